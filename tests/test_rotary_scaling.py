"""The yarn stretch at lengths where its ramp lies partly or wholly outside the pairs."""
import math

import pytest
import torch

import gated_deltanet_dual_amd as g


@pytest.mark.parametrize("n", [2, 8, 64, 128])
@pytest.mark.parametrize("length", [1, 4, 6, 7, 20, 200, 4096, 10 ** 7])
def test_slow_pairs_are_divided_and_fast_ones_kept(n, length):
    """Every pair that turns fewer than beta_slow times within the original length is
    divided by the factor, also where all of them do; every one that turns more than
    beta_fast times is kept."""
    base = g.rotary_frequencies(n, device="cpu")[0]
    y, m = g.rotary_frequencies(n, scaling="yarn", factor=4.0, original_length=length, device="cpu")
    turns = length * base / (2 * math.pi)
    assert torch.equal(y[turns < 1], base[turns < 1] / 4) and torch.equal(y[turns > 32], base[turns > 32])
    assert (y <= base).all() and (y >= base / 4).all() and m == 1 + 0.1 * math.log(4.0)


def test_ramps_without_two_ends_are_refused():
    for bad in (dict(beta_slow=0.0), dict(beta_slow=-1.0), dict(beta_fast=0.5), dict(beta_fast=math.nan)):
        with pytest.raises(g.FlareError, match="beta"):
            g.rotary_frequencies(64, scaling="yarn", factor=4.0, original_length=4096, device="cpu", **bad)
