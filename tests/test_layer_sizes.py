"""Sizes that the library's 32-bit arguments do not hold are refused by the binding,
which would otherwise pass them on cut to their lower bits."""
import pytest
import torch

import gated_deltanet_dual_amd as g
from gated_deltanet_dual_amd import layer

CPU = torch.device("cpu")


def test_cache_pages_and_heads():
    """A cache with pages of 2^32 + 16 rows is not one with pages of 16 (looked at
    without its memory: no pages)."""
    for shape in ((0, 1, 2 ** 32 + 16, 8), (0, 2 ** 32 + 2, 16, 8)):
        c = torch.empty(shape, dtype=torch.bfloat16)
        with pytest.raises(g.FlareError, match="beyond 32 bits"):
            layer._chk_cache(c, c, shape[1], 8, torch.bfloat16, CPU)
    c = torch.empty(0, 2, 16, 8, dtype=torch.bfloat16)
    assert layer._chk_cache(c, c, 2, 8, torch.bfloat16, CPU) == (0, 16)


def test_workspace_sizes():
    """A size query of cut arguments would answer for another call."""
    for call in (lambda n: g.gated_norm_bwd_workspace_bytes(4, n, 64), lambda n: g.gated_norm_bwd_workspace_bytes(4, 2, n),
                 lambda n: g.residual_norm_bwd_workspace_bytes(4, n),
                 lambda n: g.block_attention_workspace_bytes(n, 4, 8, 2, 128, 64, 512, 100),
                 lambda n: g.block_attention_workspace_bytes(2, n, 8, 2, 128, 64, 512, 100),
                 lambda n: g.block_attention_workspace_bytes(2, 4, 8, 2, 128, n, 512, 100),
                 lambda n: g.block_attention_workspace_bytes(2, 4, 8, 2, 128, 64, n, 100),
                 lambda n: g.block_attention_workspace_bytes(2, 4, 8, 2, 128, 64, 512, n)):
        with pytest.raises(g.FlareError, match="beyond 32 bits"):
            call(2 ** 32 + 64)
