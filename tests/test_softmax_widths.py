"""The q/k norms' launches at every number of turned channels of the widest heads, without
a GPU (as in test_softmax_launches.py): each call launches a kernel, and one whose lanes
have all of a head's work items between them."""
import json
import os
import re
import subprocess
import sys

import pytest

import gated_deltanet_dual_amd as g
from test_layer_launches import ROOT, kernel, symbols
from test_softmax_launches import CHILD

SWEEP = CHILD.split("out = []")[0] + """
out = []
for op, d, io, inter in json.loads(sys.argv[3]):
    for half in range(d // 2 + 1):
        stub.stub_reset()
        status = globals()[op](10, qh=2, kh=1, d=d, half=half, io=io, inter=inter)
        out.append([status, [stub.stub_function(i) for i in range(stub.stub_launches())]])
print(json.dumps([ctypes.cast(L.flare_version, ctypes.c_void_p).value, out]))
"""


def items(d, half, inter, vec):
    """Pairs of vectors of a head: those that turn, a vector of each half or, interleaved, two
    neighbours, then the other channels' two by two; a part's last one can be half."""
    up = lambda a, b: -(-a // b)  # noqa: E731
    turned = up(up(2 * half, vec), 2) if inter else up(half, vec)
    return turned + up(up(d - 2 * half, vec), 2)


@pytest.mark.parametrize("d", [1024, 1020, 1016, 1011, 528])
def test_every_turned_part_of_wide_heads(tmp_path, d):
    if not os.path.exists(g.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    stub = str(tmp_path / "launches.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-o", stub, os.path.join(ROOT, "tests", "hip_stub", "launches.c")], check=True)
    ops = ["forward", "reverse", "cache"] + (["cache4"] if d % 32 == 0 else [])
    todo = [(op, d, io, inter) for op in ops for io in (g.BF16, g.F32) for inter in (0, 1)]
    r = subprocess.run([sys.executable, "-c", SWEEP, stub, ROOT, json.dumps(todo)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    at, out = json.loads(r.stdout)
    names = dict(symbols())
    base = at - next(a for a, name in symbols() if name == "flare_version")
    bad = []
    for (status, launched), (op, io, inter, half) in zip(out, [(op, io, inter, half) for op, _, io, inter in todo for half in range(d // 2 + 1)]):
        forms = [kernel(names[f - base]) for f in launched]
        where = (op, "bf16" if io == g.BF16 else "fp32", "interleaved" if inter else "halves", half, status, forms)
        if status != 0 or len(forms) != (2 if op == "reverse" else 1):
            bad.append(where)
            continue
        # <type, channels of a vector, short vectors, items a lane[, where the rows go]>
        vec, lane_items = (int(n) for n in re.match(r"qk_norm_rotary_(?:bwd_)?kernel<[^,]+, (\d+), \w+, (\d+)", forms[0]).groups())
        # by vectors of 8 a lane has one item whatever the form; into 4 bits keys go by vectors of 4
        if items(d, half, inter, vec) > 64 * (1 if vec == 8 else lane_items):
            bad.append(where)
        elif op == "cache4" and items(d, half, inter, 4) > 64 * lane_items:
            bad.append(where)
    assert not bad, "%d of %d, the first %s" % (len(bad), len(out), bad[:3])
