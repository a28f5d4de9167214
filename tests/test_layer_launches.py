"""What the operators around the GDN step launch, without a GPU: a child process
loads a stub of HIP's launch functions before the library (device pointers are
dummies, nothing runs).  A launch dimension holds fewer than 2^32 work items:
calls that need more are refused by the host's checks, before anything is enqueued."""
import json
import os
import re
import subprocess
import sys

import pytest

import gated_deltanet_dual_amd as g

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CHILD = """
import ctypes, json, sys
stub = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
stub.stub_items.restype = ctypes.c_uint64
stub.stub_function.restype = ctypes.c_size_t
sys.path.insert(0, sys.argv[2])
import gated_deltanet_dual_amd as g
from gated_deltanet_dual_amd import layer
L = ctypes.CDLL(g.LIB_PATH)
layer.declare(L)
FAKE = 0x7F0000001000
WS = FAKE & ~255

def attention(R, block=1, qh=8, kh=8, d=64, page=1024, most=2 ** 20, n=0):
    s = g.AttentionShape(block, qh, kh, d, page, g.BF16, 0, 0.0)
    return L.flare_block_attention(R, ctypes.byref(s), FAKE, FAKE, FAKE, 100, FAKE, -(-most // page), FAKE, most, FAKE, n,
                                   FAKE, None, WS, 2 ** 62, None)

def rotary(tokens, qh=16, kh=4, d=128, half=64, io=g.BF16, inter=0):
    s = g.RotaryShape(qh, kh, d, half, io, inter, 1.0)
    return L.flare_rotary(tokens, ctypes.byref(s), FAKE, FAKE, FAKE, qh * d, FAKE, kh * d, 0, FAKE, FAKE, None)

def rotary_cache(tokens, qh=64, kh=8, d=128, half=64, io=g.BF16):
    s = g.RotaryShape(qh, kh, d, half, io, 0, 1.0)
    return L.flare_rotary_cache(tokens, ctypes.byref(s), FAKE, FAKE, FAKE, qh * d, FAKE, kh * d, FAKE, kh * d, FAKE, FAKE,
                                FAKE, FAKE, 100, 64, None)

def gated(tokens, heads=4, d=128, io=g.BF16):
    return L.flare_gated_norm(tokens, heads, d, io, FAKE, heads * d, FAKE, heads * d, FAKE, 1, 1e-6, FAKE, FAKE, None)

def residual(tokens, d=2048, io=g.BF16, res=g.F32):
    return L.flare_residual_norm(tokens, d, io, res, FAKE, d, FAKE, FAKE, d, FAKE, FAKE, FAKE, 1, 1e-6, FAKE, FAKE, FAKE, None)

def tables(R=5, tokens=40):
    return L.flare_step_tables(R, FAKE, FAKE + 64, FAKE, 4, FAKE, 10, FAKE, 16, 0, tokens, FAKE, FAKE, FAKE, FAKE + 128,
                               FAKE + 192, FAKE, None)

def gated_bwd(tokens, heads=4, d=128, io=g.BF16):
    return L.flare_gated_norm_bwd(tokens, heads, d, io, FAKE, heads * d, FAKE, heads * d, FAKE, 1, FAKE, FAKE, heads * d,
                                  FAKE, FAKE, FAKE, WS, 2 ** 40, None)

def residual_bwd(tokens, d=2048, io=g.BF16, res=g.F32):
    return L.flare_residual_norm_bwd(tokens, d, io, res, FAKE, d, FAKE, FAKE, d, FAKE, FAKE, FAKE, 1, FAKE, FAKE, FAKE,
                                     FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, WS, 2 ** 40, None)

out = []
for call in json.loads(sys.argv[3]):
    stub.stub_reset()
    stub.stub_fail_at(call.get("fail_at", -1))
    status = globals()[call["op"]](**call["args"])
    n = range(stub.stub_launches())
    out.append([status, [stub.stub_items(i) for i in n], [stub.stub_function(i) for i in n]])
print(json.dumps([ctypes.cast(L.flare_version, ctypes.c_void_p).value, out]))
"""


@pytest.fixture(scope="module")
def calls(tmp_path_factory):
    if not os.path.exists(g.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    lib = str(tmp_path_factory.mktemp("stub") / "launches.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-o", lib, os.path.join(ROOT, "tests", "hip_stub", "launches.c")],
                   check=True)

    def run(*todo, kernels=False):
        """[status, work items of each launch] of the calls; kernels: and the names."""
        r = subprocess.run([sys.executable, "-c", CHILD, lib, ROOT, json.dumps(todo)], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        at, out = json.loads(r.stdout)
        if not kernels:
            return [o[:2] for o in out]
        base = at - next(a for a, name in symbols() if name == "flare_version")
        names = dict(symbols())
        return [[s, [kernel(names[f - base]) for f in fs]] for s, _, fs in out]
    return run


def symbols():
    """(address, demangled name) of the library's own symbols."""
    rows = subprocess.run(["nm", "-C", g.LIB_PATH], check=True, capture_output=True, text=True).stdout.splitlines()
    return [(int(r[:16], 16), r[19:]) for r in rows if r[:16].strip()]


def kernel(name):
    """`attn_kernel<64, ...>` of its symbol or its launching function's, or None."""
    m = re.search(r"(\w+_kernel(?:<.*?>)?)(?:\(|$)", name.replace("__device_stub__", ""))
    return m and m.group(1)


def call(op, fail_at=-1, **args):
    return {"op": op, "fail_at": fail_at, "args": args}


def test_the_stub_sees_the_launches(calls):
    for status, items in calls(call("attention", R=2), call("gated_bwd", tokens=4000), call("residual_bwd", tokens=4000)):
        assert status == 0 and len(items) == 2 and all(0 < n < 2 ** 32 for n in items)
    (status, items), = calls(call("rotary", tokens=1000))
    assert status == 0 and len(items) == 1


def test_attention_of_more_workgroups_than_a_launch_holds(calls):
    # 8192 requests x 8 heads x 256 parts of 4096 keys are 2^24 workgroups of 256 threads
    most, fewer = calls(call("attention", R=8192), call("attention", R=8160))
    assert most == [4, []]
    assert fewer[0] == 0 and len(fewer[1]) == 2 and 2 ** 31 < fewer[1][0] < 2 ** 32
    # the prefix's workgroups count likewise, and both together
    for R, more in ((2 ** 22, dict(n=2 ** 21, most=1024)), (4096, dict(n=2 ** 21, block=64, qh=64, kh=8, most=2 ** 20))):
        status, items = calls(call("attention", R=R, **more))[0]
        assert (status == 4 and items == []) or (status == 0 and all(n < 2 ** 32 for n in items))


def test_nothing_is_enqueued_after_a_launch_that_failed(calls):
    """The join and the weights' sums read what the first launch writes."""
    todo = [call("attention", fail_at=0, R=2), call("gated_bwd", fail_at=0, tokens=4000),
            call("residual_bwd", fail_at=0, tokens=4000)]
    for status, items in calls(*todo):
        assert status == 6 and len(items) == 1


def test_rotary_of_more_workgroups_than_a_launch_holds(calls):
    wide, small = dict(qh=64, kh=8), dict(qh=1, kh=1, d=64, half=32)  # one token a workgroup, and sixteen
    for op in ("rotary", "rotary_cache"):
        got = calls(call(op, tokens=2 ** 24, **wide), call(op, tokens=2 ** 24 - 1, **wide), call(op, tokens=2 ** 31 - 1, **wide),
                    call(op, tokens=2 ** 28, **small), call(op, tokens=2 ** 28 - 16, **small))
        assert [s for s, _ in got] == [4, 0, 4, 4, 0]
        assert [len(items) for _, items in got] == [0, 1, 0, 0, 1] and all(n < 2 ** 32 for _, items in got for n in items)


def test_the_other_operators_stay_below_it(calls):
    """Norms pass their rows in rounds: the largest sizes launch."""
    for status, items in calls(call("gated_bwd", tokens=2 ** 31 - 1, heads=1, d=1), call("gated_bwd", tokens=2 ** 27, heads=15, d=128),
                               call("residual_bwd", tokens=2 ** 31 - 1, d=16384)):
        assert status == 0 and len(items) == 2 and all(n < 2 ** 32 for n in items)


KERNELS = ("attn_kernel", "attn_join_kernel", "gated_norm_kernel", "gated_norm_bwd_kernel", "residual_norm_kernel",
           "residual_norm_bwd_kernel", "norm_partials_kernel", "rotary_kernel", "step_tables_kernel")


def test_every_form_of_a_kernel_is_reached(calls):
    """What was built is what some call launches: rows of every width's class, even and
    odd, every type, few and many rows and heads."""
    widths = sorted({w for c in (1, 8, 16, 64, 128, 256, 512, 1024, 2048, 4096, 8192, 16384) for w in (c, c - 1, 3 * c // 2, 3 * c // 4)
                     if 1 <= w <= 16384})
    types = [(g.BF16, g.BF16), (g.BF16, g.F32), (g.F32, g.F32)]
    todo = [call("tables")]
    for d in widths:
        todo += [call(op, tokens=n, heads=1, d=d, io=io) for op in ("gated", "gated_bwd") for io in (g.BF16, g.F32) for n in (1, 5000)]
        todo += [call(op, tokens=n, d=d, io=io, res=r) for op in ("residual", "residual_bwd") for io, r in types for n in (1, 5000)]
    todo += [call("rotary", tokens=9, d=d, half=h, io=io, inter=i) for d in (64, 66) for h in (0, 16, 32, 7) for io in (g.BF16, g.F32)
             for i in (0, 1)]
    todo += [call("attention", R=R, block=b, qh=q, kh=2, d=d, most=own, n=n) for R in (1, 40, 300) for b in (1, 5, 20)
             for q in (2, 16) for d in (64, 128, 256) for own in (40, 1024, 20000) for n in (0, 100, 9000)]
    got = calls(*todo, kernels=True)
    assert all(status == 0 for status, _ in got)
    launched = {k for _, names in got for k in names}
    built = {k for k in map(kernel, (name for _, name in symbols())) if k and k.split("<")[0] in KERNELS}
    assert len(built) > 80 and {k.split("<")[0] for k in built} == set(KERNELS)
    assert built == launched, "never launched: %s" % sorted(built - launched)
