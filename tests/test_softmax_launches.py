"""What the softmax layers' further operators launch, without a GPU: a child process
loads a stub of HIP's launch functions before the library (device pointers are dummies,
nothing runs).  Every form that is built is launched by some call, nothing is enqueued
behind a launch that failed, and a launch dimension stays below 2^32 work items."""
import json
import os
import subprocess
import sys

import pytest

import gated_deltanet_dual_amd as g
from test_layer_launches import ROOT, call, kernel, symbols

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

def forward(tokens, qh=16, kh=4, d=128, half=64, io=g.BF16, inter=0):
    s = g.RotaryShape(qh, kh, d, half, io, inter, 1.0)
    return L.flare_qk_norm_rotary(tokens, ctypes.byref(s), FAKE, FAKE, FAKE, qh * d, FAKE, kh * d, FAKE,
                                  FAKE if kh else None, 1e-6, FAKE, FAKE, None)

def reverse(tokens, qh=16, kh=4, d=128, half=64, io=g.BF16, inter=0, weights=True):
    s = g.RotaryShape(qh, kh, d, half, io, inter, 1.0)
    w = FAKE if weights else None
    return L.flare_qk_norm_rotary_bwd(tokens, ctypes.byref(s), FAKE, FAKE, FAKE, qh * d, FAKE, kh * d, w, w, 1e-6, FAKE,
                                      qh * d, FAKE, kh * d, FAKE, FAKE, w, w, WS, 2 ** 40, None)

def cache(tokens, qh=16, kh=4, d=128, half=64, io=g.BF16, inter=0):
    s = g.RotaryShape(qh, kh, d, half, io, inter, 1.0)
    return L.flare_qk_norm_rotary_cache(tokens, ctypes.byref(s), FAKE, FAKE, FAKE, qh * d, FAKE, kh * d, FAKE, kh * d,
                                        FAKE, FAKE, 1e-6, FAKE, FAKE, FAKE, FAKE, 100, 64, None)

def cache4(tokens, qh=16, kh=4, d=128, half=64, io=g.BF16, inter=0):
    s = g.RotaryShape(qh, kh, d, half, io, inter, 1.0)
    return L.flare_qk_norm_rotary_cache_fp4(tokens, ctypes.byref(s), FAKE, FAKE, FAKE, qh * d, FAKE, kh * d, FAKE, kh * d,
                                            FAKE, FAKE, 1e-6, FAKE, FAKE, WS, FAKE, WS, FAKE, 100, 64, None)

def rows(tokens, heads=4, d=128, io=g.BF16, values=True):
    v = WS if values else None
    return L.flare_cache_fp4_rows(tokens, heads, d, io, FAKE, WS, FAKE, v, v, 100, 64, FAKE, v, None)

def attention(R, block=1, qh=8, kh=8, d=64, page=64, most=1024, n=0):
    s = g.AttentionShape(block, qh, kh, d, page, g.BF16, 0, 0.0)
    return L.flare_block_attention_fp4(R, ctypes.byref(s), WS, WS, FAKE, WS, FAKE, 100, FAKE, -(-most // page), FAKE, most,
                                       FAKE, n, WS, None, WS, 2 ** 62, None)

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

    def run(*todo):
        """[status, work items of each launch, kernels] of the calls."""
        r = subprocess.run([sys.executable, "-c", CHILD, lib, ROOT, json.dumps(todo)], capture_output=True, text=True)
        assert r.returncode == 0, r.stderr[-2000:]
        at, out = json.loads(r.stdout)
        base = at - next(a for a, name in symbols() if name == "flare_version")
        names = dict(symbols())
        return [[s, items, [kernel(names[f - base]) for f in fs]] for s, items, fs in out]
    return run


def test_every_form_is_launched(calls):
    todo = []
    for op in ("forward", "reverse", "cache"):
        for io in (g.BF16, g.F32):
            # whole vectors of 8, of 4, short ones; heads that 64 lanes do not have at a time
            for d, half in ((128, 64), (132, 64), (80, 25), (1024, 512), (1020, 300), (1021, 7)):
                todo.append(call(op, tokens=100, d=d, half=half, io=io))
    for io in (g.BF16, g.F32):
        for d, half in ((128, 64), (128, 60), (128, 25), (1024, 512), (1024, 508), (1024, 25)):
            todo.append(call("cache4", tokens=100, d=d, half=half, io=io))
        todo.append(call("rows", tokens=100, io=io))
    for d in (64, 128, 256):
        for R in (1, 5, 300, 2000):
            for block in (1, 3, 4, 8, 16, 40):
                for group in (1, 8):
                    for n in (0, 200, 20000):
                        todo.append(call("attention", R=R, block=block, d=d, qh=2 * group, kh=2, n=n, most=700))
                        todo.append(call("attention", R=R, block=block, d=d, qh=2 * group, kh=2, n=n, most=0))
    got = calls(*todo)
    assert all(s == 0 and all(0 < n < 2 ** 32 for n in items) for s, items, _ in got)
    launched = {k for _, _, ks in got for k in ks}
    built = {kernel(name) for _, name in symbols()}
    ours = {k for k in built if k and k.split("<")[0] in ("qk_norm_rotary_kernel", "qk_norm_rotary_bwd_kernel",
                                                          "cache_fp4_rows_kernel", "attend_fp4_kernel")}
    assert len(ours) > 30 and ours <= launched, sorted(ours - launched)


def test_nothing_is_enqueued_after_a_launch_that_failed(calls):
    todo = [call("reverse", fail_at=0, tokens=4000), call("attention", fail_at=0, R=2, most=2 ** 17),
            call("forward", fail_at=0, tokens=9), call("cache4", fail_at=0, tokens=9), call("rows", fail_at=0, tokens=9)]
    for status, items, _ in calls(*todo):
        assert status == 6 and len(items) == 1
    two, one, none = calls(call("reverse", tokens=4000), call("reverse", tokens=4000, weights=False), call("forward", tokens=0))
    assert (len(two[1]), len(one[1]), len(none[1])) == (2, 1, 0) and two[0] == one[0] == none[0] == 0
    assert len(calls(call("attention", R=2, most=2 ** 17))[0][1]) == 2


def test_more_workgroups_than_a_launch_holds(calls):
    wide, small = dict(qh=256, kh=8), dict(qh=1, kh=1, d=64, half=32)
    for op, kinds in (("forward", 1), ("cache", 1), ("cache4", 2)):
        (s0, i0, _), (s1, i1, _), (s2, i2, _) = calls(call(op, tokens=2 ** 24, **wide), call(op, tokens=2 ** 22, **wide),
                                                      call(op, tokens=2 ** 27, **small))
        assert (s0, i0) == (4, []) and s1 == s2 == 0
        assert all(0 < n < 2 ** 32 for n in i1 + i2) and i1[0] >= kinds * 2 ** 22 * 64
    # in rounds: the reverse mode and the rows; the attention as over bf16
    for s, items, _ in calls(call("reverse", tokens=2 ** 31 - 1, **wide), call("rows", tokens=2 ** 31 - 1)):
        assert s == 0 and all(0 < n < 2 ** 32 for n in items)
    (s, items, _), = calls(call("attention", R=2 ** 23, qh=1, kh=1, most=2 ** 20))
    assert s == 4 and items == []


def test_every_call_enqueues_its_launches(calls):
    """One of the norms and of the rows, two of the reverse mode with its weights' sums, and of an
    attention two where its workspace holds parts: a call that enqueues nothing is no success."""
    todo, want = [], []
    for inter in (0, 1):
        for io in (g.BF16, g.F32):
            for d, half in ((1, 0), (3, 1), (64, 32), (80, 25), (128, 12), (1016, 4), (1024, 0), (1024, 4), (1024, 300), (1024, 508), (1024, 512)):
                for op in ("forward", "reverse", "cache") + (("cache4",) if d % 32 == 0 else ()):
                    for tokens in (1, 3000):
                        todo.append(call(op, tokens=tokens, d=d, half=half, io=io, inter=inter))
                        want.append(2 if op == "reverse" else 1)
    for values in (False, True):
        todo.append(call("rows", tokens=1, values=values))
        want.append(1)
    for d in (64, 128, 256):
        for R in (1, 40, 300):
            for block, group in ((1, 1), (1, 17), (4, 8), (33, 1), (16, 16)):
                for n, most in ((0, 0), (0, 1), (50, 700), (0, 9000), (20000, 700), (20000, 0)):
                    todo.append(call("attention", R=R, block=block, d=d, qh=2 * group, kh=2, n=n, most=most))
                    want.append(2 if g.block_attention_fp4_workspace_bytes(R, block, 2 * group, 2, d, 64, most, n) else 1)
    got = [r for i in range(0, len(todo), 200) for r in calls(*todo[i:i + 200])]
    for (status, items, _), n, c in zip(got, want, todo):
        assert status == 0 and len(items) == n and all(0 < i < 2 ** 32 for i in items), (c, status, items)
