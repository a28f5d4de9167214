"""The GPU code that was built for the operators around the GDN step, looked at without
a GPU: what the compiler cannot know about instructions written out in the source, and
which forms of a kernel there are."""
import os
import re
import shutil
import subprocess

import pytest

import gated_deltanet_dual_amd as g
from gated_deltanet_dual_amd import build

LLVM = os.path.join(build.ROCM, "llvm", "bin")


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    """name -> disassembly of the code object that has a kernel of this name."""
    if not os.path.exists(g.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    at = tmp_path_factory.mktemp("code")
    shutil.copy(g.LIB_PATH, at)
    dump = os.path.join(LLVM, "llvm-objdump")
    subprocess.run([dump, "--offloading", os.path.basename(g.LIB_PATH)], cwd=at, check=True, capture_output=True)
    parts = {}
    for f in sorted(os.listdir(at)):
        if "gfx950" in f:
            parts[f] = subprocess.run(["nm", f], cwd=at, check=True, capture_output=True, text=True).stdout

    def find(kernel):
        f, = [f for f, names in parts.items() if kernel in names]
        return subprocess.run([dump, "-d", "--no-show-raw-insn", f], cwd=at, check=True, capture_output=True, text=True).stdout
    return find


def test_m0_is_left_as_it_was(code):
    """The block attention's loads into LDS take their place from M0, written by the same
    statement: every write is theirs and the register is restored, so that whatever the
    compiler keeps there stands."""
    text = code("attn_kernel")
    ops = [m.group(1).strip() for m in re.finditer(r"^\t(.*?)\s*//", text, re.M)]
    assert len(ops) > 10000
    loads = re.compile(r"global_load_lds_dwordx4 v\d+, s\[\d+:\d+\]( nt)?$")
    groups, i = 0, 0
    while i < len(ops):
        save = re.match(r"s_mov_b32 (s\d+), m0$", ops[i])
        if not save:
            assert not re.search(r"\bm0\b", ops[i]) and "_lds_" not in ops[i], (i, ops[max(0, i - 3):i + 4])
            i += 1
            continue
        body = ops[i + 1:i + 14]
        for k in range(4):
            assert re.match(r"s_mov_b32 m0, s\d+$", body[3 * k]) and body[3 * k + 1] == "s_nop 0" and loads.match(body[3 * k + 2]), body
        assert body[12] == "s_mov_b32 m0, " + save.group(1), body
        groups, i = groups + 1, i + 14
    assert groups > 0
