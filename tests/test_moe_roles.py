"""The roles of the tcgen05 kernel of the routed experts, as far as a CPU can tell.

The stage bookkeeping that every role walks by itself is compiled for the host
and compared with its definition.  What a role does when a wait runs out cannot
be provoked from outside and is read in the source.
"""
import ctypes
import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "binary_packed_weight_gb300", "csrc")

SHIM = r"""
#include "moe_stages.cuh"
template <bool WIDE>
static void walk(const int* cnt, int n, int each, int* again, int* at) {
    tq2::MuStages<WIDE> f;
    for (int i = 0; i < n; ++i) {
        again[i] = f.begin(cnt[i]);
        for (int j = 0; j < each; ++j, f.next()) {
            int* p = at + 4 * (i * each + j);
            p[0] = f.s, p[1] = (int)f.parity(), p[2] = f.slots(), p[3] = (int)f.slot_bytes();
        }
    }
}
extern "C" void wide(const int* c, int n, int each, int* again, int* at) { walk<true>(c, n, each, again, at); }
extern "C" void narrow(const int* c, int n, int each, int* again, int* at) { walk<false>(c, n, each, again, at); }
"""


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    d = tmp_path_factory.mktemp("stages")
    (d / "shim.cpp").write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-D__host__=", "-D__device__=", "-D__forceinline__=inline",
                    "-I", CSRC, str(d / "shim.cpp"), "-o", str(d / "shim.so")], check=True)
    return ctypes.CDLL(str(d / "shim.so"))


def walk(fn, counts, each):
    n = len(counts)
    again, at = (ctypes.c_int * n)(), (ctypes.c_int * (4 * n * each))()
    fn((ctypes.c_int * n)(*counts), n, each, again, at)
    return list(again), [tuple(at[4 * i:4 * i + 4]) for i in range(n * each)]


@pytest.mark.parametrize("each", [4, 5, 9])
def test_wide_tiles_give_up_stages_and_take_them_up_again(shim, each):
    counts = [1, 256, 257, 320, 321, 384, 320, 300, 256, 384, 31, 384, 257, 64]
    again, at = walk(shim.wide, counts, each)
    given = [2 if c > 320 else 1 if c > 256 else 0 for c in counts]
    assert again == [was - now for was, now in zip([0] + given, given)]
    uses, stage, i = [0] * 4, 0, 0
    for low in given:
        stage = max(stage, low)
        for _ in range(each):
            assert at[i] == (stage, uses[stage] & 1, 5 - low, 32768 + 8192 * low)
            assert at[i][2] * at[i][3] <= 5 * 32768                          # the slots of every cut fit the ring
            uses[stage] += 1
            stage = low if stage == 3 else stage + 1
            i += 1


def test_narrow_tiles_keep_their_stages(shim):
    again, at = walk(shim.narrow, [1, 128, 64, 128], 4)
    assert again == [0] * 4
    assert at == [(i % 3, i // 3 & 1, 4, 32768) for i in range(16)]


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_no_expression_holds_a_new_tile_and_what_it_changes():
    """C++ leaves the order of the two sides of a comparison open: one that calls begin() and reads `lowest`
    may see the old value or the new one."""
    for name in sorted(os.listdir(CSRC)):
        for statement in re.split(r"[;{}]", source(name)):
            assert not ("begin(" in statement and "lowest" in statement), (name, statement)


def test_epilogue_warps_meet_at_their_barrier_whatever_happens():
    """The epilogue warps share a named barrier.  Of one wait that runs out some of them may see the end and others
    not, so none may leave the loop early: the others would wait for it for good."""
    text = source("moe_umma.cu")
    start = text.index("warp >= MU_EPI) {")
    role = text[start:text.index("tmem_dealloc(tmem", start)]
    assert role.count("epi_bar<DRAIN>();") == 2
    assert not re.search(r"\b(break|return|goto)\b", role)


def test_mmas_end_before_their_tensor_memory_is_given_back():
    """A role that gives up leads every warp to the end of the kernel: the issuer waits for what it issued, on every
    way out of its loop."""
    text = source("moe_umma.cu")
    start = text.index("} else if (warp == 1) {")
    role = text[start:text.index("} else if (warp >= 4", start)]
    assert not re.search(r"\b(return|goto)\b", role)
    tail = role[role.rindex("umma_commit(&bars->acc_full);"):]
    assert re.search(r"}\s*umma_commit\(&bars->idle\);\s*mbar_wait\(&bars->idle, 0u\);\s*}\s*__syncwarp\(\);\s*$", tail)
    assert text.count("mbar_init(&bars->idle, 1);") == 1
