"""Which sequences of a packed call run (csrc/ssm_sequences.h, the kernels' own header, compiled for the host): any
cu_seqlens, also one that goes back, leaves disjoint sequences within the tokens, in no more segments than the
workspace is sized for."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SHIM = """
#include "ssm_sequences.h"
// writes each sequence's segments (0: it does not run), returns the bound; the walk of the kernels and the join
extern "C" int64_t walk(const int* cu, int seqs, int64_t tokens, uint32_t seg, uint32_t* segments) {
  bool back = false;
  for (int s = 0; s < seqs; ++s) {
    back = back || ssm::goes_back(cu[s], cu[s + 1]);
    segments[s] = !back && ssm::within(cu[s], cu[s + 1], tokens) ? ssm::segments_of(cu[s + 1] - cu[s], seg) : 0;
  }
  return ssm::segments_at_most(tokens, seg, seqs);
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    cxx = os.environ.get("CXX") or shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    at = tmp_path_factory.mktemp("sequences")
    (at / "shim.cpp").write_text(SHIM)
    subprocess.run([cxx, "-std=c++17", "-shared", "-fPIC", "-I", os.path.join(ROOT, "mamba_replayssm_state_gb300", "csrc"),
                    str(at / "shim.cpp"), "-o", str(at / "shim.so")], check=True)
    fn = ctypes.CDLL(str(at / "shim.so")).walk
    fn.restype = ctypes.c_int64

    def call(cu, tokens, seg):
        n = len(cu) - 1
        segments = (ctypes.c_uint32 * max(n, 1))()
        bound = fn((ctypes.c_int32 * (n + 1))(*cu), n, ctypes.c_int64(tokens), ctypes.c_uint32(seg), segments)
        return list(segments)[:n], bound

    return call


@pytest.mark.parametrize("cu,tokens,runs", [
    ([0, 5, 5, 9], 9, [1, 1, 1]), ([2, 5, 9], 12, [1, 1]),
    ([0, 20, 10, 30], 30, [1, 0, 0]),  # back, and then over the first
    ([0, 9, 0, 9, 0, 9], 9, [1, 0, 0, 0, 0]), ([0, 4, 99, 3, 9], 9, [1, 0, 0, 0]), ([-1, 4, 9], 9, [0, 1]),
    ([0, 4, 10], 9, [1, 0]), ([7, 3, 9], 9, [0, 0]), ([0, 0, 0], 0, [1, 1]), ([-9, -5, 0, 9], 9, [0, 0, 1]),
    ([2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1], 9, [0, 0])])
def test_which_sequences_run(walk, cu, tokens, runs):
    assert walk(cu, tokens, 1 << 30)[0] == runs


def test_a_call_that_starts_over_stays_within_its_segments(walk):
    segments, bound = walk([0, 32768, 0, 32768], 32768, 2816)
    assert segments == [12, 0, 0] and sum(segments) <= bound


def test_any_sequences_are_disjoint_and_within_their_segments(walk):
    rng = random.Random(1)
    for _ in range(3000):
        tokens, n = rng.choice([0, 1, 7, 300, 5000]), rng.randrange(1, 12)
        cu = [rng.randrange(-3, tokens + 4) for _ in range(n + 1)]
        kind = rng.randrange(3)
        if kind == 0:
            cu.sort()
        elif kind == 1:
            cu = [rng.choice([0, tokens, tokens // 2]) for _ in range(n + 1)]
        seg = 128 * rng.randrange(1, 9)
        segments, bound = walk(cu, tokens, seg)
        assert sum(segments) <= bound
        owner = {}
        for s, k in enumerate(segments):
            if k:
                assert 0 <= cu[s] <= cu[s + 1] <= tokens and k == max(1, -(-(cu[s + 1] - cu[s]) // seg))
                for t in range(cu[s], cu[s + 1]):
                    assert owner.setdefault(t, s) == s
        if cu == sorted(cu) and cu[0] >= 0 and cu[-1] <= tokens:
            assert all(segments)
