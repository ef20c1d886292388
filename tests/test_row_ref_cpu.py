"""The arithmetic that moves a softmax reference (csrc/row_ref.h), compiled for the host: after one move no score of a
tile asks for another, so the kernel may stop looking."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from row_ref_cases import f32, fma, limit_of, next_to_the_limit, qscale_of, two_roundings

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "hierarchical_sparse_attention_block_b200", "csrc")

SHIM = """
#include "row_ref.h"
extern "C" {
float limit_of(float q) { return hisa::rise_limit(q); }
float scale_of(float ref, float q) { return hisa::row_scale(ref, q); }
float exponent_of(float s, float ref, float q) { return hisa::exponent(s, {ref, 0.f}, q); }
// Moves (ref, limit) through a tile as the kernel does; returns how many scores still exceed the reference then.
int tile(const float* s, int n, float q, float* ref, float* limit, int* moved) {
  float top = s[0];
  bool any = false;
  for (int i = 0; i < n; ++i) {
    any = any || hisa::exceeds(s[i], {*ref, *limit});
    top = s[i] > top ? s[i] : top;
  }
  *moved = any;
  if (any != hisa::exceeds(top, {*ref, *limit})) return -1;  // the tile's largest decides as its scores do
  if (any) *ref = top, *limit = hisa::rise_limit(q);
  int left = 0;
  for (int i = 0; i < n; ++i) left += hisa::exceeds(s[i], {*ref, *limit});
  return left;
}
}
"""


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    d = tmp_path_factory.mktemp("row_ref")
    src, so = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", "-fPIC", "-shared", "-I", CSRC, str(src), "-o",
                    str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    lib.limit_of.restype = lib.scale_of.restype = lib.exponent_of.restype = ctypes.c_float
    lib.limit_of.argtypes = [ctypes.c_float]
    lib.scale_of.argtypes = [ctypes.c_float] * 2
    lib.exponent_of.argtypes = [ctypes.c_float] * 3
    return lib


def through(shim, scores, q, ref, limit):
    s = np.ascontiguousarray(scores, dtype=np.float32)
    r, lim, moved = ctypes.c_float(ref), ctypes.c_float(limit), ctypes.c_int(0)
    left = shim.tile(s.ctypes.data_as(ctypes.POINTER(ctypes.c_float)), len(s), ctypes.c_float(q), ctypes.byref(r),
                     ctypes.byref(lim), ctypes.byref(moved))
    return left, f32(r.value), f32(lim.value), bool(moved.value)


@pytest.mark.parametrize("d", [64, 128])
def test_one_move_is_enough(shim, d):
    q = qscale_of(d)
    rng = np.random.default_rng(d)
    for size in (1.0, 1e2, 1e3, 1e6, 2.0**28, 1e10, 1e12, 1e20, 1e30, 3e38):
        for _ in range(300):
            scores = (rng.standard_normal(8) * size).clip(-3.4e38, 3.4e38).astype(np.float32)
            first = scores[0]
            for ref, limit in ((first, limit_of(q)), (f32(0), f32(-np.inf))):
                left, ref2, limit2, moved = through(shim, scores, q, ref, limit)
                assert left == 0, (size, scores)
                again = through(shim, scores, q, ref2, limit2)
                assert again[0] == 0 and not again[3]
                assert all(shim.exponent_of(s, ref2, q) <= 8 * (1 + 2.0**-20) for s in scores)


def test_scores_next_to_the_limit(shim):
    """Pairs for which a rule that rounds the tested value and the moved one differently neither moves nor rests."""
    n = 0
    for d in (64, 128):
        q = qscale_of(d)
        for first, s in next_to_the_limit(q, 40, seed=d):
            old = f32(first * q)
            assert fma(s, q, -old) > 8 and not two_roundings(s, q) - old > 8
            assert through(shim, [first, s], q, first, limit_of(q))[0] == 0
            n += 1
    assert n == 80


def test_large_scores_keep_their_weights(shim):
    """The reference's own weight is 1 and a score half as large has none, whatever the scores' size."""
    q = qscale_of(128)
    rng = np.random.default_rng(1)
    for size in (2.0**28, 2.0**31, 1e12, 1e30):
        for _ in range(100):
            top = f32((1 + rng.random()) * size)
            assert shim.exponent_of(top, top, q) == 0 and shim.exponent_of(f32(top / 2), top, q) < -1e6


@pytest.mark.parametrize("q", [1e-45, 1e-38, 2.3e-38, 1e-3, 1.0, 1e30])
def test_every_scale_has_a_finite_limit(shim, q):
    x = shim.limit_of(q)
    assert 0 < x < np.inf
    for top in (0.0, 5.0, -3e38, 3e38):  # the first score moves the reference at any scale
        left, ref, _, moved = through(shim, [top], q, f32(0), f32(-np.inf))
        assert left == 0 and moved and ref == f32(top)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_by", [1.0, 1e-6, 1e6])
def test_one_multiply_add_keeps_every_weight_in_range(shim, d, q_by):
    """s c - ref c in one rounding: the largest score's exponent stays within 2^5, and beyond 2^30 it is 0 and the next
    smaller score's below -24, so that nothing else counts in fp32."""
    q = f32(qscale_of(d) * f32(q_by))
    rng = np.random.default_rng(d)
    for size in (1.0, 1e6, 2.0**28, 2.0**29.9, 2.0**30.1, 2.0**31, 1e12, 1e25, 1e31):
        for _ in range(200):
            top = f32((1 + rng.random()) * size / np.float64(q) * rng.choice([-1, 1]))
            c = f32(shim.scale_of(top, q))
            nm = f32(-top * c)
            e = fma(top, c, nm)
            assert abs(e) <= 32
            if abs(np.float64(top) * np.float64(q)) >= 2.0**30 * (1 + 2.0**-23):
                assert e == 0 and c <= q < 2 * c
                assert fma(np.nextafter(top, f32(-np.inf)), c, nm) <= -24
