"""Scores next to the point where a row's softmax reference moves (csrc/row_ref.h), in fp32."""
import numpy as np

f32 = np.float32


def qscale_of(d):
    return f32(f32(1 / np.sqrt(np.float64(d))) * f32(1.4426950408889634))


def limit_of(q):
    return f32(f32(8) / q)


def fma(a, b, c):
    """a b + c, rounded once (a b is exact in 64 bits)."""
    return f32(np.float64(a) * np.float64(b) + np.float64(c))


def two_roundings(a, b):
    return f32(a * b)


def next_to_the_limit(q, count, seed):
    """(first, s): 8 in the log2 domain apart, where fma(s, q, -first q) > 8 but the rounded product s q is not more
    than 8 above the rounded first q."""
    rng = np.random.default_rng(seed)
    found = []
    while len(found) < count:
        first = f32(rng.standard_normal() * 10.0 ** rng.uniform(1, 3.5))
        ref = two_roundings(first, q)
        s = f32((np.float64(ref) + 8) / np.float64(q))
        for _ in range(3):
            if fma(s, q, -ref) > 8 and not two_roundings(s, q) - ref > 8:
                found.append((first, s))
                break
            s = np.nextafter(s, f32(np.inf))
    return found


def three_bf16(x):
    """fp32 values as three bf16 values that add up to them exactly (the leading 8 bits, the next 8, the last 8)."""
    x = np.asarray(x, dtype=np.float32)
    out = []
    for _ in range(3):
        part = (x.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
        out.append(part)
        x = (x - part).astype(np.float32)
    assert not x.any()
    return out
