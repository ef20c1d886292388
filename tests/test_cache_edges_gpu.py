"""The cache operators at the edges of their arithmetic and of their orderings, against the definitions in 64 bits
(tolerances: test_cache_gpu.py, unless a test derives its own)."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import cache_reference as ref  # noqa: E402
from row_ref_cases import limit_of, next_to_the_limit, qscale_of, three_bf16  # noqa: E402
from test_cache_gpu import check_compact, check_tree, close, delta, hs, make_inputs, some_arrays, to_gpu  # noqa: E402, F401


def scores_next_to_the_limit(T, H, b, n_kv, d, seed):
    """One KV head whose raw scores are chosen to the last bit: q is 1 in three places, a key holds its score as three
    bf16 numbers there.  Every tile's largest score lies 8 (log2 domain) above the one before, give or take an ulp."""
    q_scale = qscale_of(d)
    rng = np.random.default_rng(seed)
    x = make_inputs(b, T, H, 1, d, n_kv, [n_kv - T - s % 3 for s in range(b)], "chain", seed, garbage=False)
    x["q"].zero_()
    x["q"][..., :3] = 1.0
    for s, (first, up) in enumerate(next_to_the_limit(q_scale, b, seed)):
        z = (first - np.float32(3) * limit_of(q_scale) * rng.random(n_kv, dtype=np.float32)).astype(np.float32)
        top = first
        for t0 in range(0, n_kv, 128):
            z[t0] = first
            if t0 == 0:
                top = up
            else:
                top = np.float32(top + limit_of(q_scale))
                for _ in range(rng.integers(0, 3)):
                    top = np.nextafter(top, np.float32(rng.choice([-np.inf, np.inf])))
            z[t0 + 1 + rng.integers(0, min(127, n_kv - t0 - 1))] = top
        for c, part in enumerate(three_bf16(z)):
            x["k"][s, :, 0, c] = torch.from_numpy(part).to(torch.bfloat16)
    return x


@pytest.mark.parametrize("T,H", [(1, 1), (3, 2), (16, 1)])
def test_scores_next_to_the_raise_of_the_reference(hs, T, H):
    x = scores_next_to_the_limit(T, H, 150, 700, 64, seed=T)
    check_tree(hs, x, H, 1, 64, True)


def rising_keys(b, Hk, d, n_kv, seed):
    """K whose raw scores against q = (1, 1, 1, 0 ..) rise by about the limit from tile to tile, at one key a tile."""
    rng = np.random.default_rng(seed)
    lim = limit_of(qscale_of(d))
    tiles = -(-n_kv // 128)
    top = np.cumsum(lim * rng.choice([0.0, 0.7, 1.0, 1.3], (b, Hk, tiles)), 2)
    z = np.repeat(top, 128, 2)[:, :, :n_kv] - lim * rng.uniform(1, 3, (b, Hk, n_kv))
    at = np.minimum(np.arange(tiles) * 128 + rng.integers(0, 128, (b, Hk, tiles)), n_kv - 1)
    np.put_along_axis(z, at, top, 2)
    k = torch.zeros(b, n_kv, Hk, d, dtype=torch.bfloat16)
    for c, part in enumerate(three_bf16(z.transpose(0, 2, 1).astype(np.float32))):
        k[..., c] = torch.from_numpy(part).to(torch.bfloat16)
    return k


@pytest.mark.parametrize("Hk,G,T", [(16, 1, 1), (4, 2, 8)])
def test_references_that_move_from_tile_to_tile(hs, Hk, G, T):
    """Dozens of tiles a share of the work, most of which move the reference, at a key of any warp: the definition's
    result, and the same bits every time."""
    b, d, n_kv = 2, 128, 24000
    H = Hk * G
    gen = torch.Generator().manual_seed(T)
    k, v = rising_keys(b, Hk, d, n_kv, T), torch.randn(b, n_kv, Hk, d, generator=gen).to(torch.bfloat16)
    q = torch.zeros(b, T, H, d, dtype=torch.bfloat16)
    q[..., :3] = 1.0
    lens = torch.tensor([n_kv - T, 17003], dtype=torch.int32)
    ro, rl, _, spread, size = ref.tree_attention(q, k, v, lens, None, 1 / math.sqrt(d))
    p = hs.params(b, T, n_kv, 128, 128, 4, 64, H, Hk, d)
    g = [x.cuda() for x in (q, k, v, lens)]
    first = hs.tree_attn(p, *g)
    dl = delta(d, size)
    close(first[1], rl, dl + 2.0**-22 * rl.abs(), "lse")
    close(first[0], ro, 2.0**-8 * ro.abs() + 2 * dl * spread, "o")
    for _ in range(40):
        assert all(torch.equal(x, y) for x, y in zip(first, hs.tree_attn(p, *g)))


def far_scores(T, H, Hk, d, n_kv, L, size, seed):
    """Keys along one direction, at a few lengths that double: a row's largest scores are about +size, equal among
    themselves to the last bit, all others at most half as large; the rows of odd slots look the other way."""
    x = make_inputs(1, T, H, Hk, d, n_kv, [L], "tree", seed, garbage=False)
    gen = torch.Generator().manual_seed(seed + 1)
    u = torch.randn(d, generator=gen).to(torch.bfloat16).float()
    e = math.log2(size * math.sqrt(d) / float((u * u).sum()))
    a, c = int(e / 2), int(e) - int(e / 2)
    level = 2.0 ** torch.randint(-6, 0, (n_kv,), generator=gen).float()
    level = torch.where(torch.rand(n_kv, generator=gen) < 0.5, level, -level)
    tops = torch.randperm(L, generator=gen)[:24]
    level[tops[:12]], level[tops[12:]] = 1.0, -1.0
    sign = 1.0 - 2.0 * (torch.arange(T) % 2)
    x["q"] = (u * 2.0**a * sign[:, None, None]).expand(1, T, H, d).to(torch.bfloat16).contiguous()
    x["k"] = (u * 2.0**c * level[None, :, None, None]).expand(1, n_kv, Hk, d).to(torch.bfloat16).contiguous()
    return x, sign, level, float((u.double() * u.double()).sum()) * 2.0 ** (a + c) / math.sqrt(d)


def check_far(hs, size, T, H, Hk, d, n_kv, L):
    """A score is off by (d + 8) 2^-23 of itself, 2e-5 of the distance of at least half to any other score, so the
    weights are those of the largest scores alone, and these are equal: o carries the roundings of the weights (equal
    ones cancel, 2^-14 for the sums) and of the output, lse the largest score's error.  Above 16 query rows a KV head
    the product holds the weights w as bf16, the sum does not: o = sum bf16(w) v / sum w is off by half a step of 8
    bits, 2^-8 sum |v| / n, unless w is 1."""
    e = 2.0**-8 if T * H // Hk > 16 else 0.0
    x, sign, level, unit = far_scores(T, H, Hk, d, n_kv, L, size, seed=int(math.log2(size)) + T)
    p = hs.params(1, T, n_kv, 128, 128, 4, 64, H, Hk, d)
    g = to_gpu(x)
    o, lse = hs.tree_attn(p, g["q"], g["k"], g["v"], g["kv_len"], parent=g["parent"])
    # The definition from the keys' lengths: 64-bit dot products beyond 2^52 no longer tell equal scores from unequal.
    assert unit > size / 4
    for i, anc in enumerate(ref.ancestors(x["parent"][0], T)):
        rows = torch.cat([torch.arange(L), L + torch.tensor(anc)])
        top = rows[sign[i] * level[rows] == 1.0]
        assert len(top) >= 12 and float((sign[i] * level[rows]).max()) == 1.0
        v = x["v"][0, top].double().repeat_interleave(H // Hk, 1)
        want = v.mean(0)
        close(o[0, i], want, 2.0**-8 * want.abs() + (2.0**-13 + e) * v.abs().mean(0), "o")
        z = torch.full((H,), unit + math.log(len(top)), dtype=torch.float64)
        close(lse[0, i], z, (d + 8) * 2.0**-23 * z + 2.0**-22 * z, "lse")


SIZES = [2.0**24, 2.0**27, 2.0**28, 2.0**31, 2.0**34, 1e12, 2.0**70, 2.0**100]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("T,H,Hk,d", [(2, 2, 2, 64), (8, 4, 2, 128)])
def test_large_finite_scores(hs, size, T, H, Hk, d):
    check_far(hs, size, T, H, Hk, d, 2000, 1900)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("T,H,Hk,d", [(17, 2, 2, 64), (40, 4, 2, 128), (90, 6, 2, 128), (150, 4, 2, 64)])
def test_large_finite_scores_of_many_rows(hs, size, T, H, Hk, d):
    check_far(hs, size, T, H, Hk, d, 2000, 1800)


@pytest.mark.parametrize("T,H", [(17, 1), (100, 1), (70, 3)])
def test_scores_next_to_the_raise_of_the_reference_of_many_rows(hs, T, H):
    x = scores_next_to_the_limit(T, H, 20, 700, 64, seed=T)
    check_tree(hs, x, H, 1, 64, True)


@pytest.mark.parametrize("scale", [1e-44, 1e-38, 1e-30, 1e30])
@pytest.mark.parametrize("T", [3, 40])
def test_scales_at_the_ends_of_their_range(hs, scale, T):
    """Tiny scales make every weight equal; with a huge one the largest score takes all (d = 64, one place of q and k
    is not 0, so a score is one product of bf16 numbers: exact in fp32, and so is its difference to another)."""
    H, Hk, d, n_kv, L = 2, 1, 64, 500, 440
    x = make_inputs(1, T, H, Hk, d, n_kv, [L], "chain", seed=T)
    gen = torch.Generator().manual_seed(T)
    x["q"].zero_()
    x["q"][..., 7] = 1.0
    held = x["k"][:, :L + T]
    held.zero_()
    held[..., 7] = (torch.randperm(L + T, generator=gen) % 97 + 1).to(torch.bfloat16)[None, :, None]
    p = hs.params(1, T, n_kv, 128, 128, 4, 64, H, Hk, d, scale=scale)
    g = to_gpu(x)
    o, lse = hs.tree_attn(p, g["q"], g["k"], g["v"], g["kv_len"])
    e = 2.0**-8 if T * H > 16 else 0.0
    z = x["k"][0, :L + T, 0, 7].double() * float(np.float32(scale))
    for i in range(T):  # the weights from differences: exp(z - lse) loses the sum's logarithm beside 1e32
        w = torch.softmax(z[:L + i + 1], 0)
        v = x["v"][0, :L + i + 1, 0].double()
        want, spread = w @ v, w @ v.abs()
        close(o[0, i], want.expand(H, d), (2.0**-8 * want.abs() + (2.0**-13 + e) * spread).expand(H, d), "o")
        rl = torch.logsumexp(z[:L + i + 1], 0).expand(H)
        close(lse[0, i], rl, 2.0**-14 + 2.0**-22 * rl.abs(), "lse")


@pytest.mark.parametrize("b,n", [(1, 20_000), (1, 4_097), (2, 9_000), (12, 1_100)])
def test_bad_entries_over_clusters(hs, b, n):
    """Lists that break the rules first in any tile, where several CTAs sweep a slice together: one fault near each
    place in turn, faults everywhere, and a list that is bad from its last entry on."""
    rng = np.random.RandomState(n)
    n_kv = 2 * n
    good = np.stack([np.sort(rng.choice(n_kv, n, replace=False)) for _ in range(b)])
    arrays = some_arrays(b, n_kv, n, ((2, 64), (3,), ()))
    for at in sorted({0, 1, 255, 256, 511, 512, 1023, 1024, 2047, 2048, 4096, n // 2, n - 2, n - 1}):
        if at >= n:
            continue
        rows = good.copy()
        rows[rng.randint(b), at] = rng.choice([-1, -7, n_kv, 0, n_kv - 1])
        check_compact(hs, rows, None, arrays)
    rows = good.copy()
    rows[rng.rand(b, n) < 0.01] = -1
    rows[rng.rand(b, n) < 0.01] = n_kv + 3
    swap = np.flatnonzero(rng.rand(n - 1) < 0.01)
    rows[:, swap], rows[:, swap + 1] = rows[:, swap + 1], rows[:, swap].copy()
    check_compact(hs, rows, None, arrays)
    check_compact(hs, rows, list(range(b)), arrays)


@pytest.mark.parametrize("T,H,Hk,d,n_kv", [(1, 4, 2, 64, 9000), (16, 2, 2, 128, 5000), (17, 2, 2, 128, 5000),
                                           (64, 4, 2, 64, 3000), (200, 6, 2, 128, 3000)])
@pytest.mark.parametrize("weigh", [False, True])
def test_scratch_of_the_stated_size_is_enough(hs, T, H, Hk, d, n_kv, weigh):
    """Bytes behind the workspace stay as they were, and the result does not depend on what the workspace held."""
    b = 3
    g = to_gpu(make_inputs(b, T, H, Hk, d, n_kv, [n_kv - T, n_kv // 3, 0], "tree", seed=T, garbage=False))
    p = hs.params(b, T, n_kv, 128, 128, 4, 64, H, Hk, d)
    need = hs.hisa_tree_attn_workspace_size(p, weigh)
    out = []
    for fill in (0x5A, 0xFF):  # 0xFF: NaN everywhere
        block = torch.full((need + 65536,), fill, dtype=torch.uint8, device="cuda")
        o, lse, w = torch.empty_like(g["q"]), torch.empty(b, T, H, device="cuda"), g["weight"].clone()
        hs.hisa_tree_attn_fwd(p, g["q"], g["k"], g["v"], g["kv_len"], o, lse, parent=g["parent"],
                              weight=w if weigh else None, workspace=block[:need])
        assert bool((block[need:] == fill).all())
        out.append((o, lse, w))
    assert all(torch.equal(x, y) for x, y in zip(*out))


@pytest.mark.parametrize("tiles", [147, 149, 210, 444])
@pytest.mark.parametrize("T,H", [(20, 1), (100, 3), (3, 1), (128, 2)])
def test_a_tile_or_a_few_for_every_sm(hs, tiles, T, H):
    """One item, or one a sequence, whose first shares of the work may hold no key tile: attention and weights."""
    rows = tiles * 128 - T - 50
    for lens in ([rows], [rows // 3, rows // 2, 0, rows - rows // 3 - rows // 2]):
        n_kv = max(lens) + T
        x = make_inputs(len(lens), T, H, 1, 64, n_kv, lens, "tree", seed=T, garbage=False)
        check_tree(hs, x, H, 1, 64, True)


@pytest.mark.parametrize("T,H,Hk", [(7, 1, 1), (8, 1, 1), (9, 1, 1), (4, 4, 2), (3, 6, 2), (1, 16, 2), (2, 10, 2)])
@pytest.mark.parametrize("d", [64, 128])
def test_weights_where_scores_are_kept_and_where_not(hs, T, H, Hk, d):
    x = make_inputs(3, T, H, Hk, d, 700, [700 - T, 128, 5], "tree", seed=T + H)
    check_tree(hs, x, H, Hk, d, True)
