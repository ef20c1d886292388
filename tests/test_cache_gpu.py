"""The cache operators on the GPU against their definitions in 64 bits.

Tolerances.  An fp32 score of d products is off by at most (d + 8) 2^-23 times scale * sum |q_c k_c| (2^-23 a step:
the tensor cores truncate), and its scaling, the exponential and the sums add a relative 2^-16; a weight that enters
the product as a pair of bf16 numbers is off by 2^-16 more.  So a softmax weight is off by a relative
delta = (d + 8) 2^-23 size + 2^-14 at most, numerator and denominator each, and
    |o - ref|   <= 2^-8 |ref| + (2 delta + e) sum p |v|      (2^-8: the output's rounding to bf16)
with e = 2^-8 where a KV head has more than 16 query rows (T H / Hk): there a weight enters the product as one bf16
number, off by half a step of 8 significant bits, 2^-8 relative, in the numerator alone; else e = 0.
    |lse - ref| <= delta + 2^-22 |ref|
    |w - ref|   <= (delta + 2^-21 max |lse|) received + 2^-20 |ref| + 2^-110
where 2^-110 covers fp32's range: a weight below 2^-126 has no relative precision and may count as 0, and at most
H T <= 2^16 of them meet in one row, 2^-110 in all.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import cache_reference as ref  # noqa: E402


@pytest.fixture(scope="module")
def hs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import hierarchical_sparse_attention_block_b200 as m

    return m


def make_parent(kind, b, T, gen):
    at = torch.arange(T, dtype=torch.int32)
    if kind == "chain":
        return None
    if kind == "chain_listed":
        return (at - 1).repeat(b, 1)
    if kind == "star":
        return torch.full((b, T), -1, dtype=torch.int32)
    parent = at[None] - torch.randint(1, 6, (b, T), generator=gen, dtype=torch.int32)
    parent = parent.clamp_min(-1)
    if kind == "holes":  # empty slots anywhere, and whole sequences without a token
        parent[torch.rand(b, T, generator=gen) < 0.3] = -2
        parent[-1] = -2
    return parent


def make_inputs(b, T, H, Hk, d, n_kv, lens, kind, seed, spread=1.0, garbage=True):
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape, by=1.0):
        return (torch.randn(shape, generator=gen) * by).to(torch.bfloat16)

    x = {"q": normal(b, T, H, d, by=spread), "k": normal(b, n_kv, Hk, d), "v": normal(b, n_kv, Hk, d),
         "kv_len": torch.tensor(lens, dtype=torch.int32), "parent": make_parent(kind, b, T, gen),
         "weight": torch.rand(b, n_kv, generator=gen)}
    if garbage:  # what no token sees: rows behind the drafted ones, and the rows of empty slots
        for s in range(b):
            L = lens[s]
            anc = ref.ancestors(None if x["parent"] is None else x["parent"][s], T)
            dead = [L + i for i in range(T) if anc[i] is None] + list(range(L + T, n_kv))
            for name, values in (("k", (math.nan, math.inf)), ("v", (math.inf, math.nan))):
                x[name][s, dead[0::2]] = values[0]
                x[name][s, dead[1::2]] = values[1]
    return x


def to_gpu(x):
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def delta(d, size):
    return (d + 8) * 2.0**-23 * size + 2.0**-14


def close(got, want, tol, what):
    got, want = got.double().cpu(), want.double()
    bad = ~((got - want).abs() <= tol) & ~((got == want) | (got.isnan() & want.isnan()))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}: "
                           f"{got[bad][0]} for {want[bad][0]}")


def check_tree(hs, x, H, Hk, d, weigh):
    b, T = x["q"].shape[:2]
    n_kv = x["k"].shape[1]
    p = hs.params(b, T, n_kv, 128, 128, 4, 64, H, Hk, d)
    g = to_gpu(x)
    o = torch.full((b, T, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b, T, H), 7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    hs.hisa_tree_attn_fwd(p, g["q"], g["k"], g["v"], g["kv_len"], o, lse, parent=g["parent"],
                          weight=g["weight"] if weigh else None, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    ro, rl, received, spread, size = ref.tree_attention(x["q"], x["k"], x["v"], x["kv_len"], x["parent"],
                                                        1 / math.sqrt(d))
    dl = delta(d, size)
    close(lse, rl, dl + 2.0**-22 * rl.abs().nan_to_num(0, 0, 0), "lse")
    e = 2.0**-8 if T * H // Hk > 16 else 0.0
    close(o, ro, 2.0**-8 * ro.abs() + (2 * dl + e) * spread, "o")
    top = float(rl[rl > -math.inf].abs().max()) if (rl > -math.inf).any() else 0.0
    if weigh:
        want = ref.weight_after(x["weight"], received, x["kv_len"], T)
        close(g["weight"], want, (dl + 2.0**-21 * top) * received + 2.0**-20 * want.abs() + 2.0**-110, "weight")
    else:
        assert torch.equal(g["weight"].cpu(), x["weight"])
    return p, g, o, lse, received, dl


# b, T, H, Hk, d, n_kv, lens, tree
TREES = [
    (1, 1, 1, 1, 64, 1, [0], "chain"),                            # one row of cache, no context
    (2, 1, 4, 4, 128, 300, [0, 299], "chain"),
    (3, 1, 16, 2, 128, 1000, [999, 128, 127], "chain"),
    (3, 5, 6, 2, 64, 140, [0, 1, 135], "tree"),
    (2, 33, 8, 2, 128, 161, [128, 127], "tree"),                  # 132 query rows a KV head: just over one tile
    (2, 64, 8, 1, 128, 400, [0, 333], "tree"),                    # 512 query rows a KV head
    (1, 256, 4, 2, 64, 700, [444], "chain"),
    (1, 256, 2, 1, 128, 513, [257], "chain_listed"),
    (4, 40, 9, 3, 128, 260, [200, 0, 220, 60], "holes"),
    (2, 100, 3, 1, 64, 229, [129, 100], "holes"),                 # 300 query rows a KV head
    (5, 7, 12, 4, 128, 1000, [0, 993, 500, 128, 121], "star"),
    (70, 3, 2, 2, 64, 40, [i % 38 for i in range(70)], "tree"),   # more sequences than a warp
    (1, 4, 2, 1, 128, 20011, [20007], "tree"),                    # one long cache split over the SMs
    (300, 2, 2, 1, 128, 90, [(7 * i) % 89 for i in range(300)], "chain"),
    (2, 2, 128, 2, 64, 300, [100, 290], "tree"),                  # 64 query heads a KV head
]


@pytest.mark.parametrize("case", TREES, ids=lambda c: "b%d_T%d_H%d_Hk%d_d%d_n%d_%s" % (*c[:6], c[7]))
@pytest.mark.parametrize("weigh", [False, True], ids=["plain", "weighed"])
def test_tree_attention(hs, case, weigh):
    b, T, H, Hk, d, n_kv, lens, kind = case
    x = make_inputs(b, T, H, Hk, d, n_kv, lens, kind, seed=n_kv + T)
    check_tree(hs, x, H, Hk, d, weigh)


@pytest.mark.parametrize("case", TREES, ids=lambda c: "b%d_T%d_H%d_Hk%d_d%d_n%d_%s" % (*c[:6], c[7]))
@pytest.mark.parametrize("path", ["all", "chain", "some", "none"])
def test_cache_weight(hs, case, path):
    b, T, H, Hk, d, n_kv, lens, kind = case
    x = make_inputs(b, T, H, Hk, d, n_kv, lens, kind, seed=2 * n_kv + T)
    rng = np.random.RandomState(T)
    lists = None
    if path != "all":
        lists = torch.full((b, T), -1, dtype=torch.int32)
        for s in range(b):
            anc = ref.ancestors(None if x["parent"] is None else x["parent"][s], T)
            take = {"chain": next((a for a in reversed(anc) if a is not None), []), "none": [],
                    "some": sorted(rng.choice(T, rng.randint(0, T + 1), replace=False))}[path]
            lists[s, :len(take)] = torch.tensor(take, dtype=torch.int32)
    _, lse, _, _, _ = ref.tree_attention(x["q"], x["k"], None, x["kv_len"], x["parent"], 1 / math.sqrt(d))
    lse = lse.float()
    lse[0, 0, 0] = -math.inf  # a row that counts nothing
    counted = None if lists is None else [set(int(i) for i in row if i >= 0) for row in lists]
    _, _, received, _, size = ref.tree_attention(x["q"], x["k"], None, x["kv_len"], x["parent"], 1 / math.sqrt(d),
                                                 counted, lse)
    want = ref.weight_after(x["weight"], received, x["kv_len"], T)
    p = hs.params(b, T, n_kv, 128, 128, 4, 64, H, Hk, d)
    g = to_gpu(x)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    first = g["weight"].clone()
    args = (p, g["q"], g["k"], g["kv_len"], lse.cuda())
    kw = dict(parent=g["parent"], path=None if lists is None else lists.cuda(), dev_status=status)
    hs.hisa_cache_weight(*args, g["weight"], **kw)
    assert int(status) == 0
    top = float(lse[lse > -math.inf].abs().max()) if (lse > -math.inf).any() else 0.0
    tol = (delta(d, size) + 2.0**-21 * top) * received + 2.0**-20 * want.abs() + 2.0**-110
    close(g["weight"], want, tol, "weight")
    hs.hisa_cache_weight(*args, first, **kw)  # the same bits again
    assert torch.equal(first, g["weight"])


def test_large_scores_and_small_rows(hs):
    """Scores of a spread of 40: most weights vanish, the running maximum moves often."""
    x = make_inputs(2, 20, 8, 2, 128, 900, [880, 500], "tree", seed=3, spread=40.0)
    check_tree(hs, x, 8, 2, 128, True)


@pytest.mark.parametrize("Hk,T", [(16, 1), (4, 3)])
def test_long_caches_of_a_batch(hs, Hk, T):
    """Hundreds of key tiles in a row for every SM, heads and sequences ending inside the SMs' shares: every row
    agrees with the definition, and with itself when the call is repeated."""
    b, H, d, n_kv = 4, 16, 128, 24000
    gen = torch.Generator(device="cuda").manual_seed(12)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)

    q, k, v = normal(b, T, H, d), normal(b, n_kv, Hk, d), normal(b, n_kv, Hk, d)
    lens = torch.tensor([23990, 23000, 17001, 23808], dtype=torch.int32, device="cuda")
    p = hs.params(b, T, n_kv, 128, 128, 4, 64, H, Hk, d)
    first = hs.tree_attn(p, q, k, v, lens)
    for _ in range(20):
        assert all(torch.equal(x, y) for x, y in zip(first, hs.tree_attn(p, q, k, v, lens)))
    for s in range(b):
        L = int(lens[s])
        z = torch.einsum("ihd,nhd->ihn", q[s].double(), k[s, :L + T].double().repeat_interleave(H // Hk, 1)) / d**0.5
        at = torch.arange(L + T, device="cuda")
        z.masked_fill_((at > L + torch.arange(T, device="cuda")[:, None])[:, None], -math.inf)
        lse = torch.logsumexp(z, -1)
        pr = (z - lse[..., None]).exp()
        vv = v[s, :L + T].double().repeat_interleave(H // Hk, 1)
        want, spread = torch.einsum("ihn,nhd->ihd", pr, vv), torch.einsum("ihn,nhd->ihd", pr, vv.abs())
        dl = delta(d, 100.0 / d**0.5 * 3)  # sum |q_c k_c| of 128 pairs of normal values: below 300
        close(first[1][s], lse.cpu(), dl + 2.0**-22 * lse.cpu().abs(), "lse")
        close(first[0][s], want.cpu(), 2.0**-8 * want.cpu().abs() + 2 * dl * spread.cpu(), "o")


def test_rising_scores(hs):
    """Every tile raises the maximum: keys grow along the cache in the query's own direction."""
    x = make_inputs(1, 8, 4, 2, 128, 2048, [2040], "tree", seed=4)
    direction = torch.randn(128, generator=torch.Generator().manual_seed(1))
    x["q"] = (x["q"].float() * 0.1 + direction).to(torch.bfloat16)
    x["k"] = (x["k"].float() * 0.1 + direction * torch.linspace(-2, 4, 2048)[None, :, None, None]).to(torch.bfloat16)
    check_tree(hs, x, 4, 2, 128, True)


def test_lowest_and_infinite_keys(hs):
    """Context keys of the type's lowest value and -inf scores keep no weight; +inf or NaN keys make a row NaN."""
    x = make_inputs(1, 3, 2, 1, 64, 300, [290], "star", seed=5, garbage=False)
    x["q"] = x["q"].abs()
    x["k"][0, :100] = torch.finfo(torch.bfloat16).min
    check_tree(hs, x, 2, 1, 64, False)
    x["k"][0, :100] = -math.inf
    p = hs.params(1, 3, 300, 128, 128, 4, 64, 2, 1, 64)
    g = to_gpu(x)
    o, lse = hs.tree_attn(p, g["q"], g["k"], g["v"], g["kv_len"], parent=g["parent"])
    assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(lse).all())
    g["k"][0, 5] = math.nan
    o, lse = hs.tree_attn(p, g["q"], g["k"], g["v"], g["kv_len"], parent=g["parent"])
    assert bool(o.isnan().all()) and bool(lse.isnan().all())


@pytest.mark.parametrize("T,H,Hk,d", [(6, 4, 2, 128), (200, 2, 1, 64)])
def test_a_branch_with_infinite_values_stays_alone(hs, T, H, Hk, d):
    """Values that are no numbers reach the rows that see them, and no other branch."""
    n_kv, L = 700, 300
    x = make_inputs(1, T, H, Hk, d, n_kv, [L], "tree", seed=6)
    x["parent"][0, 0], x["parent"][0, 1] = -1, -1
    x["v"][0, L + 1, 0, 3] = math.inf
    x["v"][0, L + 1, 0, 5] = math.nan
    x["k"][0, L + 2] = math.nan
    p = hs.params(1, T, n_kv, 128, 128, 4, 64, H, Hk, d)
    g = to_gpu(x)
    o, lse = hs.tree_attn(p, g["q"], g["k"], g["v"], g["kv_len"], parent=g["parent"])
    o = o.cpu().float()
    anc = ref.ancestors(x["parent"][0], T)
    for i in range(T):
        row = o[0, i, 0]
        if 2 in anc[i]:
            assert row.isnan().all()
        elif 1 in anc[i]:
            assert row[3] == math.inf and row[5].isnan()
            assert torch.isfinite(row[[c for c in range(d) if c not in (3, 5)]]).all()
        else:
            assert torch.isfinite(row).all(), i


def test_bad_lengths_and_parents_are_skipped_and_flagged(hs):
    b, T, H, Hk, d, n_kv = 4, 6, 4, 2, 128, 200
    x = make_inputs(b, T, H, Hk, d, n_kv, [50, 60, 70, 80], "tree", seed=7)
    p = hs.params(b, T, n_kv, 128, 128, 4, 64, H, Hk, d)
    good = hs.tree_attn(p, *[to_gpu(x)[n] for n in ("q", "k", "v", "kv_len")], parent=x["parent"].cuda())
    x["kv_len"][0], x["kv_len"][2] = -1, n_kv - T + 1
    x["parent"][3, 4] = 4  # not before itself
    g = to_gpu(x)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = torch.full_like(g["q"], 3.0), torch.full((b, T, H), 3.0, device="cuda")
    before = g["weight"].clone()
    hs.hisa_tree_attn_fwd(p, g["q"], g["k"], g["v"], g["kv_len"], o, lse, parent=g["parent"], weight=g["weight"],
                          dev_status=status)
    assert int(status) == hs.STATUS_BAD_INDEX
    for s in (0, 2):
        assert (o[s] == 0).all() and (lse[s] == -math.inf).all() and torch.equal(g["weight"][s], before[s])
    assert torch.equal(o[1], good[0][1]) and torch.equal(lse[1], good[1][1])
    assert (o[3, 4] == 0).all() and (lse[3, 4] == -math.inf).all() and torch.equal(o[3, :4], good[0][3, :4])
    status.zero_()
    path = torch.full((b, T), -1, dtype=torch.int32, device="cuda")
    path[1, :4] = torch.tensor([2, 1, 9, 3])  # 1 is not ascending, 9 no slot
    w = before.clone()
    hs.hisa_cache_weight(p, g["q"], g["k"], g["kv_len"], lse, w, parent=g["parent"], path=path, dev_status=status)
    assert int(status) == hs.STATUS_BAD_INDEX
    path[1, :4] = torch.tensor([2, 3, -1, -1])
    want = before.clone()
    hs.hisa_cache_weight(p, g["q"], g["k"], g["kv_len"], lse, want, parent=g["parent"], path=path)
    assert torch.equal(w, want)


def test_same_bits_on_every_run_and_stream(hs):
    b, T, H, Hk, d, n_kv = 3, 16, 16, 4, 128, 5000
    g = to_gpu(make_inputs(b, T, H, Hk, d, n_kv, [4900, 1234, 3], "tree", seed=8))
    p = hs.params(b, T, n_kv, 128, 128, 4, 64, H, Hk, d)
    start = g["weight"].clone()

    def once(stream=None):
        w = start.clone()
        o, lse = torch.empty_like(g["q"]), torch.empty(b, T, H, device="cuda")
        torch.cuda.synchronize()
        hs.hisa_tree_attn_fwd(p, g["q"], g["k"], g["v"], g["kv_len"], o, lse, parent=g["parent"], weight=w,
                              stream=stream)
        torch.cuda.synchronize()
        return o, lse, w

    first = once()
    for stream in (None, torch.cuda.Stream()):
        assert all(torch.equal(x, y) for x, y in zip(first, once(stream)))
    # without an LSE to write
    w = start.clone()
    o = torch.empty_like(g["q"])
    hs.hisa_tree_attn_fwd(p, g["q"], g["k"], g["v"], g["kv_len"], o, parent=g["parent"], weight=w)
    assert torch.equal(o, first[0]) and torch.equal(w, first[2])


def test_captured_steps_share_a_workspace(hs):
    """Two captured graphs with one workspace, replayed in turn with changed lengths and inputs."""
    shapes = [(2, 4, 8, 2, 128, 900, [800, 30]), (3, 9, 4, 4, 64, 400, [390, 0, 200])]
    runs, ws = [], None
    sizes = []
    for b, T, H, Hk, d, n_kv, lens in shapes:
        p = hs.params(b, T, n_kv, 128, 128, 4, 64, H, Hk, d)
        sizes += [hs.hisa_tree_attn_workspace_size(p, True), hs.hisa_cache_weight_workspace_size(p)]
    ws = torch.empty(max(sizes + [16]), dtype=torch.uint8, device="cuda")
    for b, T, H, Hk, d, n_kv, lens in shapes:
        p = hs.params(b, T, n_kv, 128, 128, 4, 64, H, Hk, d)
        x = make_inputs(b, T, H, Hk, d, n_kv, lens, "tree", seed=9)
        g = to_gpu(x)
        o, lse = torch.empty_like(g["q"]), torch.empty(b, T, H, device="cuda")

        def step(p=p, g=g, o=o, lse=lse):
            hs.hisa_tree_attn_fwd(p, g["q"], g["k"], g["v"], g["kv_len"], o, lse, parent=g["parent"],
                                  weight=g["weight"], workspace=ws)
            hs.hisa_cache_weight(p, g["q"], g["k"], g["kv_len"], lse, g["weight"], parent=g["parent"], workspace=ws)

        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        runs.append((graph, step, g, o, lse))
    for turn in range(2):
        for graph, step, g, o, lse in runs:
            g["q"].copy_(torch.roll(g["q"], 1, 1))
            g["kv_len"][0] -= 7 * turn
            start = g["weight"].clone()
            graph.replay()
            got = o.clone(), lse.clone(), g["weight"].clone()
            g["weight"].copy_(start)
            step()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(got, (o, lse, g["weight"])))


def test_offsets_beyond_32_bits(hs):
    """The second sequence's rows lie more than 2^31 elements into K and V."""
    b, T, H, Hk, d, n_kv = 2, 5, 16, 16, 128, 1_100_000
    x = make_inputs(b, T, H, Hk, d, 300, [3, 290], "tree", seed=10)
    k = torch.empty(b, n_kv, Hk, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    k[:, :300], v[:, :300] = x["k"].cuda(), x["v"].cuda()
    g = to_gpu(x)
    small = hs.params(b, T, 300, 128, 128, 4, 64, H, Hk, d)
    want = hs.tree_attn(small, g["q"], g["k"], g["v"], g["kv_len"], parent=g["parent"])
    p = hs.params(b, T, n_kv, 128, 128, 4, 64, H, Hk, d)
    w = torch.zeros(b, n_kv, device="cuda")
    o, lse = torch.empty_like(g["q"]), torch.empty(b, T, H, device="cuda")
    hs.hisa_tree_attn_fwd(p, g["q"], k, v, g["kv_len"], o, lse, parent=g["parent"], weight=w)
    close(lse, want[1].cpu(), 2.0**-14, "lse")
    close(o, want[0].cpu(), 2.0**-7 * want[0].cpu().abs().double() + 2.0**-12, "o")
    w2 = torch.zeros(b, n_kv, device="cuda")
    hs.hisa_cache_weight(p, g["q"], k, g["kv_len"], lse, w2, parent=g["parent"])
    for x_ in (w, w2):
        assert abs(float(x_[1, :295].sum()) - T * H) < 0.01 * T * H and float(x_[1, 295:].abs().max()) == 0
    # the move: rows of the far sequence
    rows = torch.tensor([[0, 1, 2], [100, 200, n_kv - 1]], dtype=torch.int32, device="cuda")
    k[1, n_kv - 1] = 3.0
    keep = k[1, [100, 200, n_kv - 1]].clone()
    hs.hisa_cache_compact(p, rows, [k])
    assert torch.equal(k[1, :3], keep) and torch.equal(k[1, 200], keep[1])


# ------------------------------------------------------------------ the choice of the kept rows

def check_keep(hs, w, lens, budget, n_first=0, n_recent=0, alias=False):
    b, n_kv = w.shape
    p = hs.params(b, 1, n_kv, 128, 128, 4, 64)
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kept = kv_len if alias else torch.full((b,), -7, dtype=torch.int32, device="cuda")
    idx = torch.full((b, budget), -7, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    hs.hisa_cache_keep(p, w.cuda(), kv_len, budget, idx, kept, n_first, n_recent, dev_status=status)
    assert int(status) == (0 if all(0 <= L <= n_kv for L in lens) else hs.STATUS_BAD_INDEX)
    for s, L in enumerate(lens):
        want = ref.keep(w[s].numpy(), L, budget, n_first, n_recent) if 0 <= L <= n_kv else []
        got = idx[s].cpu().tolist()
        assert int(kept[s]) == len(want)
        assert got[:len(want)] == want, f"sequence {s}"
        assert all(x == -1 for x in got[len(want):])


@pytest.mark.parametrize("n_kv", [1, 2, 31, 33, 1000, 4097, 70001])
@pytest.mark.parametrize("values", ["normal", "equal", "steps", "zeros", "wild"])
def test_kept_rows(hs, n_kv, values):
    gen = torch.Generator().manual_seed(n_kv)
    b = 4
    w = torch.rand(b, n_kv, generator=gen)
    if values == "equal":
        w = torch.full((b, n_kv), 0.25)
    elif values == "steps":  # few different values: ties at the border
        w = (w * 5).floor() / 5
    elif values == "zeros":
        w = torch.where(w < 0.5, 0.0, -0.0)
    elif values == "wild":
        w = torch.randn(b, n_kv, generator=gen) * torch.exp(20 * torch.randn(b, n_kv, generator=gen))
        pick = torch.randint(0, 12, (b, n_kv), generator=gen)
        for i, x in enumerate((math.inf, -math.inf, math.nan, -math.nan, 1e-42, -1e-42, 0.0, -0.0)):
            w[pick == i] = x
    lens = [n_kv, n_kv // 2, 0, max(0, n_kv - 1)]
    for budget in sorted({1, (n_kv + 1) // 2, max(1, n_kv - 1), n_kv}):
        check_keep(hs, w, lens, budget)
        check_keep(hs, w, lens, budget, budget // 3, budget // 4, alias=True)
    check_keep(hs, w, lens, (n_kv + 1) // 2, 0, (n_kv + 1) // 2)  # nothing is left to choose


def test_kept_rows_of_one_long_cache_and_many_short_ones(hs):
    gen = torch.Generator().manual_seed(1)
    check_keep(hs, torch.rand(1, 1_300_001, generator=gen).exp(), [1_300_001], 300_007, 128, 4096)
    w = (torch.rand(2, 600_000, generator=gen) * 1000).floor()
    check_keep(hs, w, [600_000, 599_999], 100_000, 3, 5)
    lens = [(i * 37) % 400 for i in range(500)]
    check_keep(hs, torch.rand(500, 400, generator=gen), lens, 64, 4, 16)


@pytest.mark.parametrize("b", [1, 3, 4])
def test_kept_rows_of_a_few_long_caches(hs, b):
    """Sequences that finish at different steps of the selection side by side: ties down to the last bit, equal
    weights, a threshold in the first digit, lengths below the budget, out of range and of zero."""
    gen = torch.Generator().manual_seed(b)
    n_kv = 540_001
    w = torch.rand(b, n_kv, generator=gen)
    w[0] = (w[0] * 50).floor() + 2.0**-10 * (w[0] < 0.3)
    w[-1, 1000:200_000] = 0.25
    for lens in ([n_kv] * b, [n_kv - 1, 70_000, 0, n_kv][:b], [n_kv + 1, n_kv, -1, 262_144][:b], [524_289] * b):
        for budget, first, recent in ((70_001, 3, 1000), (1, 0, 0), (50, 20, 30), (n_kv - 2, 1, 1)):
            check_keep(hs, w, lens, budget, first, recent, alias=budget == 70_001)
    w[0, :135_000], w[0, 135_000:] = 1.0, 2.0**40  # the first digit decides
    check_keep(hs, w, [n_kv] * b, n_kv - 135_000)


@pytest.mark.parametrize("b,n_kv", [(1, 7_900_001), (9, 800_003), (10, 400_001), (60, 110_003)])
def test_kept_rows_of_parts_beyond_shared_memory(hs, b, n_kv):
    gen = torch.Generator().manual_seed(n_kv)
    w = torch.rand(b, n_kv, generator=gen)
    w[-1] = (w[-1] * 300).floor()
    check_keep(hs, w, [n_kv - 5 * s for s in range(b)], 20_000, 5, 600)


def test_long_caches_on_two_streams(hs):
    """Choices over long caches on two streams at once, and one captured and replayed: as one after the other."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    n_kv, budget = 600_000, 9_000
    p = hs.params(2, 1, n_kv, 128, 128, 4, 64)
    w = [torch.rand(2, n_kv, generator=gen, device="cuda") for _ in range(4)]
    lens = torch.tensor([n_kv, 560_001], dtype=torch.int32, device="cuda")

    def choose(x, stream=None):
        idx = torch.empty(2, budget, dtype=torch.int32, device="cuda")
        kept = torch.empty(2, dtype=torch.int32, device="cuda")
        torch.cuda.current_stream().synchronize()
        for _ in range(5):
            hs.hisa_cache_keep(p, x, lens, budget, idx, kept, 1, 7, stream=stream)
        return idx, kept

    want = [choose(x) for x in w]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [choose(x, streams[i % 2]) for i, x in enumerate(w)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    x, idx, kept = w[0].clone(), torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hs.hisa_cache_keep(p, x, lens, budget, idx, kept, 1, 7)
    for y, z in zip(w, want):
        x.copy_(y)
        graph.replay()
        assert torch.equal(idx, z[0]) and torch.equal(kept, z[1])


def test_bad_lengths_keep_nothing(hs):
    check_keep(hs, torch.rand(3, 100), [-1, 50, 101], 20)


# ------------------------------------------------------------------ the move

def check_compact(hs, rows, begin, arrays):
    b, n_kv = arrays[0].shape[:2]
    p = hs.params(b, 1, n_kv, 128, 128, 4, 64)
    want, any_bad = [], False
    for a in arrays:
        out = []
        for s in range(b):
            x, bad = ref.compact(a[s], rows[s], 0 if begin is None else int(begin[s]))
            out.append(x)
            any_bad |= bad
        want.append(torch.stack(out))
    got = [a.cuda() for a in arrays]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    hs.hisa_cache_compact(p, torch.tensor(np.asarray(rows), dtype=torch.int32, device="cuda"), got,
                          dst_begin=None if begin is None else torch.tensor(begin, dtype=torch.int32, device="cuda"),
                          dev_status=status)
    for x, y in zip(got, want):
        assert torch.equal(x.cpu(), y)
    assert int(status) == (hs.STATUS_BAD_INDEX if any_bad else 0)


def some_arrays(b, n_kv, seed, widths=((2, 64), (3,), (), (5,), (129,))):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randint(-2**31, 2**31 - 1, (b, n_kv, *w), generator=gen, dtype=torch.int32) for w in widths]


@pytest.mark.parametrize("n_kv,n", [(1, 1), (7, 3), (300, 300), (300, 17), (5000, 1234), (5000, 4999), (70000, 30000)])
def test_moved_rows(hs, n_kv, n):
    rng = np.random.RandomState(n)
    b = 3
    rows = np.full((b, n), -1)
    for s, m in enumerate((n, max(1, n // 2), n - 1)):
        rows[s, :m] = np.sort(rng.choice(n_kv, m, replace=False))
    check_compact(hs, rows, None, some_arrays(b, n_kv, n, ((2, 64), (3,), ()) if n_kv > 6000 else ((2, 64), (3,), (), (5,), (129,))))


def test_moved_rows_of_other_types(hs):
    gen = torch.Generator().manual_seed(2)
    arrays = [torch.randn(2, 900, 4, 64, generator=gen).to(torch.bfloat16), torch.rand(2, 900, generator=gen),
              torch.randint(0, 9, (2, 900), generator=gen), torch.randn(2, 900, 6, generator=gen).to(torch.float16)]
    rows = np.stack([np.arange(450) * 2, np.arange(450) + 450])
    check_compact(hs, rows, None, arrays)


def test_commit_behind_the_context(hs):
    rows = np.array([[5, 7, 8, -1], [96, 97, 98, 99], [0, -1, -1, -1], [50, 51, 52, 60]])
    check_compact(hs, rows, [5, 96, 0, 40], some_arrays(4, 100, 3))


@pytest.mark.parametrize("n", [6, 700])
def test_bad_entries_move_nothing(hs, n):
    """Entries out of range, out of order or in front of their place, between good ones and over several tiles."""
    rng = np.random.RandomState(n)
    n_kv = 4 * n
    rows = np.stack([np.sort(rng.choice(n_kv, n, replace=False)) for _ in range(6)])
    rows[1, n // 2] = -1               # padding in the middle
    rows[2, n // 3] = n_kv             # out of range
    rows[2, n // 2] = -5
    rows[3, n // 2] = rows[3, n // 2 - 1]  # twice the same
    rows[4] = rows[4][::-1]            # descending
    rows[5] = rng.randint(-3, n_kv + 3, n)
    check_compact(hs, rows, None, some_arrays(6, n_kv, n, ((2, 64), (3,), ())))
    check_compact(hs, rows, [0, 3, n, -1, 1, 2], some_arrays(6, n_kv, n + 1, ((65,), ())))


# ------------------------------------------------------------------ streams, graphs, refused calls

def cache_of(b, T, H, Hk, d, n_kv, lens, seed):
    """A cache and its drafted tokens on the GPU, and the front ends' steps over it as one function of a stream."""
    g = to_gpu(make_inputs(b, T, H, Hk, d, n_kv, lens, "tree", seed, garbage=False))
    g["position"] = torch.arange(n_kv, device="cuda").repeat(b, 1)
    return g


def all_steps(hs, g, H, Hk, d, budget, stream=None):
    """Attention, weights of a path, its commit, an eviction: everything that changes or comes out."""
    b, T = g["q"].shape[:2]
    p = hs.params(b, T, g["k"].shape[1], 128, 128, 4, 64, H, Hk, d)
    o, lse = hs.tree_attn(p, g["q"], g["k"], g["v"], g["kv_len"], parent=g["parent"], stream=stream)
    hs.hisa_cache_weight(p, g["q"], g["k"], g["kv_len"], lse, g["weight"], parent=g["parent"], path=g["path"],
                         stream=stream)
    hs.hisa_cache_compact(p, g["rows"], [g["k"], g["v"], g["position"], g["weight"]], dst_begin=g["kv_len"],
                          stream=stream)
    keep = hs.evict(p, g["weight"], g["kv_len"], budget, [g["k"], g["v"], g["position"]], 4, 16, stream=stream)
    return [o, lse, keep, g["kv_len"], g["k"], g["v"], g["position"], g["weight"]]


def with_path(g):
    T = g["q"].shape[1]
    path = torch.full_like(g["parent"], -1)
    for s in range(path.shape[0]):
        chain = ref.ancestors(g["parent"][s].cpu(), T)[T - 1]
        path[s, :len(chain)] = torch.tensor(chain)
    g["path"] = path
    g["rows"] = torch.where(path >= 0, path + g["kv_len"][:, None], -1)
    return g


def copy_of(g):
    return {n: t.clone() for n, t in g.items()}


SETS = [(2, 9, 8, 2, 128, 700, [600, 33], 200), (1, 4, 4, 4, 64, 9000, [8990], 3000)]


def test_two_streams_at_once(hs):
    """The steps of two caches on two streams, over and over, scratch and outputs from the front ends: as alone."""
    kept, want = [], []
    for i, (b, T, H, Hk, d, n_kv, lens, budget) in enumerate(SETS):
        g = with_path(cache_of(b, T, H, Hk, d, n_kv, lens, 40 + i))
        kept.append(g)
        want.append([t.clone() for t in all_steps(hs, copy_of(g), H, Hk, d, budget)])
    turns = 12
    caches = [[copy_of(g) for _ in range(turns)] for g in kept]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for turn in range(turns):
        for i, (b, T, H, Hk, d, n_kv, lens, budget) in enumerate(SETS):
            out = all_steps(hs, caches[i][turn], H, Hk, d, budget, streams[i])
            torch.cuda.current_stream().wait_stream(streams[i])
            got[i].append([t.clone() for t in out])  # on the current stream, the originals dropped at once
            del out
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(out, want[i]))


def test_captured_evictions(hs):
    """Weights, commit and eviction captured once and replayed over changing lengths, weights and paths."""
    b, T, H, Hk, d, n_kv, lens, budget = 2, 9, 8, 2, 128, 700, [600, 33], 200
    live = with_path(cache_of(b, T, H, Hk, d, n_kv, lens, 50))
    all_steps(hs, copy_of(live), H, Hk, d, budget)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = all_steps(hs, live, H, Hk, d, budget)
    for turn, lens in enumerate(([650, 5], [199, 691], [0, 210])):
        g = with_path(cache_of(b, T, H, Hk, d, n_kv, lens, 60 + turn))
        for n, t in g.items():
            live[n].copy_(t)
        graph.replay()
        want = all_steps(hs, g, H, Hk, d, budget)
        assert all(torch.equal(x, y) for x, y in zip(out, want))


def test_a_refused_eviction_changes_nothing(hs):
    b, n_kv = 2, 300
    p = hs.params(b, 1, n_kv, 128, 128, 4, 64)
    weight, kv_len = torch.rand(b, n_kv, device="cuda"), torch.tensor([300, 120], dtype=torch.int32, device="cuda")
    k = torch.randn(b, n_kv, 8, device="cuda")
    arrays = ([k[:, ::2]], [k, k], [k, weight], [k] * 8, [k.to(torch.int8)[..., :6].contiguous()])
    before = [t.clone() for t in (k, weight, kv_len)]
    for a in arrays:
        with pytest.raises(hs.HisaError):
            hs.evict(p, weight, kv_len, 100, a)
    with pytest.raises(hs.HisaError):
        hs.evict(p, weight, kv_len, 0, [k])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(before, (k, weight, kv_len)))


@pytest.mark.parametrize("T,H,rows", [(20, 1, 95_300), (100, 2, 95_300), (100, 2, 96_700), (3, 1, 95_300)])
def test_five_tiles_for_every_sm(hs, T, H, rows):
    """One item over the whole GPU: the first share of the work may hold no key tile at all."""
    x = make_inputs(1, T, H, 1, 64, rows + T, [rows], "tree", seed=T, garbage=False)
    check_tree(hs, x, H, 1, 64, True)


@pytest.mark.parametrize("first", [-300.0, -20.0, 20.0, 300.0])
@pytest.mark.parametrize("T", [1, 5, 40])
def test_a_first_key_far_from_the_others(hs, first, T):
    """Every segment of keys starts with a score far above or below the rest, both for some rows."""
    H, Hk, d = 4, 2, 64
    x = make_inputs(3, T, H, Hk, d, 700, [660, 3, 128], "tree", seed=T)
    for t in range(0, 128 * 5, 128):
        for s, L in enumerate((660, 3, 128)):
            if t < L:
                x["k"][s, t] = (first * x["q"][s, 0, ::H // Hk].float()).to(torch.bfloat16)
    check_tree(hs, x, H, Hk, d, True)


@pytest.mark.parametrize("T,H", [(15, 1), (16, 1), (17, 1), (127, 1), (128, 1), (129, 1), (64, 4), (129, 2)])
def test_query_rows_at_the_tiles_borders(hs, T, H):
    x = make_inputs(2, T, H, 1, 64, 420, [420 - T, 128], "tree", seed=T + H)
    check_tree(hs, x, H, 1, 64, True)


# ------------------------------------------------------------------ the calls together

def test_a_bounded_cache_through_a_decode(hs):
    """A prompt's window, an eviction, two steps of drafted trees with their accepted paths and commits, and another
    eviction: every tensor of the cache follows a cache kept as plain lists of rows."""
    b, H, Hk, d, n_kv, budget = 2, 8, 2, 128, 640, 200
    gen = torch.Generator().manual_seed(11)

    def normal(*shape):
        return torch.randn(shape, generator=gen).to(torch.bfloat16)

    k, v = normal(b, n_kv, Hk, d), normal(b, n_kv, Hk, d)
    position = torch.arange(n_kv).repeat(b, 1)
    weight = torch.zeros(b, n_kv)
    g = {"k": k.cuda(), "v": v.cuda(), "position": position.cuda(), "weight": weight.cuda()}
    lens = torch.tensor([500, 333], dtype=torch.int32)
    kv_len = lens.cuda()
    scale = 1 / math.sqrt(d)

    def compare(n_rows):
        for s in range(b):
            for name, mine in (("k", k), ("v", v), ("position", position)):
                assert torch.equal(g[name][s, :n_rows[s]].cpu(), mine[s, :n_rows[s]]), name
            close(g["weight"][s, :n_rows[s]], weight[s, :n_rows[s]], 2.0**-10 * weight[s, :n_rows[s]].double() + 1e-6,
                  "weight")

    def shrink():
        idx = hs.evict(hs.params(b, 1, n_kv, 128, 128, 4, 64, H, Hk, d), g["weight"], kv_len, budget,
                       [g["k"], g["v"], g["position"]], n_first=4, n_recent=32).cpu()
        for s in range(b):
            rows = idx[s][idx[s] >= 0].long()
            want = torch.tensor(ref.keep(weight[s].numpy(), int(lens[s]), budget, 4, 32))
            # the weights agree to rounding alone, so rows at the border may change places
            assert len(rows) == len(want) and len(set(rows.tolist()) ^ set(want.tolist())) <= 2
            for a in (k, v, position, weight):
                a[s, :len(rows)] = a[s, rows].clone()
            lens[s] = len(rows)
        assert torch.equal(kv_len.cpu(), lens)
        compare(lens.tolist())

    # the window: the prompt's last 64 tokens over the whole prompt
    T = 64
    q = normal(b, T, H, d)
    p = hs.params(b, T, n_kv, 128, 128, 4, 64, H, Hk, d)
    front = kv_len - T
    _, lse = hs.tree_attn(p, q.cuda(), g["k"], g["v"], front)
    hs.hisa_cache_weight(p, q.cuda(), g["k"], front, lse, g["weight"])
    received = ref.tree_attention(q, k, None, lens - T, None, scale)[2]
    weight = ref.weight_after(weight, received, lens - T, T).float()
    compare(lens.tolist())
    shrink()
    for step in range(2):
        T = 12
        q, parent = normal(b, T, H, d), make_parent("tree", b, T, gen)
        fresh_k, fresh_v = normal(b, T, Hk, d), normal(b, T, Hk, d)
        path = torch.full((b, T), -1, dtype=torch.int32)
        for s in range(b):
            L = int(lens[s])
            k[s, L:L + T], v[s, L:L + T] = fresh_k[s], fresh_v[s]
            position[s, L:L + T] = 1000 * (step + 1) + torch.arange(T)
            for name, mine in (("k", k), ("v", v), ("position", position)):
                g[name][s, L:L + T] = mine[s, L:L + T].cuda()
            chain = ref.ancestors(parent[s], T)[T - 1 - 3 * s]
            path[s, :len(chain)] = torch.tensor(chain, dtype=torch.int32)
        p = hs.params(b, T, n_kv, 128, 128, 4, 64, H, Hk, d)
        o, lse = hs.tree_attn(p, q.cuda(), g["k"], g["v"], kv_len, parent=parent.cuda())
        counted = [set(int(i) for i in row if i >= 0) for row in path]
        ro, rl, received, spread, size = ref.tree_attention(q, k, v, lens, parent, scale, counted)
        close(o, ro, 2.0**-8 * ro.abs() + (2 * delta(d, size) + 2.0**-8) * spread, "o")
        hs.hisa_cache_weight(p, q.cuda(), g["k"], kv_len, lse, g["weight"], parent=parent.cuda(), path=path.cuda())
        weight = ref.weight_after(weight, received, lens, T).float()
        rows = torch.where(path >= 0, path + lens[:, None], -1)
        hs.hisa_cache_compact(p, rows.to(torch.int32).cuda(), [g["k"], g["v"], g["position"], g["weight"]],
                              dst_begin=kv_len)
        for s in range(b):
            for a in (k, v, position, weight):
                a[s] = ref.compact(a[s], rows[s], int(lens[s]))[0]
            lens[s] += len(counted[s])
        kv_len.copy_(lens)
        compare(lens.tolist())
    shrink()
