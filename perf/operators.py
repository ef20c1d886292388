"""The cache operators as they are measured: attention of drafted tokens over a KV cache, the attention weight each
cached row has received, the choice of the rows to keep, and the move of the kept rows.

`own` picks between the operators' plain forms (elementary torch operations) and the calls of this package.

Layouts: q [b][T][H][d], k and v [b][n_kv][Hk][d] (bf16), kv_len [b] int32 (context rows; drafted token i's row is
kv_len + i), parent [b][T] int32 (-1: child of the context, -2: empty slot), weight [b][n_kv] fp32.
"""
import math

import numpy as np
import torch

own = False

# Rows a tree's slots may hang back from the newest slot: a drafter that expands a few nodes per level.
_SPAN = 4


def _case(op, name=None, **kw):
    c = {"op": op, **kw}
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # One request with a short cache and a small tree: what counts is the latency of the call.
        _case("tree", "tree_1x1k", b=1, T=16, H=8, Hk=8, d=128, ctx=1000, chain=False, weigh=False),
        # A serving batch with shared KV heads and caches of different lengths.
        _case("tree", "tree_16x32k_gqa4", b=16, T=32, H=16, Hk=4, d=128, ctx=32768, chain=False, weigh=False),
        # Long caches and a wide tree on few KV heads: many query rows for each K/V row.
        _case("tree", "tree_4x128k_gqa8", b=4, T=64, H=16, Hk=2, d=128, ctx=131072, chain=False, weigh=False),
        # The last tokens of a prompt as a chain (the window whose weights decide an eviction), odd sizes, d = 64.
        _case("tree", "window_3x5k_d64", b=3, T=200, H=12, Hk=4, d=64, ctx=5003, chain=True, weigh=False),
        # One token per sequence, every head with its own K/V, the weights accumulated by the same call.
        _case("tree", "decode_8x64k_weighed", b=8, T=1, H=16, Hk=16, d=128, ctx=65536, chain=True, weigh=True),
        # One token of one short request: the weight call's latency.
        _case("weight", "weight_1x777_d64", b=1, T=1, H=8, Hk=2, d=64, ctx=777, chain=True, accept=0),
        # After a tree's verification: the accepted tokens of each sequence alone count.
        _case("weight", "weight_16x32k_accepted", b=16, T=32, H=16, Hk=4, d=128, ctx=32768, chain=False, accept=1),
        # A prompt's window of 128 queries over the whole prompt.
        _case("weight", "weight_2x16k_window", b=2, T=128, H=16, Hk=16, d=128, ctx=16384, chain=True, accept=0),
        # The choice of the kept rows for a decode batch.
        _case("keep", "keep_32x128k", b=32, n_kv=131072, budget=16384, first=4, recent=1024, ties=False),
        # Two long caches of odd length whose weights hold many equal values.
        _case("keep", "keep_2x1m_ties", b=2, n_kv=1000003, budget=65537, first=128, recent=4096, ties=True),
        # An eviction's move of K, V, the indexer keys and the weights to the front, in place.
        _case("compact", "evict_8x32k_to_8k", b=8, n_kv=32768, Hk=8, d=128, d_idx=128, n=8192, commit=False),
        # The accepted tokens of a step move to the end of the context.
        _case("compact", "commit_64x16", b=64, n_kv=4096, Hk=4, d=128, d_idx=128, n=16, commit=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "weight", "weight", "keep", "compact"])
    if op in ("tree", "weight"):
        d = rng.choice([64, 128, 128])
        Hk = rng.choice([1, 2, 4, 8, 16])
        H = Hk * rng.choice([1, 1, 2, 3, 4, 8])
        chain = rng.random() < 0.4
        T = _log(rng, 1, 256) if chain else _log(rng, 2, 96)
        b = _log(rng, 1, 32)
        # at most 2 GB of K and V, 1.5e11 operations and 2e8 scores
        most = min(2e9 / (b * Hk * d * 4), 1.5e11 / (4.0 * b * H * T * d), 2e8 / (b * H * T), 131072)
        ctx = _log(rng, 1, max(2, int(most)))
        if op == "tree":
            return _case("tree", b=b, T=T, H=H, Hk=Hk, d=d, ctx=ctx, chain=chain, weigh=rng.random() < 0.35)
        return _case("weight", b=b, T=T, H=H, Hk=Hk, d=d, ctx=ctx, chain=chain, accept=int(not chain and rng.random() < 0.7))
    if op == "keep":
        b = _log(rng, 1, 64)
        n_kv = _log(rng, 1, 8000000 // b)
        budget = _log(rng, 1, n_kv)
        first = rng.randint(0, min(128, budget))
        return _case("keep", b=b, n_kv=n_kv, budget=budget, first=first, recent=rng.randint(0, (budget - first) // 2),
                     ties=rng.random() < 0.5)
    Hk = rng.choice([1, 2, 4, 8, 16])
    d = rng.choice([64, 128])
    b = _log(rng, 1, 64)
    commit = rng.random() < 0.4
    n_kv = _log(rng, 64, max(65, min(262144, int(1e9 / (b * Hk * d * 4)))))
    n = rng.randint(1, min(64, n_kv)) if commit else _log(rng, 1, n_kv)
    return _case("compact", b=b, n_kv=n_kv, Hk=Hk, d=d, d_idx=rng.choice([64, 128, 256]), n=n, commit=commit)


# ------------------------------------------------------------------ inputs


def _lengths(b, top):
    """Lengths of b caches, the longest `top`: evenly between a quarter of it and all of it."""
    return [max(0, top - (3 * top * i) // (4 * b)) for i in range(b)]


def _order(values, gen):
    return torch.tensor(values, dtype=torch.int32)[torch.randperm(len(values), generator=gen)]


def _trees(b, T, gen):
    """parent [b][T]: every slot hangs from one of the _SPAN slots before it or from the context; the slots behind a
    sequence's own number of drafted tokens (at least half of T) are empty."""
    at = torch.arange(T, dtype=torch.int32)
    back = torch.randint(1, _SPAN + 1, (b, T), generator=gen, dtype=torch.int32)
    parent = (at[None] - back).clamp_min(-1)
    count = torch.randint((T + 1) // 2, T + 1, (b, 1), generator=gen, dtype=torch.int32)
    return torch.where(at[None] < count, parent, torch.full_like(parent, -2)), count[:, 0]


def _accepted(parent, count):
    """path [b][T]: the chain from the context to each sequence's last drafted token, ascending, -1 padded."""
    path = torch.full_like(parent, -1)
    for s in range(parent.shape[0]):
        chain, i = [], int(count[s]) - 1
        while i >= 0:
            chain.append(i)
            i = int(parent[s, i])
        path[s, :len(chain)] = torch.tensor(chain[::-1], dtype=torch.int32)
    return path


def prepare(case, seed):
    gen = torch.Generator().manual_seed(seed)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    b, op = case["b"], case["op"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.bfloat16)

    def spread(*shape):  # accumulated weights: most rows little, a few much
        return torch.randn(shape, generator=g, device=dev).mul_(2.0).exp_()

    if op in ("tree", "weight"):
        T, H, Hk, d = case["T"], case["H"], case["Hk"], case["d"]
        n_kv = case["ctx"] + T
        st = {"case": case, "q": normal(b, T, H, d), "k": normal(b, n_kv, Hk, d),
              "kv_len": _order(_lengths(b, case["ctx"]), gen).to(dev), "parent": None, "path": None, "weight": None}
        if op == "tree":
            st["v"] = normal(b, n_kv, Hk, d)
        if not case["chain"]:
            parent, count = _trees(b, T, gen)
            st["parent"] = parent.to(dev)
            if op == "weight" and case["accept"]:
                st["path"] = _accepted(parent, count).to(dev)
        if op == "weight" or case["weigh"]:
            st["weight"] = spread(b, n_kv) * (0.1 * H / case["ctx"])  # what a few earlier steps gave
        if op == "weight":
            # scores of unit variance: the log of the sum over L rows is about ln L + 1/2
            lse = (st["kv_len"].float() + 1).log()[:, None, None] + 0.5
            st["lse"] = lse + 0.1 * torch.randn(b, T, H, generator=g, device=dev)
        return st
    n_kv = case["n_kv"]
    if op == "keep":
        w = spread(b, n_kv)
        if case["ties"]:
            w = (w * 64).round_() / 64
        return {"case": case, "weight": w, "kv_len": _order(_lengths(b, n_kv), gen).to(dev)}
    n = case["n"]
    # The rows to move, ascending: an eviction keeps rows of the whole cache, a commit takes drafted rows behind the
    # context; every third sequence has a shorter list.
    base = _order([max(0, x - n) for x in _lengths(b, n_kv)], gen).to(dev) if case["commit"] else None
    width = 64 if case["commit"] else n_kv
    pick = torch.rand(b, min(width, n_kv), generator=g, device=dev).argsort(1)[:, :n].sort(1).values.to(torch.int32)
    if base is not None:
        room = torch.arange(n, dtype=torch.int32, device=dev) + (n_kv - n - base)[:, None]
        pick = torch.minimum(pick, room) + base[:, None]
    cut = torch.where(torch.arange(b, device=dev) % 3 == 2, (n + 1) // 2, n)
    rows = torch.where(torch.arange(n, device=dev)[None] < cut[:, None], pick, -1).to(torch.int32)
    return {"case": case, "rows": rows, "base": base, "k": normal(b, n_kv, case["Hk"], case["d"]),
            "v": normal(b, n_kv, case["Hk"], case["d"]), "k_idx": normal(b, n_kv, case["d_idx"]), "weight": spread(b, n_kv)}


# ------------------------------------------------------------------ plain forms


def _seen(kv_len, parent, T, n_kv):
    """[b][T][n_kv]: whether drafted token i sees row t."""
    b, dev = kv_len.shape[0], kv_len.device
    at = torch.arange(T, device=dev)
    if parent is None:
        up = (at[:, None] >= at[None]).expand(b, T, T)
        token = torch.ones(b, T, dtype=torch.bool, device=dev)
    else:
        # reach[i][j]: j is i or one of its ancestors (column T: the context, -1), by repeated squaring
        ok = (parent >= -1) & (parent < at)
        up_to = torch.where(ok, torch.where(parent < 0, T, parent), at).long()
        step = torch.zeros(b, T + 1, T + 1, device=dev)
        step[:, :T].scatter_(2, up_to[..., None], 1.0)
        reach = (step + torch.eye(T + 1, device=dev)).clamp_(max=1)
        for _ in range(max(1, math.ceil(math.log2(T + 1)))):
            reach = (reach @ reach).clamp_(max=1)
        token = reach[:, :T, T] > 0
        up = reach[:, :T, :T] > 0
    col = torch.arange(n_kv, device=dev)[None] - kv_len[:, None]
    draft = up.gather(2, col.clamp(0, T - 1)[:, None].expand(b, T, n_kv)) & ((col >= 0) & (col < T))[:, None]
    return ((col < 0)[:, None] | draft) & token[..., None]


def _scores(q, k):
    """[b][Hk][G][T][n_kv] scaled scores in 32 bits."""
    b, T, H, d = q.shape
    Hk = k.shape[2]
    qf = q.float().view(b, T, Hk, H // Hk, d).permute(0, 2, 3, 1, 4).reshape(b, Hk, -1, d)
    return (qf @ k.float().permute(0, 2, 3, 1)).view(b, Hk, H // Hk, T, k.shape[1]) / math.sqrt(d)


def _weigh(weight, received, kv_len, T):
    """weight += received on the context's rows, = received on the drafted rows."""
    col = torch.arange(weight.shape[1], device=weight.device)[None] - kv_len[:, None]
    weight.copy_(torch.where(col < 0, weight + received, torch.where(col < T, received, weight)))
    return weight


def _tree(st):
    q, k, v = st["q"], st["k"], st["v"]
    b, T, H, d = q.shape
    seen = _seen(st["kv_len"], st["parent"], T, k.shape[1])[:, None, None]
    z = _scores(q, k).masked_fill_(~seen, -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = z.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total > 0, total, 1.0)
    o = p.view(b, k.shape[2], -1, k.shape[1]) @ v.float().transpose(1, 2)
    o = o.view(b, k.shape[2], H // k.shape[2], T, d).permute(0, 3, 1, 2, 4).reshape(b, T, H, d).to(torch.bfloat16)
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(b, T, H)
    out = {"o": o, "lse": lse}
    if st["weight"] is not None:
        out["weight"] = _weigh(st["weight"], p.sum((1, 2, 3)), st["kv_len"], T)
    return out


def _weight(st):
    q, k, lse = st["q"], st["k"], st["lse"]
    b, T, H, d = q.shape
    seen = _seen(st["kv_len"], st["parent"], T, k.shape[1])
    if st["path"] is not None:
        hit = (st["path"][:, None] == torch.arange(T, device=q.device)[None, :, None]).any(-1)
        seen = seen & hit[..., None]
    z = _scores(q, k)
    z = z.sub_(lse.permute(0, 2, 1).reshape(b, k.shape[2], -1, T, 1)).masked_fill_(~seen[:, None, None], -math.inf)
    return {"weight": _weigh(st["weight"], z.exp_().sum((1, 2, 3)), st["kv_len"], T)}


def _keep(st):
    w, kv_len, case = st["weight"], st["kv_len"][:, None], st["case"]
    budget = case["budget"]
    at = torch.arange(w.shape[1], device=w.device)[None]
    score = torch.where((at < case["first"]) | (at >= kv_len - case["recent"]), math.inf, w)
    score = torch.where(at < kv_len, score, -math.inf)
    best = score.sort(dim=1, descending=True, stable=True).indices[:, :budget]
    best = torch.where(best < kv_len, best, w.shape[1]).sort(1).values
    kept = st["kv_len"].clamp(max=budget)
    keep = torch.where(torch.arange(budget, device=w.device)[None] < kept[:, None], best, -1).to(torch.int32)
    return {"keep_idx": keep, "kept_len": kept}


def _compact(st):
    rows, n_kv = st["rows"], st["case"]["n_kv"]
    b, n = rows.shape
    to = torch.arange(n, device=rows.device)[None] + (0 if st["base"] is None else st["base"][:, None])
    s = torch.arange(b, device=rows.device)[:, None].expand(b, n)
    ok = rows >= 0
    s, to, src = s[ok], to.expand(b, n)[ok].long(), rows[ok].long()
    out = {}
    for name in ("k", "v", "k_idx", "weight"):
        a = st[name]
        a[s, to] = a[s, src]
        out[name] = a
    return out


# ------------------------------------------------------------------ this package's calls


def _own(st):
    import hierarchical_sparse_attention_block_b200 as hs

    case = st["case"]
    op = case["op"]
    if op in ("tree", "weight"):
        q, k = st["q"], st["k"]
        b, T, H, d = q.shape
        if "p" not in st:
            st["p"] = hs.params(b, T, k.shape[1], 128, 128, 16, 512, H, k.shape[2], d)
            n = (hs.hisa_tree_attn_workspace_size(st["p"], with_weight=case["weigh"]) if op == "tree"
                 else hs.hisa_cache_weight_workspace_size(st["p"]))
            st["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)
        if op == "weight":
            hs.hisa_cache_weight(st["p"], q, k, st["kv_len"], st["lse"], st["weight"], parent=st["parent"],
                                 path=st["path"], workspace=st["ws"])
            return {"weight": st["weight"]}
        o, lse = torch.empty_like(q), torch.empty(b, T, H, device=q.device)
        hs.hisa_tree_attn_fwd(st["p"], q, k, st["v"], st["kv_len"], o, lse, parent=st["parent"], weight=st["weight"],
                              workspace=st["ws"])
        return {"o": o, "lse": lse} if st["weight"] is None else {"o": o, "lse": lse, "weight": st["weight"]}
    if op == "keep":
        w = st["weight"]
        b, budget = w.shape[0], case["budget"]
        if "p" not in st:
            st["p"] = hs.params(b, 1, w.shape[1], 128, 128, 16, 512, 1, 1, 128)
            st["ws"] = torch.empty(max(hs.hisa_cache_keep_workspace_size(st["p"]), 16), dtype=torch.uint8, device=w.device)
        keep = torch.empty(b, budget, dtype=torch.int32, device=w.device)
        kept = torch.empty(b, dtype=torch.int32, device=w.device)
        hs.hisa_cache_keep(st["p"], w, st["kv_len"], budget, keep, kept, n_first=case["first"],
                           n_recent=case["recent"], workspace=st["ws"])
        return {"keep_idx": keep, "kept_len": kept}
    if "p" not in st:
        st["p"] = hs.params(case["b"], 1, case["n_kv"], case["d_idx"], 128, 16, 512, case["Hk"], case["Hk"], case["d"])
    names = ("k", "v", "k_idx", "weight")
    hs.hisa_cache_compact(st["p"], st["rows"], [st[n] for n in names], dst_begin=st["base"])
    return {n: st[n] for n in names}


def run(state):
    if own:
        return _own(state)
    return {"tree": _tree, "weight": _weight, "keep": _keep, "compact": _compact}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without


def work(case):
    b, op = case["b"], case["op"]
    if op in ("tree", "weight"):
        T, H, Hk, d = case["T"], case["H"], case["Hk"], case["d"]
        rows = sum(_lengths(b, case["ctx"])) + b * T
        if op == "tree":
            io = b * T * H * (4 * d + 4) + (8 * rows if case["weigh"] else 0)
            return {"bytes": rows * Hk * d * 4 + io, "flops": 4 * rows * H * T * d}
        n = T if not case["accept"] else max(1, T // (2 * _SPAN))  # accepted tokens: at least the shallowest tree's
        return {"bytes": rows * Hk * d * 2 + b * n * H * (2 * d + 4) + 8 * rows, "flops": 2 * rows * H * n * d}
    if op == "keep":
        rows = sum(_lengths(b, case["n_kv"]))
        return {"bytes": 4 * rows + 4 * b * case["budget"], "flops": rows}
    full, half = b - (b // 3), b // 3
    moved = full * case["n"] + half * ((case["n"] + 1) // 2)
    return {"bytes": moved * 2 * (case["Hk"] * case["d"] * 4 + case["d_idx"] * 2 + 4) + 4 * b * case["n"], "flops": 0}


# ------------------------------------------------------------------ the definition in 64 bits


def exact(case, seed):
    op = case["op"]
    st = prepare(case, seed)
    if op == "compact":
        names = ("k", "v", "k_idx", "weight")
        for s in range(case["b"]):
            rows = st["rows"][s]
            rows = rows[rows >= 0].long()
            at = 0 if st["base"] is None else int(st["base"][s])
            for n in names:
                st[n][s, at:at + len(rows)] = st[n][s].index_select(0, rows)
        return {n: st[n] for n in names}
    if op == "keep":
        lists = np.full((case["b"], case["budget"]), -1, dtype=np.int32)
        kept = np.zeros(case["b"], dtype=np.int32)
        for s, L in enumerate(st["kv_len"].tolist()):
            keep = np.arange(L)
            if L > case["budget"]:
                keep = keep[case["first"]:L - case["recent"]]
                w = st["weight"][s, case["first"]:L - case["recent"]].double().cpu().numpy()
                keep = keep[np.lexsort((keep, -w))][:case["budget"] - case["first"] - case["recent"]]
                keep = np.concatenate([np.arange(case["first"]), np.sort(keep), np.arange(L - case["recent"], L)])
            kept[s] = len(keep)
            lists[s, :len(keep)] = keep
        return {"keep_idx": torch.from_numpy(lists).to(st["weight"].device),
                "kept_len": torch.from_numpy(kept).to(st["weight"].device)}
    q, k = st["q"], st["k"]
    b, T, H, d = q.shape
    Hk, n_kv = k.shape[2], k.shape[1]
    G = H // Hk
    o = torch.zeros(b, T, H, d, dtype=torch.float64, device=q.device)
    lse = torch.full((b, T, H), -math.inf, dtype=torch.float64, device=q.device)
    weight = None if st["weight"] is None else st["weight"].double()
    lens = st["kv_len"].tolist()
    parents = None if st["parent"] is None else st["parent"].tolist()
    paths = None if st["path"] is None else st["path"].tolist()
    for s in range(b):
        L = lens[s]
        sees = torch.zeros(T, L + T, dtype=torch.bool)
        for i in range(T):
            line, j = [], i
            while j >= 0:
                line.append(j)
                j = j - 1 if parents is None else parents[s][j]
            if j == -1:
                sees[i, :L] = True
                sees[i, [L + x for x in line]] = True
        counted = torch.ones(T, dtype=torch.bool)
        if paths is not None:
            counted = torch.zeros(T, dtype=torch.bool)
            counted[[x for x in paths[s] if x >= 0]] = True
        sees, counted = sees.to(q.device), counted.to(q.device)
        received = torch.zeros(L + T, dtype=torch.float64, device=q.device)
        for h in range(H):
            z = q[s, :, h].double() @ k[s, :L + T, h // G].double().T
            z = torch.where(sees, z * (1.0 / math.sqrt(d)), -math.inf)
            if op == "tree":
                lse[s, :, h] = torch.logsumexp(z, 1)
                p = torch.where(sees, (z - lse[s, :, h, None]).exp(), 0.0)
                o[s, :, h] = p @ st["v"][s, :L + T, h // G].double()
            else:
                p = torch.where(sees & counted[:, None], (z - st["lse"][s, :, h, None].double()).exp(), 0.0)
            received += p.sum(0)
        if weight is not None:
            weight[s, :L] += received[:L]
            weight[s, L:L + T] = received[L:]
    if op == "weight":
        return {"weight": weight}
    return {"o": o, "lse": lse} if weight is None else {"o": o, "lse": lse, "weight": weight}
