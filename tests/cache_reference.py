"""The cache operators in 64 bits, from their definitions (include/hisa.h), sequence by sequence, on the CPU."""
from __future__ import annotations

import math

import numpy as np
import torch


def ancestors(parent_row, T):
    """Per slot: the slots it sees among the drafted ones (itself included), or None for an empty slot."""
    out = []
    for i in range(T):
        p = i - 1 if parent_row is None else int(parent_row[i])
        if p == -1:
            out.append([i])
        elif 0 <= p < i and out[p] is not None:
            out.append(out[p] + [i])
        else:
            out.append(None)
    return out


def tree_attention(q, k, v, kv_len, parent, scale, counted=None, lse_in=None):
    """o, lse, received [b][n_kv], and what bounds the error of an fp32 evaluation: spread [b][T][H][d] = sum p |v|
    and size = the largest scale * sum |q_c k_c| of a visible pair.  counted: per sequence the slots that count in
    `received`; lse_in replaces the LSE there.  Rows that nothing sees are never read."""
    b, T, H, d = q.shape
    n_kv, Hk = k.shape[1], k.shape[2]
    o = torch.zeros(b, T, H, d, dtype=torch.float64)
    spread = torch.zeros_like(o)
    lse = torch.full((b, T, H), -math.inf, dtype=torch.float64)
    received = torch.zeros(b, n_kv, dtype=torch.float64)
    size = 0.0
    for s in range(b):
        L = int(kv_len[s])
        if L < 0 or L + T > n_kv:
            continue
        for i, anc in enumerate(ancestors(None if parent is None else parent[s], T)):
            if anc is None:
                continue
            rows = torch.cat([torch.arange(L), L + torch.tensor(anc)])
            kk = k[s, rows].double().repeat_interleave(H // Hk, 1)  # [n][H][d]
            z = torch.einsum("hd,nhd->nh", q[s, i].double(), kk) * scale
            size = max(size, float(torch.einsum("hd,nhd->nh", q[s, i].double().abs(), kk.abs()).max()) * scale)
            lse[s, i] = torch.logsumexp(z, 0)
            p = (z - lse[s, i]).exp()
            if v is not None:
                vv = v[s, rows].double().repeat_interleave(H // Hk, 1)
                o[s, i] = torch.einsum("nh,nhd->hd", p, vv)
                spread[s, i] = torch.einsum("nh,nhd->hd", p, vv.abs())
            if counted is None or i in counted[s]:
                if lse_in is not None:
                    fine = lse_in[s, i] != -math.inf
                    p = torch.where(fine, (z - lse_in[s, i].double()).exp(), 0.0)
                received[s, rows] += p.sum(1)
    return o, lse, received, spread, size


def weight_after(weight, received, kv_len, T):
    out = weight.double().clone()
    for s in range(weight.shape[0]):
        L = int(kv_len[s])
        if L < 0 or L + T > weight.shape[1]:
            continue
        out[s, :L] += received[s, :L]
        out[s, L:L + T] = received[s, L:L + T]
    return out


def keep(weight, L, budget, n_first, n_recent):
    """The kept rows of one sequence, ascending."""
    if L <= budget:
        return list(range(L))
    w = np.asarray(weight, dtype=np.float32)[n_first:L - n_recent]
    w = w.astype(np.float64)
    mid = np.lexsort((np.arange(len(w)), -np.where(np.isnan(w), 0.0, w), ~np.isnan(w)))[:budget - n_first - n_recent]
    return list(range(n_first)) + sorted(int(n_first + i) for i in mid) + list(range(L - n_recent, L))


def compact(a, rows, begin):
    """One sequence: (rows of array a [n_kv][...] after the move, whether an entry was skipped as bad)."""
    out, bad, last = a.clone(), begin < 0, -1
    if begin < 0:
        return out, True
    for j, r in enumerate(int(x) for x in rows):
        if r == -1:
            continue
        if not begin + j <= r < a.shape[0]:
            bad = True
            continue
        if r <= last:
            bad = True
            continue
        last = r
        out[begin + j] = a[r]
    return out, bad
