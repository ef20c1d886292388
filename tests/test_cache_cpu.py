"""The cache operators without a GPU: what the library and the binding refuse before anything is launched."""
import ctypes

import pytest
import torch

import hierarchical_sparse_attention_block_b200 as hs
from cache_reference import ancestors, compact, keep

A = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4104)  # not 16-byte aligned
BAD, UNSUP, WS = hs.HISA_ERR_INVALID_ARG, hs.HISA_ERR_UNSUPPORTED, hs.HISA_ERR_WORKSPACE


def _p(**kw):
    base = dict(batch=2, n_q=8, n_kv=512, d_idx=128, block=128, top_m=4, top_k=64, n_heads=8, n_kv_heads=2, d_head=128)
    return hs.params(**{**base, **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(n_q=257), UNSUP), (dict(n_q=513), BAD), (dict(n_q=0), BAD), (dict(n_heads=3), BAD),
    (dict(n_heads=2048), UNSUP), (dict(d_head=96), UNSUP), (dict(d_head=0), BAD), (dict(batch=0), BAD),
    (dict(scale=float("inf")), BAD), (dict(scale=float("nan")), BAD), (dict(n_kv=1 << 31), BAD),
])
def test_shapes_are_validated(kw, code):
    n = ctypes.c_size_t(0)
    p = _p(**kw)
    assert hs.lib().hisa_tree_attn_workspace_size(ctypes.byref(p), 0, ctypes.byref(n)) == code
    assert hs.lib().hisa_cache_weight_workspace_size(ctypes.byref(p), ctypes.byref(n)) == code


def test_workspace_queries_refuse_bad_arguments():
    n, p, lib = ctypes.c_size_t(0), _p(), hs.lib()
    assert lib.hisa_tree_attn_workspace_size(ctypes.byref(p), 2, ctypes.byref(n)) == BAD
    assert lib.hisa_tree_attn_workspace_size(ctypes.byref(p), 0, None) == BAD
    assert lib.hisa_tree_attn_workspace_size(None, 0, ctypes.byref(n)) == BAD
    assert lib.hisa_cache_weight_workspace_size(ctypes.byref(p), None) == BAD
    assert lib.hisa_cache_keep_workspace_size(ctypes.byref(p), None) == BAD
    assert hs.hisa_tree_attn_workspace_size(p, True) >= hs.hisa_tree_attn_workspace_size(p, False)


def test_tree_attn_pointers():
    lib, p = hs.lib(), _p()
    need = hs.hisa_tree_attn_workspace_size(p, True)

    def call(q=A, k=A, v=A, kv_len=A, parent=A, o=A, lse=A, weight=A, ws=A, n=need):
        return lib.hisa_tree_attn_fwd(ctypes.byref(p), q, k, v, kv_len, parent, o, lse, weight, None, ws, n, None)

    for name in ("q", "k", "v", "kv_len", "o"):
        assert call(**{name: None}) == BAD, name
    for name in ("q", "k", "v", "kv_len", "parent", "o", "lse", "weight"):
        assert call(**{name: ODD}) == BAD, name
    assert need > 0
    for kw in (dict(n=need - 1), dict(ws=None), dict(ws=ODD)):
        assert call(**kw) == WS


def test_cache_weight_pointers():
    lib, p = hs.lib(), _p()
    need = hs.hisa_cache_weight_workspace_size(p)

    def call(q=A, k=A, kv_len=A, parent=A, path=A, lse=A, weight=A, ws=A, n=need):
        return lib.hisa_cache_weight(ctypes.byref(p), q, k, kv_len, parent, path, lse, weight, None, ws, n, None)

    for name in ("q", "k", "kv_len", "lse", "weight"):
        assert call(**{name: None}) == BAD, name
    for name in ("q", "k", "kv_len", "parent", "path", "lse", "weight"):
        assert call(**{name: ODD}) == BAD, name
    if need:
        for kw in (dict(n=need - 1), dict(ws=None), dict(ws=ODD)):
            assert call(**kw) == WS


def test_cache_keep_arguments():
    lib, p = hs.lib(), _p()
    need = hs.hisa_cache_keep_workspace_size(p)

    def call(weight=A, kv_len=A, keep_idx=A, kept_len=A, budget=64, first=4, recent=8, ws=A, n=need):
        return lib.hisa_cache_keep(ctypes.byref(p), weight, kv_len, budget, first, recent, keep_idx, kept_len, None, ws,
                                   n, None)

    for name in ("weight", "kv_len", "keep_idx", "kept_len"):
        assert call(**{name: None}) == BAD and call(**{name: ODD}) == BAD, name
    for kw in (dict(budget=0), dict(budget=513), dict(first=-1), dict(recent=-1), dict(first=60, recent=5),
               dict(first=2**31 - 1, recent=2**31 - 1)):
        assert call(**kw) == BAD, kw
    if need:
        for kw in (dict(n=need - 1), dict(ws=None), dict(ws=ODD)):
            assert call(**kw) == WS


def test_cache_compact_arguments():
    lib, p = hs.lib(), _p()

    def call(rows=A, n=16, begin=A, arrays=((4096, 256),), count=None):
        c = (hs.HisaRows * max(1, len(arrays)))(*[hs.HisaRows(b, r) for b, r in arrays])
        return lib.hisa_cache_compact(ctypes.byref(p), rows, n, begin, c, len(arrays) if count is None else count, None,
                                      None)

    assert call(rows=None) == BAD and call(rows=ODD) == BAD and call(begin=ODD) == BAD
    assert call(n=0) == BAD and call(n=513) == BAD
    assert call(count=0) == BAD and call(arrays=((4096, 4),) * 9) == BAD
    for a in ((None, 256), (4104, 256), (4096, 0), (4096, 6), (4096, -4), (4096, (1 << 24) + 4)):
        assert call(arrays=((4096, 256), a)) == BAD, a
    assert lib.hisa_cache_compact(ctypes.byref(p), A, 16, None, None, 1, None, None) == BAD


@pytest.mark.parametrize("batch,n_kv,other", [
    (2, 512, (4096, 256)),                     # the same array twice
    (2, 512, (4096 + 2 * 512 * 256 - 16, 4)),  # begins in the last row
    (2, 512, (4096 - 16, 4)),                  # ends in the first row
    (65535, (1 << 31) - 1, (1 << 62, 4)),      # the size in bytes passes 64 bits with rows this long
])
def test_arrays_that_share_bytes_are_refused(batch, n_kv, other):
    p = _p(batch=batch, n_kv=n_kv)
    row = 256 if batch == 2 else 1 << 24
    for pair in (((4096, row), other), (other, (4096, row))):
        c = (hs.HisaRows * 2)(*[hs.HisaRows(*a) for a in pair])
        assert hs.lib().hisa_cache_compact(ctypes.byref(p), A, 16, None, c, 2, None, None) == BAD


class _OnGpu:
    """A stand-in for a CUDA tensor: what the binding looks at before it calls the library."""

    def __init__(self, shape, dtype, contiguous=True, device="cuda:0"):
        self.shape, self.dtype, self.device, self.is_cuda = torch.Size(shape), dtype, torch.device(device), True
        self._c = contiguous

    def get_device(self):
        return self.device.index

    def is_contiguous(self):
        return self._c

    def stride(self):
        return ()

    def data_ptr(self):
        return 4096

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)


def test_binding_refuses_other_types_shapes_layouts_and_devices():
    p = _p()
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    q, k, n = ((2, 8, 8, 128), bf), ((2, 512, 2, 128), bf), ((2,), i32)
    good = dict(q=q, k=k, v=k, kv_len=n, o=q, lse=((2, 8, 8), f32), parent=((2, 8), i32), weight=((2, 512), f32))

    def call(**other):
        a = {name: _OnGpu(*spec) for name, spec in good.items()}
        a.update({name: _OnGpu(*x) if isinstance(x, tuple) else x for name, x in other.items()})
        hs.hisa_tree_attn_fwd(p, **a)

    cases = [dict(q=((2, 8, 8, 64), bf)), dict(k=((2, 512, 2, 128), f32)), dict(v=((2, 512, 2, 128), bf, False)),
             dict(kv_len=((2,), torch.int64)), dict(parent=((2, 9), i32)), dict(lse=((2, 8, 8), f32, True, "cuda:1")),
             dict(weight=((2, 513), f32)), dict(q=torch.zeros(2, 8, 8, 128, dtype=bf)),
             dict(dev_status=((2,), i32), workspace=((64,), torch.uint8)),
             dict(workspace=((64,), torch.int32)), dict(workspace=((64,), torch.uint8, True, "cuda:1"))]
    for c in cases:
        with pytest.raises(hs.HisaError) as err:
            call(**c)
        assert err.value.status == BAD, c
    rows = _OnGpu((2, 16), i32)
    for arrays in ([], [_OnGpu((2, 512, 4), f32)] * 9, [_OnGpu((2, 511, 4), f32)], [_OnGpu((2,), f32)],
                   [_OnGpu((2, 512, 4), f32, False)], [torch.zeros(2, 512)]):
        with pytest.raises(hs.HisaError) as err:
            hs.hisa_cache_compact(p, rows, arrays)
        assert err.value.status == BAD
    with pytest.raises(hs.HisaError):
        hs.hisa_cache_keep(p, _OnGpu((2, 512), f32), _OnGpu((2,), i32), 64, _OnGpu((2, 65), i32), _OnGpu((2,), i32))
    with pytest.raises(hs.HisaError):
        hs.hisa_cache_weight(p, _OnGpu(*q), _OnGpu(*k), _OnGpu(*n), _OnGpu((2, 8, 8), f32), _OnGpu((2, 512), f32),
                             path=_OnGpu((2, 4), i32))


def test_the_reference_itself():
    """Hand-worked cases of the definitions that the GPU tests compare with."""
    assert ancestors(None, 3) == [[0], [0, 1], [0, 1, 2]]
    assert ancestors([-1, 0, 0, -2, 3, 5, 1], 7) == [[0], [0, 1], [0, 2], None, None, None, [0, 1, 6]]
    assert keep([5, 1, 9, 9, 2, 0], 6, 4, 1, 1) == [0, 2, 3, 5]
    assert keep([5, 1, 9, 9, 2, 0], 6, 3, 1, 1) == [0, 2, 5]
    assert keep([0.0, -0.0, 0.0], 3, 2, 0, 0) == [0, 1]
    assert keep([1.0, float("nan"), float("inf")], 3, 1, 0, 0) == [1]
    a = torch.arange(6)
    assert compact(a, [1, 3, 4, -1], 0)[0].tolist() == [1, 3, 4, 3, 4, 5]
    out, bad = compact(a, [2, 1, 9, 3, 5], 0)  # 1 is not ascending, 9 is out of range, 3 moves nowhere new
    assert out.tolist() == [2, 1, 2, 3, 5, 5] and bad
