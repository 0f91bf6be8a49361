"""Refusals of the paged-cache entry points, without a GPU: the C layer rejects
bad arguments before it touches the device (the pointers are never
dereferenced), the Python layer before it reaches the C layer."""
import ctypes

import pytest
import torch

import exact_io_aware_online_b200 as fa
from exact_io_aware_online_b200 import _build

A = 0x7f0000010000  # a 16-byte aligned fake device address
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    _build.build()
    return fa.lib()


def cache(**kw):
    a = dict(k_pages=A, v_pages=A, k_scale=A, v_scale=A, page_table=A, seqlens=A, B=3, Hkv=2, d=64, num_pages=10,
             page_size=16, max_pages=4, dtype=fa.FA_CACHE_BF16, table_stride=4)
    a["pages"] = fa._Strides(2 * 16 * 64, 16 * 64, 64)
    a["scales"] = fa._Strides(2 * 16, 16, 1)
    a.update(kw)
    return fa._PagedCache(**a)


def write(L, c, k=A, v=A, st=None, cu=A, T=5, dtype=0, fn="fa_cache_write"):
    st = None if st is None else (fa._Strides * 2)(*[fa._Strides(*s) for s in st])
    return getattr(L, fn)(ctypes.addressof(c) if c is not None else None, k, v,
                          ctypes.addressof(st) if st is not None else None, cu, T, dtype, None)


def attend(L, c, q=A, o=A, lse=A, st=None, H=4, Nq=1, scale=0.125, causal=1, window=-1, ws=A, ws_bytes=None, dtype=0):
    st = None if st is None else (fa._Strides * 2)(*[fa._Strides(*s) for s in st])
    need = max(16, L.fa_fwd_paged_workspace_size(3, 4, 2, 1, 64))
    return L.fa_fwd_paged(ctypes.addressof(c) if c is not None else None, q, o, lse,
                          ctypes.addressof(st) if st is not None else None, H, Nq, ctypes.c_float(scale), causal,
                          window, ws, need if ws_bytes is None else ws_bytes, dtype, None)


def calls(L, c):
    return {"write": write(L, c), "read": write(L, c, fn="fa_cache_read"), "attend": attend(L, c)}


CACHES = [
    (dict(k_pages=None), INVALID), (dict(v_pages=None), INVALID), (dict(page_table=None), INVALID),
    (dict(seqlens=None), INVALID), (dict(B=0), INVALID), (dict(Hkv=0), INVALID), (dict(num_pages=0), INVALID),
    (dict(page_size=0), INVALID), (dict(page_size=-16), INVALID), (dict(max_pages=0), INVALID),
    (dict(table_stride=3), INVALID), (dict(dtype=2), INVALID), (dict(dtype=1, k_scale=None), INVALID),
    (dict(dtype=1, v_scale=None), INVALID), (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED),
    (dict(page_size=1 << 20, max_pages=1 << 11, table_stride=1 << 11, pages=(1 << 31, 1 << 28, 64)), UNSUPPORTED),
    (dict(k_pages=A + 8), MISALIGNED), (dict(v_pages=A + 4), MISALIGNED),
    (dict(pages=(2 * 16 * 64, 16 * 64, 0)), INVALID), (dict(pages=(-2048, 16 * 64, 64)), INVALID),
    (dict(pages=(2 * 16 * 64 + 4, 16 * 64, 64)), MISALIGNED), (dict(pages=(1 << 40, 16 * 64, 64)), INVALID),
    (dict(dtype=1, scales=(2 * 16, 16, 0)), INVALID), (dict(dtype=1, k_scale=A + 2), MISALIGNED),
]


@pytest.mark.parametrize("kw,code", CACHES, ids=[str(i) for i in range(len(CACHES))])
def test_bad_caches_are_refused_by_every_call(L, kw, code):
    kw = {n: fa._Strides(*v) if isinstance(v, tuple) else v for n, v in kw.items()}
    assert calls(L, cache(**kw)) == {"write": code, "read": code, "attend": code}


def test_a_written_cache_must_be_one_to_one(L):
    same = fa._Strides(2 * 16 * 64, 64, 64)                                 # heads over tokens
    assert write(L, cache(pages=same)) == INVALID
    assert write(L, cache(dtype=1, scales=fa._Strides(32, 1, 1))) == INVALID


def test_move_refusals(L):
    for fn in ("fa_cache_write", "fa_cache_read"):
        go = lambda **kw: write(L, cache(), fn=fn, **kw)                    # noqa: E731
        assert write(L, None, fn=fn) == INVALID
        assert go(k=None) == INVALID and go(v=None) == INVALID and go(cu=None) == INVALID
        assert go(T=-1) == INVALID
        assert go(k=A + 8) == MISALIGNED and go(v=A + 2) == MISALIGNED
        assert go(dtype=1) == UNSUPPORTED and go(dtype=5) == INVALID
        assert go(st=[(1, 64, 128), (1, 64, 0)]) == INVALID
        assert go(st=[(1, 64, 132), (1, 64, 128)]) == MISALIGNED
        assert go(T=0) == 0                                                 # nothing to do
        assert go(T=0, k=None, v=None) == 0
    assert write(L, cache(), fn="fa_cache_read", st=[(1, 64, 64), (1, 64, 128)]) == INVALID   # output rows overlap
    assert write(L, cache(), T=1 << 30, st=[(1, 64, 128), (1, 64, 1 << 41)]) == INVALID


def test_attend_refusals(L):
    c = cache()
    assert attend(L, None) == INVALID
    for n in ("q", "o", "lse"):
        assert attend(L, c, **{n: None}) == INVALID
        assert attend(L, c, **{n: A + 8}) == MISALIGNED
    assert attend(L, c, H=3) == INVALID and attend(L, c, H=0) == INVALID and attend(L, c, Nq=0) == INVALID
    assert attend(L, c, scale=0.0) == INVALID and attend(L, c, scale=float("nan")) == INVALID
    assert attend(L, c, window=-2) == INVALID
    assert attend(L, c, dtype=1) == UNSUPPORTED and attend(L, c, dtype=9) == INVALID
    assert attend(L, c, ws=None) == WORKSPACE and attend(L, c, ws_bytes=15) == WORKSPACE
    assert attend(L, c, ws=A + 8) == MISALIGNED
    assert attend(L, c, st=[(256, 64, 68), (256, 64, 64)], Nq=2) == MISALIGNED
    assert attend(L, c, st=[(512, 128, 64), (512, 64, 64)], Nq=2) == INVALID    # output heads over rows
    assert attend(L, c, H=2, Nq=(1 << 31) - 1) == INVALID


def test_scales_out_of_range_are_refused(L):
    for scale in (-1.0, float("inf"), 2.4e38, 3.4e38):                      # the kernels work with scale * log2(e)
        assert attend(L, cache(), scale=scale) == INVALID
        assert attend(L, cache(dtype=1), scale=scale) == INVALID


def test_workspace_size(L):
    assert L.fa_fwd_paged_workspace_size(3, 4, 2, 1, 64) > 0
    for bad in ((0, 4, 2, 1, 64), (3, 5, 2, 1, 64), (3, 4, 2, 0, 64), (3, 4, 2, 1, 96)):
        assert L.fa_fwd_paged_workspace_size(*bad) == 0
    # a bound that does not grow with the batch once every SM has work
    assert L.fa_fwd_paged_workspace_size(1 << 12, 32, 8, 1, 128) == L.fa_fwd_paged_workspace_size(1 << 14, 32, 8, 1, 128)


def host(kind=torch.bfloat16):
    P, Hkv, page, d = 6, 2, 16, 64
    k = torch.zeros((P, Hkv, page, d), dtype=torch.bfloat16).to(kind)
    a = dict(k_pages=k, v_pages=k.clone(), page_table=torch.zeros((3, 2), dtype=torch.int32),
             seqlens=torch.zeros(3, dtype=torch.int32))
    if kind != torch.bfloat16:
        a |= dict(k_scale=torch.zeros((P, Hkv, page)), v_scale=torch.zeros((P, Hkv, page)))
    return a


@pytest.mark.parametrize("kw,err", [
    (dict(k_pages=torch.zeros(6, 2, 16, 64)), TypeError),
    (dict(v_pages=torch.zeros(6, 2, 8, 64, dtype=torch.bfloat16)), ValueError),
    (dict(v_pages=torch.zeros(6, 2, 16, 64)), TypeError),
    (dict(v_pages=torch.zeros(6, 16, 2, 64, dtype=torch.bfloat16).transpose(1, 2)), ValueError),
    (dict(page_table=torch.zeros(3, 2)), TypeError), (dict(seqlens=torch.zeros(3, dtype=torch.int64)), TypeError),
    (dict(seqlens=torch.zeros(2, dtype=torch.int32)), ValueError),
    (dict(page_table=torch.zeros((2, 3), dtype=torch.int32).t()), ValueError),
    (dict(seqlens=torch.zeros(6, dtype=torch.int32)[::2]), ValueError),
    (dict(page_table=torch.zeros((1, 2), dtype=torch.int32).expand(3, 2)), ValueError),
    (dict(k_scale=torch.zeros(6, 2, 16)), ValueError),
])
def test_python_checks_the_cache(kw, err):
    a = host() | kw
    q = torch.zeros((3, 4, 1, 64), dtype=torch.bfloat16)
    x = torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    cu = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(err):
        fa.fwd_paged(q, **a)
    with pytest.raises(err):
        fa.cache_write(x, x, cu_seqlens=cu, **a)
    with pytest.raises(err):
        fa.cache_read(cu_seqlens=cu, num_tokens=5, **a)


def test_python_checks_the_scales():
    a = host(torch.float8_e4m3fn)
    q = torch.zeros((3, 4, 1, 64), dtype=torch.bfloat16)
    for bad in (dict(k_scale=None), dict(v_scale=torch.zeros(6, 2, 8)), dict(k_scale=torch.zeros(6, 2, 16).half()),
                dict(v_scale=torch.zeros(6, 16, 2).transpose(1, 2))):
        with pytest.raises(ValueError):
            fa.fwd_paged(q, **(a | bad))


def test_host_tensors_never_reach_a_kernel():
    q = torch.zeros((3, 4, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fwd_paged(q, **host())


def test_positions_are_counted_with_pages_rounded_up(L):
    wide = dict(max_pages=1 << 28, table_stride=1 << 28)
    assert attend(L, cache(page_size=1, **wide)) == UNSUPPORTED                 # 2^31 places of pages of 8
    many = dict(page_size=1 << 20, max_pages=1 << 10, table_stride=1 << 10, B=1 << 20)
    many["pages"] = fa._Strides(1 << 28, 1 << 27, 64)
    assert attend(L, cache(**many), ws_bytes=1 << 40) == UNSUPPORTED            # 2^50 tokens in all


def test_more_rows_than_the_move_counts(L):
    for fn in ("fa_cache_write", "fa_cache_read"):
        assert write(L, cache(Hkv=2), T=(1 << 29), fn=fn) == UNSUPPORTED
