"""Host-side argument checks of the text side's attention (no GPU): every
refusal comes back before anything is launched, so made-up addresses do."""
import ctypes

import numpy as np
import pytest
import torch

from vision_language_model_b200 import vlm

A, B, C, E = 1 << 20, 2 << 20, 3 << 20, 4 << 20  # 256-byte aligned addresses nobody reads
STATUS = 5 << 20


@pytest.fixture(scope="module")
def L():
    return vlm.lib()


def _prompt(L, dtype=vlm.DTYPE_BF16, heads=8, kv_heads=2, dim=128, q_lens=(5,), kv_lens=(5,), q=A, qs=None, k=B, ks=None,
            v=C, vs=None, scale=0.1, out=E, os_=None, n=None):
    n = len(q_lens) if n is None else n
    arr = ctypes.c_int32 * max(1, len(q_lens))
    w, kw = heads * dim, kv_heads * dim
    return L.vlm_prompt_attention(dtype, heads, kv_heads, dim, arr(*q_lens) if q_lens else None,
                                  arr(*kv_lens) if kv_lens else None, n, q, w if qs is None else qs, k,
                                  kw if ks is None else ks, v, kw if vs is None else vs, scale, out,
                                  w if os_ is None else os_, STATUS, None)


@pytest.mark.parametrize("rc,kw", [
    (vlm.ERR_UNSUPPORTED, dict(dtype=vlm.DTYPE_F32)),
    (vlm.ERR_UNSUPPORTED, dict(dtype=7)),
    (vlm.ERR_UNSUPPORTED, dict(dim=96)),
    (vlm.ERR_UNSUPPORTED, dict(heads=9)),              # not a multiple of kv_heads
    (vlm.ERR_UNSUPPORTED, dict(heads=258, kv_heads=2)),  # 129 query heads on a key head
    (vlm.ERR_INVALID_ARG, dict(heads=0)),
    (vlm.ERR_INVALID_ARG, dict(kv_heads=0)),
    (vlm.ERR_INVALID_ARG, dict(n=0)),
    (vlm.ERR_INVALID_ARG, dict(q=0)),
    (vlm.ERR_INVALID_ARG, dict(k=None)),
    (vlm.ERR_INVALID_ARG, dict(v=C + 8)),              # misaligned
    (vlm.ERR_INVALID_ARG, dict(out=E + 2)),
    (vlm.ERR_INVALID_ARG, dict(scale=0.0)),
    (vlm.ERR_INVALID_ARG, dict(scale=float("nan"))),
    (vlm.ERR_INVALID_ARG, dict(scale=float("inf"))),
    (vlm.ERR_BAD_SHAPE, dict(q_lens=(5, -1), kv_lens=(5, 1))),
    (vlm.ERR_BAD_SHAPE, dict(kv_lens=(-1,))),
    (vlm.ERR_BAD_SHAPE, dict(q_lens=(2 ** 31 - 1, 2 ** 31 - 1), kv_lens=(1, 1))),
    (vlm.ERR_BAD_SHAPE, dict(qs=8 * 128 - 8)),         # rows overlap
    (vlm.ERR_UNSUPPORTED, dict(qs=8 * 128 + 4)),       # not a multiple of 16 bytes
    (vlm.ERR_BAD_SHAPE, dict(ks=0)),
    (vlm.ERR_BAD_SHAPE, dict(os_=64)),
    (vlm.OK, dict(q_lens=(0, 0), kv_lens=(0, 9))),     # nothing to do, nothing launched
])
def test_prompt_attention_arguments(L, rc, kw):
    before = vlm.launch_count()
    assert _prompt(L, **kw) == rc
    assert vlm.launch_count() == before


def _cache(n_pages=10, kv_heads=2, dim=128, k_sg=0.01, v_sg=0.01, pages=A):
    return vlm.Kv4CacheDesc(pages, n_pages, kv_heads, dim, k_sg, v_sg)


BAD_CACHES = [
    (vlm.ERR_INVALID_ARG, dict(pages=None)), (vlm.ERR_INVALID_ARG, dict(pages=A + 8)),
    (vlm.ERR_INVALID_ARG, dict(k_sg=0.0)), (vlm.ERR_INVALID_ARG, dict(v_sg=float("inf"))),
    (vlm.ERR_INVALID_ARG, dict(kv_heads=0)), (vlm.ERR_UNSUPPORTED, dict(dim=80)),
    (vlm.ERR_BAD_SHAPE, dict(n_pages=0)), (vlm.ERR_BAD_SHAPE, dict(n_pages=1 << 31)),
]


def _append(L, cache=None, table=B, width=4, n=3, lens=C, cu=E, n_new=7, dtype=vlm.DTYPE_F16, k=A, ks=256, v=B, vs=256):
    return L.vlm_kv4_append(ctypes.byref(cache or _cache()), table, width, n, lens, cu, n_new, dtype, k, ks, v, vs,
                            STATUS, None)


def _read(L, cache=None, table=B, width=4, n=3, start=C, cu=E, rows=7, dtype=vlm.DTYPE_F16, k=A, v=B):
    return L.vlm_kv4_read(ctypes.byref(cache or _cache()), table, width, n, start, cu, rows, dtype, k, v, STATUS, None)


def _attend(L, cache=None, table=B, width=4, n=3, lens=C, dtype=vlm.DTYPE_BF16, heads=8, q_len=1, q=A, qs=1024,
            scale=0.1, out=E, weights=None, ws=A, ws_bytes=1 << 40):
    return L.vlm_kv4_attention(ctypes.byref(cache or _cache()), table, width, n, lens, dtype, heads, q_len, q, qs, scale,
                               out, weights, ws, ws_bytes, STATUS, None)


def _evict(L, cache=None, table=B, width=4, n=3, lens=C, weights=A, budget=64, sinks=0, recent=0, to=E, to_width=1,
           to_lens=C + 4096, to_weights=6 << 20, kept=7 << 20, ws=A, ws_bytes=1 << 40):
    return L.vlm_kv4_evict(ctypes.byref(cache or _cache()), table, width, n, lens, weights, budget, sinks, recent, to,
                           to_width, to_lens, to_weights, kept, ws, ws_bytes, STATUS, None)


@pytest.mark.parametrize("call", [_append, _read, _attend, _evict])
def test_cache_calls_refuse_bad_caches_and_tables(L, call):
    before = vlm.launch_count()
    for rc, kw in BAD_CACHES:
        assert call(L, cache=_cache(**kw)) == rc, kw
    for rc, kw in [(vlm.ERR_INVALID_ARG, dict(table=None)), (vlm.ERR_INVALID_ARG, dict(table=B + 2)),
                   (vlm.ERR_BAD_SHAPE, dict(width=0)), (vlm.ERR_BAD_SHAPE, dict(n=0)), (vlm.ERR_BAD_SHAPE, dict(n=65536)),
                   (vlm.ERR_BAD_SHAPE, dict(width=(2 ** 31 - 1) // 64 + 1)),
                   (vlm.ERR_BAD_SHAPE, dict(width=1 << 20, n=1 << 12))]:
        assert call(L, **kw) == rc, kw
    assert vlm.launch_count() == before


def test_append_and_read_arguments(L):
    for rc, kw in [(vlm.ERR_UNSUPPORTED, dict(dtype=vlm.DTYPE_F32)), (vlm.ERR_INVALID_ARG, dict(k=None)),
                   (vlm.ERR_INVALID_ARG, dict(v=A + 4)), (vlm.ERR_BAD_SHAPE, dict(ks=128)),
                   (vlm.ERR_UNSUPPORTED, dict(vs=260)), (vlm.ERR_BAD_SHAPE, dict(n_new=-1)),
                   (vlm.ERR_BAD_SHAPE, dict(cu=None, n_new=4)), (vlm.ERR_INVALID_ARG, dict(cu=E + 1)),
                   (vlm.ERR_INVALID_ARG, dict(lens=C + 3)), (vlm.OK, dict(n_new=0))]:
        assert _append(L, **kw) == rc, kw
    for rc, kw in [(vlm.ERR_UNSUPPORTED, dict(dtype=vlm.DTYPE_F32)), (vlm.ERR_INVALID_ARG, dict(k=None)),
                   (vlm.ERR_BAD_SHAPE, dict(rows=-1)), (vlm.ERR_BAD_SHAPE, dict(cu=None)), (vlm.OK, dict(rows=0))]:
        assert _read(L, **kw) == rc, kw


def test_cache_attention_arguments(L):
    need = vlm.kv4_attention_workspace_size(3, 8, 2, 128)
    for rc, kw in [(vlm.ERR_INVALID_ARG, dict(lens=None)), (vlm.ERR_INVALID_ARG, dict(ws=None)),
                   (vlm.ERR_INVALID_ARG, dict(ws=A + 16)), (vlm.ERR_WORKSPACE, dict(ws_bytes=need - 1)),
                   (vlm.ERR_UNSUPPORTED, dict(heads=7)), (vlm.ERR_UNSUPPORTED, dict(heads=258)),
                   (vlm.ERR_BAD_SHAPE, dict(q_len=0)), (vlm.ERR_BAD_SHAPE, dict(q_len=16384)),
                   (vlm.ERR_INVALID_ARG, dict(q=A + 8)), (vlm.ERR_BAD_SHAPE, dict(qs=1016)),
                   (vlm.ERR_UNSUPPORTED, dict(dtype=vlm.DTYPE_F32)), (vlm.ERR_INVALID_ARG, dict(scale=-1.0)),
                   (vlm.ERR_INVALID_ARG, dict(weights=A + 2)), (vlm.ERR_INVALID_ARG, dict(out=None))]:
        assert _attend(L, **kw) == rc, kw
    assert vlm.kv4_attention_workspace_size(0, 8, 2, 128) == 0
    assert vlm.kv4_attention_workspace_size(3, 8, 3, 128) == 0
    assert vlm.kv4_attention_workspace_size(3, 8, 2, 100) == 0


def test_eviction_arguments(L):
    need = vlm.kv4_evict_workspace_size(10, 3, 2, 64)
    for rc, kw in [(vlm.ERR_BAD_SHAPE, dict(budget=0)), (vlm.ERR_BAD_SHAPE, dict(budget=65)),
                   (vlm.ERR_BAD_SHAPE, dict(sinks=-1)), (vlm.ERR_BAD_SHAPE, dict(sinks=40, recent=25)),
                   (vlm.ERR_BAD_SHAPE, dict(to_width=0)), (vlm.ERR_INVALID_ARG, dict(weights=None)),
                   (vlm.ERR_INVALID_ARG, dict(to=None)), (vlm.ERR_INVALID_ARG, dict(to_lens=None)),
                   (vlm.ERR_INVALID_ARG, dict(to_weights=None)), (vlm.ERR_INVALID_ARG, dict(to_lens=C + 8)),  # over lens
                   (vlm.ERR_INVALID_ARG, dict(to_weights=A + 1024)),  # over weights
                   (vlm.ERR_INVALID_ARG, dict(ws=A + 128)), (vlm.ERR_WORKSPACE, dict(ws_bytes=need - 1))]:
        assert _evict(L, **kw) == rc, kw


def test_page_bytes(L):
    assert vlm.kv4_page_bytes(8, 128) == 8 * 64 * 144
    assert vlm.kv4_page_bytes(1, 64) == 64 * 72
    assert vlm.kv4_page_bytes(0, 64) == 0 and vlm.kv4_page_bytes(2, 96) == 0
    assert vlm.status_string(vlm.ERR_BAD_PAGE) == "VLM_ERR_BAD_PAGE"


def test_binding_refuses_tensors_off_the_gpu_and_of_other_shapes():
    q = torch.zeros((5, 8, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        vlm.prompt_attention(q, q, q, [5])
    with pytest.raises(ValueError):
        vlm.prompt_attention(q, q, q, [5], [5, 0])
    pages = torch.zeros((4, 2, 64 * 72), dtype=torch.uint8)
    with pytest.raises(ValueError):
        vlm.kv4_attention(pages, torch.zeros((1, 2), dtype=torch.int32), None, q, 1.0, 1.0)
    with pytest.raises(ValueError):
        vlm.kv4_append(pages[:, :, :70], torch.zeros((1, 2), dtype=torch.int32), None, q, q, 1.0, 1.0)
    with pytest.raises(TypeError):
        vlm._dtype16(torch.float32)


@pytest.mark.parametrize("call", [_append, _read, _attend, _evict])
def test_tables_whose_places_leave_no_room_in_32_bits_are_refused(L, call):
    # the kernels step over places by up to 4,096, so a table may not reach to the end of 32 bits
    room = (2 ** 31 - 1 - 8192) // 64
    assert call(L, width=room + 1, n=1) == vlm.ERR_BAD_SHAPE
    if call is _evict:
        assert _evict(L, to_width=room + 1, n=1) == vlm.ERR_BAD_SHAPE
    # as many entries in all as 32-bit offsets of the sequences take, two more each
    assert call(L, width=(2 ** 31 - 1) // 64, n=64) == vlm.ERR_BAD_SHAPE


@pytest.mark.parametrize("kw", [
    dict(kept=A + 512), dict(kept=C), dict(kept=C - 1532), dict(kept=B), dict(kept=E), dict(kept=C + 4096), dict(kept=6 << 20),
    dict(to_lens=A + 4), dict(to_lens=C), dict(to_lens=B + 44), dict(to_lens=E), dict(to_lens=(6 << 20) + 64),
    dict(to_weights=C), dict(to_weights=C - 4), dict(to_weights=B - 8), dict(to_weights=E - 1532), dict(to_weights=7 << 20),
    dict(to_weights=C + 4100),
    dict(kept=None, to_lens=A), dict(to_lens=STATUS - 8), dict(to_weights=STATUS - 1532),
    dict(weights=9 << 20, ws=8 << 20, to_weights=A + (180 << 10) - 8),  # over the pool's last page
    dict(weights=9 << 20, ws=8 << 20, kept=(8 << 20) + 64),          # over the workspace
])
def test_eviction_refuses_results_over_other_buffers(L, kw):
    # kernels write the results while other CTAs still read what the call was given
    before = vlm.launch_count()
    assert _evict(L, **kw) == vlm.ERR_INVALID_ARG, kw
    assert vlm.launch_count() == before
