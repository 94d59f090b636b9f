"""The 8-bit cache's entry points, summed weights and eviction: refusals on the host (CPU).

Every call below is rejected before anything reaches CUDA; the fake pointers are never
dereferenced.
"""
import ctypes

import pytest
import torch

import query_predicted_token_b200 as asp
from query_predicted_token_b200 import _lib as L
from query_predicted_token_b200 import build as B

FAKE = 0x10000
INV, UNS, WS = L.ASP_ERR_INVALID_ARG, L.ASP_ERR_UNSUPPORTED, L.ASP_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.lib()


def kv8(**kw):
    base = dict(batch=2, n_kv_heads=2, head_dim=128, t_max=1024, kv_dtype=L.ASP_E4M3, k=FAKE, v=FAKE, page_size=0,
                page_table=None, max_pages=0, n_pages=0, seq_lens=FAKE, k_scale=FAKE, v_scale=FAKE, scale_block=64,
                src_dtype=L.ASP_BF16)
    base.update(kw)
    return L.AspKv(**base)


BAD = [
    (dict(head_dim=96), UNS),
    (dict(scale_block=8), UNS),
    (dict(scale_block=0), UNS),
    (dict(scale_block=256), UNS),
    (dict(k_scale=None), INV),
    (dict(k_scale=FAKE + 2), INV),
    (dict(kv_dtype=4), INV),
    (dict(k=FAKE + 8), INV),
    (dict(page_size=32, page_table=FAKE, max_pages=32, n_pages=64), UNS),     # blocks of 64 across 32-token pages
    (dict(page_size=64, page_table=None, max_pages=16, n_pages=64), INV),
    (dict(page_size=64, page_table=FAKE, max_pages=15, n_pages=64), INV),     # 960 tokens < t_max
]


@pytest.mark.parametrize("kw,expect", BAD)
def test_every_call_rejects_bad_caches(lib, kw, expect):
    kv = ctypes.byref(kv8(**kw))
    assert lib.asp_score_keys(FAKE, 8, kv, FAKE, None) == expect
    assert lib.asp_quantize_kv(kv, FAKE, FAKE, L.ASP_BF16, 1024, 512, 128, None) == expect
    assert lib.asp_dequantize_kv(kv, FAKE, FAKE, L.ASP_F32, 1024, 512, 128, None) == expect
    assert lib.asp_append_kv(kv, FAKE, FAKE, None, None, 16, None) == expect
    assert lib.asp_sparse_attend(FAKE, L.ASP_BF16, 8, kv, FAKE, FAKE, 64, None, 0, FAKE, None, FAKE, 1 << 40, None) == expect
    assert lib.asp_attend_accumulate(FAKE, L.ASP_BF16, 8, kv, FAKE, FAKE, 64, None, 0, FAKE, None, FAKE, FAKE, 1 << 40,
                                     None) == expect
    assert lib.asp_evict_kv(kv, FAKE, FAKE, 16, 0, 0, FAKE, FAKE, FAKE, 1 << 40, None) == expect


def test_value_side_scales_are_needed_where_values_are_read(lib):
    kv = ctypes.byref(kv8(v_scale=None))
    assert lib.asp_sparse_attend(FAKE, L.ASP_BF16, 8, kv, FAKE, FAKE, 64, None, 0, FAKE, None, FAKE, 1 << 40, None) == INV
    assert lib.asp_quantize_kv(kv, FAKE, FAKE, L.ASP_BF16, 1024, 512, 128, None) == INV


def test_calls_that_take_wide_caches_only(lib):
    kv = ctypes.byref(kv8())
    assert lib.asp_score_keys_cuda_cores(FAKE, 8, kv, FAKE, None) == UNS
    assert lib.asp_quest_build_meta(kv, 16, FAKE, None) == UNS
    assert lib.asp_quest_page_scores(FAKE, L.ASP_BF16, 8, kv, FAKE, 16, FAKE, None) == UNS
    assert lib.asp_quest_select(FAKE, L.ASP_BF16, 8, kv, FAKE, 16, 64, FAKE, FAKE, FAKE, None) == UNS
    assert lib.asp_sparse_attend_noalloc(FAKE, L.ASP_BF16, 8, kv, FAKE, FAKE, 64, None, 0, FAKE, None, None) == UNS
    assert lib.asp_append_kv(kv, FAKE, FAKE, None, FAKE, 16, None) == UNS          # page bounds of an 8-bit cache
    assert lib.asp_append_kv(ctypes.byref(kv8(src_dtype=L.ASP_I8)), FAKE, FAKE, None, None, 16, None) == INV
    wide = ctypes.byref(kv8(kv_dtype=L.ASP_BF16))
    assert lib.asp_quantize_kv(wide, FAKE, FAKE, L.ASP_BF16, 1024, 512, 128, None) == UNS
    assert lib.asp_dequantize_kv(wide, FAKE, FAKE, L.ASP_BF16, 1024, 512, 128, None) == UNS


def test_row_arguments(lib):
    kv = ctypes.byref(kv8())
    for fn in (lib.asp_quantize_kv, lib.asp_dequantize_kv):
        assert fn(kv, None, FAKE, L.ASP_BF16, 1024, 512, 128, None) == INV
        assert fn(kv, FAKE, FAKE + 8, L.ASP_BF16, 1024, 512, 128, None) == INV
        assert fn(kv, FAKE, FAKE, L.ASP_E4M3, 1024, 512, 128, None) == INV
        assert fn(kv, FAKE, FAKE, L.ASP_BF16, 1024, 512, 132, None) == INV          # 264-byte rows
        assert fn(kv, FAKE, FAKE, L.ASP_BF16, 1024, -512, 128, None) == INV
        assert fn(None, FAKE, FAKE, L.ASP_BF16, 1024, 512, 128, None) == INV


@pytest.mark.parametrize("dtype", [L.ASP_F32, L.ASP_BF16, L.ASP_E4M3, L.ASP_I8])
def test_accumulate_arguments(lib, dtype):
    kv = kv8(kv_dtype=dtype)
    r = ctypes.byref(kv)
    need = lib.asp_accumulate_workspace_bytes(r, 8, 64, 16)
    assert need > 0 and need % 256 == 0
    call = lambda q=FAKE, hq=8, idx=FAKE, C=64, tb=FAKE, mt=16, out=FAKE, acc=FAKE, ws=FAKE, n=need: \
        lib.asp_attend_accumulate(q, L.ASP_BF16, hq, r, idx, FAKE, C, tb, mt, out, None, acc, ws, n, None)
    assert call(acc=None) == INV
    assert call(q=None) == INV
    assert call(out=None) == INV
    assert call(idx=None) == INV
    if dtype == L.ASP_F32:
        assert call(q=FAKE + 4) == INV         # an fp32 cache's kernel reads the query by whole vectors
    assert call(hq=7) == INV
    assert call(hq=6) == UNS
    assert call(C=0, tb=None) == INV           # nothing to attend
    assert call(mt=-1) == INV
    assert call(n=need - 1) == WS
    assert call(ws=None) == WS
    assert call(ws=FAKE + 128) == WS           # 256-byte alignment
    assert lib.asp_accumulate_workspace_bytes(r, 7, 64, 16) == 0
    assert lib.asp_accumulate_workspace_bytes(r, 8, 0, 0) == 0
    assert lib.asp_accumulate_workspace_bytes(None, 8, 64, 16) == 0
    # the workspace does not depend on pointers
    bare = kv8(kv_dtype=dtype, k=None, v=None, k_scale=None, v_scale=None, seq_lens=None)
    assert lib.asp_accumulate_workspace_bytes(ctypes.byref(bare), 8, 64, 16) == need
    # logits of every head and row fit
    assert need >= 2 * 8 * 80 * 4


@pytest.mark.parametrize("dtype", [L.ASP_F32, L.ASP_BF16, L.ASP_E4M3, L.ASP_I8])
def test_evict_arguments(lib, dtype):
    kv = kv8(kv_dtype=dtype)
    r = ctypes.byref(kv)
    need = lib.asp_evict_workspace_bytes(r, 16)
    assert need > 0
    call = lambda r=r, acc=FAKE, out=FAKE, C=16, sink=1, recent=4, idx=FAKE, cnt=FAKE, ws=FAKE, n=need: \
        lib.asp_evict_kv(r, acc, out, C, sink, recent, idx, cnt, ws, n, None)
    assert call(acc=None) == INV
    assert call(out=None) == INV
    assert call(idx=None) == INV
    assert call(cnt=None) == INV
    assert call(C=0) == INV
    assert call(sink=-1) == INV
    assert call(recent=-1) == INV
    assert call(sink=8, recent=9) == INV
    assert call(r=ctypes.byref(kv8(kv_dtype=dtype, seq_lens=None))) == INV
    assert call(ws=None) == WS
    assert call(ws=FAKE + 16) == WS
    assert call(n=need - 1) == WS
    assert lib.asp_evict_workspace_bytes(r, 0) == 0


def test_workspace_sizes_by_cache(lib):
    wide, narrow = kv8(kv_dtype=L.ASP_BF16), kv8()
    for C, mt in [(64, 0), (64, 16), (0, 1024), (900, 100)]:
        assert lib.asp_attend_workspace_bytes_kv(ctypes.byref(wide), 8, C, mt) == \
            lib.asp_attend_workspace_bytes(2, 8, 2, 128, C, mt)
        if C:
            assert lib.asp_decode_workspace_bytes_kv(ctypes.byref(wide), 8, C, mt) == \
                lib.asp_decode_workspace_bytes(2, 8, 2, 128, C, mt)
    need = lib.asp_attend_workspace_bytes_kv(ctypes.byref(narrow), 8, 900, 100)
    assert need > 0
    a = lib.asp_sparse_attend(FAKE, L.ASP_BF16, 8, ctypes.byref(narrow), FAKE, FAKE, 900, FAKE, 100, FAKE, None, FAKE,
                              need - 1, None)
    assert a == WS
    dec = lib.asp_decode_workspace_bytes_kv(ctypes.byref(narrow), 8, 900, 100)
    assert dec >= 2 * 2 * 2048 * 4        # the selection's histogram at least
    assert lib.asp_decode_workspace_bytes_kv(ctypes.byref(narrow), 8, 0, 100) == 0
    assert lib.asp_attend_workspace_bytes_kv(ctypes.byref(kv8(head_dim=96)), 8, 64, 0) == 0


def test_the_binding_checks_scales_and_rows():
    k = torch.zeros(2, 3, 100, 64, dtype=torch.int8)
    s = torch.ones(2, 3, 4)
    assert asp.scale_shape(k, 32, False) == (2, 3, 4)
    kv = asp.KV(k, k.clone(), None, k_scale=s, v_scale=s.clone(), scale_block=32)
    assert kv.struct.kv_dtype == L.ASP_I8 and kv.struct.scale_block == 32
    with pytest.raises(ValueError, match="scale_block"):
        asp.KV(k, k, k_scale=s, v_scale=s)
    with pytest.raises(ValueError, match="k_scale"):
        asp.KV(k, k, k_scale=None, v_scale=s, scale_block=32)
    with pytest.raises(ValueError, match="v_scale"):
        asp.KV(k, k, k_scale=s, v_scale=s[:, :, :3], scale_block=32)
    with pytest.raises(ValueError, match="k_scale"):
        asp.KV(k, k, k_scale=s.double(), v_scale=s, scale_block=32)
    with pytest.raises(TypeError):
        asp.KV(k, k.float(), k_scale=s, v_scale=s, scale_block=32)
    with pytest.raises(ValueError, match="t_max"):
        asp.KV(k, k, t_max=90, k_scale=s, v_scale=s, scale_block=32)
    with pytest.raises(ValueError, match="page size"):
        asp.scale_shape(torch.zeros(4, 3, 48, 64, dtype=torch.int8), 32, True)
    rows = torch.zeros(2, 3, 100, 64)
    with pytest.raises(ValueError, match="quantize_kv"):
        asp.quantize_kv(kv, rows[:, :2], rows[:, :2], stream=0)
    with pytest.raises(ValueError, match="strides"):
        asp.quantize_kv(kv, rows, torch.zeros(2, 100, 3, 64).transpose(1, 2), stream=0)
    with pytest.raises(ValueError, match="strides"):
        asp.dequantize_kv(kv, rows, rows.bfloat16(), stream=0)
    with pytest.raises(ValueError, match="contiguous channels"):
        asp.quantize_kv(kv, torch.zeros(2, 3, 64, 100).transpose(2, 3), torch.zeros(2, 3, 64, 100).transpose(2, 3),
                        stream=0)
    with pytest.raises(TypeError):
        asp.quantize_kv(kv, rows.half(), rows.half(), stream=0)


def test_wide_caches_ignore_the_8_bit_arguments():
    k = torch.zeros(1, 2, 10, 64, dtype=torch.bfloat16)
    kv = asp.KV(k, k, k_scale=None, v_scale=None, scale_block=0, src_dtype=torch.float32)
    assert kv.struct.kv_dtype == L.ASP_BF16 and kv.struct.scale_block == 0 and not kv.struct.k_scale
