"""The Python binding's checks around the 8-bit cache (CPU): every call below is refused before the library is called."""
import pytest
import torch

import query_predicted_token_b200 as asp
from query_predicted_token_b200 import _lib as L

B, H, T, D, HQ, C = 2, 3, 64, 64, 6, 16


class NoCalls:
    """Stands in for the library: the call must not get there."""

    def __getattr__(self, name):
        raise AssertionError(f"{name} was reached")


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    monkeypatch.setattr(L, "_lib", NoCalls())


def cache8(dtype=torch.int8, **kw):
    k = torch.zeros(B, H, T, D, dtype=dtype)
    s = torch.ones(B, H, T // 16)
    return asp.KV(k, k.clone(), torch.zeros(B, dtype=torch.int32), k_scale=s, v_scale=s.clone(), scale_block=16, **kw)


def wide(dtype):
    k = torch.zeros(B, H, T, D, dtype=dtype)
    return asp.KV(k, k.clone(), torch.zeros(B, dtype=torch.int32))


def test_the_rows_type_is_fp32_or_bf16():
    assert cache8(src_dtype=torch.float32).struct.src_dtype == L.ASP_F32
    assert cache8().struct.src_dtype == L.ASP_BF16
    for t in (torch.float16, torch.float64, torch.int8, torch.float8_e4m3fn):
        with pytest.raises(TypeError, match="src_dtype"):
            cache8(src_dtype=t)


@pytest.mark.parametrize("src,rows", [(torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16),
                                      (torch.bfloat16, torch.float16)])
def test_appended_rows_have_the_declared_type(src, rows):
    """bf16 rows read as fp32 would be read past their end."""
    kv = cache8(src_dtype=src)
    good, bad = torch.zeros(B, H, D, dtype=src), torch.zeros(B, H, D, dtype=rows)
    for k, v in ((bad, bad), (good, bad), (bad, good)):
        with pytest.raises(TypeError, match="append_kv"):
            asp.append_kv(kv, k, v, stream=0)


@pytest.mark.parametrize("q,out", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)])
def test_an_8bit_caches_output_has_the_querys_type(q, out):
    """An fp32 query writes fp32: a bf16 output would be written past its end."""
    kv = cache8()
    qt, ot, acc = torch.zeros(B, HQ, D, dtype=q), torch.zeros(B, HQ, D, dtype=out), torch.zeros(B, H, T)
    with pytest.raises(TypeError, match="sparse_attend"):
        asp.sparse_attend(qt, kv, None, None, 0, ot, stream=0)
    with pytest.raises(TypeError, match="attend_accumulate"):
        asp.attend_accumulate(qt, kv, None, None, 0, ot, acc, stream=0)


@pytest.mark.parametrize("cache,out", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)])
def test_a_wide_caches_accumulated_output_has_its_type(cache, out):
    q, acc = torch.zeros(B, HQ, D), torch.zeros(B, H, T)
    with pytest.raises(TypeError, match="attend_accumulate"):
        asp.attend_accumulate(q, wide(cache), None, None, 0, torch.zeros(B, HQ, D, dtype=out), acc, stream=0)


def test_a_decode_step_checks_the_same_types():
    kv = cache8()
    st = asp.DecodeState.__new__(asp.DecodeState)       # the checks come before any buffer is looked at
    st.kv = kv
    q, new = torch.zeros(B, HQ, D, dtype=torch.bfloat16), torch.zeros(B, H, D, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="step"):
        st.step(q, torch.zeros(B, HQ, D), None, new, new)
    with pytest.raises(TypeError, match="step"):
        st.step(q, torch.zeros_like(q), None, new.float(), new.float())


@pytest.mark.parametrize("fmt", [torch.int8, torch.bfloat16])
def test_sums_are_fp32_of_every_token(fmt):
    kv = cache8() if fmt == torch.int8 else wide(fmt)
    q = torch.zeros(B, HQ, D, dtype=torch.bfloat16)
    out = torch.zeros_like(q)
    idx, cnt = torch.zeros(B, H, C, dtype=torch.int32), torch.zeros(B, H, dtype=torch.int32)
    good = torch.zeros(B, H, T)
    for acc in (good.double(), good[:, :, :-1].contiguous(), good.transpose(1, 2)):
        with pytest.raises((TypeError, ValueError), match="acc"):
            asp.attend_accumulate(q, kv, None, None, 0, out, acc, stream=0)
        with pytest.raises((TypeError, ValueError), match="acc"):
            asp.evict_kv(kv, acc, C, idx, cnt, stream=0)
        with pytest.raises((TypeError, ValueError), match="acc"):
            asp.evict_kv(kv, good, C, idx, cnt, acc_out=acc, stream=0)
    for i, c in ((idx.long(), cnt), (idx[:, :, 1:].contiguous(), cnt), (idx, cnt.long()), (idx, cnt[:1])):
        with pytest.raises((TypeError, ValueError), match="idx|count"):
            asp.evict_kv(kv, good, C, i, c, stream=0)


@pytest.mark.parametrize("call", ["quantize_kv", "dequantize_kv"])
@pytest.mark.parametrize("nk,nv", [(40, 40), (64, 64), (80, 50), (17, 80)])
def test_the_rows_token_count_bounds_the_call(monkeypatch, call, nk, nv):
    """Lengths live on the device: the kernels must learn how many tokens the rows hold."""
    seen = []

    class Record:
        def __getattr__(self, name):
            return lambda *args: seen.append((name, args)) or L.ASP_OK

    monkeypatch.setattr(L, "_lib", Record())
    k = torch.zeros(B, H, 80, D)
    getattr(asp, call)(cache8(), k[:, :, :nk], k[:, :, :nv], stream=0)
    (name, args), = seen
    assert name == f"asp_{call}_bounded"
    assert args[3:8] == (L.ASP_F32, min(nk, nv), H * 80 * D, 80 * D, D)


def test_the_bound_is_at_least_one_token(monkeypatch):
    monkeypatch.setattr(L, "_lib", None)
    from query_predicted_token_b200 import build
    build.build()
    kv = L.AspKv(2, 2, 128, 1024, L.ASP_I8, 0x10000, 0x10000, 0, None, 0, 0, 0x10000, 0x10000, 0x10000, 64, L.ASP_BF16)
    for fn in (L.lib().asp_quantize_kv_bounded, L.lib().asp_dequantize_kv_bounded):
        for n in (0, -1):
            assert fn(kv, 0x10000, 0x10000, L.ASP_BF16, n, 1024, 512, 128, None) == L.ASP_ERR_INVALID_ARG


@pytest.mark.parametrize("dtype", [L.ASP_F32, L.ASP_BF16, L.ASP_E4M3, L.ASP_I8])
def test_rows_past_the_sums_grid_are_refused_before_the_attention_runs(monkeypatch, dtype):
    """The sums' launch has 65535 CTAs of 1024 rows per unit at most."""
    monkeypatch.setattr(L, "_lib", None)
    from query_predicted_token_b200 import build
    build.build()
    lib, p = L.lib(), 0x10000
    kv = L.AspKv(1, 1, 64, 1024, dtype, p, p, 0, None, 0, 0, p, p, p, 64, L.ASP_BF16)
    most = 65535 * 1024
    assert lib.asp_accumulate_workspace_bytes(kv, 1, 0, most) > 4 * most
    for C, tail in ((0, most + 1), (1, most), (most, 1), (0, 1 << 30)):
        assert lib.asp_accumulate_workspace_bytes(kv, 1, C, tail) == 0
        st = lib.asp_attend_accumulate(p, L.ASP_BF16, 1, kv, p, p, C, p, tail, p, None, p, p, 1 << 60, None)
        assert st == L.ASP_ERR_UNSUPPORTED


def test_rows_read_back_must_not_coincide(monkeypatch):
    """A destination with a stride of 0, as expand() gives, would be written by many rows at once; a source may have one."""
    monkeypatch.setattr(L, "_lib", None)
    from query_predicted_token_b200 import build
    build.build()
    lib, p = L.lib(), 0x10000
    for paged in (False, True):
        kv = L.AspKv(2, 2, 128, 1024, L.ASP_I8, p, p, 64 if paged else 0, p, 16, 64, p, p, p, 64, L.ASP_BF16)
        for st in ((0, 512, 128), (1024, 0, 128), (1024, 512, 0), (1024, 512, 64)):
            assert lib.asp_dequantize_kv(kv, p, p, L.ASP_BF16, *st, None) == L.ASP_ERR_INVALID_ARG
            assert lib.asp_dequantize_kv_bounded(kv, p, p, L.ASP_BF16, 8, *st, None) == L.ASP_ERR_INVALID_ARG
