"""Filling from and reading back into rows that hold fewer tokens than a sequence has (GPU)."""
import numpy as np
import pytest
import torch

import query_predicted_token_b200 as asp
from oracle import cache8
from parity_util import np64
from test_gpu_cache8 import DEV, WIDE, Cache, _built, gen  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("wide", ["bf16", "f32"])
@pytest.mark.parametrize("d,page,block", [(64, 0, 16), (128, 32, 32), (128, 0, 128)])
@pytest.mark.parametrize("n", [1, 40, 130])
def test_longer_sequences_are_cut_and_flagged(fmt, wide, d, page, block, n):
    lens, T, H = [200, n, 0, n + 1], 200, 2
    c = Cache(fmt, 4, H, d, T, lens, page, block, seed=n)
    x = torch.randn(2, 4, H, n + 40, d, generator=gen(2)).to(WIDE[wide]).to(DEV)
    x[:, :, :, n:] = float("nan")                       # what lies past the rows must not be read
    before = {s: [c.codes(s, b) for b in range(4)] for s in "kv"}
    asp.quantize_kv(c.kv, x[0, :, :, :n], x[1, :, :, :n])
    assert asp.device_status() == asp.ASP_DEV_ROW_LIMIT
    for i, s in enumerate("kv"):
        for b, T_b in enumerate(lens):
            m = min(n, T_b)
            codes, scales = c.codes(s, b)
            for h in range(H):
                rc, rs = cache8.quantize(np64(x[i, b, h, :m].float()), block, fmt)
                assert np.array_equal(codes[h][:m], rc) and np.array_equal(scales[h][:len(rs)], rs)
                assert np.array_equal(codes[h][m:], before[s][b][0][h][m:])
                assert np.array_equal(scales[h][len(rs):], before[s][b][1][h][len(rs):])
    buf = torch.full((2, 4, H, n + 40, d), -7.0, device=DEV, dtype=WIDE[wide])
    asp.dequantize_kv(c.kv, buf[0, :, :, :n], buf[1, :, :, :n])
    assert asp.device_status() == asp.ASP_DEV_ROW_LIMIT
    assert (buf[:, :, :, n:] == -7).all()
    for i, s in enumerate("kv"):
        for b, T_b in enumerate(lens):
            m = min(n, T_b)
            want = torch.from_numpy(c.rows(s, b)[:, :m]).float().to(WIDE[wide])
            assert torch.equal(buf[i, b, :, :m].cpu(), want) and (buf[i, b, :, m:] == -7).all()
    # rows that hold every sequence are not flagged
    c.seq_lens.clamp_(max=n)
    asp.quantize_kv(c.kv, x[0, :, :, :n], x[1, :, :, :n])
    asp.dequantize_kv(c.kv, buf[0, :, :, :n], buf[1, :, :, :n])
    assert asp.device_status() == 0


def test_a_cache_without_lengths_is_cut_at_the_rows():
    k = torch.zeros(1, 1, 64, 64, dtype=torch.int8, device=DEV)
    s = torch.ones(1, 1, 4, device=DEV)
    kv = asp.KV(k, k.clone(), k_scale=s, v_scale=s.clone(), scale_block=16)
    buf = torch.full((2, 1, 1, 48, 64), -7.0, device=DEV)
    asp.dequantize_kv(kv, buf[0, :, :, :20], buf[1, :, :, :20])
    assert asp.device_status() == asp.ASP_DEV_ROW_LIMIT
    assert (buf[:, :, :, :20] == 0).all() and (buf[:, :, :, 20:] == -7).all()
