"""Eviction at the lengths it is for: every row width of the choice, and moves of several chunks (GPU).

Everything is compared exactly.  With scales that are no powers of two a code moves as the kernel's steps say: the
block's largest |code * scale| in fp32 sets the new scale, code * (scale / new scale) in fp32 is rounded to the code.
"""
import numpy as np
import pytest
import torch

import query_predicted_token_b200 as asp
from oracle import cache8
from parity_util import np64
from test_gpu_cache8 import CODE, DEV, WIDE, Cache, _built, gen  # noqa: F401

pytestmark = pytest.mark.gpu


def recoded(codes, scales, keep, block, fmt):
    """The kept rows of ``codes [n, d]`` (``scales`` per row) as new blocks."""
    c, s = codes[keep].astype(np.float32), scales[keep].astype(np.float32)
    nb = -(-len(keep) // block)
    out, new = np.zeros(c.shape), np.zeros(nb)
    for i in range(nb):
        rows = slice(i * block, min(len(keep), (i + 1) * block))
        top = np.abs(c[rows]).max(axis=1) * s[rows]
        new[i] = cache8.block_scale(top, fmt)
        f = (s[rows] / np.float32(new[i])).astype(np.float32)
        out[rows] = cache8.code_values(c[rows] * f[:, None], fmt)
    return out, new


def run_evict(fmt, T, lens, C, sink, recent, in_place, sums, d=64, page=0, block=16, odd=False, H=2, seed=1):
    B = len(lens)
    c = Cache(fmt, B, H, d, T, lens, page, block, seed=seed, odd_scales=odd, spread=1.5)
    g = gen(seed)
    if sums == "spread":
        acc = torch.rand(B, H, T, generator=g).pow_(6)
    elif sums == "ties":
        acc = torch.randint(0, 9, (B, H, T), generator=g).float()
    else:
        acc = torch.zeros(B, H, T)
    acc = acc.to(DEV)
    a = np64(acc)
    before = {s: [c.codes(s, b) for b in range(B)] for s in "kv"}
    idx = torch.full((B, H, C), 12345, dtype=torch.int32, device=DEV)
    cnt = torch.full((B, H), 12345, dtype=torch.int32, device=DEV)
    ws = torch.empty(asp.evict_workspace_bytes(c.kv, C), dtype=torch.uint8, device=DEV)
    out = acc if in_place else torch.full_like(acc, -3.0)
    asp.evict_kv(c.kv, acc, C, idx, cnt, n_sink=sink, n_recent=recent, acc_out=None if in_place else out, workspace=ws)
    assert asp.device_status() == 0
    assert c.seq_lens.tolist() == [min(C, n) for n in lens]
    got_acc, got_idx, got_cnt = np64(out), idx.cpu().numpy(), cnt.cpu().numpy()
    for b, n in enumerate(lens):
        after = {s: c.codes(s, b) for s in "kv"}
        for h in range(H):
            keep = cache8.kept_tokens(a[b, h, :n], n, C, sink, recent)
            m = len(keep)
            assert got_cnt[b, h] == m
            assert np.array_equal(got_idx[b, h, :m], keep) and (got_idx[b, h, m:] == -1).all(), (b, h)
            assert np.array_equal(got_acc[b, h, :m], a[b, h, keep]) and (got_acc[b, h, m:] == 0).all(), (b, h)
            for s in "kv":
                codes, scales = after[s]
                oc, osc = before[s][b]
                if n <= C or fmt in WIDE:
                    assert np.array_equal(codes[h], oc[h][keep]), (s, b, h)
                    assert scales is None or np.array_equal(scales[h], osc[h]), (s, b, h)
                else:
                    rc, rs = recoded(oc[h], np.repeat(osc[h], block)[:n], keep, block, fmt)
                    assert np.array_equal(scales[h], rs), (s, b, h)
                    assert np.array_equal(codes[h], rc), (s, b, h)


@pytest.mark.parametrize("T", [4096, 4097, 5000, 8192, 8193, 12000, 16385, 20000, 32768, 32769, 40000, 49152, 49153, 60001])
@pytest.mark.parametrize("sums", ["spread", "ties", "zero"])
@pytest.mark.parametrize("in_place", [False, True])
def test_the_choice_at_every_row_width(T, sums, in_place):
    """Rows kept in 4, 8, 16 and 32 registers a thread, in shared memory, and re-read."""
    C = T // 3
    run_evict("bf16", T, [T, T - 3, C + 1, C, 2], C, 4, 30, in_place, sums)


@pytest.mark.parametrize("C,sink,recent", [(1, 0, 0), (64, 0, 0), (500, 500, 0), (500, 0, 500), (39000, 100, 100)])
@pytest.mark.parametrize("T", [20000, 40000, 60000])
def test_the_choice_with_few_and_many_kept(T, C, sink, recent):
    run_evict("bf16", T, [T, T - 1], min(C, T - 2), sink, recent, False, "spread")


@pytest.mark.parametrize("fmt", ["e4m3", "int8", "f32"])
@pytest.mark.parametrize("d,page,block", [(64, 0, 16), (128, 0, 128), (64, 48, 16), (128, 256, 64)])
@pytest.mark.parametrize("odd", [False, True])
def test_moves_of_many_chunks(fmt, d, page, block, odd):
    """5000 kept rows: 5 chunks of 8-bit rows at d = 64, 10 at d = 128, up to 40 of fp32 rows."""
    run_evict(fmt, 9000, [9000, 5003, 100], 5000, 4, 1000, True, "spread", d, page, block, odd)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_a_long_8bit_row_cut_in_half(fmt):
    run_evict(fmt, 33000, [33000], 16500, 4, 64, False, "ties", 128, 0, 64, True, H=1)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_blocks_whose_scales_lie_far_apart(fmt):
    """Rows of one new block come from scales up to 2^30 apart: small ones become subnormal or zero codes."""
    for odd in (False, True):
        B, H, T, d, block, C = 1, 2, 2600, 64, 16, 1300
        c = Cache(fmt, B, H, d, T, [T], 0, block, seed=4, odd_scales=odd, spread=9.0)
        acc = torch.rand(B, H, T, generator=gen(2)).to(DEV)
        a, before = np64(acc), {s: c.codes(s, 0) for s in "kv"}
        idx = torch.empty(B, H, C, dtype=torch.int32, device=DEV)
        cnt = torch.empty(B, H, dtype=torch.int32, device=DEV)
        ws = torch.empty(asp.evict_workspace_bytes(c.kv, C), dtype=torch.uint8, device=DEV)
        asp.evict_kv(c.kv, acc, C, idx, cnt, n_sink=1, n_recent=7, workspace=ws)
        assert asp.device_status() == 0
        for h in range(H):
            keep = cache8.kept_tokens(a[0, h], T, C, 1, 7)
            for s in "kv":
                oc, osc = before[s]
                rc, rs = recoded(oc[h], np.repeat(osc[h], block)[:T], keep, block, fmt)
                codes, scales = c.codes(s, 0)
                assert np.array_equal(scales[h], rs) and np.array_equal(codes[h], rc), (odd, s, h)
