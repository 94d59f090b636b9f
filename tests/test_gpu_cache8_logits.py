"""Attention of every cache type at logits of any finite size (GPU).

Keys and queries differ from zero in channel 0 alone and sqrt(d) = 8, so a row's logit is one product: rows with equal
keys get the same float whatever its rounding error, and the others lie at half or twice that logit, further away than
any rounding.  The softmax is then uniform over the best rows, exactly, at every size of the logits, and the bounds of
test_gpu_cache8.py hold with D = 0: out within 2^-19 (exponentials and sums) + (n + 17 n) / 16 2^-23 (the fp32 sums over
n rows) + the weights' parts (2^-11 for one fp16 part, 2^-18 for two) of sum w |v|, plus half a step of its own type; acc
within 2^-19 + n / 16 2^-23 of each weight.
"""
import numpy as np
import pytest
import torch

import query_predicted_token_b200 as asp
from parity_util import np64
from test_gpu_cache8 import CODE, DEV, WIDE, Cache, _built, attend_ref, check, gen, logit_bound  # noqa: F401

pytestmark = pytest.mark.gpu


def uniform_case(fmt, qd, T, logit, seed, G=2, unit=2.0 ** -7):
    """(cache, q, best rows): natural logits `logit` on every third row, and twice or half of it, below,
    elsewhere.  Keys are codes times `unit`."""
    lens = [T, max(1, T - 5), 1]
    c = Cache(fmt, 3, 2, 64, T, lens, 0, 16, seed=seed, odd_scales=seed % 2 == 1, spread=2.0)
    k, ks = c.side["k"]
    best, other = (64.0, 32.0) if logit > 0 else (-32.0, -64.0)
    val = torch.full((T,), other)
    val[0::3] = best
    k.view(torch.uint8).zero_()
    if fmt in CODE:
        ks.fill_(unit)
        k[..., 0] = val.to(CODE[fmt]).to(DEV)
    else:
        k[..., 0] = (val * unit).to(WIDE[fmt]).to(DEV)
    q = torch.zeros(3, 2 * G, 64)
    q[..., 0] = abs(logit) * 8 / (abs(best) * unit)
    return c, q.to(WIDE[qd]).to(DEV), lens


def run(c, q, lens, T, accumulate):
    G = q.shape[1] // 2
    out = torch.full(q.shape, float("nan"), dtype=q.dtype if c.fmt in CODE else WIDE[c.fmt], device=DEV)
    lse = torch.full(q.shape[:2], float("nan"), device=DEV)
    acc = torch.zeros(3, 2, T, device=DEV)
    tb = torch.zeros(3, dtype=torch.int32, device=DEV)
    if accumulate:
        ws = torch.full((asp.accumulate_workspace_bytes(c.kv, 2 * G, 0, T),), 255, dtype=torch.uint8, device=DEV)
        asp.attend_accumulate(q, c.kv, None, None, 0, out, acc, lse, tail_begin=tb, max_tail=T, workspace=ws)
    else:
        ws = torch.full((max(16, asp.attend_workspace_bytes_kv(c.kv, 2 * G, 0, T)),), 255, dtype=torch.uint8, device=DEV)
        asp.sparse_attend(q, c.kv, None, None, 0, out, lse, tail_begin=tb, max_tail=T, workspace=ws)
    assert asp.device_status() == 0
    return np64(out.float()), np64(lse), np64(acc)


def check_uniform(c, q, lens, T, accumulate):
    out, lse, acc = run(c, q, lens, T, accumulate)
    G = q.shape[1] // 2
    one = c.fmt in CODE and q.dtype == torch.bfloat16
    eps = 2.0 ** -8 if (q.dtype if c.fmt in CODE else WIDE[c.fmt]) == torch.bfloat16 else 2.0 ** -22
    for b, n in enumerate(lens):
        K, V, vs = c.rows("k", b), c.rows("v", b), c.row_scales("v", b)
        S = np.arange(0, n, 3)
        for h in range(2):
            w = 1 / len(S)
            o, mag = V[h][S].mean(axis=0), np.abs(V[h][S]).mean(axis=0)
            ob = (2.0 ** -19 + 18 * n / 16 * 2.0 ** -23 + (2.0 ** -11 if one else 2.0 ** -18)) * mag + eps * np.abs(o) + 1e-30
            if vs[h] is not None:
                ob = ob + 2.0 ** -38 * w * vs[h][S].max() * (np.abs(V[h][S]) / vs[h][S, None]).sum(axis=0)
            for g in range(h * G, (h + 1) * G):
                check(out[b, g], o, ob, f"out b{b} head {g}")
                x, D = logit_bound(np64(q[b, g:g + 1].float()), K[h])
                ref = x[0].max() + np.log(len(S))
                check(lse[b, g:g + 1], np.array([ref]), np.array([D[0].max() + 2.0 ** -19 + 2.0 ** -21 * abs(ref)]), f"lse b{b}")
            if accumulate:
                full = np.zeros(T)
                full[S] = G * w
                check(acc[b, h], full, full * (2.0 ** -19 + n / 16 * 2.0 ** -23) + 1e-30, f"acc b{b} h{h}")


LOGITS = [9e6, -9e6, 1.2e7, 2.1e7, -2.1e7, 2.0 ** 25 + 64, 1e8, -1e8, 1.9e8, 1e12, -1e12, 1e30, -1e30]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("qd", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 40, 700, 6000])
@pytest.mark.parametrize("accumulate", [False, True])
def test_large_logits_8bit(fmt, qd, T, accumulate):
    for i, logit in enumerate(LOGITS):
        c, q, lens = uniform_case(fmt, qd, T, logit, seed=T + i)
        check_uniform(c, q, lens, T, accumulate)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_logits_next_to_the_lowest_float(fmt):
    """The best logit is -2.2e38 (-3.2e38 in base 2); the others overflow to -inf."""
    for T in (1, 40, 700):
        c, q, lens = uniform_case(fmt, "f32", T, -2.2e38, seed=T, unit=1.0)
        check_uniform(c, q, lens, T, True)


@pytest.mark.parametrize("qd", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 40, 700])
def test_large_logits_bf16_cache(qd, T):
    for i, logit in enumerate(LOGITS):
        c, q, lens = uniform_case("bf16", qd, T, logit, seed=T + i)
        check_uniform(c, q, lens, T, True)


@pytest.mark.parametrize("qd", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 40, 700])
def test_large_logits_fp32_cache(qd, T):
    for i, logit in enumerate(LOGITS):
        c, q, lens = uniform_case("f32", qd, T, logit, seed=T + i)
        check_uniform(c, q, lens, T, True)


@pytest.mark.parametrize("fmt", ["e4m3", "int8", "bf16", "f32"])
@pytest.mark.parametrize("T", [40, 500, 900])
@pytest.mark.parametrize("G", [2, 8])
def test_sums_where_one_heads_logit_overflows(fmt, T, G):
    """Head 0's logit of one row is -inf: the other heads' weights of that row still count."""
    c = Cache(fmt, 1, 1, 64, T, [T], 0, 16, seed=T)
    k, ks = c.side["k"]
    if ks is not None:
        ks.fill_(2.0 ** -6)
    k[..., 0] = 0
    r = T - 7
    k[0, 0, r, 0] = 64.0 if fmt in CODE else 1.0
    if ks is not None:
        ks[0, 0, r // 16] = 1.0
    K = c.rows("k", 0)[0]
    q = torch.randn(1, G, 64, generator=gen(5))
    q[..., 0] = 0
    q[0, 0] = 0
    q[0, 0, 0] = -1.9375 * 2.0 ** 127      # one part in bf16 and fp16
    if fmt not in CODE:        # a wide cache's keys are not scaled: one of 2^12 overflows
        k[0, 0, r, 0] = 2.0 ** 12
        K = c.rows("k", 0)[0]
    out = torch.empty(1, G, 64, dtype=torch.float32 if fmt != "bf16" else torch.bfloat16, device=DEV)
    lse, acc = torch.empty(1, G, device=DEV), torch.zeros(1, 1, T, device=DEV)
    tb = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.empty(asp.accumulate_workspace_bytes(c.kv, G, 0, T), dtype=torch.uint8, device=DEV)
    asp.attend_accumulate(q.to(DEV), c.kv, None, None, 0, out, acc, lse, tail_begin=tb, max_tail=T, workspace=ws)
    _, _, _, _, w, wb = attend_ref(np64(q[0, 1:]), K, c.rows("v", 0)[0], np.arange(T), False, 2.0 ** -8)
    w0 = np.full(T, 1 / (T - 1))      # head 0: equal logits on the other rows
    w0[r] = 0
    check(np64(acc[0, 0]), w + w0, wb + w0 * (2.0 ** -19 + T / 16 * 2.0 ** -23) + 2.0 ** -23 * (w + w0), "acc")
    assert np.isfinite(np64(lse)).all()
