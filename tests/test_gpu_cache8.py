"""The 8-bit cache, the attention that sums weights and the eviction, against float64 (GPU).

Bounds, derived once.  One logit x = q . k s / sqrt(d): products are exact, the fp32 sum of d
terms over d / 16 matrix steps of at most 17 additions errs by at most 17 (d / 16) 2^-23 of
A = sum |q_c k_c| s / sqrt(d) (additions that truncate), the parts of the query by 2^-21 of
its largest channel times sum |k_c| s / sqrt(d) <= B, and the factors (scales, 1 / sqrt(d)) by
2^-21 |x|:   D = 17 (d / 16) 2^-23 A + 2^-21 B + 2^-21 A.
A softmax weight then errs by at most e^(2 D) - 1 relative, plus 2^-19 for its exponentials and
sums (ex2.approx within 2^-22, a few of them, the sum over n rows by n / 16 2^-23), and the
output by that times sum w |v|, the fp32 sum over the rows (17 n / 16 2^-23) and, where the
weights are one fp16 part, 2^-11 of them; a bf16 output adds half a step, 2^-8.
fp16 also has a smallest step, 2^-24.  An 8-bit cache's weight times V's scale, w_j s_j, is held as
u_j = 2^(x_j + e_j - M + 14) mant_j with M = ceil(max(x_j + e_j)): at the row of that maximum
x + e - M > -1, so max u > 2^13, and rounding to a multiple of 2^-24 moves any u_j by at most
2^-25 < 2^-38 max u.  On the output that is at most 2^-38 max(w s) sum_j |code_j|.
"""
import math

import numpy as np
import pytest
import torch

import query_predicted_token_b200 as asp
from oracle import cache8
from parity_util import assert_valid_topk, np64

pytestmark = pytest.mark.gpu
DEV = "cuda"
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
WIDE = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from query_predicted_token_b200 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    asp.lib()
    asp.device_status()
    yield
    assert asp.device_status() == 0


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


class Cache:
    """A cache of any type on the GPU with a host view of its values."""

    def __init__(self, fmt, B, Hkv, d, T, lens, page=0, block=32, seed=0, src=torch.bfloat16, odd_scales=False,
                 spread=0.5):
        g = gen(seed)
        self.fmt, self.B, self.Hkv, self.d, self.T, self.page, self.block = fmt, B, Hkv, d, T, page, block
        self.lens = list(lens)
        N, L = (B, T) if not page else (sum(-(-max(n, 1) // page) for n in lens) + 3, page)
        shape = (N, Hkv, L, d)
        self.table = None
        if page:
            perm = torch.randperm(N, generator=g).to(torch.int32)
            self.table = torch.full((B, -(-T // page)), -1, dtype=torch.int32)
            at = 0
            for b, n in enumerate(lens):
                m = -(-max(n, 1) // page)
                self.table[b, :m] = perm[at:at + m]
                at += m
            self.free = perm[at:].tolist()
        self.side = {}
        for s in ("k", "v"):
            if fmt in WIDE:
                self.side[s] = (torch.randn(shape, generator=g).to(WIDE[fmt]).to(DEV), None)
                continue
            nb = -(-L // block)
            if fmt == "int8":
                code = torch.randint(-127, 128, shape, generator=g).to(torch.int8)
            else:
                code = (torch.randn(shape, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
            e = spread * torch.randn(N, Hkv, nb, generator=g) - (6 if fmt == "int8" else 5)
            sc = torch.exp2(e if odd_scales else e.round())
            self.side[s] = (code.to(DEV), sc.to(DEV))
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        ks, vs = self.side["k"][1], self.side["v"][1]
        self.table_dev = self.table.to(DEV) if page else None
        self.kv = asp.KV(self.side["k"][0], self.side["v"][0], self.seq_lens, self.table_dev, t_max=T, k_scale=ks,
                         v_scale=vs, scale_block=block if fmt in CODE else 0, src_dtype=src)

    def rows(self, s, b, n=None):
        """Sequence b's first n rows as float64 values [Hkv, n, d]."""
        codes, scales = self.codes(s, b, n)
        return codes if scales is None else codes * np.repeat(scales, self.block, axis=1)[:, :codes.shape[1], None]

    def row_scales(self, s, b, n=None):
        codes, scales = self.codes(s, b, n)
        return [None] * self.Hkv if scales is None else np.repeat(scales, self.block, axis=1)[:, :codes.shape[1]]

    def codes(self, s, b, n=None):
        n = int(self.seq_lens[b]) if n is None else n
        x, sc = self.side[s]
        if self.page:
            m = -(-n // self.page)
            pages = self.table[b, :m].long()
            if not m:
                return np.zeros((self.Hkv, 0, self.d)), None if sc is None else np.zeros((self.Hkv, 0))
            x = torch.cat([x[p] for p in pages], dim=1)
            sc = None if sc is None else torch.cat([sc[p] for p in pages], dim=1)
        else:
            x, sc = x[b], None if sc is None else sc[b]
        return np64(x[:, :n].float()), None if sc is None else np64(sc)[:, :-(-n // self.block)]


def logit_bound(q, K):
    """D of the module's docstring, q [G, d], K [n, d] -> (logits, D) [G, n]."""
    d = q.shape[-1]
    x = q @ K.T / math.sqrt(d)
    A = np.abs(q) @ np.abs(K).T / math.sqrt(d)
    Bq = np.abs(q).max(axis=1, keepdims=True) * np.abs(K).sum(axis=1)[None] / math.sqrt(d)
    return x, 17 * (d / 16) * 2.0 ** -23 * A + 2.0 ** -21 * Bq + 2.0 ** -21 * A


def attend_ref(q, K, V, S, one_part, out_eps, vs=None):
    """vs: V's scale per row (8-bit caches).  (out, out bound, lse, lse bound, summed weights, their bound) of a group."""
    G, d = q.shape
    if len(S) == 0:
        z = np.zeros
        return z((G, d)), z((G, d)), np.full(G, -np.inf), z(G), z(K.shape[0]), z(K.shape[0])
    x, D = logit_bound(q, K[S])
    m = x.max(axis=1, keepdims=True)
    e = np.exp(x - m)
    w = e / e.sum(axis=1, keepdims=True)
    n = len(S)
    dmax = D.max(axis=1, keepdims=True)
    rel = np.expm1(2 * dmax) + 2.0 ** -19 + n / 16 * 2.0 ** -23
    o = w @ V[S]
    mag = w @ np.abs(V[S])
    ob = (rel + 17 * n / 16 * 2.0 ** -23 + (2.0 ** -11 if one_part else 2.0 ** -18)) * mag + out_eps * np.abs(o) + 1e-30
    if vs is not None:
        ob = ob + 2.0 ** -38 * (w * vs[S]).max(axis=1, keepdims=True) * (np.abs(V[S]) / vs[S, None]).sum(axis=0)
    lse = m[:, 0] + np.log(e.sum(axis=1))
    lb = dmax[:, 0] + 2.0 ** -19 + n / 16 * 2.0 ** -23 + 2.0 ** -22 * np.abs(lse)
    acc, accb = np.zeros(K.shape[0]), np.zeros(K.shape[0])
    acc[S] = w.sum(axis=0)
    accb[S] = (w * rel).sum(axis=0) + 1e-30
    return o, ob, lse, lb, acc, accb


def check(got, ref, bound, what):
    err = np.abs(got - ref)
    bad = err > bound
    assert np.isfinite(got).all() and not bad.any(), \
        f"{what}: {bad.sum()} out of bounds, worst {np.max(err - bound):.3e} at error {err[bad][:3]}, bound {bound[bad][:3]}"


# ---- filling and reading back ---------------------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("src", ["bf16", "f32"])
@pytest.mark.parametrize("d,page,block", [(64, 0, 16), (128, 0, 64), (128, 0, 128), (64, 32, 32), (128, 16, 16),
                                          (128, 128, 64)])
def test_quantize_matches_the_definition_bit_for_bit(fmt, src, d, page, block):
    lens, T, H = [0, 1, block - 1, block, 197], 200, 3
    c = Cache(fmt, len(lens), H, d, T, lens, page, block, seed=d + page)
    before = {s: (c.side[s][0].view(torch.uint8).clone(), c.side[s][1].clone()) for s in "kv"}
    g = gen(7)
    # values of every size: normal ones, whole blocks of zeros, tiny, subnormal and huge rows; and a projection's
    # layout [batch, token, head, channel], one row longer than the longest sequence
    x = torch.randn(2, 5, T + 1, H, d, generator=g) * torch.exp2(torch.randint(-20, 20, (2, 5, T + 1, H, 1), generator=g).float())
    x[:, :, 16:32] = 0
    x[:, 4, 64:70] = 1e-39
    x[:, 4, 128:130] = 3.3e38
    x = x.to(WIDE[src]).to(DEV)
    k, v = x[0].transpose(1, 2), x[1].transpose(1, 2)
    asp.quantize_kv(c.kv, k, v)
    kd = torch.full((5, H, T, d), -7.0, device=DEV)
    vd = torch.full((5, H, T, d), -7.0, device=DEV)
    asp.dequantize_kv(c.kv, kd, vd)
    kb = torch.full((5, T, H, d), -7.0, device=DEV, dtype=torch.bfloat16)
    vb = torch.full((5, T, H, d), -7.0, device=DEV, dtype=torch.bfloat16)
    asp.dequantize_kv(c.kv, kb.transpose(1, 2), vb.transpose(1, 2))
    assert asp.device_status() == 0
    for s, src_t, wide, half in (("k", k, kd, kb), ("v", v, vd, vb)):
        for b, n in enumerate(lens):
            codes, scales = c.codes(s, b)
            for h in range(H):
                rc, rs = cache8.quantize(np64(src_t[b, h, :n].float()), block, fmt)
                assert np.array_equal(scales[h], rs)
                assert np.array_equal(codes[h], rc)
                val = rc * np.repeat(rs, block)[:n, None]
                with np.errstate(over="ignore"):      # a code next to fp32's largest value may stand for 2^128
                    val = val.astype(np.float32).astype(np.float64)
                assert np.array_equal(np64(wide[b, h, :n]), val)
                assert np.array_equal(np64(half[b, :n, h].float()), np64(torch.from_numpy(val).float().bfloat16().float()))
            assert (wide[b, :, n:] == -7).all() and (half[b, n:] == -7).all()
    # nothing else of the cache was written
    for s in "kv":
        code, scale = before[s]
        now = c.side[s][0].view(torch.uint8)
        live = torch.zeros_like(code, dtype=torch.bool)
        live_s = torch.zeros_like(scale, dtype=torch.bool)
        for b, n in enumerate(lens):
            for t in range(n):
                p, r = (int(c.table[b, t // page]), t % page) if page else (b, t)
                live[p, :, r] = True
                live_s[p, :, r // block] = True
        assert torch.equal(now[~live], code[~live])
        assert torch.equal(c.side[s][1][~live_s], scale[~live_s])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_infinities_and_nan_saturate_and_are_flagged(fmt):
    c = Cache(fmt, 1, 1, 64, 32, [20], block=16)
    x = torch.randn(1, 1, 32, 64, generator=gen(1)).to(DEV)
    x[0, 0, 3, 5], x[0, 0, 3, 6], x[0, 0, 17, 0] = float("inf"), float("-inf"), float("nan")
    y = x.clone()
    asp.quantize_kv(c.kv, x, x.clone())
    assert asp.device_status() == asp.ASP_DEV_NONFINITE
    codes, scales = c.codes("k", 0)
    y[0, 0, 3, 5:7] = 0
    y[0, 0, 17, 0] = 0
    rc, rs = cache8.quantize(np64(y[0, 0, :20]), 16, fmt)     # the finite values set the scales
    q = cache8.QMAX[fmt]
    assert np.array_equal(scales[0], rs)
    assert codes[0][3, 5] == q and codes[0][3, 6] == -q
    assert np.isnan(codes[0][17, 0]) if fmt == "e4m3" else codes[0][17, 0] == 0
    codes[0][3, 5:7] = 0
    codes[0][17, 0] = 0
    assert np.array_equal(codes[0], rc)
    # rows past the length, NaN or not, do not matter
    x2 = torch.randn(1, 1, 32, 64, generator=gen(1)).to(DEV)
    x2[0, 0, 20:] = float("nan")
    asp.quantize_kv(c.kv, x2, x2)
    assert asp.device_status() == 0


def test_bad_pages_are_skipped_and_flagged():
    c = Cache("e4m3", 2, 2, 64, 64, [60, 40], page=16, block=16)
    c.table_dev[0, 1] = 10 ** 6
    c.table_dev[1, 0] = -1
    x = torch.randn(2, 2, 64, 64, generator=gen(3)).to(DEV)
    asp.quantize_kv(c.kv, x, x)
    assert asp.device_status() == asp.ASP_DEV_BAD_PAGE
    y = torch.full((2, 2, 64, 64), -7.0, device=DEV)
    asp.dequantize_kv(c.kv, y, y.clone())
    assert asp.device_status() == asp.ASP_DEV_BAD_PAGE
    assert (y[0, :, 16:32] == -7).all() and (y[1, :, :16] == -7).all() and (y[0, :, :16] != -7).any()
    q = torch.randn(2, 4, 64, generator=gen(4)).to(DEV)
    s = torch.empty(2, 2, 64, device=DEV)
    asp.score_keys(q, c.kv, s)
    assert asp.device_status() == asp.ASP_DEV_BAD_PAGE
    out, acc = torch.empty(2, 4, 64, device=DEV), torch.zeros(2, 2, 64, device=DEV)
    zero = torch.zeros(2, dtype=torch.int32, device=DEV)
    ws = torch.empty(asp.accumulate_workspace_bytes(c.kv, 4, 0, 64), dtype=torch.uint8, device=DEV)
    asp.attend_accumulate(q, c.kv, None, None, 0, out, acc, tail_begin=zero, max_tail=64, workspace=ws)
    assert asp.device_status() == asp.ASP_DEV_BAD_PAGE
    assert (acc[0, :, 16:32] == 0).all() and (acc[1, :, :16] == 0).all()
    assert torch.allclose(acc.sum(-1), torch.full((2, 2), 2.0, device=DEV), atol=1e-4)
    c.seq_lens.copy_(torch.tensor([20, 5], dtype=torch.int32))
    new = torch.randn(2, 2, 64, generator=gen(5)).to(torch.bfloat16).to(DEV)
    asp.append_kv(c.kv, new, new)
    assert asp.device_status() == asp.ASP_DEV_BAD_PAGE
    assert c.seq_lens.tolist() == [20, 5]


# ---- append -----------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("src", ["bf16", "f32"])
@pytest.mark.parametrize("d,page,block", [(64, 0, 16), (128, 16, 16), (128, 0, 128), (64, 64, 32)])
def test_append_token_by_token(fmt, src, d, page, block):
    H, T = 9, 70          # more heads and sides than a CTA has warps
    lens = [0, 13, 31, 70]
    c = Cache(fmt, 4, H, d, T, [40, 60, 70, 70], page, block, seed=3, src=WIDE[src])
    c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    ref = {(s, b, h): [a[h] for a in c.codes(s, b)] for s in "kv" for b in range(4) for h in range(H)}
    tail = torch.full((4,), -1, dtype=torch.int32, device=DEV)
    g = gen(11)
    for step in range(20):
        x = torch.randn(2, 4, H, d, generator=g) * torch.exp2(torch.randint(-9, 5, (2, 4, H, 1), generator=g).float())
        if step == 5:
            x[0] = 0
        x = x.to(WIDE[src]).to(DEV)
        asp.append_kv(c.kv, x[0], x[1], tail)
        assert asp.device_status() == asp.ASP_DEV_BAD_PAGE       # the last sequence is at its capacity
        assert tail.tolist()[:3] == [n + step for n in lens[:3]]
        assert c.seq_lens.tolist() == [n + step + 1 for n in lens[:3]] + [70]
        for (s, b, h), (codes, scales) in ref.items():
            if b < 3:
                ref[s, b, h] = list(cache8.append(codes, scales, np64(x["kv".index(s), b, h].float()), block, fmt))
    for s in "kv":
        for b in range(4):
            codes, scales = c.codes(s, b)
            for h in range(H):
                assert np.array_equal(scales[h], ref[s, b, h][1]), (s, b, h)
                assert np.array_equal(codes[h], ref[s, b, h][0]), (s, b, h)


# ---- the key scan -----------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("page,block", [(0, 32), (16, 16), (48, 16), (256, 128)])
def test_score_keys(fmt, d, G, page, block):
    lens, H, T = [1000, 0, 517, 1, 33], 2, 1003
    c = Cache(fmt, 5, H, d, T, lens, page, block, seed=G + d, odd_scales=True, spread=4.0)
    q = torch.randn(5, H * G, d, generator=gen(5)) * torch.exp2(torch.randint(-30, 10, (5, H * G, 1), generator=gen(6)).float())
    q[0, 0] = 0
    q = q.to(DEV)
    scores = torch.full((5, H, T), float("nan"), device=DEV)
    asp.score_keys(q, c.kv, scores)
    assert asp.device_status() == 0
    got = np64(scores)
    for b, n in enumerate(lens):
        K = c.rows("k", b)
        for h in range(H):
            x, D = logit_bound(np64(q[b, h * G:(h + 1) * G]), K[h])
            if n:
                check(got[b, h, :n], x.max(axis=0), D.max(axis=0) + 1e-37, f"b{b} h{h}")
            assert np.isnan(got[b, h, n:]).all()


def test_score_keys_of_many_short_sequences():
    lens = [int(n) for n in np.random.default_rng(3).integers(0, 41, 300)]
    c = Cache("int8", 300, 3, 64, 41, lens, 16, 16, seed=2)
    q = torch.randn(300, 6, 64, generator=gen(5)).to(DEV)
    scores = torch.full((300, 3, 41), float("nan"), device=DEV)
    asp.score_keys(q, c.kv, scores)
    got = np64(scores)
    for b, n in enumerate(lens):
        K = c.rows("k", b)
        for h in range(3):
            if n:
                x, D = logit_bound(np64(q[b, 2 * h:2 * h + 2]), K[h])
                check(got[b, h, :n], x.max(axis=0), D.max(axis=0), f"b{b} h{h}")
            assert np.isnan(got[b, h, n:]).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_score_keys_of_the_largest_batch(fmt):
    """8192 sequences: the lengths in shared memory leave room for fewer stages."""
    B, T, d = 8192, 40, 128
    lens = [int(n) for n in np.random.default_rng(4).integers(0, T + 1, B)]
    c = Cache(fmt, B, 1, d, T, lens, 0, 32, seed=2)
    q = torch.randn(B, 2, d, generator=gen(5)).to(DEV)
    scores = torch.full((B, 1, T), float("nan"), device=DEV)
    asp.score_keys(q, c.kv, scores)
    assert asp.device_status() == 0
    live = torch.arange(T) < torch.tensor(lens)[:, None]
    got = scores[:, 0].cpu()
    assert torch.equal(torch.isnan(got), ~live)
    for b in range(0, B, 97):
        if lens[b]:
            x, D = logit_bound(np64(q[b]), c.rows("k", b)[0])
            check(np64(got[b, :lens[b]]), x.max(axis=0), D.max(axis=0), f"b{b}")


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_nan_and_infinite_queries_reach_the_scores(fmt):
    """A head whose query is not finite gives scores that are not finite; its neighbours' stay."""
    c = Cache(fmt, 1, 4, 128, 50, [50], 0, 16, seed=2)
    q = torch.randn(1, 4, 128, generator=gen(5)).to(DEV)
    clean = torch.empty(1, 4, 50, device=DEV)
    asp.score_keys(q, c.kv, clean)
    q[0, 1, 3], q[0, 2, 100] = float("nan"), float("inf")
    scores = torch.empty(1, 4, 50, device=DEV)
    asp.score_keys(q, c.kv, scores)
    assert not torch.isfinite(scores[0, 1:3]).any()
    assert torch.equal(scores[0, [0, 3]], clean[0, [0, 3]])


# ---- attention and summed weights ---------------------------------------------------------------------------------------

def selection(B, H, C, lens, tails, seed):
    """Distinct random indices (ascending, -1 past the count), some inside the tail."""
    r = np.random.default_rng(seed)
    idx, cnt = np.full((B, H, max(C, 1)), -1, np.int32), np.zeros((B, H), np.int32)
    for b in range(B):
        for h in range(H):
            n = min(C, lens[b])
            n = 0 if n == 0 else int(r.integers(n // 2, n + 1))
            idx[b, h, :n] = np.sort(r.choice(lens[b], n, replace=False)) if n else []
            cnt[b, h] = n
    return idx, cnt


def run_attention(c, q, C, tail, seed, accumulate, lse=True):
    """Runs the call and checks out, lse and acc; tail: tokens before the end, None for none, "all" for dense."""
    B, Hq, d = q.shape
    H, G = c.Hkv, Hq // c.Hkv
    lens = c.seq_lens.tolist()
    tb = None if tail is None else [0 if tail == "all" else max(0, n - tail) for n in lens]
    idx, cnt = selection(B, H, C, lens, tb, seed)
    tbd = None if tb is None else torch.tensor(tb, dtype=torch.int32, device=DEV)
    mt = 0 if tail is None else (c.T if tail == "all" else tail)
    idxd, cntd = torch.from_numpy(idx).to(DEV), torch.from_numpy(cnt).to(DEV)
    odt = q.dtype if c.fmt in CODE else WIDE[c.fmt]
    out = torch.full((B, Hq, d), float("nan"), dtype=odt, device=DEV)
    ls = torch.full((B, Hq), float("nan"), device=DEV) if lse else None
    acc0 = torch.rand(B, H, c.T, generator=gen(seed)).to(DEV)
    acc = acc0.clone()
    args = (idxd if C else None, cntd if C else None, C, out)
    if accumulate:
        ws = torch.full((asp.accumulate_workspace_bytes(c.kv, Hq, C, mt),), 255, dtype=torch.uint8, device=DEV)
        asp.attend_accumulate(q, c.kv, *args, acc, ls, tail_begin=tbd, max_tail=mt, workspace=ws)
    else:
        ws = torch.full((max(16, asp.attend_workspace_bytes_kv(c.kv, Hq, C, mt)),), 255, dtype=torch.uint8, device=DEV)
        asp.sparse_attend(q, c.kv, *args, ls, tail_begin=tbd, max_tail=mt, workspace=ws)
    assert asp.device_status() == 0
    go, gl, ga, a0 = np64(out.float()), np64(ls) if lse else None, np64(acc), np64(acc0)
    for b in range(B):
        K, V, vs = c.rows("k", b), c.rows("v", b), c.row_scales("v", b)
        for h in range(H):
            S = cache8.attended_set(idx[b, h], int(cnt[b, h]) if C else 0, tb and tb[b], lens[b]) if tb else \
                np.unique(idx[b, h, :cnt[b, h]])
            hs = slice(h * G, (h + 1) * G)
            one = c.fmt in CODE and q.dtype == torch.bfloat16
            o, ob, l, lb, w, wb = attend_ref(np64(q[b, hs].float()), K[h], V[h], S.astype(np.int64), one,
                                             2.0 ** -8 if odt == torch.bfloat16 else 2.0 ** -22, vs[h])
            check(go[b, hs], o, ob, f"out b{b} h{h}")
            if lse:
                assert np.array_equal(np.isneginf(gl[b, hs]), np.isneginf(l))
                if len(S):
                    check(gl[b, hs], l, lb, f"lse b{b} h{h}")
            if accumulate:
                full, fb = np.zeros(c.T), np.zeros(c.T)
                full[:len(w)], fb[:len(w)] = w, wb
                out_of = np.ones(c.T, bool)
                out_of[S] = False
                assert np.array_equal(ga[b, h, out_of], a0[b, h, out_of])
                check(ga[b, h], a0[b, h] + full, fb + 2.0 ** -23 * (np.abs(a0[b, h]) + full), f"acc b{b} h{h}")
    return out, ls, acc


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("qd", ["bf16", "f32"])
@pytest.mark.parametrize("d,G", [(64, 1), (64, 8), (128, 2), (128, 4), (128, 8)])
@pytest.mark.parametrize("page,block", [(0, 64), (32, 16)])
@pytest.mark.parametrize("C,tail", [(0, "all"), (300, 3), (37, None)])
def test_attend_8bit(fmt, qd, d, G, page, block, C, tail):
    lens, H, T = [700, 0, 1, 40, 333], 2, 703
    c = Cache(fmt, 5, H, d, T, lens, page, block, seed=d + G, odd_scales=True)
    q = torch.randn(5, H * G, d, generator=gen(5)).to(WIDE[qd]).to(DEV)
    run_attention(c, q, C, tail, seed=C + G, accumulate=False)


@pytest.mark.parametrize("fmt", ["e4m3", "int8", "bf16", "f32"])
@pytest.mark.parametrize("qd", ["bf16", "f32"])
@pytest.mark.parametrize("d,G,page", [(64, 4, 0), (128, 8, 0), (128, 1, 16), (64, 2, 64)])
@pytest.mark.parametrize("C,tail", [(0, "all"), (100, 5), (500, 2), (64, None)])
def test_attend_accumulate(fmt, qd, d, G, page, C, tail):
    lens, H, T = [900, 0, 1, 130, 17], 3, 905
    c = Cache(fmt, 5, H, d, T, lens, page, 16, seed=d + G)
    q = torch.randn(5, H * G, d, generator=gen(5)).to(WIDE[qd]).to(DEV)
    run_attention(c, q, C, tail, seed=C + G, accumulate=True, lse=C != 100)


@pytest.mark.parametrize("fmt", ["e4m3", "bf16", "f32"])
@pytest.mark.parametrize("T", [1, 16, 250, 256, 257, 512, 513])
def test_short_caches(fmt, T):
    c = Cache(fmt, 2, 2, 128, T, [T, max(0, T - 1)], 0, 16, seed=T)
    q = torch.randn(2, 8, 128, generator=gen(5)).to(torch.bfloat16).to(DEV)
    run_attention(c, q, 0, "all", seed=T, accumulate=True)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("qd", ["bf16", "f32"])
def test_scales_far_apart_and_large_logits(fmt, qd):
    """Blocks of values 2^40 apart on either side: weights of the small ones keep their precision where the large
    ones' weights are nothing, and the other way round."""
    c = Cache(fmt, 2, 1, 128, 600, [600, 600], 0, 16, seed=9)
    ks, vs = c.side["k"][1], c.side["v"][1]
    vs[0, 0, 3] *= 2.0 ** 40           # a block of huge values ...
    ks[0, 0, 3] *= 64.0                # ... under logits far from the others'
    vs[1, 0, :20] *= 2.0 ** -50
    ks[1] *= 8.0
    q = torch.randn(2, 4, 128, generator=gen(5)).to(WIDE[qd]).to(DEV)
    run_attention(c, q, 0, "all", seed=1, accumulate=True)


def test_a_uniform_long_tail_is_not_lost():
    """One row with a weight 2^20 times the others': 40000 small weights still count."""
    T, d = 40001, 64
    c = Cache("e4m3", 1, 1, d, T, [T], 0, 64, seed=1)
    code, sc = c.side["k"]
    sc.fill_(1.0)
    c.side["v"][1].fill_(1.0)
    code.view(torch.uint8).zero_()
    q = torch.zeros(1, 2, d, device=DEV)
    q[..., 0] = 1.0
    code[0, 0, 777, 0] = torch.tensor(112.0).to(torch.float8_e4m3fn)      # logit 14 against 0
    v = c.side["v"][0]
    v.copy_((torch.rand(v.shape, generator=gen(2)) + 1).to(torch.float8_e4m3fn))
    for dt in (torch.float32, torch.bfloat16):
        run_attention(c, q.to(dt), 0, "all", seed=1, accumulate=True)


@pytest.mark.parametrize("fmt", ["e4m3", "int8", "bf16"])
def test_queries_off_the_16_byte_boundary(fmt):
    """A query tensor that starts at an odd element is read correctly."""
    c = Cache(fmt, 2, 2, 64, 700, [700, 9], 0, 16, seed=4)
    for dt in (torch.bfloat16, torch.float32):
        flat = torch.randn(2 * 8 * 64 + 1, generator=gen(5)).to(dt).to(DEV)
        q = flat[1:].view(2, 8, 64)
        assert q.data_ptr() % 16
        run_attention(c, q, 0, "all", seed=1, accumulate=True)


def test_many_captured_calls_back_to_back():
    """Unsynchronised calls in a row over ragged lengths and units shared by CTAs: each waits for the one before."""
    lens = [int(n) for n in np.random.default_rng(11).integers(1, 4000, 16)]
    c = Cache("bf16", 16, 4, 128, 4000, lens, 0, 16, seed=3)
    q = torch.randn(16, 16, 128, generator=gen(5)).to(torch.bfloat16).to(DEV)
    tb = torch.zeros(16, dtype=torch.int32, device=DEV)
    ws = torch.empty(asp.accumulate_workspace_bytes(c.kv, 16, 0, 4000), dtype=torch.uint8, device=DEV)
    out, lse, acc = (torch.empty(16, 16, 128, dtype=torch.bfloat16, device=DEV), torch.empty(16, 16, device=DEV),
                     torch.zeros(16, 4, 4000, device=DEV))
    call = lambda: asp.attend_accumulate(q, c.kv, None, None, 0, out, acc, lse, tail_begin=tb, max_tail=4000, workspace=ws)
    call()
    torch.cuda.synchronize()
    one, first = acc.clone(), out.clone()
    acc.zero_()
    for _ in range(40):
        call()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    # 40 additions of the same value: at most 39 roundings of half a step of the largest sum
    assert (acc - 40 * one).abs().max() <= 40 * 2.0 ** -24 * float(acc.max())
    for b in range(16):
        assert torch.allclose(one[b, :, :lens[b]].sum(-1), torch.full((4,), 4.0, device=DEV), rtol=1e-4)
        assert (one[b, :, lens[b]:] == 0).all()


def test_duplicate_free_selection_inside_the_tail_counts_once():
    c = Cache("int8", 1, 1, 64, 64, [50], 0, 16, seed=4)
    q = torch.randn(1, 2, 64, generator=gen(5)).to(DEV)
    idx = torch.tensor([[[3, 10, 45, 48]]], dtype=torch.int32, device=DEV)
    cnt = torch.tensor([[4]], dtype=torch.int32, device=DEV)
    tb = torch.tensor([44], dtype=torch.int32, device=DEV)
    out, acc = torch.empty(1, 2, 64, device=DEV), torch.zeros(1, 1, 64, device=DEV)
    ws = torch.empty(asp.accumulate_workspace_bytes(c.kv, 2, 4, 6), dtype=torch.uint8, device=DEV)
    asp.attend_accumulate(q, c.kv, idx, cnt, 4, out, acc, tail_begin=tb, max_tail=6, workspace=ws)
    S = np.array([3, 10, 44, 45, 46, 47, 48, 49])
    o, ob, _, _, w, wb = attend_ref(np64(q[0]), c.rows("k", 0)[0], c.rows("v", 0)[0], S, False, 2.0 ** -22)
    check(np64(out[0]), o, ob, "out")
    check(np64(acc[0, 0, :50]), w, wb, "acc")
    # an index outside the sequence is skipped and flagged
    idx[0, 0, 3] = 60
    asp.attend_accumulate(q, c.kv, idx, cnt, 4, out, acc.zero_(), tail_begin=tb, max_tail=6, workspace=ws)
    assert asp.device_status() == asp.ASP_DEV_BAD_INDEX
    check(np64(out[0]), o, ob, "out")
    # a tail longer than max_tail is cut and flagged
    asp.attend_accumulate(q, c.kv, None, None, 0, out, acc.zero_(), tail_begin=tb, max_tail=4, workspace=ws)
    assert asp.device_status() == asp.ASP_DEV_TAIL_LIMIT
    assert (acc[0, 0, 44:48] > 0).all() and (acc[0, 0, 48:] == 0).all()


@pytest.mark.parametrize("fmt", ["e4m3", "bf16"])
def test_many_units_and_equal_shares(fmt):
    """Hundreds of units of very different lengths: ranges that cut units, hold many, and empty units."""
    r = np.random.default_rng(5)
    lens = [int(n) for n in r.integers(0, 2, 150) * r.integers(0, 700, 150)]
    c = Cache(fmt, 150, 3, 64, 700, lens, 0, 32, seed=3)
    q = torch.randn(150, 6, 64, generator=gen(5)).to(torch.bfloat16).to(DEV)
    run_attention(c, q, 0, "all", seed=1, accumulate=True)


@pytest.mark.parametrize("accumulate", [False, True])
def test_two_streams_and_a_captured_call(accumulate):
    """Two calls at once on streams of their own, each with its workspace, and a captured and replayed call give
    what one call alone gives, bit for bit."""
    cs = [Cache("e4m3", 3, 2, 128, 2000, [2000, 700, 1], 0, 64, seed=s) for s in (1, 2)]
    qs = [torch.randn(3, 8, 128, generator=gen(s)).to(torch.bfloat16).to(DEV) for s in (1, 2)]
    tb = torch.zeros(3, dtype=torch.int32, device=DEV)

    def buffers(c):
        return (torch.empty(3, 8, 128, dtype=torch.bfloat16, device=DEV), torch.empty(3, 8, device=DEV),
                torch.zeros(3, 2, 2000, device=DEV),
                torch.empty(asp.accumulate_workspace_bytes(c.kv, 8, 0, 2000), dtype=torch.uint8, device=DEV))

    def call(i, buf):
        out, lse, acc, ws = buf
        if accumulate:
            asp.attend_accumulate(qs[i], cs[i].kv, None, None, 0, out, acc, lse, tail_begin=tb, max_tail=2000, workspace=ws)
        else:
            asp.sparse_attend(qs[i], cs[i].kv, None, None, 0, out, lse, tail_begin=tb, max_tail=2000, workspace=ws)

    alone = [buffers(c) for c in cs]
    for i in range(2):
        call(i, alone[i])
    torch.cuda.synchronize()
    both = [buffers(c) for c in cs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, s in enumerate(streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            call(i, both[i])
    torch.cuda.synchronize()
    graph_buf = buffers(cs[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(0, graph_buf)
    for _ in range(3):
        graph_buf[2].zero_()
        g.replay()
    torch.cuda.synchronize()
    for a, b in [(alone[0], both[0]), (alone[1], both[1]), (alone[0], graph_buf)]:
        for x, y in zip(a[:3], b[:3]):
            assert torch.equal(x, y)


# ---- eviction -----------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["e4m3", "int8", "bf16", "f32"])
@pytest.mark.parametrize("d,page,block", [(64, 0, 16), (128, 0, 64), (128, 32, 16), (64, 64, 32)])
@pytest.mark.parametrize("C,sink,recent", [(1, 0, 1), (100, 4, 30), (700, 0, 0), (130, 130, 0)])
def test_evict(fmt, d, page, block, C, sink, recent):
    lens, H, T = [1500, 0, 1, 700, 1031, C], 2, 1503
    c = Cache(fmt, 6, H, d, T, lens, page, block, seed=d + C, odd_scales=False)
    g = gen(C)
    acc = torch.rand(6, H, T, generator=g).pow_(6)
    acc[0] = (acc[0] * 20).round() / 20          # ties
    acc[4] = 0
    acc = acc.to(DEV)
    before = {s: [c.codes(s, b) for b in range(6)] for s in "kv"}
    raw = {s: c.side[s][0].view(torch.uint8).clone() for s in "kv"}
    idx = torch.full((6, H, C), 12345, dtype=torch.int32, device=DEV)
    cnt = torch.full((6, H), 12345, dtype=torch.int32, device=DEV)
    ws = torch.empty(asp.evict_workspace_bytes(c.kv, C), dtype=torch.uint8, device=DEV)
    in_place = C == 100
    acc_in = acc.clone()
    out = acc_in if in_place else torch.full_like(acc, -3.0)
    asp.evict_kv(c.kv, acc_in, C, idx, cnt, n_sink=sink, n_recent=recent, acc_out=None if in_place else out, workspace=ws)
    assert asp.device_status() == 0
    assert c.seq_lens.tolist() == [min(C, n) for n in lens]
    a = np64(acc)
    written = {s: torch.zeros(c.side[s][0].shape[:3], dtype=torch.bool) for s in "kv"}
    for b, n in enumerate(lens):
        for h in range(H):
            keep = cache8.kept_tokens(a[b, h, :n], n, C, sink, recent)
            m = len(keep)
            assert int(cnt[b, h]) == m
            assert np.array_equal(idx[b, h].cpu().numpy(), np.concatenate([keep, np.full(C - m, -1)]))
            assert np.array_equal(np64(out[b, h]), np.concatenate([a[b, h, keep], np.zeros(T - m)]))
            for s in "kv":
                codes, scales = c.codes(s, b)
                oc, osc = before[s][b]
                if n <= C:
                    assert np.array_equal(codes[h], oc[h][:m])
                    assert scales is None or np.array_equal(scales[h], osc[h])
                    continue
                for i in range(m):
                    p, r = (int(c.table[b, i // page]), i % page) if page else (b, i)
                    written[s][p, h, r] = True
                if fmt in WIDE:
                    assert np.array_equal(codes[h], oc[h][keep])
                else:
                    val = (oc[h] * np.repeat(osc[h], block)[:n, None])[keep]
                    rc, rs = cache8.quantize(val, block, fmt)
                    assert np.array_equal(scales[h], rs)
                    assert np.array_equal(codes[h], rc)
    for s in "kv":
        now = c.side[s][0].view(torch.uint8)
        keep = ~written[s].to(DEV)
        assert torch.equal(now[keep], raw[s][keep])


def test_evict_captured_and_repeated():
    """A captured eviction replayed on restored contents gives the same cache."""
    c = Cache("e4m3", 2, 2, 64, 400, [400, 90], 0, 16, seed=8)
    acc = torch.rand(2, 2, 400, generator=gen(1)).to(DEV)
    saved = [x.clone() for s in "kv" for x in (c.side[s][0].view(torch.uint8), c.side[s][1])] + [c.seq_lens.clone()]
    live = [x for s in "kv" for x in (c.side[s][0].view(torch.uint8), c.side[s][1])] + [c.seq_lens]
    idx, cnt = torch.empty(2, 2, 100, dtype=torch.int32, device=DEV), torch.empty(2, 2, dtype=torch.int32, device=DEV)
    out = torch.empty_like(acc)
    ws = torch.empty(asp.evict_workspace_bytes(c.kv, 100), dtype=torch.uint8, device=DEV)
    call = lambda: asp.evict_kv(c.kv, acc, 100, idx, cnt, 2, 20, out, ws)
    call()
    first = [x.clone() for x in live] + [idx.clone(), cnt.clone(), out.clone()]
    for x, y in zip(live, saved):
        x.copy_(y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(2):
        for x, y in zip(live, saved):
            x.copy_(y)
        g.replay()
    torch.cuda.synchronize()
    for x, y in zip(live + [idx, cnt, out], first):
        assert torch.equal(x, y)


def test_evict_flags_nan_sums_and_bad_pages():
    c = Cache("bf16", 1, 1, 64, 128, [100], page=16, block=16, seed=2)
    acc = torch.rand(1, 1, 128, generator=gen(1)).to(DEV)
    acc[0, 0, 7] = float("nan")
    idx, cnt = torch.empty(1, 1, 32, dtype=torch.int32, device=DEV), torch.empty(1, 1, dtype=torch.int32, device=DEV)
    ws = torch.empty(asp.evict_workspace_bytes(c.kv, 32), dtype=torch.uint8, device=DEV)
    asp.evict_kv(c.kv, acc, 32, idx, cnt, workspace=ws)
    assert asp.device_status() == asp.ASP_DEV_NAN_SCORE
    c.seq_lens.fill_(100)
    c.table_dev[0, 1] = -1
    acc = torch.rand(1, 1, 128, generator=gen(1)).to(DEV)
    old = c.codes("k", 0, 16)[0]
    asp.evict_kv(c.kv, acc, 32, idx, cnt, n_sink=16, workspace=ws)
    assert asp.device_status() == asp.ASP_DEV_BAD_PAGE
    assert np.array_equal(c.codes("k", 0, 16)[0], old)      # the sinks stay where they are


# ---- together -------------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("page,block", [(0, 64), (16, 16)])
def test_a_generation_in_a_bounded_8bit_cache(fmt, page, block):
    """Prompt in, then steps of append, dense attention with summed weights and, when the budget is passed, an
    eviction: codes, scales and lengths follow the oracle bit for bit given the device's sums; outputs stay in
    bounds."""
    B, H, G, d, T, C = 2, 2, 4, 64, 160, 64
    lens = [75, 150]
    c = Cache(fmt, B, H, d, T, [T, T], page, block, seed=1)
    c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    g = gen(21)
    prompt = torch.randn(2, B, H, T, d, generator=g).to(torch.bfloat16).to(DEV)
    asp.quantize_kv(c.kv, prompt[0], prompt[1])
    ref = {(s, b, h): list(cache8.quantize(np64(prompt[i, b, h, :lens[b]].float()), block, fmt))
           for i, s in enumerate("kv") for b in range(B) for h in range(H)}
    acc = torch.zeros(B, H, T, device=DEV)
    tail, zero = torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    idx, cnt = torch.empty(B, H, C, dtype=torch.int32, device=DEV), torch.empty(B, H, dtype=torch.int32, device=DEV)
    ws = torch.empty(asp.accumulate_workspace_bytes(c.kv, H * G, 0, T), dtype=torch.uint8, device=DEV)
    wse = torch.empty(asp.evict_workspace_bytes(c.kv, C), dtype=torch.uint8, device=DEV)
    out, lse = torch.empty(B, H * G, d, dtype=torch.bfloat16, device=DEV), torch.empty(B, H * G, device=DEV)
    for step in range(8):
        new = (torch.randn(2, B, H, d, generator=g) * 2.0 ** step).to(torch.bfloat16).to(DEV)
        q = torch.randn(B, H * G, d, generator=g).to(torch.bfloat16).to(DEV)
        asp.append_kv(c.kv, new[0], new[1], tail)
        for (s, b, h), (cs, sc) in ref.items():
            ref[s, b, h] = list(cache8.append(cs, sc, np64(new["kv".index(s), b, h].float()), block, fmt))
        asp.attend_accumulate(q, c.kv, None, None, 0, out, acc, lse, tail_begin=zero, max_tail=T, workspace=ws)
        val = {k: cs * np.repeat(sc, block)[:len(cs), None] for k, (cs, sc) in ref.items()}
        for b in range(B):
            for h in range(H):
                hs = slice(h * G, (h + 1) * G)
                n = len(val["k", b, h])
                o, ob, l, lb, _, _ = attend_ref(np64(q[b, hs].float()), val["k", b, h], val["v", b, h], np.arange(n), True,
                                                2.0 ** -8, np.repeat(ref["v", b, h][1], block)[:n])
                check(np64(out[b, hs].float()), o, ob, f"step {step} out")
                check(np64(lse[b, hs]), l, lb, f"step {step} lse")
        if step % 4 == 3:
            a = np64(acc)
            asp.evict_kv(c.kv, acc, C, idx, cnt, n_sink=2, n_recent=8, workspace=wse)
            for (s, b, h), (cs, sc) in ref.items():
                n = len(cs)
                keep = cache8.kept_tokens(a[b, h, :n], n, C, 2, 8)
                if n > C:
                    ref[s, b, h] = list(cache8.quantize(val[s, b, h][keep], block, fmt))
                if s == "k":
                    assert np.array_equal(idx[b, h, :len(keep)].cpu().numpy(), keep)
                    assert np.array_equal(np64(acc[b, h, :len(keep)]), a[b, h, keep])
    assert asp.device_status() == 0
    for (s, b, h), (cs, sc) in ref.items():
        codes, scales = c.codes(s, b)
        assert np.array_equal(codes[h], cs) and np.array_equal(scales[h], sc)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("page,block", [(0, 32), (16, 16)])
def test_decode_steps_on_an_8bit_cache(fmt, page, block):
    """The asynchronous decode step with appends: every step's output over the previous selection and the tail,
    scores and selection of the step, and captured replays equal to eager steps."""
    B, H, G, d, T, C, W = 3, 2, 4, 128, 900, 64, 8
    lens = [800, 333, 50]

    def fresh():
        c = Cache(fmt, B, H, d, T, [T] * B, page, block, seed=1)
        c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        g = gen(31)
        qhist = torch.randn(B, H * G, W + 1, d, generator=g).to(DEV).contiguous()
        idx0, cnt0 = selection(B, H, C, lens, None, 3)
        tail = torch.zeros(B, dtype=torch.int32, device=DEV)
        st = asp.DecodeState(c.kv, H * G, asp.PredCfg(W, (4, 8), 1e-2), C, qhist, max_tail=2, tail_begin=tail)
        st.set_selection(torch.from_numpy(idx0).to(DEV), torch.from_numpy(cnt0).to(DEV))
        return c, st, tail

    steps = 20
    g = gen(41)
    new = (torch.randn(steps, 2, B, H, d, generator=g)).to(torch.bfloat16).to(DEV)
    qs = torch.randn(steps, B, H * G, d, generator=g).to(torch.bfloat16).to(DEV)
    c, st, tail = fresh()
    out, lse = torch.empty(B, H * G, d, dtype=torch.bfloat16, device=DEV), torch.empty(B, H * G, device=DEV)
    eager = []
    for i in range(steps):
        idx, cnt = (t.cpu().numpy().copy() for t in st.selection)
        st.step(qs[i], out, lse, new[i, 0], new[i, 1])
        assert asp.wait_selection(st.ev_sel_done, 60_000_000) == 0
        torch.cuda.synchronize()
        n = [m + i + 1 for m in lens]
        assert c.seq_lens.tolist() == n and tail.tolist() == [m - 1 for m in n]
        idx1, cnt1 = (t.cpu().numpy() for t in st.selection)
        scores = st.scores.cpu().numpy()
        pred = np64(st.qpred)
        for b in range(B):
            K, V = c.rows("k", b), c.rows("v", b)
            for h in range(H):
                hs = slice(h * G, (h + 1) * G)
                S = cache8.attended_set(idx[b, h], int(cnt[b, h]), n[b] - 1, n[b])
                o, ob, l, lb, _, _ = attend_ref(np64(qs[i, b, hs].float()), K[h], V[h], S, True, 2.0 ** -8)
                check(np64(out[b, hs].float()), o, ob, f"step {i} out")
                check(np64(lse[b, hs]), l, lb, f"step {i} lse")
                x, D = logit_bound(pred[b, hs], K[h])
                check(scores[b, h, :n[b]].astype(np.float64), x.max(axis=0), D.max(axis=0), f"step {i} scores")
                assert_valid_topk(scores[b, h], n[b], C, idx1[b, h], int(cnt1[b, h]), f"step {i}")
        eager.append((out.clone(), lse.clone(), st.idx[st.cur].clone()))
    assert asp.device_status() == 0
    c, st, tail = fresh()
    q_in, k_in, v_in = torch.empty_like(qs[0]), torch.empty_like(new[0, 0]), torch.empty_like(new[0, 1])
    st.step(qs[0], out, lse, new[0, 0], new[0, 1])
    torch.cuda.synchronize()
    st.capture(q_in, out, lse, k_in, v_in)
    for i in range(1, steps):
        q_in.copy_(qs[i])
        k_in.copy_(new[i, 0])
        v_in.copy_(new[i, 1])
        st.replay()
        torch.cuda.synchronize()
        for x, y in zip((out, lse, st.idx[st.cur]), eager[i]):
            assert torch.equal(x, y), i
    st.release_graphs()
    assert asp.device_status() == 0


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes per side: the last sequence's rows."""
    B, H, T, d = 5, 8, 900_000, 128
    assert B * H * T * d > 1 << 32
    k = torch.zeros(B, H, T, d, dtype=torch.int8, device=DEV)
    v = torch.zeros_like(k)
    nb = -(-T // 64)
    ks, vs = torch.full((B, H, nb), 2.0 ** -6, device=DEV), torch.full((B, H, nb), 2.0 ** -5, device=DEV)
    n = 300
    g = gen(3)
    rows = torch.randint(-127, 128, (2, H, n, d), generator=g).to(torch.int8).to(DEV)
    k[B - 1, :, T - n:], v[B - 1, :, T - n:] = rows[0], rows[1]
    lens = torch.tensor([0, 5, 0, 0, T], dtype=torch.int32, device=DEV)
    kv = asp.KV(k, v, lens, k_scale=ks, v_scale=vs, scale_block=64, src_dtype=torch.float32)
    q = torch.randn(B, H * 2, d, generator=g).to(DEV)
    scores = torch.empty(B, H, T, device=DEV)
    asp.score_keys(q, kv, scores)
    tb = torch.tensor([0, 0, 0, 0, T - n], dtype=torch.int32, device=DEV)
    out, acc = torch.empty(B, H * 2, d, device=DEV), torch.zeros(B, H, T, device=DEV)
    ws = torch.empty(asp.accumulate_workspace_bytes(kv, H * 2, 0, n), dtype=torch.uint8, device=DEV)
    asp.attend_accumulate(q, kv, None, None, 0, out, acc, tail_begin=tb, max_tail=n, workspace=ws)
    assert asp.device_status() == 0
    assert (scores[B - 1, :, :T - n] == 0).all()
    assert (acc[B - 1, :, :T - n] == 0).all()
    for h in range(H):
        K, V = np64(rows[0, h].float()) * 2.0 ** -6, np64(rows[1, h].float()) * 2.0 ** -5
        qq = np64(q[B - 1, 2 * h:2 * h + 2])
        x, D = logit_bound(qq, K)
        check(np64(scores[B - 1, h, T - n:]), x.max(axis=0), D.max(axis=0), "scores")
        o, ob, _, _, w, wb = attend_ref(qq, K, V, np.arange(n), False, 2.0 ** -22)
        check(np64(out[B - 1, 2 * h:2 * h + 2]), o, ob, "out")
        check(np64(acc[B - 1, h, T - n:]), w, wb, "acc")
    # append at the end of the last sequence, then evict down to its tail
    lens[B - 1] = T - 1
    x = torch.randn(B, H, d, generator=g).to(DEV)
    lens[1] = 4
    asp.append_kv(kv, x, x)
    assert lens.tolist() == [1, 5, 1, 1, T]
    sc = np64(ks[B - 1, :, (T - 1) // 64])
    for h in range(H):
        need = cache8.block_scale(np64(x[B - 1, h]), "int8")
        assert sc[h] == max(need, 2.0 ** -6)
        assert np.array_equal(np64(k[B - 1, h, T - 1].float()), cache8.code_values(np64(x[B - 1, h]) / sc[h], "int8"))
    idx, cnt = torch.empty(B, H, n, dtype=torch.int32, device=DEV), torch.empty(B, H, dtype=torch.int32, device=DEV)
    wse = torch.empty(asp.evict_workspace_bytes(kv, n), dtype=torch.uint8, device=DEV)
    before = k[B - 1, :, T - n:].float() * ks[B - 1, :, torch.arange(T - n, T, device=DEV) // 64][..., None]
    asp.evict_kv(kv, acc, n, idx, cnt, n_recent=n, workspace=wse)
    assert lens.tolist() == [1, 5, 1, 1, n]
    for h in range(H):
        rc, rs = cache8.quantize(np64(before[h]), 64, "int8")
        assert np.array_equal(np64(k[B - 1, h, :n].float()), rc) and np.array_equal(np64(ks[B - 1, h, :len(rs)]), rs)
