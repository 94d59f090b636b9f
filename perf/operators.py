"""The operators around a KV cache held in 8 bits, as they are measured: filling the cache, appending to it,
scoring its keys, attending over it, summing the attention each cached token gets, and evicting by that sum.

A cache in 8 bits holds a code per value and one scale per block of tokens, KV head and side (K or V); a value is
code * scale.  ``run`` computes each operator in its plain form, or, where ``own`` is true, by the library's calls.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
QMAX = {"e4m3": 448.0, "int8": 127.0}
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
WIDE = {"bf16": torch.bfloat16, "f32": torch.float32}
MIN_EXP = -100           # the smallest scale is 2^-100


def _case(name, op, fmt, B, Hkv, G, d, T, tmin, page=0, block=64, q="bf16", C=0, sink=0, recent=0):
    return dict(name=name, op=op, fmt=fmt, B=B, Hkv=Hkv, G=G, d=d, T=T, tmin=tmin, page=page, block=block, q=q, C=C,
                sink=sink, recent=recent)


def listed():
    return [
        # a long prompt's K and V, as the projections leave them ([batch, token, head, channel]), into the cache
        _case("quantize prompt 8 x 32k", "quantize", "e4m3", 8, 8, 4, 128, 32768, 32768, block=64),
        # a short prompt of one sequence, fp32 activations, codes of 8-bit integers
        _case("quantize one short prompt", "quantize", "int8", 1, 2, 2, 64, 512, 500, block=32, q="f32"),
        # the token of a decode step for 8 sequences: the call of every layer and step, where latency counts
        _case("append 8 sequences", "append", "e4m3", 8, 8, 4, 128, 32768, 20000, block=64),
        # the token of a decode step for 64 ragged sequences in 16-token pages
        _case("append 64 ragged paged", "append", "int8", 64, 8, 4, 128, 16384, 1024, page=16, block=16),
        # the key scan of a decode step at long contexts (the step's largest part)
        _case("score 8 x 32k", "score", "e4m3", 8, 8, 4, 128, 32768, 32768, block=64, q="f32"),
        # the key scan over ragged sequences in shuffled 16-token pages, GQA group 8
        _case("score 8 ragged paged", "score", "int8", 8, 8, 8, 128, 65536, 8192, page=16, block=16, q="f32"),
        # attention over every cached token (the fallback and baseline of the sparse step)
        _case("attend all 8 x 32k", "attend", "e4m3", 8, 8, 4, 128, 32768, 32768, block=64),
        # attention over the 2048 selected tokens of each of 64 long ragged sequences
        _case("attend 2048 of 64 ragged", "attend", "e4m3", 64, 8, 4, 128, 32768, 8192, page=16, block=16, C=2048),
        # decode of one small sequence, fp32 query: latency alone
        _case("accumulate one short", "accumulate", "int8", 1, 2, 2, 64, 512, 512, block=32, q="f32"),
        # a decode step that also sums each token's attention, over a bf16 cache with ragged lengths
        _case("accumulate 32 ragged bf16", "accumulate", "bf16", 32, 8, 4, 128, 8192, 1, block=0),
        # eviction from 8192 tokens down to 2048, the first 4 and the last 256 always kept
        _case("evict 8 x 8k to 2k", "evict", "e4m3", 8, 8, 4, 128, 8192, 8192, block=64, C=2048, sink=4, recent=256),
        # eviction in a ragged batch in pages, bf16 cache; some sequences are under the budget already
        _case("evict 16 ragged paged bf16", "evict", "bf16", 16, 4, 4, 128, 5000, 500, page=32, block=0, C=1024, sink=1,
              recent=64),
    ]


def draw(rng):
    op = rng.choice(["quantize", "append", "score", "attend", "accumulate", "evict"])
    d = rng.choice([64, 128])
    G = rng.choice([1, 2, 4, 8])
    q = "f32" if op == "score" else rng.choice(["bf16", "bf16", "f32"])
    fmt = rng.choice(["e4m3", "int8"] + (["bf16", "f32"] if op in ("accumulate", "evict") else []))
    page = rng.choice([0, 0, 16, 32, 64, 128])
    block = 0 if fmt in WIDE else rng.choice([b for b in (16, 32, 64, 128) if not page or page % b == 0])
    B = int(round(math.exp(rng.uniform(0, math.log(64)))))
    Hkv = rng.choice([1, 2, 4, 8])
    T = int(math.exp(rng.uniform(0, math.log(32768))))
    while B * Hkv * T * d > 1 << 27:      # at most half of the largest listed cache
        B, T = max(1, B // 2), max(1, int(T * 0.8))
    tmin = rng.choice([0, 1, max(1, T // 4), T])
    C = sink = recent = 0
    if op == "attend":
        C = rng.choice([0, 0, max(1, T // 16), max(1, T // 3)])
    elif op == "accumulate":
        C = rng.choice([0, 0, 0, max(1, T // 8)])
    elif op == "evict":
        C = max(4, T // rng.choice([2, 3, 8]))
        sink, recent = rng.choice([0, 1, 4]), rng.randint(0, C // 2)
        sink = min(sink, C - recent)
    if op == "append":
        T, tmin = T + 1, min(tmin, T)
    return {k: v for k, v in _case("", op, fmt, B, Hkv, G, d, T, tmin, page, block, q, C, sink, recent).items()
            if k != "name"}


# ---- inputs -------------------------------------------------------------------------------------------------------

def _scale_of(amax, fmt):
    """The smallest power of two s with amax <= qmax * s, at least 2^MIN_EXP."""
    m, e = torch.frexp(amax)
    top, shift = (0.875, 9) if fmt == "e4m3" else (0.9921875, 7)     # qmax = top * 2^shift
    e = torch.where(amax > 0, e - shift + (m > top).to(e.dtype), torch.full_like(e, MIN_EXP)).clamp_(min=MIN_EXP)
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _encode(x, fmt):
    """Codes of values already divided by their scale."""
    if fmt == "int8":
        return x.round().clamp_(-127, 127).to(torch.int8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _new_cache(c, g, gc):
    """Random codes and scales (or wide values) of one side of the cache, everywhere, lengths or not: quantised normal
    values with a scale per channel and per block."""
    B, H, T, d, P, bl = c["B"], c["Hkv"], c["T"], c["d"], c["page"], c["block"]
    N, L = (gc["n_pages"], P) if P else (B, T)
    chan = 0.5 + 1.5 * torch.rand(H, 1, d, generator=g, device=DEV)
    x = torch.empty(N, H, L, d, dtype=WIDE.get(c["fmt"]) or CODE[c["fmt"]], device=DEV)
    nb = -(-L // bl) if bl else 0
    sc = torch.empty(N, H, nb, dtype=torch.float32, device=DEV) if bl else None
    step = max(1, (1 << 26) // (H * L * d))
    for n in range(0, N, step):
        m = min(N, n + step) - n
        y = torch.randn(m, H, L, d, generator=g, device=DEV).mul_(chan)
        if not bl:
            x[n:n + m] = y
            continue
        y.mul_(torch.exp(0.5 * torch.randn(m, H, nb, generator=g, device=DEV)).repeat_interleave(bl, 2)[:, :, :L, None])
        a = torch.nn.functional.pad(y.abs().amax(-1), (0, nb * bl - L)).view(m, H, nb, bl).amax(-1)
        s = _scale_of(a, c["fmt"])
        sc[n:n + m] = s
        x[n:n + m] = _encode(y.div_(s.repeat_interleave(bl, 2)[:, :, :L, None]), c["fmt"])
    return x, sc


def prepare(case, seed):
    c = dict(case)
    B, H, G, T, d, P = c["B"], c["Hkv"], c["G"], c["T"], c["d"], c["page"]
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 1)
    h = torch.Generator().manual_seed(int(seed) * 7919 + 2)
    most = T - 1 if c["op"] == "append" else T
    lens = torch.randint(min(c["tmin"], most), most + 1, (B,), generator=h)
    s = {"c": c, "len0": lens.to(torch.int32).to(DEV)}
    s["seq_lens"] = s["len0"].clone()
    if P:
        maxp = -(-T // P)
        need = (lens + (1 if c["op"] == "append" else 0) + P - 1) // P
        n_pages = B * maxp
        perm = torch.randperm(n_pages, generator=h).to(torch.int32)
        at = torch.cumsum(need, 0) - need
        slot = at[:, None] + torch.arange(maxp)
        s["table"] = torch.where(torch.arange(maxp) < need[:, None], perm[slot.clamp(max=n_pages - 1)],
                                 torch.tensor(-1, dtype=torch.int32)).to(DEV)
        s["n_pages"] = n_pages
    s["k"], s["ks"] = _new_cache(c, g, s)
    s["v"], s["vs"] = _new_cache(c, g, s)
    wide = WIDE[c["q"]]
    if c["op"] == "quantize":        # the projections' layout, [batch, token, head, channel], seen head-first
        src = torch.randn(2, B, T, H, d, generator=g, device=DEV).to(wide)
        s["k_src"], s["v_src"] = src[0].transpose(1, 2), src[1].transpose(1, 2)
    if c["op"] == "append":
        new = torch.randn(2, B, H, d, generator=g, device=DEV).mul_(1.5).to(wide)
        s["k_new"], s["v_new"] = new[0].contiguous(), new[1].contiguous()
    if c["op"] in ("quantize", "evict") and c["fmt"] in CODE:      # where the cache is read back as values
        rows = T if c["op"] == "quantize" else min(c["C"], T)
        s["k_val"] = torch.zeros(B, H, rows, d, dtype=torch.bfloat16, device=DEV)
        s["v_val"] = torch.zeros_like(s["k_val"])
    if c["op"] == "append":
        s["tail"] = torch.zeros(B, dtype=torch.int32, device=DEV)
        bl, n0 = c["block"], s["len0"].long()
        rows = ((n0 // bl * bl)[:, None] + torch.arange(bl, device=DEV))[:, None].expand(B, H, bl)
        s["rows"], s["place"] = rows, _place(s, rows.clamp(max=T - 1))        # the blocks that get the tokens
        s["held"] = (rows <= n0[:, None, None])[..., None]
    if c["op"] in ("score", "attend", "accumulate"):
        s["q"] = torch.randn(B, H * G, d, generator=g, device=DEV).to(wide)
    if c["op"] == "score":
        s["scores"] = torch.zeros(B, H, T, device=DEV)
    if c["op"] in ("attend", "accumulate"):
        s["out"] = torch.zeros(B, H * G, d, dtype=WIDE.get(c["fmt"], wide), device=DEV)
        s["lse"] = torch.zeros(B, H * G, device=DEV)
        C = c["C"]
        if C:        # the selection of a sparse step, and the tokens appended since it was made
            tail = (s["len0"] - 3).clamp_(min=0)
            s["tail_begin"], s["max_tail"] = tail, 3
            r = torch.rand(B, H, T, generator=g, device=DEV)
            r = r.masked_fill_(torch.arange(T, device=DEV) >= tail[:, None, None], -1.0)
            idx = r.topk(C, dim=-1).indices.sort(-1).values.to(torch.int32)
            cnt = tail.clamp(max=C)[:, None].expand(B, H).contiguous()
            del r
            big = torch.where(idx < tail[:, None, None], idx, T + 1).sort(-1).values
            s["idx"] = torch.where(torch.arange(C, device=DEV) < cnt[..., None], big, -1).to(torch.int32)
            s["count"] = cnt
        else:
            s["tail_begin"], s["max_tail"] = torch.zeros(B, dtype=torch.int32, device=DEV), T
    if c["op"] in ("accumulate", "evict"):     # heavy-tailed, as sums of attention weights are
        s["acc"] = torch.rand(B, H, T, generator=g, device=DEV).pow_(6.0)
    if c["op"] == "evict":
        s["idx"] = torch.full((B, H, c["C"]), -1, dtype=torch.int32, device=DEV)
        s["count"] = torch.zeros(B, H, dtype=torch.int32, device=DEV)
        s["acc_out"] = torch.zeros_like(s["acc"])
    return s


# ---- plain forms --------------------------------------------------------------------------------------------------

def _all_values(s, side):
    """The cache as fp32 [B, H, T, d] in token order (rows past a sequence's pages hold another page's values)."""
    c, x, sc = s["c"], s[side], s[side + "s"]
    y = x.float()
    if sc is not None:
        y = y * sc.repeat_interleave(c["block"], 2)[:, :, :y.shape[2], None]
    if c["page"]:
        y = y[s["table"].clamp(min=0).long()].transpose(1, 2).flatten(2, 3)[:, :, :c["T"]]
    return y


def _place(s, tok):
    """Where tokens tok [B, H, n] of the cache lie: (page or sequence, head, row) indices."""
    c = s["c"]
    h = torch.arange(c["Hkv"], device=DEV)[None, :, None].expand_as(tok)
    b = torch.arange(c["B"], device=DEV)[:, None, None].expand_as(tok)
    if not c["page"]:
        return b, h, tok
    return s["table"].long()[b, tok // c["page"]].clamp(min=0), h, tok % c["page"]


def _take(x, n, h, r):
    return x[n, h, r] if x.dtype in WIDE.values() else x.view(torch.uint8)[n, h, r].view(x.dtype)


def _values_at(s, side, tok):
    n, h, r = _place(s, tok)
    y = _take(s[side], n, h, r).float()
    if s[side + "s"] is not None:
        y = y * s[side + "s"][n, h, r // s["c"]["block"]][..., None]
    return y


def _plain_quantize(s):
    c = s["c"]
    B, H, T, d, P, bl = c["B"], c["Hkv"], c["T"], c["d"], c["page"], c["block"]
    live = torch.arange(T, device=DEV) < s["seq_lens"][:, None]                 # [B, T]
    for side in ("k", "v"):
        x = s[side + "_src"].float()
        a = torch.where(live[:, None], x.abs().amax(-1), 0.0)
        nb = -(-T // bl)
        a = torch.nn.functional.pad(a, (0, nb * bl - T)).view(B, H, nb, bl).amax(-1)
        sc = _scale_of(a, c["fmt"])
        code = _encode(x / sc.repeat_interleave(bl, 2)[:, :, :T, None], c["fmt"])
        if not P:
            s[side] = torch.where(live[:, None, :, None], code.view(torch.uint8), s[side].view(torch.uint8)).view(code.dtype)
            used = live[:, ::bl]
            s[side + "s"] = torch.where(used[:, None], sc, s[side + "s"])
        else:
            b, t = live.nonzero(as_tuple=True)
            page = s["table"].long()[b, t // P]
            s[side].view(torch.uint8)[page, :, t % P] = code.view(torch.uint8)[b, :, t]
            s[side + "s"][page, :, (t % P) // bl] = sc[b, :, t // bl]
        val = code.float() * sc.repeat_interleave(bl, 2)[:, :, :T, None]
        s[side + "_val"] = torch.where(live[:, None, :, None], val, 0.0).to(torch.bfloat16)
    return {"k": s["k_val"], "v": s["v_val"], "k_scale": _scales(s, "k"), "v_scale": _scales(s, "v")}


def _scales(s, side):
    """The scales of the blocks that hold tokens, in token order, zeros elsewhere."""
    c, sc = s["c"], s[side + "s"]
    nb = -(-c["T"] // c["block"])
    if c["page"]:
        sc = sc[s["table"].clamp(min=0).long()].transpose(1, 2).flatten(2, 3)[:, :, :nb]
    used = torch.arange(nb, device=DEV) * c["block"] < s["seq_lens"][:, None]
    return torch.where(used[:, None], sc, 0.0)


def _plain_append(s):
    c, rows = s["c"], s["rows"]
    bl = c["block"]
    T = s["seq_lens"].long()
    inside = rows < c["T"]
    old = rows < T[:, None, None]
    n, h, r = s["place"]
    for side in ("k", "v"):
        new = s[side + "_new"].float()
        need = _scale_of(new.abs().amax(-1), c["fmt"])
        was = s[side + "s"][n[..., 0], h[..., 0], r[..., 0] // bl]
        opens = (T % bl == 0)[:, None]
        sc = torch.where(opens, need, torch.maximum(need, was))
        val = _take(s[side], n, h, r).float()
        again = _encode(val * (was / sc)[..., None, None], c["fmt"]).view(torch.uint8)
        code = torch.where(old[..., None], again, _encode(new / sc[..., None], c["fmt"]).view(torch.uint8)[:, :, None])
        touch = inside & (rows <= T[:, None, None])
        s[side].view(torch.uint8)[n[touch], h[touch], r[touch]] = code[touch]
        s[side + "s"][n[..., 0], h[..., 0], r[..., 0] // bl] = sc
    s["tail"].copy_(s["seq_lens"])
    s["seq_lens"] += 1
    return _appended(s)


def _appended(s):
    """The blocks that got the token, as values, with their scales, and the lengths."""
    n, h, r = s["place"]
    out = {"tail": s["tail"], "seq_lens": s["seq_lens"]}
    for side in ("k", "v"):
        sc = s[side + "s"][n[..., 0], h[..., 0], r[..., 0] // s["c"]["block"]]
        out[side] = torch.where(s["held"], _take(s[side], n, h, r).float() * sc[..., None, None], 0.0)
        out[side + "_scale"] = sc
    return out


def _plain_score(s):
    c = s["c"]
    B, H, G, T, d = c["B"], c["Hkv"], c["G"], c["T"], c["d"]
    k = _all_values(s, "k")
    x = (s["q"].view(B, H, G, d) @ k.transpose(-1, -2)).amax(2) / math.sqrt(d)
    live = torch.arange(T, device=DEV) < s["seq_lens"][:, None, None]
    return torch.where(live, x, s["scores"])


def _attended(s):
    """(tokens [B, H, n], which of them count) of the selection and the tail."""
    c = s["c"]
    T, tb = s["seq_lens"].long()[:, None, None], s["tail_begin"].long()[:, None, None]
    i = s["idx"].long()
    ok = (torch.arange(c["C"], device=DEV) < s["count"][..., None]) & (i >= 0) & (i < T) & (i < tb)
    t = (tb + torch.arange(s["max_tail"], device=DEV)).expand(c["B"], c["Hkv"], s["max_tail"])
    return torch.cat([i, t], -1), torch.cat([ok, t < T], -1)


def _plain_attend(s):
    c = s["c"]
    B, H, G, T, d = c["B"], c["Hkv"], c["G"], c["T"], c["d"]
    if c["C"]:
        tok, ok = _attended(s)
        tok = torch.where(ok, tok, 0)
        k, v = _values_at(s, "k", tok), _values_at(s, "v", tok)
        v = torch.where(ok[..., None], v, 0.0)
    else:
        tok = None
        ok = (torch.arange(T, device=DEV) < s["seq_lens"][:, None, None]).expand(B, H, T)
        k, v = _all_values(s, "k"), _all_values(s, "v")
    x = (s["q"].float().view(B, H, G, d) @ k.transpose(-1, -2)) / math.sqrt(d)
    x = torch.where(ok[:, :, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    z = p.sum(-1, keepdim=True)
    p = torch.where(z > 0, p / z, 0.0)
    s["lse"] = (m + torch.log(z)).view(B, H * G)
    s["out"] = (p @ v).view(B, H * G, d).to(s["out"].dtype)
    out = {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "accumulate":
        w = p.sum(2)
        if tok is None:
            s["acc"] += w
        else:
            s["acc"].scatter_add_(2, tok, w)
        out["acc"] = s["acc"]
    return out


def _plain_evict(s):
    c = s["c"]
    B, H, T, d, C, bl = c["B"], c["Hkv"], c["T"], c["d"], c["C"], c["block"]
    n0 = s["seq_lens"].long()[:, None, None]
    j = torch.arange(T, device=DEV)
    a = torch.where((j < c["sink"]) | (j >= n0 - c["recent"]), math.inf, s["acc"])
    a = torch.where(j < n0, a, -math.inf)
    kept = torch.sort(a, dim=-1, descending=True, stable=True).indices[..., :C]
    kept = torch.where(kept < n0, kept, T).sort(-1).values              # ascending, past the end where there are fewer
    ok = kept < n0
    tok = torch.where(ok, kept, 0)
    cnt = ok.sum(-1)
    moved = (n0 > C).expand(B, H, 1)
    acc = torch.where(ok, s["acc"].gather(-1, tok), 0.0)
    s["acc_out"] = torch.nn.functional.pad(acc, (0, T - acc.shape[-1]))
    C = kept.shape[-1]
    dst = torch.arange(C, device=DEV).expand(B, H, C)
    n, h, r = _place(s, dst)
    write = moved & ok
    out = {}
    for side in ("k", "v"):
        if c["fmt"] not in CODE:
            x = s[side][_place(s, tok)]
            s[side][n[write], h[write], r[write]] = x[write]
            out[side] = s[side]
            continue
        x = _values_at(s, side, tok)
        nb = -(-C // bl)
        amax = torch.nn.functional.pad(torch.where(ok, x.abs().amax(-1), 0.0), (0, nb * bl - C))
        sc = _scale_of(amax.view(B, H, nb, bl).amax(-1), c["fmt"])
        code = _encode(x / sc.repeat_interleave(bl, 2)[:, :, :C, None], c["fmt"])
        s[side].view(torch.uint8)[n[write], h[write], r[write]] = code.view(torch.uint8)[write]
        at = torch.arange(nb, device=DEV).mul(bl)
        w = write[..., ::bl]
        s[side + "s"][n[..., at][w], h[..., at][w], r[..., at][w] // bl] = sc[w]
        val = torch.where(ok[..., None], _values_at(s, side, dst), 0.0)
        s[side + "_val"] = val.to(torch.bfloat16)
        out[side] = s[side + "_val"]
    s["idx"] = torch.nn.functional.pad(torch.where(ok, kept, -1), (0, c["C"] - C), value=-1).to(torch.int32)
    s["count"] = cnt.to(torch.int32)
    s["seq_lens"] = s["seq_lens"].clamp(max=c["C"])
    return {**out, "acc": s["acc_out"], "idx": s["idx"], "count": s["count"], "seq_lens": s["seq_lens"]}


# ---- the library's calls ------------------------------------------------------------------------------------------

def _handle(s, asp):
    """The cache's handle and the workspace that a program keeps beside it."""
    c = s["c"]
    kv = asp.KV(s["k"], s["v"], s["seq_lens"], s.get("table"), t_max=c["T"], k_scale=s["ks"], v_scale=s["vs"],
                scale_block=c["block"], src_dtype=WIDE[c["q"]])
    need = 0
    if c["op"] == "attend":
        need = asp.attend_workspace_bytes_kv(kv, c["Hkv"] * c["G"], c["C"], s["max_tail"])
    elif c["op"] == "accumulate":
        need = asp.accumulate_workspace_bytes(kv, c["Hkv"] * c["G"], c["C"], s["max_tail"])
    elif c["op"] == "evict":
        need = asp.evict_workspace_bytes(kv, c["C"])
    return kv, torch.empty(max(16, need), dtype=torch.uint8, device=DEV)


def _own_run(s):
    import query_predicted_token_b200 as asp
    c = s["c"]
    if "handle" not in s:
        s["handle"] = _handle(s, asp)
    kv, ws = s["handle"]
    op = c["op"]
    if op == "quantize":
        asp.quantize_kv(kv, s["k_src"], s["v_src"])
        asp.dequantize_kv(kv, s["k_val"], s["v_val"])
        return {"k": s["k_val"], "v": s["v_val"], "k_scale": _scales(s, "k"), "v_scale": _scales(s, "v")}
    if op == "append":
        asp.append_kv(kv, s["k_new"], s["v_new"], s["tail"])
        return _appended(s)
    if op == "score":
        asp.score_keys(s["q"], kv, s["scores"])
        return s["scores"]
    if op == "attend":
        asp.sparse_attend(s["q"], kv, s.get("idx"), s.get("count"), c["C"], s["out"], s["lse"],
                          tail_begin=s["tail_begin"], max_tail=s["max_tail"], workspace=ws)
        return {"out": s["out"], "lse": s["lse"]}
    if op == "accumulate":
        asp.attend_accumulate(s["q"], kv, s.get("idx"), s.get("count"), c["C"], s["out"], s["acc"], s["lse"],
                              tail_begin=s["tail_begin"], max_tail=s["max_tail"], workspace=ws)
        return {"out": s["out"], "lse": s["lse"], "acc": s["acc"]}
    asp.evict_kv(kv, s["acc"], c["C"], s["idx"], s["count"], n_sink=c["sink"], n_recent=c["recent"],
                 acc_out=s["acc_out"], workspace=ws)
    out = {"k": s["k"], "v": s["v"]}
    if c["fmt"] in CODE:
        asp.dequantize_kv(kv, s["k_val"], s["v_val"])
        out = {"k": s["k_val"], "v": s["v_val"]}
    return {**out, "acc": s["acc_out"], "idx": s["idx"], "count": s["count"], "seq_lens": s["seq_lens"]}


def run(state):
    op = state["c"]["op"]
    if op in ("append", "evict"):        # the call moves the lengths: each pass starts from the same ones
        state["seq_lens"].copy_(state["len0"])
    if own:
        return _own_run(state)
    return {"quantize": _plain_quantize, "append": _plain_append, "score": _plain_score, "attend": _plain_attend,
            "accumulate": _plain_attend, "evict": _plain_evict}[op](state)


# ---- the definitions in 64 bits -----------------------------------------------------------------------------------

def _np_scale(amax, fmt):
    """The smallest 2^e with amax <= qmax 2^e, by its definition."""
    if not amax > 0:
        return 2.0 ** MIN_EXP
    e = math.floor(math.log2(amax / QMAX[fmt])) - 1
    while amax > QMAX[fmt] * 2.0 ** e:
        e += 1
    return 2.0 ** max(e, MIN_EXP)


def _grid(x, fmt):
    """Doubles rounded to the nearest value a code stands for, ties to even."""
    if fmt == "int8":
        return torch.round(x).clamp(-127, 127)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _sequence(s, side, b, n):
    """Sequence b's first n rows of the cache as doubles [H, n, d]."""
    c = s["c"]
    P, bl = c["page"], c["block"]
    t = torch.arange(n, device=DEV)
    page = s["table"][b].long()[t // P] if P else torch.full_like(t, b)
    row = t % P if P else t
    x = (s[side].view(torch.uint8)[page, :, row].view(s[side].dtype) if bl else s[side][page, :, row]).double()
    if bl:
        x = x * s[side + "s"][page, :, row // bl].double()[..., None]
    return x.transpose(0, 1)


def _requantised(x, fmt, bl):
    """Values [H, n, d] after a trip through codes with one scale per bl rows, and the scales [H, blocks]."""
    H, n, _ = x.shape
    nb = -(-n // bl)
    a = x.abs().amax(-1).cpu().numpy()
    sc = np.array([[_np_scale(a[h, i * bl:(i + 1) * bl].max(), fmt) for i in range(nb)] for h in range(H)]).reshape(H, nb)
    per = torch.from_numpy(sc).to(DEV).repeat_interleave(bl, 1)[:, :n, None]
    return _grid(x / per, fmt) * per, torch.from_numpy(sc).to(DEV)


def exact(case, seed):
    s = prepare(case, seed)
    c = s["c"]
    B, H, G, T, d, bl, fmt = c["B"], c["Hkv"], c["G"], c["T"], c["d"], c["block"], c["fmt"]
    lens = s["len0"].tolist()
    f64 = dict(dtype=torch.float64, device=DEV)
    if c["op"] == "quantize":
        out = {k: torch.zeros(B, H, T, d, dtype=torch.float32, device=DEV) for k in ("k", "v")}
        nb = -(-T // bl)
        out |= {k + "_scale": torch.zeros(B, H, nb, **f64) for k in ("k", "v")}
        for side in ("k", "v"):
            for b, n in enumerate(lens):
                if n:
                    y, sc = _requantised(s[side + "_src"][b, :, :n].double(), fmt, bl)
                    out[side][b, :, :n] = y.float()           # codes times a power of two: exact in 32 bits
                    out[side + "_scale"][b, :, :sc.shape[1]] = sc
        return out
    if c["op"] == "append":
        out = {"tail": None, "seq_lens": None}
        for side in ("k", "v"):
            val, scs = torch.zeros(B, H, bl, d, **f64), torch.zeros(B, H, **f64)
            for b, n in enumerate(lens):
                new = s[side + "_new"][b].double()
                amax = new.abs().amax(-1).tolist()
                P, first = c["page"], n // bl * bl
                page, row = (int(s["table"][b, first // P]), first % P) if P else (b, first)
                for h in range(H):
                    was = float(s[side + "s"][page, h, row // bl])
                    need = _np_scale(amax[h], fmt)
                    sc = need if n == first else max(need, was)
                    old = s[side][page, h, row:row + n - first].float().double() * was
                    val[b, h, :n - first] = _grid(old / sc, fmt) * sc
                    val[b, h, n - first] = _grid(new[h] / sc, fmt) * sc
                    scs[b, h] = sc
            out[side], out[side + "_scale"] = val, scs
        return out
    if c["op"] == "score":
        out = torch.zeros(B, H, T, **f64)
        for b, n in enumerate(lens):
            if n:
                x = torch.einsum("hgd,hnd->hgn", s["q"][b].double().view(H, G, d), _sequence(s, "k", b, n))
                out[b, :, :n] = x.max(1).values / d ** 0.5
        return out
    if c["op"] in ("attend", "accumulate"):
        o, lse = torch.zeros(B, H * G, d, **f64), torch.full((B, H * G), -math.inf, **f64)
        acc = s["acc"].double() if "acc" in s else None
        for b, n in enumerate(lens):
            if not n:
                continue
            k, v = _sequence(s, "k", b, n), _sequence(s, "v", b, n)
            x = torch.einsum("hgd,hnd->hgn", s["q"][b].double().view(H, G, d), k) / d ** 0.5
            if c["C"]:
                seen = torch.zeros(H, n, dtype=torch.bool, device=DEV)
                seen[:, int(s["tail_begin"][b]):] = True
                for h in range(H):
                    seen[h, s["idx"][b, h, :int(s["count"][b, h])].long()] = True
                x = x.masked_fill(~seen[:, None], -math.inf)
            w = torch.softmax(x, -1)
            o[b] = torch.einsum("hgn,hnd->hgd", w, v).reshape(H * G, d)
            lse[b] = torch.logsumexp(x, -1).reshape(-1)
            if acc is not None:
                acc[b, :, :n] += w.sum(1)
        return {"out": o, "lse": lse, "acc": acc} if c["op"] == "accumulate" else {"out": o, "lse": lse}
    C = c["C"]
    out = {"acc": torch.zeros(B, H, T, **f64), "idx": None, "count": None, "seq_lens": None}
    kept = []
    a = s["acc"].cpu().numpy()
    for b, n in enumerate(lens):
        kept.append([])
        for h in range(H):
            must = set(range(min(c["sink"], n))) | set(range(max(0, n - c["recent"]), n))
            rest = [int(i) for i in np.lexsort((np.arange(n), -a[b, h, :n].astype(np.float64))) if int(i) not in must]
            keep = sorted(list(must) + rest[:max(0, C - len(must))]) if n > C else list(range(n))
            kept[b].append(keep)
            out["acc"][b, h, :len(keep)] = s["acc"][b, h, keep].double()
    for side in ("k", "v"):
        if fmt not in CODE:
            out[side] = s[side].double()
            for b, n in enumerate(lens):
                if n <= C:
                    continue
                seq = _sequence(s, side, b, n)
                t = torch.arange(C, device=DEV)
                page = s["table"][b].long()[t // c["page"]] if c["page"] else torch.full_like(t, b)
                row = t % c["page"] if c["page"] else t
                for h in range(H):
                    out[side][page, h, row] = seq[h, kept[b][h]]
            continue
        out[side] = torch.zeros(B, H, min(C, T), d, **f64)
        for b, n in enumerate(lens):
            if not n:
                continue
            seq = _sequence(s, side, b, n)
            rows = torch.stack([seq[h, kept[b][h]] for h in range(H)])
            out[side][b, :, :min(n, C)] = _requantised(rows, fmt, bl)[0] if n > C else rows
    return out


def work(case):
    c = case
    B, H, G, T, d = c["B"], c["Hkv"], c["G"], c["T"], c["d"]
    mean = min(T, (c["tmin"] + T) / 2)
    e = {"e4m3": 1, "int8": 1, "bf16": 2, "f32": 4}[c["fmt"]]
    w = 4 if c["q"] == "f32" else 2
    row = d * e + (4.0 / c["block"] if c["block"] else 0.0)         # one side's row, with its share of the scale
    toks = B * H * mean
    if c["op"] == "quantize":       # the source read, the codes written, and read back as bf16 values
        return {"bytes": toks * 2 * (d * w + 2 * row + 2 * d), "flops": toks * 2 * 4 * d}
    if c["op"] == "append":         # the new rows, and the block's scales
        return {"bytes": B * H * 2 * (d * w + d + 8), "flops": B * H * 2 * 4 * d}
    if c["op"] == "score":
        return {"bytes": toks * (row + 4) + B * H * G * d * w, "flops": toks * G * 2 * d}
    if c["op"] in ("attend", "accumulate"):
        rows = B * H * min(mean, c["C"] + 3) if c["C"] else toks
        moved = rows * 2 * row + B * H * G * (2 * d * w + 4) + (rows * 4 if c["C"] else 0)
        return {"bytes": moved + (8 * rows if c["op"] == "accumulate" else 0), "flops": rows * G * 4 * d}
    kept = B * H * min(mean, c["C"])
    return {"bytes": 4 * toks + kept * (4 * row + 12) + (kept * 2 * (row + 2 * d) if e == 1 else 0), "flops": kept * 2 * 4 * d}
