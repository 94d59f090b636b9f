"""Append to 8-bit blocks whose scales are any positive normal fp32, not only powers of two (GPU).

A token that fits its block's scale (max |x| <= qmax * scale) leaves the scale and the older codes alone; its codes are
x / scale in fp32, rounded.  One that does not fit raises the scale to the power of two it needs.  Compared exactly.
"""
import numpy as np
import pytest
import torch

import query_predicted_token_b200 as asp
from oracle import cache8
from parity_util import np64
from test_gpu_cache8 import DEV, WIDE, Cache, _built, gen  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("src", ["bf16", "f32"])
@pytest.mark.parametrize("page,block", [(0, 16), (32, 32)])
def test_append_to_blocks_with_any_scale(fmt, src, page, block):
    B, H, T, d = 3, 4, 64, 64
    lens = [5, 20, 33]
    c = Cache(fmt, B, H, d, T, [T] * B, page, block, seed=3, src=WIDE[src], odd_scales=True, spread=1.0)
    c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    qmax = cache8.QMAX[fmt]
    ref = {(s, b, h): [a[h].copy() for a in c.codes(s, b)] for s in "kv" for b in range(B) for h in range(H)}
    g = gen(8)
    kept, raised = 0, 0
    for step in range(12):
        x = torch.randn(2, B, H, d, generator=g)
        for (s, b, h), (codes, scales) in ref.items():     # rows whose largest value is near what the block takes
            i = "kv".index(s)
            n = len(codes)
            if n % block:
                want = qmax * scales[-1] * (0.7, 0.999, 1.001, 3.0)[(step + h + b) % 4]
                x[i, b, h] *= want / float(x[i, b, h].abs().max())
        x = x.to(WIDE[src])
        asp.append_kv(c.kv, x[0].to(DEV), x[1].to(DEV))
        for key, (codes, scales) in ref.items():
            s, b, h = key
            row = np64(x["kv".index(s), b, h].float())
            n = len(codes)
            if n % block == 0:
                scales = np.append(scales, cache8.block_scale(row, fmt))
            elif np.abs(row).max() > np.float32(qmax) * np.float32(scales[-1]):
                need = cache8.block_scale(row, fmt)
                f = np.float32(scales[-1]) / np.float32(need)
                first = n // block * block
                codes[first:] = cache8.code_values(codes[first:].astype(np.float32) * f, fmt)
                scales[-1] = need
                raised += 1
            else:
                kept += 1
            code = cache8.code_values(row.astype(np.float32) / np.float32(scales[-1]), fmt)
            ref[key] = [np.concatenate([codes, code[None]]), scales]
    assert asp.device_status() == 0
    assert kept > 20 and raised > 20
    for s in "kv":
        for b in range(B):
            codes, scales = c.codes(s, b)
            for h in range(H):
                assert np.array_equal(scales[h], ref[s, b, h][1]), (s, b, h)
                assert np.array_equal(codes[h], ref[s, b, h][0]), (s, b, h)
