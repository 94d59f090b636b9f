"""Oracle of the 8-bit cache, the summed attention weights and the eviction (test infrastructure).

Float64 throughout; codes are represented by the values they stand for.

C1  scale of a block: the smallest power of two s >= 2^-100 with max |x| <= qmax s over the
    block's finite values (qmax 448 for E4M3, 127 for 8-bit integers).
C2  code of x: x / s rounded to the nearest representable value, ties to even; infinities
    become +-qmax, NaN stays NaN (E4M3) or becomes 0 (integers).
C3  append: a token that opens a block sets its scale by C1; a later one that does not fit (max |x|
    > qmax s over its finite values) raises it to what it needs by C1, and the older codes of the
    block are rounded again at the new scale.
C4  summed weights: acc_j += sum over the group's query heads of softmax_j over the attended
    set.
C5  eviction: a sequence longer than C keeps its first n_sink and last n_recent tokens and the
    C - n_sink - n_recent others with the largest acc, ties to the lowest index, in order.
"""
from __future__ import annotations

import math

import numpy as np

from .attend import attended_set

QMAX = {"e4m3": 448.0, "int8": 127.0}


def block_scale(x: np.ndarray, fmt: str) -> float:
    x = np.abs(np.asarray(x, dtype=np.float64))
    x = x[np.isfinite(x)]
    amax = float(x.max()) if x.size else 0.0
    if amax == 0.0:
        return 2.0 ** -100
    e = math.floor(math.log2(amax / QMAX[fmt])) - 1
    while amax > QMAX[fmt] * 2.0 ** e:
        e += 1
    return 2.0 ** max(e, -100)


def code_values(y: np.ndarray, fmt: str) -> np.ndarray:
    """The codes of ``y`` (already divided by the scale), as values."""
    y = np.asarray(y, dtype=np.float64)
    if fmt == "int8":
        return np.clip(np.rint(np.nan_to_num(y, nan=0.0, posinf=127, neginf=-127)), -127, 127)
    z = np.nan_to_num(y, nan=0.0, posinf=448, neginf=-448)
    e = np.floor(np.log2(np.maximum(np.abs(z), 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    r = np.clip(np.rint(z / step) * step, -448, 448)
    return np.where(np.isnan(y), np.nan, r)


def quantize(x: np.ndarray, scale_block: int, fmt: str):
    """``x [T, d]`` -> (code values ``[T, d]``, scales ``[ceil(T / scale_block)]``)."""
    T = x.shape[0]
    nb = -(-T // scale_block)
    codes, scales = np.zeros(x.shape), np.zeros(nb)
    for i in range(nb):
        rows = slice(i * scale_block, min(T, (i + 1) * scale_block))
        scales[i] = block_scale(x[rows], fmt)
        codes[rows] = code_values(x[rows] / scales[i], fmt)
    return codes, scales


def append(codes: np.ndarray, scales: np.ndarray, x: np.ndarray, scale_block: int, fmt: str):
    """One token ``x [d]`` after ``codes [T, d]``, ``scales`` of its blocks (new arrays)."""
    T = codes.shape[0]
    need = block_scale(x, fmt)
    amax = np.abs(x[np.isfinite(x)]).max(initial=0.0)
    codes, scales = codes.copy(), list(scales)
    if T % scale_block == 0:
        scales.append(need)
    elif amax > QMAX[fmt] * scales[-1]:
        first = T // scale_block * scale_block
        codes[first:] = code_values(codes[first:] * (scales[-1] / need), fmt)
        scales[-1] = need
    return np.concatenate([codes, code_values(x / scales[-1], fmt)[None]]), np.array(scales)


def attention_weights(q: np.ndarray, K: np.ndarray, S: np.ndarray) -> np.ndarray:
    """``q [G, d]``, ``K [T, d]``, attended tokens ``S`` -> summed weights ``[T]``."""
    w = np.zeros(K.shape[0])
    if len(S) == 0:
        return w
    x = np.asarray(q, np.float64) @ np.asarray(K[S], np.float64).T / math.sqrt(q.shape[-1])
    e = np.exp(x - x.max(axis=1, keepdims=True))
    w[S] = (e / e.sum(axis=1, keepdims=True)).sum(axis=0)
    return w


def kept_tokens(acc: np.ndarray, T: int, C: int, n_sink: int, n_recent: int) -> np.ndarray:
    if T <= C:
        return np.arange(T)
    must = np.zeros(T, bool)
    must[:n_sink] = True
    must[T - n_recent:] = True
    rest = np.nonzero(~must)[0]
    rest = rest[np.lexsort((rest, -acc[rest]))][:C - int(must.sum())]
    return np.sort(np.concatenate([np.nonzero(must)[0], rest]))


__all__ = ["QMAX", "append", "attended_set", "attention_weights", "block_scale", "code_values", "kept_tokens", "quantize"]
