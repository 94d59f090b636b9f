"""Pins of the 8-bit cache's oracle against independent definitions (CPU)."""
import numpy as np
import pytest
import torch

from oracle import cache8


def test_e4m3_codes_are_the_nearest_of_all_representable_values():
    grid = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    grid = np.unique(grid[np.isfinite(grid)])
    x = np.random.default_rng(0).normal(size=4000) * np.exp2(np.random.default_rng(1).integers(-12, 9, 4000))
    x = np.clip(x, -448, 448)
    best = np.abs(x[:, None] - grid[None]).min(axis=1)
    assert np.array_equal(np.abs(cache8.code_values(x, "e4m3") - x), best)
    # ties to even, as torch's conversion rounds: halfway between neighbouring codes (fp32 holds it)
    mid = (grid[1:] + grid[:-1]) / 2
    t = torch.from_numpy(mid).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(cache8.code_values(mid, "e4m3"), t)


def test_integer_codes():
    x = np.array([-200.0, -127.4, -0.5, 0.5, 1.5, 126.5, 127.49, np.inf, -np.inf, np.nan])
    assert np.array_equal(cache8.code_values(x, "int8"), [-127, -127, 0, 0, 2, 126, 127, 127, -127, 0])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_scale_is_the_smallest_power_of_two_that_holds_the_block(fmt):
    q = cache8.QMAX[fmt]
    for e in (-90, -3, 0, 7, 100):
        assert cache8.block_scale(np.array([q * 2.0 ** e]), fmt) == 2.0 ** e
        assert cache8.block_scale(np.array([-np.nextafter(q * 2.0 ** e, np.inf)]), fmt) == 2.0 ** (e + 1)
    assert cache8.block_scale(np.zeros(4), fmt) == 2.0 ** -100
    assert cache8.block_scale(np.array([1e-40]), fmt) == 2.0 ** -100
    assert cache8.block_scale(np.array([np.inf, np.nan, 1.0]), fmt) == cache8.block_scale(np.array([1.0]), fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_appending_token_by_token_errs_as_stated(fmt):
    """E4M3: within half a step of 3 fraction bits (or half the smallest step) of every value, once
    more for values that a raise makes subnormal; integers: less than one step of the final scale."""
    rng = np.random.default_rng(2)
    x = rng.normal(size=(37, 8)) * np.exp2(rng.integers(-2, 6, (37, 1)))
    c, s = np.zeros((0, 8)), np.zeros(0)
    for row in x:
        c, s = cache8.append(c, s, row, 16, fmt)
    per = np.repeat(s, 16)[:37, None]
    err = np.abs(c * per - x)
    if fmt == "int8":
        assert (err < per).all()
    else:
        assert (err <= np.maximum(2.0 ** -4 * np.abs(x), 2 * 2.0 ** -10 * per)).all()


def test_kept_tokens_ties_sinks_and_recents():
    acc = np.array([0.0, 5, 5, 1, 5, 0, 0, 0])
    assert cache8.kept_tokens(acc, 8, 4, 1, 1).tolist() == [0, 1, 2, 7]
    assert cache8.kept_tokens(acc, 8, 3, 0, 0).tolist() == [1, 2, 4]
    assert cache8.kept_tokens(acc, 3, 4, 1, 1).tolist() == [0, 1, 2]
    assert cache8.kept_tokens(acc, 8, 4, 2, 2).tolist() == [0, 1, 6, 7]


def test_attention_weights_sum_to_the_group_size():
    rng = np.random.default_rng(3)
    q, K = rng.normal(size=(4, 16)), rng.normal(size=(9, 16))
    w = cache8.attention_weights(q, K, np.array([1, 4, 8]))
    assert abs(w.sum() - 4) < 1e-12 and w[[0, 2, 3, 5, 6, 7]].sum() == 0
    assert cache8.attention_weights(q, K, np.array([], dtype=int)).sum() == 0
