"""A query head that is not finite in the 8-bit scan: its whole group's scores are NaN, other groups' stay (GPU)."""
import pytest
import torch

import query_predicted_token_b200 as asp
from test_gpu_cache8 import DEV, Cache, _built, gen  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_a_head_that_is_not_finite_reaches_its_groups_scores(fmt, d, G):
    T = 70
    c = Cache(fmt, 1, 3, d, T, [T], 0, 16, seed=2)
    q = torch.randn(1, 3 * G, d, generator=gen(5)).to(DEV)
    clean = torch.empty(1, 3, T, device=DEV)
    asp.score_keys(q, c.kv, clean)
    assert torch.isfinite(clean).all()
    for head in range(G):
        for bad in (float("nan"), float("inf")):
            x = q.clone()
            x[0, G + head, (7 * head) % d] = bad
            scores = torch.empty(1, 3, T, device=DEV)
            asp.score_keys(x, c.kv, scores)
            assert torch.isnan(scores[0, 1]).all(), (head, bad)
            assert torch.equal(scores[0, [0, 2]], clean[0, [0, 2]])


def test_a_nan_key_of_an_e4m3_cache_reaches_its_score_alone():
    c = Cache("e4m3", 1, 1, 64, 40, [40], 0, 16, seed=2)
    c.side["k"][0].view(torch.uint8)[0, 0, 17, 9] = 0x7f
    q = torch.randn(1, 8, 64, generator=gen(5)).to(DEV)
    scores = torch.empty(1, 1, 40, device=DEV)
    asp.score_keys(q, c.kv, scores)
    nan = torch.isnan(scores[0, 0]).cpu()
    assert nan[17] and int(nan.sum()) == 1
