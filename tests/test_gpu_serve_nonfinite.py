"""Infinities and NaN in what the prompt attention reads: in keys that a row sees, in keys that it does not see, and in
V on either side of the mask."""
import math

import pytest
import torch

from tests.serve_ref import attend, check
from tests.test_gpu_serve_prompt import _inputs

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16]
# lq, lk, Hq, Hk, D, causal, first row tile's heads to look at
FORMS = {
    "pairs over heads": (260, 260, 600, 100, 64, True, [0, 299, 599]),
    "pairs over rows": (256, 640, 100, 100, 128, False, [0, 57, 99]),
    "alone": (400, 400, 2, 1, 128, True, [0, 1]),
    "alone, narrow": (100, 500, 3, 1, 64, True, [0, 2]),
    "clusters": (60, 2000, 2, 1, 128, True, [0, 1]),
}


def _one(name, dtype):
    lq, lk, Hq, Hk, D, causal, heads = FORMS[name]
    q, k, v = _inputs([lq], [lk], Hq, Hk, D, dtype, seed=len(name))
    q = q.clone()
    q[..., 0] = q[..., 0].abs() + 0.25                      # an infinity in K's channel 0 keeps its sign in every score
    n = torch.arange(lq, device="cuda") + 1 + lk - lq
    return q, k.clone(), v, n if causal else torch.full_like(n, lk), causal, heads


def _run(adt, q, k, v, causal):
    lse = torch.full((q.shape[1], q.shape[0]), 9.0, device="cuda")
    out = adt.sage_attn_prompt(q, k, v, [0, q.shape[0]], [0, k.shape[0]], lse=lse, causal=causal)
    return out, lse


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name", list(FORMS))
def test_a_score_that_is_no_number_reaches_every_row_that_sees_it(adt, dtype, name):
    """A NaN or +inf score makes the row's softmax NaN, wherever in a tile its key lies; other rows are as before."""
    q, k, v, visible, causal, _ = _one(name, dtype)
    clean, clean_lse = _run(adt, q, k, v, causal)
    assert bool(torch.isfinite(clean).all())
    for j in range(34):
        for bad in (math.nan, math.inf):
            x = k.clone()
            x[j, :, 0] = bad
            out, lse = _run(adt, q, x, v, causal)
            sees = visible > j
            assert bool(torch.isnan(out[sees]).all()) and bool(torch.isnan(lse[:, sees]).all()), (j, bad)
            assert torch.equal(out[~sees], clean[~sees]) and torch.equal(lse[:, ~sees], clean_lse[:, ~sees]), (j, bad)
    adt.sage_check()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name", list(FORMS))
def test_scores_of_minus_infinity(adt, dtype, name):
    """One such key weighs nothing; a row that sees no other has no softmax."""
    q, k, v, visible, causal, heads = _one(name, dtype)
    G, D = q.shape[1] // k.shape[1], q.shape[2]
    for j in (0, 17):
        x = k.clone()
        x[j, :, 0] = -math.inf
        out, lse = _run(adt, q, x, v, causal)
        rows = visible > j + 1
        for h in heads:
            ref = attend(q[rows, h].double(), x[:, h // G].double(), v[:, h // G].double(), visible[rows], D ** -0.5,
                         torch.finfo(dtype).eps / 2)
            check(out[rows, h], lse[h, rows], *ref, what=(j, h))
    k[:, :, 0] = -math.inf
    out, _ = _run(adt, q, k, v, causal)
    assert bool(torch.isnan(out[visible > 0]).all())
    adt.sage_check()


def test_a_query_that_is_no_number(adt):
    for dtype in TYPES:
        q, k, v, visible, causal, _ = _one("alone", dtype)
        clean, _ = _run(adt, q, k, v, causal)
        k[..., 1] = -k[..., 1].abs() - 0.25
        clean, _ = _run(adt, q, k, v, causal)
        q[137, 1, 1], q[391, 0, 1] = math.inf, math.nan          # every score of row 137 is -inf
        out, _ = _run(adt, q, k, v, causal)
        assert bool(torch.isnan(out[137, 1]).all()) and bool(torch.isnan(out[391, 0]).all())
        q[137, 1, 1], q[391, 0, 1] = 1, 1
        same = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
        same[137, 1] = same[391, 0] = False
        assert torch.equal(out[same], clean[same])
