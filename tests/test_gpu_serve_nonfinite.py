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


# ---------------------------------------------------------------------------------------------- V on either side
def _check_v(out, lse, q, k, v, cq, ck, causal, heads):
    """Every channel against the definition: sums over the visible keys alone, so a NaN or infinity among them decides
    the channel (each weight is above 0), and what the others hold does not matter."""
    G, D = q.shape[1] // k.shape[1], q.shape[2]
    for s in range(len(cq) - 1):
        a, b, c, d = cq[s], cq[s + 1], ck[s], ck[s + 1]
        n = torch.arange(b - a, device="cuda") + 1 + (d - c) - (b - a)
        vis = n.clamp(0, d - c) if causal else torch.full_like(n, d - c)
        for h in heads:
            y = v[c:d, h // G].double()
            ref, ref_lse, tol, tol_lse = attend(q[a:b, h].double(), k[c:d, h // G].double(), y, vis, D ** -0.5,
                                                torch.finfo(q.dtype).eps / 2)
            upto = lambda m: torch.cat([torch.zeros(1, D, device="cuda"), m.double().cumsum(0)])[vis] > 0  # noqa: E731
            nan, up, down = upto(torch.isnan(y)), upto(y == math.inf), upto(y == -math.inf)
            ref = torch.where(up, math.inf, torch.where(down, -math.inf, ref))
            ref = torch.where(nan | (up & down), math.nan, ref)
            fine = torch.isfinite(ref)
            got = out[a:b, h]
            assert torch.equal(torch.isnan(got), torch.isnan(ref)), (s, h)
            assert torch.equal(got.double()[torch.isinf(ref)], ref[torch.isinf(ref)]), (s, h)
            check(got[fine], None, ref[fine], None, tol[fine], None, what=(s, h))
            assert bool(((lse[h, a:b].double() - ref_lse).abs()[vis > 0] <= tol_lse[vis > 0]).all()), (s, h)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lq,lk,Hq,Hk,D,causal,heads", [
    ([300], [300], 320, 80, 64, True, [0, 159, 319]),              # pairs over heads
    ([200, 56], [640, 130], 100, 100, 128, True, [0, 57]),         # pairs over rows
    ([400, 3, 250], [400, 300, 251], 3, 1, 128, True, [0, 2]),     # row tiles alone
    ([150, 100], [333, 200], 4, 2, 64, False, [0, 3]),
    ([60], [2000], 2, 1, 128, True, [0, 1]),                       # clusters
    ([130, 40], [1500, 1100], 4, 2, 64, False, [0, 2]),
])
@pytest.mark.parametrize("kind", ["a few", "some channels", "often", "the next sequence"])
def test_v_that_is_no_number(adt, dtype, lq, lk, Hq, Hk, D, causal, heads, kind):
    g = torch.Generator(device="cuda").manual_seed(sum(lk) + D)
    q, k, v = _inputs(lq, lk, Hq, Hk, D, dtype, seed=sum(lk))
    cq = [sum(lq[:i]) for i in range(len(lq) + 1)]
    ck = [sum(lk[:i]) for i in range(len(lk) + 1)]
    v = v.contiguous()
    rate = {"a few": 0.3 / D / sum(lk) * 16, "some channels": 0.05, "often": 0.02, "the next sequence": 0.5}[kind]
    at = torch.rand(v.shape, generator=g, device="cuda") < rate
    if kind == "some channels":
        at[..., 5:] = False
    if kind == "a few":
        at[lk[0] * 2 // 3, :, 7] = True
    if kind == "the next sequence":
        at[: ck[1]] = False
    bad = torch.tensor([math.nan, math.inf, -math.inf], device="cuda", dtype=dtype)
    v[at] = bad[torch.randint(0, 3, (int(at.sum()),), generator=g, device="cuda")]
    out = torch.full((sum(lq), Hq, D), 9.0, device="cuda").to(dtype)
    lse = torch.full((Hq, sum(lq)), 9.0, device="cuda")
    adt.sage_attn_prompt(q, k, v, cq, ck, out, lse, causal=causal)
    adt.sage_check()
    _check_v(out, lse, q, k, v, cq, ck, causal, heads)
    again = torch.empty_like(out)
    adt.sage_attn_prompt(q, k, v, cq, ck, again, causal=causal)
    assert torch.equal(torch.nan_to_num(out, 1.5, 2.5, 3.5), torch.nan_to_num(again, 1.5, 2.5, 3.5))


def test_v_near_the_end_of_its_type(adt):
    """Finite values whose sum before the division would not be."""
    q, k, v = _inputs([300], [300], 2, 1, 64, torch.bfloat16, seed=5)
    v = v.contiguous()
    v[40:, :, 3] = 1e38
    lse = torch.empty(2, 300, device="cuda")
    out = adt.sage_attn_prompt(q, k, v, [0, 300], lse=lse)
    _check_v(out, lse, q, k, v, [0, 300], [0, 300], True, [0, 1])


@pytest.mark.parametrize("lq,lk,Hq", [(2048, 2048, 8), (100, 4096, 8)])
@pytest.mark.parametrize("bad", ["one token", "channels", "all"])
def test_what_is_seen_costs_no_second_pass(adt, lq, lk, Hq, bad):
    """A NaN or an infinity in a visible row of V is the row's own: scores are not formed again for it.  (They took a
    few hundred times as long; what is left is a look at V.)"""
    q, k, v = _inputs([lq], [lk], Hq, Hq, 128, torch.bfloat16, seed=8)
    p = v.contiguous()
    if bad == "one token":
        p[0] = math.nan
    elif bad == "channels":
        p[::7, :, 11] = math.inf
    else:
        p[:] = math.nan
    out = torch.empty(lq, Hq, 128, dtype=torch.bfloat16, device="cuda")

    def us(y):
        adt.sage_attn_prompt(q, k, y, [0, lq], [0, lk], out)
        best = math.inf
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            adt.sage_attn_prompt(q, k, y, [0, lq], [0, lk], out)
            b.record()
            b.synchronize()
            best = min(best, 1e3 * a.elapsed_time(b))
        return best

    clean, poisoned = us(v), us(p)
    assert poisoned < 12 * clean, (clean, poisoned)
