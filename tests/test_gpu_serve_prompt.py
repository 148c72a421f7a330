"""sage_attn_prompt against plain attention in 64 bits (tests/serve_ref.py states the bound)."""
import math

import pytest
import torch

from tests.serve_ref import attend, check

pytestmark = pytest.mark.gpu


def _offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _inputs(lq, lk, Hq, Hk, D, dtype, seed=0, pad=8):
    g = torch.Generator(device="cuda").manual_seed(seed)
    Tq, Tk = sum(lq), sum(lk)
    q = (1.5 * torch.randn(Tq, Hq * D + pad, generator=g, device="cuda")).to(dtype)[:, : Hq * D].view(Tq, Hq, D)
    kv = torch.randn(Tk, 2 * Hk * D + pad, generator=g, device="cuda").to(dtype)
    return q, kv[:, : Hk * D].view(Tk, Hk, D), kv[:, Hk * D: 2 * Hk * D].view(Tk, Hk, D)


def _compare(out, lse, q, k, v, cq, ck, causal, scale=None, heads=None):
    Hq, D = q.shape[1], q.shape[2]
    G = Hq // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    for s in range(len(cq) - 1):
        a, b, c, d = cq[s], cq[s + 1], ck[s], ck[s + 1]
        if a == b:
            continue
        n = torch.arange(b - a, device="cuda") + 1 + (d - c) - (b - a)
        vis = n.clamp(0, d - c) if causal else torch.full_like(n, d - c)
        for h in (range(Hq) if heads is None else heads):
            ref = attend(q[a:b, h].double(), k[c:d, h // G].double(), v[c:d, h // G].double(), vis, scale,
                         torch.finfo(q.dtype).eps / 2)
            check(out[a:b, h], lse[h, a:b], *ref, what=(s, h))


CASES = [
    # lq, lk, Hq, Hk, D, causal
    ([1], [1], 1, 1, 64, True),
    ([1], [300], 4, 2, 128, True),
    ([128], [128], 2, 1, 128, True),
    ([256], [256], 2, 2, 64, True),
    ([129], [129], 3, 1, 128, True),
    ([257, 1, 127], [257, 1, 127], 4, 1, 64, True),
    ([77, 130, 1, 333, 64, 19, 256, 100], None, 4, 2, 128, True),
    ([100, 40, 0, 200], [1000, 40, 77, 333], 2, 1, 128, True),      # continued prompts, an empty one
    ([300, 129], [7, 128], 2, 1, 64, True),                        # fewer keys than queries: rows without any
    ([200, 50], [0, 60], 2, 2, 128, True),                         # no keys at all
    ([300], [500], 2, 2, 128, False),
    ([50, 200], [1, 129], 6, 2, 64, False),
    ([1500], [1500], 7, 1, 128, True),
    ([900], [2600], 2, 1, 64, True),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lq,lk,Hq,Hk,D,causal", CASES)
def test_prompt(adt, dtype, lq, lk, Hq, Hk, D, causal):
    lk = lq if lk is None else lk
    q, k, v = _inputs(lq, lk, Hq, Hk, D, dtype, seed=sum(lq) + D)
    cq, ck = _offsets(lq), _offsets(lk)
    out = torch.full((sum(lq), Hq, D), 9.0, device="cuda").to(dtype)
    lse = torch.full((Hq, sum(lq)), 9.0, device="cuda")
    adt.sage_attn_prompt(q, k, v, cq, ck, out, lse, causal=causal)
    adt.sage_check()
    _compare(out, lse, q, k, v, cq, ck, causal)
    again = torch.empty_like(out)
    adt.sage_attn_prompt(q, k, v, cq, torch.tensor(ck, dtype=torch.int32), again, causal=causal)
    assert torch.equal(out, again)


def test_scale_and_large_scores(adt):
    """Scores that grow along the row move the reference often; an own sm_scale."""
    L, D = 700, 128
    q, k, v = _inputs([L], [L], 2, 1, D, torch.bfloat16, seed=4)
    k = (k.float() * torch.linspace(0.05, 6, L, device="cuda")[:, None, None]).bfloat16()
    lse = torch.empty(2, L, device="cuda")
    out = adt.sage_attn_prompt(q, k, v, [0, L], lse=lse, sm_scale=0.2)
    _compare(out, lse, q, k, v, [0, L], [0, L], True, scale=0.2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_what_masked_places_hold_does_not_matter(adt, dtype):
    """Infinities and NaN in the K and V of later tokens and of the next sequence."""
    L, D = 200, 64
    q, k, v = _inputs([L, 90], [L, 90], 2, 1, D, dtype, seed=6)
    clean = adt.sage_attn_prompt(q, k, v, [0, L, L + 90])
    q2, k2, v2 = q.clone(), k.clone(), v.clone()
    k2[L:], v2[L:] = float("nan"), float("inf")                     # the next sequence
    k2[150:L], v2[150:L] = float("inf"), float("nan")               # later tokens of the first
    v2[149, :, 5] = float("-inf")                                   # one channel of one token
    got = adt.sage_attn_prompt(q2, k2, v2, [0, L, L + 90])
    adt.sage_check()
    lim = 2 * torch.finfo(dtype).eps * clean[:149].double().abs() + 4 * torch.finfo(dtype).eps
    assert bool(((got[:149].double() - clean[:149].double()).abs() <= lim).all())
    assert bool(torch.isinf(got[149, :, 5]).all()) and bool(torch.isfinite(got[149, :, :5]).all())
    assert bool(torch.isnan(got[150:L]).all())


def test_more_sequences_than_one_launch(adt):
    lens = [(7 * i) % 23 for i in range(300)]
    cu = _offsets(lens)
    q, k, v = _inputs(lens, lens, 2, 1, 64, torch.float16, seed=9)
    lse = torch.empty(2, cu[-1], device="cuda")
    out = adt.sage_attn_prompt(q, k, v, cu, lse=lse)
    _compare(out, lse, q, k, v, cu, cu, True)


def test_no_sequences(adt):
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    for cu in ([0], [0, 0, 0]):
        assert adt.sage_attn_prompt(e, e, e, cu).shape == (0, 2, 64)


def test_graph_and_side_stream(adt):
    L, D = 500, 128
    q, k, v = _inputs([L], [L], 4, 2, D, torch.bfloat16, seed=11)
    want = adt.sage_attn_prompt(q, k, v, [0, L])
    out = torch.zeros_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    adt.sage_attn_prompt(q, k, v, [0, L], out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        adt.sage_attn_prompt(q, k, v, [0, L], out=out)
    q.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    adt.sage_check()
    assert torch.equal(out, adt.sage_attn_prompt(q, k, v, [0, L]))
    assert not math.isclose(float((out.float() - want.float()).abs().max()), 0.0)


@pytest.mark.parametrize("lq,lk,Hq,Hk,D,causal,heads", [
    ([700, 300], None, 64, 16, 128, True, [0, 3, 33, 63]),             # two waves of pairs, the last ones parted
    ([600, 90, 1], [2000, 90, 1500], 64, 16, 64, True, [0, 30, 63]),   # long and short pairs mixed
    ([256], [700], 100, 100, 128, False, [0, 57, 99]),                 # one wave of pairs
    ([128, 1], [128, 900], 3, 3, 128, True, None),                     # an item alone with one key tile, with several
    ([64], [640], 5, 1, 64, True, None),
    ([30], [257], 1, 1, 128, False, None),
])
def test_pairs_and_items_alone(adt, lq, lk, Hq, Hk, D, causal, heads):
    """Row tiles that share a CTA, and row tiles alone whose keys are taken by both halves of one."""
    lk = lq if lk is None else lk
    q, k, v = _inputs(lq, lk, Hq, Hk, D, torch.bfloat16, seed=sum(lk) + Hq)
    cq, ck = _offsets(lq), _offsets(lk)
    out = torch.full((sum(lq), Hq, D), 9.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((Hq, sum(lq)), 9.0, device="cuda")
    adt.sage_attn_prompt(q, k, v, cq, ck, out, lse, causal=causal)
    adt.sage_check()
    _compare(out, lse, q, k, v, cq, ck, causal, heads=heads)
    again = torch.empty_like(out)
    adt.sage_attn_prompt(q, k, v, cq, ck, again, causal=causal)
    assert torch.equal(out, again)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lq,lk,Hq,Hk,D,causal", [
    ([1], [5000], 4, 2, 128, True),                        # 8 CTAs per row tile
    ([100, 3], [4096, 130], 4, 4, 64, True),               # a sequence with fewer key tiles than CTAs
    ([257], [4000], 3, 1, 128, False),
    ([128], [2049], 16, 8, 64, True),
    ([300, 20], [1300, 0], 8, 2, 128, True),               # 4; rows without any key
    ([1000], [700], 2, 2, 64, True),                       # rows without any key beside rows with some
    ([640], [640], 13, 13, 128, True),                     # 2
])
def test_row_tiles_shared_by_a_cluster(adt, dtype, lq, lk, Hq, Hk, D, causal):
    """Few row tiles over many keys: several CTAs take the keys of one and join what they found."""
    q, k, v = _inputs(lq, lk, Hq, Hk, D, dtype, seed=sum(lk) + D)
    cq, ck = _offsets(lq), _offsets(lk)
    out = torch.full((sum(lq), Hq, D), 9.0, device="cuda").to(dtype)
    lse = torch.full((Hq, sum(lq)), 9.0, device="cuda")
    adt.sage_attn_prompt(q, k, v, cq, ck, out, lse, causal=causal)
    adt.sage_check()
    _compare(out, lse, q, k, v, cq, ck, causal)
    again = torch.empty_like(out)
    adt.sage_attn_prompt(q, k, v, cq, ck, again, causal=causal)
    assert torch.equal(out, again)


def test_what_masked_places_hold_does_not_matter_to_a_cluster(adt):
    Lq, Lk, D = 60, 3000, 128
    q, k, v = _inputs([Lq], [Lk], 2, 1, D, torch.bfloat16, seed=21)
    clean = adt.sage_attn_prompt(q, k, v, [0, Lq], [0, Lk])
    k2, v2 = k.clone(), v.clone()
    k2[Lk - 20:], v2[Lk - 20:] = float("nan"), float("inf")         # seen by the last 20 rows alone
    v2[7, :, 5] = float("-inf")                                     # one channel of one token, seen by all
    got = adt.sage_attn_prompt(q, k2, v2, [0, Lq], [0, Lk])
    adt.sage_check()
    rest = [c for c in range(D) if c != 5]
    a, b = got[:40][..., rest].double(), clean[:40][..., rest].double()
    lim = 2 * torch.finfo(torch.bfloat16).eps * b.abs() + 4 * torch.finfo(torch.bfloat16).eps
    assert bool(((a - b).abs() <= lim).all())
    assert bool(torch.isinf(got[:40, :, 5]).all()) and bool(torch.isnan(got[40:]).all())


def test_more_pairs_than_are_sorted(adt):
    lens = [1 + (53 * i) % 290 for i in range(150)]
    past = [(31 * i) % 70 for i in range(150)]
    lk = [a + b for a, b in zip(lens, past)]
    cq, ck = _offsets(lens), _offsets(lk)
    q, k, v = _inputs(lens, lk, 9, 1, 64, torch.bfloat16, seed=31)
    lse = torch.empty(9, cq[-1], device="cuda")
    out = adt.sage_attn_prompt(q, k, v, cq, ck, lse=lse)
    adt.sage_check()
    _compare(out, lse, q, k, v, cq, ck, True, heads=[0, 8])


def test_graph_with_clusters_beside_an_eager_call(adt):
    Lq, Lk, D = 100, 3000, 128
    q, k, v = _inputs([Lq], [Lk], 4, 2, D, torch.float16, seed=33)
    cu = [0, Lq], [0, Lk]
    want = adt.sage_attn_prompt(q, k, v, *cu)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        adt.sage_attn_prompt(q, k, v, *cu, out=out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = torch.empty_like(want)
    for _ in range(3):
        graph.replay()
        adt.sage_attn_prompt(q, k, v, *cu, out=other, stream=side)
    torch.cuda.synchronize()
    adt.sage_check()
    assert torch.equal(out, want) and torch.equal(other, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("low", [-0.125, -0.25, -0.3125, -0.5, -0.75])
def test_log_sum_exp_keeps_32_bits(adt, dtype, low):
    """Scores without rounding (one channel, powers and short fractions): key 2 scores 0, keys 0 and 1 of every 16
    `low`, the others -40.  Each weight is off by 2^-21 at most (its exponential, with the argument's rounding), the sum
    of 256 of them by 256 2^-24, the logarithm and the result by 2^-22 of themselves each."""
    L, D = 256, 64
    q, k = torch.zeros(128, 1, D, device="cuda"), torch.full((L, 1), -40.0, device="cuda")
    q[..., 0] = 1
    at = torch.arange(L, device="cuda") % 16 < 2
    k[at] = low
    k[2] = 0
    k = torch.nn.functional.pad(k[..., None], (0, D - 1))
    lse = torch.empty(1, 128, device="cuda")
    out = adt.sage_attn_prompt(q.to(dtype), k.to(dtype), torch.ones_like(k).to(dtype), [0, 128], [0, L], lse=lse,
                               causal=False, sm_scale=1.0)
    want = math.log(1 + 32 * math.exp(low) + 223 * math.exp(-40.0))
    tol = 2.0 ** -21 + L * 2.0 ** -24 + 2 * 2.0 ** -22 * abs(want)
    assert float((lse.double() - want).abs().max()) <= tol
    assert bool((out == 1).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lq", [1, 300])
def test_many_small_weights(adt, dtype, lq):
    """65535 keys of e^-18 of the largest weight each, a thousandth together, carry a channel of their own."""
    L, D = 65536, 64
    q = torch.zeros(lq, 2, D, device="cuda", dtype=dtype)
    q[..., 0] = 1
    k = torch.zeros(L, 1, D, device="cuda", dtype=dtype)
    k[1:, :, 0] = -18
    v = torch.zeros(L, 1, D, device="cuda", dtype=dtype)
    v[0, :, 32:], v[1:, :, :32] = 1, 1
    lse = torch.empty(2, lq, device="cuda")
    out = adt.sage_attn_prompt(q, k, v, [0, lq], [0, L], lse=lse, causal=False, sm_scale=1.0)
    _compare(out, lse, q, k, v, [0, lq], [0, L], False, scale=1.0)


def test_own_output_on_a_given_stream(adt):
    """An output that the call makes belongs to the stream that writes it: released at once, its memory is not handed
    to the current stream while that one still writes."""
    q, k, v = _inputs([300], [300], 2, 1, 64, torch.bfloat16, seed=40)
    want = adt.sage_attn_prompt(q, k, v, [0, 300])
    torch.cuda.synchronize()
    for side in (torch.cuda.Stream(),):
        for given in (side, side.cuda_stream):
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                torch.cuda._sleep(20_000_000)
            out = adt.sage_attn_prompt(q, k, v, [0, 300], stream=given)
            at = out.data_ptr()
            keep = [torch.zeros_like(want) for _ in range(4)]
            del out
            keep += [torch.zeros_like(want) for _ in range(4)]
            side.synchronize()
            assert at not in [t.data_ptr() for t in keep] and all(not bool(t.any()) for t in keep)
            out = adt.sage_attn_prompt(q, k, v, [0, 300], stream=given)
            side.synchronize()
            assert torch.equal(out, want)
