"""sage_attn_token against plain attention in 64 bits over the dequantized cache.

On top of the bound of tests/serve_ref.py: P is rounded to f16 (half a step, 2^-11), and q to f16 after a power of two
(off by at most 2^-25 of its largest channel, so a score by D 2^-25 max|q| max|k| * scale)."""
import math

import pytest
import torch

from tests.serve_ref import attend, check

pytestmark = pytest.mark.gpu


def _setup(adt, lens, Hq, Hk, D, ps, fmt, dtype, seed=0, garbage=True, spread=0.5):
    """A cache whose pages are shuffled; slots that no sequence holds are filled with bytes of every kind."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B = len(lens)
    need = [-(-n // ps) for n in lens]
    pages = sum(need) + 2
    cache = adt.KVCache(pages, ps, Hk, D, fmt)
    if garbage:
        cache.k_codes.view(torch.uint8).random_(0, 256, generator=g)
        cache.v_codes.view(torch.uint8).fill_(0x7F)                # an E4M3 NaN
        cache.k_scale.fill_(float("nan"))
        cache.v_scale.fill_(float("inf"))
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).int()
    table = torch.full((B, max(need + [1]) + 1), -7, dtype=torch.int32)
    at, slots = 0, []
    for b, n in enumerate(need):
        table[b, :n] = order[at: at + n]
        at += n
        i = torch.arange(lens[b])
        slots.append(table[b].long()[i // ps] * ps + i % ps)
    slots = torch.cat(slots).cuda()
    T = sum(lens)
    k = torch.randn(T, Hk, D, generator=g, device="cuda") + torch.randn(Hk, D, generator=g, device="cuda")
    v = torch.randn(T, Hk, D, generator=g, device="cuda")
    v = v * torch.exp(spread * torch.randn(T, Hk, 1, generator=g, device="cuda"))
    if T:
        cache.write(k.to(dtype), v.to(dtype), slots)
    q = (1.5 * torch.randn(B, Hq * D + 8, generator=g, device="cuda")).to(dtype)[:, : Hq * D].view(B, Hq, D)
    return cache, q, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), slots


def _workspace(adt, q, cache, table):
    n = adt.attn_token_workspace_bytes(q.shape[0], q.shape[1], cache.Hk, cache.D, table.shape[1] * cache.page_size)
    return torch.empty(max(256, n), dtype=torch.uint8, device="cuda")


def _compare(out, lse, cache, q, lens, slots, scale=None):
    B, Hq, D = q.shape
    G = Hq // cache.Hk
    scale = D ** -0.5 if scale is None else scale
    T = int(sum(lens))
    flat = lambda c, s: (c.double() * s.double()[..., None]).permute(0, 2, 1, 3).reshape(-1, cache.Hk, D)  # noqa: E731
    k, v = flat(cache.k_codes.float(), cache.k_scale)[slots], flat(cache.v_codes.float(), cache.v_scale)[slots]
    at = 0
    for b, n in enumerate(lens):
        for h in range(Hq):
            x, y = k[at: at + n, h // G], v[at: at + n, h // G]
            ref, ref_lse, tol, tol_lse = attend(q[b, h][None].double(), x, y, torch.tensor([n], device="cuda"), scale,
                                                2.0 ** -11)
            if n:
                e = 2.0 ** -25 * D * float(q[b, h].abs().max()) * float(x.abs().max()) * scale
                tol = tol + 4 * e * tol / (2.0 ** -11)
                tol_lse = tol_lse + 2 * e
            check(out[b, h][None], None if lse is None else lse[b, h][None], ref, ref_lse, tol, tol_lse, what=(b, h))
        at += n
    assert at == T


CASES = [
    # lens, Hq, Hk, D, page
    ([1], 1, 1, 64, 16),
    ([15, 16, 17, 1], 8, 2, 128, 16),
    ([0, 5, 0], 4, 4, 64, 32),
    ([100, 3000, 64], 24, 8, 128, 64),
    ([777, 2049], 7, 1, 64, 128),
    ([130, 1], 32, 2, 128, 16),          # 16 heads to a KV head
    ([500], 40, 1, 64, 1024),            # 40 heads to a KV head: three blocks
    ([4097] + [33] * 40, 16, 8, 128, 16),
    ([9000], 9, 3, 128, 256),
]


@pytest.mark.parametrize("fmt,dtype", [("int8", torch.bfloat16), ("e4m3", torch.float16), ("e4m3", torch.bfloat16),
                                       ("int8", torch.float16)])
@pytest.mark.parametrize("lens,Hq,Hk,D,ps", CASES)
def test_token(adt, fmt, dtype, lens, Hq, Hk, D, ps):
    cache, q, table, ln, slots = _setup(adt, lens, Hq, Hk, D, ps, fmt, dtype, seed=sum(lens))
    B = len(lens)
    ws = _workspace(adt, q, cache, table)
    out = torch.full((B, Hq, D), 9.0, device="cuda").to(dtype)
    lse = torch.full((B, Hq), 9.0, device="cuda")
    cache.attend(q, table, ln, out, ws, lse=lse)
    adt.sage_check()
    _compare(out, lse, cache, q, lens, slots)
    # a tighter bound on the lengths splits the keys otherwise; the same launch twice gives the same bits
    m = max(lens)
    a, b = torch.empty_like(out), torch.empty_like(out)
    cache.attend(q, table, ln, a, ws, max_len=m)
    ws.fill_(0xFF)
    cache.attend(q, table, ln, b, ws, max_len=m)
    adt.sage_check()
    assert torch.equal(a, b)
    _compare(a, None, cache, q, lens, slots)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_v_scales_of_very_different_size(adt, fmt):
    """Heavy V rows that get almost no weight beside small ones that get all of it: the weights' power of two follows."""
    L, Hq, Hk, D, ps = 600, 4, 2, 64, 16
    cache, q, table, ln, slots = _setup(adt, [L], Hq, Hk, D, ps, fmt, torch.bfloat16, seed=3)
    g = torch.Generator(device="cuda").manual_seed(1)
    k = 0.05 * torch.randn(L, Hk, D, generator=g, device="cuda")
    v = torch.randn(L, Hk, D, generator=g, device="cuda")
    qm = q.float().reshape(Hk, 2, D).mean(1)
    k[300:310] = 4 * qm                                           # the keys that matter, late
    v[:300] *= 3e3
    v[300:310] *= 1e-4
    cache.write(k.bfloat16(), v.bfloat16(), slots)
    ws = _workspace(adt, q, cache, table)
    out, lse = torch.empty_like(q.contiguous()), torch.empty(1, Hq, device="cuda")
    cache.attend(q, table, ln, out, ws, lse=lse, sm_scale=0.5)
    _compare(out, lse, cache, q, [L], slots, scale=0.5)


def test_queries_of_every_size(adt):
    """q near the ends of its type's range: the scale of the scores absorbs the power of two."""
    lens, Hq, Hk, D, ps = [200, 200, 200], 4, 4, 64, 16
    cache, q, table, ln, slots = _setup(adt, lens, Hq, Hk, D, ps, "int8", torch.bfloat16, seed=5)
    q = q.clone()
    q[0] *= 1e-30
    q[1] = 0
    ws = _workspace(adt, q, cache, table)
    out, lse = torch.empty_like(q), torch.empty(3, Hq, device="cuda")
    cache.attend(q, table, ln, out, ws, lse=lse)
    _compare(out, lse, cache, q, lens, slots)
    q[2] *= 1e30
    cache.attend(q, table, ln, out, ws, sm_scale=1e-30)
    _compare(out[2:], None, cache, q[2:], [200], slots[400:], scale=1e-30)


def test_a_poisoned_row_reaches_its_sequence_only(adt):
    lens, Hq, Hk, D, ps = [70, 90], 4, 2, 64, 16
    cache, q, table, ln, slots = _setup(adt, lens, Hq, Hk, D, ps, "e4m3", torch.float16, seed=7)
    bad = torch.full((1, Hk, D), float("inf"), device="cuda", dtype=torch.float16)
    fine = torch.ones_like(bad)
    cache.write(fine, bad, slots[30:31].clone())
    ws = _workspace(adt, q, cache, table)
    out = torch.empty_like(q.contiguous())
    cache.attend(q, table, ln, out, ws)
    assert bool(torch.isnan(out[0]).all()) and bool(torch.isfinite(out[1]).all())
    ln[0] = 30                                                    # not seen any more
    cache.attend(q, table, ln, out, ws)
    assert bool(torch.isfinite(out).all())


def test_bad_pages_and_lengths_are_left_out_and_reported(adt):
    lens, Hq, Hk, D, ps = [64, 64], 2, 1, 64, 16
    cache, q, table, ln, slots = _setup(adt, lens, Hq, Hk, D, ps, "int8", torch.bfloat16, seed=8)
    ws = _workspace(adt, q, cache, table)
    out = torch.empty_like(q.contiguous())
    lse = torch.empty(2, Hq, device="cuda")
    cache.attend(q, table, ln, out, ws, lse=lse, max_len=64)
    keep = out.clone()
    t2 = table.clone()
    t2[0, 1], t2[0, 2] = cache.num_pages, -1
    cache.attend(q, t2, ln, out, ws, lse=lse, max_len=64)
    assert adt.sage_check_status() == 1 and adt.sage_check_status() == 0
    sub = torch.cat([slots[:16], slots[48:64], slots[64:]])
    _compare(out[:1], lse[:1], cache, q[:1], [32], sub[:32])
    assert torch.equal(out[1], keep[1])
    ln2 = ln.clone()
    ln2[1], ln2[0] = 1 << 30, -5
    cache.attend(q, table, ln2, out, ws, lse=lse, max_len=64)
    assert adt.sage_check_status() == 1
    assert torch.equal(out[1], keep[1]) and bool((out[0] == 0).all()) and bool(torch.isinf(lse[0]).all())


def test_graph_replay_follows_lens_and_pages(adt):
    lens, Hq, Hk, D, ps = [400, 900], 8, 2, 128, 32
    cache, q, table, ln, slots = _setup(adt, lens, Hq, Hk, D, ps, "int8", torch.bfloat16, seed=12)
    ws = _workspace(adt, q, cache, table)
    out, lse = torch.empty_like(q.contiguous()), torch.empty(2, Hq, device="cuda")
    cache.attend(q, table, ln, out, ws, lse=lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.attend(q, table, ln, out, ws, lse=lse)
    ln.copy_(torch.tensor([17, 333], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    adt.sage_check()
    _compare(out, lse, cache, q, [17, 333], torch.cat([slots[:17], slots[400:733]]))


def test_no_sequences(adt):
    cache = adt.KVCache(1, 16, 2, 64)
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    out = cache.attend(q, torch.empty(0, 3, dtype=torch.int32, device="cuda"),
                       torch.empty(0, dtype=torch.int32, device="cuda"), q.clone(), None)
    assert out.shape == (0, 4, 64) and math.prod(out.shape) == 0


def _one_long(adt, L, fmt, dtype, D=128, seed=0):
    """One sequence of L keys among 56 with 8 KV heads: its keys are one chunk, so each warp takes many tiles."""
    return _setup(adt, [L] + [1] * 55, 16, 8, D, 32, fmt, dtype, seed=seed)


@pytest.mark.parametrize("fmt,dtype", [("int8", torch.bfloat16), ("e4m3", torch.float16), ("e4m3", torch.bfloat16),
                                       ("int8", torch.float16)])
@pytest.mark.parametrize("amax", [1.0, 1e-2, 1e-4])
def test_v_rows_of_zeros_first(adt, fmt, dtype, amax):
    """The power of two on the weights waits for the first weight that is not zero."""
    L = 1500
    cache, q, table, ln, slots = _one_long(adt, L, fmt, dtype, seed=17)
    g = torch.Generator(device="cuda").manual_seed(2)
    k = 0.2 * torch.randn(L, 8, 128, generator=g, device="cuda")
    k[:200] *= 4                                                  # the reference does not rise any more
    v = torch.randn(L, 8, 128, generator=g, device="cuda")
    v = amax * v / v.abs().amax(-1, keepdim=True)
    v[:200] = 0
    cache.write(k.to(dtype), v.to(dtype), slots[:L])
    out, lse = torch.empty_like(q.contiguous()), torch.empty(56, 16, device="cuda")
    cache.attend(q, table, ln, out, _workspace(adt, q, cache, table), lse=lse)
    adt.sage_check()
    _compare(out[:1], lse[:1], cache, q[:1], [L], slots[:L])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_v_of_every_size(adt, fmt):
    """V near both ends of bfloat16's range, and both in one sequence.  A weight below 2^-126 of the largest is 0 in 32
    bits, so the earlier values may be missing from the third case: up to L 2^-126 3e38 < 2^13 = 8192."""
    L = 1500
    cache, q, table, ln, slots = _one_long(adt, L, fmt, torch.bfloat16, seed=18)
    g = torch.Generator(device="cuda").manual_seed(3)
    ws = _workspace(adt, q, cache, table)
    out, lse = torch.empty_like(q.contiguous()), torch.empty(56, 16, device="cuda")
    n = torch.randn(L, 8, 128, generator=g, device="cuda")
    n = n / n.abs().amax(-1, keepdim=True)
    plain = 0.2 * torch.randn(L, 8, 128, generator=g, device="cuda")
    late = plain.clone()
    late[700:] += 8 * q[0].float().view(8, 2, 128).mean(1)       # scores far above the earlier ones
    for k, first, then in ((plain, 3e38, 3e38), (plain, 1e-27, 1e-27), (late, 3e38, 1e-27), (late, 1e-27, 3e38),
                           (plain, 1e-27, 3e38)):
        v = n * first
        v[700:] = n[700:] * then
        cache.write(k.bfloat16(), v.bfloat16(), slots[:L])
        cache.attend(q, table, ln, out, ws, lse=lse)
        if first > then and k is late:
            x, y = cache.k_codes.double() * cache.k_scale.double()[..., None], cache.v_codes.double() * cache.v_scale.double()[..., None]
            x, y = (z.permute(0, 2, 1, 3).reshape(-1, 8, 128)[slots[:L]] for z in (x, y))
            for h in range(16):
                ref, _, tol, _ = attend(q[0, h][None].double(), x[:, h // 2], y[:, h // 2],
                                        torch.tensor([L], device="cuda"), 128 ** -0.5, 2.0 ** -11)
                err = (out[0, h][None].double() - ref).abs()
                assert bool((err <= 2.0 ** -8 * (ref.abs() + tol) + tol + 8192).all()), h
        else:
            _compare(out[:1], lse[:1], cache, q[:1], [L], slots[:L])


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_query_that_is_no_number(adt, bad):
    """Every score of such a head is an infinity or no number, so it has no softmax; its neighbours are as before."""
    lens, Hq, Hk, D, ps = [70, 300, 0], 4, 2, 64, 16
    for fmt, dtype in (("int8", torch.bfloat16), ("e4m3", torch.float16)):
        cache, q, table, ln, slots = _setup(adt, lens, Hq, Hk, D, ps, fmt, dtype, seed=19, garbage=False)
        k = torch.randn(370, Hk, D, device="cuda").abs() + 0.25
        cache.write(-k.to(dtype), k.to(dtype), slots)            # one sign: no score is 0 times an infinity
        ws = _workspace(adt, q, cache, table)
        clean = cache.attend(q, table, ln, torch.empty_like(q.contiguous()), ws)
        q = q.clone()
        q[0, 1, 7] = q[1, 2, 7] = q[2, 0, 7] = bad
        lse = torch.empty(3, Hq, device="cuda")
        out = cache.attend(q, table, ln, torch.empty_like(clean), ws, lse=lse)
        for b, h in ((0, 1), (1, 2)):
            assert bool(torch.isnan(out[b, h]).all()) and bool(torch.isnan(lse[b, h]))
            out[b, h] = clean[b, h]
        assert torch.equal(out, clean) and bool((out[2] == 0).all())      # without keys: zeros


@pytest.mark.parametrize("lens", [[70, 0, 300], [9000]])
def test_in_place(adt, lens):
    """out may be q: with the keys in one chunk, and in many."""
    cache, q, table, ln, slots = _setup(adt, lens, 8, 2, 64, 16, "int8", torch.bfloat16, seed=23)
    ws = _workspace(adt, q, cache, table)
    want = cache.attend(q, table, ln, torch.empty_like(q.contiguous()), ws)
    got = q.clone()
    assert cache.attend(got, table, ln, got, ws) is got
    adt.sage_check()
    assert torch.equal(got, want)


def test_any_page_outside_the_cache_is_reported(adt):
    """The lowest int32 too, in each half of a tile; in entries behind the length nothing is."""
    lens, ps = [64, 40], 16
    cache, q, table, ln, slots = _setup(adt, lens, 2, 1, 64, ps, "int8", torch.bfloat16, seed=24)
    ws = _workspace(adt, q, cache, table)
    out = torch.empty_like(q.contiguous())
    want = cache.attend(q, table, ln, torch.empty_like(out), ws)
    for entry, value, status in ((1, -2 ** 31, 1), (2, -2 ** 31, 1), (3, 2 ** 31 - 1, 1), (4, -2 ** 31, 0), (4, 2 ** 31 - 1, 0)):
        bad = table.clone()
        bad[0, entry] = value
        cache.attend(q, bad, ln, out, ws)
        assert adt.sage_check_status() == status, (entry, value)
        assert torch.equal(out[1], want[1]) and torch.equal(out[0], want[0]) == (status == 0)
