"""Rotary positions and the quantized KV cache against plain implementations.

sage_rope: the angle is exact to 2^-25 half revolutions (one rounding of the fraction to 32 bits) and cos / sin to a
unit or two of 2^-24, so each of the two products is off by less than 2^-22 of its factor; the result is rounded once.
|err| <= (eps / 2) |ref| + 2^-21 m (|a| + |b|) (+ half the smallest FP16 step).
sage_kv_write and sage_kv_read follow rules whose every rounding is fixed: compared bit for bit.
"""
import math

import numpy as np
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]


def _rope_ref(x, angle, m, r, pairs, transpose=False):
    """(result, |a| + |b| of each channel) in 64 bits; angle [T, r/2]."""
    y, size = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    c, s = (angle.cos() * m)[:, None], (angle.sin() * m * (-1 if transpose else 1))[:, None]
    ia = torch.arange(0, r, 2) if pairs else torch.arange(r // 2)
    ib = ia + 1 if pairs else ia + r // 2
    a, b = y[..., ia].clone(), y[..., ib].clone()
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    size[..., ia] = size[..., ib] = (a.abs() + b.abs()) * m
    return y, size


def _rope_check(got, ref, size, r):
    t = got.dtype
    tol = torch.finfo(t).eps / 2 * ref.abs() + 2.0 ** -21 * size + (2.0 ** -25 if t == torch.float16 else 0.0)
    assert bool(((got.double() - ref).abs() <= tol)[..., :r].all()), float(((got.double() - ref).abs() - tol).max())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,Hq,Hk,D,r,pairs", [
    (1, 32, 8, 128, 128, False), (1, 1, 1, 64, 64, True), (3, 4, 4, 64, 40, False), (5, 3, 1, 96, 30, False),
    (7, 6, 2, 128, 36, True), (130, 5, 2, 64, 16, False), (700, 24, 24, 128, 128, True), (2049, 32, 4, 128, 64, False),
    (33, 2, 2, 256, 256, False), (9, 2, 1, 256, 2, True), (11, 40, 8, 8, 8, False),
])
def test_rope(adt, dtype, T, Hq, Hk, D, r, pairs):
    g = torch.Generator(device="cuda").manual_seed(T + D)
    qkv = torch.randn(T, (Hq + 2 * Hk) * D + 8, generator=g, device="cuda").to(dtype)
    q = qkv[:, : Hq * D].view(T, Hq, D)
    k = qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
    before = qkv.clone()
    pos = torch.randint(-5, 1_000_000, (T,), generator=g, device="cuda")
    plan = adt.RopePlan(r, base=10000.0, interleaved=pairs)
    f = 10000.0 ** (-2.0 * torch.arange(r // 2, dtype=torch.float64, device="cuda") / r)
    angle = pos.double()[:, None] * f
    q_out, k_out = torch.full((T, Hq, D), 7.0, device="cuda").to(dtype), torch.empty(T, Hk, D, dtype=dtype, device="cuda")
    adt.sage_rope(q, k, pos, plan, q_out, k_out)
    adt.sage_check()
    assert torch.equal(qkv, before)
    for x, y in ((q, q_out), (k, k_out)):
        ref, size = _rope_ref(x, angle, 1.0, r, pairs)
        _rope_check(y, ref, size, r)
        assert torch.equal(y[..., r:], x[..., r:])
    # in place, on the strided view: the same bits, and nothing beside the heads changes
    adt.sage_rope(q, k, pos, plan)
    assert torch.equal(q, q_out) and torch.equal(k, k_out)
    assert torch.equal(qkv[:, (Hq + Hk) * D:], before[:, (Hq + Hk) * D:])
    # one of the two alone
    q2, _ = adt.sage_rope(before[:, : Hq * D].view(T, Hq, D), None, pos, plan, q_out=torch.empty_like(q_out))
    assert torch.equal(q2, q_out)


@pytest.mark.parametrize("D,r,pairs", [(8, 2, True), (8, 2, False), (16, 6, False)])
def test_rope_of_many_narrow_rows(adt, D, r, pairs):
    """A million one-head rows: many tokens to a CTA, the angles bounded in shared memory."""
    T = 1_300_003
    g = torch.Generator(device="cuda").manual_seed(D)
    x = torch.randn(T, 1, D, generator=g, device="cuda").half()
    pos = torch.arange(T, device="cuda")
    f = 10000.0 ** (-2.0 * torch.arange(r // 2, dtype=torch.float64, device="cuda") / r)
    got, _ = adt.sage_rope(x, None, pos, adt.RopePlan(r, interleaved=pairs), q_out=torch.empty_like(x))
    adt.sage_check()
    ref, size = _rope_ref(x, pos.double()[:, None] * f, 1.0, r, pairs)
    _rope_check(got, ref, size, r)
    assert torch.equal(got[..., r:], x[..., r:])


@pytest.mark.parametrize("scaling,factor", [(None, 1.0), ("linear", 8.0), ("ntk", 4.0), ("yarn", 16.0)])
def test_rope_scaling_far_out(adt, scaling, factor):
    T, H, D, r, L0 = 64, 2, 128, 128, 4096
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, H, D, generator=g, device="cuda")
    pos = torch.randint(0, 1 << 40, (T,), generator=g, device="cuda")
    pos[:16] = torch.randint(0, 100_000, (16,), generator=g, device="cuda")
    pos[0] = 0
    i = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    base = 500000.0 * (factor ** (r / (r - 2)) if scaling == "ntk" else 1.0)
    f, m = base ** (-2 * i / r), 1.0
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        ramp = ((L0 * f / (2 * math.pi) - 1.0) / 31.0).clamp(0, 1)
        f, m = ramp * f + (1 - ramp) * f / factor, 0.1 * math.log(factor) + 1
    plan = adt.RopePlan(r, base=500000.0, scaling=scaling, factor=factor, orig_len=L0)
    assert np.allclose(np.array(plan.struct.turns[: r // 2]) * 2 * math.pi, f.cpu().numpy(), rtol=1e-14, atol=0)
    got, _ = adt.sage_rope(x, None, pos, plan, q_out=torch.empty_like(x))
    near = pos < 1_000_000      # the reference's own angles are exact enough up to there
    ref, size = _rope_ref(x, pos.double()[:, None] * f, m, r, False)
    _rope_check(got[near], ref[near], size[near], r)
    # far out: the plan's revolutions, in exact integer arithmetic
    turns = [plan.struct.turns[j] for j in range(r // 2)]
    frac = torch.tensor([[float((int(p) * int(t * 2.0 ** 90)) % (1 << 90)) / 2.0 ** 90 for t in turns]
                         for p in pos.tolist()], dtype=torch.float64, device="cuda")
    ref, size = _rope_ref(x, frac * 2 * math.pi, m, r, False)
    slack = 2 * math.pi * 2.0 ** -52 * pos.double()[:, None, None] * torch.tensor(turns, device="cuda").repeat(2)
    assert bool(((got.double() - ref).abs() <= 2.0 ** -24 * ref.abs() + (2.0 ** -21 + slack) * size).all())


def test_rope_axes_match_the_joint_tables(adt):
    """The 4-axis tables of the joint blocks, as a plan: frequencies restart on every axis."""
    w = synth.custom(1, 300, 2, 128, seed=5, cu_seqlens=(0, 100, 300))
    inp = synth.normrope_inputs(w)
    n = 16                                                      # pairs per axis at D = 128
    plan = adt.RopePlan(128, interleaved=True, axis=[i // n for i in range(64)],
                        inv_freq=[10000.0 ** (-(i % n) / n) for i in range(64)])
    assert plan.n_axes == 4
    T = 300
    pos = torch.randint(0, 300, (4, T), generator=torch.Generator().manual_seed(1)).cuda()
    x = torch.randn(T, 2, 128, device="cuda")
    got, _ = adt.sage_rope(x, None, pos, plan, q_out=torch.empty_like(x))
    f = torch.tensor([10000.0 ** (-(i % n) / n) for i in range(64)], dtype=torch.float64, device="cuda")
    angle = pos.double().repeat_interleave(n, 0).t() * f
    ref, size = _rope_ref(x, angle, 1.0, 128, True)
    _rope_check(got, ref, size, 128)
    assert inp["cos"].shape == (300, 64)                        # the same pair layout as the tables


@pytest.mark.parametrize("pairs", [False, True])
def test_rope_gradient(adt, pairs):
    """transpose=True is the gradient: against the formula's, and <g, R x> = <R^T g, x> by differences."""
    T, H, D, r = 17, 3, 64, 32
    g = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn(T, H, D, generator=g, device="cuda")
    gy = torch.randn(T, H, D, generator=g, device="cuda")
    pos = torch.randint(0, 5000, (T,), generator=g, device="cuda")
    plan = adt.RopePlan(r, interleaved=pairs, scaling="yarn", factor=4.0, orig_len=512)
    new = lambda: torch.empty_like(x)  # noqa: E731
    gx, _ = adt.sage_rope(gy, None, pos, plan, q_out=new(), transpose=True)
    f = torch.tensor(plan.struct.turns[: r // 2], dtype=torch.float64, device="cuda") * 2 * math.pi
    ref, size = _rope_ref(gy, pos.double()[:, None] * f, plan.struct.mscale, r, pairs, transpose=True)
    _rope_check(gx, ref, size, r)
    # differences: the map is linear, so (loss(x + d) - loss(x)) = <gx, d> for any step
    d = torch.randn(T, H, D, generator=g, device="cuda")
    y0, _ = adt.sage_rope(x, None, pos, plan, q_out=new())
    y1, _ = adt.sage_rope(x + d, None, pos, plan, q_out=new())
    lhs = ((y1.double() - y0.double()) * gy.double()).sum()
    rhs = (gx.double() * ((x + d).double() - x.double())).sum()
    # each of the T H D terms is off by at most 2^-20 of |gy| (|x| + |d|) sizes
    assert abs(float(lhs - rhs)) <= 2.0 ** -20 * float((gy.abs() * (x.abs() + d.abs() + 2)).sum()) * 4


# ------------------------------------------------------------------------------------------------------ the cache
def _quant_ref(x, fmt):
    """Codes as values and scales, in numpy binary32 steps."""
    x = x.float().cpu().numpy()
    top = np.float32(127 if fmt == "int8" else 448)
    amax = np.abs(x).max(-1)
    bad = ~np.isfinite(amax)
    some = ~bad & (amax >= np.float32(2.0 ** -100))
    safe = np.where(some, amax, np.float32(1))
    y = x * (top / safe)[..., None].astype(np.float32)
    y = np.where(some[..., None], y, np.float32(0)).astype(np.float32)
    if fmt == "int8":
        codes = torch.from_numpy(np.rint(y).astype(np.int8))
    else:
        codes = torch.from_numpy(y).clamp(-448, 448).to(torch.float8_e4m3fn)
    scale = np.where(some, safe / top, np.float32(0)).astype(np.float32)
    return codes, torch.from_numpy(np.where(bad, np.float32(np.nan), scale))


def _rows_with_corners(T, H, D, dtype, g):
    x = (torch.randn(T, H, D, generator=g, device="cuda") * torch.exp(2 * torch.randn(T, H, 1, generator=g, device="cuda")))
    x = x.to(dtype)
    if T > 6:
        x[0] = 0
        x[1, :, 3] = float("inf")
        x[2, :, D - 1] = float("nan")
        x[3] = x[3].sign() * torch.finfo(dtype).tiny          # below 2^-100 for bf16 and fp32
        x[4] = 1.0                                            # every element is the largest
        x[5] = torch.finfo(dtype).max
    return x


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,D,ps", [(1, 1, 64, 16), (3, 2, 128, 16), (257, 8, 128, 64), (1000, 3, 64, 1024), (70, 5, 128, 32)])
def test_write_then_read(adt, fmt, dtype, T, H, D, ps):
    g = torch.Generator(device="cuda").manual_seed(T)
    pages = -(-T // ps) + 3
    cache = adt.KVCache(pages, ps, H, D, fmt)
    for t in cache.tensors:
        t.view(torch.uint8).fill_(0x33)
    old = [t.clone() for t in cache.tensors]
    kv = torch.empty(T, 2 * H * D + 16, dtype=dtype, device="cuda")
    k, v = kv[:, : H * D].view(T, H, D), kv[:, H * D: 2 * H * D].view(T, H, D)
    k.copy_(_rows_with_corners(T, H, D, dtype, g))
    v.copy_(_rows_with_corners(T, H, D, dtype, g).flip(-1))
    slots = torch.randperm(pages * ps, generator=g, device="cuda")[:T]
    if T > 9:
        slots[8] = -1
        slots[9] = -(1 << 40)
    cache.write(k, v, slots)
    adt.sage_check()
    keep = torch.ones(pages * ps, dtype=torch.bool)
    ok = (slots >= 0).cpu()
    keep[slots.cpu()[ok]] = False
    for x, codes, scale, oc, osc in ((k, cache.k_codes, cache.k_scale, old[0], old[1]),
                                     (v, cache.v_codes, cache.v_scale, old[2], old[3])):
        rc, rs = _quant_ref(x, fmt)
        flat = codes.view(torch.uint8).permute(0, 2, 1, 3).reshape(pages * ps, H, D).cpu()
        fsc = scale.permute(0, 2, 1).reshape(pages * ps, H).cpu()
        assert torch.equal(flat[slots.cpu()[ok]], rc.view(torch.uint8)[ok])
        got = fsc[slots.cpu()[ok]]
        assert torch.equal(got.isnan(), rs[ok].isnan()) and torch.equal(got.nan_to_num(), rs[ok].nan_to_num())
        # slots that were not named keep their bytes
        oflat = oc.view(torch.uint8).permute(0, 2, 1, 3).reshape(pages * ps, H, D).cpu()
        assert torch.equal(flat[keep], oflat[keep])
        assert torch.equal(fsc[keep], osc.permute(0, 2, 1).reshape(pages * ps, H).cpu()[keep])
    # read back, into a strided view, some slots twice, negative ones left alone
    rs = torch.cat([slots, slots.flip(0)])
    out = torch.full((2 * T, 2 * H * D + 8), 5.0, device="cuda").to(dtype)
    ko, vo = out[:, : H * D].view(2 * T, H, D), out[:, H * D: 2 * H * D].view(2 * T, H, D)
    cache.read(rs, ko, vo)
    adt.sage_check()
    for codes, scale, o in ((cache.k_codes, cache.k_scale, ko), (cache.v_codes, cache.v_scale, vo)):
        vals = codes.float().permute(0, 2, 1, 3).reshape(pages * ps, H, D)
        sc = scale.permute(0, 2, 1).reshape(pages * ps, H, 1)
        ref = (vals * sc)[rs.clamp(min=0)].to(dtype)
        ref[rs < 0] = 5.0
        assert torch.equal(o.isnan(), ref.isnan()) and torch.equal(o.nan_to_num(), ref.nan_to_num())
    assert bool((out[:, 2 * H * D:] == 5.0).all())


def test_slots_outside_the_cache_are_skipped_and_reported(adt):
    T, H, D, ps = 20, 2, 64, 16
    cache = adt.KVCache(2, ps, H, D)
    x = torch.randn(T, H, D, device="cuda").bfloat16()
    slots = torch.arange(T, device="cuda")
    slots[3], slots[4] = 2 * ps, 1 << 60
    cache.write(x, x, slots)
    assert adt.sage_check_status() == 1
    assert adt.sage_check_status() == 0                          # reported once
    flat = cache.k_scale.permute(0, 2, 1).reshape(-1, H)
    assert bool((flat[3:5] == 0).all()) and bool((flat[5:T] > 0).all())
    ko, vo = torch.full_like(x, 5.0), torch.full_like(x, 5.0)
    cache.read(slots, ko, vo)
    assert adt.sage_check_status() == 1
    assert bool((ko[3:5] == 5.0).all()) and not bool((ko[5] == 5.0).any())


def test_no_tokens(adt):
    cache = adt.KVCache(1, 16, 2, 64)
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    cache.write(e, e, none)
    cache.read(none, e, e)
    adt.sage_rope(e, e, none, adt.RopePlan(64))
    adt.sage_check()


def test_a_bad_slot_and_a_wait_that_ran_out_are_both_reported(adt):
    cache = adt.KVCache(2, 16, 2, 64)
    x = torch.ones(1, 2, 64, device="cuda", dtype=torch.bfloat16)
    cache.write(x, x, torch.tensor([32], device="cuda"))
    adt.selftest_wait_timeout(1_000_000)
    assert [adt.sage_check_status() for _ in range(3)] == [5, 1, 0]
