"""Plain attention in 64 bits for the serving tests, with the error bound of a 16-bit kernel beside each value."""
import math

import torch


def attend(q, k, v, visible, scale, p_half):
    """One head.  q [Lq, D], k, v [Lk, D] in 64 bits; visible [Lq]: keys 0 .. visible - 1 are seen.
    Returns out, lse, tol_out (without the output's own rounding), tol_lse.

    The bound: a score is off by at most s = scale * |q| . |k| * D 2^-23 (32-bit sums, their order open) + 2^-22 of
    its size (the factor and the exponent's argument), a weight by (1 + 2 s + 2^-21) (exp2) and by its rounding to 16
    bits (p_half), the sum of the products by Lk 2^-23 of sum p |v|.  With A = sum p |v| / sum p that is
    A (p_half + 4 s + Lk 2^-23 + 2^-19) for the quotient."""
    Lk, D = k.shape
    out = torch.zeros(q.shape[0], D, dtype=torch.float64, device=q.device)
    lse = torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    tol_lse = torch.zeros_like(lse)
    some = visible > 0
    if Lk and bool(some.any()):
        seen = torch.arange(Lk, device=q.device) < visible[some][:, None]
        kk = torch.where(torch.isfinite(k), k, torch.zeros_like(k))
        x = (q[some] @ k.t()) * scale
        x = torch.where(seen, x, torch.full_like(x, -math.inf))
        size = torch.where(seen, (q[some].abs() @ kk.abs().t()) * scale, torch.zeros_like(x)).amax(-1, keepdim=True)
        s = size * (D * 2.0 ** -23 + 2.0 ** -22)
        p = torch.softmax(x, -1)
        # only visible rows of V take part, whatever the others hold
        vis_v = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
        out[some] = p @ vis_v
        A = p @ vis_v.abs()
        lse[some] = torch.logsumexp(x, -1)
        tol[some] = A * (p_half + 4 * s + Lk * 2.0 ** -23 + 2.0 ** -19)
        tol_lse[some] = (2 * s[:, 0] + Lk * 2.0 ** -23 + 2.0 ** -19) + lse[some].abs() * 2.0 ** -22
    return out, lse, tol, tol_lse


def check(got, lse, ref, ref_lse, tol, tol_lse, what=""):
    t = got.dtype
    half = torch.finfo(t).eps / 2
    floor = 2.0 ** -25 if t == torch.float16 else 0.0
    err = (got.double() - ref).abs()
    lim = half * (ref.abs() + tol) + tol + floor
    assert bool((err <= lim).all()), (what, float((err - lim).max()), float((err / lim.clamp(min=1e-30)).max()))
    if lse is not None:
        inf = torch.isinf(ref_lse)
        assert torch.equal(torch.isinf(lse), inf), what
        d = (lse.double() - ref_lse).abs()[~inf]
        assert bool((d <= tol_lse[~inf]).all()), (what, float((d - tol_lse[~inf]).max()))
