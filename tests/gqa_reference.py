"""Plain 64-bit forms of the grouped-head attention operators for the tests, and
the tolerances that follow from the kernels' arithmetic.

Attention (`tolerance`).  With p_i = e^(l_i - M) / den and u the half step of the
output type (bf16 2^-8, fp32 2^-24):
  * logits: a dot product of d fp32 products, summed in any order, is off by at
    most d 2^-23 sum|q_c k_c| (2^-24 for a rounded sum, 2^-23 for a truncating
    adder), and scaling it and taking the maximum off adds 4 2^-24 (|l_i| + |M|).
    A probability then is off by the factor e^(2 e_l), its own and the
    denominator's, where e_l is the largest such error of a visible logit;
  * 2^(x): 2^-20 on either side covers CUDA's ex2.approx and exp2f and a
    polynomial of that accuracy;
  * p is rounded once to 16 bits before the product with v (bf16 kernels): u_p =
    2^-8, 0 for fp32 kernels;
  * sums over n keys: n 2^-23 of sum p|v|;
  * the result is rounded once: u |out|.
  tol = sum p|v| (2 e_l (1 + small) + 2 2^-20 + u_p + (2 n + 8) 2^-23) + u |out| + 2^-126
"""
import math

import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def attend(q, k, v, scale, visible, sinks, out_dtype, p_half):
    """One sequence: q [n][H][d], k, v [m][HK][d] (float64), visible [n][m]; (out, tol),
    both [n][H][d] float64."""
    n, H, d = q.shape
    m, HK = k.shape[:2]
    out, tol = torch.zeros(n, H, d, dtype=torch.float64), torch.full((n, H, d), 2.0 ** -126, dtype=torch.float64)
    rows = visible.any(1)
    # what nobody sees takes no part
    seen = visible.any(0)
    kz, vz = (torch.where(seen[:, None, None], x, 0.0) for x in (k, v))
    for h in range(H):
        kh, vh = kz[:, h // (H // HK)], vz[:, h // (H // HK)]
        lg = (q[:, h] @ kh.T) * scale
        mag = (q[:, h].abs() @ kh.abs().T) * abs(scale)
        lg = torch.where(visible, lg, -math.inf)
        top = lg.amax(1) if m else torch.full((n,), -math.inf, dtype=torch.float64)
        if sinks is not None:
            top = torch.maximum(top, sinks[h].double())
        top = torch.where(top == -math.inf, 0.0, top)
        p = torch.exp(lg - top[:, None])
        den = p.sum(1) + (torch.exp(sinks[h].double() - top) if sinks is not None else 0.0)
        p = p / torch.where(den == 0, 1.0, den)[:, None]
        o = p @ vh
        e_l = torch.where(visible, mag * d * 2.0 ** -23 + 4 * 2.0 ** -24 * (lg.nan_to_num(neginf=0.0).abs() + top.abs()[:, None]),
                          0.0).amax(1) if m else torch.zeros(n, dtype=torch.float64)
        nk = visible.sum(1).double()
        rel = 2 * torch.expm1(e_l) + 2 * 2.0 ** -20 + p_half + (2 * nk + 8) * 2.0 ** -23
        out[:, h] = torch.where(rows[:, None], o, 0.0)
        tol[:, h] += (p @ vh.abs()) * rel[:, None] * 1.01 + HALF[out_dtype] * o.abs()
    return out, tol


def causal(n, m, window):
    t = torch.arange(n)[:, None] + m - n
    j = torch.arange(m)[None]
    see = j <= t
    if window:
        see &= j > t - window
    return see


def rotate(x, pos, inv_freq, rot, pairs):
    """x [n][heads][d] float64, pos [n]."""
    y = x.clone()
    if rot:
        ang = pos.double()[:, None] * inv_freq.double()[None]
        c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
        lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if pairs else (slice(0, rot // 2), slice(rot // 2, rot))
        a, b = x[..., lo], x[..., hi]
        y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
    return y


def partner(x, rot, pairs):
    """|a| + |b| of each element's pair: what a rotated value's fp32 error scales with."""
    y = x.abs().clone()
    if rot:
        lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if pairs else (slice(0, rot // 2), slice(rot // 2, rot))
        both = x[..., lo].abs() + x[..., hi].abs()
        y[..., lo], y[..., hi] = both, both
    return y


def assert_within(got, ref, tol, what=""):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (got.shape, ref.shape)
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = tuple(int(x) for x in torch.nonzero(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {i}: got {got[i]:.9g}, "
                             f"reference {ref[i]:.9g}, tolerance {tol[i]:.3g}")


def paged_rows(cache, table_row, n, page):
    """Rows 0..n-1 of one sequence as [n][HK][d] float64 (values of an FP8 cache: code * scale)."""
    ids = table_row[: -(-n // page)].long().clamp(min=0)
    x = cache.data[ids.to(cache.data.device)].cpu()
    if cache.scales is not None:
        s = cache.scales[ids.to(cache.data.device)].cpu().double()
        x = x.view(torch.float8_e4m3fn).double() * s.repeat_interleave(64, -1)
    return x.double().transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])[:n]
