"""The 64-bit form of one query over rows of a paged cache, with the tolerance of each kernel's own rounding of P."""
import torch

from gqa_reference import attend

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def attend_paged(q, k, v, v_scales, scale, sinks, act, cache):
    """One query [1][H][d] over the rows k, v [n][HK][d] (float64; v_scales [n][HK][d/64] of FP8 rows): (out, tol).

    P is rounded to 16 bits before the product with v by the kernel for bf16 queries: to bf16 (half a step is 2^-8) over
    bf16 rows, to f16 (2^-11) over FP8 rows, whose codes are f16 exactly.  There p * scale is held in units of the largest
    one so far of its head and 64 channels, which lies above 2^12 of them: where f16 ends below 2^-14, a step is 2^-24
    units, and a key adds at most half of it, 2^-37 of the largest p * scale, times its code (448 at most).  The units
    end at 2^-100, so that half a step is never below 2^-125."""
    n, HK, d = k.shape
    half = 0.0 if act == "f32" or cache == "f32" else 2.0 ** -8 if cache == "bf16" else 2.0 ** -11
    out, tol = attend(q, k, v, scale, torch.ones(1, n, dtype=torch.bool), sinks, DT[act], half)
    if act == "bf16" and cache == "fp8":
        G = q.shape[1] // HK
        for h in range(q.shape[1]):
            lg = (k[:, h // G] @ q[0, h]) * scale
            top = max(float(lg.max()), float(sinks[h]) if sinks is not None else -float("inf"))
            w = torch.exp(lg - top)
            den = w.sum() + (torch.exp(sinks[h].double() - top) if sinks is not None else 0.0)
            most = (w[:, None] * v_scales[:, h // G]).amax(0)              # [d/64]
            unit = torch.clamp(2.0 ** -37 * most, min=2.0 ** -125) / den
            tol[0, h] += n * 448 * unit.repeat_interleave(64)
    return out, tol


def scale_rows(cache, table_row, n, page):
    """The scales of rows 0..n-1 of one sequence, [n][HK][d/64] float64."""
    ids = table_row[:-(-n // page)].long().clamp(min=0)
    s = cache.scales[ids.to(cache.scales.device)].cpu().double()
    return s.transpose(1, 2).reshape(-1, s.shape[1], s.shape[3])[:n]
