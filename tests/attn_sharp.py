"""What include/w4a8.h promises of decode attention's weights, as bounds that
see a lost second part of a weight, and a check that takes an output's rounding
for what it is instead of adding half a step of slack."""
import torch

from attn_refs import U, gather

# a weight, as its two parts: off by PART of it, or by LEAST of the row's largest weight
PART = {torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -22}
LEAST = {torch.bfloat16: 2.0 ** -88, torch.float16: 2.0 ** -38}


def attention(q, k_cache, v_cache, table, lens, k_scales=None, v_scales=None, scale=None, window=0):
    """(out in 64 bits, bound on its error before the last rounding).

    A score of n products that are not zero is off by (n + 16) 2^-23 of the sum
    of their magnitudes and 4 U of itself, the hardware's exp2 by 2^-22: E.  Weights
    and their sum carry it once each, the sums over the keys lose (2 keys + 64) U."""
    B, Hq, D = q.shape
    num_pages, page_size, Hkv, _ = k_cache.shape
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device=q.device)
    err = torch.zeros_like(out)
    for b, n in enumerate(lens.tolist()):
        start, end = max(0, n - window) if window else 0, min(max(n, 0), table.shape[1] * page_size)
        if start >= end:
            continue
        k = gather(k_cache, k_scales, table[b], start, end, num_pages)
        v = gather(v_cache, v_scales, table[b], start, end, num_pages)
        if not k.shape[0]:
            continue
        qb = q[b].double().reshape(Hkv, Hq // Hkv, D)
        kt = k.permute(1, 2, 0).contiguous()
        s = qb @ kt * scale
        products = int((q[b] != 0).sum(-1).max())
        E = ((qb.abs() @ kt.abs()) * abs(scale) * (products + 16) * 2.0 ** -23 + 4 * U * s.abs()).amax(-1) + 2.0 ** -22
        p = (s - s.amax(-1, keepdim=True)).exp()
        total = p.sum(-1, keepdim=True)
        vt = v.transpose(0, 1).contiguous()
        mag = p @ vt.abs() / total
        e = mag * (PART[q.dtype] + 2 * E[..., None] + (2 * k.shape[0] + 64) * U)
        e = e + LEAST[q.dtype] * vt.abs().sum(1)[:, None] / total
        out[b], err[b] = (p @ vt / total).reshape(Hq, D), e.reshape(Hq, D)
    return out, err


def outside(got, want, err):
    """How many elements are no rounding of a number within err of want.  Rounding
    keeps order, so they lie between the roundings of the two ends."""
    lo, hi = (want - err).to(got.dtype), (want + err).to(got.dtype)
    return int(((got < lo) | (got > hi) | torch.isnan(got)).sum())
