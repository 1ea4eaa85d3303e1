"""Plain 64-bit forms of the attention half (gemm_fp8, rope, kv_append,
attn_decode) and the bounds on what rounding may do to them.

Bounds count roundings: U = 2^-24 is half a step of fp32, 2^-8 of bf16, 2^-11
of fp16."""
import math

import torch

from block_refs import GROUP, U, activate, dequant

TURN = 2e-7  # what w4a8.h promises for sine and cosine


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounded(want, err, dtype):
    """The bound after one rounding to dtype (half the smallest subnormal below the normal range)."""
    tiny = {torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134}[dtype]
    return err + half_step(dtype) * (want.abs() + err) + tiny


def block_weights(w, scales):
    rows, K = w.shape
    s = scales.double().repeat_interleave(GROUP, 0)[:rows].repeat_interleave(GROUP, 1)
    return w.view(torch.float8_e4m3fn).double() * s


def gemm_fp8(a_q, a_scales, w, w_scales, bias=None, activation="none", residual=None):
    """(out in 64 bits, bound on the error before the last rounding).

    The fp8 matrix instruction cuts each product to 2^-13 of the largest of
    eight, the largest itself not: a group's sum is off by at most 7 * 2^-13
    of the sum of its products' magnitudes.  The promotion over G groups adds (2 G
    + 2) U of it.  The activations' slopes are below 1.2, and each is evaluated
    to 8 U."""
    a, b = dequant(a_q.view(torch.uint8), a_scales), block_weights(w.view(torch.uint8), w_scales)
    G = a_scales.shape[1]
    y = a @ b.t().contiguous()
    err = (a.abs() @ b.abs().t().contiguous()) * (7 * 2.0 ** -13 + (2 * G + 2) * U)
    if bias is not None:
        y = y + bias.double()
        err = err + U * y.abs()
    if activation == "swiglu":
        g, u = y.chunk(2, 1)
        eg, eu = err.chunk(2, 1)
        out = activate(g, "silu") * u
        err = 1.2 * eg * (u.abs() + eu) + activate(g, "silu").abs() * eu + 12 * U * out.abs()
    else:
        out = activate(y, activation)
        err = 1.2 * err + 8 * U * (out.abs() + (y.abs() if activation != "none" else 0))
    if residual is not None:
        out = out + residual.double()
        err = err + U * out.abs()
    return out, err


def frequencies(R, base=10000.0, scaling="none", factor=1.0, original_length=0.0, beta_fast=32.0, beta_slow=1.0):
    if scaling == "ntk":
        base = base * factor ** (R / (R - 2))
    f = [base ** (-2 * i / R) for i in range(R // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "yarn":
        def pair(beta):
            return R * math.log(original_length / (beta * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), R - 1)
        r = [min(max((i - lo) / max(hi - lo, 0.001), 0), 1) for i in range(R // 2)]
        f = [x / factor * k + x * (1 - k) for x, k in zip(f, r)]
    return torch.tensor(f, dtype=torch.float64)


def rope(x, positions, freq, interleaved=False, magnitude=1.0):
    """(rotated x in 64 bits, bound on the error before the last rounding): sine and cosine to TURN (and what
    64 bits lose of a far angle), two products and a sum."""
    R = 2 * freq.numel()
    angle = positions.double()[:, None] * freq
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    far = (angle.abs() * 2.0 ** -50)[:, None]
    y = x.double().clone()
    err = torch.zeros_like(y)
    if R == 0:
        return y, err
    first, second = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    a, b = y[..., first].clone(), y[..., second].clone()
    y[..., first], y[..., second] = magnitude * (a * cos - b * sin), magnitude * (a * sin + b * cos)
    e = abs(magnitude) * (a.abs() + b.abs()) * (TURN + far + 4 * U)
    err[..., first] = e
    err[..., second] = e
    return y, err


def gather(cache, scales, table, start, end, num_pages):
    """The rows of the positions [start, end) that hold something, [n, Hkv, D] in 64 bits."""
    page_size = cache.shape[1]
    at = torch.arange(start, end, device=cache.device)
    held = table[at // page_size].long()
    at, held = at[(held >= 0) & (held < num_pages)], held[(held >= 0) & (held < num_pages)]
    rows = cache[held, at % page_size]
    if scales is None:
        return rows.double()
    return rows.view(torch.float8_e4m3fn).double() * scales[held, :, at % page_size].double()[..., None]


def attn_decode(q, k_cache, v_cache, table, lens, k_scales=None, v_scales=None, scale=None, window=0):
    """(out, bound on it before the last rounding, lse, bound on it).

    A score is off by E = (D + 16) 2^-23 of the sum of its products' magnitudes
    (the matrix instruction may cut where it aligns) and 4 U of itself, the hardware's exp2 by 2^-22.  The weights are rounded to q's type (fp16: at least 2^-25
    of the reference, which the largest is not below), and a sum over n keys loses n U of its terms' magnitudes."""
    B, Hq, D = q.shape
    num_pages, page_size, Hkv, _ = k_cache.shape
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device=q.device)
    err = torch.zeros_like(out)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=q.device)
    lse_err = torch.zeros_like(lse)
    for b, n in enumerate(lens.tolist()):
        start, end = max(0, n - window) if window else 0, min(max(n, 0), table.shape[1] * page_size)
        k = gather(k_cache, k_scales, table[b], start, max(start, end), num_pages)
        if not k.shape[0]:
            continue
        v = gather(v_cache, v_scales, table[b], start, end, num_pages)
        qb = q[b].double().reshape(Hkv, Hq // Hkv, D)
        kt = k.permute(1, 2, 0).contiguous()
        s = qb @ kt * scale
        E = ((qb.abs() @ kt.abs()) * abs(scale) * (D + 16) * 2.0 ** -23 + 4 * U * s.abs()).amax(-1) + 2.0 ** -22
        vt = v.transpose(0, 1).contiguous()
        p = torch.softmax(s, -1)
        o, mag = p @ vt, p @ vt.abs()
        keys = k.shape[0]
        lse[b] = torch.logsumexp(s, -1).reshape(-1)
        lse_err[b] = (E + keys * U).reshape(-1) + 2.0 ** -21 * (lse[b].abs() + s.abs().amax(-1).reshape(-1) + 1)
        e = mag * (half_step(q.dtype) + 2 * E[..., None] + (2 * keys + 64) * U)
        if q.dtype == torch.float16:
            e = e + 2.0 ** -25 * vt.abs().sum(1)[:, None]
        out[b], err[b] = o.reshape(Hq, D), e.reshape(Hq, D)
    return out, err, lse, lse_err
