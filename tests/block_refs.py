"""Plain 64-bit forms of the operators around the expert forward, written from
their definitions in include/w4a8.h (torch float64, any device)."""
import math

import torch

GROUP = 128
U = 2.0 ** -24  # half a step of fp32, relative


def norm_residual(x, residual, post_weight=None, gate=None, residual_scale=1.0, pre_weight=None,
                  weight_offset=0.0, eps=1e-6):
    """(r', y or None, m): m bounds the terms that r' is the sum of."""
    def d(t):
        return None if t is None else t.double()

    def rms(v):
        return 1 / torch.sqrt(v.pow(2).mean(-1, keepdim=True) + eps)

    r, m = 0.0, 0.0
    if residual is not None:
        r = residual_scale * d(residual)
        m = r.abs()
    if x is not None:
        u = d(x)
        if post_weight is not None:
            u = u * rms(u) * (d(post_weight) + weight_offset)
        if gate is not None:
            u = d(gate) * u
        r, m = r + u, m + u.abs()
    y = None
    if pre_weight is not None:
        y = r * rms(r) * (d(pre_weight) + weight_offset)
    return r, y, m


def quant_values(y):
    """(y * 448/amax, amax/448) per 128, before the rounding to e4m3."""
    b = y.reshape(y.shape[0], -1, GROUP)
    amax = b.abs().amax(-1, keepdim=True).clamp_min(1e-10)
    return (b * (448 / amax)).reshape(y.shape), (amax / 448).squeeze(-1)


def route(logits, topk, score="sigmoid", bias=None, num_groups=1, topk_groups=1, group_top=2,
          renormalize=True, scale=1.0, num_tokens=None):
    """Row by row, expert by expert: (ids list of lists, weights list of lists)."""
    L = logits.double().tolist()
    B = [0.0] * logits.shape[1] if bias is None else bias.double().tolist()
    inf = math.inf
    all_ids, all_w = [], []
    for t, x in enumerate(L):
        E = len(x)
        if num_tokens is not None and t >= num_tokens:
            all_ids.append([-1] * topk)
            all_w.append([0.0] * topk)
            continue
        ok = [v > -inf for v in x]  # NaN: False
        s = [0.0] * E
        if score == "softmax":
            m = max([v for v, o in zip(x, ok) if o], default=0.0)
            s = [(1.0 if v == m else math.exp(v - m)) if o else 0.0 for v, o in zip(x, ok)]
            total = math.fsum(s)
            s = [v / total if total > 0 else 0.0 for v in s]
        else:
            s = [(1 / (1 + math.exp(-v)) if v > -700 else 0.0) if o else 0.0 for v, o in zip(x, ok)]
        c = [v + b if o and v + b > -inf else -inf for v, b, o in zip(s, B, ok)]
        if num_groups > 1:
            n = E // num_groups
            value = []
            for g in range(num_groups):
                best = sorted(((c[e], e) for e in range(g * n, (g + 1) * n) if c[e] > -inf), reverse=True)[:group_top]
                value.append((sum(v for v, _ in best) if best else -inf,
                              max((x[e] for e in range(g * n, (g + 1) * n) if c[e] > -inf), default=-inf)
                              if bias is None and group_top == 1 else 0.0))
            order = sorted(range(num_groups), key=lambda g: (-value[g][0], -value[g][1], g))
            kept = set(order[:topk_groups])
            c = [v if e // n in kept else -inf for e, v in enumerate(c)]
        # without a bias the logits order the scores, also where 64 bits round them alike
        key = [(c[e], x[e] if bias is None and ok[e] else 0.0) for e in range(E)]
        order = sorted((e for e in range(E) if c[e] > -inf), key=lambda e: (-key[e][0], -key[e][1], e))[:topk]
        w = [s[e] for e in order]
        total = math.fsum(w)
        if renormalize:
            w = [v / total if total > 0 else 0.0 for v in w]
        rest = topk - len(order)
        all_ids.append(order + [-1] * rest)
        all_w.append([scale * v for v in w] + [0.0] * rest)
    return all_ids, all_w


def dequant(codes, scales):
    return codes.view(torch.float8_e4m3fn).double() * scales.double().repeat_interleave(GROUP, 1)


def int4(w, scales):
    v = torch.stack((w & 15, w >> 4), -1).reshape(w.shape[0], -1).double()
    v = torch.where(v > 7, v - 16, v)
    return v * scales.double().repeat_interleave(GROUP, 1)


def activate(y, act):
    if act == "relu":
        return y.clamp_min(0)
    if act == "silu":
        return y * torch.sigmoid(y)
    if act == "gelu":
        return 0.5 * y * torch.special.erfc(-y / math.sqrt(2))
    if act == "gelu_tanh":
        return y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
    return y


def gemm_epilogue(a_q, a_scales, w, w_scales, bias=None, activation="none", residual=None):
    """(out in 64 bits, bound on the error before the last rounding).

    The fp8 matrix instruction keeps 13 bits below the largest product of a
    group, so a group's sum is off by at most 2^-13 of the sum of its
    products' magnitudes; the fp32 promotion adds (2 G + 2) U of it.  The
    activations' slopes are below 1.2, and each is evaluated to 8 U."""
    a, b = dequant(a_q, a_scales), int4(w, w_scales)
    G = a_scales.shape[1]
    y = a @ b.t().contiguous()
    err = (a.abs() @ b.abs().t().contiguous()) * (2.0 ** -13 + (2 * G + 2) * U)
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
