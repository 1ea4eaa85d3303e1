"""The operators of the attention half of a served MoE block, and the cases they are timed on.

  gemm    gemm_fp8     the dense fp8 product: scales per token and 128 K, and per 128 x 128 weights
  rope    rope         rotary positions of heads
  append  kv_append    rotates queries and keys and writes keys and values into a paged cache
  attn    attn_decode  attention of one new token of each sequence over that cache

With `own` false, run() computes them from elementary torch operations; with `own` true it calls
w4a8_moe_grouped_amd.lib.
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 128
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2, "fp8": 1, "none": 0}


# ---- cases ---------------------------------------------------------------------------

def _gemm(M, K, N, act="none", bias="none", residual=False):
    return dict(op="gemm", M=M, K=K, N=N, act=act, bias=bias, residual=residual)


def _rope(T, heads, D, R, type, interleaved=False, far=8192, scaled="none"):
    return dict(op="rope", T=T, heads=heads, D=D, R=R, type=type, interleaved=interleaved, far=far, scaled=scaled)


def _append(T, Hq, Hkv, D, R, type, cache, page, interleaved=False, far=8192, pad=0):
    return dict(op="append", T=T, Hq=Hq, Hkv=Hkv, D=D, R=R, type=type, cache=cache, page=page,
                interleaved=interleaved, far=far, pad=pad)


def _attn(B, Hq, Hkv, D, L, type, cache, page, ragged=False, window=0, empty=0):
    return dict(op="attn", B=B, Hq=Hq, Hkv=Hkv, D=D, L=L, type=type, cache=cache, page=page, ragged=ragged,
                window=window, empty=empty)


def listed():
    return [
        # one token of a single stream: the projection to 64 query and 2 x 8 key and value heads
        dict(_gemm(1, 7168, 10240), name="fp8_one_token"),
        # a decode batch: the projection back from the heads, added to the residual stream
        dict(_gemm(64, 8192, 7168, residual=True), name="fp8_decode"),
        # a prefill chunk: the projection to the heads
        dict(_gemm(4096, 7168, 10240), name="fp8_prefill"),
        # odd sizes: a short prompt through a biased projection with an activation
        dict(_gemm(333, 1664, 2050, act="gelu", bias="bf16", residual=True), name="fp8_ragged"),
        # the queries and keys of a decode batch
        dict(_rope(64, 72, 128, 128, "bf16"), name="rope_decode"),
        # a long prefill in 32 bits: pairs side by side, half of the head, positions of a scaled context
        dict(_rope(16384, 40, 128, 64, "fp32", interleaved=True, far=1 << 20, scaled="yarn"), name="rope_long"),
        # a decode batch's keys and values into the cache, its queries rotated on the way
        dict(_append(64, 64, 8, 128, 128, "bf16", "bf16", 16), name="append_decode"),
        # a prefill into an fp8 cache, with a padded tail
        dict(_append(16384, 64, 8, 128, 128, "bf16", "fp8", 64, far=131072, pad=100), name="append_prefill_fp8"),
        # one stream with a short history
        dict(_attn(1, 64, 8, 128, 1000, "bf16", "bf16", 16), name="attn_one_stream"),
        # a decode batch of equal histories
        dict(_attn(64, 64, 8, 128, 4096, "bf16", "bf16", 16), name="attn_decode"),
        # few long histories of very different lengths in an fp8 cache
        dict(_attn(16, 64, 8, 128, 65536, "bf16", "fp8", 64, ragged=True), name="attn_long_fp8"),
        # odd sizes: heads of 80, pages of 24 tokens, a window, new sequences without a history
        dict(_attn(37, 20, 5, 80, 3001, "fp16", "fp16", 24, ragged=True, window=1000, empty=3), name="attn_ragged"),
    ]


def _log(rng, lo, hi):
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def draw(rng):
    op = rng.choice(["gemm", "rope", "append", "attn", "attn"])
    if op == "gemm":
        while True:
            M, K, N = _log(rng, 1, 4096), GROUP * rng.randint(1, 64), _log(rng, 16, 10240)
            act = rng.choice(["none", "none", "relu", "silu", "gelu", "gelu_tanh", "swiglu"])
            if act == "swiglu":  # gate and up are each cut into blocks
                N = max(GROUP, N // GROUP * GROUP)
            if M * K * N * (2 if act == "swiglu" else 1) <= 4096 * 7168 * 10240:
                return _gemm(M, K, N, act, rng.choice(["none", "bf16", "fp32"]), rng.random() < 0.5)
    D = rng.choice([64, 128, 128, 128, 256, 8 * rng.randint(2, 32)])
    R = rng.choice([D, D, D // 2, 2 * rng.randint(1, D // 2)])
    far, page = rng.choice([2048, 32768, 1 << 20]), rng.choice([16, 32, 64, 8 * rng.randint(1, 32), rng.randint(1, 100)])
    while op == "rope":
        T, heads = _log(rng, 1, 16384), _log(rng, 1, 128)
        if T * heads * D <= 16384 * 40 * 128:
            return _rope(T, heads, D, R, rng.choice(["bf16", "fp16", "fp32"]), rng.random() < 0.5, far,
                         rng.choice(["none", "linear", "yarn"]))
    Hkv, group = rng.choice([1, 2, 4, 5, 8, 8, 16]), rng.choice([1, 4, 7, 8, 8, 16])
    type = rng.choice(["bf16", "bf16", "fp16"])
    cache = rng.choice(["fp8", type]) if type == "bf16" else type
    while op == "append":
        T = _log(rng, 1, 16384)
        if T * (group + 2) * Hkv * D <= 16384 * 80 * 128:
            return _append(T, group * Hkv, Hkv, D, R, type, cache, page, rng.random() < 0.5, far, rng.choice([0, T // 5]))
    while True:
        B, L = _log(rng, 1, 256), _log(rng, 1, 65536)
        if B * L * Hkv * D * SIZE[cache] <= 64 * 4096 * 8 * 128 * 2 and B * (group * Hkv) * L * D <= 64 * 64 * 4096 * 128:
            return _attn(B, group * Hkv, Hkv, D, L, type, cache, page, rng.random() < 0.6,
                         rng.choice([0, 0, max(1, L // 3)]), rng.choice([0, 0, B // 8]))


# ---- inputs --------------------------------------------------------------------------

def _lengths(case):
    """The lengths of a batch, known from the case; a seed only shuffles them."""
    B, L = case["B"], case["L"]
    n = torch.full((B,), L, dtype=torch.int32)
    if case["ragged"]:  # from a 32nd of the longest up, evenly over the logarithm
        n = (L * 32.0 ** -torch.linspace(0, 1, B, dtype=torch.float64)).ceil().int()
    n[B - case["empty"]:] = 0
    return n


def _quantised(x, dims=1):
    """e4m3 codes (uint8) and the scales of the rows along the last axis."""
    amax = x.abs().amax(-1, keepdim=True).clamp_min(1e-10)
    codes = (x * (448 / amax)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, (amax / 448).squeeze(-1)


def _frequencies(R, scaled, far):
    i = torch.arange(R // 2, dtype=torch.float64, device=DEV)
    f = 10000.0 ** (-2 * i / R)
    if scaled == "linear":
        return f / 8
    if scaled == "yarn":  # turns over the first context decide how much of a frequency is kept
        turns = far / 32 * f / (2 * math.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        return f * keep + f / 32 * (1 - keep)
    return f


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=DEV)

    def shuffled(n):
        return torch.randperm(n, generator=g, device=DEV)

    s = dict(case=case)
    if case["op"] == "gemm":
        M, K, N = case["M"], case["K"], case["N"]
        rows = 2 * N if case["act"] == "swiglu" else N
        codes, s["a_scales"] = _quantised(normal(M, K // GROUP, GROUP).bfloat16().float())
        s["a_q"] = codes.reshape(M, K)
        s["w"] = (100 * normal(rows, K)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s["w_scales"] = (0.5 + uniform(-(-rows // GROUP), K // GROUP)) * 2e-4
        s["bias"] = normal(rows).to(TYPES[case["bias"]]) if case["bias"] != "none" else None
        s["residual"] = normal(M, N).bfloat16() if case["residual"] else None
        return s
    D, type = case["D"], TYPES[case["type"]]
    if case["op"] == "attn":
        B, Hkv, page, fp8 = case["B"], case["Hkv"], case["page"], case["cache"] == "fp8"
        lens = _lengths(case)
        used = (lens + page - 1) // page
        most = max(1, -(-case["L"] // page))
        pages = int(used.sum()) + 1
        place = torch.arange(most, device=DEV) + (used.cumsum(0) - used).to(DEV)[:, None]
        order = shuffled(pages)
        table = torch.where(torch.arange(most, device=DEV) < used.to(DEV)[:, None],
                            order[place.clamp_max(pages - 1)], -1).int()
        mixed = shuffled(B)
        s["seq_lens"], s["page_table"] = lens.to(DEV)[mixed], table[mixed].contiguous()
        s["q"] = normal(B, case["Hq"], D).to(type)
        for name in ("k", "v"):
            rows = torch.empty(pages, page, Hkv, D, dtype=torch.uint8 if fp8 else type, device=DEV)
            scales = torch.empty(pages, Hkv, page, device=DEV) if fp8 else None
            step = max(1, (1 << 26) // (page * Hkv * D))
            for at in range(0, pages, step):
                x = normal(min(step, pages - at), page, Hkv, D)
                if fp8:
                    rows[at:at + step], r = _quantised(x)
                    scales[at:at + step] = r.transpose(1, 2)
                else:
                    rows[at:at + step] = x
            s[name + "_cache"], s[name + "_scales"] = rows, scales
        return s
    T, R = case["T"], case["R"]
    s["positions"] = torch.randint(0, case["far"], (T,), generator=g, device=DEV, dtype=torch.int32)
    s["frequencies"] = _frequencies(R, case.get("scaled", "none"), case["far"])
    if case["op"] == "rope":
        s["x"] = normal(T, case["heads"], D).to(type)
        return s
    Hq, Hkv, page, fp8 = case["Hq"], case["Hkv"], case["page"], case["cache"] == "fp8"
    qkv = normal(T, Hq + 2 * Hkv, D).to(type)  # one product's output, read in place
    s["q"], s["k"], s["v"] = qkv.split((Hq, Hkv, Hkv), 1)
    pages = -(-(T + T // 4 + 1) // page)
    s["slots"] = shuffled(pages * page)[:T].long()
    s["slots"][T - case["pad"]:] = -1
    for name in ("k", "v"):
        old = normal(pages, page, Hkv, D)
        s[name + "_cache"], r = _quantised(old) if fp8 else (old.to(type), None)
        s[name + "_scales"] = r.transpose(1, 2).contiguous() if fp8 else None
    return s


# ---- the plain forms -------------------------------------------------------------------

def _plain_act(y, act):
    if act == "relu":
        return torch.where(y < 0, 0.0, y)
    if act == "silu":
        return y / (1 + torch.exp(-y))
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    if act == "swiglu":
        gate, up = y.chunk(2, -1)
        return gate / (1 + torch.exp(-gate)) * up
    return y


def _plain_gemm(s):
    rows, K = s["w"].shape
    w = s["w"].view(torch.float8_e4m3fn).float().reshape(rows, K // GROUP, GROUP)
    w = w * s["w_scales"].repeat_interleave(GROUP, 0)[:rows, :, None]
    a = s["a_q"].view(torch.float8_e4m3fn).float().reshape(-1, K // GROUP, GROUP) * s["a_scales"][..., None]
    y = a.reshape(-1, K) @ w.reshape(rows, K).t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = _plain_act(y, s["case"]["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return [y.bfloat16()]


def _rotated(x, s):
    """x [T, heads, D] rotated, in 32 bits."""
    R = s["case"]["R"]
    angle = s["positions"].double()[:, None] * s["frequencies"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x = x.float()
    turned, rest = x[..., :R], x[..., R:]
    if s["case"]["interleaved"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = turned[..., :R // 2], turned[..., R // 2:]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, rest), -1)


def _values(s):
    """What an append changes and returns; codes as the values they stand for."""
    if s["k_scales"] is None:
        return [s["k_cache"], s["v_cache"]]
    return [s["k_cache"].view(torch.float8_e4m3fn), s["v_cache"].view(torch.float8_e4m3fn), s["k_scales"], s["v_scales"]]


def _plain_append(s):
    case = s["case"]
    n, Hkv, D = case["T"] - case["pad"], case["Hkv"], case["D"]
    slots = s["slots"][:n]
    k, v = _rotated(s["k"], s)[:n], s["v"][:n].float()
    if s["k_scales"] is not None:
        page, place = slots // case["page"], slots % case["page"]
        k, r = _quantised(k)
        s["k_scales"][page, :, place] = r
        v, r = _quantised(v)
        s["v_scales"][page, :, place] = r
    s["k_cache"].view(-1, Hkv, D)[slots] = k.to(s["k_cache"].dtype)
    s["v_cache"].view(-1, Hkv, D)[slots] = v.to(s["v_cache"].dtype)
    return [_rotated(s["q"], s).to(s["q"].dtype)] + _values(s)


def _history(cache, scales, table):
    """The cached rows of each sequence, [B, Hkv, positions, D] in 32 bits."""
    rows = cache[table]
    if scales is None:
        rows = rows.float()
    else:
        rows = rows.view(torch.float8_e4m3fn).float() * scales[table].transpose(2, 3)[..., None]
    return rows.flatten(1, 2).transpose(1, 2)


def _plain_attn(s):
    case = s["case"]
    B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]
    table = s["page_table"].clamp_min(0).long()
    k = _history(s["k_cache"], s["k_scales"], table)
    q = s["q"].float().reshape(B * Hkv, Hq // Hkv, D)
    n = k.shape[2]
    scores = torch.bmm(q, k.transpose(2, 3).reshape(B * Hkv, D, n)).reshape(B, Hq, n) * D ** -0.5
    del k
    at, length = torch.arange(n, device=DEV), s["seq_lens"][:, None]
    seen = at < length
    if case["window"]:
        seen = seen & (at >= length - case["window"])
    scores = torch.where(seen[:, None], scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top > -math.inf, top, 0.0)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    v = _history(s["v_cache"], s["v_scales"], table).reshape(B * Hkv, n, D)
    out = torch.bmm(p.reshape(B * Hkv, Hq // Hkv, n), v).reshape(B, Hq, D)
    out = torch.where(total > 0, out / total, 0.0)
    return [out.to(s["q"].dtype), (top + torch.log(total)).squeeze(-1)]


def run(state):
    case = state["case"]
    s = state
    if own:
        from w4a8_moe_grouped_amd import lib
        if case["op"] == "gemm":
            return [lib.gemm_fp8(s["a_q"], s["a_scales"], s["w"], s["w_scales"], bias=s["bias"], activation=case["act"],
                                 residual=s["residual"])]
        if case["op"] == "rope":
            return [lib.rope(s["x"], s["positions"], s["frequencies"], interleaved=case["interleaved"])]
        if case["op"] == "append":
            q = lib.kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], k_scales=s["k_scales"],
                              v_scales=s["v_scales"], positions=s["positions"], frequencies=s["frequencies"],
                              interleaved=case["interleaved"], q=s["q"])
            return [q] + _values(s)
        return list(lib.attn_decode(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["seq_lens"],
                                    k_scales=s["k_scales"], v_scales=s["v_scales"], window=case["window"],
                                    return_lse=True))
    if case["op"] == "rope":
        return [_rotated(s["x"], s).to(s["x"].dtype)]
    return {"gemm": _plain_gemm, "append": _plain_append, "attn": _plain_attn}[case["op"]](s)


# ---- the definitions in 64 bits --------------------------------------------------------

def _exact_gemm(case, s):
    w = s["w"].view(torch.float8_e4m3fn).double()
    w *= s["w_scales"].double().repeat_interleave(GROUP, 1).repeat_interleave(GROUP, 0)[:w.shape[0]]
    a = s["a_q"].view(torch.float8_e4m3fn).double() * s["a_scales"].double().repeat_interleave(GROUP, 1)
    y = torch.mm(a, w.T.contiguous())
    if s["bias"] is not None:
        y += s["bias"].double()
    act = case["act"]
    if act == "swiglu":
        y = y[:, :case["N"]] * torch.sigmoid(y[:, :case["N"]]) * y[:, case["N"]:]
    elif act == "silu":
        y = y * torch.sigmoid(y)
    elif act == "relu":
        y = y.clamp(min=0)
    elif act == "gelu":
        y = y * 0.5 * torch.special.erfc(-y / math.sqrt(2.0))
    elif act == "gelu_tanh":
        y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
    return [y if s["residual"] is None else y + s["residual"].double()]


def _exact_turned(case, s, x):
    """The pairs as complex numbers, times e^(i angle)."""
    R, y = case["R"], x.double().clone()
    turn = torch.exp(1j * (s["positions"].double()[:, None] * s["frequencies"][None]))[:, None, :]
    if case["interleaved"]:
        first, second = slice(0, R, 2), slice(1, R, 2)
    else:
        first, second = slice(0, R // 2), slice(R // 2, R)
    z = torch.complex(y[:, :, first], y[:, :, second]) * turn
    y[:, :, first], y[:, :, second] = z.real, z.imag
    return y


def _exact_append(case, s):
    n, Hkv, D, page = case["T"] - case["pad"], case["Hkv"], case["D"], case["page"]
    fp8 = s["k_scales"] is not None

    def filled(cache, scales, rows):
        cache = cache.view(torch.float8_e4m3fn).double() if fp8 else cache.double()
        if not fp8:
            cache.reshape(-1, Hkv, D)[s["slots"][:n]] = rows[:n]
            return cache, None
        r = rows.abs().max(2)[0].clamp(min=1e-10) / 448
        cache.reshape(-1, Hkv, D)[s["slots"][:n]] = (rows / r[:, :, None])[:n]
        r_all = scales.double().transpose(1, 2).reshape(-1, Hkv)
        r_all[s["slots"][:n]] = r[:n]
        return cache, r_all.reshape(-1, page, Hkv).transpose(1, 2).contiguous()

    k, kr = filled(s["k_cache"], s["k_scales"], _exact_turned(case, s, s["k"]))
    v, vr = filled(s["v_cache"], s["v_scales"], s["v"].double())
    return [_exact_turned(case, s, s["q"]), k, v] + ([kr, vr] if fp8 else [])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "gemm":
        return _exact_gemm(case, s)
    if case["op"] == "rope":
        return [_exact_turned(case, s, s["x"])]
    if case["op"] == "append":
        return _exact_append(case, s)
    B, Hq, Hkv, D, page = (case[x] for x in ("B", "Hq", "Hkv", "D", "page"))
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=DEV)
    for b, length in enumerate(s["seq_lens"].tolist()):
        at = torch.arange(max(0, length - case["window"]) if case["window"] else 0, length, device=DEV)
        if not at.numel():
            continue
        held, place = s["page_table"][b].long()[at // page], at % page
        k, v = s["k_cache"][held, place], s["v_cache"][held, place]  # [n, Hkv, D]
        if case["cache"] == "fp8":
            k = k.view(torch.float8_e4m3fn).double() * s["k_scales"][held, :, place].double()[..., None]
            v = v.view(torch.float8_e4m3fn).double() * s["v_scales"][held, :, place].double()[..., None]
        q = s["q"][b].double().reshape(Hkv, Hq // Hkv, D)
        scores = torch.matmul(q, k.double().permute(1, 2, 0).contiguous()) / math.sqrt(D)
        lse[b] = torch.logsumexp(scores, -1).reshape(-1)
        out[b] = torch.matmul(torch.softmax(scores, -1), v.double().transpose(0, 1).contiguous()).reshape(Hq, D)
    return [out, lse]


# ---- what a pass cannot do without -------------------------------------------------------

def work(case):
    if case["op"] == "gemm":
        M, K, N = case["M"], case["K"], case["N"]
        rows = 2 * N if case["act"] == "swiglu" else N
        return {"bytes": rows * K + 4 * -(-rows // GROUP) * (K // GROUP) + M * (K + 4 * (K // GROUP))
                + M * N * (4 if case["residual"] else 2) + rows * SIZE[case["bias"]], "flops": 2 * M * K * rows}
    D = case["D"]
    if case["op"] == "attn":
        lens = _lengths(case).long()
        keys = int((lens.clamp_max(case["window"]) if case["window"] else lens).sum())
        row = D * SIZE[case["cache"]] + (4 if case["cache"] == "fp8" else 0)
        pages = int(((lens + case["page"] - 1) // case["page"]).sum())
        return {"bytes": 2 * keys * case["Hkv"] * row + case["B"] * case["Hq"] * (2 * D * SIZE[case["type"]] + 4) + 4 * pages,
                "flops": 4 * case["Hq"] * D * keys}
    T, size = case["T"], SIZE[case["type"]]
    if case["op"] == "rope":
        return {"bytes": 2 * T * case["heads"] * D * size + 4 * T, "flops": 3 * T * case["heads"] * case["R"]}
    n = T - case["pad"]
    row = D * SIZE[case["cache"]] + (4 if case["cache"] == "fp8" else 0)
    return {"bytes": 2 * T * case["Hq"] * D * size + 2 * n * case["Hkv"] * (D * size + row) + 12 * T,
            "flops": 3 * (T * case["Hq"] + n * case["Hkv"]) * case["R"]}
