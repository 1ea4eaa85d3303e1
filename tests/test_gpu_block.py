"""The operators around the expert forward (moe_route, norm_residual,
gemm_epilogue) on the GPU against their plain 64-bit forms (block_refs.py).

Bounds count roundings: U = 2^-24 is half a step of fp32, 2^-8 of bf16; e4m3
codes are off by half a step, 2^-4 of the value or 2^-10 below 2^-6."""
import math

import numpy as np
import pytest
import torch

import block_refs as ref
from block_refs import U
from w4a8_moe_grouped_amd import lib as w4
from w4a8_moe_grouped_amd import synth

pytestmark = pytest.mark.gpu

BF16, FP32, FP16 = torch.bfloat16, torch.float32, torch.float16
INF = math.inf


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "the gpu tests need an MI355X"
    w4.load()
    return torch.device("cuda:0")


def gen(dev, seed):
    return torch.Generator(device=dev).manual_seed(seed)


def padded(t, extra):
    """The same rows with a larger row stride."""
    big = torch.full((t.shape[0], t.shape[1] + extra), 7, dtype=t.dtype, device=t.device)
    big[:, :t.shape[1]] = t
    return big[:, :t.shape[1]]


# ---- moe_route -----------------------------------------------------------------------

def check_route(logits, topk, got=None, **kw):
    want_ids, want_w = ref.route(logits, topk, **{k: (int(v) if k == "num_tokens" and v is not None else v)
                                                  for k, v in kw.items()})
    ids, w = got if got is not None else w4.moe_route(logits, topk, **kw)
    torch.cuda.synchronize()
    assert ids.dtype == torch.int32 and w.dtype == FP32 and ids.shape == w.shape == (logits.shape[0], topk)
    if logits.shape[0] == 0:
        return
    assert ids.tolist() == want_ids
    want = torch.tensor(want_w, dtype=torch.float64)
    # one rounding to fp32 (2^-150: half a step of the subnormals), the rest in 64 bits
    torch.testing.assert_close(w.double().cpu(), want, rtol=U * (1 + 1e-6), atol=2.0 ** -150)


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T, E, k, groups, kept", [
    (1, 8, 2, 1, 1), (64, 256, 8, 8, 4), (5, 256, 8, 1, 1), (33, 90, 6, 6, 3), (7, 1, 1, 1, 1), (9, 64, 32, 2, 2),
    (3, 1000, 10, 8, 2), (2, 1024, 32, 64, 64), (17, 384, 8, 1, 1), (6, 130, 5, 13, 4), (130, 60, 4, 1, 1),
    (4, 64, 3, 64, 5), (11, 160, 6, 8, 3), (3, 512, 7, 4, 1), (9, 256, 16, 8, 4), (10, 100, 13, 1, 1), (6, 48, 16, 16, 9),
    (7, 234, 9, 13, 5), (5, 256, 15, 16, 16), (8, 75, 10, 5, 2), (6, 128, 16, 2, 1), (5, 33, 12, 3, 3)])
def test_route(dev, dtype, score, T, E, k, groups, kept):
    g = gen(dev, T * E + k)
    x = torch.randn(T, E, generator=g, device=dev).to(dtype)
    bias = 0.2 * torch.randn(E, generator=g, device=dev)
    for b in (None, bias):
        for renorm, scale, top in ((True, 2.5, 2), (False, 1.0, 1)):
            print("route", dtype, score, T, E, k, groups, kept, b is not None, renorm, top, flush=True)
            check_route(x, k, score=score, bias=b, num_groups=groups, topk_groups=kept, group_top=top,
                        renormalize=renorm, scale=scale)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups, kept", [(1, 1), (8, 3)])
def test_route_masked_and_special_values(dev, score, groups, kept):
    E, k = 64, 6
    g = gen(dev, 5)
    x = torch.randn(14, E, generator=g, device=dev)
    x[0] = -INF                       # nothing can be chosen
    x[1, 3:] = -INF                   # fewer than k
    x[2] = torch.finfo(FP32).min      # the type's lowest value is a value
    x[3, 10:] = torch.finfo(FP32).min
    x[4, 5] = math.nan
    x[5] = math.nan
    x[6, [7, 9]] = INF
    x[7] = INF
    x[8] = 1.25                       # all tie: the lowest indexes
    x[9, ::2] = x[9, 1::2]            # pairs tie
    x[10] = 0.0
    x[10, 1::2] = -0.0
    x[11, :32] = -INF                 # whole groups are masked
    x[12] = -1e4                      # scores that underflow
    x[13] = x[13].round()             # many ties
    bias = torch.zeros(E, device=dev)
    bias[::3] = 0.5
    special = bias.clone()
    special[[1, 20]] = -INF
    special[[2, 40]] = math.nan
    special[33] = INF
    for b in (None, bias, special):
        for top in (1, 2):
            check_route(x, k, score=score, bias=b, num_groups=groups, topk_groups=kept, group_top=top)
            check_route(x, k, score=score, bias=b, num_groups=groups, topk_groups=kept, group_top=top,
                        renormalize=False)
            check_route(x.to(FP16), 12, score=score, bias=b, num_groups=groups, topk_groups=kept, group_top=top)


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("E, groups, kept", [(256, 8, 4), (256, 16, 5), (256, 2, 1), (192, 6, 2), (64, 8, 3), (128, 4, 2),
                                             (100, 1, 1), (250, 1, 1), (90, 6, 3), (77, 7, 3), (165, 11, 4)])
def test_route_near_ties(dev, dtype, E, groups, kept):
    """Logits a few steps of their type apart, and sums of choices whose parts
    cancel: the order is that of 64 bits."""
    g = gen(dev, E + groups)
    step = torch.finfo(dtype).eps
    x = (1 + step * torch.randint(0, 9, (60, E), generator=g, device=dev)).to(dtype)
    x[30:] *= -1
    wide = 1000 * torch.randint(-1, 2, (E,), generator=g, device=dev).float()
    for score in ("sigmoid", "softmax"):
        for bias in (None, torch.zeros(E, device=dev), wide, 1e-7 * torch.randn(E, generator=g, device=dev)):
            for top in (1, 2):
                check_route(x[::3], 14, score=score, bias=bias, num_groups=groups, topk_groups=kept, group_top=top)
                check_route(x, 8, score=score, bias=bias, num_groups=groups, topk_groups=kept, group_top=top)


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("T, E, k, groups, kept", [
    (37, 512, 8, 1, 1), (37, 257, 16, 1, 1), (5, 440, 8, 8, 4), (70, 512, 8, 16, 3), (9, 444, 7, 2, 2), (3, 384, 12, 6, 2)])
def test_route_with_32_experts_a_lane(dev, dtype, T, E, k, groups, kept):
    """Random logits, logits a few steps apart, strides, specials."""
    g = gen(dev, T + E)
    x = padded(torch.randn(T, E, generator=g, device=dev).to(dtype), 3)
    x[0] = -INF
    x[1, ::2] = math.nan
    x[2, 5:] = -INF
    near = (1 + torch.finfo(dtype).eps * torch.randint(0, 9, (30, E), generator=g, device=dev)).to(dtype)
    bias = 0.2 * torch.randn(E, generator=g, device=dev)
    for score in ("sigmoid", "softmax"):
        for b in (None, bias, torch.zeros(E, device=dev)):
            for renorm, top in ((True, 2), (False, 1)):
                for rows in (x, near):
                    check_route(rows, k, score=score, bias=b, num_groups=groups, topk_groups=kept, group_top=top,
                                renormalize=renorm)


def test_route_orders_scores_that_32_bits_round_alike(dev):
    """sigmoid(x) + b around 1e-4 with a bias of 1000: 32 bits see ties."""
    E = 128
    g = gen(dev, 8)
    x = -9 + 0.01 * torch.randn(40, E, generator=g, device=dev)
    for bias in (torch.full((E,), 1000.0, device=dev), torch.full((E,), -1000.0, device=dev), None):
        for groups, kept in ((1, 1), (8, 3)):
            check_route(x, 8, bias=bias, num_groups=groups, topk_groups=kept)
            check_route(x, 8, score="softmax", bias=bias, num_groups=groups, topk_groups=kept)


def test_route_without_a_bias_orders_by_the_logits(dev):
    """Scores that round to 1 in 64 bits still differ by their logits."""
    x = torch.linspace(30, 60, 96, device=dev)[torch.randperm(96, generator=gen(dev, 1), device=dev)].repeat(3, 1)
    check_route(x, 8)


@pytest.mark.parametrize("num", [0, 1, 5, 6, 7, -3])
def test_route_padded_batch(dev, num):
    x = torch.randn(6, 64, device=dev, generator=gen(dev, 2))
    x[max(num, 0):] = math.nan  # the padding is not read
    n = torch.tensor([num], dtype=torch.int32, device=dev)
    check_route(x, 4, num_tokens=n)


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("E, extra", [(64, 8), (90, 1), (256, 3), (256, 4), (33, 0)])
def test_route_strides(dev, dtype, E, extra):
    x = padded(torch.randn(9, E, device=dev, generator=gen(dev, 3)).to(dtype), extra)
    check_route(x, 5, score="softmax")


def test_route_empty_and_many_tokens(dev):
    ids, w = w4.moe_route(torch.empty(0, 64, device=dev), 4)
    assert ids.shape == w.shape == (0, 4)
    # more rows than one chunk of any grid: equal rows give equal answers
    row = torch.randn(1, 16, device=dev, generator=gen(dev, 4)).to(BF16)
    x = row.repeat(300_001, 1)
    x[-1, 3] = 50.0
    ids, w = w4.moe_route(x, 2)
    one = w4.moe_route(row, 2)
    assert torch.equal(ids[:-1], one[0].expand(300_000, 2)) and torch.equal(w[:-1], one[1].expand(300_000, 2))
    assert ids[-1, 0] == 3


# ---- norm_residual -------------------------------------------------------------------

def check_norm(x, residual, quantize=False, got=None, **kw):
    args = {k: v for k, v in kw.items() if k not in ("residual_out", "out", "out_scales", "keep_residual")}
    r, y, m = ref.norm_residual(x, residual, **args)
    out, yo, scales = got if got is not None else w4.norm_residual(x, residual, quantize=quantize, **kw)
    torch.cuda.synchronize()
    like = residual if residual is not None else x
    H = like.shape[1]
    if like.shape[0] == 0:
        return
    # u: two factors and the product with rsqrt, whose sum of H squares takes
    # at most 48 roundings (32 a thread, 6 + 16 across waves, one root's half
    # of them) and the residual's fma: below 40 U of the terms
    tol = 40 * U * m
    if out is not None:
        half = 2.0 ** -8 if out.dtype == BF16 else U
        assert out.dtype == like.dtype
        diff = (out.double() - r).abs()
        assert bool((diff <= tol + half * r.abs() + 1e-38).all()), float((diff - tol - half * r.abs()).max())
    if y is None:
        assert yo is None
        return
    # y = r' * mul * w: r' as above, mul by 24 U and by the rows' own error
    rms = lambda v: v.pow(2).mean(-1, keepdim=True).sqrt()  # noqa: E731
    w = (kw["pre_weight"].double() + kw.get("weight_offset", 0.0)).abs()
    mul = 1 / torch.sqrt(r.pow(2).mean(-1, keepdim=True) + kw.get("eps", 1e-6))
    tol = tol * mul * w + y.abs() * (30 * U + 40 * U * rms(m) * mul)
    if not quantize:
        assert yo.dtype == BF16 and scales is None
        diff = (yo.double() - y).abs()
        assert bool((diff <= tol * 1.01 + 2.0 ** -8 * y.abs() + 1e-38).all()), float((diff - tol).max())
        return
    v, s = ref.quant_values(y)
    block = tol.reshape(-1, H // 128, 128).amax(-1)
    sdiff = (scales.double() - s).abs()
    assert bool((sdiff <= block / 448 + 4 * U * s).all()), float((sdiff / s).max())
    codes = yo.view(torch.float8_e4m3fn).double()
    vt = (tol + block.repeat_interleave(128, 1)) / s.repeat_interleave(128, 1) + 4 * U * v.abs()
    cdiff = (codes - v).abs()
    assert bool((cdiff <= torch.maximum(2.0 ** -4 * (v.abs() + vt), torch.full_like(v, 2.0 ** -10)) + vt).all()), \
        float(cdiff.max())


def norm_inputs(dev, T, H, xt, rt, pt, seed=0):
    g = gen(dev, seed + T + H)
    r = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    return dict(x=r(T, H).to(xt), residual=(3 * r(T, H)).to(rt), post=(1 + 0.3 * r(H)).to(pt),
                pre=(1 + 0.3 * r(H)).to(pt), channel=r(H).to(pt), token=r(T, 1).to(pt), full=r(T, H).to(pt))


SIZES = [(1, 7168), (5, 128), (3, 1), (4, 7), (9, 512), (6, 520), (2, 513), (3, 1000), (2, 8192), (2, 8200), (3, 16384),
         (1, 32768), (2, 20001), (70, 256)]


@pytest.mark.parametrize("T, H", SIZES)
@pytest.mark.parametrize("xt, rt, pt", [(BF16, BF16, BF16), (BF16, FP32, FP32), (FP32, BF16, FP32), (FP32, FP32, BF16)])
def test_norm(dev, T, H, xt, rt, pt):
    d = norm_inputs(dev, T, H, xt, rt, pt)
    for gate in (None, "channel", "token", "full"):
        print("norm", T, H, xt, rt, pt, gate, flush=True)
        kw = dict(post_weight=d["post"], gate=d[gate] if gate else None, residual_scale=0.5, pre_weight=d["pre"])
        check_norm(d["x"], d["residual"], **kw)
        if H % 128 == 0:
            check_norm(d["x"], d["residual"], quantize=True, **kw)


@pytest.mark.parametrize("T, H", [(3, 384), (2, 7168), (4, 1001)])
def test_norm_parts(dev, T, H):
    """Each operand left out in turn, the (1 + w) form, and r' not kept."""
    d = norm_inputs(dev, T, H, BF16, FP32, FP32)
    x, r, post, pre = d["x"], d["residual"], d["post"], d["pre"]
    check_norm(x, r)
    check_norm(x, r, post_weight=post)
    check_norm(x, r, pre_weight=pre, weight_offset=1.0, eps=1e-3)
    check_norm(x, r, post_weight=post, gate=d["channel"], weight_offset=1.0, pre_weight=pre)
    check_norm(x, None, post_weight=post, pre_weight=pre)
    check_norm(None, r, pre_weight=pre, residual_scale=2.0)
    check_norm(None, r, residual_scale=2.0)
    check_norm(x, r, gate=d["token"], pre_weight=pre, keep_residual=False)


@pytest.mark.parametrize("H", [100, 256, 7168])
def test_norm_strides_and_given_outputs(dev, H):
    d = norm_inputs(dev, 5, H, BF16, BF16, BF16)
    for extra in (1, 8):
        x, r, gate = padded(d["x"], extra), padded(d["residual"], 2 * extra), padded(d["full"], 3 * extra)
        big = torch.full((5, H + 3 * extra), 3.0, dtype=BF16, device=dev)
        y = torch.full((5, H + extra), 3.0, dtype=BF16, device=dev)
        kw = dict(post_weight=d["post"], gate=gate, pre_weight=d["pre"])
        got = w4.norm_residual(x, r, residual_out=big[:, :H], out=y[:, :H], **kw)
        check_norm(x, r, got=got, **kw)
        assert bool((big[:, H:] == 3).all()) and bool((y[:, H:] == 3).all())  # behind the rows
        # in place on the residual
        kept = r.clone()
        rr = padded(kept, 2 * extra)
        got = w4.norm_residual(x, rr, residual_out=rr, **kw)
        check_norm(x, kept, got=got, **kw)


def test_norm_special_rows(dev):
    """Rows of zeros, one huge and one tiny value, inf and NaN in one row only."""
    H = 256
    x = torch.randn(6, H, device=dev, generator=gen(dev, 1)).to(BF16)
    r = torch.zeros(6, H, dtype=FP32, device=dev)
    w = torch.ones(H, device=dev)
    x[0] = 0
    x[1, 5] = 2.0 ** 50
    x[2] *= 2.0 ** -60
    for q in (False, True):
        check_norm(x[:3], r[:3], post_weight=w, pre_weight=w, quantize=q)
    x[3, 7], x[4, 9] = INF, math.nan
    out, y, _ = w4.norm_residual(x, r, post_weight=w, pre_weight=w)
    assert bool(torch.isfinite(out[[0, 1, 2, 5]]).all()) and bool(torch.isfinite(y[[0, 1, 2, 5]]).all())
    assert bool(torch.isnan(y[[3, 4]]).any(-1).all())
    # codes hold no NaN that the clamp leaves: the block's scale is NaN
    _, q, scale = w4.norm_residual(x, r, post_weight=w, pre_weight=w, quantize=True)
    assert torch.isnan(scale).any(-1).tolist() == [False, False, False, True, True, False]
    # a NaN stays one in bf16 too
    _, y, _ = w4.norm_residual(None, x, pre_weight=w.to(BF16))
    assert bool(torch.isnan(y[4]).all())


def test_norm_empty(dev):
    for q in (False, True):
        out, y, s = w4.norm_residual(torch.empty(0, 256, device=dev), torch.empty(0, 256, device=dev),
                                     pre_weight=torch.ones(256, device=dev), quantize=q)
        assert out.shape == y.shape == (0, 256)


def test_norm_both_outputs_through_the_c_abi(dev):
    """bf16 and codes of one call are those of the two separate calls."""
    L, T, H = w4.load(), 37, 1024
    d = norm_inputs(dev, T, H, BF16, BF16, FP32)
    kw = dict(post_weight=d["post"], pre_weight=d["pre"], residual_scale=0.5)
    r, y, _ = w4.norm_residual(d["x"], d["residual"], **kw)
    _, q, s = w4.norm_residual(d["x"], d["residual"], quantize=True, **kw)
    r2, y2, q2, s2 = (torch.full_like(t, 1) for t in (r, y, q, s))
    p = lambda t: t.data_ptr()  # noqa: E731
    assert L.w4a8_norm_residual(p(d["x"]), 1, H, p(d["residual"]), 1, H, T, H, 0, p(d["post"]), None, 0, 0, 0.5, p(d["pre"]),
                                0.0, 1e-6, p(r2), H, p(y2), H, p(q2), p(s2),
                                torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in ((r, r2), (y, y2), (q, q2), (s, s2)))


def test_norm_codes_are_quantize_act_of_the_same_values(dev):
    """Rows whose normed values are bf16 numbers: the codes and scales are
    those of quantize_act on them, bit for bit."""
    H = 1024
    x = torch.where(torch.randn(8, H, device=dev, generator=gen(dev, 6)) > 0, 1.0, -1.0).to(BF16)  # mean square 1
    w = (1 + torch.randint(0, 64, (H,), device=dev, generator=gen(dev, 7)) / 64).to(BF16)
    _, y, _ = w4.norm_residual(x, None, pre_weight=w, eps=1e-30)
    assert torch.equal(y, x * w)
    _, q, s = w4.norm_residual(x, None, pre_weight=w, eps=1e-30, quantize=True)
    q2, s2 = w4.quantize_act(y)
    assert torch.equal(q, q2) and torch.equal(s, s2)


# ---- gemm_epilogue ---------------------------------------------------------------------

def gemm_inputs(dev, M, K, R, seed=0, dist="normal"):
    g = gen(dev, seed + M + K + R)
    x = torch.randn(M, K, generator=g, device=dev)
    if dist == "positive":
        x = x.abs() + 0.5
    x = x.to(BF16)
    q = (x.double() * 0).reshape(M, -1, 128)
    v, s = ref.quant_values(x.double())
    q = v.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    w = torch.randint(0, 256, (R, K // 2), generator=g, device=dev, dtype=torch.uint8)
    sw = 0.002 + 0.018 * torch.rand(R, K // 128, generator=g, device=dev)
    return q.contiguous(), s.float().contiguous(), w, sw


def check_gemm(ops, got=None, **kw):
    want, err = ref.gemm_epilogue(*ops, **{k: v for k, v in kw.items() if k not in ("out", "workspace")})
    out = got if got is not None else w4.gemm_epilogue(*ops, **kw)
    torch.cuda.synchronize()
    assert out.dtype == BF16 and out.shape == want.shape
    if out.numel() == 0:
        return
    diff = (out.double() - want).abs()
    assert bool((diff <= err + 2.0 ** -8 * (want.abs() + err)).all()), float((diff - err - 2.0 ** -8 * want.abs()).max())
    near = want.to(BF16).double()  # the library's bar for bf16 outputs
    fro = float((out.double() - near).norm() / near.norm().clamp_min(1e-300))
    print("gemm_epilogue", tuple(want.shape), "rel_fro %.2e" % fro, flush=True)
    assert fro <= 1e-3


SHAPES = [(1, 128, 16), (1, 7168, 512), (3, 256, 48), (16, 384, 33), (17, 640, 64), (33, 1152, 130), (64, 2048, 256),
          (65, 128, 72), (129, 896, 200), (200, 1664, 1), (257, 512, 260), (300, 256, 1030), (512, 1024, 512),
          (700, 384, 771), (1025, 256, 384)]


@pytest.mark.parametrize("M, K, N", SHAPES)
@pytest.mark.parametrize("act", list(w4.ACTIVATIONS))
def test_gemm_epilogue(dev, M, K, N, act):
    R = 2 * N if act == "swiglu" else N
    ops = gemm_inputs(dev, M, K, R)
    g = gen(dev, 99)
    bias = torch.randn(R, generator=g, device=dev)
    res = torch.randn(M, N, generator=g, device=dev).to(BF16)
    check_gemm(ops, activation=act)
    check_gemm(ops, activation=act, bias=bias, residual=res)
    check_gemm(ops, activation=act, bias=bias.to(BF16))


# sizes that run on tiles: whole ones, and ones whose last tiles hold one row,
# one column, half a unit; one and several groups
@pytest.mark.parametrize("M, K, N, act", [
    (4096, 128, 4096, "none"), (4097, 256, 4001, "silu"), (4001, 384, 2050, "swiglu"), (2000, 1152, 4097, "gelu"),
    (8000, 256, 1000, "relu"), (3000, 1024, 3001, "none"), (2570, 2048, 2049, "swiglu"), (2100, 7168, 4096, "none"),
    (2500, 640, 4230, "gelu_tanh")])
def test_gemm_epilogue_tiles(dev, M, K, N, act):
    assert w4.gemm_epilogue_workspace_bytes(M, K, N, act) > 0
    R = 2 * N if act == "swiglu" else N
    ops = gemm_inputs(dev, M, K, R)
    g = gen(dev, 98)
    bias = torch.randn(R, generator=g, device=dev)
    res = torch.randn(M, N, generator=g, device=dev).to(BF16)
    check_gemm(ops, activation=act, bias=bias, residual=res)
    # a workspace full of NaN, a row stride, the residual updated in place
    ws = torch.full((w4.gemm_epilogue_workspace_bytes(M, K, N, act),), 0xFF, dtype=torch.uint8, device=dev)
    rr = padded(res, 5)
    check_gemm(ops, activation=act, residual=res,
               got=w4.gemm_epilogue(*ops, activation=act, residual=rr, out=rr, workspace=ws))
    with pytest.raises(w4.W4A8Error):
        w4.gemm_epilogue(*ops, activation=act, workspace=ws[:-16])


def test_gemm_epilogue_tiles_same_sign_and_extremes(dev):
    q, s, w, sw = ops = gemm_inputs(dev, 4096, 256, 4096, dist="positive")
    assert w4.gemm_epilogue_workspace_bytes(4096, 256, 4096) > 0
    check_gemm(ops)
    check_gemm((torch.full_like(q, 0x7E), s, torch.full_like(w, 0x88), sw))
    s2, sw2 = s.clone(), sw.clone()
    s2[300, 1], sw2[9, 0] = math.nan, INF
    want, got = w4.gemm_epilogue(*ops), w4.gemm_epilogue(q, s2, w, sw2)
    assert bool(torch.isnan(got[300]).all()) and not bool(torch.isfinite(got[:, 9]).any())
    keep = torch.ones(4096, 4096, dtype=torch.bool, device=dev)
    keep[300], keep[:, 9] = False, False
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("M", [1, 40, 300, 600])
def test_gemm_epilogue_same_sign_and_extremes(dev, M):
    """Sums that do not cancel; codes of +-448; weights of -8 everywhere."""
    ops = gemm_inputs(dev, M, 2048, 96, dist="positive")
    check_gemm(ops)
    q, s, w, sw = ops
    check_gemm((torch.full_like(q, 0x7E), s, torch.full_like(w, 0x88), sw))
    check_gemm((torch.full_like(q, 0xFE), s, torch.full_like(w, 0x78), sw), activation="gelu")
    check_gemm((torch.zeros_like(q), s, w, sw), activation="silu")
    check_gemm((q, torch.full_like(s, 1e-12), w, sw), bias=torch.ones(96, device=dev))


@pytest.mark.parametrize("M, N", [(5, 64), (40, 36), (300, 100), (600, 260)])
@pytest.mark.parametrize("extra", [1, 4])
def test_gemm_epilogue_strides_and_in_place(dev, M, N, extra):
    ops = gemm_inputs(dev, M, 384, N)
    res = padded(torch.randn(M, N, device=dev, generator=gen(dev, 5)).to(BF16), extra)
    big = torch.full((M + 2, N + 3 * extra), 5.0, dtype=BF16, device=dev)
    out = big[:M, :N]
    check_gemm(ops, residual=res, got=w4.gemm_epilogue(*ops, residual=res, out=out))
    assert bool((big[:, N:] == 5).all()) and bool((big[M:] == 5).all())  # beside and behind
    rr = padded(res, extra)
    check_gemm(ops, residual=res, got=w4.gemm_epilogue(*ops, residual=rr, out=rr))


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh", "swiglu"])
def test_gemm_epilogue_activation_of_every_size(dev, act):
    """The activation alone, on biases from -60 to 60 and near 0 (zero codes)."""
    v = torch.cat([torch.linspace(-60, 60, 4001, device=dev), torch.logspace(-30, 0, 200, device=dev),
                   -torch.logspace(-30, 0, 200, device=dev), torch.zeros(3, device=dev)])
    bias = torch.cat([v, torch.ones_like(v)]) if act == "swiglu" else v
    q, s, w, sw = gemm_inputs(dev, 2, 128, bias.numel())
    check_gemm((torch.zeros_like(q), s, w, sw), activation=act, bias=bias)
    bias[0], bias[1] = INF, math.nan
    out = w4.gemm_epilogue(torch.zeros_like(q), s, w, sw, activation=act, bias=bias)
    assert bool((out[:, 0] == INF).all()) and bool(torch.isnan(out[:, 1]).all())


def test_gemm_epilogue_special_values(dev):
    """Scales of inf and NaN reach their own outputs and no others."""
    q, s, w, sw = gemm_inputs(dev, 40, 512, 64)
    want = w4.gemm_epilogue(q, s, w, sw)
    s2, sw2 = s.clone(), sw.clone()
    s2[3, 1], sw2[9, 2] = math.nan, INF
    got = w4.gemm_epilogue(q, s2, w, sw2)
    assert bool(torch.isnan(got[3]).all()) and not bool(torch.isfinite(got[:, 9]).any())
    keep = torch.ones(40, 64, dtype=torch.bool, device=dev)
    keep[3], keep[:, 9] = False, False
    assert torch.equal(got[keep], want[keep])


def test_gemm_epilogue_empty_batch(dev):
    q, s, w, sw = gemm_inputs(dev, 4, 256, 32)
    assert w4.gemm_epilogue(q[:0], s[:0], w, sw).shape == (0, 32)


def test_gemm_epilogue_agrees_with_gemm(dev):
    """Without an epilogue it computes what w4a8_gemm does."""
    for M in (1, 48, 500):
        ops = gemm_inputs(dev, M, 1024, 128)
        a, b = w4.gemm(*ops).double(), w4.gemm_epilogue(*ops).double()
        assert float((a - b).norm() / a.norm()) < 1e-3


@pytest.mark.parametrize("R", [64])
def test_gemm_epilogue_operands_over_4_gib(dev, R):
    """M * K past 2^32 bytes: the last rows are those of a small call."""
    K = 7168
    M = (1 << 32) // K + 300
    q, s, w, sw = gemm_inputs(dev, 64, K, R)
    big = torch.zeros(M, K, dtype=torch.uint8, device=dev)
    bs = torch.ones(M, K // 128, device=dev)
    for at in (0, M // 2, M - 64):
        big[at:at + 64], bs[at:at + 64] = q, s
    out = w4.gemm_epilogue(big, bs, w, sw)
    for at in (0, M // 2, M - 64):
        check_gemm((q, s, w, sw), got=out[at:at + 64].contiguous())
    assert int((out != 0).any(-1).sum()) == 3 * 64


# ---- together, on streams, in graphs -----------------------------------------------------

class Block:
    """One MoE block as a serving program runs it: norm, router, experts, the
    shared expert added to their output, then the norm before the next block."""

    def __init__(self, dev, T=96, H=512, I=256, E=16, local=8, k=4, seed=0):
        self.cfg, d = synth.random_moe(T, H, I, E, k, 0, local, seed=11)
        put = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        self.w = [put(d[n]) for n in ("w13", "s13", "w2", "s2")]
        self.packed = w4.prepack_weights(*self.w[:2]) + w4.prepack_weights(*self.w[2:])
        g = gen(dev, seed)
        self.router = torch.randn(E, H, generator=g, device=dev) / H ** 0.5
        self.bias = 0.1 * torch.randn(E, generator=g, device=dev)
        self.w1, self.w2 = (1 + 0.2 * torch.randn(H, generator=g, device=dev) for _ in range(2))
        self.sw = [t for t in gemm_inputs(dev, 1, H, 2 * I)[2:]] + [t for t in gemm_inputs(dev, 1, I, H)[2:]]
        self.ws = torch.empty(w4.fused_moe_workspace_bytes(T, H, k, local, I), dtype=torch.uint8, device=dev)
        self.num = torch.full((1,), T, dtype=torch.int32, device=dev)

    def __call__(self, x, stream):
        c = self.cfg
        r, h, _ = w4.norm_residual(x, stream, pre_weight=self.w1)
        logits = h.float() @ self.router.t()
        ids, wts = w4.moe_route(logits, c.topk, bias=self.bias, num_groups=4, topk_groups=2, scale=2.5,
                                num_tokens=self.num)
        moe = w4.fused_moe(h, ids, wts, c.expert_begin, c.E_local, *self.w, workspace=self.ws, prepacked=self.packed)
        _, q, s = w4.norm_residual(x, stream, pre_weight=self.w1, quantize=True, keep_residual=False)
        mid = w4.gemm_epilogue(q, s, *self.sw[:2], activation="swiglu")
        both = w4.gemm_epilogue(*w4.quantize_act(mid), *self.sw[2:], residual=moe)
        r2, y, _ = w4.norm_residual(both, r, post_weight=self.w2, gate=None, residual_scale=0.5, pre_weight=self.w1)
        return dict(r=r, h=h, logits=logits, ids=ids, wts=wts, moe=moe, q=q, s=s, mid=mid, both=both, r2=r2, y=y)


def test_block_chain(dev, orc):
    T, H = 96, 512
    b = Block(dev, T, H)
    b.num.fill_(T - 7)
    g = gen(dev, 3)
    x = torch.randn(T, H, generator=g, device=dev).to(BF16)
    stream = torch.randn(T, H, generator=g, device=dev)
    o = b(x, stream)
    torch.cuda.synchronize()
    check_norm(x, stream, got=(o["r"], o["h"], None), pre_weight=b.w1)
    check_norm(x, stream, got=(None, o["q"], o["s"]), quantize=True, pre_weight=b.w1)
    check_route(o["logits"], 4, got=(o["ids"], o["wts"]), bias=b.bias, num_groups=4, topk_groups=2, scale=2.5,
                num_tokens=b.num)
    assert bool((o["ids"][-7:] == -1).all()) and bool((o["moe"][-7:] == 0).all())  # padding costs no expert
    bits = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
    want = synth.bf16_bits_to_f32(orc.fused_moe(
        bits(o["h"]), o["ids"].cpu().numpy(), o["wts"].cpu().numpy(), 0, 8, *[t.cpu().numpy() for t in b.w]))
    got = o["moe"].float().cpu().numpy()
    assert np.linalg.norm(got - want) <= 1e-3 * np.linalg.norm(want)
    check_gemm((o["q"], o["s"], *b.sw[:2]), got=o["mid"], activation="swiglu")
    check_gemm((*w4.quantize_act(o["mid"]), *b.sw[2:]), got=o["both"], residual=o["moe"])
    check_norm(o["both"], o["r"], got=(o["r2"], o["y"], None), post_weight=b.w2, residual_scale=0.5, pre_weight=b.w1)


@pytest.mark.parametrize("T", [3, 96, 400])
def test_block_in_a_graph(dev, T):
    """Captured once and replayed on new inputs and another number of valid
    tokens, with eager calls and synchronisations in between."""
    H = 512
    b, eager = Block(dev, T, H), Block(dev, T, H)
    x, stream = torch.zeros(T, H, dtype=BF16, device=dev), torch.zeros(T, H, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b(x, stream)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = b(x, stream)
    for k in range(4):
        g = gen(dev, 20 + k)
        x.copy_(torch.randn(T, H, generator=g, device=dev))
        stream.copy_(torch.randn(T, H, generator=g, device=dev))
        for m in (b, eager):
            m.num.fill_(max(1, T - 5 * k))
        graph.replay()
        want = eager(x.clone(), stream.clone())
        torch.cuda.synchronize()
        for name in ("r", "h", "ids", "wts", "moe", "q", "s", "mid", "both", "r2", "y"):
            assert torch.equal(o[name], want[name]), (k, name)
    del graph


def test_block_on_another_stream(dev):
    """Work queued on a side stream reads what that stream wrote before it."""
    T, H = 64, 512
    b = Block(dev, T, H)
    g = gen(dev, 7)
    x = torch.randn(T, H, generator=g, device=dev).to(BF16)
    stream = torch.randn(T, H, generator=g, device=dev)
    want = {k: v.clone() for k, v in b(x, stream).items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x2, s2 = torch.zeros_like(x), torch.zeros_like(stream)
        busy = torch.ones(2048, 2048, device=dev)
        for _ in range(20):
            busy = busy @ busy * 1e-4
        x2.copy_(x)
        s2.copy_(stream)
        got = b(x2, s2)
    side.synchronize()
    for name in ("r", "h", "q", "s", "r2", "y"):
        assert torch.equal(got[name], want[name]), name
    # the same call twice gives the same bits
    again = b(x, stream)
    for name, v in want.items():
        if name != "logits":
            assert torch.equal(again[name], v), name


def test_gemm_epilogue_tiles_in_a_graph(dev):
    """The two launches of the tiles, captured and replayed on new operands,
    with eager calls and synchronisations in between."""
    M, K, N = 4096, 256, 4096
    ops = [t.clone() for t in gemm_inputs(dev, M, K, N)]
    assert w4.gemm_epilogue_workspace_bytes(M, K, N) > 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        w4.gemm_epilogue(*ops)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = w4.gemm_epilogue(*ops, activation="silu")
    for k in range(4):
        new = gemm_inputs(dev, M, K, N, seed=k)
        for t, u in zip(ops, new):
            t.copy_(u)
        graph.replay()
        want = w4.gemm_epilogue(*new, activation="silu")
        torch.cuda.synchronize()
        assert torch.equal(out, want), k
    del graph


@pytest.mark.parametrize("M, K, N", [(64, 2048, 512), (4096, 256, 4096)])
def test_two_streams_at_once(dev, M, K, N):
    """Calls that overlap on two streams, each with its own outputs."""
    sets = [gemm_inputs(dev, M, K, N, seed=k) for k in range(2)]
    rows = [norm_inputs(dev, M, 1024, BF16, FP32, FP32, seed=k) for k in range(2)]
    logits = [torch.randn(M, 256, device=dev, generator=gen(dev, k)) for k in range(2)]

    def calls(k):
        d = rows[k]
        return (w4.gemm_epilogue(*sets[k], activation="gelu"),
                *w4.norm_residual(d["x"], d["residual"], post_weight=d["post"], pre_weight=d["pre"], quantize=True),
                *w4.moe_route(logits[k], 8, num_groups=8, topk_groups=4))

    want = [calls(k) for k in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got[k].append(calls(k))
    torch.cuda.synchronize()
    for k in range(2):
        for one in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(one, want[k]))


def test_binding_refuses_a_workspace_with_holes_and_a_cut_group_top(dev):
    ops = gemm_inputs(dev, 2100, 7168, 1024)
    with pytest.raises(w4.W4A8Error, match="contiguous"):
        w4.gemm_epilogue(*ops, workspace=torch.zeros(16, 1, dtype=torch.uint8, device=dev).expand(16, 4096))
    with pytest.raises(w4.W4A8Error):
        w4.moe_route(torch.zeros(4, 16, device=dev), 4, group_top=2 + 2 ** 32)


def test_binding_checks_on_the_gpu(dev):
    x = torch.zeros(4, 256, dtype=BF16, device=dev)
    w = torch.ones(256, device=dev)
    for call in (
        lambda: w4.norm_residual(x, x, pre_weight=w, gate=w.to(BF16)),          # two parameter types
        lambda: w4.norm_residual(x, x.cpu(), pre_weight=w),                     # another device
        lambda: w4.norm_residual(x.to(FP16), x, pre_weight=w),
        lambda: w4.norm_residual(x, x[:, :128], pre_weight=w),
        lambda: w4.norm_residual(x.t().contiguous().t(), x, pre_weight=w),      # column stride
        lambda: w4.norm_residual(x, x, quantize=True),
        lambda: w4.norm_residual(x[:, :200].contiguous(), None, pre_weight=w[:200].contiguous(), quantize=True),
        lambda: w4.norm_residual(x, x, pre_weight=w, gate=torch.ones(4, 2, device=dev)),
        lambda: w4.norm_residual(x, x, pre_weight=w, residual_out=x.float()),
        lambda: w4.norm_residual(x[:, 1:], x[:, 1:], pre_weight=w[:255].contiguous()),  # not 16-byte aligned
        lambda: w4.moe_route(x, 300),
        lambda: w4.moe_route(x, 4, score="max"),
        lambda: w4.moe_route(x, 4, bias=torch.zeros(8, device=dev)),
        lambda: w4.moe_route(x, 4, num_tokens=torch.ones(1, dtype=torch.int64, device=dev)),
        lambda: w4.moe_route(x.double(), 4),
        lambda: w4.moe_route(x, 4, topk_ids=torch.zeros(4, 4, device=dev)),
    ):
        with pytest.raises(w4.W4A8Error):
            call()
    ops = gemm_inputs(dev, 4, 256, 32)
    for bad in (dict(activation="tanh"), dict(bias=torch.zeros(31, device=dev)), dict(bias=torch.zeros(32, device=dev).half()),
                dict(residual=torch.zeros(4, 32, device=dev)), dict(residual=torch.zeros(4, 31, device=dev, dtype=BF16)),
                dict(out=torch.zeros(3, 32, device=dev, dtype=BF16)), dict(activation="swiglu", bias=torch.zeros(16, device=dev))):
        with pytest.raises(w4.W4A8Error):
            w4.gemm_epilogue(*ops, **bad)
    with pytest.raises(w4.W4A8Error):
        w4.gemm_epilogue(ops[0], ops[1], ops[2][:31], ops[3][:31], activation="swiglu")


@pytest.mark.parametrize("M", [1, 64, 333])
def test_gemm_epilogue_with_an_empty_workspace(dev, M):
    """Sizes that need no workspace take an empty one, whose address is null."""
    K, N = 1664, 130
    ops = gemm_inputs(dev, M, K, N)
    assert w4.gemm_epilogue_workspace_bytes(M, K, N) == 0
    whole = torch.zeros(64, dtype=torch.uint8, device=dev)
    for ws in (torch.empty(0, dtype=torch.uint8, device=dev), whole[:0], whole):
        out = torch.full((M, N), math.nan, dtype=BF16, device=dev)
        assert w4.gemm_epilogue(*ops, out=out, workspace=ws) is out
        check_gemm(ops, got=out)


def test_gemm_epilogue_refuses_an_empty_workspace_for_tiles(dev):
    ops = gemm_inputs(dev, 4096, 256, 4096)
    need = w4.gemm_epilogue_workspace_bytes(4096, 256, 4096)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    for bad in (ws[:0], torch.empty(0, dtype=torch.uint8, device=dev), ws[:need - 1]):
        with pytest.raises(w4.W4A8Error, match="workspace"):
            w4.gemm_epilogue(*ops, workspace=bad)
    for bad in (torch.empty(0, dtype=torch.uint8), torch.empty(need, dtype=torch.uint8)):  # in host memory
        with pytest.raises(w4.W4A8Error, match="one GPU"):
            w4.gemm_epilogue(*ops, workspace=bad)


def test_gemm_with_an_empty_workspace(dev):
    """gemm and the fused forward, too: computed where none is needed, else
    refused."""
    for M, K, N in ((1, 1024, 64), (48, 1024, 128), (700, 1024, 64)):
        ops = gemm_inputs(dev, M, K, N)
        out = torch.full((M, N), math.nan, dtype=BF16, device=dev)
        empty = torch.empty(0, dtype=torch.uint8, device=dev)
        if w4.gemm_workspace_bytes(M, K, N) == 0:
            assert torch.equal(w4.gemm(*ops, out=out, workspace=empty), w4.gemm(*ops))
        else:
            with pytest.raises(w4.W4A8Error, match="workspace"):
                w4.gemm(*ops, out=out, workspace=empty)
    b = Block(dev, 8)
    x = torch.randn(8, 512, device=dev, generator=gen(dev, 3)).to(BF16)
    ids = torch.zeros(8, b.cfg.topk, dtype=torch.int32, device=dev)
    for packed in (None, b.packed):
        with pytest.raises(w4.W4A8Error, match="workspace"):
            w4.fused_moe(x, ids, ids.float(), 0, 8, *b.w, workspace=b.ws[:0], prepacked=packed)


def test_gemm_refuses_a_workspace_with_holes(dev):
    """An expanded tensor names more elements than it holds."""
    ops = gemm_inputs(dev, 128, 7168, 512)
    need = w4.gemm_workspace_bytes(128, 7168, 512)
    assert need > 0
    holes = torch.zeros(16, 1, dtype=torch.uint8, device=dev).expand(16, need)
    with pytest.raises(w4.W4A8Error, match="contiguous"):
        w4.gemm(*ops, workspace=holes)
    b = Block(dev, 8)
    x = torch.zeros(8, 512, dtype=BF16, device=dev)
    ids = torch.zeros(8, b.cfg.topk, dtype=torch.int32, device=dev)
    with pytest.raises(w4.W4A8Error, match="contiguous"):
        w4.fused_moe(x, ids, ids.float(), 0, 8, *b.w, workspace=holes[:, :b.ws.numel()])


@pytest.mark.parametrize("M, K, N", [(1, 2048, 96), (40, 2048, 96), (300, 2048, 96), (600, 2048, 96), (2500, 1024, 900),
                                     (4096, 256, 4096)])
def test_gemm_epilogue_small_weights(dev, M, K, N):
    """The bound counts the products themselves: weights of 0 give 0 whatever
    the activations, weights of -1, 0 and 1 are as exact as larger ones, and a
    large activation under a weight of 0 costs its neighbours nothing."""
    q, s, w, sw = gemm_inputs(dev, M, K, N, dist="positive")
    zero = torch.zeros_like(w)
    check_gemm((q, s, zero, sw))
    check_gemm((torch.full_like(q, 0x7E), s, zero, sw), bias=torch.ones(N, device=dev))
    some = zero.clone()
    some[::2] = w[::2]  # every other weight row
    check_gemm((q, s, some, sw))
    g = gen(dev, K + N)
    unit = lambda: torch.randint(0, 3, w.shape, generator=g, device=dev, dtype=torch.uint8)  # noqa: E731
    signs = torch.tensor([0, 1, 15], dtype=torch.uint8, device=dev)
    check_gemm((q, s, signs[unit().long()] | signs[unit().long()] << 4, sw))
    check_gemm((torch.full_like(q, 0x7E), s, signs[unit().long()] | signs[unit().long()] << 4, sw))
    # +-448 under a weight of 0 in every group, codes of 2^-4 to 2^-2 elsewhere
    small = (0x18 + torch.randint(0, 16, q.shape, generator=g, device=dev, dtype=torch.uint8)) \
        | torch.randint(0, 2, q.shape, generator=g, device=dev, dtype=torch.uint8) << 7
    small[:, 10::128] = 0x7E
    small[:, 75::128] = 0xFE
    clear = w.clone()
    clear[:, 5::64] &= 0xF0   # k = 10 of 128
    clear[:, 37::64] &= 0x0F  # k = 75
    check_gemm((small, s, clear, sw))


@pytest.mark.parametrize("M, K, N", [(1, 256, 40), (40, 256, 36), (300, 256, 100), (2500, 256, 2500)])
def test_gemm_epilogue_largest_scale(dev, M, K, N):
    """Activations up to the largest bf16 have scales up to 2^128 / 448: their
    products stay finite where the result does."""
    q, _, w, sw = gemm_inputs(dev, M, K, N)
    top = torch.finfo(BF16).max / 448
    s = torch.full((M, K // 128), top, device=dev)
    s[1::2] = 2.0
    few = torch.zeros_like(q)
    few[:, ::32] = q[:, ::32]
    assert float(ref.gemm_epilogue(few, s, w, sw)[0].abs().max()) < torch.finfo(BF16).max
    check_gemm((few, s, w, sw))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E, groups, kept", [(16, 2, 1), (64, 8, 1), (64, 8, 3), (256, 8, 1), (256, 8, 4), (512, 4, 1),
                                             (512, 4, 2), (90, 6, 1), (1000, 8, 2), (128, 32, 5)])
def test_route_groups_whose_sums_pass_32_bits(dev, score, E, groups, kept):
    """Sums of two finite choices that 32 bits hold as an infinity: biases of
    the type's lowest value as a mask, and of +-2e38 and +-3e38."""
    size = E // groups
    g = gen(dev, E)
    x = torch.randn(40, E, generator=g, device=dev)
    x[:20, :size] = -INF                       # the first group is empty
    x[10:20, size + 1:2 * size] = -INF         # the next holds one expert
    low = torch.finfo(FP32).min
    biases = [torch.full((E,), low, device=dev), torch.full((E,), 3e38, device=dev)]
    for values in ((low, -3e38, -2e38), (3e38, 2e38, 2.5e38), (low, 3e38, -INF), (low, 0.0, 3e38), (-2e38, 2e38, INF)):
        b = torch.tensor(values, device=dev)[torch.randint(0, 3, (E,), generator=g, device=dev)]
        biases += [b, b.reshape(groups, size)[:, :1].expand(-1, size).reshape(E).contiguous()]
    for b in biases:
        for top in (1, 2):
            for rows in (x, x.to(BF16)):
                check_route(rows, min(4, kept * size), score=score, bias=b, num_groups=groups, topk_groups=kept,
                            group_top=top)


@pytest.mark.parametrize("T, H", [(513, 520), (600, 1000), (517, 7168), (514, 8192), (530, 2085), (600, 512), (513, 513)])
@pytest.mark.parametrize("xt, rt, pt", [(BF16, BF16, BF16), (BF16, FP32, FP32), (FP32, BF16, FP32)])
def test_norm_many_rows(dev, T, H, xt, rt, pt):
    """More rows than get a workgroup of one chunk a thread, every row its own."""
    d = norm_inputs(dev, T, H, xt, rt, pt, seed=40)
    x, r = padded(d["x"], 3), padded(d["residual"], 5)
    for gate in ("channel", "token", "full"):
        g = padded(d["full"], 1) if gate == "full" else d[gate]
        kw = dict(post_weight=d["post"], gate=g, residual_scale=0.5, pre_weight=d["pre"])
        y = torch.full((T, H + 1), 3.0, dtype=BF16, device=dev)
        check_norm(x, r, got=w4.norm_residual(x, r, out=y[:, :H], **kw), **kw)
        assert bool((y[:, H:] == 3).all())
        if H % 128 == 0:
            check_norm(x, r, quantize=True, **kw)


@pytest.mark.parametrize("dtype", [FP32, BF16])
@pytest.mark.parametrize("T, E, k, groups, kept", [(4097, 64, 6, 8, 3), (4099, 40, 4, 1, 1), (4110, 33, 12, 3, 2), (4111, 160, 8, 4, 2)])
def test_route_many_tokens(dev, dtype, T, E, k, groups, kept):
    """More tokens than get a workgroup of one wave, every row its own: random
    ones, near ties, and padding that begins inside the last workgroup."""
    g = gen(dev, T)
    x = torch.randn(T, E, generator=g, device=dev)
    x[1::3] = 1 + torch.finfo(dtype).eps * torch.randint(0, 9, (T, E), generator=g, device=dev)[1::3]
    x[7::50] = -INF
    x = padded(x.to(dtype), 5)
    bias = 0.2 * torch.randn(E, generator=g, device=dev)
    for score, b, num in (("sigmoid", None, T), ("sigmoid", bias, T - 1), ("softmax", torch.zeros_like(bias), T - 6),
                          ("softmax", None, 4094)):
        n = torch.tensor([num], dtype=torch.int32, device=dev)
        check_route(x, k, score=score, bias=b, num_groups=groups, topk_groups=kept, num_tokens=n, renormalize=b is None)


@pytest.mark.parametrize("M, K, N", [(1, 512, 48), (40, 512, 48), (300, 512, 100), (4096, 256, 4096)])
def test_gemm_epilogue_keeps_13_bits_below_the_largest_product(dev, M, K, N):
    """Large activations under weights of +-1, whose products cancel, and small
    ones beside them: the matrix instruction cuts a product to 2^-13 of the
    largest of its eight neighbours in K, so each eight are off by at most 7
    2^-13 of that."""
    g = gen(dev, M + N)
    s = 0.5 + torch.rand(M, K // 128, generator=g, device=dev)
    sw = 0.002 + 0.018 * torch.rand(N, K // 128, generator=g, device=dev)
    for small, unit in ((0x20, 1), (0x20, 0), (0x28, 0), (0x18, 0)):
        # codes of about 2^-3, 2^-2 and 2^-4; +448 and -448 in turn at one place of every eight
        q = small + torch.randint(0, 1 if unit else 8, (M, K), generator=g, device=dev, dtype=torch.uint8)
        q[:, 3::16], q[:, 11::16] = 0x7E, 0xFE
        v = torch.ones(N, K, dtype=torch.uint8, device=dev) if unit else \
            torch.randint(0, 8, (N, K), generator=g, device=dev, dtype=torch.uint8)
        v[:, 3::8] = 1
        v[::2, 3::8] = 15  # -1
        w = v[:, ::2] | v[:, 1::2] << 4
        out = w4.gemm_epilogue(q, s, w, sw).double()
        want, _ = ref.gemm_epilogue(q, s, w, sw)
        # the eights' largest products: 448 times 1, the small ones' are below 4
        top = torch.full((N, K // 8), 448.0, dtype=torch.float64, device=dev)
        err = 7 * 2.0 ** -13 * (s.double() @ (top.reshape(N, -1, 16).sum(-1) * sw.double()).t().contiguous())
        err = err + (2 * (K // 128) + 2) * U * (ref.dequant(q, s).abs() @ ref.int4(w, sw).abs().t().contiguous())
        diff = (out - want).abs()
        assert bool((diff <= err + 2.0 ** -8 * (want.abs() + err)).all()), float((diff - err - 2.0 ** -8 * want.abs()).max())
