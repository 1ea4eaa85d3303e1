"""The attention half of a served block (gemm_fp8, rope, kv_append,
attn_decode) on the GPU against its plain 64-bit forms (attn_refs.py)."""
import math

import pytest
import torch

import attn_refs as ref
import block_refs
from attn_refs import rounded
from block_refs import U
from w4a8_moe_grouped_amd import lib as w4

pytestmark = pytest.mark.gpu

BF16, FP32, FP16, FP8 = torch.bfloat16, torch.float32, torch.float16, torch.float8_e4m3fn
INF = math.inf


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "the gpu tests need an MI355X"
    w4.load()
    return torch.device("cuda:0")


def gen(dev, seed):
    return torch.Generator(device=dev).manual_seed(seed)


def near(got, want, err, dtype=None):
    """Every element within its bound; infinities and NaN in the same places."""
    got = got.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)])
    if dtype is not None:
        err = rounded(want, err, dtype)
    diff = (got - want).abs()[fine]
    assert bool((diff <= err[fine]).all()), float((diff - err[fine]).max())


def quantised(x):
    """e4m3 codes and scales of the rows along the last axis."""
    amax = x.double().abs().amax(-1, keepdim=True).clamp_min(1e-10)
    return (x.double() / amax * 448).float().to(FP8).view(torch.uint8), (amax / 448).float().squeeze(-1)


# ---- gemm_fp8 ------------------------------------------------------------------------

def gemm_inputs(dev, M, K, R, seed=0, dist="normal"):
    g = gen(dev, seed + M + K + R)
    x = torch.randn(M, K // 128, 128, generator=g, device=dev)
    w = torch.randn(R, K, generator=g, device=dev)
    if dist == "positive":
        x, w = x.abs() + 0.5, w.abs() + 0.1
    q, s = quantised(x)
    wq = (100 * w).clamp(-448, 448).to(FP8).view(torch.uint8)
    sw = (0.5 + torch.rand(-(-R // 128), K // 128, generator=g, device=dev)) * 2e-4
    return q.reshape(M, K), s, wq, sw


def check_gemm(ops, got=None, **kw):
    want, err = ref.gemm_fp8(*ops, **{k: v for k, v in kw.items() if k not in ("out", "workspace")})
    out = got if got is not None else w4.gemm_fp8(*ops, **kw)
    torch.cuda.synchronize()
    assert out.dtype == BF16 and out.shape == want.shape
    if out.numel() == 0:
        return
    near(out, want, err, BF16)
    close = want.to(BF16).double()  # the library's bar for bf16 outputs
    fro = float((out.double() - close).norm() / close.norm().clamp_min(1e-300))
    print("gemm_fp8", tuple(want.shape), "rel_fro %.2e" % fro, flush=True)
    assert fro <= 1e-3


SHAPES = [(1, 128, 16), (1, 7168, 512), (3, 256, 48), (8, 384, 33), (9, 640, 100), (16, 1152, 130), (17, 640, 64),
          (33, 1664, 130), (64, 2048, 256), (65, 128, 72), (128, 1280, 300), (129, 896, 200), (200, 1664, 1),
          (257, 512, 260), (300, 256, 1030), (700, 384, 771), (1025, 256, 384)]


@pytest.mark.parametrize("M, K, N", SHAPES)
@pytest.mark.parametrize("act", list(w4.ACTIVATIONS))
def test_gemm_fp8(dev, M, K, N, act):
    if act == "swiglu":
        N = -(-N // 128) * 128
    R = 2 * N if act == "swiglu" else N
    ops = gemm_inputs(dev, M, K, R)
    g = gen(dev, 99)
    bias = torch.randn(R, generator=g, device=dev)
    res = torch.randn(M, N, generator=g, device=dev).to(BF16)
    check_gemm(ops, activation=act)
    check_gemm(ops, activation=act, bias=bias, residual=res)
    check_gemm(ops, activation=act, bias=bias.to(BF16))


# sizes of both tiles: whole ones, and ones whose last tiles hold one row, one
# column, half of a scale's block; one and several groups, in fours and not
@pytest.mark.parametrize("M, K, N, act", [
    (4096, 128, 4096, "none"), (4097, 256, 4001, "silu"), (4001, 384, 2048, "swiglu"), (2000, 1152, 4097, "gelu"),
    (8000, 512, 1000, "relu"), (3000, 1024, 3001, "none"), (2570, 2048, 2176, "swiglu"), (2100, 7168, 4096, "none"),
    (130, 512, 5000, "none"), (515, 640, 256, "swiglu")])
def test_gemm_fp8_tiles(dev, M, K, N, act):
    R = 2 * N if act == "swiglu" else N
    ops = gemm_inputs(dev, M, K, R)
    g = gen(dev, 98)
    bias = torch.randn(R, generator=g, device=dev)
    res = torch.randn(M, N, generator=g, device=dev).to(BF16)
    check_gemm(ops, activation=act, bias=bias, residual=res)
    check_gemm(ops, activation=act)


# some row blocks times column counts around a multiple of 8 blocks of 32 and of 64
@pytest.mark.parametrize("M, K, N", [(96, 1024, 5000), (70, 512, 545), (100, 384, 1030), (200, 1024, 1500),
                                     (333, 256, 2050), (128, 2048, 991), (33, 256, 513), (65, 1024, 4100)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_gemm_fp8_several_row_blocks(dev, M, K, N, act):
    N = N if act == "none" else N // 128 * 128
    check_gemm(gemm_inputs(dev, M, K, 2 * N if act == "swiglu" else N), activation=act)


@pytest.mark.parametrize("M", [1, 40, 300, 2500])
def test_gemm_fp8_same_sign_and_extremes(dev, M):
    check_gemm(gemm_inputs(dev, M, 2048, 96 if M < 2000 else 2500, dist="positive"))
    q, s, w, sw = gemm_inputs(dev, M, 512, 64 if M < 2000 else 2500)
    s[:, 1] = 2.0 ** 100   # scales far apart, and weights of zero
    sw[:, 1] = 2.0 ** -110
    s[0, 0] = 0.0
    w[:, 128:160] = 0
    check_gemm((q, s, w, sw))


@pytest.mark.parametrize("M, N", [(1, 40), (40, 36), (300, 260), (2500, 2500)])
def test_gemm_fp8_largest_scale(dev, M, N):
    """The largest activation scale (a bf16 maximum / 448) under small weight scales."""
    q, s, w, sw = gemm_inputs(dev, M, 256, N)
    check_gemm((q, torch.full_like(s, 3.38e38 / 448), w, sw * 2.0 ** -60))


@pytest.mark.parametrize("M, N", [(5, 64), (40, 36), (300, 100), (2500, 2500)])
@pytest.mark.parametrize("extra", [1, 4])
def test_gemm_fp8_strides_and_in_place(dev, M, N, extra):
    ops = gemm_inputs(dev, M, 256, N)
    wide = torch.full((M, N + extra), 7.0, dtype=BF16, device=dev)
    wide[:, :N] = torch.randn(M, N, generator=gen(dev, 4), device=dev)
    res = wide[:, :N].clone()
    out = w4.gemm_fp8(*ops, residual=wide[:, :N], out=wide[:, :N])
    assert out.data_ptr() == wide.data_ptr()
    check_gemm(ops, got=out, residual=res)
    assert bool((wide[:, N:] == 7.0).all())


@pytest.mark.parametrize("M", [1, 8, 9, 64, 300, 2500])
def test_gemm_fp8_nan_stays_in_its_row(dev, M):
    N = 40 if M < 2000 else 2500
    q, s, w, sw = gemm_inputs(dev, M, 384, N)
    q[M // 2, 130] = 0x7F
    w[N // 3, 5] = 0x7F
    want, _ = ref.gemm_fp8(q, s, w, sw)
    out = w4.gemm_fp8(q, s, w, sw)
    assert torch.equal(torch.isnan(out), torch.isnan(want))


def test_gemm_fp8_types_and_empty_batch(dev):
    ops = gemm_inputs(dev, 5, 256, 40)
    a = w4.gemm_fp8(*ops)
    b = w4.gemm_fp8(ops[0].view(FP8), ops[1], ops[2].view(FP8), ops[3], workspace=torch.empty(0, device=dev))
    assert torch.equal(a, b)
    out = w4.gemm_fp8(ops[0][:0], ops[1][:0], ops[2], ops[3])
    assert out.shape == (0, 40)


# ---- rope ----------------------------------------------------------------------------

def check_rope(x, positions, freq, got=None, **kw):
    want, err = ref.rope(x, positions, freq, **{k: v for k, v in kw.items() if k != "out"})
    out = got if got is not None else w4.rope(x, positions, freq, **kw)
    torch.cuda.synchronize()
    assert out.dtype == x.dtype and out.shape == x.shape
    near(out, want, err, x.dtype)


HEADS = [(128, 128), (128, 64), (64, 64), (80, 80), (80, 20), (80, 32), (96, 48), (112, 112), (192, 64), (256, 256),
         (256, 64), (8, 8), (8, 2), (24, 14), (136, 34), (248, 248), (128, 0), (40, 40)]


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D, R", HEADS)
def test_rope(dev, dtype, interleaved, D, R):
    freq = ref.frequencies(R).to(dev)
    for T, heads in ((1, 1), (7, 5), (33, 72), (300, 80)):
        g = gen(dev, T + D)
        x = torch.randn(T, heads, D, generator=g, device=dev).to(dtype)
        pos = torch.randint(0, 1 << 20, (T,), generator=g, device=dev, dtype=torch.int32)
        check_rope(x, pos, freq, interleaved=interleaved)
    check_rope(x, pos, freq, interleaved=interleaved, magnitude=1.25)


def test_rope_positions_of_every_size(dev):
    """Small, far, negative and the largest positions; the sine and cosine of every eighth of a turn."""
    p = [0, 1, 2, 3, -1, -5, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31] + [7 ** k for k in range(11)]
    pos = torch.tensor(p, dtype=torch.int32, device=dev)
    x = torch.randn(len(p), 4, 128, generator=gen(dev, 1), device=dev)
    check_rope(x, pos, ref.frequencies(128).to(dev))
    turns = torch.arange(64, dtype=torch.float64, device=dev) / 64 * (2 * math.pi)
    pos = torch.arange(-130, 130, dtype=torch.int32, device=dev)
    x = torch.randn(260, 2, 128, generator=gen(dev, 2), device=dev)
    check_rope(x, pos, turns)
    check_rope(x, pos, -turns, interleaved=True)


@pytest.mark.parametrize("D, R, interleaved", [(128, 128, False), (80, 20, False), (128, 64, True)])
def test_rope_strides_and_in_place(dev, D, R, interleaved):
    freq = ref.frequencies(R).to(dev)
    big = torch.randn(9, 12, D + 8, generator=gen(dev, 3), device=dev).to(BF16)
    keep = big.clone()
    view = big[:, 2:7, :D]
    x = view.clone()
    pos = torch.arange(100, 109, dtype=torch.int32, device=dev)
    out = w4.rope(view, pos, freq, interleaved=interleaved, out=view)
    assert out.data_ptr() == view.data_ptr()
    check_rope(x, pos, freq, got=out, interleaved=interleaved)
    big[:, 2:7, :D] = x
    assert torch.equal(big, keep)
    # heads before tokens
    turned = torch.randn(5, 9, D, generator=gen(dev, 4), device=dev).to(BF16).transpose(0, 1)
    check_rope(turned, pos, freq, interleaved=interleaved)


def test_rope_empty(dev):
    freq = ref.frequencies(64).to(dev)
    none = torch.empty(0, dtype=torch.int32, device=dev)
    assert w4.rope(torch.empty(0, 4, 64, device=dev), none, freq).shape == (0, 4, 64)
    assert w4.rope(torch.empty(3, 0, 64, device=dev), torch.zeros(3, dtype=torch.int32, device=dev), freq).shape == (3, 0, 64)


@pytest.mark.parametrize("R, kw", [
    (128, {}), (2, {}), (64, dict(base=500000.0)), (128, dict(scaling="linear", factor=4.0)),
    (96, dict(scaling="ntk", factor=8.0)), (128, dict(scaling="yarn", factor=16.0, original_length=4096.0)),
    (64, dict(scaling="yarn", factor=40.0, original_length=4096.0, base=1e6, beta_fast=16.0, beta_slow=2.0)),
    (64, dict(scaling="yarn", factor=4.0, original_length=8.0))])
def test_rope_frequencies(dev, R, kw):
    want = ref.frequencies(R, **kw)
    got = w4.rope_frequencies(R, device=dev, **kw).cpu()
    torch.testing.assert_close(got, want, rtol=1e-13, atol=0)


# ---- kv_append -----------------------------------------------------------------------

def make_cache(dev, pages, page, Hkv, D, kind, layout="tokens", seed=0):
    """k, v caches and scales with contents, [pages, page, Hkv, D] views of the layout."""
    g = gen(dev, seed)
    out = []
    for _ in range(2):
        x = torch.randn(pages, page, Hkv, D, generator=g, device=dev)
        x, s = quantised(x) if kind == "fp8" else (x.to(kind), None)
        if layout == "heads":
            x = x.transpose(1, 2).contiguous().transpose(1, 2)
        out += [x, None if s is None else s.transpose(1, 2).contiguous()]
    if layout == "joined":  # keys and values of a page side by side
        both = torch.stack((out[0], out[2]), 1)
        out[0], out[2] = both[:, 0], both[:, 1]
    return out[0], out[2], out[1], out[3]


def check_rows(cache, scales, old, old_scales, rows, err, slots, page):
    """Rows in their slots, all else as it was."""
    kept = (slots >= 0) & (slots < cache.shape[0] * page)
    at, rows, err = slots[kept], rows[kept], err[kept]
    p, t = at // page, at % page
    got = cache[p, t]
    if scales is None:
        near(got, rows, err, cache.dtype)
    else:
        s = rows.abs().amax(-1).clamp_min(1e-10) / 448
        worst = err.amax(-1) / 448
        near(scales[p, :, t], s, worst + 3 * U * s)
        # half a step of e4m3 (2^-10 below its normal range), the scale's error and two roundings
        want = rows / s[..., None]
        bound = 2.0 ** -4 * want.abs() + 2.0 ** -10 + (err + worst[..., None] * want.abs()) / s[..., None] * 1.1 + 1e-4
        near(got.view(FP8), want, bound)
        old_scales[p, :, t] = scales[p, :, t]
        assert torch.equal(scales, old_scales)
    old[p, t] = got
    assert torch.equal(cache, old)


def check_append(dev, T, Hq, Hkv, D, R, dtype, kind, page, layout="tokens", interleaved=False, drop=True, fused=True,
                 magnitude=1.0, with_q=True):
    print("append", T, Hq, Hkv, D, R, dtype, kind, page, layout, interleaved, flush=True)
    g = gen(dev, T + D + page)
    pages = -(-(T + 5) // page) + 1
    kc, vc, ks, vs = make_cache(dev, pages, page, Hkv, D, kind, layout)
    old = [None if t is None else t.clone() for t in (kc, vc, ks, vs)]
    if fused:
        q, k, v = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=dev).to(dtype).split((Hq, Hkv, Hkv), 1)
    else:
        q, k, v = (torch.randn(T, h, D, generator=g, device=dev).to(dtype) for h in (Hq, Hkv, Hkv))
    slots = torch.randperm(pages * page, generator=g, device=dev)[:T]
    if drop:
        slots[T // 2] = -1
        slots[-1] = pages * page
    pos = torch.randint(0, 100000, (T,), generator=g, device=dev, dtype=torch.int32)
    freq = ref.frequencies(R).to(dev) if R else None
    kw = dict(positions=pos, frequencies=freq) if R else {}
    got = w4.kv_append(k, v, kc, vc, slots, k_scales=ks, v_scales=vs, interleaved=interleaved, magnitude=magnitude,
                       q=q if with_q else None, **kw)
    torch.cuda.synchronize()
    none = torch.empty(0, dtype=torch.float64, device=dev)
    turn = lambda x: ref.rope(x, pos, none if freq is None else freq, interleaved, magnitude)  # noqa: E731
    if with_q:
        near(got, *turn(q), dtype)
    else:
        assert got is None
    check_rows(kc, ks, old[0], old[2], *turn(k), slots, page)
    check_rows(vc, vs, old[1], old[3], v.double(), torch.zeros_like(v, dtype=torch.float64), slots, page)


@pytest.mark.parametrize("kind", [BF16, FP16, "fp8"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D, R", [(128, 128), (64, 32), (80, 20), (256, 256), (8, 8), (24, 10), (192, 64), (136, 136)])
def test_kv_append(dev, kind, interleaved, D, R):
    dtype = BF16 if kind == "fp8" else kind
    for T, Hq, Hkv, page, layout in ((3, 4, 2, 16, "tokens"), (37, 14, 2, 7, "heads"), (40, 5, 5, 1, "joined")):
        check_append(dev, T, Hq, Hkv, D, R, dtype, kind, page, layout, interleaved)


@pytest.mark.parametrize("kind", [BF16, "fp8"])
def test_kv_append_forms(dev, kind):
    check_append(dev, 5, 0, 3, 64, 64, BF16, kind, 16, fused=False)                 # no query heads
    check_append(dev, 5, 4, 3, 64, 64, BF16, kind, 16, with_q=False)
    check_append(dev, 5, 4, 3, 128, 0, BF16, kind, 16)                              # no rotation
    check_append(dev, 1, 64, 8, 128, 128, BF16, kind, 64, drop=False, magnitude=1.5)
    check_append(dev, 2000, 64, 8, 128, 128, BF16, kind, 64)                        # four rows a lane group
    check_append(dev, 2100, 20, 5, 200, 24, BF16, kind, 24, interleaved=True)
    if kind == "fp8":
        check_append(dev, 9, 4, 2, 128, 64, FP16, kind, 16)


@pytest.mark.parametrize("T, heads, D, dtype", [(8193, 1, 128, FP32), (8200, 3, 256, BF16), (2731, 24, 64, FP16), (8192, 8, 128, BF16)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_many_tokens(dev, T, heads, D, dtype, interleaved):
    """Either side of where a lane group takes four rows, and fewer rows than it could take."""
    g = gen(dev, T)
    x = torch.randn(T, heads, D, generator=g, device=dev).to(dtype)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device=dev, dtype=torch.int32)
    check_rope(x, pos, w4.rope_frequencies(D, device=dev), interleaved=interleaved)


@pytest.mark.parametrize("kind", [BF16, "fp8"])
@pytest.mark.parametrize("T, Hq, Hkv, D, page", [(8193, 2, 2, 256, 61), (8200, 1, 1, 128, 16), (4100, 4, 1, 256, 64)])
def test_kv_append_many_tokens(dev, kind, T, Hq, Hkv, D, page):
    check_append(dev, T, Hq, Hkv, D, 128, BF16, kind, page)


def test_kv_append_codes_are_those_of_quantize_act(dev):
    T, H = 50, 4
    x = torch.randn(T, 2 * H, 128, generator=gen(dev, 5), device=dev).to(BF16)
    x[3, 1] = 0.0
    x[4, 2] *= 1e-30
    kc, vc, ks, vs = make_cache(dev, 4, 16, H, 128, "fp8")
    w4.kv_append(x[:, :H], x[:, H:], kc, vc, torch.arange(T, device=dev), k_scales=ks, v_scales=vs)
    q, s = w4.quantize_act(x.reshape(T, -1))
    q, s = q.reshape(T, 2 * H, 128), s.reshape(T, 2 * H)
    for cache, scales, at in ((kc, ks, slice(0, H)), (vc, vs, slice(H, 2 * H))):
        assert torch.equal(cache.reshape(-1, H, 128)[:T], q[:, at])
        assert torch.equal(scales.transpose(1, 2).reshape(-1, H)[:T], s[:, at])


def test_cache_of_float8_tensors(dev):
    """Codes may come as uint8 or as float8_e4m3fn."""
    d = make_batch(dev, [40, 3], 4, 2, 64, "fp8", 16)
    f8 = {k: v.view(FP8) if k in ("k_cache", "v_cache") else v for k, v in d.items()}
    assert torch.equal(w4.attn_decode(**d)[0], w4.attn_decode(**f8)[0])
    x = torch.randn(2, 2, 64, generator=gen(dev, 5), device=dev).to(BF16)
    slots = torch.tensor([5, 17], device=dev)
    before = d["k_cache"].clone()
    w4.kv_append(x, x, f8["k_cache"], f8["v_cache"], slots, k_scales=d["k_scales"], v_scales=d["v_scales"])
    assert not torch.equal(d["k_cache"], before)


def test_kv_append_nan_shows_in_the_scale(dev):
    x = torch.randn(3, 2, 64, generator=gen(dev, 5), device=dev).to(BF16)
    x[1, 0, 9] = math.nan
    kc, vc, ks, vs = make_cache(dev, 1, 16, 2, 64, "fp8")
    w4.kv_append(x, x, kc, vc, torch.arange(3, device=dev), k_scales=ks, v_scales=vs)
    for s in (ks, vs):
        assert torch.isnan(s[0, :, :3]).tolist() == [[False, True, False], [False, False, False]]


def test_kv_append_in_place_and_empty(dev):
    q = torch.randn(4, 6, 64, generator=gen(dev, 6), device=dev).to(BF16)
    k = torch.randn(4, 2, 64, generator=gen(dev, 7), device=dev).to(BF16)
    kc, vc, _, _ = make_cache(dev, 2, 16, 2, 64, BF16)
    pos = torch.arange(4, dtype=torch.int32, device=dev)
    freq = ref.frequencies(64).to(dev)
    slots = torch.arange(4, device=dev)
    want, err = ref.rope(q, pos, freq)
    got = w4.kv_append(k, k, kc, vc, slots, positions=pos, frequencies=freq, q=q, q_out=q)
    assert got.data_ptr() == q.data_ptr()
    near(q, want, err, BF16)
    before = kc.clone()
    got = w4.kv_append(k[:0], k[:0], kc, vc, slots[:0], positions=pos[:0], frequencies=freq, q=q[:0])
    assert got.shape == (0, 6, 64) and torch.equal(kc, before)


# ---- attn_decode ---------------------------------------------------------------------

def make_batch(dev, lens, Hq, Hkv, D, kind, page, layout="tokens", extra=2, seed=0, share=False):
    """q, caches, a table of shuffled pages (-1 behind a sequence's last) and lengths."""
    g = gen(dev, seed + len(lens) + D)
    need = [-(-max(n, 0) // page) for n in lens]
    most = max(need + [1]) + extra
    pages = sum(need) + 1
    kc, vc, ks, vs = make_cache(dev, pages, page, Hkv, D, kind, layout, seed)
    order = torch.randperm(pages, generator=g, device=dev).tolist()
    table = torch.full((len(lens), most), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    q = torch.randn(len(lens), Hq, D, generator=g, device=dev).to(BF16 if kind == "fp8" else kind)
    return dict(q=q, k_cache=kc, v_cache=vc, page_table=table.to(dev),
                seq_lens=torch.tensor(lens, dtype=torch.int32, device=dev), k_scales=ks, v_scales=vs)


def check_attn(d, got=None, **kw):
    args = {k: v for k, v in kw.items() if k in ("scale", "window")}
    want, err, lse, lse_err = ref.attn_decode(d["q"], d["k_cache"], d["v_cache"], d["page_table"], d["seq_lens"],
                                              d["k_scales"], d["v_scales"], **args)
    out, l = got if got is not None else w4.attn_decode(**d, return_lse=True, **kw)
    torch.cuda.synchronize()
    assert out.dtype == d["q"].dtype and out.shape == d["q"].shape and l.shape == lse.shape
    near(out, want, err, out.dtype)
    near(l, lse, lse_err, FP32)
    fine = torch.isfinite(want)
    print("attn", tuple(out.shape), d["k_cache"].dtype, "rel %.2e" % float(
        (out.double() - want)[fine].norm() / want[fine].norm().clamp_min(1e-300)), flush=True)


LENS = [1, 0, 33, 128, 7, 31, 32, 129, 500, 64, 255, 257]


@pytest.mark.parametrize("kind", [BF16, FP16, "fp8"])
@pytest.mark.parametrize("D", [128, 64, 256, 80, 8, 48, 96, 192, 112, 248])
@pytest.mark.parametrize("page, layout", [(16, "tokens"), (64, "heads"), (24, "joined"), (7, "tokens"), (1, "heads"), (100, "tokens")])
def test_attn_decode(dev, kind, D, page, layout):
    for Hq, Hkv in ((8, 2), (3, 3)):
        check_attn(make_batch(dev, LENS, Hq, Hkv, D, kind, page, layout))


@pytest.mark.parametrize("kind", [BF16, "fp8"])
@pytest.mark.parametrize("Hq, Hkv", [(1, 1), (64, 8), (16, 1), (17, 1), (40, 1), (48, 2), (7, 7), (128, 1), (35, 5)])
def test_attn_decode_heads(dev, kind, Hq, Hkv):
    check_attn(make_batch(dev, [300, 5, 0, 1000], Hq, Hkv, 128, kind, 16))


# heads of 64 side by side are taken two by two where there are enough of them
@pytest.mark.parametrize("kind", [BF16, FP16, "fp8"])
@pytest.mark.parametrize("page, layout", [(16, "tokens"), (64, "heads"), (24, "joined"), (5, "tokens")])
@pytest.mark.parametrize("group, Hkv", [(1, 8), (3, 4), (4, 8), (7, 6), (8, 4), (9, 4), (4, 5)])
@pytest.mark.parametrize("wide", [False, True])
def test_attn_decode_heads_of_64(dev, kind, page, layout, group, Hkv, wide):
    lens = LENS * (2 if wide else -(-512 // (Hkv * len(LENS))))
    d = make_batch(dev, lens, group * Hkv, Hkv, 64, kind, page, layout, extra=5000 // page if wide else 2)
    check_attn(d)
    check_attn(d, window=70)


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("page, start, gap", [(16, 8, 0), (5, 8, 0), (16, 0, 8), (16, 16, 16)])
def test_attn_decode_codes_of_8_aligned_bytes(dev, D, page, start, gap):
    """Codes that begin at, or whose tokens lie apart by, an odd multiple of 8 bytes."""
    d = make_batch(dev, LENS * 3, 8, 2, D, "fp8", page, extra=3000 // page)
    for name in ("k_cache", "v_cache"):
        pages = d[name].shape[0]
        buf = torch.zeros(start + pages * page * (2 * D + gap), dtype=d[name].dtype, device=dev)
        view = buf[start:].view(pages, page, 2 * D + gap)[:, :, :2 * D].unflatten(2, (2, D))
        view.copy_(d[name])
        d[name] = view
    check_attn(d)


@pytest.mark.parametrize("kind", [BF16, "fp8"])
@pytest.mark.parametrize("lens", [[700] * 70, [3000] * 5 + [9, 0, 4100]])
def test_attn_decode_heads_of_64_stay_apart(dev, kind, lens):
    """A NaN in one head's keys or values shows in its own query heads and nowhere else."""
    d = make_batch(dev, lens, 32, 8, 64, kind, 16)
    whole = w4.attn_decode(**d, return_lse=True)
    page = d["page_table"][0, 1].long()
    for name, kv in (("k_cache", 2), ("v_cache", 5)):
        at = d[name][page, 3, kv]
        at[7] = 0x7F if kind == "fp8" else float("nan")
    out, lse = w4.attn_decode(**d, return_lse=True)
    bad = torch.zeros(len(lens), 32, dtype=torch.bool, device=dev)
    bad[0, 8:12] = True
    assert torch.equal(torch.isnan(lse), bad)
    assert torch.isnan(out[0, 8:12]).all() and torch.isnan(out[0, 20:24, 7]).all()
    bad[0, 20:24] = True
    assert torch.equal(out[~bad], whole[0][~bad]) and torch.equal(lse[~bad], whole[1][~bad])


@pytest.mark.parametrize("kind", [BF16, FP16, "fp8"])
@pytest.mark.parametrize("window", [1, 5, 32, 100, 128, 129, 250, 100000])
def test_attn_decode_window(dev, kind, window):
    for page in (16, 5):
        check_attn(make_batch(dev, LENS + [1500], 8, 2, 64, kind, page), window=window)


@pytest.mark.parametrize("kind", [BF16, "fp8"])
@pytest.mark.parametrize("lens", [[20000], [1, 9000, 3, 0, 700], [4096] * 40, [0, 0, 0], list(range(0, 330)), [130] * 600,
                                  [0] * 500 + [5000] + [0] * 200])
def test_attn_decode_batches(dev, kind, lens):
    """Work cut over the workgroups: one long sequence, very unequal ones, many, none."""
    check_attn(make_batch(dev, lens, 8, 2, 64, kind, 64))


@pytest.mark.parametrize("kind", [BF16, FP16, "fp8"])
@pytest.mark.parametrize("D", [64, 128, 256, 72])
@pytest.mark.parametrize("page", [16, 5])
def test_attn_decode_short_sequences_in_wide_tables(dev, kind, D, page):
    """Tables for far more tokens than there are: what little there is, is cut."""
    for lens in (LENS, [1], [0, 0], [129] * 70, [5, 900, 1, 0, 0, 2000, 64]):
        check_attn(make_batch(dev, lens, 8, 2, D, kind, page, extra=3000))
        check_attn(make_batch(dev, lens, 8, 2, D, kind, page, extra=3000), window=70)


def test_attn_decode_many_sequences_most_of_them_empty(dev):
    """More sequences than the lanes of a wave, at the borders of 64 too, and long runs without a token."""
    lens = [0] * 6400
    for at, n in ((0, 3), (63, 300), (64, 1), (127, 128), (128, 129), (3000, 2000), (3001, 5), (6335, 40), (6399, 1000)):
        lens[at] = n
    check_attn(make_batch(dev, lens, 2, 1, 64, BF16, 64, extra=100))
    lens[6399] = lens[0] = 0
    check_attn(make_batch(dev, lens, 2, 1, 64, BF16, 64, extra=100), window=100)


def test_attn_decode_one_page_each(dev):
    """Tables that hold no more than one unit are not cut."""
    for page in (16, 64, 128, 9):
        check_attn(make_batch(dev, [min(page, n) for n in (0, 1, 16, 64, 9, 128, 100)], 8, 2, 128, BF16, page, extra=0))


@pytest.mark.parametrize("kind", [BF16, FP16, "fp8"])
@pytest.mark.parametrize("page", [16, 6])
def test_attn_decode_missing_pages_and_long_lengths(dev, kind, page):
    """Entries outside the cache hold nothing, whatever the length says."""
    d = make_batch(dev, [200, 64, 300, 90, 4], 8, 2, 64, kind, page)
    pages = d["k_cache"].shape[0]
    d["page_table"][0, 1] = -1
    d["page_table"][0, 3] = pages
    d["page_table"][1] = -7
    d["page_table"][2, ::2] = 2 ** 31 - 1
    d["page_table"][3, -1] = -2 ** 31
    d["seq_lens"][3] = 10 ** 6   # past the table
    d["seq_lens"][4] = -3
    check_attn(d)
    check_attn(d, window=150)


@pytest.mark.parametrize("kind", [BF16, FP16, "fp8"])
@pytest.mark.parametrize("page", [16, 6])
def test_attn_decode_reads_nothing_behind_a_sequence(dev, kind, page):
    """What lies in a page behind the last token, before the window, or in another page may be anything."""
    d = make_batch(dev, [37, 130, 1, 75], 8, 2, 64, kind, page)
    clean = {k: v.clone() if torch.is_tensor(v) else v for k, v in d.items()}
    for window in (0, 20):
        used = torch.zeros(d["k_cache"].shape[:2], dtype=torch.bool, device=dev)
        for b, n in enumerate(d["seq_lens"].tolist()):
            for j in range(max(0, n - window) if window else 0, n):
                used[d["page_table"][b, j // page], j % page] = True
        for name in ("k", "v"):
            c = d[name + "_cache"]
            c[~used] = 0x7F if kind == "fp8" else math.nan
            if kind == "fp8":
                s = d[name + "_scales"]
                s[~used[:, None].expand_as(s)] = math.nan
        check_attn(d, window=window)
        a, b = w4.attn_decode(**d, window=window, return_lse=True), w4.attn_decode(**clean, window=window, return_lse=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("kind", [BF16, FP16])
def test_attn_decode_special_values(dev, kind):
    d = make_batch(dev, [50, 50, 50, 50, 50, 300], 4, 2, 64, kind, 16)
    k = lambda b, j: d["k_cache"][d["page_table"][b, j // 16], j % 16]  # noqa: E731
    v = lambda b, j: d["v_cache"][d["page_table"][b, j // 16], j % 16]  # noqa: E731
    v(0, 7)[0, 3] = math.nan
    k(1, 20)[1, 5] = math.nan
    v(2, 9)[1, 6] = INF
    d["q"][3] = 0.0              # equal weights
    d["q"][4] *= 60.0            # scores in the hundreds
    k(5, 299)[:] *= 30.0         # the maximum comes last
    check_attn(d)
    check_attn(d, scale=-0.3)
    check_attn(d, scale=0.0)


def test_attn_decode_scores_far_below_zero(dev):
    """Scores of -10^6 and lower: the softmax does not see the offset."""
    d = make_batch(dev, [200, 3], 4, 1, 64, BF16, 16)
    d["k_cache"].copy_(d["k_cache"].abs() * 100)
    d["q"].copy_(-d["q"].abs() * 1000)
    check_attn(d)


def test_attn_decode_rising_scores(dev):
    """Each key beats all before it: the reference moves on at every tile."""
    d = make_batch(dev, [700], 8, 1, 64, BF16, 16)
    n = torch.arange(700, device=dev)
    d["k_cache"][d["page_table"][0, n // 16].long(), n % 16] = (n[:, None, None] / 64).to(BF16).expand(700, 1, 64)
    d["q"].copy_(d["q"].abs() + 0.5)
    check_attn(d)


def test_attn_decode_strides_outputs_and_workspace(dev):
    d = make_batch(dev, [70, 300, 1], 8, 2, 80, BF16, 16)
    wide = torch.randn(3, 12, 96, generator=gen(dev, 8), device=dev).to(BF16)
    wide[:, 2:10, :80] = d["q"]
    d["q"] = wide[:, 2:10, :80]
    big = torch.zeros(3, 2010, dtype=torch.int32, device=dev) - 1  # wide enough for a workspace
    big[:, :d["page_table"].shape[1]] = d["page_table"]
    d["page_table"] = big[:, :2000]
    need = w4.attn_decode_workspace_bytes(3, 8, 2, 80, d["page_table"].shape[1], 16)
    out = torch.full((3, 9, 80), 7.0, dtype=BF16, device=dev)
    lse = torch.empty(3, 8, device=dev)
    got = w4.attn_decode(**d, out=out[:, :8], lse=lse, workspace=torch.empty(need, dtype=torch.uint8, device=dev))
    assert got[0].data_ptr() == out.data_ptr() and got[1] is lse
    check_attn(d, got=got)
    assert bool((out[:, 8] == 7.0).all())
    assert w4.attn_decode(**d)[1] is None
    with pytest.raises(w4.W4A8Error, match="bytes"):
        w4.attn_decode(**d, workspace=torch.empty(need - 1, dtype=torch.uint8, device=dev))
    none = w4.attn_decode(d["q"][:0], d["k_cache"], d["v_cache"], d["page_table"][:0], d["seq_lens"][:0], return_lse=True)
    assert none[0].shape == (0, 8, 80) and none[1].shape == (0, 8)


@pytest.mark.parametrize("kind", [BF16, "fp8"])
def test_attn_decode_and_append_beyond_4_gib(dev, kind):
    """Pages whose offsets pass 32 bits, in bytes and in elements."""
    Hkv, D, page = 8, 128, 64
    pages = (1 << 33) // (page * Hkv * D * (1 if kind == "fp8" else 2)) // (2 if kind == "fp8" else 1) + 40
    dtype = torch.uint8 if kind == "fp8" else BF16
    kc = torch.zeros(pages, page, Hkv, D, dtype=dtype, device=dev)
    vc = torch.zeros(pages, page, Hkv, D, dtype=dtype, device=dev)
    ks = torch.ones(pages, Hkv, page, device=dev) if kind == "fp8" else None
    vs = torch.ones(pages, Hkv, page, device=dev) if kind == "fp8" else None
    n = 150
    table = torch.tensor([[pages - 1, 3, pages // 2 + 1]], dtype=torch.int32, device=dev)
    j = torch.arange(n, device=dev)
    slots = table[0, j // page].long() * page + j % page
    k, v = (torch.randn(n, Hkv, D, generator=gen(dev, s), device=dev).to(BF16) for s in (1, 2))
    w4.kv_append(k, v, kc, vc, slots, k_scales=ks, v_scales=vs)
    if kind != "fp8":
        assert torch.equal(kc.reshape(-1, Hkv, D)[slots], k) and torch.equal(vc.reshape(-1, Hkv, D)[slots], v)
    q = torch.randn(1, 16, D, generator=gen(dev, 3), device=dev).to(BF16)
    check_attn(dict(q=q, k_cache=kc, v_cache=vc, page_table=table, seq_lens=torch.tensor([n], dtype=torch.int32, device=dev),
                    k_scales=ks, v_scales=vs))


# ---- together ------------------------------------------------------------------------

class Attention:
    """The attention half of a block as a server runs it on a decode batch: norm
    to codes, the projection to heads, append, attention, the projection back."""

    def __init__(self, dev, B, H, Hq, Hkv, D, fp8, pages=40, page=16):
        g = gen(dev, 11)
        N = (Hq + 2 * Hkv) * D
        self.dims = Hq, Hkv, D
        self.norm = 1 + 0.1 * torch.randn(H, generator=g, device=dev)
        self.qkv = gemm_inputs(dev, 1, H, N, seed=1)[2:]
        self.back = gemm_inputs(dev, 1, Hq * D, H, seed=2)[2:]
        self.kc, self.vc, self.ks, self.vs = make_cache(dev, pages, page, Hkv, D, "fp8" if fp8 else BF16)
        self.freq = w4.rope_frequencies(D, device=dev)
        self.table = torch.randperm(pages, generator=g, device=dev).int()[:B * (pages // B)].reshape(B, -1).contiguous()
        self.lens = torch.zeros(B, dtype=torch.int32, device=dev)
        self.page = page

    def __call__(self, x):
        Hq, Hkv, D = self.dims
        o = {}
        pos = self.lens - 1
        o["pos"] = pos
        o["slots"] = self.table.gather(1, (pos // self.page).long()[:, None])[:, 0].long() * self.page + pos % self.page
        _, o["codes"], o["scales"] = w4.norm_residual(x, None, pre_weight=self.norm, quantize=True, keep_residual=False)
        o["heads"] = w4.gemm_fp8(o["codes"], o["scales"], *self.qkv).view(-1, Hq + 2 * Hkv, D)
        q, k, v = o["heads"].split((Hq, Hkv, Hkv), 1)
        o["q"] = w4.kv_append(k, v, self.kc, self.vc, o["slots"], k_scales=self.ks, v_scales=self.vs, positions=pos,
                              frequencies=self.freq, q=q)
        o["attn"], o["lse"] = w4.attn_decode(o["q"], self.kc, self.vc, self.table, self.lens, k_scales=self.ks,
                                             v_scales=self.vs, return_lse=True)
        o["out"] = w4.gemm_fp8(*w4.quantize_act(o["attn"].reshape(len(x), -1)), *self.back, residual=x)
        return o


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_chain(dev, fp8):
    """Several tokens of a batch, one step at a time, each step against the 64-bit forms of its parts."""
    B, H, Hq, Hkv, D = 4, 512, 8, 2, 128
    m = Attention(dev, B, H, Hq, Hkv, D, fp8)
    m.lens += torch.tensor([0, 14, 100, 31], dtype=torch.int32, device=dev)
    for step in range(4):
        m.lens += 1
        x = torch.randn(B, H, generator=gen(dev, step), device=dev).to(BF16)
        o = m(x)
        torch.cuda.synchronize()
        check_gemm((o["codes"], o["scales"], *m.qkv), got=o["heads"].reshape(B, -1))
        near(o["q"], *ref.rope(o["heads"][:, :Hq], o["pos"], m.freq), BF16)
        d = dict(q=o["q"], k_cache=m.kc, v_cache=m.vc, page_table=m.table, seq_lens=m.lens, k_scales=m.ks, v_scales=m.vs)
        check_attn(d, got=(o["attn"], o["lse"]))
        check_gemm((*w4.quantize_act(o["attn"].reshape(B, -1)), *m.back), got=o["out"], residual=x)


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_in_a_graph(dev, fp8):
    """Captured once and replayed for token after token, with eager work in between."""
    B, H, Hq, Hkv, D = 3, 256, 8, 2, 64
    m, eager = (Attention(dev, B, H, Hq, Hkv, D, fp8, pages=60) for _ in range(2))
    x = torch.zeros(B, H, dtype=BF16, device=dev)
    for a in (m, eager):
        a.lens.fill_(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m(x)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = m(x)
    eager(x.clone())
    for k in range(40):
        x.copy_(torch.randn(B, H, generator=gen(dev, 30 + k), device=dev))
        for a in (m, eager):
            a.lens += 1 if k % 7 else 20
        graph.replay()
        want = eager(x.clone())
        torch.cuda.synchronize()
        for name in ("codes", "heads", "q", "attn", "lse", "out"):
            assert torch.equal(o[name], want[name]), (k, name)
    assert torch.equal(m.kc, eager.kc) and torch.equal(m.vc, eager.vc)
    del graph


def test_attention_on_two_streams_at_once(dev):
    """Calls that overlap, each with its own cache and outputs."""
    sets = [make_batch(dev, [900, 40, 0, 3000], 8, 2, 128, BF16, 16, seed=k) for k in range(2)]
    gemms = [gemm_inputs(dev, 64, 2048, 512, seed=k) for k in range(2)]
    xs = [torch.randn(64, 72, 128, generator=gen(dev, k), device=dev).to(BF16) for k in range(2)]
    pos = torch.arange(64, dtype=torch.int32, device=dev)
    freq = ref.frequencies(128).to(dev)

    def calls(k):
        return (*w4.attn_decode(**sets[k], return_lse=True), w4.gemm_fp8(*gemms[k]), w4.rope(xs[k], pos, freq))

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
