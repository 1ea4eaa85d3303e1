"""Host-only checks of the operators around the expert forward: refusals of the
C ABI (no kernel is launched, the pointers are never followed) and of the
binding, and the plain 64-bit forms the GPU tests compare with."""
import ctypes
import math
import os
import random

import pytest
import torch

import block_refs as ref
from w4a8_moe_grouped_amd import lib as w4

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = ctypes.c_void_p(0x1000)
P2 = ctypes.c_void_p(0x2000)
ODD = ctypes.c_void_p(0x1004)


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(w4.LIB_PATH):
        from w4a8_moe_grouped_amd import build
        build.build()
    return w4.load()


def _route(L, logits=P, kind=0, T=0, E=64, ld=64, bias=None, score=0, groups=1, kept=1, top=2, k=8,
           num=None, ids=P, wts=P):
    return L.w4a8_moe_route(logits, kind, T, E, ld, bias, score, groups, kept, top, k, 1, 1.0, num, ids, wts, None)


@pytest.mark.parametrize("change, want", [
    (dict(), OK), (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(ld=63), INVALID), (dict(k=0), INVALID),
    (dict(kind=3), INVALID), (dict(score=2), INVALID), (dict(top=0), INVALID), (dict(top=3), INVALID),
    (dict(groups=0), INVALID), (dict(groups=3), INVALID), (dict(groups=8, kept=0), INVALID),
    (dict(groups=8, kept=9), INVALID), (dict(groups=8, kept=1, k=9), INVALID), (dict(k=33), UNSUPPORTED),
    (dict(E=8, ld=8, k=9), INVALID), (dict(E=1025, ld=1025), UNSUPPORTED), (dict(E=130, ld=130, groups=65, kept=65), UNSUPPORTED),
    (dict(T=4, logits=None), INVALID), (dict(T=4, ids=None), INVALID), (dict(T=4, wts=None), INVALID),
    (dict(T=4, logits=ODD), UNSUPPORTED), (dict(T=4, bias=ODD), UNSUPPORTED), (dict(T=4, ids=ODD), UNSUPPORTED),
    (dict(T=4, num=ctypes.c_void_p(0x1002)), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED),
])
def test_route_arguments(L, change, want):
    assert _route(L, **change) == want


def _norm(L, x=P, xt=1, ldx=256, r=P2, rt=1, ldr=256, T=0, H=256, pt=1, post=None, gate=None, grs=0, gcs=0,
          pre=P, eps=1e-6, ro=P2, ldo=256, y=P, ldy=256, q=None, qs=None):
    return L.w4a8_norm_residual(x, xt, ldx, r, rt, ldr, T, H, pt, post, gate, grs, gcs, 1.0, pre, 0.0, eps, ro, ldo,
                                y, ldy, q, qs, None)


@pytest.mark.parametrize("change, want", [
    (dict(), OK), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(eps=0.0), INVALID), (dict(eps=math.nan), INVALID), (dict(eps=1e-40), INVALID),
    (dict(xt=2), INVALID), (dict(rt=3), INVALID), (dict(pt=2), INVALID), (dict(q=P), INVALID), (dict(qs=P), INVALID),
    (dict(ldx=255), INVALID), (dict(ldr=255), INVALID), (dict(ldo=255), INVALID), (dict(ldy=255), INVALID),
    (dict(gate=P, gcs=2), INVALID), (dict(gate=P, gcs=1, grs=255), INVALID), (dict(gate=P, grs=-1), INVALID),
    (dict(T=4, x=None, r=None), INVALID), (dict(T=4, x=None, post=P), INVALID), (dict(T=4, x=None, gate=P), INVALID),
    (dict(T=4, pre=None), INVALID), (dict(T=4, y=None), INVALID), (dict(T=4, pre=None, y=None, ro=None), INVALID),
    (dict(ldo=264), INVALID),  # in place with another stride
    (dict(H=32776, ldx=32776, ldr=32776, ldo=32776, ldy=32776), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED),
    (dict(H=200, q=P, qs=P), UNSUPPORTED), (dict(T=4, x=ODD), UNSUPPORTED), (dict(T=4, r=ODD, ro=P), UNSUPPORTED),
    (dict(T=4, y=ODD), UNSUPPORTED), (dict(T=4, pre=ODD), UNSUPPORTED), (dict(T=4, gate=ODD), UNSUPPORTED),
    (dict(T=4, q=ODD, qs=P), UNSUPPORTED),
])
def test_norm_arguments(L, change, want):
    assert _norm(L, **change) == want


@pytest.mark.parametrize("T, H, want", [(1 << 22, 520, UNSUPPORTED), ((1 << 25) + 1, 512, UNSUPPORTED)])
def test_norm_rows_of_one_launch(L, T, H, want):
    """A launch holds less than 2^32 threads."""
    assert _norm(L, T=T, H=H, ldx=H, ldr=H, ldo=H, ldy=H) == want


def test_route_tokens_of_one_launch(L):
    assert _route(L, T=(1 << 25) + 1) == UNSUPPORTED


def _gemm(L, a=P, sa=P, M=0, K=256, b=P, sb=P, N=64, bias=None, bt=0, act=0, res=None, ldr=64, out=P2, ldo=64, ws=P,
          nbytes=1 << 50):
    n = ctypes.c_size_t(nbytes)
    return L.w4a8_gemm_epilogue(a, sa, M, K, b, sb, N, bias, bt, act, res, ldr, out, ldo, ws, ctypes.byref(n), None)


@pytest.mark.parametrize("change, want", [
    (dict(), OK), (dict(M=-1), INVALID), (dict(K=0), INVALID), (dict(N=0), INVALID), (dict(act=6), INVALID),
    (dict(act=-1), INVALID), (dict(K=200), UNSUPPORTED), (dict(K=(1 << 22) + 128), UNSUPPORTED),
    (dict(M=1 << 31), UNSUPPORTED), (dict(N=1 << 31), UNSUPPORTED), (dict(N=1 << 30, act=5), UNSUPPORTED),
    (dict(M=1 << 30, N=1 << 11, ldo=1 << 11), UNSUPPORTED),
    (dict(M=4, a=None), INVALID), (dict(M=4, sa=None), INVALID), (dict(b=None), INVALID), (dict(sb=None), INVALID),
    (dict(M=4, out=None), INVALID), (dict(ldo=63), INVALID), (dict(res=P, ldr=63), INVALID),
    (dict(bias=P, bt=2), INVALID), (dict(res=P2, ldr=72), INVALID), (dict(M=4, a=ODD), UNSUPPORTED),
    (dict(sa=ODD), UNSUPPORTED), (dict(b=ODD), UNSUPPORTED), (dict(sb=ODD), UNSUPPORTED), (dict(bias=ODD), UNSUPPORTED),
    (dict(res=ODD), UNSUPPORTED), (dict(out=ODD), UNSUPPORTED), (dict(ws=ODD), UNSUPPORTED),
])
def test_gemm_epilogue_arguments(L, change, want):
    assert _gemm(L, **change) == want


def test_gemm_epilogue_workspace(L):
    for M, K, N, act in ((1, 7168, 2048, "swiglu"), (4096, 7168, 2048, "swiglu"), (4096, 2048, 7168, "none")):
        need = w4.gemm_epilogue_workspace_bytes(M, K, N, act)
        assert need >= 0 and need == w4.gemm_epilogue_workspace_bytes(M, K, N, act)
        if need:
            assert _gemm(L, M=M, K=K, N=N, act=w4.ACTIVATIONS[act], ldo=N, nbytes=need - 1) == WORKSPACE


def test_binding_refuses():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(w4.W4A8Error):
        w4.moe_route(x, 2)
    with pytest.raises(w4.W4A8Error):
        w4.norm_residual(x, x)
    with pytest.raises(w4.W4A8Error):
        w4.norm_residual(None, None)
    with pytest.raises(w4.W4A8Error):
        w4.gemm_epilogue(x.view(torch.uint8), x, x, x)


# ---- the plain forms ----------------------------------------------------------------

def test_ref_route_small_by_hand():
    x = torch.tensor([[1.0, 3.0, 3.0, -1.0], [0.0, -math.inf, math.nan, 2.0], [-math.inf] * 4])
    ids, w = ref.route(x, 3, "softmax")
    e = [math.exp(v) for v in (1.0, 3.0, 3.0)]
    assert ids[0] == [1, 2, 0] and w[0] == pytest.approx([e[1] / sum(e), e[2] / sum(e), e[0] / sum(e)], rel=1e-14)
    assert ids[1] == [3, 0, -1] and w[1] == pytest.approx([1 / (1 + math.exp(-2)), 1 / (1 + math.exp(2)), 0], rel=1e-14)
    assert ids[2] == [-1, -1, -1] and w[2] == [0, 0, 0]
    ids, w = ref.route(x[:1], 1, "sigmoid", torch.tensor([0.0, 0.0, 0.0, 5.0]), renormalize=False, scale=2.0)
    assert ids == [[3]] and w[0][0] == pytest.approx(2 / (1 + math.exp(1)), rel=1e-14)
    # two groups of two: the first has the larger sum; by the best alone they tie, and the first wins
    assert ref.route(x[:1], 2, "softmax", num_groups=2, topk_groups=1)[0] == [[1, 0]]
    assert ref.route(x[:1], 2, "softmax", num_groups=2, topk_groups=1, group_top=1)[0] == [[1, 0]]
    assert ref.route(x[:1], 2, num_tokens=0)[0] == [[-1, -1]]


def test_ref_norm_is_torch_rms_norm():
    g = torch.Generator().manual_seed(0)
    x, r = torch.randn(3, 40, generator=g), torch.randn(3, 40, generator=g)
    w = torch.randn(40, generator=g)
    n = torch.nn.functional.rms_norm
    out, y, _ = ref.norm_residual(x, r, post_weight=w, residual_scale=0.5, pre_weight=w, eps=1e-5)
    want = 0.5 * r.double() + n(x.double(), (40,), w.double(), 1e-5)
    torch.testing.assert_close(out, want, rtol=1e-13, atol=1e-13)
    torch.testing.assert_close(y, n(want, (40,), w.double(), 1e-5), rtol=1e-13, atol=1e-13)


def test_ref_gemm_is_the_oracle(orc):
    import numpy as np
    rng = np.random.default_rng(3)
    codes = rng.integers(0, 0x78, (5, 256)).astype(np.uint8)
    sa = rng.random((5, 2)).astype(np.float32)
    w = rng.integers(0, 256, (24, 128)).astype(np.uint8)
    sw = rng.random((24, 2)).astype(np.float32)
    t = torch.from_numpy
    got, _ = ref.gemm_epilogue(t(codes), t(sa), t(w), t(sw))
    np.testing.assert_allclose(got.numpy(), orc.gemm_f64(codes, sa, w, sw), rtol=1e-12, atol=1e-9)


@pytest.mark.parametrize("M, K, N, act, want", [
    # 128 x 128 tiles of 256 threads: 8192 x 257
    (1 << 20, 128, 1 << 13, 5, OK), (1 << 20, 128, (1 << 14) + 32, 5, OK),
    # 512 threads for 32 weight rows; 256 threads for 32 rows x 64 weight rows
    (16, 128, (1 << 28) + 32, 0, UNSUPPORTED), (17, 128, (1 << 30) + 64, 0, UNSUPPORTED), (17, 128, 1 << 29, 0, OK),
    # the first pass: 256 threads for 8192 weights
    (1 << 13, 4096, 1 << 13, 0, OK), (1 << 17, 1 << 20, 1 << 18, 0, UNSUPPORTED)])
def test_gemm_epilogue_threads_of_one_launch(L, M, K, N, act, want):
    """Both kernels' launches hold less than 2^32 threads; the query says so."""
    assert _gemm(L, M=M, K=K, N=N, act=act, ldo=N, ws=None) == want


def test_gemm_epilogue_without_workspace_bytes(L):
    """0 bytes are enough where the query says so, at an address that is not null."""
    assert w4.gemm_epilogue_workspace_bytes(64, 2048, 7168) == 0
    assert _gemm(L, K=2048, N=7168, ldo=7168, nbytes=0) == OK
    assert _gemm(L, M=4, a=None, nbytes=0) == INVALID  # not taken for a query
    assert _gemm(L, M=4, a=None, ws=None, nbytes=0) == OK


@pytest.mark.parametrize("M, K, N, act, want", [
    # 32 rows of one weight row take as many threads as of 64
    (1 << 29, 128, 1, 0, UNSUPPORTED), (1 << 29, 128, 16, 0, UNSUPPORTED), ((1 << 29) - 32, 128, 64, 0, OK),
    (16, 128, (1 << 28) - 32, 0, OK)])
def test_gemm_epilogue_threads_of_narrow_weights(L, M, K, N, act, want):
    assert _gemm(L, M=M, K=K, N=N, act=act, ldo=N, ws=None) == want


def test_gemm_epilogue_sizes_that_always_fit(L):
    """The sizes that include/w4a8.h promises, at random over the whole range."""
    rng = random.Random(5)
    up = lambda a, b: -(-a // b)  # noqa: E731
    checked = 0
    for _ in range(20000):
        act = rng.choice([0, 5])
        M, N, G = (int(2 ** rng.uniform(0, top)) for top in (30.9, 29.9 if act else 30.9, 15))
        R, K = (2 * N if act else N), 128 * G
        if R <= 2 ** 28 - 32 and up(M, 32) * up(R, 64) < 2 ** 24 and up(R, 128) * up(K, 256) <= 2 ** 21 \
                and up(M, 128) * up(K, 1024) <= 2 ** 22:
            checked += 1
            assert _gemm(L, M=M, K=K, N=N, act=act, ldo=N, ws=None) == OK, (M, K, N, act)
    assert checked > 1000
