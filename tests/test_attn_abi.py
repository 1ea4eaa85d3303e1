"""The C ABI and the binding of the attention half of a block on the CPU:
refusals, queries and the plain forms the GPU tests compare with."""
import ctypes
import math

import pytest
import torch

import attn_refs as ref
from w4a8_moe_grouped_amd import lib as w4

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
A = ctypes.c_void_p(0x10000)  # aligned addresses that are never followed
B = ctypes.c_void_p(0x20000)
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(w4.LIB_PATH):
        from w4a8_moe_grouped_amd import build
        build.build()
    return w4.load()


def _gemm(L, M=0, K=256, N=64, act=0, a=A, w=A, sw=A, bias=None, btype=0, res=None, ldr=None, out=B, ldo=None, ws=A,
          nbytes=0):
    n = ctypes.c_size_t(nbytes)
    return L.w4a8_gemm_fp8(a, A, M, K, w, sw, N, bias, btype, act, res, ldr or N, out, ldo or N, ws, ctypes.byref(n), None)


def test_gemm_fp8_refusals(L):
    assert _gemm(L) == OK  # M = 0
    for kw in (dict(M=-1), dict(K=0), dict(N=0), dict(act=6), dict(act=-1), dict(w=None), dict(sw=None), dict(ldo=63),
               dict(M=1, a=None), dict(M=1, out=None), dict(res=A, ldr=63), dict(bias=A, btype=2),
               dict(res=B, ldr=70, ldo=64)):
        assert _gemm(L, **kw) == INVALID, kw
    for kw in (dict(K=130), dict(K=1 << 23), dict(M=1 << 31), dict(N=1 << 31), dict(act=5, N=64), dict(w=ODD), dict(a=ODD),
               dict(out=ODD), dict(ws=ODD), dict(res=ODD), dict(bias=ODD), dict(M=1 << 30, N=1 << 30),
               dict(N=(1 << 31) - 128, K=1 << 22), dict(M=(1 << 31) - 1, K=128, N=1 << 20)):
        assert _gemm(L, **kw) == UNSUPPORTED, kw
    assert _gemm(L, M=1, ws=None) == OK  # a query
    assert w4.gemm_fp8_workspace_bytes(4096, 7168, 2048, "swiglu") >= 0


def test_gemm_fp8_sizes_that_always_fit(L):
    """The sizes that include/w4a8.h promises, at random over the whole range."""
    import random
    rng = random.Random(5)
    up = lambda a, b: -(-a // b)  # noqa: E731
    checked = 0
    for _ in range(20000):
        act = rng.choice([0, 5])
        M, N, G = (int(2 ** rng.uniform(0, top)) for top in (30.9, 29.9 if act else 30.9, 15))
        N = up(N, 128) * 128 if act else N
        R = 2 * N if act else N
        if up(M, 16) * up(R, 32) < 2 ** 23 - 8 and up(R, 128) * G * 4 < 2 ** 32:
            checked += 1
            assert _gemm(L, M=M, K=128 * G, N=N, act=act, ws=None) == OK, (M, N, G, act)
    assert checked > 1000


def test_rope_frequencies_refusals(L):
    def f(R=64, base=1e4, kind=0, factor=2.0, length=4096.0, fast=32.0, slow=1.0, out=None):
        return L.w4a8_rope_frequencies(R, base, kind, factor, length, fast, slow, out, None)
    for kw in (dict(), dict(R=0, out=A), dict(R=3, out=A), dict(R=258, out=A), dict(base=1.0, out=A),
               dict(base=math.inf, out=A), dict(base=math.nan, out=A), dict(kind=4, out=A), dict(kind=-1, out=A),
               dict(kind=1, factor=0.0, out=A), dict(kind=1, factor=math.inf, out=A), dict(kind=2, R=2, out=A),
               dict(kind=3, length=0.0, out=A), dict(kind=3, fast=0.5, out=A), dict(kind=3, slow=0.0, out=A),
               dict(kind=3, fast=math.inf, out=A)):
        assert f(**kw) == INVALID, kw
    assert f(out=ctypes.c_void_p(0x10004)) == UNSUPPORTED


def _rope(L, x=A, type=1, T=0, H=4, D=64, xs=(256, 64), pos=A, freq=A, R=64, out=B, os=(256, 64)):
    return L.w4a8_rope(x, type, T, H, D, *xs, pos, freq, R, 0, 1.0, out, *os, None)


def test_rope_refusals(L):
    assert _rope(L) == OK and _rope(L, T=3, H=0) == OK
    for kw in (dict(T=-1), dict(H=-1), dict(D=0), dict(type=3), dict(type=-1), dict(R=-2), dict(R=66), dict(R=3),
               dict(T=1, x=None), dict(T=1, out=None), dict(T=1, pos=None), dict(T=1, freq=None),
               dict(T=1, out=A, os=(512, 64)), dict(T=1, out=A, os=(256, 72)), dict(T=2, os=(0, 64)), dict(T=1, os=(256, 0))):
        assert _rope(L, **kw) == INVALID, kw
    for kw in (dict(D=60, R=2), dict(D=264, R=2), dict(T=1, x=ODD), dict(T=1, out=ODD), dict(xs=(-8, 64)), dict(xs=(256, 4)),
               dict(os=(256, 63)), dict(os=(-256, 64)), dict(T=(1 << 25) + 1), dict(H=4097), dict(pos=ctypes.c_void_p(0x10002)),
               dict(freq=ctypes.c_void_p(0x10004)), dict(T=1 << 25, H=4096)):
        assert _rope(L, **kw) == UNSUPPORTED, kw


def _cache(**kw):
    c = dict(k=0x10000, v=0x20000, k_scales=None, v_scales=None, type=1, num_pages=4, page_size=16, kv_heads=2, head_dim=64,
             k_page_stride=2048, k_token_stride=128, k_head_stride=64, v_page_stride=2048, v_token_stride=128, v_head_stride=64)
    c.update(kw)
    return w4.KVCache(**c)


BAD_CACHES = [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(num_pages=0), INVALID), (dict(page_size=0), INVALID),
              (dict(kv_heads=0), INVALID), (dict(head_dim=0), INVALID), (dict(type=0), INVALID), (dict(type=4), INVALID),
              (dict(type=3), INVALID), (dict(k_scales=0x10000), INVALID), (dict(type=3, k_scales=0x10000), INVALID),
              (dict(head_dim=60), UNSUPPORTED), (dict(head_dim=264), UNSUPPORTED), (dict(k=0x10008), UNSUPPORTED),
              (dict(v=0x10002), UNSUPPORTED), (dict(k_page_stride=-8), UNSUPPORTED), (dict(v_token_stride=4), UNSUPPORTED),
              (dict(v_head_stride=1 << 50), UNSUPPORTED), (dict(num_pages=1 << 31), UNSUPPORTED),
              (dict(kv_heads=4097), UNSUPPORTED), (dict(num_pages=1 << 30, page_size=1 << 12), UNSUPPORTED),
              (dict(type=3, k_scales=0x10000, v_scales=0x10008), UNSUPPORTED),
              (dict(type=3, k=0x10004, k_scales=0x10000, v_scales=0x10000), UNSUPPORTED)]


def _append(L, cache=None, q=A, qs=(256, 64), Hq=4, k=A, v=A, ks=(128, 64), type=1, T=0, slots=A, pos=A, freq=A, R=64, qo=B,
            qos=(256, 64)):
    c = _cache() if cache is None else cache
    return L.w4a8_kv_append(q, *qs, Hq, k, *ks, v, *ks, type, T, slots, pos, freq, R, 0, 1.0, ctypes.byref(c), qo, *qos, None)


def test_kv_append_refusals(L):
    assert _append(L) == OK
    assert L.w4a8_kv_append(A, 256, 64, 4, A, 128, 64, A, 128, 64, 1, 0, A, A, A, 64, 0, 1.0, None, B, 256, 64, None) == INVALID
    for kw, want in BAD_CACHES:
        assert _append(L, cache=_cache(**kw)) == want, kw
    for kw in (dict(T=-1), dict(Hq=-1), dict(type=0), dict(type=2), dict(type=3), dict(q=None), dict(qo=None), dict(T=1, k=None),
               dict(T=1, v=None), dict(T=1, slots=None), dict(T=1, q=None, qo=None), dict(T=1, pos=None), dict(T=1, freq=None),
               dict(R=66), dict(R=1), dict(qo=A, qos=(512, 64)), dict(T=2, qos=(0, 64)), dict(T=1, qos=(256, 0))):
        assert _append(L, **kw) == INVALID, kw
    for name in ("k_page", "k_token", "k_head", "v_page", "v_token", "v_head"):  # rows that are written lie apart
        assert _append(L, cache=_cache(**{name + "_stride": 0})) == INVALID, name
    for kw in (dict(T=1 << 26), dict(Hq=4093), dict(qs=(4, 64)), dict(ks=(-8, 64)), dict(qos=(256, 1)), dict(k=ODD), dict(v=ODD),
               dict(q=ODD), dict(qo=ODD), dict(slots=ctypes.c_void_p(0x10004))):
        assert _append(L, **kw) == UNSUPPORTED, kw


def _attn(L, cache=None, q=A, type=1, n=0, Hq=8, qs=(512, 64), table=A, pages=4, ld=4, lens=A, window=0, out=B, os=(512, 64),
          lse=None, ws=A, nbytes=1 << 40):
    c = _cache() if cache is None else cache
    b = ctypes.c_size_t(nbytes)
    return L.w4a8_attn_decode(q, type, n, Hq, *qs, ctypes.byref(c), table, pages, ld, lens, 1.0, window, out, *os, lse, ws,
                              ctypes.byref(b), None)


def test_attn_decode_refusals(L):
    assert _attn(L) == OK
    for kw, want in BAD_CACHES:
        if kw not in (dict(num_pages=1 << 30, page_size=1 << 12), dict(kv_heads=4097)):
            assert _attn(L, cache=_cache(**kw)) == want, kw
    assert _attn(L, cache=_cache(kv_heads=4097), Hq=4097) == UNSUPPORTED
    for kw in (dict(n=-1), dict(Hq=0), dict(Hq=3), dict(pages=0), dict(type=0), dict(type=2), dict(type=3), dict(window=-1),
               dict(ld=3), dict(n=1, q=None), dict(n=1, out=None), dict(n=1, table=None), dict(n=1, lens=None), dict(n=1, out=A)):
        assert _attn(L, **kw) == INVALID, kw
    for kw in (dict(n=65537), dict(Hq=8192), dict(pages=1 << 27, ld=1 << 27), dict(q=ODD), dict(out=ODD), dict(qs=(4, 64)),
               dict(os=(512, -64)), dict(table=ctypes.c_void_p(0x10002)), dict(lens=ctypes.c_void_p(0x10001)),
               dict(lse=ctypes.c_void_p(0x10002)), dict(ws=ODD)):
        assert _attn(L, **kw) == UNSUPPORTED, kw
    assert _attn(L, n=2, os=(0, 64)) == INVALID and _attn(L, n=1, os=(512, 0)) == INVALID
    assert _attn(L, n=65536, cache=_cache(kv_heads=65), Hq=65, ws=None) == UNSUPPORTED  # workgroups of one launch
    assert _attn(L, n=65536, cache=_cache(kv_heads=64), Hq=1024, ws=None) == OK
    assert _attn(L, n=65536, cache=_cache(kv_heads=64), Hq=1088, ws=None) == UNSUPPORTED
    assert _attn(L, cache=_cache(k_head_stride=0, v_token_stride=0)) == OK  # read only: any strides
    assert _attn(L, cache=_cache(type=3, k_scales=0x10000, v_scales=0x10000)) == OK  # bf16 queries of codes
    assert _attn(L, cache=_cache(type=3, k_scales=0x10000, v_scales=0x10000), type=2) == INVALID


def test_attn_decode_workspace(L):
    assert w4.attn_decode_workspace_bytes(4, 8, 2, 64, 8, 16) == 0  # one unit of keys: nothing is cut
    n = w4.attn_decode_workspace_bytes(4, 8, 2, 64, 100, 16)
    assert n > 0 and _attn(L, n=4, pages=100, ld=100, nbytes=n - 1) == WORKSPACE
    assert w4.attn_decode_workspace_bytes(4, 8, 2, 64, 1 << 26, 16) == n  # whatever the length


def test_binding_refuses_on_the_cpu(L):
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    cache = torch.zeros(2, 16, 4, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    f = torch.zeros(32, dtype=torch.float64)
    for call in (lambda: w4.rope(x, i, f), lambda: w4.kv_append(x, x, cache, cache, i.long()),
                 lambda: w4.attn_decode(x, cache, cache, i[:, None], i),
                 lambda: w4.gemm_fp8(x, x, x, x), lambda: w4.gemm_fp8(None, x, x, x),
                 lambda: w4.gemm_fp8(x, x, x, x, activation="tanh"), lambda: w4.rope_frequencies(64, scaling="cubic"),
                 lambda: w4.rope_frequencies(64, device="cpu"), lambda: w4.rope("x", i, f)):
        with pytest.raises(w4.W4A8Error):
            call()


# ---- the plain forms ----------------------------------------------------------------

def test_ref_rope_turns_by_hand():
    x = torch.tensor([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    f = torch.tensor([math.pi / 2, math.pi])
    pos = torch.tensor([1], dtype=torch.int32)
    y, _ = ref.rope(x, pos, f)
    torch.testing.assert_close(y, torch.tensor([[[-3.0, -2.0, 1.0, -4.0, 5.0]]], dtype=torch.float64), rtol=1e-6, atol=1e-6)
    y, _ = ref.rope(x, pos, f, interleaved=True, magnitude=2.0)
    torch.testing.assert_close(y, torch.tensor([[[-4.0, 2.0, -6.0, -8.0, 5.0]]], dtype=torch.float64), rtol=1e-6, atol=1e-6)


def test_ref_frequencies():
    plain = ref.frequencies(8)
    torch.testing.assert_close(plain, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64))
    torch.testing.assert_close(ref.frequencies(8, scaling="linear", factor=4.0), plain / 4)
    y = ref.frequencies(128, scaling="yarn", factor=16.0, original_length=4096.0)
    f = ref.frequencies(128)
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(y[turns > 40], f[turns > 40])          # fast pairs stay
    torch.testing.assert_close(y[turns < 0.8], f[turns < 0.8] / 16)  # slow ones are interpolated
    assert bool((y[1:] < y[:-1]).all())


def test_ref_attention_is_torch():
    g = torch.Generator().manual_seed(0)
    kc, vc = torch.randn(5, 4, 2, 8, generator=g), torch.randn(5, 4, 2, 8, generator=g)
    q = torch.randn(2, 6, 8, generator=g)
    table = torch.tensor([[3, 0, -1], [1, 4, 2]], dtype=torch.int32)
    out, _, lse, _ = ref.attn_decode(q, kc, vc, table, torch.tensor([7, 12]))
    for b, pages, n in ((0, [3, 0], 7), (1, [1, 4, 2], 12)):
        k, v = (c[pages].reshape(-1, 2, 8)[:n].double().permute(1, 0, 2) for c in (kc, vc))
        want = torch.nn.functional.scaled_dot_product_attention(
            q[b].double().reshape(2, 3, 8), k, v).reshape(6, 8)
        torch.testing.assert_close(out[b], want, rtol=1e-12, atol=1e-12)
    out, _, lse, _ = ref.attn_decode(q, kc, vc, table, torch.tensor([0, 1]))
    assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all())
    torch.testing.assert_close(out[1], vc[1, 0].double().repeat_interleave(3, 0))


def test_sine_and_cosine_series():
    """The series of the kernel, in fp32, over an eighth of a turn each way: within the promised 2e-7."""
    import numpy as np
    f = np.float32
    x = np.linspace(-math.pi / 4, math.pi / 4, 200001)
    v = x.astype(f)
    z = v * v
    s = z * f(1 / 362880) + f(-1 / 5040)
    for c in (1 / 120, -1 / 6):
        s = z * s + f(c)
    s = z * v * s + v
    c = z * f(-1 / 3628800) + f(1 / 40320)
    for k in (-1 / 720, 1 / 24, -0.5, 1.0):
        c = z * c + f(k)
    assert np.abs(s - np.sin(x)).max() < 2e-7 and np.abs(c - np.cos(x)).max() < 2e-7
