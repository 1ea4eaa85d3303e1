"""The bounds of attn_sharp.py on the CPU: a weight's two parts meet them, and
what they are there to see does not: one part alone, or parts that are raised."""
import pytest
import torch

import attn_sharp

BF16, FP16 = torch.bfloat16, torch.float16


def cut(w, dtype):
    """w (fp32, not negative) cut to the type."""
    if dtype == BF16:
        return (w.view(torch.int32) & -65536).view(torch.float32)
    h = w.half()
    return torch.where(h.float() > w, torch.nextafter(h, torch.zeros_like(h)), h).float()


def emulated(q, k, v, scale, shift, parts, raised=0.0):
    """One sequence and kv head with weights in 32 bits held times 2^shift, as parts of q's type."""
    s = (q.double() @ k.double().T * scale * 1.4426950408889634).float()
    w = torch.exp2((s - s.amax(-1, keepdim=True) + shift).double()).float()
    hi = cut(w, q.dtype)
    lo = (w - hi).to(q.dtype).float().clamp_min(raised)
    total = hi.double() + (lo.double() if parts == 2 else 0.0)
    return ((total @ v.double()) / w.double().sum(-1, keepdim=True)).to(q.dtype)


def batch(dtype, n, positive, D=64, seed=0):
    """Queries of eight elements that are not zero, and few keys: there the bounds on scores and sums
    are well below what a lost part costs."""
    g = torch.Generator().manual_seed(seed)
    q, k, v = torch.randn(8, D, generator=g), torch.randn(n, D, generator=g), torch.randn(n, D, generator=g)
    q[:, 8:] = 0
    return q.to(dtype), k.to(dtype), (v.abs() + 0.5 if positive else v).to(dtype)


def misses(got, q, k, v, scale):
    n = k.shape[0]
    table = torch.zeros(1, 1, dtype=torch.int32)
    want, err = attn_sharp.attention(q[None], k[None, :, None], v[None, :, None], table, torch.tensor([n]), scale=scale)
    return attn_sharp.outside(got[None], want, err)


@pytest.mark.parametrize("dtype, shift", [(BF16, 0), (FP16, 14)])
@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("n", [33, 128])
def test_two_parts_are_within_and_one_is_not(dtype, shift, positive, n):
    q, k, v = batch(dtype, n, positive)
    assert misses(emulated(q, k, v, 0.125, shift, 2), q, k, v, 0.125) == 0
    one = misses(emulated(q, k, v, 0.125, shift, 1), q, k, v, 0.125)
    assert one > 100, one


def test_parts_raised_for_every_key_are_seen():
    """Small weights under a peak whose value is 0: 2^-31 more for every key is far outside."""
    q, k, v = batch(FP16, 4096, True)
    q.zero_()
    q[:, 0] = 8.0
    k[:, 0] /= 8
    k[1000, 0] = 20 / 8
    v *= 1000
    v[1000] = 0
    assert misses(emulated(q, k, v, 1.0, 14, 2), q, k, v, 1.0) == 0
    assert misses(emulated(q, k, v, 1.0, 7, 2, raised=2.0 ** -24), q, k, v, 1.0) > 400
