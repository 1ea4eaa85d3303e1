"""Rotation at far positions against 80-bit angles: sine and cosine are good to
the promised 2e-7 wherever a position lies."""
import numpy as np
import pytest
import torch

from attn_refs import TURN, U
from test_gpu_attn import BF16, dev, gen  # noqa: F401
from w4a8_moe_grouped_amd import lib as w4

pytestmark = pytest.mark.gpu

# 64 bits of mantissa: a product below 2^36 is off by 2^-28 of a turn at most, 4e-9
assert np.finfo(np.longdouble).nmant >= 63


def turned(positions, freq):
    """cos and sin of positions * freq in 64 bits."""
    angle = np.multiply.outer(positions.cpu().numpy().astype(np.longdouble), freq.cpu().numpy().astype(np.longdouble))
    return (torch.from_numpy(f(angle).astype(np.float64)).to(positions.device) for f in (np.cos, np.sin))


def far_positions(dev, n, lowest):  # noqa: F811
    g = gen(dev, lowest)
    p = torch.randint(2 ** lowest, 2 ** 31 - 1, (n,), generator=g, device=dev, dtype=torch.int64)
    p[::2] = -p[::2]
    p[:4] = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 30, -2 ** 30 - 1], device=dev)
    return p.int()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("lowest", [1, 24, 30])
@pytest.mark.parametrize("freq", ["plain", "all", "far"])
def test_sine_and_cosine_at_far_positions(dev, interleaved, lowest, freq):  # noqa: F811
    g = gen(dev, 5)
    pairs = 64
    if freq == "plain":
        f = w4.rope_frequencies(2 * pairs, device=dev)
    else:  # up to a turn a position, and beyond
        f = torch.rand(pairs, generator=g, device=dev, dtype=torch.float64) * (2 * np.pi if freq == "all" else 30.0)
        f[0], f[1] = 1.0, -np.pi
    pos = far_positions(dev, 2000, lowest)
    x = torch.zeros(len(pos), 2, 2 * pairs, device=dev)
    first, second = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, pairs), slice(pairs, None))
    x[:, 0, first] = 1.0   # (1, 0) turns to (cos, sin), (0, 1) to (-sin, cos)
    x[:, 1, second] = 1.0
    out = w4.rope(x, pos, f, interleaved=interleaved).double()
    cos, sin = turned(pos, f)
    for got, want in ((out[:, 0, first], cos), (out[:, 0, second], sin), (out[:, 1, first], -sin), (out[:, 1, second], cos)):
        worst = float((got - want).abs().max())
        print("rope", freq, lowest, "%.2e" % worst, flush=True)
        assert worst <= TURN + U


def test_append_turns_far_keys_alike(dev):  # noqa: F811
    """The append's keys are the rotation's, bit for bit."""
    pos = far_positions(dev, 64, 30)
    f = w4.rope_frequencies(64, device=dev)
    k = torch.randn(64, 2, 64, generator=gen(dev, 3), device=dev).to(BF16)
    cache = torch.zeros(2, 4, 16, 2, 64, dtype=BF16, device=dev)
    w4.kv_append(k, k, cache[0], cache[1], torch.arange(64, device=dev), positions=pos, frequencies=f)
    assert torch.equal(cache[0].view(64, 2, 64), w4.rope(k, pos, f))
