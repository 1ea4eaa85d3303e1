"""The attention half at the ends of what it accepts: the most sequences, tokens and positions, no tokens."""
import pytest
import torch

import attn_refs as ref
from test_gpu_attn import BF16, check_attn, dev, gen, make_batch, near  # noqa: F401
from w4a8_moe_grouped_amd import lib as w4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages", [1, 300])
@pytest.mark.parametrize("D", [64, 128])
def test_most_sequences(dev, pages, D):  # noqa: F811
    """65536 sequences of 0 to 16 tokens, whole and (by the table's width) cut; garbage behind the tables' first page."""
    B, page, Hkv = 65536, 16, 2
    g = gen(dev, pages + D)
    kc, vc = (torch.randn(1000, page, Hkv, D, generator=g, device=dev).to(BF16) for _ in range(2))
    q = torch.randn(B, 4, D, generator=g, device=dev).to(BF16)
    table = torch.randint(-5, 1005, (B, pages), generator=g, device=dev, dtype=torch.int32)
    lens = torch.randint(0, page + 1, (B,), generator=g, device=dev, dtype=torch.int32)
    lens[:70] = 0
    out, lse = w4.attn_decode(q, kc, vc, table, lens, return_lse=True)
    held = (table[:, 0] >= 0) & (table[:, 0] < 1000)
    for at in range(0, B, 8192):
        rows = slice(at, at + 8192)
        p = table[rows, 0].clamp(0, 999).long()
        k, v = (c[p].float().permute(0, 2, 3, 1).contiguous() for c in (kc, vc))  # [b, kv head, D, token]
        s = torch.matmul(q[rows].float().view(-1, Hkv, 2, D), k) * D ** -0.5
        seen = (torch.arange(page, device=dev) < lens[rows, None]) & held[rows, None]
        s = s.masked_fill(~seen[:, None, None], -torch.inf)
        some = seen.any(1)[:, None, None]
        w = torch.softmax(s, -1).masked_fill(~seen[:, None, None], 0.0)
        want = torch.matmul(w, v.transpose(2, 3).contiguous()).view(-1, 4, D)
        torch.testing.assert_close(out[rows].float(), torch.where(some, want, 0.0), rtol=2 ** -8, atol=2e-3)
        torch.testing.assert_close(lse[rows], torch.logsumexp(s, -1).view(-1, 4), rtol=1e-5, atol=1e-4)


def test_widest_table(dev):  # noqa: F811
    """A table for 2^30 tokens, lengths of few; and a length past all of it with one page that holds something."""
    d = make_batch(dev, [300, 0, 5], 4, 2, 64, BF16, 1024, extra=0)
    wide = torch.full((3, 1 << 20), -1, dtype=torch.int32, device=dev)
    wide[:, :1] = d["page_table"]
    d["page_table"] = wide
    check_attn(d)
    d["seq_lens"][:] = 2 ** 31 - 1
    d["k_cache"][:], d["v_cache"][:] = 0.0, 1.0
    wide[:, 0] = 0
    wide[1, 0], wide[1, -1] = -1, 1
    out, lse = w4.attn_decode(**d, return_lse=True)
    assert bool((out == 1.0).all())
    near(lse, torch.full_like(lse, 1024).double().log(), torch.full_like(lse, 1e-5).double())
    out, lse = w4.attn_decode(**d, return_lse=True, window=2 ** 62)
    assert bool((out == 1.0).all())
    # the last 2^30 of 2^31 - 1 tokens begin at the table's last, which the second sequence alone holds
    out, lse = w4.attn_decode(**d, return_lse=True, window=2 ** 30)
    assert bool((out[1] == 1.0).all()) and bool((lse[1].abs() < 1e-6).all())
    assert bool((out[::2] == 0.0).all()) and bool((lse[::2] == -torch.inf).all())


def test_most_tokens(dev):  # noqa: F811
    T = 1 << 25
    x = torch.randn(T, 1, 8, generator=gen(dev, 1), device=dev).to(BF16)
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    freq = w4.rope_frequencies(8, device=dev)
    out = w4.rope(x, pos, freq)
    for rows in (slice(0, 1000), slice(T // 2 - 500, T // 2 + 500), slice(T - 1000, T)):
        near(out[rows], *ref.rope(x[rows], pos[rows], freq), BF16)
    kc, vc = (torch.zeros(T // 64, 64, 1, 8, dtype=BF16, device=dev) for _ in range(2))
    slots = torch.arange(T - 1, -1, -1, device=dev)
    assert w4.kv_append(x, x, kc, vc, slots, positions=pos, frequencies=freq) is None
    assert torch.equal(kc.view(T, 1, 8).flip(0), out) and torch.equal(vc.view(T, 1, 8).flip(0), x)
    with pytest.raises(w4.W4A8Error, match="unsupported"):
        w4.rope(torch.empty(1, 1, 8, dtype=BF16, device=dev).expand(T + 1, 1, 8), pos.new_zeros(T + 1), freq, out=None)
