"""Values that decode attention has to get right beside the ordinary ones:
infinite, far below the largest score, of the type's largest size."""
import pytest
import torch

import attn_refs
import attn_sharp
from test_gpu_attn import BF16, FP16, INF, dev, make_batch, near  # noqa: F401
from w4a8_moe_grouped_amd import lib as w4

pytestmark = pytest.mark.gpu


def scored(dev, lens, kind, page=16, group=4, Hkv=2, D=64, extra=2, seed=0):
    """A batch whose scores are set by each key's first element: q is 8 there and
    0 elsewhere, keys are 0 in it, so with scale 1 a key's score is 8 times its
    first element (exact in the cache's type)."""
    d = make_batch(dev, lens, group * Hkv, Hkv, D, kind, page, extra=extra, seed=seed)
    d["q"].zero_()
    d["q"][..., 0] = 8.0
    d["k_cache"][..., 0] = 0.0
    return d


def check(d, got, scale):
    """Against the 64-bit form on the CPU (on the GPU torch's softmax of a long row makes 0 of e^-100 in 64 bits too)."""
    host = {k: v if v is None else v.cpu() for k, v in d.items()}
    want, err, lse, lse_err = attn_refs.attn_decode(
        host["q"], host["k_cache"], host["v_cache"], host["page_table"], host["seq_lens"], scale=scale)
    near(got[0].cpu(), want, err, d["q"].dtype)
    near(got[1].cpu(), lse, lse_err, torch.float32)


# uncut, cut over workgroups by the table's width, long, heads taken two by two
FORMS = [dict(lens=[50, 3], extra=2), dict(lens=[50, 700], extra=3000), dict(lens=[20000], extra=0),
         dict(lens=[70] * 130, Hkv=4), dict(lens=[400] * 16, extra=3000)]


@pytest.mark.parametrize("kind", [BF16, FP16])
@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("below", [0, 5, 12, 25, 40, 100, 250])
def test_infinite_values_of_any_weight(dev, kind, page, below):  # noqa: F811
    """An infinite value makes its element infinite however small its weight is (250 below: 2^-360, as a number of
    64 bits still above 0); one of each sign makes it NaN; the other elements do not see it."""
    for form in FORMS:
        d = scored(dev, kind=kind, page=page, **form)
        clean = w4.attn_decode(**d, scale=1.0)[0]
        last = len(form["lens"]) - 1
        n = form["lens"][last]
        for j, h, e, v in ((0, 0, 5, INF), (n // 2, 1, 6, -INF), (n - 1, 0, 7, INF), (1, 1, 8, INF), (n - 2, 1, 8, -INF)):
            d["k_cache"][d["page_table"][last, j // page].long(), j % page, :, 0] = -below / 8
            d["v_cache"][d["page_table"][last, j // page].long(), j % page, h, e] = v
        out, lse = w4.attn_decode(**d, scale=1.0, return_lse=True)
        check(d, (out, lse), 1.0)
        group = d["q"].shape[1] // d["k_cache"].shape[2]
        assert bool((out[last, :group, 5] == INF).all()) and bool((out[last, group:2 * group, 6] == -INF).all())
        assert bool((out[last, :group, 7] == INF).all())
        both = out[last, group:2 * group, 8]
        assert bool(torch.isnan(both).all() if n > 3 else (both == -INF).all())  # of 3 tokens they are the same
        assert torch.equal(out[:last], clean[:last])


@pytest.mark.parametrize("kind", [BF16, FP16])
def test_infinite_values_before_the_maximum(dev, kind):  # noqa: F811
    """Scores that rise by 200 behind an infinite value: what was summed before is scaled to nothing, but it stays infinite."""
    for n, extra in ((300, 0), (6000, 0), (900, 3000)):
        d = scored(dev, [n], kind, extra=extra)
        j = torch.arange(n, device=dev)
        rise = ((j * 4 // n) * 200.0 / 8).to(kind)  # four steps
        d["k_cache"][d["page_table"][0, j // 16].long(), j % 16, :, 0] = rise[:, None]
        d["v_cache"][d["page_table"][0, 0].long(), 2, 1, 9] = -INF
        out, lse = w4.attn_decode(**d, scale=1.0, return_lse=True)
        assert bool((out[0, 4:, 9] == -INF).all()) and int(torch.isfinite(out).sum()) == out.numel() - 4
        check(d, (out, lse), 1.0)


@pytest.mark.parametrize("kind", [BF16, FP16])
def test_infinite_values_under_a_score_of_minus_infinity(dev, kind):  # noqa: F811
    """The definition's 0 times infinity: neither finite nor seen by another element."""
    d = scored(dev, [40], kind)
    page = d["page_table"][0, 0].long()
    d["k_cache"][page, 3, :, 0] = -INF
    clean = w4.attn_decode(**d, scale=1.0)[0]
    d["v_cache"][page, 3, 0, 5] = INF
    out = w4.attn_decode(**d, scale=1.0)[0]
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[0, :4, 5] = True
    assert torch.equal(~torch.isfinite(out), bad)
    near(out[~bad], clean[~bad].double(), torch.zeros((), dtype=torch.float64, device=dev).expand(int((~bad).sum())), kind)


# ---- weights -------------------------------------------------------------------------

def check_sharp(d, **kw):
    want, err = attn_sharp.attention(d["q"], d["k_cache"], d["v_cache"], d["page_table"], d["seq_lens"], d["k_scales"],
                                     d["v_scales"], **kw)
    out = w4.attn_decode(**d, **kw)[0]
    torch.cuda.synchronize()
    bad = attn_sharp.outside(out, want, err)
    print("sharp", tuple(out.shape), d["k_cache"].dtype, "outside", bad, flush=True)
    assert bad == 0


@pytest.mark.parametrize("kind", [BF16, FP16, "fp8"])
@pytest.mark.parametrize("D", [64, 128, 256, 80])
@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("positive", [False, True])
def test_weights_have_two_parts(dev, kind, D, page, positive):  # noqa: F811
    """Outputs are roundings of what the promised error allows; with a weight's second part
    lost a quarter of them are not.  Queries of eight elements and few keys keep the other errors small."""
    for extra in (0, 3000):
        d = make_batch(dev, [128, 33, 100, 7, 128, 1], 8, 2, D, kind, page, extra=extra)
        d["q"][..., 8:] = 0
        if positive and kind == "fp8":
            d["v_cache"] &= 0x7F
        elif positive:
            d["v_cache"].copy_(d["v_cache"].abs() + 0.5)
        check_sharp(d)


@pytest.mark.parametrize("kind", [BF16, FP16])
@pytest.mark.parametrize("above", [10, 15, 17, 20, 23])
@pytest.mark.parametrize("peaks", [1, 16])
def test_small_weights_under_peaks_of_no_value(dev, kind, above, peaks):  # noqa: F811
    """Keys of unit variance below peaks whose values are 0: the output is theirs alone, in weights of e^-above and less."""
    for form in (dict(lens=[4096], extra=0), dict(lens=[4096] * 70, Hkv=4, extra=0), dict(lens=[500], extra=0, page=100)):
        d = scored(dev, kind=kind, **form)
        n, page = form["lens"][0], d["k_cache"].shape[1]
        g = torch.Generator(device=dev).manual_seed(above)
        d["k_cache"][..., 0] = (torch.randn(d["k_cache"].shape[:3], generator=g, device=dev) / 8).to(kind)
        d["v_cache"].copy_(1000 * (d["v_cache"].abs() + 0.5))
        for b in range(len(form["lens"])):
            j = torch.arange(peaks, device=dev) * (n // peaks) + 3
            at = d["page_table"][b, j // page].long(), j % page
            d["k_cache"][at[0], at[1], :, 0] = above / 8
            d["v_cache"][at] = 0
        check_sharp(d, scale=1.0)


def test_very_many_small_weights(dev):  # noqa: F811
    """2^20 keys of no weight to speak of, all of one value, and in each wave's share of them one that has all the weight.

    The small ones are e^-30 of a large one and 8000 times its value: 512 to each add 4e-7.  What the format may
    add is 2^-37 * 512 * 8000, 3e-5; sums of 512 keys and of 512 parts lose 2^-15 each: below half a step under 1, 2^-12."""
    n = 1 << 20
    d = scored(dev, [n], FP16, page=64, group=2, Hkv=1, extra=0)
    d["k_cache"][..., 0] = -30 / 8
    d["v_cache"].fill_(8000.0)
    j = torch.arange(n, device=dev)
    j = j[(j % 2048 < 128) & (j % 32 == 5)]
    at = d["page_table"][0, j // 64].long(), j % 64
    d["k_cache"][at[0], at[1], :, 0] = 0.0
    d["v_cache"][at] = 1.0
    assert bool((w4.attn_decode(**d, scale=1.0)[0] == 1.0).all())


# ---- the largest values --------------------------------------------------------------

@pytest.mark.parametrize("kind", [BF16, FP16, "fp8"])
@pytest.mark.parametrize("rise", [0, 1, 5, 30])
@pytest.mark.parametrize("mixed", [False, True])
def test_largest_values(dev, kind, rise, mixed):  # noqa: F811
    """Values of the type's largest size (e4m3: under the largest scale) have a mean of that size at most, under equal
    scores and under scores that rise by `rise` nats every 32 keys."""
    for lens, extra, Hkv in (([700, 40], 0, 2), ([20000], 0, 2), ([3000, 300], 3000, 2), ([300] * 130, 0, 4)):
        d = scored(dev, lens, BF16 if kind == "fp8" else kind, extra=extra, Hkv=Hkv)
        pages, page = d["k_cache"].shape[:2]
        for b, n in enumerate(lens):
            j = torch.arange(n, device=dev)
            steps = (j // 32 % 12 * rise / 8).to(d["k_cache"].dtype)
            d["k_cache"][d["page_table"][b, j // page].long(), j % page, :, 0] = steps[:, None]
        sign = torch.where(d["v_cache"] > 0, 1.0, -1.0) if mixed else torch.ones_like(d["v_cache"])
        most = torch.finfo(d["v_cache"].dtype).max
        if kind == "fp8":
            d["k_cache"] = d["k_cache"].to(torch.float8_e4m3fn).view(torch.uint8)
            d["v_cache"] = (448 * sign).to(torch.float8_e4m3fn).view(torch.uint8)
            d["k_scales"] = torch.ones(pages, Hkv, page, device=dev)
            d["v_scales"] = torch.full((pages, Hkv, page), most / 448, device=dev)
        else:
            d["v_cache"] = (most * sign).to(d["v_cache"].dtype)
        check_sharp(d, scale=1.0)
        assert bool(torch.isfinite(w4.attn_decode(**d, scale=1.0)[0]).all())


@pytest.mark.parametrize("least", ["all", "half"])
def test_smallest_scales_of_codes(dev, least):  # noqa: F811
    """Rows of (nearly) nothing, whose scales are the least that an append writes."""
    for extra in (0, 3000):
        d = make_batch(dev, [128, 33, 700, 1], 8, 2, 64, "fp8", 16, extra=extra)
        d["q"][..., 8:] = 0
        scales = d["v_scales"] if least == "all" else d["v_scales"][..., ::2]
        scales.fill_(1e-10 / 448)
        check_sharp(d)


@pytest.mark.parametrize("kind", [BF16, FP16])
@pytest.mark.parametrize("extra", [0, 3000])
def test_infinite_scores(dev, kind, extra):  # noqa: F811
    """+infinity and NaN make their rows NaN, -infinity weighs nothing, and a row of nothing else is 0."""
    d = scored(dev, [70, 70, 70, 70, 600], kind, extra=extra)
    clean = w4.attn_decode(**d, scale=1.0, return_lse=True)
    for b, value, tokens in ((0, INF, [33]), (1, float("nan"), [69]), (2, -INF, [0, 5, 64]), (3, -INF, list(range(70)))):
        for j in tokens:
            d["k_cache"][d["page_table"][b, j // 16].long(), j % 16, 0, 0] = value  # of the first kv head
    out, lse = w4.attn_decode(**d, scale=1.0, return_lse=True)
    assert bool(torch.isnan(out[:2, :4]).all()) and bool(torch.isnan(lse[:2, :4]).all())
    assert bool((out[3, :4] == 0).all()) and bool((lse[3, :4] == -INF).all())
    near(lse[2, :4], torch.full((4,), 67.0, dtype=torch.float64, device=dev).log(),
         torch.full((4,), 1e-5, dtype=torch.float64, device=dev))
    assert bool(torch.isfinite(out[2]).all())
    for got, want in zip((out, lse), clean):
        assert torch.equal(got[:, 4:], want[:, 4:]) and torch.equal(got[4], want[4])


@pytest.mark.parametrize("kind", [BF16, FP16])
@pytest.mark.parametrize("value", [INF, float("nan"), "largest"])
@pytest.mark.parametrize("below", [8, 60, 110, 400, INF])
def test_values_that_are_far_off_stay_where_they_are(dev, kind, value, below):  # noqa: F811
    """One element of one key that is infinite, NaN or of the type's largest size: no other element, head or sequence
    changes by a bit; and the largest adds no more than its weight has it (nothing, where that is below 2^-150)."""
    for form in FORMS:
        d = scored(dev, kind=kind, **form)
        last = len(form["lens"]) - 1
        n = form["lens"][last]
        places = [(j, h, 3 + 7 * i) for i, (j, h) in enumerate(((0, 0), (n // 2, 1), (n - 1, 0)))]
        for j, h, e in places:
            at = d["page_table"][last, j // 16].long(), j % 16
            d["k_cache"][at[0], at[1], :, 0] = -below / 8
            d["v_cache"][at[0], at[1], h, e] = 0.0
        clean = w4.attn_decode(**d, scale=1.0, return_lse=True)
        assert bool(torch.isfinite(clean[0]).all())
        for j, h, e in places:
            d["v_cache"][d["page_table"][last, j // 16].long(), j % 16, h, e] = (
                torch.finfo(kind).max if value == "largest" else value)
        out, lse = w4.attn_decode(**d, scale=1.0, return_lse=True)
        assert torch.equal(lse, clean[1])
        group = d["q"].shape[1] // d["k_cache"].shape[2]
        changed = torch.zeros_like(out, dtype=torch.bool)
        for j, h, e in places:
            changed[last, h * group:(h + 1) * group, e] = True
        if value == "largest" and below > 104 and (n > 3 or below == INF):  # of three tokens all are so far below
            changed[:] = False
        assert torch.equal(out[~changed], clean[0][~changed])
        if value != "largest":
            assert not bool(torch.isfinite(out[changed]).any())
        elif changed.any():
            check(d, (out, lse), 1.0)


@pytest.mark.parametrize("D", [64, 128, 200])
@pytest.mark.parametrize("R", [0, 32])
def test_infinite_elements_in_an_appended_row_of_codes(dev, D, R):  # noqa: F811
    """By the rule an infinity's row has an infinite scale, its own code is that of infinity times 0, NaN, and the
    others' are 0: what attends to the row is NaN, whatever signs meet (an infinite key was passed over where its
    score came out as -infinity)."""
    T, H = 40, 2
    g = torch.Generator(device=dev).manual_seed(D)
    x = torch.randn(T, 2 * H, D, generator=g, device=dev).to(BF16)
    k, v = x[:, :H], x[:, H:]
    k[3, 0, 40], k[20, 1, 41], v[30, 0, 42] = INF, -INF, INF  # not among those that are turned
    kc, vc = (torch.zeros(3, 16, H, D, dtype=torch.uint8, device=dev) for _ in range(2))
    ks, vs = (torch.zeros(3, H, 16, device=dev) for _ in range(2))
    kw = dict(positions=torch.arange(T, dtype=torch.int32, device=dev), frequencies=w4.rope_frequencies(R, device=dev)) if R else {}
    w4.kv_append(k, v, kc, vc, torch.arange(T, device=dev), k_scales=ks, v_scales=vs, **kw)
    for cache, scales, j, h, e in ((kc, ks, 3, 0, 40), (kc, ks, 20, 1, 41), (vc, vs, 30, 0, 42)):
        row = cache.view(-1, H, D)[j, h].clone()
        assert float(scales[j // 16, h, j % 16]) == INF and int(row[e]) & 0x7F == 0x7F
        row[e] = 0
        assert bool((row & 0x7F == 0).all())
    assert int(torch.isfinite(ks).sum()) == ks.numel() - 2 and int(torch.isfinite(vs).sum()) == vs.numel() - 1
    table = torch.arange(3, dtype=torch.int32, device=dev).expand(4, 3).contiguous()
    q = torch.randn(4, 4, D, generator=g, device=dev).to(BF16)
    q[:, ::2] = q[:, 1::2] * -1  # both signs in every element
    lens = torch.tensor([3, 20, 30, 40], dtype=torch.int32, device=dev)
    out, lse = w4.attn_decode(q, kc, vc, table, lens, k_scales=ks, v_scales=vs, return_lse=True)
    bad = torch.tensor([[0, 0], [1, 0], [1, 1], [1, 1]], dtype=torch.bool, device=dev).repeat_interleave(2, 1)
    assert torch.equal(torch.isnan(lse), bad)
    assert torch.equal(torch.isnan(out).all(-1), bad) and torch.equal(torch.isnan(out).any(-1), bad)
