"""The decoder's row operators on a GPU against plain 64-bit forms, with
tolerances derived in decoder_util."""
import math

import pytest
import torch

import row_reduction_gb300 as mt
from decoder_util import (DTYPES, LARGEST, check, half_step, logits_ref,
                          quantise_ref, rotary_backward_ref, rotary_ref)

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


class Sentinel:
    """A [tokens, heads, dim] view into a larger buffer whose every other
    value must stay as it is.  pad: values between heads and behind a
    token."""

    def __init__(self, tokens, heads, dim, dtype, pad=8, offset=16):
        self.width = heads * (dim + pad) + pad
        self.buf = torch.full((2 * offset + tokens * self.width,), -77.0,
                              dtype=dtype, device="cuda")
        self.view = torch.as_strided(
            self.buf, (tokens, heads, dim), (self.width, dim + pad, 1),
            offset)

    def check(self):
        keep = self.buf.clone()
        torch.as_strided(keep, self.view.shape, self.view.stride(),
                         self.view.storage_offset()).fill_(-77.0)
        assert bool((keep == -77.0).all()), "written outside the rows"


# ---- rotary -----------------------------------------------------------------
def rot_inputs(seed, tokens, hq, hk, dim, dtype, far=4096, pos64=True):
    g = gen(seed)
    fused = randn(g, tokens, hq + 2 * hk, dim, dtype=dtype)
    pos = torch.randint(0, far, (tokens,), generator=g, device="cuda")
    w = [(1 + 0.1 * randn(g, dim)).to(dtype) for _ in range(2)]
    return (fused[:, :hq], fused[:, hq:hq + hk],
            pos if pos64 else pos.to(torch.int32), *w)


def table(rotary, **kw):
    f, s = mt.mt_rotary_frequencies(rotary, 10000.0)
    t = mt.rotary_frequencies(rotary, **kw)
    return (f, s, t)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,hq,hk,dim,rotary", [
    (1, 1, 1, 2, 2), (1, 32, 8, 128, 128), (3, 2, 1, 64, 32), (7, 5, 3, 80, 40),
    (5, 3, 1, 96, 24), (2, 4, 4, 256, 256), (2, 3, 1, 512, 512),
    (4, 1, 1, 130, 66), (3, 2, 2, 17, 6), (2, 2, 1, 77, 70), (33, 9, 1, 20, 20),
    (2, 1, 1, 511, 510), (300, 4, 2, 64, 64), (3, 2, 1, 264, 264),
    (3, 3, 1, 132, 132), (2600, 3, 1, 64, 32), (2500, 41, 9, 64, 64),
    (2700, 6, 2, 96, 96), (2600, 9, 3, 128, 128), (1250, 15, 5, 80, 40),
    (2500, 15, 3, 64, 16), (2450, 8, 1, 128, 128),
])
def test_rotary(dt, norm, interleaved, tokens, hq, hk, dim, rotary):
    dtype = DTYPES[dt]
    q, k, pos, wq, wk = rot_inputs(tokens + dim, tokens, hq, hk, dim, dtype,
                                   pos64=dim % 4 == 0)
    freqs, scale, tab = table(rotary)
    kw = dict(q_weight=wq, k_weight=wk, eps=1e-6) if norm else {}
    oq, ok = (Sentinel(tokens, h, dim, dtype) for h in (hq, hk))
    got = mt.rotary(q, k, pos, tab, interleaved=interleaved,
                    out=(oq.view, ok.view), **kw)
    plain = mt.rotary(q, k, pos, tab, interleaved=interleaved, **kw)
    for x, y, o, p, w in ((q, got[0], oq, plain[0], wq),
                          (k, got[1], ok, plain[1], wk)):
        ref, err = rotary_ref(x, pos, freqs, scale, rotary, interleaved,
                              w if norm else None, 1e-6 if norm else None)
        tol = err + half_step(ref, dtype)
        check(y, ref, tol, "rotary")
        check(p, ref, tol, "rotary, new outputs")
        o.check()
        if not norm:  # values that pass are copied bit for bit
            assert torch.equal(y[..., rotary:], x[..., rotary:])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rotary_far_and_negative_positions(dt):
    """The angle is exact in 64 bits: positions to 2^31 and below zero."""
    dtype = DTYPES[dt]
    q, k, _, _, _ = rot_inputs(3, 8, 2, 1, 64, dtype)
    pos = torch.tensor([0, -1, 2 ** 20 + 1, -2 ** 20, 2 ** 24 + 3, 2 ** 31 - 1,
                        -2 ** 31, 123456789], device="cuda")
    freqs, scale, tab = table(64)
    for p in (pos, pos.to(torch.int32)):
        y, _ = mt.rotary(q, k, p, tab)
        ref, err = rotary_ref(q, pos, freqs, scale, 64, False, None, None)
        # the 64-bit reference itself rounds the product at 2^-53 of 2^31
        check(y, ref, err + half_step(ref, dtype) + 1e-6, "far positions")


@pytest.mark.parametrize("scaling", [
    dict(type="linear", factor=4.0), dict(type="ntk", factor=4.0),
    dict(type="yarn", factor=8.0, original_length=2048),
    dict(type="bands", factor=8.0, original_length=2048)])
def test_rotary_scaled_for_long_contexts(scaling):
    kinds = dict(linear=1, ntk=2, yarn=3, bands=4)
    s = mt.MtRotaryScaling(
        type=kinds[scaling["type"]], factor=scaling["factor"],
        original_length=scaling.get("original_length", 0), low=1.0,
        high=32.0 if scaling["type"] == "yarn" else 4.0)
    freqs, factor = mt.mt_rotary_frequencies(96, 500000.0, s)
    tab = mt.rotary_frequencies(96, base=500000.0, scaling=scaling)
    assert tab.scale == factor
    q, k, pos, wq, wk = rot_inputs(5, 40, 4, 2, 128, torch.float32, far=16384)
    y, _ = mt.rotary(q, k, pos, tab, q_weight=wq, k_weight=wk, eps=1e-5)
    ref, err = rotary_ref(q, pos, freqs, factor, 96, False, wq, 1e-5)
    check(y, ref, err + half_step(ref, torch.float32), scaling["type"])


def test_rotary_custom_frequencies_and_scale():
    freqs = [2.0, -0.5, 7.5, 0.0]
    tab = mt.rotary_frequencies(8, freqs=freqs, scale=0.75)
    q, k, pos, _, _ = rot_inputs(6, 9, 3, 1, 24, torch.float32)
    y = mt.rotary(q, None, pos, tab, interleaved=True)
    ref, err = rotary_ref(q, pos, freqs, 0.75, 8, True, None, None)
    check(y, ref, err + half_step(ref, torch.float32))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("norm", [False, True])
def test_rotary_in_place_and_other_layouts(dt, norm):
    """In place in a fused projection; heads before tokens; reversed and
    repeated rows; addresses off a 16-byte boundary."""
    dtype = DTYPES[dt]
    q, k, pos, wq, wk = rot_inputs(7, 21, 6, 2, 64, dtype)
    freqs, scale, tab = table(64)
    kw = dict(q_weight=wq, k_weight=wk, eps=1e-6) if norm else {}
    want = mt.rotary(q, k, pos, tab, **kw)
    fused = torch.cat((q, k), 1).contiguous()
    a, b = fused[:, :6], fused[:, 6:]
    mt.rotary(a, b, pos, tab, out=(a, b), **kw)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    swapped = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k)]
    got = mt.rotary(*swapped, pos, tab, out=tuple(
        torch.empty_like(t.transpose(0, 1).contiguous()).transpose(0, 1)
        for t in (q, k)), **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # every other row of a larger buffer, a broadcast row
    thick = torch.repeat_interleave(q, 2, 0)[::2]
    assert torch.equal(mt.rotary(thick, None, pos, tab, **{
        n: v for n, v in kw.items() if n != "k_weight"}), want[0])
    wide = q[:1].expand(21, -1, -1)
    got = mt.rotary(wide, None, pos, tab, **{
        n: v for n, v in kw.items() if n != "k_weight"})
    ref, err = rotary_ref(wide, pos, freqs, scale, 64, False,
                          wq if norm else None, 1e-6 if norm else None)
    check(got, ref, err + half_step(ref, dtype), "broadcast")
    for off in (1, 2, 3, 4):
        buf = torch.zeros(off + q.numel(), dtype=dtype, device="cuda")
        x = buf[off:].view(21, 6, 64)
        x.copy_(q)
        got = mt.rotary(x, None, pos, tab, **{
            n: v for n, v in kw.items() if n != "k_weight"})
        ref, err = rotary_ref(q, pos, freqs, scale, 64, False,
                              wq if norm else None, 1e-6 if norm else None)
        check(got, ref, err + half_step(ref, dtype), f"offset {off}")


def test_rotary_non_finite_rows_stay_in_their_heads():
    q, k, pos, wq, wk = rot_inputs(8, 6, 3, 1, 32, torch.float32)
    q = q.clone()
    q[1, 1, 3] = math.nan
    q[2, 0, 5] = math.inf
    _, _, tab = table(32)
    clean = mt.rotary(torch.nan_to_num(q, posinf=0.0), None, pos, tab,
                      q_weight=wq, eps=1e-6)
    got = mt.rotary(q, None, pos, tab, q_weight=wq, eps=1e-6)
    hit = torch.zeros(6, 3, dtype=torch.bool, device="cuda")
    hit[1, 1] = hit[2, 0] = True
    assert torch.equal(got[~hit], clean[~hit])
    assert bool(torch.isnan(got[1, 1]).all())
    # a zero row stays zero under eps
    z = torch.zeros(2, 1, 32, device="cuda")
    assert bool((mt.rotary(z, None, pos[:2], tab, eps=1e-6) == 0).all())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rotary", [(64, 32), (80, 40), (18, 6)])
def test_rotary_values_that_pass_keep_infinities_and_nan(dim, rotary,
                                                         interleaved):
    """A value that is not turned is nobody's partner: infinities and NaN stay
    in their places there, forward and backward."""
    q, _, pos, _, _ = rot_inputs(16, 5, 2, 1, dim, torch.bfloat16)
    q = q.clone()
    q[1, 0, rotary] = math.inf
    q[2, 1, dim - 1] = -math.inf
    q[3, 0, rotary + 1] = math.nan
    _, _, tab = table(rotary)
    for y in (mt.rotary(q, None, pos, tab, interleaved=interleaved),
              mt.rotary_backward(q, None, pos, tab,
                                 interleaved=interleaved)[0]):
        assert torch.equal(y[..., rotary:].view(torch.int16),
                           q[..., rotary:].contiguous().view(torch.int16))
        assert bool(torch.isfinite(y[..., :rotary]).all())


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,hq,hk,dim,rotary", [
    (1, 1, 1, 2, 2), (1, 8, 2, 128, 128), (3, 2, 1, 64, 32), (7, 5, 3, 80, 40),
    (2, 3, 1, 512, 512), (4, 1, 1, 130, 66), (3, 2, 2, 17, 6),
    (2, 2, 1, 77, 70), (33, 9, 1, 20, 20), (5, 3, 0, 64, 64),
    (200, 2, 1, 64, 64), (3, 2, 1, 264, 264), (3, 3, 1, 132, 132),
    (2, 1, 1, 511, 510), (700, 33, 5, 64, 64),
])
def test_rotary_backward(dt, norm, interleaved, tokens, hq, hk, dim, rotary):
    dtype = DTYPES[dt]
    q, k, pos, wq, wk = rot_inputs(tokens + dim, tokens, hq, max(hk, 1), dim,
                                   dtype)
    dq, dk, _, _, _ = rot_inputs(999, tokens, hq, max(hk, 1), dim, dtype)
    if hk == 0:
        k, dk, wk = None, None, None
    freqs, scale, tab = table(rotary)
    kw = dict(q=q, k=k, q_weight=wq, k_weight=wk, eps=1e-6) if norm else {}
    oq = Sentinel(tokens, hq, dim, dtype)
    ok = Sentinel(tokens, hk, dim, dtype) if hk else None
    got = mt.rotary_backward(dq, dk, pos, tab, interleaved=interleaved,
                             out=(oq.view, ok.view if hk else None), **kw)
    again = mt.rotary_backward(dq, dk, pos, tab, interleaved=interleaved, **kw)
    for i, (dy, x, w, o) in enumerate(((dq, q, wq, oq), (dk, k, wk, ok))):
        if dy is None:
            assert got[i] is None
            continue
        dx, err, dw, werr = rotary_backward_ref(
            dy, x, pos, freqs, scale, rotary, interleaved, w,
            1e-6 if norm else None)
        check(got[i], dx, err + half_step(dx, dtype), "dx")
        assert torch.equal(got[i], again[i])
        o.check()
        if norm:
            assert got[2 + i].dtype == torch.float32
            check(got[2 + i], dw, werr, "dweight")
            assert torch.equal(got[2 + i], again[2 + i])


def test_rotary_backward_forms():
    """No weights; gradients in place of dy and of x; many tokens (several
    rounds per CTA); a call without tokens."""
    q, k, pos, wq, wk = rot_inputs(11, 6000, 3, 1, 64, torch.bfloat16)
    dq, dk, _, _, _ = rot_inputs(12, 6000, 3, 1, 64, torch.bfloat16)
    freqs, scale, tab = table(64)
    kw = dict(q=q, k=k, q_weight=wq, k_weight=wk, eps=1e-6)
    want = mt.rotary_backward(dq, dk, pos, tab, **kw)
    dx, err, dw, werr = rotary_backward_ref(dq, q, pos, freqs, scale, 64,
                                            False, wq, 1e-6)
    check(want[0], dx, err + half_step(dx, torch.bfloat16))
    check(want[2], dw, werr)
    a, b = dq.clone(), dk.clone()
    got = mt.rotary_backward(a, b, pos, tab, out=(a, b), **kw)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    assert torch.equal(got[2], want[2])
    a, b = q.clone(), k.clone()
    mt.rotary_backward(dq, dk, pos, tab, out=(a, b), **{**kw, "q": a, "k": b})
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    got = mt.rotary_backward(dq, None, pos, tab, q=q, eps=1e-6)
    assert got[1] is None and got[2] is None and got[3] is None
    ones = torch.ones_like(wq)
    assert torch.equal(got[0], mt.rotary_backward(
        dq, None, pos, tab, q=q, q_weight=ones, eps=1e-6)[0])
    e = torch.empty(0, 3, 64, dtype=torch.bfloat16, device="cuda")
    got = mt.rotary_backward(e, None, pos[:0], tab, q=e, q_weight=wq,
                             eps=1e-6)
    assert got[0].shape == (0, 3, 64) and bool((got[2] == 0).all())


def test_rotary_backward_matches_differences_of_the_kernel():
    """<dy, f(x + h v) - f(x - h v)> / 2h of the FP32 forward kernel against
    <dx, v>.  The forward's error is that of angle and norm, of sqrt(2) times a value of
    about 1, at most 2e-6 each, summed with random signs over n values of dy
    ~ 1: below 2e-6 sqrt(n) * 4 / h; the third derivative adds h^2 sqrt(n)."""
    n, h = 40 * 4 * 64, 1e-2
    q, _, pos, wq, _ = rot_inputs(13, 40, 4, 1, 64, torch.float32)
    g = gen(14)
    dy, v = randn(g, 40, 4, 64), randn(g, 40, 4, 64)
    _, _, tab = table(64)

    def f(x):
        return mt.rotary(x, None, pos, tab, q_weight=wq, eps=1e-6).double()
    want = float((dy.double() * (f(q + h * v) - f(q - h * v))).sum() / (2 * h))
    dx = mt.rotary_backward(dy, None, pos, tab, q=q, q_weight=wq, eps=1e-6)[0]
    got = float((dx.double() * v.double()).sum())
    assert abs(got - want) <= math.sqrt(n) * (8e-6 / h + 4 * h * h)


def test_rotary_refuses_on_the_device():
    q, k, pos, wq, wk = rot_inputs(15, 4, 2, 1, 16, torch.bfloat16)
    _, _, tab = table(16)
    with pytest.raises(ValueError, match="eps"):
        mt.rotary(q, k, pos, tab, q_weight=wq)
    with pytest.raises(ValueError, match="k_weight without k"):
        mt.rotary(q, None, pos, tab, k_weight=wk, eps=1e-6)
    with pytest.raises(TypeError, match="positions"):
        mt.rotary(q, k, pos.float(), tab)
    with pytest.raises(ValueError, match="positions"):
        mt.rotary(q, k, pos[:3], tab)
    with pytest.raises(TypeError):
        mt.rotary(q, k.float(), pos, tab)
    with pytest.raises(TypeError):
        mt.rotary(q.long(), None, pos, tab)
    with pytest.raises(ValueError):
        mt.rotary(q, k[:3], pos, tab)
    with pytest.raises(ValueError, match="dense"):
        mt.rotary(q.transpose(1, 2), None, pos, tab)
    with pytest.raises(mt.MTError):
        mt.rotary(q[..., :8], None, pos, tab)          # rotary_dim > dim
    with pytest.raises(mt.MTError):                     # output rows overlap
        mt.rotary(q, None, pos, tab, out=q[:1].expand(4, -1, -1))
    with pytest.raises(ValueError, match="needs q"):
        mt.rotary_backward(q, None, pos, tab, eps=1e-6)
    with pytest.raises(ValueError, match="give eps"):
        mt.rotary_backward(q, None, pos, tab, q=q)


# ---- cache ----------------------------------------------------------------------
def paged_slots(g, tokens, pool, page=16):
    order = torch.randperm(pool // page, generator=g, device="cuda")
    at = torch.arange(tokens, device="cuda")
    return order[at // page] * page + at % page


def snapshot(cache):
    return cache[0].view(torch.int8).clone(), cache[1].clone()


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("tokens,heads,dim,group", [
    (1, 1, 1, 1), (1, 8, 128, 128), (5, 3, 80, 80), (64, 2, 64, 32),
    (7, 1, 96, 24), (3, 2, 256, 256), (9, 4, 128, 16), (2, 1, 576, 576),
    (4, 3, 20, 5), (3, 5, 33, 11), (130, 1, 8, 8), (3, 2, 1024, 512),
    (9001, 4, 64, 64), (3000, 1, 40, 8), (2, 700, 16, 16),
])
def test_cache_write_and_read(dt, fmt, tokens, heads, dim, group):
    dtype = DTYPES[dt]
    g = gen(tokens * dim + group)
    fused = (randn(g, tokens, 2 * heads, dim) *
             torch.exp(2 * randn(g, 2 * heads, dim))).to(dtype)
    k, v = fused[:, :heads], fused[:, heads:]
    pool = (tokens + 40) // 16 * 16 + 16
    slots = paged_slots(g, tokens, pool)
    slots[tokens // 2] = -1 if tokens > 1 else slots[0]
    if tokens > 4:
        slots[1] = pool
        slots[2] = 2 ** 40
    caches = [mt.cache_alloc(pool, heads, dim, group, fmt) for _ in range(2)]
    for c in caches:
        c[0].view(torch.int8).fill_(55)
        c[1].fill_(-3.0)
    before = [snapshot(c) for c in caches]
    mt.cache_write(k, v, *caches, slots)
    live = (slots >= 0) & (slots < pool)
    rest = torch.ones(pool, dtype=torch.bool, device="cuda")
    rest[slots[live]] = False
    outs = [Sentinel(tokens, heads, dim, dtype) for _ in range(2)]
    got = mt.cache_read(*caches, slots, out=tuple(o.view for o in outs))
    for x, c, b, o, y in zip((k, v), caches, before, outs, got):
        codes, scales = quantise_ref(x, fmt, group)
        held = c[0][slots[live]]
        # the operator's own FP32 steps are exactly rounded: equal bits
        assert torch.equal(held.float().cpu(), codes[live.cpu()])
        assert torch.equal(c[1][slots[live]].cpu(), scales[live.cpu()])
        assert torch.equal(c[0].view(torch.int8)[rest], b[0][rest])
        assert torch.equal(c[1][rest], b[1][rest])
        want = codes.unflatten(-1, (-1, group)) * scales[..., None]
        want = want.flatten(-2).to(dtype)
        assert torch.equal(y[live].cpu(), want[live.cpu()])
        assert bool((y[~live] == -77.0).all()), "a padding row was written"
        o.check()
        # from the definition: half a step of the format (the smallest e4m3
        # step is 2^-9), widened by the two roundings of scale and 1/scale
        x64 = x[live].double().cpu()
        s64 = scales[live.cpu()].double().repeat_interleave(group, -1)
        back = (codes.double().unflatten(-1, (-1, group)) *
                scales.double()[..., None]).flatten(-2)[live.cpu()]
        step = torch.maximum(x64.abs() * 2.0 ** -4, s64 * 2.0 ** -10) \
            if fmt == "e4m3" else s64 / 2
        assert bool(((back - x64).abs() <= step + x64.abs() * 2.0 ** -21).all())


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("group", [32, 11])
def test_cache_special_groups(dt, fmt, group):
    """Zeros, subnormals, the type's largest values, one spike, NaN and
    infinities (whose group reads back as NaN, and no other)."""
    dtype = DTYPES[dt]
    info = torch.finfo(dtype)
    x = torch.zeros(8, 1, 2 * group, dtype=dtype, device="cuda")
    x[1] = info.smallest_normal / 4
    x[2] = info.max
    x[3, 0, 3] = 1000.0
    x[4, 0, 0] = math.nan
    x[5, 0, group + 1] = -math.inf
    x[6] = -info.max
    x[7] = torch.linspace(-1, 1, 2 * group).to(dtype)
    c = mt.cache_alloc(8, 1, 2 * group, group, fmt)
    slots = torch.arange(8, device="cuda")
    mt.cache_write(x, None, c, None, slots)
    y = mt.cache_read(c, None, slots, dtype=dtype)
    codes, scales = quantise_ref(x, fmt, group)
    assert torch.equal(c[0].float().cpu(), codes)
    assert torch.equal(torch.nan_to_num(c[1].cpu(), nan=-1.0),
                       torch.nan_to_num(scales, nan=-1.0))
    nan = torch.isnan(y[:, 0].unflatten(-1, (2, group)))
    want = torch.zeros(8, 2, dtype=torch.bool)
    want[4, 0] = want[5, 1] = True
    assert torch.equal(nan.all(-1).cpu(), want)
    assert torch.equal(nan.any(-1).cpu(), want)
    assert bool((y[0] == 0).all())


def test_cache_read_repeats_slots_and_new_outputs_are_zero_where_padding():
    g = gen(20)
    c = mt.cache_alloc(64, 2, 32, 32, "int8")
    x = randn(g, 64, 2, 32)
    mt.cache_write(x, None, c, None, torch.arange(64, device="cuda"))
    slots = torch.tensor([5, 5, -1, 63, 64, 5, 0], device="cuda")
    y = mt.cache_read(c, None, slots, dtype=torch.float32)
    whole = mt.cache_read(c, None, torch.arange(64, device="cuda"),
                          dtype=torch.float32)
    assert torch.equal(y[[0, 1, 3, 5, 6]], whole[[5, 5, 63, 5, 0]])
    assert bool((y[[2, 4]] == 0).all())


def test_cache_off_alignment():
    """Codes and rows at addresses that rule out wide accesses."""
    g = gen(21)
    for off in (1, 3, 4):
        x = randn(g, off + 5 * 2 * 64, dtype=torch.bfloat16)[off:].view(
            5, 2, 64)
        raw = torch.zeros(off + 16 * 2 * 64, dtype=torch.int8, device="cuda")
        c = (raw[off:].view(16, 2, 64), torch.zeros(16, 2, 2, device="cuda"))
        slots = torch.tensor([3, 0, 15, 7, -1], device="cuda")
        mt.cache_write(x, None, c, None, slots)
        codes, scales = quantise_ref(x, "int8", 32)
        assert torch.equal(c[0][slots[:4]].float().cpu(), codes[:4])
        out = torch.zeros(off + 5 * 2 * 64, dtype=torch.bfloat16,
                          device="cuda")[off:].view(5, 2, 64)
        mt.cache_read(c, None, slots, out=out)
        want = (codes.unflatten(-1, (2, 32)) * scales[..., None]).flatten(
            -2).bfloat16()
        assert torch.equal(out[:4].cpu(), want[:4])
        assert bool((raw[:off] == 0).all()) and bool((out[4] == 0).all())


def test_cache_larger_than_32_bits():
    """Slots beyond 2^32 bytes of codes: 4.6 GB of codes, one tensor."""
    slots_n, heads, dim = 4_500_000, 8, 128
    c = mt.cache_alloc(slots_n, heads, dim, 128, "e4m3")
    x = randn(gen(22), 4, heads, dim, dtype=torch.bfloat16)
    slots = torch.tensor([slots_n - 1, 0, 4_194_304, 2_097_152],
                         device="cuda")
    mt.cache_write(x, None, c, None, slots)
    y = mt.cache_read(c, None, slots)
    codes, scales = quantise_ref(x, "e4m3", 128)
    assert torch.equal(y.cpu(), (codes * scales).bfloat16())
    assert int((c[1] != 0).sum()) == 4 * heads


@pytest.mark.parametrize("page", [1, 7, 16])
@pytest.mark.parametrize("sequences", [0, 1, 3, 100])
def test_cache_slots(page, sequences):
    g = torch.Generator().manual_seed(page + sequences)
    lens = torch.randint(0, 30, (sequences,), generator=g)
    lens[::3] = 0
    offsets = torch.zeros(sequences + 1, dtype=torch.int64)
    offsets[1:] = torch.cumsum(lens, 0)
    offsets += 2                       # two rows in front of the batch
    starts = torch.randint(-3, 40, (sequences,), generator=g)
    width = 50 // page + 1
    tab = torch.randint(-2, 200000000, (sequences, width + 3), generator=g)
    rows = int(offsets[-1]) + 5
    want = [-1] * rows
    for s in range(sequences):
        for r in range(int(offsets[s]), int(offsets[s + 1])):
            p = int(starts[s]) + r - int(offsets[s])
            if p >= 0 and p // page < width and int(tab[s, p // page]) >= 0:
                want[r] = int(tab[s, p // page]) * page + p % page
    i32 = dict(dtype=torch.int32, device="cuda")
    got = mt.cache_slots(tab.to(**i32)[:, :width], offsets.to(**i32),
                         starts.to(**i32), page, rows)
    assert got.dtype == torch.int64 and got.tolist() == want


def test_cache_refuses_on_the_device():
    x = torch.zeros(4, 2, 16, dtype=torch.bfloat16, device="cuda")
    c = mt.cache_alloc(8, 2, 16)
    s = torch.arange(4, device="cuda")
    with pytest.raises(ValueError, match="together"):
        mt.cache_write(x, x, c, None, s)
    with pytest.raises(ValueError):
        mt.cache_write(x[:3], None, c, None, s)
    with pytest.raises(TypeError):
        mt.cache_write(x, None, c, None, s.to(torch.int32))
    with pytest.raises(TypeError, match="codes"):
        mt.cache_write(x, None, (c[0].view(torch.uint8), c[1]), None, s)
    with pytest.raises(TypeError):
        mt.cache_write(x, None, (c[0], c[1].half()), None, s)
    with pytest.raises(ValueError, match="scales"):
        mt.cache_write(x, None, (c[0], c[1].expand(8, 2, 3)), None, s)
    with pytest.raises(ValueError, match="contiguous"):
        mt.cache_write(x, None, (c[0][::2], c[1][::2]), None, s)
    with pytest.raises(mt.MTError):   # output rows overlap
        mt.cache_read(c, None, s, out=x[:1].expand(4, -1, -1))
    with pytest.raises(TypeError):
        mt.cache_read(c, None, s, dtype=torch.float64)


# ---- logits -----------------------------------------------------------------
def logits_inputs(seed, rows, vocab, history=0, biases=0, mask=False,
                  dtype=torch.float32):
    g = gen(seed)
    kw = {}
    x = (3 * randn(g, rows, vocab)).to(dtype)
    uni = lambda *s: torch.rand(s, generator=g, device="cuda")  # noqa: E731
    if history:
        ids = (uni(rows, history) ** 3 * (vocab + 4)).int() - 2
        kw = dict(tokens=ids,
                  lengths=(uni(rows) * (history + 1)).int(),
                  prompt_lengths=(uni(rows) * history).int(),
                  repetition=0.8 + 0.6 * uni(rows),
                  frequency=uni(rows) - 0.3, presence=uni(rows))
    if biases:
        kw["bias_ids"] = (uni(rows, biases) * (vocab + 2)).int() - 1
        kw["bias_ids"][:, biases // 2:] = \
            kw["bias_ids"][:, :biases - biases // 2].flip(1)  # twice
        kw["bias"] = 2 * randn(g, rows, biases)
    if mask:
        words = (vocab + 31) // 32
        kw["mask"] = torch.randint(-2 ** 31, 2 ** 31, (rows, words),
                                   generator=g, device="cuda").int()
    kw["temperature"] = 0.5 + uni(rows)
    return x, kw


def check_logits(x, kw, mode, got, what=""):
    ref, err = logits_ref(x, mode=mode, **kw)
    check(got, ref, err + half_step(torch.nan_to_num(
        ref, nan=0.0, posinf=0.0, neginf=0.0), x.dtype), what or mode)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("mode", ["logits", "softmax", "log_softmax"])
@pytest.mark.parametrize("rows,vocab,history,biases,mask", [
    (1, 1, 1, 1, True), (2, 2, 3, 2, True), (3, 7, 20, 0, True),
    (2, 31, 0, 4, True), (2, 32, 5, 0, True), (2, 33, 5, 3, True),
    (1, 1000, 0, 0, False), (5, 4099, 700, 33, True), (3, 32000, 2000, 300, True),
    (2, 50257, 4000, 17, True), (1, 131072, 1, 1, True),
    (300, 511, 64, 8, True), (1, 262144, 3000, 1024, False),
])
def test_process_logits(dt, mode, rows, vocab, history, biases, mask):
    dtype = DTYPES[dt]
    x, kw = logits_inputs(rows + vocab, rows, vocab, history, biases, mask,
                          dtype)
    y = mt.process_logits(x, mode=mode, **kw)
    check_logits(x, kw, mode, y)
    assert torch.equal(y, mt.process_logits(x, mode=mode, **kw))
    z = x.clone()
    assert mt.process_logits(z, mode=mode, out=z, **kw) is z
    assert torch.equal(z, y)


@pytest.mark.parametrize("mode", ["logits", "softmax", "log_softmax"])
@pytest.mark.parametrize("parts", [
    ("tokens", "repetition"), ("tokens", "lengths", "frequency"),
    ("tokens", "presence", "prompt_lengths"), ("tokens",),
    ("bias_ids", "bias"), ("mask",), ("temperature",), (),
    ("tokens", "repetition", "mask")])
def test_process_logits_each_part_alone(mode, parts):
    x, kw = logits_inputs(31, 4, 5003, 300, 20, True, torch.bfloat16)
    kw = {n: kw[n] for n in parts}
    check_logits(x, kw, mode, mt.process_logits(x, mode=mode, **kw))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [100, 32000, 131077])
def test_process_logits_masks(dt, vocab):
    """Rows of which nothing, one token or everything is left; NaN, infinities
    and the type's lowest value in masked places; -inf and the lowest value
    in allowed ones."""
    dtype = DTYPES[dt]
    x, _ = logits_inputs(32, 6, vocab, dtype=dtype)
    words = (vocab + 31) // 32
    mask = torch.zeros(6, words + 3, dtype=torch.int32, device="cuda")
    mask[1, (vocab - 1) // 32] = 1 << ((vocab - 1) % 32) \
        if (vocab - 1) % 32 < 31 else -2 ** 31
    mask[2] = -1
    mask[3, 0] = 0b1011
    mask[4:] = -1
    x[0] = math.nan
    x[1, 0] = math.inf
    x[3, 2] = math.nan
    x[3, 4] = math.inf
    x[3, 5] = torch.finfo(dtype).min
    x[4, :vocab - 1] = -math.inf
    x[5] = torch.finfo(dtype).min
    for mode in ("logits", "softmax", "log_softmax"):
        y = mt.process_logits(x, mask=mask, mode=mode)
        check_logits(x, dict(mask=mask), mode, y, f"{mode} masks")
    assert bool((mt.process_logits(x, mask=mask, mode="softmax")[0] == 0).all())
    # one mask for all rows
    y = mt.process_logits(x[2:4], mask=mask[3], mode="softmax")
    check_logits(x[2:4], dict(mask=mask[3]), "softmax", y, "shared mask")


def test_process_logits_nan_and_infinity_where_allowed():
    x, _ = logits_inputs(33, 3, 40000)
    x[0, 39999] = math.nan
    x[1, 5] = math.inf
    p = mt.process_logits(x, mode="softmax")
    assert bool(torch.isnan(p[:2]).all())
    check_logits(x[2:], {}, "softmax", p[2:])
    z = mt.process_logits(x)
    assert torch.equal(torch.nan_to_num(z), torch.nan_to_num(x))


@pytest.mark.parametrize("mode", ["softmax", "log_softmax"])
@pytest.mark.parametrize("vocab", [100, 5003, 131072])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_process_logits_nan_rows_are_nan_as_a_whole(mode, vocab, value):
    """One NaN (or +infinity, whose softmax is NaN) that the mask leaves, most
    of the row masked out: every value of that row is NaN, no other row's."""
    x, _ = logits_inputs(39, 3, vocab)
    x[1, vocab - 2] = value
    mask = torch.zeros(3, (vocab + 31) // 32, dtype=torch.int32,
                       device="cuda")
    mask[:, 0] = 0b110
    at = vocab - 2
    mask[:, at // 32] |= 1 << (at % 32) if at % 32 < 31 else -2 ** 31
    y = mt.process_logits(x, mask=mask, mode=mode)
    assert bool(torch.isnan(y[1]).all())
    check_logits(x[::2], dict(mask=mask[::2].contiguous()), mode, y[::2])


@pytest.mark.parametrize("dt", ["f32", "f16"])
@pytest.mark.parametrize("mode", ["logits", "softmax"])
def test_process_logits_strided_rows(dt, mode):
    """Rows of a padded matrix, odd strides, outputs of another phase; the
    padding stays as it is."""
    dtype = DTYPES[dt]
    for vocab, stride, ostride, off in ((1001, 1003, 1009, 0),
                                        (32000, 32003, 32000, 1),
                                        (129, 136, 131, 3)):
        x, kw = logits_inputs(34, 5, vocab, 40, 6, True, dtype)
        buf = torch.full((off + 5 * stride,), math.nan, dtype=dtype,
                         device="cuda")
        xs = torch.as_strided(buf, (5, vocab), (stride, 1), off)
        xs.copy_(x)
        out = torch.full((8 + 5 * ostride,), -77.0, dtype=dtype,
                         device="cuda")
        ys = torch.as_strided(out, (5, vocab), (ostride, 1), 5)
        mt.process_logits(xs, mode=mode, out=ys, **kw)
        check_logits(x, kw, mode, ys)
        keep = out.clone()
        torch.as_strided(keep, (5, vocab), (ostride, 1), 5).fill_(-77.0)
        assert bool((keep == -77.0).all()), "written outside the rows"


def test_process_logits_history_edges():
    """Lengths of zero, below zero and past the end; a prompt longer than the
    history; ids outside the vocabulary; a token 100000 times."""
    x, kw = logits_inputs(35, 6, 700, 50)
    kw["lengths"] = torch.tensor([0, -5, 1000, 50, 1, 50], dtype=torch.int32,
                                 device="cuda")
    kw["prompt_lengths"] = torch.tensor([0, 3, 1000, -2, 1, 50],
                                        dtype=torch.int32, device="cuda")
    kw["tokens"][2] = -2 ** 31
    kw["tokens"][3] = 2 ** 31 - 1
    check_logits(x, kw, "logits", mt.process_logits(x, **kw))
    ids = torch.full((1, 100003), 5, dtype=torch.int32, device="cuda")
    freq = torch.full((1,), 2.0 ** -10, device="cuda")
    y = mt.process_logits(x[:1], tokens=ids, frequency=freq)
    want = float(x[0, 5].double()) - 100003 * 2.0 ** -10
    assert abs(float(y[0, 5]) - want) <= 4 * 2.0 ** -24 * 100
    assert torch.equal(y[0, :5], x[0, :5]) and torch.equal(y[0, 6:], x[0, 6:])
    none = torch.zeros(6, 0, dtype=torch.int32, device="cuda")
    assert torch.equal(mt.process_logits(x, tokens=none), x)


def test_process_logits_temperatures():
    x, _ = logits_inputs(36, 7, 300)
    t = torch.tensor([0.0, -1.0, math.nan, 1e-42, 2.0, math.inf, 1e-3],
                     device="cuda")
    y = mt.process_logits(x, temperature=t)
    assert torch.equal(y[:3], x[:3])
    check_logits(x[4:5], dict(temperature=t[4:5]), "logits", y[4:5])
    check_logits(x[6:], dict(temperature=t[6:]), "logits", y[6:])
    assert torch.equal(y[5], x[5] * 2.0 ** -126)
    assert torch.equal(y[3], torch.sign(x[3]) * torch.where(
        x[3].abs() >= 4, math.inf, (x[3].abs() * 2.0 ** 126)))


def test_process_logits_largest_vocabulary():
    x, kw = logits_inputs(37, 2, 524280, 100, 5, True, torch.bfloat16)
    for mode in ("logits", "softmax"):
        y = mt.process_logits(x, mode=mode, **kw)
        check_logits(x, kw, mode, y)


def test_process_logits_more_than_2_31_values():
    rows, vocab = 17000, 131072
    x = torch.empty(rows, vocab, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=gen(38))
    ids = torch.full((rows, 1), 7, dtype=torch.int32, device="cuda")
    rep = torch.full((rows,), 1.5, device="cuda")
    mt.process_logits(x[:1], tokens=ids[:1], repetition=rep[:1])
    keep = x[[0, 9000, rows - 1]].clone()
    mt.process_logits(x, tokens=ids, repetition=rep, mode="softmax", out=x)
    check_logits(keep, dict(tokens=ids[:3], repetition=rep[:3]), "softmax",
                 x[[0, 9000, rows - 1]])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("mode", ["logits", "softmax", "log_softmax"])
@pytest.mark.parametrize("rows,vocab,history,biases,mask", [
    (1300, 32000, 300, 20, True), (700, 33008, 0, 0, False),
    (400, 131072, 2500, 3, True), (5000, 4008, 40, 0, False)])
def test_process_logits_many_rows(dt, mode, rows, vocab, history, biases,
                                  mask):
    """More rows than the device holds at once: some against the 64-bit form
    (rows masked out as a whole among them), others against a call on few
    rows, which shares a row out between more CTAs; then in place."""
    x, kw = logits_inputs(rows, rows, vocab, history, biases, mask,
                          DTYPES[dt])
    if mask:
        kw["mask"][5] = 0
        kw["mask"][rows - 2] = 0
    y = mt.process_logits(x, mode=mode, **kw)
    for r in (0, 5, rows // 2, rows - 2, rows - 1):
        one = {n: t[r:r + 1].contiguous() for n, t in kw.items()}
        check_logits(x[r:r + 1], one, mode, y[r:r + 1], f"row {r}")
    for lo in range(0, rows, 97):
        some = {n: t[lo:lo + 3].contiguous() for n, t in kw.items()}
        z = mt.process_logits(x[lo:lo + 3], mode=mode, **some)
        if mode == "logits":  # the same FP32 steps
            assert torch.equal(y[lo:lo + 3], z)
            continue
        # Each is within |d| 2^-22 (the exponent's roundings) + 200 U (the
        # sum's) of the exact value, relative for a softmax and absolute for
        # its logarithm, d the distance to the row's maximum: |d| <= |ln p|,
        # since the sum is at least 1.  Twice that, and a step of storage.
        z = z.double()
        log = z if mode == "log_softmax" else torch.log(z)
        off = 2 * (torch.nan_to_num(log, neginf=0.0).abs() * 2.0 ** -22 +
                   200 * 2.0 ** -24)
        size = torch.nan_to_num(z, neginf=0.0).abs()
        check(y[lo:lo + 3], z, (off if mode == "log_softmax" else off * size) +
              torch.finfo(x.dtype).eps * size + 1e-37, f"rows from {lo}")
    w = x.clone()
    mt.process_logits(w, mode=mode, out=w, **kw)
    assert torch.equal(w, y)


def test_process_logits_refuses_on_the_device():
    x = torch.zeros(2, 100, device="cuda")
    ids = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    f = torch.zeros(2, device="cuda")
    bad = [dict(repetition=f), dict(bias=f[:, None]),
           dict(tokens=ids, repetition=f[:1]), dict(tokens=ids[:1]),
           dict(tokens=ids.t().contiguous().t()), dict(mode="argmax"),
           dict(mask=ids), dict(mask=ids.repeat(2, 2)),
           dict(bias_ids=ids, bias=f[:, None]), dict(temperature=f[:1])]
    for kw in bad:
        with pytest.raises(ValueError):
            mt.process_logits(x, **kw)
    for kw in (dict(tokens=ids.long()), dict(tokens=ids, repetition=f.half()),
               dict(mask=ids.float()), dict(out=x.half())):
        with pytest.raises(TypeError):
            mt.process_logits(x, **kw)
    with pytest.raises(mt.MTError):
        mt.process_logits(x, out=x[:1].expand(2, -1))
    with pytest.raises(mt.MTError):
        mt.process_logits(torch.zeros(1, 524281, device="cuda"))


def test_calls_with_nothing_to_do():
    """Empty batches: outputs of the right shapes, nothing written."""
    _, _, tab = table(16)
    q = torch.empty(0, 2, 16, dtype=torch.bfloat16, device="cuda")
    pos = torch.empty(0, dtype=torch.int64, device="cuda")
    y, z = mt.rotary(q, q[:, :1], pos, tab, eps=1e-6)
    assert y.shape == (0, 2, 16) and z.shape == (0, 1, 16)
    c = mt.cache_alloc(4, 2, 16)
    s = torch.empty(0, dtype=torch.int64, device="cuda")
    mt.cache_write(q, q, c, mt.cache_alloc(4, 2, 16), s)
    assert mt.cache_read(c, None, s).shape == (0, 2, 16)
    none = mt.cache_alloc(0, 2, 16)         # a cache without slots
    x = torch.ones(3, 2, 16, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1, -1], device="cuda")
    mt.cache_write(x, None, none, None, at)
    assert bool((mt.cache_read(none, None, at) == 0).all())
    e = torch.empty(0, 50, device="cuda")
    for mode in ("logits", "softmax"):
        assert mt.process_logits(e, mode=mode, tokens=torch.empty(
            0, 4, dtype=torch.int32, device="cuda")).shape == (0, 50)
    t = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    o = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert mt.cache_slots(t, o, o[:0], 16, 2).tolist() == [-1, -1]


@pytest.mark.parametrize("norm", [False, True])
def test_rotary_keys_alone_and_more_keys_than_queries(norm):
    q, k, pos, wq, wk = rot_inputs(17, 30, 1, 9, 32, torch.bfloat16)
    freqs, scale, tab = table(32)
    kw = dict(eps=1e-6) if norm else {}
    eps = 1e-6 if norm else None
    for a in (q, q[:, :0]):  # one query head, none
        y, z = mt.rotary(a, k, pos, tab, **(
            dict(kw, q_weight=wq, k_weight=wk) if norm else {}))
        ref, err = rotary_ref(k, pos, freqs, scale, 32, False,
                              wk if norm else None, eps)
        check(z, ref, err + half_step(ref, torch.bfloat16))
        assert y.shape == a.shape
        g = mt.rotary_backward(a, k, pos, tab, **(
            dict(kw, q=a, k=k, q_weight=wq, k_weight=wk) if norm else {}))
        dx, err, dw, werr = rotary_backward_ref(
            k, k, pos, freqs, scale, 32, False, wk, eps)
        check(g[1], dx, err + half_step(dx, torch.bfloat16))
        if norm:
            check(g[3], dw, werr)
            if a.shape[1] == 0:
                assert bool((g[2] == 0).all())


@pytest.mark.parametrize("norm", [False, True])
def test_rotary_backward_with_a_scale(norm):
    """The factor of a scaled rotation, part of a head, float32."""
    f, s = mt.mt_rotary_frequencies(24, 10000.0, mt.MtRotaryScaling(
        type=mt.MT_ROTARY_YARN, factor=4.0, original_length=64.0, low=1.0,
        high=32.0))
    tab = mt.rotary_frequencies(24, scaling=dict(
        type="yarn", factor=4.0, original_length=64))
    q, _, pos, wq, _ = rot_inputs(18, 13, 2, 1, 40, torch.float32)
    dq, _, _, _, _ = rot_inputs(19, 13, 2, 1, 40, torch.float32)
    kw = dict(q=q, q_weight=wq, eps=1e-6) if norm else {}
    g = mt.rotary_backward(dq, None, pos, tab, interleaved=True, **kw)
    dx, err, dw, werr = rotary_backward_ref(
        dq, q, pos, f, s, 24, True, wq, 1e-6 if norm else None)
    check(g[0], dx, err + half_step(dx, torch.float32))
    if norm:
        check(g[2], dw, werr)


def test_rotary_rows_of_zeros_without_eps():
    """eps = 0: a zero row is 0/0, and no head that is not there adds a NaN to
    the weight's gradient."""
    q, _, pos, wq, _ = rot_inputs(20, 9, 3, 1, 32, torch.float32)
    freqs, scale, tab = table(32)
    g = mt.rotary_backward(q, None, pos, tab, q=q, q_weight=wq, eps=0.0)
    dx, err, dw, werr = rotary_backward_ref(q, q, pos, freqs, scale, 32,
                                            False, wq, 0.0)
    check(g[0], dx, err + half_step(dx, torch.float32))
    check(g[2], dw, werr)


@pytest.mark.parametrize("rows,vocab,history", [
    (3, 200, 30000), (1, 64, 5000), (40, 1000, 2047), (2, 9000, 33333)])
def test_process_logits_long_histories_of_small_vocabularies(rows, vocab,
                                                            history):
    """Every CTA's queue fills and drains many times; counts stay exact (a
    frequency of 2^-12 makes the sums exact in FP32)."""
    x, kw = logits_inputs(rows + history, rows, vocab, history, 40, True)
    kw["frequency"] = torch.full((rows,), 2.0 ** -12, device="cuda")
    for mode in ("logits", "softmax"):
        y = mt.process_logits(x, mode=mode, **kw)
        check_logits(x, kw, mode, y)


# ---- streams, graphs, together -----------------------------------------------
def test_other_stream_and_large_offsets():
    """Work on a stream of its own; more than 2^31 values of rows."""
    tokens, heads, dim = 600_000, 30, 128
    x = torch.empty(tokens, heads, dim, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=gen(40))
    assert x.numel() > 2 ** 31
    pos = torch.arange(tokens, device="cuda")
    freqs, scale, tab = table(128)
    keep = x[[0, 300_000, tokens - 1]].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mt.rotary(x, None, pos, tab, out=x, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    ref, err = rotary_ref(keep, pos[[0, 300_000, tokens - 1]], freqs, scale,
                          128, False, None, None)
    check(x[[0, 300_000, tokens - 1]], ref,
          err + half_step(ref, torch.bfloat16))
    # the stream as a raw handle, 0 for the default stream
    z = mt.process_logits(torch.ones(2, 10, device="cuda"), stream=0)
    torch.cuda.synchronize()
    assert bool((z == 1).all())
    y = mt.process_logits(torch.ones(2, 10, device="cuda"), mode="softmax",
                          stream=s.cuda_stream)
    s.synchronize()
    check(y, torch.full((2, 10), 0.1, dtype=torch.float64), 1e-6)


def test_a_decode_step_of_the_operators_together():
    """norm -> projection -> heads normed and turned -> cache -> attention
    over what the cache holds -> add and norm -> logits -> probabilities,
    each stage held against its 64-bit form on what the stage before gave;
    then the step captured into a graph and replayed on new inputs."""
    g = gen(50)
    B, E, HQ, HK, D, V, PAGE, LONG = 5, 256, 8, 2, 64, 5000, 16, 40
    dt = torch.bfloat16
    wn, wo = (1 + 0.1 * randn(g, E)).to(dt), (1 + 0.1 * randn(g, E)).to(dt)
    wqkv = (randn(g, E, (HQ + 2 * HK) * D) / 16).to(dt)
    wout = (randn(g, HQ * D, E) / 22).to(dt)
    whead = (randn(g, E, V) / 16).to(dt)
    wq, wk = (1 + 0.1 * randn(g, D)).to(dt), (1 + 0.1 * randn(g, D)).to(dt)
    freqs, scale, tab = table(D)
    pages = 5 * B
    caches = [mt.cache_alloc(pages * PAGE, HK, D, 32, f)
              for f in ("e4m3", "int8")]
    ptab = torch.randperm(pages, generator=g, device="cuda").int().view(B, 5)
    lens = torch.tensor([0, 1, 15, 16, LONG], dtype=torch.int32,
                        device="cuda")
    # what the sequences hold so far
    offs = torch.cat((torch.zeros(1, dtype=torch.int32, device="cuda"),
                      torch.cumsum(lens, 0).int()))
    n = int(offs[-1])
    old = mt.cache_slots(ptab, offs, torch.zeros_like(lens), PAGE, n)
    mt.cache_write(randn(g, n, HK, D, dtype=dt), None, caches[0], None, old)
    mt.cache_write(randn(g, n, HK, D, dtype=dt), None, caches[1], None, old)
    x = randn(g, B, E, dtype=dt)
    ids = torch.randint(0, V, (B, 30), generator=g, device="cuda").int()
    rep = 1 + 0.5 * torch.rand(B, generator=g, device="cuda")
    mask = torch.randint(-2 ** 31, 2 ** 31, (B, (V + 31) // 32), generator=g,
                         device="cuda").int()
    one = torch.arange(B + 1, device="cuda").int()
    width = LONG + 1
    all_offs = (torch.arange(B + 1, device="cuda") * width).int()
    zeros = torch.zeros_like(lens)

    def step():
        t = {}
        t["h"] = mt.rmsnorm(x, wn)
        t["qkv"] = (t["h"] @ wqkv).view(B, HQ + 2 * HK, D)
        q, k, v = t["qkv"].split((HQ, HK, HK), 1)
        t["q"], t["k"] = mt.rotary(q, k, lens, tab, q_weight=wq, k_weight=wk,
                                   eps=1e-6)
        slots = mt.cache_slots(ptab, one, lens, PAGE, B)
        mt.cache_write(t["k"], None, caches[0], None, slots)
        mt.cache_write(v, None, caches[1], None, slots)
        at = mt.cache_slots(ptab, all_offs, zeros, PAGE, B * width)
        t["K"] = mt.cache_read(caches[0], None, at)
        t["V"] = mt.cache_read(caches[1], None, at)
        K = t["K"].view(B, width, HK, D).repeat_interleave(HQ // HK, 2)
        W = t["V"].view(B, width, HK, D).repeat_interleave(HQ // HK, 2)
        s = torch.einsum("bhd,blhd->bhl", t["q"].float(), K.float()) / 8
        s = s.masked_fill((torch.arange(width, device="cuda") >
                           lens[:, None])[:, None], -math.inf)
        p = mt.softmax(s.reshape(B * HQ, width)).view(B, HQ, width)
        o = torch.einsum("bhl,blhd->bhd", p, W.float()).to(dt)
        t["o"] = o.reshape(B, HQ * D) @ wout
        t["y"], t["r"] = mt.residual_rmsnorm(t["o"], x, wo, return_h=True)
        t["logits"] = t["y"] @ whead
        t["p"] = mt.process_logits(t["logits"], tokens=ids, repetition=rep,
                                   mask=mask, mode="softmax")
        return t

    def verify(t):
        q, k, v = t["qkv"].split((HQ, HK, HK), 1)
        for a, y, w in ((q, t["q"], wq), (k, t["k"], wk)):
            ref, err = rotary_ref(a, lens, freqs, scale, D, False, w, 1e-6)
            check(y, ref, err + half_step(ref, dt), "rotary")
        for name, fmt, new in (("K", "e4m3", t["k"]), ("V", "int8", v)):
            held = t[name].view(B, width, HK, D)
            codes, scales = quantise_ref(new, fmt, 32)
            want = (codes.unflatten(-1, (2, 32)) * scales[..., None]).flatten(
                -2).to(dt)
            for b in range(B):
                assert torch.equal(held[b, int(lens[b])].cpu(), want[b])
        check_logits(t["logits"], dict(tokens=ids, repetition=rep, mask=mask),
                     "softmax", t["p"])
        allowed = (mask[:, torch.arange(V) >> 5].cpu() >>
                   (torch.arange(V) & 31)) & 1
        assert bool((t["p"].cpu()[allowed == 0] == 0).all())

    eager = step()
    verify(eager)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    graph.replay()
    torch.cuda.synchronize()
    for name in ("q", "k", "p"):
        assert torch.equal(held[name], eager[name]), name
    x.copy_(randn(g, B, E, dtype=dt))
    graph.replay()
    torch.cuda.synchronize()
    verify(held)
    assert not torch.equal(held["p"], eager["p"])


def test_training_pass_captured():
    """Forward and backward captured with their workspace, replayed twice on
    new inputs; two graphs hold workspaces of their own."""
    q, k, pos, wq, wk = rot_inputs(60, 500, 4, 2, 64, torch.float32)
    dq, dk, _, _, _ = rot_inputs(61, 500, 4, 2, 64, torch.float32)
    q, k, dq, dk = (t.contiguous() for t in (q, k, dq, dk))
    _, _, tab = table(64)

    def both():
        kw = dict(q_weight=wq, k_weight=wk, eps=1e-6)
        return (*mt.rotary(q, k, pos, tab, **kw),
                *mt.rotary_backward(dq, dk, pos, tab, q=q, k=k, **kw))
    both()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = both()
        graphs.append((graph, outs))
    for seed in (62, 63):
        nq, nk, _, _, _ = rot_inputs(seed, 500, 4, 2, 64, torch.float32)
        q.copy_(nq)
        k.copy_(nk)
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for (graph, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        want = both()
        for _, outs in graphs:
            for a, b in zip(outs, want):
                assert torch.equal(a, b)


def test_calls_from_several_threads():
    from concurrent.futures import ThreadPoolExecutor
    x, kw = logits_inputs(70, 4, 40000, 100, 5, True, torch.bfloat16)
    want = mt.process_logits(x, mode="softmax", **kw)
    q, k, pos, wq, wk = rot_inputs(71, 50, 4, 2, 64, torch.bfloat16)
    _, _, tab = table(64)
    turned = mt.rotary(q, k, pos, tab)
    torch.cuda.synchronize()

    def work(_):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            outs = [(mt.process_logits(x, mode="softmax", **kw),
                     mt.rotary(q, k, pos, tab)) for _ in range(10)]
        s.synchronize()
        return all(torch.equal(a, want) and torch.equal(b[0], turned[0])
                   for a, b in outs)
    with ThreadPoolExecutor(8) as ex:
        assert all(ex.map(work, range(8)))
