"""Edges of the decoder's row operators on a GPU: values and sizes at which a
result can go wrong without a usual input showing it."""
import math

import pytest
import torch

import row_reduction_gb300 as mt
from decoder_util import (DTYPES, NORM, U, angle_error, check, half_step,
                          logits_ref, norm64, pair_sum, rotate)

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ---- logits: lengths of the prompt ---------------------------------------------
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("history", [40, 41, 4096, 4099])
def test_process_logits_prompt_lengths_of_any_value(dt, history):
    """A prompt length below zero is none, one past the history all of it,
    down to the type's bounds, whatever the alignment of the rows of ids."""
    g = gen(history)
    prompts = [-2 ** 31, -2 ** 31 + 1, -history, -1, 0, 3, history,
               history + 1, 2 ** 31 - 1]
    rows, vocab = len(prompts), 300
    x = (3 * torch.randn(rows, vocab, generator=g, device="cuda")).to(
        DTYPES[dt])
    parts = dict(
        tokens=torch.randint(0, vocab, (rows, history), generator=g,
                             device="cuda", dtype=torch.int32),
        prompt_lengths=torch.tensor(prompts, dtype=torch.int32,
                                    device="cuda"),
        frequency=torch.linspace(0.1, 0.9, rows, device="cuda"),
        presence=torch.linspace(0.5, 0.2, rows, device="cuda"))
    ref, err = logits_ref(x, **parts)
    check(mt.process_logits(x, **parts), ref, err + half_step(ref, DTYPES[dt]))


# ---- rotary: gradients of weights -------------------------------------------------
def backward_inputs(seed, tokens, hq, hk, dim, dtype):
    g = gen(seed)

    def t():
        x = torch.randn(tokens, hq + hk, dim, generator=g, device="cuda")
        return x.to(dtype)
    x, dy = t(), t()
    return x[:, :hq], x[:, hq:], dy[:, :hq], dy[:, hq:]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads", [5, 13])
def test_weight_gradients_keep_an_infinity(dt, interleaved, heads):
    """A gradient that holds an infinity gives an infinite gradient of the
    weight there, of its sign, and finite ones elsewhere: the places of a
    warp that stand for no head add nothing.  (Values that pass unrotated, so
    that no product of the rotation is infinity times zero.)"""
    dtype, tokens, dim, rotary = DTYPES[dt], 3000, 64, 32
    q, _, dq, _ = backward_inputs(heads, tokens, heads, 0, dim, dtype)
    q, dq = q.clone(), dq.clone()
    pos = torch.arange(tokens, device="cuda")
    tab = mt.rotary_frequencies(rotary)
    w = torch.ones(dim, dtype=dtype, device="cuda")
    want = {}
    for i in range(12):
        at = (100 + 31 * i, i % heads, rotary + i)
        q[at] = 1.0 + i / 8
        dq[at] = -math.inf if i % 3 else math.inf
        want[rotary + i] = float(dq[at])
    dw = mt.rotary_backward(dq, None, pos, tab, interleaved=interleaved, q=q,
                            q_weight=w, eps=1e-6)[2].tolist()
    assert {d: v for d, v in enumerate(dw) if not math.isfinite(v)} == want


WEIGHT_SHAPES = [
    # tokens, query heads, key heads, dim, rotary_dim: many items per warp,
    # of a number that does not divide evenly; odd, padded and wide heads
    (3001, 5, 3, 64, 64), (2999, 13, 2, 64, 32), (700, 33, 5, 64, 64),
    (6007, 3, 1, 64, 64), (1999, 7, 7, 96, 48), (1003, 9, 1, 128, 128),
    (901, 5, 2, 80, 40), (301, 6, 2, 512, 512), (303, 7, 1, 130, 66),
    (203, 3, 2, 77, 70), (151, 3, 1, 511, 510), (12001, 1, 1, 64, 64),
]


def weight_sum_roundings(tokens, hq, hk):
    """Most roundings on the way of one term into a weight's gradient: a lane
    adds up its warp's items (a token's group of heads, at most one per head;
    a tensor has a part of 304 blocks of 8 warps or more in proportion to its
    groups, rounded down but at least one, so at least half its due), then 5
    exchanges, up to 12 warps, 10 of 304 rows of partial sums, and 32 sums of
    those."""
    items = -(-2 * tokens * (hq + hk) // (304 * 8)) + 1
    return items + 5 + 12 + 10 + 32


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,hq,hk,dim,rotary", WEIGHT_SHAPES)
def test_weight_gradients_add_every_row_once(dt, interleaved, tokens, hq, hk,
                                             dim, rotary):
    """Whole numbers in dy, x of +-1 and position 0 without eps: the mean
    square is 1 (its sum is exact, the mean within one rounding), the factor
    1/sqrt within 2 ulp of 1, the rotation the identity, and every term a
    whole number of 1 or more but for that factor: a row that is left out or
    taken twice shows in every column."""
    dtype = DTYPES[dt]
    g = gen(dim + tokens)
    tab = mt.rotary_frequencies(rotary)
    pos = torch.zeros(tokens, dtype=torch.int32, device="cuda")
    args, want = [], []
    for h in (hq, hk):
        x = torch.randint(0, 2, (tokens, h, dim), generator=g,
                          device="cuda") * 2 - 1
        dy = torch.randint(1, 3, (tokens, h, dim), generator=g,
                           device="cuda") * (torch.randint(
                               0, 2, (tokens, h, dim), generator=g,
                               device="cuda") * 2 - 1)
        args.append((x.to(dtype), dy.to(dtype)))
        want.append(((x * dy).sum((0, 1)), dy.abs().sum((0, 1))))
    ones = torch.ones(dim, dtype=dtype, device="cuda")
    got = mt.rotary_backward(args[0][1], args[1][1], pos, tab,
                             interleaved=interleaved, q=args[0][0],
                             k=args[1][0], q_weight=ones, k_weight=ones,
                             eps=0.0)
    roundings = weight_sum_roundings(tokens, hq, hk)
    for i in range(2):
        ref, size = want[i]
        # 1/sqrt: 2 ulp are 2^-22, half a rounding of the mean, its own; then
        # g r, and the sums where r is not 1 exactly
        tol = size.double() * (2.0 ** -22 + (3 + roundings) * U)
        assert float(tol.max()) < 0.5   # a term is 1 or more
        check(got[2 + i], ref.double(), tol, "dweight")


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,hq,hk,dim,rotary", WEIGHT_SHAPES)
def test_weight_gradients_to_the_longest_sum(dt, interleaved, tokens, hq, hk,
                                             dim, rotary):
    """Random rows, with the error that the longest way of a term into its
    sum allows (however many rows there are)."""
    dtype = DTYPES[dt]
    q, k, dq, dk = backward_inputs(tokens, tokens, hq, hk, dim, dtype)
    pos = torch.randint(0, 8192, (tokens,), generator=gen(1), device="cuda")
    tab = mt.rotary_frequencies(rotary)
    freqs, scale = mt.mt_rotary_frequencies(rotary, 10000.0)
    w = torch.ones(dim, dtype=dtype, device="cuda")
    got = mt.rotary_backward(dq, dk, pos, tab, interleaved=interleaved, q=q,
                             k=k, q_weight=w, k_weight=w, eps=1e-6)
    roundings = weight_sum_roundings(tokens, hq, hk)
    for i, (x, dy) in enumerate(((q, dq), (k, dk))):
        g = rotate(dy, pos, freqs, scale, rotary, interleaved, -1.0)
        xr = norm64(x, None, 1e-6)[0]
        mag = pair_sum(dy, rotary, interleaved, scale) * xr.abs()
        # angle, 1/sqrt and its sum, g r and the term's product, the sums
        tol = mag.sum((0, 1)) * (angle_error(dtype) + NORM +
                                 (3 + roundings) * U)
        terms = (g * xr).sum(1)
        # one token left out would show
        assert bool((terms[-1].abs() > tol).any())
        check(got[2 + i], terms.sum(0), tol, "dweight")


# ---- cache: sizes do not depend on addresses ---------------------------------------
def cache_in(buf, slots, heads, dim, group, off):
    """A cache whose codes start `off` bytes into `buf`."""
    return (buf[off:off + slots * heads * dim].view(slots, heads, dim),
            torch.zeros(slots, heads, dim // group, device="cuda"))


@pytest.mark.parametrize("off", [0, 1])
def test_cache_accepts_the_same_sizes_at_any_address(off):
    """More than 2^32 values of one call, the codes on a 16-byte boundary and
    off it.  (One row of values for all tokens; most have no slot.)"""
    heads, dim, slots = 1024, 1024, 3
    tokens = 4099                               # of 2^20 values
    assert tokens * heads * dim > 2 ** 32
    row = torch.randn(1, heads, dim, generator=gen(1), device="cuda").to(
        torch.bfloat16)
    at = torch.full((tokens,), -1, dtype=torch.int64, device="cuda")
    at[0], at[2050], at[tokens - 1] = 2, 0, 1
    buf = torch.full((slots * heads * dim + 16,), 55, dtype=torch.int8,
                     device="cuda")
    cache = cache_in(buf, slots, heads, dim, 256, off)
    mt.cache_write(row.expand(tokens, -1, -1), None, cache, None, at)
    want = cache_in(torch.zeros_like(buf), slots, heads, dim, 256, 0)
    mt.cache_write(row.expand(3, -1, -1), None, want, None,
                   torch.arange(3, device="cuda"))
    assert torch.equal(cache[0], want[0]) and torch.equal(cache[1], want[1])
    assert bool((buf[:off] == 55).all())
    assert bool((buf[off + slots * heads * dim:] == 55).all())
    # every token reads slot 1, but for a few that keep what was there
    at = torch.full((tokens,), 1, dtype=torch.int64, device="cuda")
    at[0] = at[2050] = -1
    out = torch.full((tokens, heads, dim), 7.0, dtype=torch.bfloat16,
                     device="cuda")
    mt.cache_read(cache, None, at, out=out)
    value = mt.cache_read(want, None, torch.tensor([1], device="cuda"))[0]
    for t in range(0, tokens, 512):
        part = out[t:t + 512]
        keep = (at[t:t + 512] < 0)
        assert bool((part[keep] == 7.0).all())
        assert bool((part[~keep] == value).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_cache_of_many_odd_groups(dt, fmt):
    """Groups of any size, many of them: every row of a call of 2200003 tokens
    against the same rows in calls of 1000."""
    tokens, heads, dim, group = 2_200_003, 3, 10, 5
    dtype = DTYPES[dt]
    g = gen(3)
    base = torch.randn(1000, heads, dim, generator=g, device="cuda").to(dtype)
    x = base.repeat(tokens // 1000 + 1, 1, 1)[:tokens]
    at = torch.randperm(tokens, generator=g, device="cuda")
    k, v = (mt.cache_alloc(tokens, heads, dim, group, fmt) for _ in range(2))
    mt.cache_write(x, -x, k, v, at)
    few = [mt.cache_alloc(1000, heads, dim, group, fmt) for _ in range(2)]
    rows = torch.arange(1000, device="cuda")
    mt.cache_write(base, -base, *few, rows)
    kr, vr = mt.cache_read(k, v, at, dtype=dtype)
    fk, fv = mt.cache_read(*few, rows, dtype=dtype)
    of = torch.arange(tokens, device="cuda") % 1000
    assert torch.equal(kr, fk[of]) and torch.equal(vr, fv[of])
    assert torch.equal(k[1][at], few[0][1][of])
