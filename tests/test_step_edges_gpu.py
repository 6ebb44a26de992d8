"""Edges of the operators around a decoder's cache on a GPU: what their calls
allow and few callers use, against the plain 64-bit forms."""
import pytest
import torch

import row_reduction_gb300 as mt
from decoder_util import DTYPES, U, check, half_step
from step_util import attention_ref, block_norm_back_ref
from test_step_gpu import attention_inputs, gen, i32, randn

pytestmark = pytest.mark.gpu

CODES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


# ---- attention over the cache ------------------------------------------------
@pytest.mark.parametrize("dt,dim,group", [
    ("bf16", 128, 128), ("bf16", 128, 64), ("f16", 64, 64), ("f32", 96, 96),
    ("bf16", 40, 40)])
@pytest.mark.parametrize("rows", [(3, 5), (100, 130), (400, 300)], ids=str)
@pytest.mark.parametrize("kind", ["last", "both", "window"])
def test_rows_before_position_zero_see_nothing(dt, dim, group, rows, kind):
    """... with bounds of their own too, which would let them see keys."""
    batch = [(rows[0], rows[0] - 2), (rows[1], rows[1] // 2), (4, 60)]
    a = attention_inputs(dim, batch, 4, 1, dim, group, 16, "e4m3", DTYPES[dt])
    n = sum(r for r, _ in batch)
    p = torch.cat([torch.arange(k - r, k) for r, k in batch])
    last = torch.where(p % 3 == 0, p + 40, 2)
    kw = {}
    if kind == "both":
        kw["first"] = i32(torch.where(p % 5 == 0, p, -1).tolist())
    if kind == "window":
        kw["window"] = 50
    out = torch.full(a["q"].shape, 7.0, dtype=a["q"].dtype, device="cuda")
    got, lse = mt.cache_attention(
        a["q"], a["k_cache"], a["v_cache"], a["table"], a["offsets"],
        a["starts"], 16, out=out, return_lse=True, last=i32(last.tolist()),
        **kw)
    assert bool((got[p < 0] == 0).all())
    assert bool((lse[p < 0] == -torch.inf).all())
    # the same as with bounds that let those rows see nothing
    ref, err, rlse, lerr, there = attention_ref(
        a["q"], a["k_cache"], a["v_cache"], a["table"], a["offsets"],
        a["starts"], 16, last=i32(torch.where(p < 0, -1, last).tolist()), **kw)
    assert bool(there.all()) and len(there) == n
    check(got, ref, err + half_step(ref, got.dtype), "out")
    check(lse, rlse, lerr + torch.nan_to_num(rlse, neginf=0.0).abs() * 2e-7,
          "lse")


def capped_ref(a, cap, scale):
    """(out, its bound, lse, its bound) of a causal batch with capped scores.

    The bound is attention_ref's but for the cap, by which a score is off by 36
    roundings of what it becomes and no multiple of the cap: towards 0 the series
    by 4 (t 3, which moves it by a sixth of that and less, Horner's scheme 2, the
    last product, and 0.2 left out); from |t| = 1/4 on, where the value is 0.24
    cap or more, sech^2(t) / 2 times the exponential's 4 + 6 |t|, which it makes
    of 3 in its argument and its own 2^-22, and 2 / (1 + e^2t) times 3 (the sum,
    the reciprocal), 6.3 of cap together at t = -1/4, where they are most of the
    value, 2 of cap for the sum with what the score is compared with, and 2 of
    the value for cap log2(e) and the last sum."""
    q, page = a["q"], a["page"]
    dim, times = q.shape[2], q.shape[1] // a["k_cache"][0].shape[1]
    part = 2.0 ** -11 if q.dtype == torch.bfloat16 else 2.0 ** -22
    outs = []
    offs = a["offsets"].tolist()
    for s, start in enumerate(a["starts"].tolist()):
        r0, r1 = offs[s], offs[s + 1]
        j = torch.arange(start + r1 - r0, device="cuda")
        slot = a["table"][s].long()[j // page] * page + j % page
        k, v = ((c.view(torch.int8)[slot].view(c.dtype).float().double() *
                 x[slot].double().repeat_interleave(dim // x.shape[-1], -1))
                .repeat_interleave(times, 1)
                for c, x in (a["k_cache"], a["v_cache"]))
        x = q[r0:r1].double()
        see = (j <= start + torch.arange(r1 - r0, device="cuda")[:, None])[
            :, None]
        z = scale * torch.einsum("rhd,jhd->rhj", x, k)
        dz = scale * torch.einsum("rhd,jhd->rhj", x.abs(), k.abs()) * \
            ((dim / 16 + 5) * 2.0 ** -22 + 2.0 ** -22 + 6 * U) + \
            scale * x.abs().amax(-1)[..., None] * k.abs().sum(-1).T[None] * \
            2.0 ** -39
        z = cap * torch.tanh(z / cap)
        dz = torch.where(see, dz + 36 * U * z.abs(), 0.0)
        z = torch.where(see, z, -torch.inf)
        w, top = z.softmax(-1), z.amax(-1)
        dw = dz + torch.where(see, (z - top[..., None]).abs(), 0.0) * 2.0 ** -23
        most = dw.amax(-1)
        n = len(j)
        # (values as attention_inputs makes them: nothing near the smallest)
        outs.append((
            torch.einsum("rhj,jhd->rhd", w, v),
            torch.einsum("rhj,jhd->rhd", w, v.abs()) *
            (2 * most[..., None] + part + 2.0 ** -20 + (n + 8) * U) +
            n * 2.0 ** -37 * v.abs().amax(),
            torch.logsumexp(z, -1),
            most + 2.0 ** -20 + (n + 8) * U + 4 * U * top.abs()))
    return [torch.cat(t) for t in zip(*outs)]


@pytest.mark.parametrize("cap", [0.02, 1.0, 7.0, 50.0, 1e3, 1e5, 1e8, 1e30,
                                 3e38])
@pytest.mark.parametrize("dt,dim,group,rows", [
    ("f32", 128, 64, 1), ("f16", 64, 64, 1), ("bf16", 128, 128, 3),
    ("f32", 96, 96, 90), ("f16", 128, 32, 90), ("bf16", 64, 32, 90),
    ("bf16", 128, 128, 300), ("bf16", 64, 64, 300), ("f32", 40, 8, 5),
    ("bf16", 72, 72, 5)])
def test_capped_scores(cap, dt, dim, group, rows):
    """Caps from far below the scores to far above them, where they change
    nothing."""
    a = attention_inputs(dim + rows, [(rows, rows + 330), (rows, rows)], 4, 1,
                         dim, group, 16, "e4m3", DTYPES[dt])
    out, lse = mt.cache_attention(
        a["q"], a["k_cache"], a["v_cache"], a["table"], a["offsets"],
        a["starts"], 16, cap=cap, return_lse=True)
    ref, err, rlse, lerr = capped_ref(a, cap, dim ** -0.5)
    check(out, ref, err + half_step(ref, out.dtype), "out")
    check(lse, rlse, lerr + rlse.abs() * 2e-7, "lse")


@pytest.mark.parametrize("cap", [1.0, 50.0, 1e4])
def test_capped_scores_across_the_bend(cap):
    """Scores all along the curve, both signs, in one chunk and in chunks of
    their own: one key apart from the rest of a head, two keys."""
    n, dim = 257, 64
    t = torch.linspace(-12, 12, n, device="cuda")
    t[::7] = torch.linspace(-0.26, 0.26, len(t[::7]), device="cuda")
    kc, vc = (mt.cache_alloc(2 * n, 1, dim) for _ in range(2))
    key = torch.zeros(2 * n, 1, dim, device="cuda")
    key[0::2, 0, 0] = t        # a sequence of two keys: z_1 and 0
    value = torch.zeros_like(key)
    value[0::2] = 1.0
    mt.cache_write(key, value, kc, vc, torch.arange(2 * n, device="cuda"))
    q = torch.zeros(n, 1, dim, device="cuda")
    q[:, 0, 0] = 1.0
    table = torch.arange(n, dtype=torch.int32, device="cuda")[:, None]
    ones = torch.ones(n, dtype=torch.int32, device="cuda")
    offsets = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    _, lse = mt.cache_attention(q, kc, vc, table, offsets, ones, 2, scale=cap,
                                cap=cap, return_lse=True)
    held = mt.cache_read(kc, None, torch.arange(2 * n, device="cuda"),
                         dtype=torch.float32)[0::2, 0, 0].double()
    z = cap * torch.tanh(held)
    want = torch.logaddexp(z, torch.zeros_like(z))
    # 6 roundings of the score before the cap (its slope is at most 1), 36 of
    # what it becomes; the sum's and the logarithm's as in attention_ref
    tol = (6 * cap * held.abs() / torch.cosh(held).square() + 36 * z.abs() +
           4 * want.abs()) * U + 2.0 ** -20 + 10 * U + want.abs() * 2e-7
    check(lse[:, 0], want, tol, "lse")


# ---- norms around a block ----------------------------------------------------
def back_call(c, dtype):
    """The C call, on a workspace of the size that it asks for."""
    n = mt.mt_block_norm_backward_workspace(CODES[dtype], c)
    room = torch.empty(n, dtype=torch.uint8, device="cuda")
    mt.mt_block_norm_backward(CODES[dtype], c, room.data_ptr() if n else None,
                              n, torch.cuda.current_stream().cuda_stream)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 2, 5, 200, 700])
@pytest.mark.parametrize("cols", [8, 7, 256, 1024, 1235, 2048, 4096, 8190,
                                  16384, 40001])
def test_backward_keeps_to_its_workspace(dt, rows, cols):
    """Every way that rows go, with as many bytes as the call asks for."""
    if rows * cols > 4_000_000:
        rows = 4_000_000 // cols
    dtype, g = DTYPES[dt], gen(rows + cols)
    dy, x, h = (randn(g, rows, cols, dtype=dtype) for _ in range(3))
    gate, w, w2 = (randn(g, cols, dtype=dtype) for _ in range(3))
    dx, dres = torch.empty_like(dy), torch.empty_like(dy)
    sums = torch.empty(3, cols, device="cuda")
    c = mt.MtBlockNormBack(
        dy=dy.data_ptr(), x=x.data_ptr(), h=h.data_ptr(), gate=gate.data_ptr(),
        weight=w.data_ptr(), next_weight=w2.data_ptr(), dx=dx.data_ptr(),
        dresidual=dres.data_ptr(), dgate_sum=sums[0].data_ptr(),
        dweight=sums[1].data_ptr(), dnext_weight=sums[2].data_ptr(),
        dy_stride=cols, x_stride=cols, h_stride=cols, dx_stride=cols,
        dresidual_stride=cols, rows=rows, cols=cols, norms=3, eps=1e-5,
        residual_scale=1.0)
    n = mt.mt_block_norm_backward_workspace(CODES[dtype], c)
    assert n <= rows * 12 * cols
    # what lies behind belongs to the buffer, as much as the largest call needs
    room = torch.full((n + 608 * 12 * cols,), 171, dtype=torch.uint8,
                      device="cuda")
    mt.mt_block_norm_backward(CODES[dtype], c, room.data_ptr(), n,
                              torch.cuda.current_stream().cuda_stream)
    assert bool((room[n:] == 171).all())
    want = block_norm_back_ref(dy, None, x, h, w, gate, w2, "both", 1.0, 1e-5)
    for name, got, (ref, err) in zip(
            ("dx", "dresidual", "dgate", "dweight", "dnext_weight"),
            (dx, dres, *sums), want):
        check(got, ref, err + half_step(ref, got.dtype), name)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(7, 1024), (1, 4096), (9, 1235),
                                       (1, 8190), (4, 24), (5, 7), (3, 20000),
                                       (2, 40001)], ids=str)
@pytest.mark.parametrize("matrix", [False, True])
def test_gradients_of_a_gate_without_x(dt, rows, cols, matrix):
    """norms "before": x is not needed while the gate's gradient is not."""
    dtype, g = DTYPES[dt], gen(rows * cols)
    dy, dh, h = (randn(g, rows, cols, dtype=dtype) for _ in range(3))
    gate = randn(g, *((rows, cols) if matrix else (cols,)), dtype=dtype)
    w = randn(g, cols, dtype=dtype)
    dx, dres = torch.empty_like(dy), torch.empty_like(dy)
    dw = torch.empty(cols, device="cuda")
    back_call(mt.MtBlockNormBack(
        dy=dy.data_ptr(), dh=dh.data_ptr(), h=h.data_ptr(),
        gate=gate.data_ptr(), next_weight=w.data_ptr(), dx=dx.data_ptr(),
        dresidual=dres.data_ptr(), dnext_weight=dw.data_ptr(), dy_stride=cols,
        dh_stride=cols, h_stride=cols, gate_stride=cols if matrix else 0,
        dx_stride=cols, dresidual_stride=cols, rows=rows, cols=cols, norms=2,
        eps=1e-5, residual_scale=0.75), dtype)
    want = block_norm_back_ref(dy, dh, torch.zeros_like(dy), h, None, gate, w,
                               "before", 0.75, 1e-5)
    for name, got, (ref, err) in zip(("dx", "dresidual", "dnext_weight"),
                                     (dx, dres, dw),
                                     (want[0], want[1], want[3])):
        check(got, ref, err + half_step(ref, got.dtype), name)
