"""Edges of the operators around a decoder's cache on a GPU: what their calls
allow and few callers use, against the plain 64-bit forms."""
import pytest
import torch

import row_reduction_gb300 as mt
from decoder_util import DTYPES, check, half_step
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


# ---- norms around a block ----------------------------------------------------
def back_call(c, dtype):
    """The C call, on a workspace of the size that it asks for."""
    n = mt.mt_block_norm_backward_workspace(CODES[dtype], c)
    room = torch.empty(n, dtype=torch.uint8, device="cuda")
    mt.mt_block_norm_backward(CODES[dtype], c, room.data_ptr() if n else None,
                              n, torch.cuda.current_stream().cuda_stream)


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
