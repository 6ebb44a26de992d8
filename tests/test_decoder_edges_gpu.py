"""Edges of the decoder's row operators on a GPU: values and sizes at which a
result can go wrong without a usual input showing it."""
import math

import pytest
import torch

import row_reduction_gb300 as mt
from decoder_util import DTYPES, U, check, half_step, logits_ref

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
