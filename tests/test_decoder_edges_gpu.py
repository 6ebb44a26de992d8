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
