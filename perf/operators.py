"""The row work of a decoder's step between its matrix products, measured: rotary positions of the query and key heads (with the
per-head RMSNorm in front of them, forward and backward), the quantised cache (rows written as 8-bit codes and read back), and the
logits (penalties, biases, grammar mask, temperature, then the row's softmax or log-softmax).

`run` computes each in plain torch operations, or, where `own` is true, through the calls of row_reduction_gb300.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
FORMATS = {"e4m3": (torch.float8_e4m3fn, 448.0), "int8": (torch.int8, 127.0)}
EPS = 1e-6


def listed():
    return [
        # One decode step of eight sequences far into their contexts: launch and Python latency.
        dict(name="rotary decode 8", op="rotary", dtype="bf16", tokens=8, q_heads=32, k_heads=8, dim=128, rotary=128,
             interleaved=False, norm=True, scaling="yarn", far=100000, wide_positions=True),
        # The prefill of a long batch, query and key heads normed and rotated in one pass.
        dict(name="rotary prefill 16384", op="rotary", dtype="bf16", tokens=16384, q_heads=32, k_heads=8, dim=128, rotary=128,
             interleaved=False, norm=True, scaling="bands", far=131072, wide_positions=True),
        # Odd sizes: half of an 80-wide head rotated, interleaved pairs, a ragged token count.
        dict(name="rotary odd 1237", op="rotary", dtype="f16", tokens=1237, q_heads=15, k_heads=5, dim=80, rotary=40,
             interleaved=True, norm=False, scaling="ntk", far=1048576, wide_positions=False),
        # The training step's backward pass through norm and rotation, weight gradients included.
        dict(name="rotary backward 8192", op="rotary_backward", dtype="bf16", tokens=8192, q_heads=32, k_heads=8, dim=128, rotary=128,
             interleaved=False, norm=True, scaling="none", far=8192, wide_positions=True),
        # A small FP32 training step: the rotation's own backward, odd token count.
        dict(name="rotary backward f32 333", op="rotary_backward", dtype="f32", tokens=333, q_heads=12, k_heads=4, dim=64, rotary=32,
             interleaved=True, norm=True, scaling="linear", far=4096, wide_positions=False),
        # One decode step of 64 sequences: each writes its row and has it back.
        dict(name="cache write 64", op="cache", dtype="bf16", format="e4m3", tokens=64, heads=8, dim=128, group=128, pool=65536),
        # A prefill chunk written to integer codes with small groups, and read back for the chunk's attention.
        dict(name="cache write 16384", op="cache", dtype="bf16", format="int8", tokens=16384, heads=8, dim=128, group=64, pool=32768),
        # Long contexts of a batch read back from their pages.
        dict(name="cache read 100003", op="cache_read", dtype="bf16", format="e4m3", tokens=100003, heads=8, dim=128, group=128, pool=131072),
        # One sequence's step over a small vocabulary: latency.
        dict(name="logits 1x32000", op="logits", dtype="f32", rows=1, vocab=32000, history=700, prompt=500, bias=16, mask=True,
             mode="logits"),
        # A batch's step with every option, long histories.
        dict(name="logits 64x131072", op="logits", dtype="bf16", rows=64, vocab=131072, history=8192, prompt=6000, bias=300, mask=True,
             mode="logits"),
        # The largest batch: probabilities under grammar masks, in one pass.
        dict(name="softmax 256x131072", op="logits", dtype="bf16", rows=256, vocab=131072, history=1024, prompt=800, bias=0, mask=True,
             mode="softmax"),
        # An odd vocabulary, long histories, log-probabilities.
        dict(name="log_softmax 17x50257", op="logits", dtype="f16", rows=17, vocab=50257, history=32768, prompt=30000, bias=100, mask=False,
             mode="log_softmax"),
    ]


def draw(rng):
    def log_uniform(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rotary", "rotary", "rotary_backward", "cache", "cache", "cache_read", "logits", "logits", "logits"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("rotary", "rotary_backward"):
        dim = rng.choice([64, 80, 96, 128, 256])
        k_heads = rng.choice([1, 2, 3, 4, 5, 8])
        heads = k_heads * rng.choice([2, 3, 4, 5])
        most = 16384 * 40 * 128 if op == "rotary" else 8192 * 40 * 128
        tokens = log_uniform(1, most // ((heads + k_heads) * dim * BYTES[dtype] // 2))
        return dict(op=op, dtype=dtype, tokens=tokens, q_heads=heads, k_heads=k_heads, dim=dim, rotary=dim // rng.choice([1, 1, 2, 4]),
                    interleaved=rng.random() < 0.4, norm=rng.random() < 0.6, scaling=rng.choice(["none", "linear", "ntk", "yarn", "bands"]),
                    far=log_uniform(1024, 1048576), wide_positions=rng.random() < 0.5)
    if op in ("cache", "cache_read"):
        dim = rng.choice([64, 80, 96, 128, 256])
        heads = rng.choice([1, 2, 3, 4, 8])
        most = (16384 if op == "cache" else 100003) * 8 * 128 // (heads * dim * BYTES[dtype] // 2)
        tokens = log_uniform(1, most)
        return dict(op=op, dtype=dtype, format=rng.choice(["e4m3", "int8"]), tokens=tokens, heads=heads, dim=dim,
                    group=dim // rng.choice([1, 1, 2, 4]) if dim % 64 == 0 else dim, pool=tokens + log_uniform(64, 30000))
    vocab = log_uniform(1000, 262144)
    mode = rng.choice(["logits", "softmax", "log_softmax"])
    rows = log_uniform(1, 128 * 131072 * 2 // (vocab * BYTES[dtype]) if vocab > 2000 else 512)
    history = rng.choice([0, log_uniform(1, 32768)]) if rows <= 256 else log_uniform(1, 2048)
    return dict(op="logits", dtype=dtype, rows=rows, vocab=vocab, history=history, prompt=rng.randint(0, history),
                bias=rng.choice([0, log_uniform(1, 300)]), mask=rng.random() < 0.6, mode=mode)


# ---- inputs -----------------------------------------------------------------------------------------------------------------------


def frequencies(rotary, scaling):
    """Radians per position of each pair, in 64 bits, and the factor on the rotated values. The scaled forms are for contexts eight times
    as long as the 4096 positions of the training."""
    factor, original, base = 8.0, 4096.0, 10000.0
    i = torch.arange(rotary // 2, dtype=torch.float64)
    if scaling == "ntk":
        base = base * factor ** (rotary / (rotary - 2))
    f = base ** (-2.0 * i / rotary)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        def pair_of(turns):
            return rotary * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(pair_of(32.0)), 0), min(math.ceil(pair_of(1.0)), rotary - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    if scaling == "bands":
        length, low, high = 2 * math.pi / f, 1.0, 4.0
        smooth = ((original / length - low) / (high - low)).clamp(0, 1)
        return f * (smooth + (1 - smooth) / factor), 1.0
    return f, 1.0


SCALINGS = {"none": None, "linear": dict(type="linear", factor=8.0), "ntk": dict(type="ntk", factor=8.0),
            "yarn": dict(type="yarn", factor=8.0, original_length=4096),
            "bands": dict(type="bands", factor=8.0, original_length=4096)}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return dict(globals()["_prepare_" + case["op"]](case, gen), case=case)


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _heads(case, gen, count, k_heads):
    """Heads as a fused projection leaves them: views into one row per token, some channels far larger than the rest."""
    dim, dtype = case["dim"], TYPES[case["dtype"]]
    gain = torch.exp(0.7 * _normal(gen, (count + k_heads) * dim))
    x = torch.empty(case["tokens"], (count + k_heads) * dim, device="cuda")
    x.normal_(generator=gen)
    x = (x * gain).to(dtype).view(case["tokens"], count + k_heads, dim)
    return x[:, :count], x[:, count:]


def _prepare_rotary(case, gen):
    q, k = _heads(case, gen, case["q_heads"], case["k_heads"])
    tokens, dim, dtype = case["tokens"], case["dim"], TYPES[case["dtype"]]
    # packed sequences, each from a position of its own
    starts = torch.randint(0, case["far"], (tokens // 512 + 1,), generator=gen, device="cuda")
    at = torch.arange(tokens, device="cuda")
    positions = starts[at // 512] + at % 512
    freqs, factor = frequencies(case["rotary"], case["scaling"])
    state = dict(q=q, k=k, positions=positions if case["wide_positions"] else positions.to(torch.int32), freqs=freqs.cuda(), factor=factor,
                 q_weight=(1 + 0.1 * _normal(gen, dim)).to(dtype), k_weight=(1 + 0.1 * _normal(gen, dim)).to(dtype))
    if own:
        import row_reduction_gb300 as mt
        state["table"] = mt.rotary_frequencies(case["rotary"], base=10000.0, scaling=SCALINGS[case["scaling"]])
    return state


def _prepare_rotary_backward(case, gen):
    state = _prepare_rotary(case, gen)
    state["dq"], state["dk"] = (t * 0.1 for t in _heads(case, gen, case["q_heads"], case["k_heads"]))
    return state


def _slots(case, gen):
    """Rows in pages of 16 slots, the pages in no order; one row in 64 or so is padding and has no slot."""
    pages = (case["pool"] + 15) // 16
    order = torch.randperm(pages, generator=gen, device="cuda")
    at = torch.arange(case["tokens"], device="cuda")
    slots = order[at // 16] * 16 + at % 16
    return torch.where(torch.rand(case["tokens"], generator=gen, device="cuda") < 1 / 64, -1, slots), pages * 16


def _prepare_cache(case, gen):
    k, v = _heads(case, gen, case["heads"], case["heads"])
    slots, count = _slots(case, gen)
    heads, dim, groups = case["heads"], case["dim"], case["dim"] // case["group"]
    code = FORMATS[case["format"]][0]
    empty = lambda: (torch.zeros(count, heads, dim, device="cuda", dtype=torch.int8).view(code),  # noqa: E731
                     torch.zeros(count, heads, groups, device="cuda"))
    read = lambda: torch.zeros(case["tokens"], heads, dim, device="cuda", dtype=TYPES[case["dtype"]])  # noqa: E731
    return dict(k=k, v=v, slots=slots, k_cache=empty(), v_cache=empty(), out=(read(), read()))


def _prepare_cache_read(case, gen):
    slots, count = _slots(case, gen)
    heads, dim, groups = case["heads"], case["dim"], case["dim"] // case["group"]
    code, largest = FORMATS[case["format"]]

    def filled():
        x = (torch.randn(count, heads, dim, generator=gen, device="cuda", dtype=torch.float16) * (largest / 4)).clamp(-largest, largest)
        return x.round().to(code) if case["format"] == "int8" else x.to(code), torch.rand(count, heads, groups, generator=gen, device="cuda") / largest
    read = lambda: torch.zeros(case["tokens"], heads, dim, device="cuda", dtype=TYPES[case["dtype"]])  # noqa: E731
    return dict(slots=slots, k_cache=filled(), v_cache=filled(), out=(read(), read()))


def _prepare_logits(case, gen):
    rows, vocab, history = case["rows"], case["vocab"], case["history"]
    uniform = lambda *shape: torch.rand(shape, generator=gen, device="cuda")  # noqa: E731
    state = dict(logits=(3.0 * _normal(gen, rows, vocab)).to(TYPES[case["dtype"]]), mode=case["mode"],
                 temperature=0.5 + uniform(rows), tokens=None, lengths=None, prompt_lengths=None, repetition=None, frequency=None,
                 presence=None, bias_ids=None, bias=None, mask=None)
    if history:
        # few tokens are frequent, most are rare; rows of different lengths, the rest of a row is padding
        state["tokens"] = (uniform(rows, history) ** 4 * vocab).to(torch.int32).clamp(max=vocab - 1)
        state["lengths"] = (history - (uniform(rows) * (history // 4 + 1)).to(torch.int32)).to(torch.int32)
        state["prompt_lengths"] = (uniform(rows) * (case["prompt"] + 1)).to(torch.int32).clamp(max=case["prompt"])
        state["repetition"] = 1.0 + 0.3 * uniform(rows)
        state["frequency"] = 0.2 * uniform(rows)
        state["presence"] = 0.5 * uniform(rows)
    if case["bias"]:
        state["bias_ids"] = (uniform(rows, case["bias"]) * vocab).to(torch.int32).clamp(max=vocab - 1)
        state["bias"] = 2.0 * _normal(gen, rows, case["bias"])
    if case["mask"]:
        # a grammar allows anything, half of the words, or one in some hundreds; some row of a batch has come to its end: nothing
        words = (vocab + 31) // 32
        dense = torch.randint(-2 ** 31, 2 ** 31, (rows, words), generator=gen, device="cuda").to(torch.int32)
        few = torch.where(uniform(rows, words) < 0.05, dense & (dense >> 3) & (dense >> 7), 0)
        kind = torch.arange(rows, device="cuda")[:, None] % 4
        mask = torch.where(kind == 0, -1, torch.where(kind == 1, dense, few))
        state["mask"] = torch.where(torch.arange(rows, device="cuda")[:, None] % 64 == 10, 0, mask).to(torch.int32).contiguous()
    return state


# ---- one pass -----------------------------------------------------------------------------------------------------------------------


def run(state):
    return globals()[("_own_" if own else "_plain_") + state["case"]["op"]](state)


def _own_rotary(s):
    import row_reduction_gb300 as mt
    c = s["case"]
    if not c["norm"]:
        return mt.rotary(s["q"], s["k"], s["positions"], s["table"], interleaved=c["interleaved"])
    return mt.rotary(s["q"], s["k"], s["positions"], s["table"], interleaved=c["interleaved"], q_weight=s["q_weight"],
                     k_weight=s["k_weight"], eps=EPS)


def _own_rotary_backward(s):
    import row_reduction_gb300 as mt
    c = s["case"]
    if not c["norm"]:
        return mt.rotary_backward(s["dq"], s["dk"], s["positions"], s["table"], interleaved=c["interleaved"])
    return mt.rotary_backward(s["dq"], s["dk"], s["positions"], s["table"], interleaved=c["interleaved"], q=s["q"], k=s["k"],
                              q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS)


def _own_cache(s):
    import row_reduction_gb300 as mt
    mt.cache_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"])
    return mt.cache_read(s["k_cache"], s["v_cache"], s["slots"], out=s["out"]), s["k_cache"][1], s["v_cache"][1]


def _own_cache_read(s):
    import row_reduction_gb300 as mt
    return mt.cache_read(s["k_cache"], s["v_cache"], s["slots"], out=s["out"])


def _own_logits(s):
    import row_reduction_gb300 as mt
    return mt.process_logits(s["logits"], tokens=s["tokens"], lengths=s["lengths"], prompt_lengths=s["prompt_lengths"],
                             repetition=s["repetition"], frequency=s["frequency"], presence=s["presence"], bias_ids=s["bias_ids"],
                             bias=s["bias"], mask=s["mask"], temperature=s["temperature"], mode=s["mode"])


def _cos_sin(s):
    """cos and sin of each token's angles, [tokens, 1, pairs]: far positions lose their angle in 32 bits, so the angle has 64."""
    angle = s["positions"].double()[:, None, None] * s["freqs"]
    return (torch.cos(angle) * s["factor"]).float(), (torch.sin(angle) * s["factor"]).float()


def _turned(x, cos, sin, rotary, interleaved):
    """The rotation of the first `rotary` values of each head of an FP32 tensor; with -sin its transpose."""
    a, b = (x[..., 0:rotary:2], x[..., 1:rotary:2]) if interleaved else (x[..., :rotary // 2], x[..., rotary // 2:rotary])
    a, b = a * cos - b * sin, a * sin + b * cos
    y = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((y, x[..., rotary:]), -1)


def _plain_rotary(s):
    cos, sin = _cos_sin(s)
    return _rotary_of(s, s["q"], s["q_weight"], cos, sin), _rotary_of(s, s["k"], s["k_weight"], cos, sin)


def _rotary_of(s, x, weight, cos, sin):
    c, y = s["case"], x.float()
    if c["norm"]:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * weight.float()
    return _turned(y, cos, sin, c["rotary"], c["interleaved"]).to(x.dtype)


def _plain_rotary_backward(s):
    cos, sin = _cos_sin(s)
    dq, dq_weight = _rotary_backward_of(s, s["dq"], s["q"], s["q_weight"], cos, sin)
    dk, dk_weight = _rotary_backward_of(s, s["dk"], s["k"], s["k_weight"], cos, sin)
    return (dq, dk, dq_weight, dk_weight) if s["case"]["norm"] else (dq, dk)


def _rotary_backward_of(s, dy, x, weight, cos, sin):
    c = s["case"]
    g = _turned(dy.float(), cos, -sin, c["rotary"], c["interleaved"])
    if not c["norm"]:
        return g.to(dy.dtype), None
    x = x.float()
    rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    xh, gw = x * rstd, g * weight.float()
    return (rstd * (gw - xh * (gw * xh).mean(-1, keepdim=True))).to(dy.dtype), (g * xh).sum((0, 1))


def _quantised(x, fmt, group):
    """Codes and FP32 scales of the rows of an FP32 tensor [rows, heads, dim], one scale to each group of a row."""
    code, largest = FORMATS[fmt]
    x = x.unflatten(-1, (-1, group))
    scale = (x.abs().amax(-1) * (1 / largest)).clamp(min=2.0 ** -126)
    codes = (x * (1 / scale)[..., None]).clamp(-largest, largest)
    return (codes.round() if fmt == "int8" else codes).to(code).flatten(-2), scale


def _plain_cache(s):
    c = s["case"]
    rows = torch.nonzero(s["slots"] >= 0)[:, 0]
    at = s["slots"][rows]
    codes, scales = _quantised(torch.stack((s["k"][rows], s["v"][rows])).float(), c["format"], c["group"])
    s["k_cache"][0].view(torch.int8)[at], s["k_cache"][1][at] = codes[0].view(torch.int8), scales[0]
    s["v_cache"][0].view(torch.int8)[at], s["v_cache"][1][at] = codes[1].view(torch.int8), scales[1]
    return _plain_cache_read(s), s["k_cache"][1], s["v_cache"][1]


def _plain_cache_read(s):
    rows = torch.nonzero(s["slots"] >= 0)[:, 0]
    at = s["slots"][rows]
    s["out"][0][rows] = _values(s["k_cache"], at, s["case"]["group"]).to(s["out"][0].dtype)
    s["out"][1][rows] = _values(s["v_cache"], at, s["case"]["group"]).to(s["out"][1].dtype)
    return s["out"]


def _values(cache, at, group):
    codes = cache[0].view(torch.int8)[at].view(cache[0].dtype).float()
    return (codes.unflatten(-1, (-1, group)) * cache[1][at][..., None]).flatten(-2)


def _plain_logits(s):
    z = s["logits"].float()
    rows, vocab = z.shape
    if s["tokens"] is not None:
        at = torch.arange(s["tokens"].shape[1], device="cuda")
        there, prompt = at < s["lengths"][:, None], at < s["prompt_lengths"][:, None]
        ids = torch.where(there, s["tokens"].long(), vocab)
        ones = torch.ones_like(ids, dtype=torch.int32)
        count = torch.zeros(rows, vocab + 1, dtype=torch.int32, device="cuda").scatter_add_(1, torch.where(prompt, vocab, ids), ones)[:, :vocab]
        seen = torch.zeros(rows, vocab + 1, dtype=torch.bool, device="cuda").scatter_(1, ids, True)[:, :vocab]
        rho = s["repetition"][:, None]
        z = torch.where(seen, torch.where(z > 0, z / rho, z * rho), z)
        z = z - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
    if s["bias"] is not None:
        z = z.scatter_add(1, s["bias_ids"].long(), s["bias"])
    z = z / s["temperature"][:, None]
    if s["mask"] is not None:
        v = torch.arange(vocab, device="cuda")
        z = torch.where((s["mask"][:, v >> 5] >> (v & 31)) & 1 != 0, z, -math.inf)
    if s["mode"] != "logits":
        top = z.amax(1, keepdim=True)
        d = z - torch.where(top == -math.inf, 0.0, top)
        e = torch.exp(d)
        total = e.sum(1, keepdim=True)
        z = e / torch.where(total == 0, 1.0, total) if s["mode"] == "softmax" else torch.where(total == 0, d, d - torch.log(total))
    return z.to(s["logits"].dtype)


# ---- what a pass has to move and to compute ----------------------------------------------------------------------------------------


def work(case):
    if case["op"] in ("rotary", "rotary_backward"):
        values = case["tokens"] * (case["q_heads"] + case["k_heads"]) * case["dim"]
        back = case["op"] == "rotary_backward" and case["norm"]
        moved = values * BYTES[case["dtype"]] * (3 if back else 2) + case["tokens"] * (8 if case["wide_positions"] else 4)
        return {"bytes": moved, "flops": values * (4 + (14 if back else 4 if case["norm"] else 0))}
    if case["op"] in ("cache", "cache_read"):
        values = 2 * case["tokens"] * case["heads"] * case["dim"]
        wide = BYTES[case["dtype"]]
        # written: values in, codes and scales out; read back: codes and scales in, values out
        one = values * (wide + 1) + values // case["group"] * 4 + case["tokens"] * 8
        return {"bytes": one * (2 if case["op"] == "cache" else 1), "flops": values * (4 if case["op"] == "cache" else 1)}
    cells = case["rows"] * case["vocab"]
    extra = case["rows"] * (case["history"] * 4 + case["bias"] * 8 + (case["vocab"] // 8 if case["mask"] else 0))
    return {"bytes": cells * 2 * BYTES[case["dtype"]] + extra, "flops": cells * (2 if case["mode"] == "logits" else 6)}


# ---- in 64 bits, from the definitions ----------------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](s, case)


def _exact_spin(s, case):
    """exp(i angle) times the factor, [tokens, 1, pairs]."""
    angle = s["positions"].double()[:, None] * s["freqs"][None]
    return torch.polar(torch.full_like(angle, s["factor"]), torch.remainder(angle, 2 * math.pi))[:, None]


def _exact_spun(x, spin, case):
    r = case["rotary"]
    head, rest = x[..., :r], x[..., r:]
    if case["interleaved"]:
        z = torch.view_as_complex(head.reshape(*head.shape[:-1], r // 2, 2).contiguous()) * spin
        return torch.cat((torch.view_as_real(z).reshape(head.shape), rest), -1)
    z = torch.complex(head[..., :r // 2].contiguous(), head[..., r // 2:].contiguous()) * spin
    return torch.cat((z.real, z.imag, rest), -1)


def _exact_rotary(s, case):
    spin, got = _exact_spin(s, case), []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        x = x.double()
        if case["norm"]:
            x = x * w.double() * torch.rsqrt(x.square().sum(-1, keepdim=True) / case["dim"] + EPS)
        got.append(_exact_spun(x, spin, case))
    return tuple(got)


def _exact_rotary_backward(s, case):
    """Through the norm as d/dx of x w r(x), r = (mean x^2 + eps)^-1/2: w r g - x r^3 (x . w g) / dim."""
    spin, grads, weights = _exact_spin(s, case).conj(), [], []
    for dy, x, w in ((s["dq"], s["q"], s["q_weight"]), (s["dk"], s["k"], s["k_weight"])):
        g = _exact_spun(dy.double(), spin, case)
        if case["norm"]:
            x, w = x.double(), w.double()
            r = torch.rsqrt(x.square().sum(-1, keepdim=True) / case["dim"] + EPS)
            weights.append(torch.einsum("thd,thd->d", g, x * r))
            g = r * w * g - x * r ** 3 * torch.einsum("thd,thd->th", x, w * g)[..., None] / case["dim"]
        grads.append(g)
    return tuple(grads + weights)


def _exact_quantised(x, case):
    """Values that the codes stand for, and the scales; codes are rounded to the format's own grid."""
    largest = FORMATS[case["format"]][1]
    x = x.double().reshape(*x.shape[:-1], -1, case["group"])
    scale = torch.clamp(x.abs().max(-1).values / largest, min=2.0 ** -126)
    y = x / scale[..., None]
    if case["format"] == "int8":
        y = torch.round(y)
    else:  # three bits of fraction; the smallest exponent is -6
        step = torch.exp2(torch.clamp(torch.frexp(y).exponent.double() - 1, min=-6.0) - 3)
        y = torch.round(y / step) * step
    return (torch.clamp(y, -largest, largest) * scale[..., None]).reshape(*x.shape[:-2], -1), scale


def _exact_cache(s, case):
    live, outs, scales = s["slots"] >= 0, [], []
    for x, cache in ((s["k"], s["k_cache"]), (s["v"], s["v_cache"])):
        values, scale = _exact_quantised(x, case)
        outs.append(torch.where(live[:, None, None], values, 0.0))
        held = cache[1].double()
        held[s["slots"][live]] = scale[live]
        scales.append(held)
    return tuple(outs), *scales


def _exact_cache_read(s, case):
    outs = []
    for codes, scales in (s["k_cache"], s["v_cache"]):
        held = codes.float()
        got = held[s["slots"].clamp(min=0)].double() * torch.repeat_interleave(scales[s["slots"].clamp(min=0)].double(), case["group"], -1)
        outs.append(torch.where((s["slots"] >= 0)[:, None, None], got, 0.0))
    return tuple(outs)


def _exact_logits(s, case):
    z = s["logits"].double()
    rows, vocab = z.shape
    if s["tokens"] is not None:
        at = torch.arange(case["history"], device="cuda").expand(rows, -1)
        flat = s["tokens"].long() + vocab * torch.arange(rows, device="cuda")[:, None]
        whole = at < s["lengths"][:, None]
        output = whole & (at >= s["prompt_lengths"][:, None])
        count = torch.bincount(flat[output], minlength=rows * vocab).view(rows, vocab).double()
        seen = torch.bincount(flat[whole], minlength=rows * vocab).view(rows, vocab) > 0
        rho = s["repetition"].double()[:, None]
        z = torch.where(seen, torch.where(z > 0, z / rho, z * rho), z)
        z = z - s["frequency"].double()[:, None] * count - s["presence"].double()[:, None] * torch.sign(count)
    if s["bias"] is not None:
        flat = s["bias_ids"].long() + vocab * torch.arange(rows, device="cuda")[:, None]
        z = z + torch.bincount(flat.flatten(), weights=s["bias"].double().flatten(), minlength=rows * vocab).view(rows, vocab)
    z = z / s["temperature"].double()[:, None]
    if s["mask"] is not None:
        bits = (s["mask"].cpu().view(torch.uint8).cuda()[..., None] >> torch.arange(8, device="cuda", dtype=torch.uint8)) & 1
        z = z.masked_fill(bits.reshape(rows, -1)[:, :vocab] == 0, -math.inf)
    if case["mode"] == "logits":
        return z
    z = z - torch.nan_to_num(torch.logsumexp(z, 1, keepdim=True), neginf=0.0)
    return torch.exp(z) if case["mode"] == "softmax" else z
