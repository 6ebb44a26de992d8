"""A decoder's step around its quantised cache, measured: the pages, slots and positions of the step's rows (cache_extend), attention over
the cached codes (cache_attention), and the norms after a block and before the next one with the block's gate and the residual's scale
(block_norm, forward and backward).

`run` computes each in plain torch operations, or, where `own` is true, through the calls of row_reduction_gb300.
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
FORMATS = {"e4m3": (torch.float8_e4m3fn, 448.0), "int8": (torch.int8, 127.0)}
EPS = 1e-6


def listed():
    return [
        # One decode step of eight chats: launch and Python latency.
        dict(name="attention decode 8", op="attention", dtype="bf16", format="e4m3", sequences=8, keys=2048, rows=1, q_heads=32, k_heads=8,
             dim=128, group=128, page=16, cap=0.0, slopes=False, window=0, mask="causal"),
        # The largest decode batch: contexts of every length up to 16384.
        dict(name="attention decode 64", op="attention", dtype="bf16", format="e4m3", sequences=64, keys=16384, rows=1, q_heads=32,
             k_heads=8, dim=128, group=128, page=16, cap=0.0, slopes=False, window=0, mask="causal"),
        # One far context alone, capped scores, integer codes with small groups: split along the keys or most of the device is idle.
        dict(name="attention decode 1 far", op="attention", dtype="bf16", format="int8", sequences=1, keys=131072, rows=1, q_heads=32,
             k_heads=8, dim=128, group=64, page=32, cap=50.0, slopes=False, window=0, mask="causal"),
        # Tokens guessed ahead and checked in one step: one to four rows a sequence, odd heads, a bias by distance, a window.
        dict(name="attention guessed 17", op="attention", dtype="f16", format="e4m3", sequences=17, keys=5003, rows=4, q_heads=15,
             k_heads=5, dim=80, group=80, page=24, cap=0.0, slopes=True, window=1000, mask="causal"),
        # Chunks of prompts after what the cache holds already, a prefix that all its rows see, capped.
        dict(name="attention chunk 2x512", op="attention", dtype="bf16", format="e4m3", sequences=2, keys=4096, rows=512, q_heads=32,
             k_heads=8, dim=128, group=128, page=16, cap=30.0, slopes=False, window=0, mask="prefix"),
        # A small model checked in FP32, documents packed into its sequences.
        dict(name="attention f32 documents", op="attention", dtype="f32", format="int8", sequences=5, keys=1200, rows=33, q_heads=12,
             k_heads=4, dim=64, group=32, page=16, cap=0.0, slopes=False, window=0, mask="document"),
        # One decode step's residual rows: latency.
        dict(name="block norm 8", op="block_norm", dtype="bf16", rows=8, cols=4096, gate="vector", norms="both", residual_scale=1.0),
        # A long batch's prefill, both norms and a gate per channel in one pass.
        dict(name="block norm 16384", op="block_norm", dtype="bf16", rows=16384, cols=4096, gate="vector", norms="both",
             residual_scale=1.0),
        # The training step's backward pass, gradients of both weights and of the gate included.
        dict(name="block norm backward 8192", op="block_norm_backward", dtype="bf16", rows=8192, cols=4096, gate="vector", norms="both",
             residual_scale=1.0),
        # A small FP32 training step, a gate of its own for each row, a scaled residual, odd sizes.
        dict(name="block norm backward f32 333", op="block_norm_backward", dtype="f32", rows=333, cols=1237, gate="matrix", norms="both",
             residual_scale=0.7),
        # One decode step of 256 sequences: a page for one in sixteen of them.
        dict(name="extend decode 256", op="extend", sequences=256, most=1, keys=8192, page=16, short=False),
        # Prompts and single tokens mixed, more than there are pages for.
        dict(name="extend mixed 1024", op="extend", sequences=1024, most=512, keys=16384, page=16, short=True),
    ]


# ---- drawn cases ------------------------------------------------------------------------------------------------------------------


def draw(rng):
    def log_uniform(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))

    op = rng.choice(["attention", "attention", "attention", "block_norm", "block_norm", "block_norm_backward", "block_norm_backward",
                     "extend"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "attention":
        dim = rng.choice([64, 80, 96, 128, 128, 256])
        k_heads = rng.choice([1, 2, 3, 4, 5, 8])
        times = rng.choice([1, 2, 3, 4, 5, 8])
        sequences = log_uniform(1, 128)
        rows = rng.choice([1, 1, 1, log_uniform(2, 8), log_uniform(9, 300)])
        # no more to read, and no more scores, than the largest listed ones have
        most = 131072 if rows == 1 else 8192
        most = min(most, 64 * 16384 * 1024 // (sequences * k_heads * dim), (2 * 32 * 512 * 4096) // (sequences * k_heads * times * rows))
        keys = max(rows, log_uniform(1, max(1, most)))
        group = rng.choice([dim, dim, dim // 2, 32]) if dim % 64 == 0 else dim
        return dict(op=op, dtype=dtype, format=rng.choice(["e4m3", "int8"]), sequences=sequences, keys=keys, rows=rows,
                    q_heads=k_heads * times, k_heads=k_heads, dim=dim, group=group, page=rng.choice([1, 16, 16, 24, 32, 64, 128]),
                    cap=rng.choice([0.0, 0.0, 30.0, 50.0]), slopes=rng.random() < 0.3,
                    window=rng.choice([0, 0, log_uniform(1, 4096)]), mask=rng.choice(["causal", "causal", "prefix", "document"]))
    if op == "extend":
        sequences = log_uniform(1, 1024)
        return dict(op=op, sequences=sequences, most=log_uniform(1, 512), keys=log_uniform(600, 16384), page=rng.choice([1, 16, 24, 32, 64]),
                    short=rng.random() < 0.4)
    cols = rng.choice([log_uniform(64, 16384), 64 * log_uniform(1, 128), 1024 * rng.choice([1, 2, 4, 5, 8])])
    most = (16384 if op == "block_norm" else 8192) * 4096 * 2 // (cols * BYTES[dtype] * 2)
    return dict(op=op, dtype=dtype, rows=log_uniform(1, max(1, most)), cols=cols, gate=rng.choice(["none", "vector", "vector", "matrix"]),
                norms=rng.choice(["both", "both", "before", "after"]), residual_scale=rng.choice([1.0, 1.0, 0.5, 0.7071]))


# ---- inputs -----------------------------------------------------------------------------------------------------------------------


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return dict(globals()["_prepare_" + case["op"]](case, gen), case=case)


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _batch(case):
    """(rows, keys) of each sequence, by the case alone: the longest has all of its keys and rows, the others from one on."""
    rng = random.Random(case["keys"] * 1000003 + case["sequences"] * 101 + case["rows"])
    batch = [(case["rows"], case["keys"])]
    for _ in range(case["sequences"] - 1):
        rows = rng.randint(1, case["rows"])
        batch.append((rows, rng.randint(rows, max(rows, case["keys"]))))
    rng.shuffle(batch)
    return batch


def _sees(case):
    """For each row of each sequence the first and the last key that it sees, and the document or prefix bound among them."""
    rng = random.Random(case["keys"] + case["sequences"])
    got = []
    for rows, keys in _batch(case):
        start, cut = keys - rows, rng.randint(1, keys)
        for p in range(start, keys):
            # a document that begins inside the sequence; a prefix that all of its rows see to its end
            first = cut if case["mask"] == "document" and p >= cut else 0
            last = max(p, cut - 1) if case["mask"] == "prefix" else p
            bound = max(first, p - case["window"] + 1) if case["window"] else first
            got.append((bound, last, first))
    return got


def _prepare_attention(case, gen):
    batch = _batch(case)
    heads, dim, groups, page = case["k_heads"], case["dim"], case["dim"] // case["group"], case["page"]
    need = [(keys + page - 1) // page for _, keys in batch]
    width, pool = max(need), sum(need) + 3
    order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    begin = torch.tensor([sum(need[:s]) for s in range(len(need))], device="cuda")
    at = torch.arange(width, device="cuda")
    table = torch.where(at < torch.tensor(need, device="cuda")[:, None], order[(begin[:, None] + at).clamp(max=pool - 1)], -1)
    code, largest = FORMATS[case["format"]]

    def filled():
        x = torch.empty(pool * page, heads, dim, device="cuda", dtype=torch.float16).normal_(generator=gen).mul_(largest / 4)
        x = x.clamp_(-largest, largest)
        scales = torch.empty(pool * page, heads, groups, device="cuda").uniform_(0.5, 1.5, generator=gen).mul_(4 / largest)
        return (x.round_() if case["format"] == "int8" else x).to(code), scales
    total = sum(rows for rows, _ in batch)
    offsets = [0]
    for rows, _ in batch:
        offsets.append(offsets[-1] + rows)
    sees = _sees(case)
    dtype = TYPES[case["dtype"]]
    # queries as a fused projection leaves them; the batch is padded to a multiple of four rows
    padded = (total + 3) // 4 * 4
    q = _normal(gen, padded, case["q_heads"] + 2 * heads, dim).to(dtype)[:, :case["q_heads"]]
    pad = [0] * (padded - total)
    slopes = torch.exp2(-8.0 * torch.arange(1, case["q_heads"] + 1, device="cuda") / case["q_heads"]) if case["slopes"] else None
    return dict(q=q, k_cache=filled(), v_cache=filled(), table=table.to(torch.int32).contiguous(), offsets=_int32(offsets),
                starts=_int32([keys - rows for rows, keys in batch]), slopes=slopes,
                first=_int32([f for _, _, f in sees] + pad) if case["mask"] == "document" else None,
                last=_int32([b for _, b, _ in sees] + pad) if case["mask"] == "prefix" else None,
                sees=(_int32([a for a, _, _ in sees]), _int32([b for _, b, _ in sees])), rows=total, most_rows=case["rows"],
                most_keys=max(keys for _, keys in batch), out=torch.zeros(padded, case["q_heads"], dim, dtype=dtype, device="cuda"))


def _matrix(case, gen):
    """A matrix of the residual stream: some channels far larger than the rest."""
    gain = torch.exp(0.7 * _normal(gen, case["cols"]))
    x = torch.empty(case["rows"], case["cols"], device="cuda").normal_(generator=gen)
    return x.mul_(gain).to(TYPES[case["dtype"]])


def _prepare_block_norm(case, gen):
    dtype, cols = TYPES[case["dtype"]], case["cols"]
    weight = lambda: (1 + 0.1 * _normal(gen, cols)).to(dtype)  # noqa: E731
    gate = None
    if case["gate"] != "none":
        gate = (0.5 + 0.3 * _normal(gen, *((cols,) if case["gate"] == "vector" else (case["rows"], cols)))).to(dtype)
    return dict(x=_matrix(case, gen), residual=_matrix(case, gen), gate=gate,
                weight=weight() if case["norms"] != "before" else None, next_weight=weight() if case["norms"] != "after" else None)


def _prepare_block_norm_backward(case, gen):
    s = _prepare_block_norm(case, gen)
    s["h"] = s.pop("residual")  # the stream behind the block, kept by the forward pass
    s["dh"] = _matrix(case, gen) * 0.1
    s["dy"] = _matrix(case, gen) * 0.1 if case["norms"] != "after" else None
    return s


def _prepare_extend(case, gen):
    n, page = case["sequences"], case["page"]
    width = (case["keys"] + case["most"] + page - 1) // page
    uniform = lambda: torch.rand(n, generator=gen, device="cuda")  # noqa: E731
    lengths = (uniform() * case["keys"]).int()
    # most sequences go on by one token, some by a part of their prompt, some not at all
    kind = uniform()
    counts = torch.where(kind < 0.05, 0, torch.where(kind < 0.7, 1, 1 + (uniform() * case["most"]).int())).to(torch.int32)
    held = (lengths + page - 1) // page
    wanted = (lengths + counts + page - 1) // page - held
    total = int(held.sum()) + int(wanted.sum()) + 16
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    begin = torch.cumsum(held, 0) - held
    at = torch.arange(width, device="cuda")
    table = torch.where(at < held[:, None], order[(begin[:, None] + at).clamp(max=total - 1)], -1).to(torch.int32)
    free = order[int(held.sum()):].contiguous()
    count = int(wanted.sum()) * 3 // 4 if case["short"] else free.numel() - 3
    # a captured step's rows: room for what a batch of these sequences brings on most days, the rest padding
    rows = (n * (5 + case["most"]) // 5 + 2 * case["most"] + 255) // 256 * 256
    return dict(table=table.contiguous(), lengths=lengths, counts=counts, free=free, free_count=_int32([count]), rows=rows)


# ---- one pass ---------------------------------------------------------------------------------------------------------------------


def run(state):
    return globals()[("_own_" if own else "_plain_") + state["case"]["op"]](state)


def _own_attention(s):
    import row_reduction_gb300 as mt
    c = s["case"]
    return mt.cache_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["offsets"], s["starts"], c["page"],
                              cap=c["cap"] or None, slopes=s["slopes"], window=c["window"] or None, first=s["first"], last=s["last"],
                              out=s["out"])


def _own_block_norm(s):
    import row_reduction_gb300 as mt
    c = s["case"]
    return mt.block_norm(s["x"], s["residual"], gate=s["gate"], weight=s["weight"], next_weight=s["next_weight"], norms=c["norms"],
                         residual_scale=c["residual_scale"], eps=EPS)


def _own_block_norm_backward(s):
    import row_reduction_gb300 as mt
    c = s["case"]
    return mt.block_norm_backward(s["dy"], s["dh"], s["x"], s["h"], gate=s["gate"], weight=s["weight"], next_weight=s["next_weight"],
                                  norms=c["norms"], residual_scale=c["residual_scale"], eps=EPS)


def _own_extend(s):
    import row_reduction_gb300 as mt
    step = mt.cache_extend(s["table"], s["lengths"], s["counts"], s["free"], s["free_count"], s["case"]["page"], s["rows"])
    return s["table"], step.offsets, step.slots, step.positions, step.lengths, step.free_count


def _plain_attention(s):
    c, rows = s["case"], s["rows"]
    heads, times, page = c["k_heads"], c["q_heads"] // c["k_heads"], c["page"]
    key = torch.arange(s["most_keys"], device="cuda")
    slot = s["table"][:, key // page].long()
    slot = torch.where(slot < 0, 0, slot * page + key % page)
    # every sequence padded to the most rows and keys
    row = torch.arange(rows, device="cuda")
    at = torch.searchsorted(s["offsets"], row.to(torch.int32), right=True) - 1, row - s["offsets"][:-1].long().repeat_interleave(
        s["offsets"][1:].long() - s["offsets"][:-1], output_size=rows)
    q = torch.zeros(c["sequences"], s["most_rows"], heads, times, c["dim"], device="cuda")
    q[at] = s["q"][:rows].float().unflatten(1, (heads, times))
    score = torch.einsum("srhtd,skhd->srhtk", q, _values(s["k_cache"], slot, c["group"])) / math.sqrt(c["dim"])
    if c["cap"]:
        score = c["cap"] * torch.tanh(score / c["cap"])
    if s["slopes"] is not None:
        place = s["starts"][:, None] + torch.arange(s["most_rows"], device="cuda")
        far = (place[:, :, None] - key).abs()
        score = score - s["slopes"].view(heads, times, 1) * far[:, :, None, None]
    see = torch.zeros(2, c["sequences"], s["most_rows"], dtype=torch.int32, device="cuda")
    see[1] = -1
    see[0][at], see[1][at] = s["sees"]
    seen = (key >= see[0][..., None]) & (key <= see[1][..., None])
    score = torch.where(seen[:, :, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    e = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total == 0, 1.0, total)
    o = torch.einsum("srhtk,skhd->srhtd", p, _values(s["v_cache"], slot, c["group"]))
    s["out"][:rows] = o[at].flatten(1, 2).to(s["out"].dtype)
    return s["out"]


def _values(cache, slot, group):
    codes = cache[0].view(torch.int8)[slot].view(cache[0].dtype).float()
    return codes.unflatten(-1, (-1, group)).mul_(cache[1][slot][..., None]).flatten(-2)


def _rms(x):
    return 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)


def _plain_block_norm(s):
    c, x = s["case"], s["x"].float()
    if c["norms"] != "before":
        x = x * _rms(x) * s["weight"].float()
    if s["gate"] is not None:
        x = x * s["gate"].float()
    h = s["residual"].float() * c["residual_scale"] + x
    y = None if c["norms"] == "after" else (h * _rms(h) * s["next_weight"].float()).to(s["x"].dtype)
    h = h.to(s["x"].dtype)
    return h if y is None else (y, h)


def _plain_block_norm_backward(s):
    """Gradients of x, the residual, the gate, the weight of the norm behind the block and that of the norm before the next one."""
    c, x, h, d, dtype = s["case"], s["x"].float(), s["h"].float(), s["dh"].float(), s["x"].dtype
    dnext = dweight = dgate = None
    if c["norms"] != "after":
        r, g = _rms(h), s["dy"].float()
        hh, gw = h * r, g * s["next_weight"].float()
        d = d + r * (gw - hh * (gw * hh).mean(-1, keepdim=True))
        dnext = (g * hh).sum(0)
    dresidual = d * c["residual_scale"]
    r = _rms(x) if c["norms"] != "before" else 1.0
    xh = x * r
    if s["gate"] is not None:
        u = xh * s["weight"].float() if c["norms"] != "before" else x
        dgate = (d * u).sum(0) if c["gate"] == "vector" else (d * u).to(dtype)
        d = d * s["gate"].float()
    if c["norms"] != "before":
        dweight = (d * xh).sum(0)
        gw = d * s["weight"].float()
        d = r * (gw - xh * (gw * xh).mean(-1, keepdim=True))
    return tuple(t for t in (d.to(dtype), dresidual.to(dtype), dgate, dweight, dnext) if t is not None)


def _plain_extend(s):
    page, rows, width = s["case"]["page"], s["rows"], s["table"].shape[1]
    lengths, counts = s["lengths"].long(), s["counts"].long()
    held, wanted = (lengths + page - 1) // page, (lengths + counts + page - 1) // page
    fits = wanted <= width
    need = torch.where(fits, wanted - held, 0)
    upto = torch.cumsum(need, 0)
    free = s["free_count"].long()
    served = fits & ((upto <= free) | (need == 0))
    # pages from the end of the list, in the order of the sequences
    at = torch.arange(width, device="cuda")
    new = served[:, None] & (at >= held[:, None]) & (at < wanted[:, None])
    take = (free - 1 - (upto - need)[:, None] - (at - held[:, None])).clamp(0, s["free"].shape[0] - 1)
    s["table"].copy_(torch.where(new, s["free"][take], s["table"]))
    offsets = torch.cat((torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(counts, 0)))
    row = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(offsets, row, right=True) - 1
    there = seq < lengths.shape[0]
    seq = seq.clamp(max=lengths.shape[0] - 1)
    place = torch.where(there, lengths[seq] + row - offsets[seq], 0)
    slots = s["table"][seq, (place // page).clamp(max=width - 1)].long() * page + place % page
    slots = torch.where(there & served[seq], slots, -1)
    used = torch.where(served & (need > 0), upto, 0).amax()
    return (s["table"], offsets.int(), slots, place.int(), torch.where(served, lengths + counts, lengths).int(),
            (free - used).int())


# ---- what a pass has to move and to compute ---------------------------------------------------------------------------------------


def work(case):
    if case["op"] == "attention":
        # a key is read once for each sequence that sees it; a pair of a row and a key that it sees costs two products of the head's width
        sees, at, read = _sees(case), 0, 0
        for rows, _ in _batch(case):
            mine = sees[at:at + rows]
            read += max(b for _, b, _ in mine) + 1 - min(a for a, _, _ in mine)
            at += rows
        pairs = sum(b + 1 - a for a, b, _ in sees)
        one = 2 * case["k_heads"] * (case["dim"] + 4 * case["dim"] // case["group"])
        return {"bytes": read * one + 2 * len(sees) * case["q_heads"] * case["dim"] * BYTES[case["dtype"]],
                "flops": 4 * pairs * case["q_heads"] * case["dim"]}
    if case["op"] == "extend":
        # lengths, counts, new lengths and offsets of a sequence, slots and positions of its rows (some 0.3 most of them), their new pages
        rows = case["sequences"] * (0.65 + 0.15 * (1 + case["most"]))
        return {"bytes": int(16 * case["sequences"] + 12 * rows + 8 * rows / case["page"]), "flops": int(4 * rows)}
    cells, wide = case["rows"] * case["cols"], BYTES[case["dtype"]]
    matrix = 1 if case["gate"] == "matrix" else 0
    both = 2 if case["norms"] == "both" else 1
    if case["op"] == "block_norm":
        return {"bytes": cells * wide * ((3 if case["norms"] == "after" else 4) + matrix), "flops": cells * (4 + 3 * both)}
    # two gradients out; in: the stream's gradient, with the norm before the next block its own and h, and x where a norm or a gate takes it
    matrices = 3 + (2 if case["norms"] != "after" else 0) + (1 if case["norms"] != "before" or case["gate"] != "none" else 0)
    return {"bytes": cells * wide * (matrices + 2 * matrix), "flops": cells * (4 + 9 * both)}


# ---- in 64 bits, from the definitions ---------------------------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](s, case)


def _exact_attention(s, case):
    """Sequence by sequence, its keys picked out page by page."""
    got = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    sees, at, page, times = _sees(case), 0, case["page"], case["q_heads"] // case["k_heads"]
    for n, (rows, keys) in enumerate(_batch(case)):
        mine = sees[at:at + rows]
        low = min(a for a, _, _ in mine)
        j = torch.arange(low, keys, device="cuda")
        slot = s["table"][n].long()[j // page] * page + j % page
        k, v = (codes.view(torch.int8)[slot].view(codes.dtype).double() * torch.repeat_interleave(scales[slot].double(), case["group"], -1)
                for codes, scales in (s["k_cache"], s["v_cache"]))
        a, b = torch.tensor([m[:2] for m in mine], device="cuda").T
        hidden = (j < a[:, None]) | (j > b[:, None])
        place = torch.arange(keys - rows, keys, device="cuda")
        for h in range(case["q_heads"]):
            z = s["q"][at:at + rows, h].double() @ k[:, h // times].T * case["dim"] ** -0.5
            if case["cap"]:
                z = torch.tanh(z / case["cap"]) * case["cap"]
            if s["slopes"] is not None:
                z = z - float(s["slopes"][h]) * torch.abs(j - place[:, None])
            p = torch.softmax(z.masked_fill(hidden, -math.inf), -1)
            got[at:at + rows, h] = torch.nan_to_num(p) @ v[:, h // times]
        at += rows
    return got


def _exact_block_norm(s, case):
    x = s["x"].double()
    if case["norms"] != "before":
        x = x * torch.rsqrt(x.square().sum(1, keepdim=True) / case["cols"] + EPS) * s["weight"].double()
    h = case["residual_scale"] * s["residual"].double() + (1.0 if s["gate"] is None else s["gate"].double()) * x
    if case["norms"] == "after":
        return h
    return h * torch.rsqrt(h.square().sum(1, keepdim=True) / case["cols"] + EPS) * s["next_weight"].double(), h


def _exact_norm_gradient(g, x, w):
    """Through x w r, r = (mean x^2 + eps)^-1/2: gradients of x and w."""
    r = torch.rsqrt(x.square().sum(1, keepdim=True) / x.shape[1] + EPS)
    dot = torch.einsum("rc,rc->r", g * w, x)[:, None]
    return r * w * g - x * r ** 3 * dot / x.shape[1], torch.einsum("rc,rc->c", g, x * r)


def _exact_block_norm_backward(s, case):
    x, h, d = s["x"].double(), s["h"].double(), s["dh"].double()
    last = []
    if case["norms"] != "after":
        through, dnext = _exact_norm_gradient(s["dy"].double(), h, s["next_weight"].double())
        d, last = d + through, [dnext]
    got = [d * case["residual_scale"]]
    if s["gate"] is not None:
        u = x
        if case["norms"] != "before":
            u = x * torch.rsqrt(x.square().sum(1, keepdim=True) / case["cols"] + EPS) * s["weight"].double()
        got.append(torch.einsum("rc,rc->c", d, u) if case["gate"] == "vector" else d * u)
        d = d * s["gate"].double()
    if case["norms"] != "before":
        d, dweight = _exact_norm_gradient(d, x, s["weight"].double())
        got.append(dweight)
    return (d, *got, *last)


def _exact_extend(s, case):
    """Sequence by sequence, on the host."""
    page, width, rows = case["page"], s["table"].shape[1], s["rows"]
    table, free = s["table"].tolist(), s["free"].tolist()
    left, asked, offsets, slots, positions, lengths = int(s["free_count"]), 0, [0], [], [], []
    most = left
    for n, (length, count) in enumerate(zip(s["lengths"].tolist(), s["counts"].tolist())):
        held, wanted = -(-length // page), -(-(length + count) // page)
        fits = wanted <= width
        need = wanted - held if fits else 0
        asked += need
        served = fits and (need == 0 or asked <= most)
        if served:
            for p in range(held, wanted):
                left -= 1
                table[n][p] = free[left]
        offsets.append(offsets[-1] + count)
        for p in range(length, length + count):
            slots.append(table[n][p // page] * page + p % page if served else -1)
            positions.append(p)
        lengths.append(length + count if served else length)
    slots = slots[:rows] + [-1] * (rows - len(slots))
    positions = positions[:rows] + [0] * (rows - len(positions))
    return (_int32(table), _int32(offsets), torch.tensor(slots, device="cuda"), _int32(positions), _int32(lengths), _int32([left]))
