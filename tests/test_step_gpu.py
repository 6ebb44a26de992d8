"""The operators around a decoder's cache on a GPU, against their plain 64-bit
forms: pages of a step, attention over the cache, norms around a block."""
import math
import random

import pytest
import torch

import row_reduction_gb300 as mt
from decoder_util import DTYPES, check, half_step
from step_util import (attention_ref, block_norm_back_ref, block_norm_ref,
                       extend_ref)

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---- pages of a step ---------------------------------------------------------
def extend_check(table, lengths, counts, free, free_count, page, rows,
                 out=None):
    want = extend_ref(table, lengths, counts, free, free_count, page, rows)
    width = len(table[0]) if table else 3
    t = i32(table) if table else torch.empty(0, width, dtype=torch.int32,
                                             device="cuda")
    step = mt.cache_extend(t, i32(lengths), i32(counts), i32(free),
                           i32([free_count]), page, rows, out=out)
    got = (t, step.offsets, step.slots, step.positions, step.lengths,
           step.free_count[0])
    assert step.slots.dtype == torch.int64
    for name, g, w in zip(("table", "offsets", "slots", "positions",
                           "lengths", "free_count"), got, want):
        assert g.tolist() == w, name
    return step


@pytest.mark.parametrize("sequences", [0, 1, 2, 31, 33, 257, 1025, 4097,
                                       9000])
@pytest.mark.parametrize("page", [1, 16, 24])
@pytest.mark.parametrize("short", [False, True])
def test_extend(sequences, page, short):
    rng = random.Random(sequences * 100 + page)
    most = 40 if sequences < 2000 else 3
    lengths = [rng.choice([0, 1, page, rng.randint(0, 200)])
               for _ in range(sequences)]
    counts = [rng.choice([0, 1, 1, rng.randint(0, most)])
              for _ in range(sequences)]
    width = -(-(200 + most) // page)
    pages = list(range(5 * sequences * width + 50))
    rng.shuffle(pages)
    table = [[pages.pop() if p < -(-n // page) else -1 for p in range(width)]
             for n in lengths]
    need = sum(-(-(a + b) // page) - -(-a // page)
               for a, b in zip(lengths, counts))
    free = pages[:need + 7]
    extend_check(table, lengths, counts, free,
                 need // 2 if short else need + 3, page, sum(counts) + 5)


def test_extend_edges():
    free = list(range(100, 160))
    # nothing free; nothing needed beside what is needed
    extend_check([[1, -1], [2, -1]], [3, 4], [1, 1], free, 0, 4, 4)
    # a sequence past its table's width gets none, the next one does
    extend_check([[1, 2], [3, -1]], [7, 3], [2, 5], free, 9, 4, 9)
    # the first that fails leaves none for those after that need some, though
    # there would be enough; those that need none go on
    extend_check([[-1] * 9, [-1] * 9, [5] + [-1] * 8], [0, 0, 1],
                 [33, 4, 2], free, 8, 4, 50)
    # exactly enough; one too few
    for left in (3, 2):
        extend_check([[-1, -1], [-1, -1]], [0, 0], [8, 4], free, left, 4, 12)
    # fewer rows than the batch has, and none
    extend_check([[-1, -1], [-1, -1]], [0, 0], [8, 4], free, 9, 4, 5)
    extend_check([[-1, -1], [-1, -1]], [0, 0], [8, 4], free, 9, 4, 0)
    # negative lengths, counts and free counts, one past the list
    extend_check([[-1, -1], [-1, -1]], [-5, 0], [3, -2], free, -1, 4, 5)
    extend_check([[-1, -1], [-1, -1]], [-5, 0], [3, -2], free, 1000, 4, 5)
    # a length that passes 31 bits; a hole in the pages that are there
    extend_check([[1, -1], [2, -1]], [2 ** 31 - 2, 1], [2, 1], free, 9, 4, 5)
    extend_check([[-1, -1]], [2], [1], free, 9, 4, 3)
    # no width, no list
    t = torch.empty(2, 0, dtype=torch.int32, device="cuda")
    step = mt.cache_extend(t, i32([0, 0]), i32([1, 0]), i32([]), i32([5]), 16,
                           3)
    assert step.slots.tolist() == [-1, -1, -1]
    assert step.lengths.tolist() == [0, 0]
    assert step.free_count.tolist() == [0]
    # huge counts: the offsets end at the type's largest
    big = 2 ** 31 - 1
    step = mt.cache_extend(i32([[-1]] * 3), i32([0] * 3), i32([big] * 3),
                           i32([1]), i32([1]), 2 ** 31 - 1, 4)
    assert step.offsets.tolist() == [0, big, big, big]
    assert step.slots.tolist() == [2 ** 31 - 1 + r for r in range(4)]


def test_extend_step_by_step():
    """Sequences grow token by token from their own outputs; every slot is
    given out once."""
    rng = random.Random(5)
    n, page, width = 37, 8, 40
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    free = i32(rng.sample(range(400), 400))
    lengths, left = i32([0] * n), i32([400])
    seen = set()
    for _ in range(30):
        counts = [rng.choice([0, 1, 1, 5]) for _ in range(n)]
        rows = sum(counts)
        step = mt.cache_extend(table, lengths, i32(counts), free, left, page,
                               rows + 2)
        slots = step.slots.tolist()
        assert slots[rows:] == [-1, -1]
        assert not seen & set(slots[:rows]) and len(set(slots[:rows])) == rows
        seen |= set(slots[:rows])
        # the slots are those that the table names
        again = mt.cache_slots(table, step.offsets, lengths, page, rows + 2)
        assert torch.equal(again, step.slots)
        lengths, left = step.lengths, step.free_count
    used = int((table >= 0).sum())
    assert used == 400 - int(left) and \
        used == sum(-(-v // page) for v in lengths.tolist())


# ---- attention over the cache ------------------------------------------------
def cache_of(g, slots, heads, dim, group, fmt, spread=0.5):
    codes, scales = mt.cache_alloc(slots, heads, dim, group, fmt)
    top = 448.0 if fmt == "e4m3" else 127.0
    x = (torch.randn(slots, heads, dim, generator=g, device="cuda") * top /
         4).clamp(-top, top)
    codes = x.to(codes.dtype) if fmt == "e4m3" else x.round().to(torch.int8)
    scales = torch.exp(spread * torch.randn(scales.shape, generator=g,
                                            device="cuda")) * 4 / top
    return codes, scales


def attention_inputs(seed, batch, q_heads, heads, dim, group, page, fmt,
                     dtype, before=0, behind=0, extra=1, spread=0.5):
    """batch: (rows, keys) of each sequence."""
    g = gen(seed)
    need = [-(-max(k, 0) // page) for _, k in batch]
    pool = sum(need) + 2
    order = torch.randperm(pool, generator=g, device="cuda").int()
    width = max(need + [0]) + extra
    table = torch.full((len(batch), width), -1, dtype=torch.int32,
                       device="cuda")
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    offs = [before]
    for r, _ in batch:
        offs.append(offs[-1] + r)
    q = randn(g, offs[-1] + behind, q_heads, dim, dtype=dtype)
    return dict(
        q=q, k_cache=cache_of(g, pool * page, heads, dim, group, fmt, spread),
        v_cache=cache_of(g, pool * page, heads, dim, group, fmt, spread),
        table=table, offsets=i32(offs), starts=i32([k - r for r, k in batch]),
        page=page)


def attention_check(a, out=None, **kw):
    """Runs and compares; rows outside the batch keep what was there."""
    q = a["q"]
    if out is None:
        out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    got, lse = mt.cache_attention(
        q, a["k_cache"], a["v_cache"], a["table"], a["offsets"], a["starts"],
        a["page"], out=out, return_lse=True, **kw)
    assert got is out
    ref, err, rlse, lerr, there = attention_ref(
        q, a["k_cache"], a["v_cache"], a["table"], a["offsets"], a["starts"],
        a["page"], **kw)
    ref[~there] = 7.0
    check(out, ref, err + half_step(torch.nan_to_num(ref), q.dtype), "out")
    check(lse, rlse, lerr + torch.nan_to_num(rlse, neginf=0.0).abs() * 2e-7,
          "lse")
    return out


SHAPES = [
    # query heads, key heads, dim, group, page
    (8, 2, 128, 128, 16), (8, 2, 128, 64, 16), (6, 3, 128, 32, 24),
    (4, 4, 64, 64, 1), (10, 2, 64, 32, 32), (15, 5, 80, 80, 24),
    (3, 1, 96, 96, 7), (16, 2, 96, 48, 16), (4, 2, 256, 256, 16),
    (9, 1, 256, 64, 64), (2, 1, 256, 32, 16), (24, 1, 128, 128, 16),
    (4, 2, 32, 32, 16), (4, 2, 64, 16, 16), (5, 1, 112, 16, 16),
    # sizes that no matrix instruction takes
    (2, 1, 1, 1, 3), (4, 2, 7, 7, 16), (2, 2, 100, 20, 16), (3, 1, 72, 8, 16),
    (4, 1, 512, 512, 16), (2, 1, 320, 160, 16), (1, 1, 511, 73, 5),
]
BATCHES = {
    "one": [(1, 1)],
    "tokens": [(1, 1), (1, 15), (1, 16), (1, 17), (1, 33), (1, 200)],
    "ragged": [(3, 40), (0, 10), (1, 300), (5, 5), (2, 65), (0, 0), (9, 129)],
    "long": [(1, 2900), (2, 1)],
    "chunk": [(70, 100), (33, 33), (1, 64)],
}


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("batch", sorted(BATCHES))
def test_attention(dt, fmt, shape, batch):
    hq, hk, dim, group, page = shape
    rows = [(r, max(r, k)) for r, k in BATCHES[batch]]
    a = attention_inputs(hq * 1000 + dim, rows, hq, hk, dim, group, page, fmt,
                         DTYPES[dt], before=2, behind=3)
    attention_check(a)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(8, 2, 128, 64, 16), (3, 1, 80, 80, 24),
                                   (2, 1, 20, 10, 16)], ids=str)
@pytest.mark.parametrize("batch", ["tokens", "ragged", "chunk"])
@pytest.mark.parametrize("kind", ["cap", "slopes", "window", "first", "last",
                                  "empty", "all", "holes"])
def test_attention_options(dt, shape, batch, kind):
    hq, hk, dim, group, page = shape
    rows = [(r, max(r, k)) for r, k in BATCHES[batch]]
    a = attention_inputs(hq + dim, rows, hq, hk, dim, group, page, "e4m3",
                         DTYPES[dt], behind=1)
    n = a["q"].shape[0]
    rng = random.Random(dim + n)
    p = []
    for r, k in rows:
        p += range(k - r, k)
    p += [0]
    slopes = torch.exp2(-torch.arange(1, hq + 1, device="cuda").float())
    kw = {}
    if kind in ("cap", "all"):
        kw["cap"] = 1.5     # most scores are well inside the bend
    if kind in ("slopes", "all"):
        kw["slopes"] = slopes
    if kind in ("window", "all"):
        kw["window"] = 13
    if kind in ("first", "all"):
        kw["first"] = i32([rng.choice([-3, 0, v // 2, v]) for v in p])
    if kind in ("last", "all"):
        # a prefix behind the row itself, past all keys, and before the row
        kw["last"] = i32([rng.choice([v, v + 9, 2 ** 31 - 1, v // 2])
                          for v in p])
    if kind == "empty":
        # bounds that leave nothing, at their extremes too
        kw["first"] = i32([rng.choice([v + 1, 2 ** 31 - 1, 0]) for v in p])
        kw["last"] = i32([rng.choice([v, -1, -2 ** 31]) for v in p])
    if kind == "holes":
        # pages that are not there: some, and all of a sequence's
        t = a["table"]
        t[torch.rand(t.shape, generator=gen(3), device="cuda") < 0.4] = -1
        t[0] = -1
        t[-1, 0] = 2 ** 31 - 1    # past the cache's slots
        kw["scale"] = -0.2
    attention_check(a, **kw)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("heads", [(80, 1), (70, 2), (9, 3), (130, 1)],
                         ids=str)
@pytest.mark.parametrize("batch", ["tokens", "chunk"])
def test_attention_many_query_heads(dt, fmt, heads, batch):
    """Query heads of a key head that take several tiles, and numbers that
    fill none."""
    rows = [(r, max(r, k)) for r, k in BATCHES[batch]]
    a = attention_inputs(sum(heads), rows, *heads, 64, 64, 16, fmt,
                         DTYPES[dt], behind=2)
    attention_check(a, window=100)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(8, 2, 128, 128), (4, 1, 96, 96),
                                   (6, 2, 64, 32)], ids=str)
@pytest.mark.parametrize("kind", ["plain", "prefix", "documents", "window"])
def test_attention_prompts(dt, shape, kind):
    """Prompts whose rows fill tiles of 64 columns, cut wherever the CTAs'
    shares of the work end."""
    hq, hk, dim, group = shape
    rows = [(200, 900), (64, 64), (0, 0), (65, 1000), (1, 700), (130, 131)]
    a = attention_inputs(dim, rows, hq, hk, dim, group, 16, "e4m3",
                         DTYPES[dt], before=1, behind=2)
    p = [0] + [v for r, k in rows for v in range(k - r, k)] + [0, 0]
    kw = {}
    if kind == "prefix":
        kw = dict(last=i32([max(v, 333) for v in p]), cap=5.0)
    elif kind == "documents":
        kw = dict(first=i32([v // 50 * 50 for v in p]),
                  slopes=torch.rand(hq, generator=gen(1), device="cuda") / 9)
    elif kind == "window":
        kw = dict(window=70)
    out = attention_check(a, **kw).clone()
    assert torch.equal(out, attention_check(a, **kw))


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim,group", [(128, 128), (64, 32), (30, 10)])
def test_attention_strided_views(dt, dim, group):
    """q out of a fused projection, out into a wider buffer, heads before
    tokens."""
    dtype = DTYPES[dt]
    a = attention_inputs(4, [(3, 50), (1, 9)], 6, 2, dim, group, 16, "int8",
                         dtype)
    q = a["q"]
    wide = randn(gen(5), 4, 10, dim, dtype=dtype)
    wide[:, 2:8] = q
    a["q"] = wide[:, 2:8]
    room = torch.full((4, 9, dim), 3.0, dtype=dtype, device="cuda")
    attention_check(a, out=room[:, 1:7])
    assert bool((room[:, 0] == 3).all() and (room[:, 7:] == 3).all())
    flat = torch.full((6, 4, dim + 3), 3.0, dtype=dtype, device="cuda")
    a["q"] = q.transpose(0, 1).contiguous().transpose(0, 1)
    attention_check(a, out=flat[:, :, 1:-2].transpose(0, 1))
    assert bool((flat[:, :, 0] == 3).all() and (flat[:, :, -2:] == 3).all())
    # the same query for all rows
    a["q"] = q[:1].expand(4, -1, -1)
    attention_check(a)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("dim,group", [(128, 64), (64, 64), (24, 8)])
def test_attention_not_a_number(dt, dim, group):
    """What a row does not see has no effect on it, NaN included; a NaN that
    it sees makes it NaN, out of the values in its group alone."""
    dtype = DTYPES[dt]
    batch = [(6, 40), (1, 30), (1, 1), (2, 50)]
    a = attention_inputs(6, batch, 4, 2, dim, group, 16, "e4m3", dtype)
    flat = [i for i in range(10)]
    slot = mt.cache_slots(a["table"], i32([0, 64, 128, 192, 256]),
                          i32([0] * 4), 16, 256)

    def where(s, j):
        return int(slot[64 * s + j])
    # keys and values behind the last row, on pages' ends
    for s, (_, n) in enumerate(batch):
        for j in range(n, -(-n // 16) * 16):
            for c in (a["k_cache"], a["v_cache"]):
                c[1][where(s, j)] = math.nan
                c[0].view(torch.int8)[where(s, j)] = 0x7f  # a NaN code
    attention_check(a)
    # key 37 of sequence 0: rows 3, 4, 5 see it, and head 1 alone
    for name in ("k_cache", "v_cache"):
        b = dict(a)
        codes, scales = a[name]
        scales, codes = scales.clone(), codes.clone()
        scales[where(0, 37), 1, 0] = math.nan
        codes.view(torch.int8)[where(0, 37), 1, :group] = 0
        b[name] = (codes, scales)
        out = attention_check(b)
        bad = torch.isnan(out)
        want = torch.zeros_like(bad)
        want[3:6, 2:4] = True
        if name == "v_cache":
            want[3:6, 2:4, group:] = False
        assert torch.equal(bad, want)
        # and with a window or a document that leaves it out none
        assert not bool(torch.isnan(attention_check(
            b, last=i32([min(v, 36) for v in
                         list(range(34, 40)) + [29, 0, 48, 49]]))).any())
    # a query's NaN or infinity
    for v in (math.nan, math.inf):
        b = dict(a, q=a["q"].clone())
        b["q"][6, 1, dim // 2] = v
        out, lse = mt.cache_attention(b["q"], b["k_cache"], b["v_cache"],
                                      b["table"], b["offsets"], b["starts"],
                                      16, return_lse=True)
        bad = torch.isnan(out)
        assert bool(bad[6, 1].all()) and int(bad.sum()) == dim
        assert torch.isnan(lse).nonzero().tolist() == [[6, 1]]
    assert flat


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("dim,group", [(128, 32), (64, 64), (12, 12)])
def test_attention_extreme_scales(dt, dim, group):
    """Scales far apart, between keys and between the groups of a key, of the
    seen and of the unseen; queries large and tiny; scores so large that one
    key takes all."""
    dtype = DTYPES[dt]
    a = attention_inputs(8, [(1, 90), (3, 70)], 4, 2, dim, group, 16, "int8",
                         dtype, spread=8.0)
    attention_check(a, scale=1e-3)
    # one key's values 2^60 times the others', with next to no weight
    b = attention_inputs(9, [(1, 90), (3, 70)], 4, 2, dim, group, 16, "int8",
                         dtype)
    slot = mt.cache_slots(b["table"], i32([0, 90, 160]), i32([0, 0]), 16, 160)
    b["v_cache"][1][slot[5]] *= 2.0 ** 60
    sl = torch.full((4,), 1.0, device="cuda")
    attention_check(b, slopes=sl)
    b["v_cache"][1][slot[5]] *= 2.0 ** 30
    attention_check(b, slopes=sl)
    for big in (1e-20, 1e-30, 1e10):
        c = dict(b, q=(b["q"].double() * big).to(dtype))
        attention_check(c, scale=1.0 / big / 8)
    attention_check(b, scale=30.0)


def test_attention_far_slots():
    """Slots whose codes lie behind 2^32 bytes."""
    slots, heads, dim, page = 4_300_000, 8, 128, 16
    g = gen(10)
    base = slots // page - 8
    codes = torch.zeros(slots, heads, dim, dtype=torch.int8, device="cuda")
    scales = torch.ones(slots, heads, 1, device="cuda")
    small = cache_of(g, 128, heads, dim, dim, "int8")
    codes[-128:], scales[-128:] = small
    table = (base + torch.randperm(8, generator=g, device="cuda")).int()[None]
    q = randn(g, 2, 16, dim, dtype=torch.bfloat16)
    offs, starts = i32([0, 2]), i32([101])
    got = mt.cache_attention(q, (codes, scales), (codes, scales), table, offs,
                             starts, page)
    want = mt.cache_attention(q, small, small, table - base, offs, starts,
                              page)
    assert torch.equal(got, want)


@pytest.mark.parametrize("sequences", [700, 5000])
def test_attention_many_sequences(sequences):
    rng = random.Random(sequences)
    batch = [(rng.choice([0, 1, 1, 1, 2]), rng.randint(2, 40))
             for _ in range(sequences)]
    a = attention_inputs(11, batch, 4, 2, 64, 64, 16, "e4m3", torch.bfloat16,
                         behind=2)
    out = torch.full(a["q"].shape, 7.0, dtype=torch.bfloat16, device="cuda")
    mt.cache_attention(a["q"], a["k_cache"], a["v_cache"], a["table"],
                       a["offsets"], a["starts"], 16, out=out)
    # a sample of them by themselves
    offs = a["offsets"].tolist()
    for s in rng.sample(range(sequences), 60):
        lo, hi = offs[s], offs[s + 1]
        if lo == hi:
            continue
        ref, err, *_ = attention_ref(
            a["q"][lo:hi], a["k_cache"], a["v_cache"], a["table"][s:s + 1],
            i32([0, hi - lo]), a["starts"][s:s + 1], 16)
        check(out[lo:hi], ref, err + half_step(ref, torch.bfloat16))
    assert bool((out[offs[-1]:] == 7).all())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("keys", [5000, 40000])
def test_attention_one_long_context(dt, keys):
    """Few rows and many keys: the keys are shared out and joined."""
    a = attention_inputs(12, [(2, keys), (1, 3)], 8, 2, 128, 128, 16, "int8",
                         DTYPES[dt])
    first = attention_check(a).clone()
    again = attention_check(a)
    assert torch.equal(first, again)      # the same bits each time
    attention_check(a, window=keys // 2, cap=20.0)
    # all of the weight on single keys near a far end
    sl = torch.full((8,), 3.0, device="cuda")
    attention_check(a, slopes=sl)
    attention_check(a, slopes=-sl / 1000)


# ---- norms around a block ----------------------------------------------------
def norm_inputs(seed, rows, cols, dtype, gate, norms, weights=True):
    g = gen(seed)
    w = (lambda: (1 + 0.3 * randn(g, cols)).to(dtype)) if weights else \
        (lambda: None)
    gates = {"none": lambda: None,
             "vector": lambda: (0.5 + 0.5 * randn(g, cols)).to(dtype),
             "matrix": lambda: (0.5 + 0.5 * randn(g, rows, cols)).to(dtype)}
    gain = torch.exp(randn(g, cols))
    return dict(x=(randn(g, rows, cols) * gain).to(dtype),
                residual=(2 * randn(g, rows, cols)).to(dtype),
                weight=w() if norms != "before" else None,
                gate=gates[gate](),
                next_weight=w() if norms != "after" else None, norms=norms)


def norm_check(a, residual_scale=1.0, eps=1e-6, **kw):
    got = mt.block_norm(**a, residual_scale=residual_scale, eps=eps, **kw)
    y, h = (None, got) if a["norms"] == "after" else got
    ry, ye, rh, he = block_norm_ref(
        a["x"], a["residual"], a["weight"], a["gate"], a["next_weight"],
        a["norms"], residual_scale, eps)
    dtype = a["x"].dtype
    check(h, rh, he + half_step(rh, dtype), "h")
    if y is not None:
        check(y, ry, ye + half_step(ry, dtype), "y")
    return y, h


def back_check(a, seed, residual_scale=1.0, eps=1e-6, dh=True, **kw):
    dtype, (rows, cols), norms = a["x"].dtype, a["x"].shape, a["norms"]
    g = gen(seed)
    dy = None if norms == "after" else randn(g, rows, cols).to(dtype)
    dh = randn(g, rows, cols).to(dtype) if dh else None
    h = None if norms == "after" else a["residual"]
    x = a["x"] if norms != "before" or a["gate"] is not None else None
    rest = (a["weight"], a["gate"], a["next_weight"], norms, residual_scale,
            eps)
    want = block_norm_back_ref(dy, dh, x, h, *rest)
    got = mt.block_norm_backward(dy, dh, x, h, *rest, **kw)
    assert len(got) == len(want)
    for i, (d, (ref, err)) in enumerate(zip(got, want)):
        t = dtype if d.dim() == 2 else torch.float32
        assert d.dtype == t
        check(d, ref, err + half_step(ref, t), f"gradient {i}")
    return got


NORM_SHAPES = [(1, 1), (3, 2), (5, 31), (2, 64), (7, 100), (4, 256), (9, 333),
               (3, 1000), (5, 1024), (6, 1237), (2, 2048), (3, 4096),
               (2, 5000), (3, 5120), (2, 7168), (3, 8191), (2, 8192),
               (2, 16384), (2, 16390), (1, 40001), (1, 65536), (333, 96),
               (1000, 24), (700, 1536)]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gate", ["none", "vector", "matrix"])
@pytest.mark.parametrize("norms", ["both", "before", "after"])
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=str)
def test_block_norm(dt, gate, norms, shape):
    a = norm_inputs(sum(shape), *shape, DTYPES[dt], gate, norms)
    norm_check(a, residual_scale=0.7)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("gate", ["none", "vector", "matrix"])
@pytest.mark.parametrize("norms", ["both", "before", "after"])
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=str)
def test_block_norm_backward(dt, gate, norms, shape):
    a = norm_inputs(sum(shape), *shape, DTYPES[dt], gate, norms)
    back_check(a, 1, residual_scale=0.7)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("off", [1, 2, 3, 7])
@pytest.mark.parametrize("cols", [513, 1026, 3001, 8190])
def test_block_norm_off_the_packs_bounds(dt, off, cols):
    """Matrices that begin anywhere among 16-byte packs, each somewhere else,
    rows one after the other and apart; more rows than CTAs; in place."""
    dtype, rows = DTYPES[dt], 700 if cols < 2000 else 310
    a = norm_inputs(off, rows, cols, dtype, "matrix", "both")

    def moved(t, by, stride):
        flat = torch.full((rows * stride + by + 8,), 5.0, dtype=dtype,
                          device="cuda")
        v = flat.as_strided((rows, cols), (stride, 1), by)
        v.copy_(t)
        return v
    b = dict(a, x=moved(a["x"], off, cols),
             residual=moved(a["residual"], off + 2, cols + 1),
             gate=moved(a["gate"], 2 * off, cols + 3))
    out = moved(a["x"], off + 1, cols + 1)
    y, h = norm_check(b, out=out, h_out=b["residual"].clone())
    y0, h0 = norm_check(a)
    assert torch.equal(y, y0) and torch.equal(h, h0)
    got = back_check(b, 1)
    assert len(got) == 5
    g = gen(1)
    dy, dh = (randn(g, rows, cols, dtype=dtype) for _ in range(2))
    args = (a["weight"], a["gate"], a["next_weight"])
    want = mt.block_norm_backward(dy, dh, a["x"], h0, *args)
    dy, dh = moved(dy, off, cols), moved(dh, off + 5, cols)
    got = mt.block_norm_backward(dy, dh, a["x"], h0, *args, out=(dy, dh))
    for p, q in zip(got, want):
        assert torch.equal(p, q)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("norms", ["both", "before", "after"])
@pytest.mark.parametrize("shape", [(11, 1024), (5, 333), (2, 20000)], ids=str)
def test_block_norm_without_weights(dt, norms, shape):
    a = norm_inputs(3, *shape, DTYPES[dt], "none", norms, weights=False)
    norm_check(a)
    got = back_check(a, 2, dh=norms == "after")
    assert len(got) == 2


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(9, 1024), (9, 1237)], ids=str)
def test_block_norm_strides_and_in_place(dt, shape):
    """Rows out of wider matrices, one row for all, outputs in place."""
    rows, cols = shape
    dtype = DTYPES[dt]
    a = norm_inputs(4, rows, cols, dtype, "matrix", "both")
    wide = torch.full((rows, 2 * cols + 8), 5.0, dtype=dtype, device="cuda")
    b = dict(a, x=wide[:, 3:cols + 3], gate=wide[:, -cols:])
    wide[:, 3:cols + 3] = a["x"]
    wide[:, -cols:] = a["gate"]
    y, h = norm_check(b)
    y0, h0 = norm_check(a)
    room = torch.full((rows, cols + 5), 5.0, dtype=dtype, device="cuda")
    norm_check(a, out=room[:, 2:cols + 2])
    assert bool((room[:, :2] == 5).all() and (room[:, cols + 2:] == 5).all())
    # the same residual for all rows
    norm_check(dict(a, residual=a["residual"][:1].expand(rows, -1)))
    # one row's gate as a matrix: its gradient is a matrix
    back_check(dict(a, gate=a["gate"][:1].expand(rows, -1)), 3)
    # in place of the inputs
    c = {k: v.clone() if isinstance(v, torch.Tensor) else v
         for k, v in a.items()}
    y1, h1 = mt.block_norm(**c, out=c["x"], h_out=c["residual"])
    assert y1 is c["x"] and h1 is c["residual"]
    assert torch.equal(y1, y0) and torch.equal(h1, h0)
    g = gen(5)
    dy, dh = randn(g, rows, cols, dtype=dtype), randn(g, rows, cols,
                                                      dtype=dtype)
    args = (a["weight"], a["gate"], a["next_weight"])
    want = mt.block_norm_backward(dy, dh, a["x"], h0, *args)
    for dx, dres in ((0, 1), (1, 0), (2, 3)):
        t = [v.clone() for v in (dy, dh, a["x"], h0)]
        got = mt.block_norm_backward(*t, *args, out=(t[dx], t[dres]))
        for p, q in zip(got, want):
            assert torch.equal(p, q)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cols", [64, 1024, 1235, 4096])
def test_block_norm_gradients_add_every_row_once(dt, cols):
    """Whole numbers, and means of squares of 1: every term of a weight's and
    a gate's gradient is a whole number (within a few roundings), so a row
    left out or taken twice shows in every column."""
    rows, dtype = 1237, DTYPES[dt]
    g = gen(cols)

    def sign():
        return torch.randint(0, 2, (rows, cols), generator=g,
                             device="cuda") * 2 - 1
    x, h, dy = sign(), sign(), 2 * sign()
    # dy h sums to zero in pairs of columns, so that its mean adds nothing
    half = cols // 2
    x[:, half:2 * half], h[:, half:2 * half] = x[:, :half], h[:, :half]
    dy[:, half:2 * half] = -dy[:, :half]
    if cols % 2:
        dy[:, -1] = 0
    dh = 3 * sign()
    ones = torch.ones(cols, dtype=dtype, device="cuda")
    t = [v.to(dtype) for v in (dy, dh, x, h)]
    got = mt.block_norm_backward(*t, ones, ones, ones, eps=0.0)
    e = (dh + dy).double()
    for d, want, size in ((got[2], e * x, e.abs()), (got[3], e * x, e.abs()),
                          (got[4], dy * h, dy.abs())):
        # 1/sqrt within 2 ulp, the mean's rounding; few roundings a row
        tol = size.double().sum(0) * 2.0 ** -20
        assert float(tol.max()) < 0.5
        check(d, want.double().sum(0), tol, "sum")


def test_block_norm_of_many_rows():
    """More rows than 2^31 values; many rows per block of the backward
    pass."""
    rows, cols = 540_000, 4096
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=gen(7))
    y, h = mt.block_norm(x, x, residual_scale=2.0)
    for r in (0, 1, 262_144, rows - 1):
        ry, ye, rh, he = block_norm_ref(x[r:r + 1], x[r:r + 1], None, None,
                                        None, "both", 2.0, 1e-6)
        check(y[r:r + 1], ry, ye + half_step(ry, torch.bfloat16))
        check(h[r:r + 1], rh, he + half_step(rh, torch.bfloat16))
    dx, dres = mt.block_norm_backward(y, None, x, h)
    for r in (0, 262_145, rows - 1):
        want = block_norm_back_ref(y[r:r + 1], None, x[r:r + 1], h[r:r + 1],
                                   None, None, None, "both", 1.0, 1e-6)
        for d, (ref, err) in zip((dx, dres), want):
            check(d[r:r + 1], ref, err + half_step(ref, torch.bfloat16))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [128, 1000, 1237, 20000])
def test_block_norm_keeps_rows_apart(dt, cols):
    """An infinity or a NaN stays in its row, and in a weight's gradient in
    its column (dh's: through no norm's sum)."""
    dtype = DTYPES[dt]
    a = norm_inputs(8, 9, cols, dtype, "vector", "both")
    y0, h0 = mt.block_norm(**a)
    a["x"][4, cols // 3] = math.nan
    a["residual"][6, 1] = math.inf
    y, h = mt.block_norm(**a)
    keep = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(y[keep], y0[keep]) and torch.equal(h[keep], h0[keep])
    assert bool(torch.isnan(h[4]).all() and torch.isnan(y[4]).all())
    assert int(torch.isinf(h[6]).sum()) == 1
    b = norm_inputs(9, 700, cols, dtype, "vector", "before")
    dy = randn(gen(1), 700, cols, dtype=dtype)
    dh = randn(gen(2), 700, cols, dtype=dtype)
    dh[300, cols - 1] = -math.inf
    out = mt.block_norm_backward(dy, dh, b["x"], b["residual"], None,
                                 b["gate"], b["next_weight"], "before")
    bad = ~torch.isfinite(out[0])
    assert bad.nonzero().tolist() == [[300, cols - 1]]
    assert (~torch.isfinite(out[2])).nonzero().flatten().tolist() == \
        [cols - 1]
    assert bool(torch.isfinite(out[3]).all())


@pytest.mark.parametrize("cols", [16, 1030])
def test_block_norm_zero_rows_and_empty_calls(cols):
    """Rows of zeros with and without eps, calls without rows."""
    z = torch.zeros(3, cols, device="cuda")
    y, h = mt.block_norm(z, z)
    assert bool((y == 0).all() and (h == 0).all())
    y, h = mt.block_norm(z, z, eps=0.0)
    assert bool(torch.isnan(y).all())
    none = torch.empty(0, cols, device="cuda")
    w = torch.ones(cols, device="cuda")
    y, h = mt.block_norm(none, none, w, w, w)
    assert y.shape == h.shape == (0, cols)
    got = mt.block_norm_backward(none, none, none, none, w, w, w)
    assert [tuple(t.shape) for t in got] == [(0, cols)] * 2 + [(cols,)] * 3
    assert all(bool((t == 0).all()) for t in got[2:])


# ---- streams, graphs, together -----------------------------------------------
def test_a_decode_step_around_the_cache():
    """Pages -> rows into the cache -> attention -> projection -> norms around
    the block, for three steps; then a step captured and replayed from new
    inputs and lengths, in two graphs on two streams at once."""
    g = gen(20)
    S, E, HQ, HK, D, PAGE, WIDTH = 5, 256, 8, 2, 64, 8, 12
    dt = torch.bfloat16
    wqkv = (randn(g, E, (HQ + 2 * HK) * D) / 16).to(dt)
    wout = (randn(g, HQ * D, E) / 22).to(dt)
    w1, w2, gate = ((1 + 0.1 * randn(g, E)).to(dt) for _ in range(3))
    tab = mt.rotary_frequencies(D)
    sl = torch.full((HQ,), 0.01, device="cuda")

    class Run:
        def __init__(self, seed):
            gg = gen(seed)
            self.k, self.v = (mt.cache_alloc(S * WIDTH * PAGE, HK, D, 32, f)
                              for f in ("e4m3", "e4m3"))
            self.table = torch.full((S, WIDTH), -1, dtype=torch.int32,
                                    device="cuda")
            self.free = torch.randperm(S * WIDTH, generator=gg,
                                       device="cuda").int()
            self.left = i32([S * WIDTH])
            self.lengths = i32([0] * S)
            self.counts = i32([3, 0, 9, 1, 30])
            self.rows = 48
            self.x = randn(gg, self.rows, E, dtype=dt)

        def step(self):
            st = mt.cache_extend(self.table, self.lengths, self.counts,
                                 self.free, self.left, PAGE, self.rows)
            q, k, v = (self.x @ wqkv).view(-1, HQ + 2 * HK, D).split(
                (HQ, HK, HK), 1)
            q, k = mt.rotary(q, k, st.positions, tab)
            mt.cache_write(k, v, self.k, self.v, st.slots)
            o = mt.cache_attention(q, self.k, self.v, self.table, st.offsets,
                                   self.lengths, PAGE, cap=20.0, slopes=sl,
                                   window=40)
            y, h = mt.block_norm(o.flatten(1) @ wout, self.x, w1, gate, w2)
            return st, q, o, y, h

        def verify(self, lengths, got):
            st, q, o, y, h = got
            ref, err, *_ = attention_ref(q, self.k, self.v, self.table,
                                         st.offsets, lengths, PAGE, cap=20.0,
                                         slopes=sl, window=40)
            check(o, ref, err + half_step(ref, dt))
            ry, ye, rh, he = block_norm_ref(o.flatten(1) @ wout, self.x, w1,
                                            gate, w2, "both", 1.0, 1e-6)
            check(y, ry, ye + half_step(ry, dt))
            check(h, rh, he + half_step(rh, dt))

    r = Run(21)
    for counts in ([3, 0, 9, 1, 30], [1, 1, 1, 1, 1], [0, 20, 4, 1, 2]):
        r.counts.copy_(i32(counts))
        got = r.step()
        assert got[0].offsets.tolist()[-1] == sum(counts)
        r.verify(r.lengths, got)
        r.lengths, r.left = got[0].lengths, got[0].free_count
    runs, graphs = [Run(22), Run(23)], []
    for run in runs:
        # one uncaptured step, on another stream
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            run.step()
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = run.step()
            old = run.lengths.clone()
            run.lengths.copy_(outs[0].lengths)
            run.left.copy_(outs[0].free_count)
        graphs.append((graph, outs, old))
    for counts in ([3, 0, 9, 1, 30], [1, 1, 1, 1, 1], [2, 5, 0, 1, 1]):
        for run in runs:
            run.counts.copy_(i32(counts))
            run.x.copy_(randn(g, run.rows, E, dtype=dt))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in runs]
        for (graph, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for run, (_, outs, old) in zip(runs, graphs):
            run.verify(old, outs)


def test_training_pass_captured():
    """Forward and backward captured with their workspace, in two graphs
    replayed at once on new inputs."""
    a = norm_inputs(30, 500, 1024, torch.bfloat16, "vector", "both")
    dy, dh = (randn(gen(s), 500, 1024, dtype=torch.bfloat16)
              for s in (31, 32))

    def both():
        y, h = mt.block_norm(**a)
        return (y, h, *mt.block_norm_backward(
            dy, dh, a["x"], h, a["weight"], a["gate"], a["next_weight"]))
    both()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = both()
        graphs.append((graph, outs))
    for seed in (33, 34):
        a["x"].copy_(randn(gen(seed), 500, 1024))
        torch.cuda.synchronize()
        for graph, _ in graphs:
            with torch.cuda.stream(torch.cuda.Stream()):
                graph.replay()
        torch.cuda.synchronize()
        want = both()
        for _, outs in graphs:
            for p, q in zip(outs, want):
                assert torch.equal(p, q)


def test_calls_from_several_threads():
    from concurrent.futures import ThreadPoolExecutor
    a = attention_inputs(40, [(2, 900), (1, 30)], 8, 2, 128, 128, 16, "e4m3",
                         torch.bfloat16)
    n = norm_inputs(41, 64, 1024, torch.bfloat16, "vector", "both")

    def both():
        o = mt.cache_attention(a["q"], a["k_cache"], a["v_cache"], a["table"],
                               a["offsets"], a["starts"], 16)
        y, h = mt.block_norm(**n)
        return (o, *mt.block_norm_backward(y, h, n["x"], h, n["weight"],
                                           n["gate"], n["next_weight"]))
    want = both()
    torch.cuda.synchronize()

    def work(_):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            outs = [both() for _ in range(10)]
        s.synchronize()
        return all(torch.equal(p, q) for o in outs for p, q in zip(o, want))
    with ThreadPoolExecutor(8) as ex:
        assert all(ex.map(work, range(8)))


def test_explicit_streams():
    a = attention_inputs(42, [(2, 90)], 4, 2, 64, 64, 16, "e4m3",
                         torch.bfloat16)
    want = mt.cache_attention(a["q"], a["k_cache"], a["v_cache"], a["table"],
                              a["offsets"], a["starts"], 16)
    n = norm_inputs(43, 7, 333, torch.float32, "vector", "both")
    wn = mt.block_norm(**n)
    ext = (i32([[-1, -1]]), i32([0]), i32([5]), i32([4, 3, 2]), i32([3]), 4,
           6)
    we = mt.cache_extend(*ext)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for st in (s, s.cuda_stream, 0):
        got = mt.cache_attention(a["q"], a["k_cache"], a["v_cache"],
                                 a["table"], a["offsets"], a["starts"], 16,
                                 stream=st)
        gn = mt.block_norm(**n, stream=st)
        ge = mt.cache_extend(*ext, stream=st)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        assert all(torch.equal(p, q) for p, q in zip(gn, wn))
        assert all(torch.equal(p, q) for p, q in zip(ge, we))


# ---- prompts on tensor memory -----------------------------------------------------
TALL = [(200, 900), (0, 0), (130, 131), (257, 64 * 12)]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("shape", [(8, 2, 128, 16), (6, 1, 64, 24), (3, 3, 128, 1),
                                   (140, 1, 64, 16), (7, 1, 128, 32)], ids=str)
@pytest.mark.parametrize("kind", ["plain", "cap", "prefix", "documents",
                                  "window", "empty", "holes"])
def test_attention_tall(fmt, shape, kind):
    """BF16 prompts of several tiles of 128 columns, cut wherever the CTAs'
    shares end; chunks that some rows, or none, see."""
    hq, hk, dim, page = shape
    rows = TALL if hq < 100 else [(5, 300), (3, 64)]
    if hq == hk:
        rows = [(500, 700), (410, 410)]
    a = attention_inputs(dim + hq, rows, hq, hk, dim, dim, page, fmt,
                         torch.bfloat16, before=1, behind=2)
    p = [0] + [v for r, k in rows for v in range(k - r, k)] + [0, 0]
    rng, kw = random.Random(hq), {}
    if kind == "cap":
        kw = dict(cap=1.5)
    elif kind == "prefix":
        kw = dict(last=i32([max(v, 333) for v in p]), cap=5.0)
    elif kind == "documents":
        kw = dict(first=i32([v // 50 * 50 for v in p]),
                  slopes=torch.rand(hq, generator=gen(1), device="cuda") / 9)
    elif kind == "window":
        kw = dict(window=70, slopes=torch.rand(hq, generator=gen(2),
                                               device="cuda"))
    elif kind == "empty":
        kw = dict(first=i32([rng.choice([v + 1, 2 ** 31 - 1, 0]) for v in p]),
                  last=i32([rng.choice([v, -1, -2 ** 31]) for v in p]))
    elif kind == "holes":
        t = a["table"]
        t[torch.rand(t.shape, generator=gen(3), device="cuda") < 0.4] = -1
        t[-1, 0] = 2 ** 31 - 1
        kw["scale"] = -0.2
    out = attention_check(a, **kw).clone()
    assert torch.equal(out, attention_check(a, **kw))


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("grow", [1e-4, 1.0, 30.0])
@pytest.mark.parametrize("values", [1e-30, 1.0, 1e30])
def test_attention_tall_moving_references(dim, grow, values):
    """Scores that run ahead of every chunk's reference, values' scales that
    leave the power of two of the chunks before, up and down."""
    a = attention_inputs(9, [(250, 640), (170, 170)], 4, 1, dim, dim, 16, "e4m3",
                         torch.bfloat16)
    a["q"] = a["q"].abs()
    a["k_cache"][0].copy_(a["k_cache"][0].float().abs().to(torch.float8_e4m3fn))
    # a key's place in its sequence, by its slot
    place = torch.zeros(a["k_cache"][0].shape[0], device="cuda")
    for row in a["table"]:
        for j, page in enumerate(row.tolist()):
            if page >= 0:
                place[page * 16:page * 16 + 16] = \
                    j * 16 + torch.arange(16, device="cuda")
    ks, vs = a["k_cache"][1], a["v_cache"][1]
    ks.mul_((1 + grow * place / 64)[:, None, None])
    vs.mul_((values * torch.exp2(12 * torch.sin(place / 40)))[:, None, None])
    attention_check(a)


def test_attention_tall_not_a_number():
    """What a row does not see has no effect on it; what it does has, on its own
    columns alone."""
    a = attention_inputs(10, [(300, 400)], 4, 2, 128, 128, 16, "int8",
                         torch.bfloat16)
    clean = attention_check(a).clone()
    at = int(a["table"][0, 250 // 16]) * 16 + 250 % 16   # seen from row 150 on
    for which, value in (("v_cache", math.nan), ("k_cache", math.nan),
                         ("v_cache", math.inf)):
        s = a[which][1]
        old = s[at, 1].clone()
        s[at, 1] = value
        got = mt.cache_attention(a["q"], a["k_cache"], a["v_cache"], a["table"],
                                 a["offsets"], a["starts"], 16)
        s[at, 1] = old
        assert torch.equal(got[:, :2], clean[:, :2])
        assert torch.equal(got[:150], clean[:150])
        assert not bool(torch.isfinite(got[150:, 2:]).any())
    q = a["q"].clone()
    q[7, 3, 5], q[200, 0, 0] = math.nan, -math.inf
    got = mt.cache_attention(q, a["k_cache"], a["v_cache"], a["table"],
                             a["offsets"], a["starts"], 16)
    bad = torch.zeros(300, 4, dtype=torch.bool, device="cuda")
    bad[7, 3] = bad[200, 0] = True
    assert torch.equal(got.isnan().all(-1), bad)
    assert torch.equal(got[~bad], clean[~bad])


def test_attention_tall_streams_and_graphs():
    """Two calls at once on two streams, of both head sizes (tensor memory is
    shared by what runs on an SM), and a captured one, replayed."""
    a = [attention_inputs(11 + d, [(300, 900), (200, 333)], 8, 2, d, d, 16,
                          "e4m3", torch.bfloat16) for d in (64, 128)]

    def call(x, out=None):
        return mt.cache_attention(x["q"], x["k_cache"], x["v_cache"], x["table"],
                                  x["offsets"], x["starts"], 16, out=out)
    want = [call(x) for x in a]
    streams = [torch.cuda.Stream() for _ in a]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for x, s in zip(a, streams):
            with torch.cuda.stream(s):
                got.append(call(x))
    torch.cuda.synchronize()
    for i, t in enumerate(got):
        assert torch.equal(t, want[i % 2])
    out = torch.zeros_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(a[1], out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[1])


@pytest.mark.parametrize("dim", [64, 128])
def test_attention_tall_strided_views(dim):
    a = attention_inputs(12, [(150, 300), (60, 61)], 6, 1, dim, dim, 16, "int8",
                         torch.bfloat16)
    q = a["q"]
    wide = randn(gen(5), 210, 9, dim + 1, dtype=torch.bfloat16)
    wide[:, 2:8, 1:] = q
    a["q"] = wide[:, 2:8, 1:]       # off any bound
    room = torch.full((6, 210, dim + 3), 3.0, dtype=torch.bfloat16,
                      device="cuda")
    attention_check(a, out=room[:, :, 1:-2].transpose(0, 1))
    assert bool((room[:, :, 0] == 3).all() and (room[:, :, -2:] == 3).all())


# ---- what device arrays may hold -----------------------------------------------
@pytest.mark.parametrize("dim,group", [(128, 64), (64, 64), (40, 40)])
@pytest.mark.parametrize("rows", [(3, 5), (100, 130), (400, 300)])
@pytest.mark.parametrize("window", [None, 20, 2 ** 40])
def test_attention_negative_starts(dim, group, rows, window):
    """Rows at negative positions see nothing; those behind them, in the same
    sequence, what a window leaves."""
    batch = [(rows[0], rows[0] - 2), (rows[1], rows[1] // 2), (4, 60)]
    a = attention_inputs(dim, batch, 4, 1, dim, group, 16, "e4m3",
                         torch.bfloat16)
    assert a["starts"].tolist()[:2] == [-2, rows[1] // 2 - rows[1]]
    attention_check(a, window=window)


@pytest.mark.parametrize("dim,group", [(128, 64), (64, 64), (40, 40)])
@pytest.mark.parametrize("rows", [5, 150])
def test_attention_offsets_past_the_rows(dim, group, rows):
    """Offsets that leave the call's rows are cut at them: fewer rows of q
    than the step has."""
    a = attention_inputs(dim, [(rows, rows + 40), (rows, 2 * rows)], 4, 1, dim,
                         group, 16, "int8", torch.float16)
    q = a["q"][:rows + 3]
    args = (a["k_cache"], a["v_cache"], a["table"])
    want = mt.cache_attention(q, *args, i32([0, rows, rows + 3]), a["starts"],
                              16)
    for offs in ([0, rows, 2 * rows], [-7, rows, 2 ** 31 - 1]):
        room = torch.full((2 * rows, 4, dim), 3.0, dtype=q.dtype,
                          device="cuda")
        mt.cache_attention(q, *args, i32(offs), a["starts"], 16,
                           out=room[:rows + 3])
        assert torch.equal(room[:rows + 3], want)
        assert bool((room[rows + 3:] == 3).all())


@pytest.mark.parametrize("sequences", [3, 5000])
def test_extend_fewer_rows_than_tokens(sequences):
    n = torch.arange(sequences, dtype=torch.int32, device="cuda") % 5
    free = torch.arange(2 * sequences, dtype=torch.int32, device="cuda")
    count = i32([2 * sequences])
    got = []
    for rows in (int(n.sum()), 4):
        table = torch.full((sequences, 2), -1, dtype=torch.int32,
                           device="cuda")
        got.append((mt.cache_extend(table, n, n, free, count, 4, rows), table))
    (all_, t0), (few, t1) = got
    assert torch.equal(t0, t1)
    for name in ("offsets", "lengths", "free_count"):
        assert torch.equal(getattr(all_, name), getattr(few, name))
    n = min(4, all_.slots.shape[0])   # behind all of them: padding
    assert torch.equal(all_.slots[:n], few.slots[:n])
    assert torch.equal(all_.positions[:n], few.positions[:n])


def test_more_refusals():
    a = attention_inputs(51, [(1, 9), (2, 5)], 4, 2, 64, 32, 16, "e4m3",
                         torch.bfloat16)
    args = (a["q"], a["k_cache"], a["v_cache"], a["table"], a["offsets"],
            a["starts"])
    with pytest.raises(mt.MTError):
        mt.cache_attention(*args, 16, out=a["q"])
    for kw in (dict(page_size=2 ** 31), dict(page_size=16, cap=1e-50),
               dict(page_size=16, scale=1e39)):
        with pytest.raises((ValueError, mt.MTError)):
            mt.cache_attention(*args, **kw)
    x = torch.ones(2, 8, device="cuda")
    with pytest.raises((ValueError, mt.MTError)):
        mt.block_norm(x, x, residual_scale=1e39)
    one = i32([0])
    with pytest.raises(ValueError):
        mt.cache_extend(i32([[0]]), one, one, i32([]), i32([0]), 2 ** 31, 1)


# ---- refusals of the binding -------------------------------------------------
def test_extend_refuses():
    t, n, f, c = i32([[-1, -1]]), i32([0]), i32([4, 3]), i32([2])
    for err, args in (
            (TypeError, (t.long(), n, n, f, c, 4, 2)),
            (ValueError, (i32([[-1], [-1]]), n, n, f, c, 4, 2)),
            (ValueError, (t.cpu(), n, n, f, c, 4, 2)),
            (ValueError, (t.expand(1, 2)[:, ::2].expand(1, 1), i32([0, 1]), n,
                          f, c, 4, 2)),
            (TypeError, (t, n.long(), n, f, c, 4, 2)),
            (ValueError, (t, n, i32([0, 1]), f, c, 4, 2)),
            (ValueError, (t, n, n, f.view(1, 2), c, 4, 2)),
            (ValueError, (t, n, n, f, i32([1, 2]), 4, 2)),
            (TypeError, (t, n, n, f, c.float(), 4, 2)),
            (TypeError, (t, n, n, f, 2, 4, 2)),
            (mt.MTError, (t, n, n, f, c, 0, 2))):
        with pytest.raises(err):
            mt.cache_extend(*args)
    step = mt.cache_extend(t, n, n, f, c, 4, 2)
    with pytest.raises(mt.MTError):   # an output that is an input
        mt.cache_extend(t, step.lengths, n, f, c, 4, 2, out=step)
    with pytest.raises(ValueError, match="slots"):
        mt.cache_extend(t, n, n, f, c, 4, 3, out=step)


def test_attention_refuses():
    a = attention_inputs(50, [(1, 9), (2, 5)], 4, 2, 64, 32, 16, "e4m3",
                         torch.bfloat16)
    base = dict(q=a["q"], k_cache=a["k_cache"], v_cache=a["v_cache"],
                table=a["table"], offsets=a["offsets"], starts=a["starts"],
                page_size=16)
    codes, scales = a["k_cache"]
    for err, kw in (
            (ValueError, dict(q=a["q"][0])),
            (ValueError, dict(q=a["q"].cpu())),
            (TypeError, dict(q=a["q"].double())),
            (ValueError, dict(q=a["q"][:, :3])),
            (ValueError, dict(q=a["q"][:, :0])),
            (ValueError, dict(q=a["q"][..., :32])),
            (ValueError, dict(q=a["q"].transpose(1, 2))),
            (TypeError, dict(k_cache=(codes.float(), scales))),
            (ValueError, dict(v_cache=(codes[1:], scales[1:]))),
            (TypeError, dict(v_cache=(codes.view(torch.int8), scales))),
            (TypeError, dict(table=a["table"].long())),
            (ValueError, dict(table=a["table"][:1])),
            (ValueError, dict(offsets=a["offsets"][:2])),
            (TypeError, dict(offsets=a["offsets"].long())),
            (TypeError, dict(starts=a["starts"].long())),
            (ValueError, dict(first=i32([0, 0]))),
            (TypeError, dict(last=torch.zeros(3, device="cuda"))),
            (ValueError, dict(slopes=torch.zeros(3, device="cuda"))),
            (ValueError, dict(cap=0.0)), (ValueError, dict(cap=-1.0)),
            (ValueError, dict(cap=math.nan)), (ValueError, dict(window=0)),
            (mt.MTError, dict(cap=math.inf)), (mt.MTError, dict(page_size=0)),
            (mt.MTError, dict(scale=math.nan)),
            (ValueError, dict(out=a["q"][:2])),
            (TypeError, dict(out=a["q"].float())),
            (mt.MTError, dict(out=a["q"][:1].expand(3, -1, -1)))):
        with pytest.raises(err):
            mt.cache_attention(**dict(base, **kw))
    # a head that is too wide
    w = mt.cache_alloc(16, 1, 1024)
    with pytest.raises(mt.MTError) as e:
        mt.cache_attention(torch.zeros(1, 1, 1024, device="cuda"), w, w,
                           i32([[0]]), i32([0, 1]), i32([0]), 16)
    assert e.value.status == mt.MT_ERR_UNSUPPORTED
    # nothing to do
    empty = mt.cache_attention(**dict(base, q=a["q"][:0]))
    assert empty.shape == (0, 4, 64)
    none = mt.cache_attention(a["q"], a["k_cache"], a["v_cache"],
                              a["table"][:0], i32([0]), i32([]), 16)
    assert bool((none == 0).all())


def test_block_norm_refuses():
    a = norm_inputs(51, 3, 64, torch.bfloat16, "vector", "both")
    dy = a["x"]
    for err, kw in (
            (ValueError, dict(x=a["x"][0])), (TypeError, dict(x=a["x"].int())),
            (ValueError, dict(residual=a["x"][:2])),
            (TypeError, dict(residual=a["x"].float())),
            (ValueError, dict(residual=a["x"].t().contiguous().t())),
            (ValueError, dict(gate=a["gate"][:63])),
            (ValueError, dict(gate=a["x"][:2])),
            (TypeError, dict(weight=a["weight"].float())),
            (ValueError, dict(next_weight=a["weight"].cpu())),
            (ValueError, dict(norms="all")),
            (ValueError, dict(norms="before")),
            (ValueError, dict(norms="after")),
            (ValueError, dict(norms="after", next_weight=None, out=dy)),
            (ValueError, dict(h_out=a["x"][:2])),
            (mt.MTError, dict(eps=-1.0)),
            (mt.MTError, dict(out=a["x"], h_out=a["x"])),
            (mt.MTError, dict(out=a["x"][:1].expand(3, -1)))):
        with pytest.raises(err):
            mt.block_norm(**dict(a, **kw))
    b = dict(dy=dy, dh=dy, x=dy, h=dy, weight=a["weight"], gate=a["gate"],
             next_weight=a["next_weight"])
    for err, kw in (
            (ValueError, dict(dy=None)), (ValueError, dict(h=None)),
            (ValueError, dict(x=None)), (ValueError, dict(dy=dy[0])),
            (ValueError, dict(dh=dy[:2])), (TypeError, dict(h=dy.float())),
            (ValueError, dict(norms="after")),
            (ValueError, dict(norms="after", next_weight=None)),
            (ValueError, dict(norms="after", next_weight=None, dy=None,
                              dh=None)),
            (ValueError, dict(norms="before")),
            (ValueError, dict(out=(dy[:2], None))),
            (mt.MTError, dict(out=(dy, dy)))):
        with pytest.raises(err):
            mt.block_norm_backward(**dict(b, **kw))
