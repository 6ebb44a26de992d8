"""Plain 64-bit forms of the operators around a decoder's cache, written from
their definitions, and the tolerances of the GPU tests (half a step at the
store, and the FP32 arithmetic before it: see each bound)."""
import math

import torch

from decoder_util import U

LARGEST = {"e4m3": 448.0, "int8": 127.0}
MAX32 = 2 ** 31 - 1


# ---- pages of a step ---------------------------------------------------------
def extend_ref(table, lengths, counts, free, free_count, page, rows):
    """(table, offsets, slots, positions, lengths, free_count) as lists,
    sequence by sequence."""
    table = [list(r) for r in table]
    width = len(table[0]) if table else 0
    left = most = min(max(free_count, 0), len(free))
    asked, offsets, slots, positions, new = 0, [0], [], [], []
    for s, (length, count) in enumerate(zip(lengths, counts)):
        length, count = max(length, 0), max(count, 0)
        held, want = -(-length // page), -(-(length + count) // page)
        fits = length + count <= MAX32 and (want == held or want <= width)
        need = want - held if fits else 0
        asked += need
        served = fits and (need == 0 or asked <= most)
        if served:
            for p in range(held, want):
                left -= 1
                table[s][p] = free[left]
        offsets.append(min(offsets[-1] + count, MAX32))
        new.append(length + count if served else length)
        for p in range(length, length + min(count, rows - len(slots))):
            id_ = table[s][p // page] if p // page < width else -1
            slots.append(id_ * page + p % page if served and id_ >= 0 else -1)
            positions.append(min(p, MAX32))
    pad = rows - len(slots)
    return (table, offsets, slots + [-1] * pad, positions + [0] * pad, new,
            left)


# ---- attention over the cache ------------------------------------------------
def cache_values(cache):
    """64-bit values of a whole cache tensor [slots, heads, dim]."""
    codes, scales = cache
    return codes.float().double() * scales.double().repeat_interleave(
        codes.shape[-1] // scales.shape[-1], -1)


def attention_ref(q, k_cache, v_cache, table, offsets, starts, page,
                  scale=None, cap=None, slopes=None, window=None, first=None,
                  last=None):
    """(out, its FP32 error bound, lse, its bound, rows that have a value):
    sequence by sequence, row by row of the mask.

    The bound.  A score: queries as one or two FP16 parts of a power of two
    times their value (FP32: 2^-22 of each; smaller ones 2^-39 of the head's
    largest), products exact, at most dim / 16 + 5 sums (each within 2^-22 of
    what it adds up, as a matrix instruction may cut off), the scale, factors
    and, in cap, five roundings of cap; the distance's product and difference.
    A weight: its score's error, |z - top| 2^-23 (the exponent's product) and
    2^-21 (the instruction, and rescaling at most twice); as FP16 times the
    value's scale 2^-11 (two such parts: 2^-22, kept for FP32 and FP16).  The
    sums over keys: one rounding a key at most.

    The smallest.  Weights below 2^-126 of a row's largest are zero (the
    instruction flushes) and so are products below that: 2^-126 (1 + |v|) a
    key.  A weight times a value's scale in FP16 is held against the largest
    of some keys, 2^14 or more: half a step of the smallest such numbers,
    2^-25, is 2^-39 of it, times a code, a key."""
    rows, heads, dim = q.shape
    times = heads // k_cache[0].shape[1]
    scale = dim ** -0.5 if scale is None else scale
    out = torch.zeros(rows, heads, dim, dtype=torch.float64, device=q.device)
    err = torch.zeros_like(out)
    lse = torch.full((rows, heads), -math.inf, dtype=torch.float64,
                     device=q.device)
    lse_err = torch.zeros_like(lse)
    there = torch.zeros(rows, dtype=torch.bool, device=q.device)
    offs, begin = offsets.tolist(), starts.tolist()
    slots = k_cache[0].shape[0]
    part = 2.0 ** -11 if q.dtype == torch.bfloat16 else 2.0 ** -22
    for s, start in enumerate(begin):
        a, b = max(offs[s], 0), min(offs[s + 1], rows)
        if b <= a:
            continue
        there[a:b] = True
        held = min(start + offs[s + 1] - offs[s], table.shape[1] * page)
        j = torch.arange(max(held, 0), device=q.device)
        id_ = table[s].long()[j // page] if held > 0 else j
        slot = id_ * page + j % page
        good = (id_ >= 0) & (slot < slots)
        slot = torch.where(good, slot, 0)
        pick = [tuple(t.view(torch.int8)[slot].view(t.dtype)
                      if t.element_size() == 1 else t[slot] for t in c)
                for c in (k_cache, v_cache)]
        k, v = (cache_values(c).repeat_interleave(times, 1) for c in pick)
        p = start + torch.arange(a - offs[s], b - offs[s], device=q.device)
        lo = torch.zeros_like(p) if first is None else first[a:b].long()
        hi = p if last is None else last[a:b].long()
        if window is not None:
            lo = torch.maximum(lo, p - window + 1)
        see = (j >= lo[:, None]) & (j <= hi[:, None]) & good
        if held <= 0:
            continue
        x = q[a:b].double()
        # what a row does not see must not reach it, NaN included
        z = scale * torch.einsum("rhd,jhd->rhj", x, k)
        mag = abs(scale) * torch.einsum("rhd,jhd->rhj", x.abs(), k.abs())
        big = abs(scale) * x.abs().amax(-1)[..., None] * \
            k.abs().sum(-1).T[None]
        dz = mag * ((dim / 16 + 5) * 2.0 ** -22 + 2.0 ** -22 + 6 * U) + \
            big * 2.0 ** -39
        if cap is not None:
            z = cap * torch.tanh(z / cap)
            dz = dz + 5 * U * cap
        if slopes is not None:
            far = (p[:, None] - j).abs().double()
            bias = slopes.double()[:, None] * far[:, None]
            z = z - bias
            dz = dz + 3 * U * bias.abs() + 2 * U * z.abs()
        m = see[:, None].expand_as(z)
        z = torch.where(m, z, -math.inf)
        dz = torch.where(m, dz, 0.0)
        top = z.amax(-1, keepdim=True)
        ref = torch.where(top == -math.inf, 0.0, top)
        e = torch.exp(z - ref)
        total = e.sum(-1, keepdim=True)
        w = torch.where(m, e / torch.where(total == 0, 1.0, total), 0.0)
        vm = torch.where(see.any(0)[:, None, None], v, 0.0)
        # rows that do not see a NaN of v that others see
        if bool(torch.isnan(vm).any()):
            nan = torch.einsum("rhj,jhd->rhd", m.double(),
                               torch.isnan(vm).double()) > 0
            vm = torch.nan_to_num(vm)
        else:
            nan = None
        o = torch.einsum("rhj,jhd->rhd", w, vm)
        away = torch.where(m, (z - ref).abs(), 0.0)
        dw = dz + away * 2.0 ** -23
        most = dw.amax(-1, keepdim=True)
        spread = torch.einsum("rhj,jhd->rhd", w, vm.abs())
        err[a:b] = spread * (2 * most + part + 2.0 ** -20 + (len(j) + 8) * U)
        vs = torch.nan_to_num(pick[1][1].double()).repeat_interleave(
            dim // pick[1][1].shape[-1], -1).repeat_interleave(times, 1)
        vs = torch.where(see.any(0)[:, None, None], vs, 0.0)
        top_code = 448.0 if k_cache[0].is_floating_point() else 127.0
        large = torch.zeros_like(o)
        for d in range(0, dim, dim // pick[1][1].shape[-1]):
            g = slice(d, d + dim // pick[1][1].shape[-1])
            large[..., g] = (w * vs[..., d].T[None]).amax(-1)[..., None]
        err[a:b] += len(j) * (2.0 ** -39 * top_code * large + 2.0 ** -126) + \
            2.0 ** -126 * vm.abs().sum(0)
        out[a:b] = o if nan is None else torch.where(nan, math.nan, o)
        lse[a:b] = torch.where(total[..., 0] == 0, -math.inf,
                               ref[..., 0] + torch.log(total[..., 0]))
        lse_err[a:b] = most[..., 0] + 2.0 ** -20 + (len(j) + 8) * U + \
            4 * U * ref[..., 0].abs()
    return out, err, lse, lse_err, there


# ---- norms around a block ----------------------------------------------------
# A sum of `cols` squares or products: however they are split, at most
# cols / 8 + 40 roundings touch a term (256 threads or more from 2048 columns
# on, ten exchanges; a thread's own terms one after the other).
def sum_roundings(cols):
    return max(cols / 128, min(cols, 64)) + 40


def block_norm_ref(x, residual, weight, gate, next_weight, norms,
                   residual_scale, eps):
    """(y, its bound, h, its bound)."""
    x, res = x.double(), residual.double()
    n = sum_roundings(x.shape[1])
    u, rel = x, 0.0
    if norms != "before":
        r = 1 / torch.sqrt(x.square().mean(1, keepdim=True) + eps)
        u = x * r * (1.0 if weight is None else weight.double())
        rel = (n / 2 + 8) * U
    b = u * (1.0 if gate is None else gate.double())
    h = residual_scale * res + b
    dh = (residual_scale * res).abs() * 3 * U + b.abs() * (rel + 3 * U)
    if norms == "after":
        return None, None, h, dh
    ms = h.square().mean(1, keepdim=True) + eps
    r = 1 / torch.sqrt(ms)
    w = 1.0 if next_weight is None else next_weight.double()
    y = h * r * w
    # the mean of squares moves by 2 h dh
    dm = (2 * h.abs() * dh + dh.square()).mean(1, keepdim=True) / ms / 2
    dy = (w * r * dh if next_weight is None else w.abs() * r * dh) + \
        y.abs() * (dm + (n / 2 + 8) * U)
    return y, dy, h, dh


def block_norm_back_ref(dy, dh, x, h, weight, gate, next_weight, norms,
                        residual_scale, eps):
    """[(gradient, its bound)] in the order of the operator's results."""
    some = dy if dy is not None else dh
    rows, cols = some.shape
    n = sum_roundings(cols)
    g = torch.zeros(rows, cols, dtype=torch.float64, device=some.device) \
        if dh is None else dh.double()
    ge = torch.zeros_like(g)
    last = []
    w2 = 1.0 if next_weight is None else next_weight.double()
    if norms != "after":
        hd, d = h.double(), dy.double()
        r = 1 / torch.sqrt(hd.square().mean(1, keepdim=True) + eps)
        dot = (d * w2 * hd).mean(1, keepdim=True)
        big = (d * w2 * hd).abs().mean(1, keepdim=True)
        a, b = r * d * w2, r * hd * r * r * dot
        g = g + a - b
        ge = (g.abs() + a.abs() * (n / 2 + 10) + b.abs() * (2 * n + 12)) * U \
            + r * hd.abs() * r * r * big * (n + 4) * U
        if next_weight is not None:
            t = d * hd * r
            last.append((t.sum(0), t.abs().sum(0) * (n / 2 + 10 + rows) * U))
    got = [(residual_scale * g, abs(residual_scale) * ge + (residual_scale *
                                                            g).abs() * U)]
    xd = None if x is None else x.double()
    r1 = 1.0
    w1 = 1.0 if weight is None else weight.double()
    if norms != "before":
        r1 = 1 / torch.sqrt(xd.square().mean(1, keepdim=True) + eps)
    e, ee = g, ge
    if gate is not None:
        u = xd * r1 * w1
        dg, dge = g * u, ge * u.abs() + (g * u).abs() * (n / 2 + 12) * U
        if gate.dim() == 1:
            got.append((dg.sum(0), dge.sum(0) +
                        dg.abs().sum(0) * (rows + 4) * U))
        else:
            got.append((dg, dge))
        gd = gate.double()
        e, ee = g * gd, ge * gd.abs() + (g * gd).abs() * U
    if norms == "before":
        return [(e, ee)] + got + last
    if weight is not None:
        t = e * xd * r1
        got.append((t.sum(0), (ee * (xd * r1).abs()).sum(0) +
                    t.abs().sum(0) * (n / 2 + 12 + rows) * U))
    dot = (e * w1 * xd).mean(1, keepdim=True)
    big = ((e * w1 * xd).abs() * (n + 6) * U + ee * (w1 * xd).abs()).mean(
        1, keepdim=True)
    a, b = r1 * e * w1, r1 * xd * r1 * r1 * dot
    dx = a - b
    dxe = r1 * ee * (abs(w1) if weight is None else w1.abs()) + \
        a.abs() * (n / 2 + 10) * U + b.abs() * (2 * n + 12) * U + \
        r1 * xd.abs() * r1 * r1 * big + dx.abs() * U
    return [(dx, dxe)] + got + last
