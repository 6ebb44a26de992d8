"""Plain 64-bit forms of the decoder's row operators, written from their
definitions, and the tolerances of the GPU tests.

Tolerances.  A stored value is rounded once, by at most half a step
(finfo.eps/2 relative; half the smallest subnormal near zero).  Before that,
FP32 arithmetic adds an error that each bound below derives from the number of
roundings (2^-24 relative each) and the accuracy of the functions used."""
import math

import torch

U = 2.0 ** -24  # one FP32 rounding, relative

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def half_step(ref, dtype):
    """Largest error of rounding `ref` (64-bit) once to dtype; a value that
    the FP32 error carries over a power of two costs a step of the next."""
    info = torch.finfo(dtype)
    return (ref.abs() * (1 + 2.0 ** -6) * (info.eps / 2) +
            info.smallest_normal * info.eps / 2)


def check(got, ref, tol, what=""):
    """|got - ref| <= tol element by element; NaN matches NaN, an infinity
    the same infinity."""
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    got, ref = got.double().cpu(), ref.double().cpu()
    tol = tol.double().cpu() if isinstance(tol, torch.Tensor) else tol
    ok = ((got - ref).abs() <= tol) & torch.isfinite(ref)
    ok |= (got == ref) | (torch.isnan(got) & torch.isnan(ref))
    if not bool(ok.all()):
        at = tuple(int(i) for i in torch.nonzero(~ok)[0])
        bad = int((~ok).sum())
        raise AssertionError(
            f"{what}: {bad} of {ok.numel()} values off; first at {at}: got "
            f"{got[at].item()!r}, want {ref[at].item()!r}, tolerance "
            f"{tol[at].item() if isinstance(tol, torch.Tensor) else tol!r}")


# ---- rotary -------------------------------------------------------------------
def rotate(x, positions, freqs, scale, rotary_dim, interleaved, sign=1.0):
    """64-bit rotation of [tokens, heads, dim]."""
    x = x.double()
    f = torch.as_tensor(freqs, dtype=torch.float64, device=x.device)
    ang = positions.double()[:, None] * f
    c, s = scale * torch.cos(ang)[:, None], sign * scale * torch.sin(ang)[:, None]
    y = x.clone()
    n = rotary_dim // 2
    ia = (torch.arange(n) * 2 if interleaved else torch.arange(n)).to(x.device)
    ib = ia + (1 if interleaved else n)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    return y


def pair_sum(x, rotary_dim, interleaved, scale):
    """scale (|a| + |b|) of the pair that each value belongs to; |x| where it
    is not rotated."""
    x = x.double().abs()
    m = x.clone()
    n = rotary_dim // 2
    ia = (torch.arange(n) * 2 if interleaved else torch.arange(n)).to(x.device)
    ib = ia + (1 if interleaved else n)
    t = abs(scale) * (x[..., ia] + x[..., ib])
    m[..., ia] = t
    m[..., ib] = t
    return m


# Cosine and sine of an angle in turns: the angle is rounded at 2^-25 of half
# a turn (9.4e-8 radians), sincospif is off by at most 2 ulp of 1 (1.2e-7),
# and the factor and the two products and the sum round once each.
#
# 16-bit storage takes __sinf and __cosf, off by at most 2^-21.19 on
# [-pi, pi], of an angle in radians that rounds three times at pi 2^-24.
def angle_error(dtype):
    if dtype == torch.float32:
        return 9.4e-8 + 1.2e-7 + 4 * U
    return 2.0 ** -21.19 + 3 * math.pi * U + 4 * U


def norm64(x, weight, eps):
    x = x.double()
    r = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    w = 1.0 if weight is None else weight.double()
    return x * r * w, r


# r: 16 squares added one after the other in a lane, 5 exchanges, the mean and
# eps (at most 24 roundings, halved by the square root), rsqrtf within 2 ulp,
# two products.
NORM = 12 * U + 4 * U + 2 * U


def rotary_ref(x, positions, freqs, scale, rotary_dim, interleaved, weight,
               eps):
    """(value, FP32 error bound) of the forward pass."""
    rel, angle = 0.0, angle_error(x.dtype)
    x = x.double()
    if eps is not None:
        x, _ = norm64(x, weight, eps)
        rel = NORM
    y = rotate(x, positions, freqs, scale, rotary_dim, interleaved)
    mag = pair_sum(x, rotary_dim, interleaved, scale)
    err = mag * (angle + rel)
    if eps is None:  # values that pass are copied
        err[..., rotary_dim:] = 0.0
    return y, err


def rotary_backward_ref(dy, x, positions, freqs, scale, rotary_dim,
                        interleaved, weight, eps):
    """(dx, its bound, dweight, its bound); the last two None without norm."""
    angle = angle_error(dy.dtype)
    g = rotate(dy, positions, freqs, scale, rotary_dim, interleaved, -1.0)
    mag = pair_sum(dy, rotary_dim, interleaved, scale)
    if eps is None:
        err = mag * angle
        err[..., rotary_dim:] = 0.0
        return g, err, None, None
    x = x.double()
    dim = x.shape[-1]
    _, r = norm64(x, None, eps)
    w = 1.0 if weight is None else weight.double()
    m = (g * w * x).mean(-1, keepdim=True) * r * r
    dx = r * (g * w - x * m)
    big = (mag * abs(w) * x.abs()).mean(-1, keepdim=True) * r * r
    # g: the angle; r three times over in the second term; the mean 24 roundings;
    # a handful of products.
    err = r * (mag * abs(w) * (angle + NORM + 4 * U) +
               x.abs() * big * (angle + 3 * NORM + 30 * U))
    terms = g * x * r
    count = terms.shape[0] * terms.shape[1]
    # however the rows are added up, at most `count` roundings touch a term
    werr = ((mag * x.abs() * r).sum((0, 1)) *
            (angle + NORM + 3 * U + count * U))
    return dx, err, terms.sum((0, 1)), werr


# ---- cache ----------------------------------------------------------------------
LARGEST = {"e4m3": 448.0, "int8": 127.0}


def quantise_ref(x, fmt, group):
    """Codes (as numbers) and scales in the operator's own FP32 steps, which
    are exactly rounded and so the same everywhere: x [..., dim]."""
    q = LARGEST[fmt]
    x = x.float().cpu().unflatten(-1, (-1, group))
    amax = x.abs().amax(-1)
    bad = ~torch.isfinite(amax)
    scale = torch.maximum(amax * torch.tensor(1 / q, dtype=torch.float32),
                          torch.tensor(2.0 ** -126))
    codes = x * (1 / scale)[..., None]
    codes = codes.round() if fmt == "int8" else \
        codes.clamp(-q, q).to(torch.float8_e4m3fn).float()
    codes = torch.where(bad[..., None], 0.0, codes)
    scale = torch.where(bad, math.nan, scale)
    return codes.flatten(-2), scale


# ---- logits -------------------------------------------------------------------
def logits_ref(x, tokens=None, lengths=None, prompt_lengths=None,
               repetition=None, frequency=None, presence=None, bias_ids=None,
               bias=None, mask=None, temperature=None, mode="logits"):
    """(value, FP32 error bound), row by row and token by token (CPU)."""
    x = x.double().cpu()
    rows, vocab = x.shape
    z, mag = x.clone(), x.abs().clone()
    for r in range(rows):
        if tokens is not None:
            ids = [int(t) for t in tokens[r]]
            n = len(ids) if lengths is None else \
                min(len(ids), max(0, int(lengths[r])))
            p = 0 if prompt_lengths is None else int(prompt_lengths[r])
            counts, seen = {}, set()
            for i, t in enumerate(ids[:n]):
                if 0 <= t < vocab:
                    seen.add(t)
                    if i >= p:
                        counts[t] = counts.get(t, 0) + 1
            rho = 1.0 if repetition is None else float(repetition[r])
            for t in seen:
                z[r, t] = z[r, t] / rho if z[r, t] > 0 else z[r, t] * rho
                mag[r, t] = z[r, t].abs()
            phi = 0.0 if frequency is None else float(frequency[r])
            pi = 0.0 if presence is None else float(presence[r])
            for t, c in counts.items():
                z[r, t] -= phi * c + pi
                mag[r, t] += abs(phi * c) + abs(pi)
        if bias_ids is not None:
            for t, b in zip(bias_ids[r].tolist(), bias[r].tolist()):
                if 0 <= t < vocab:
                    z[r, t] += b
                    mag[r, t] += abs(b) * bias_ids.shape[1] / 4 + abs(b)
        if temperature is not None:
            t = float(temperature[r])
            t = min(max(t, 2.0 ** -126), 2.0 ** 126) if t > 0 else 1.0
            z[r] /= t
            mag[r] /= t
    if mask is not None:
        m = mask.cpu().to(torch.int64)
        m = m[None].expand(rows, -1) if m.dim() == 1 else m
        v = torch.arange(vocab)
        allowed = (m[:, v >> 5] >> (v & 31)) & 1 != 0
        z = torch.where(allowed, z, -math.inf)
        mag = torch.where(allowed, mag, 0.0)
    # penalty 1 or 2 roundings, count * frequency + presence 2, the sums 1
    # each (a bias list's are counted in mag), 1/temperature and product 2
    zerr = torch.nan_to_num(mag, posinf=0.0) * 8 * U
    if mode == "logits":
        return z, zerr
    top = z.amax(1, keepdim=True)
    d = z - torch.where(top == -math.inf, 0.0, top)
    total = torch.exp(d).sum(1, keepdim=True)
    dz = zerr + zerr.amax(1, keepdim=True)
    # a term: the difference and its product round at |d| 2^-23, ex2.approx
    # within 2^-22; a thread adds at most 128 terms, the block 9, 16 slices
    weight = dz.amax(1, keepdim=True) + 180 * U
    far = torch.nan_to_num(d.abs(), posinf=0.0) * 2.0 ** -22
    if mode == "softmax":
        p = torch.where(total == 0, 0.0, torch.exp(d) / total)
        return p, torch.nan_to_num(p, nan=0.0) * (dz + far + weight + 8 * U) + 2.0 ** -125
    y = torch.where(total == 0, d, d - torch.log(total))
    return y, dz + far + weight + torch.nan_to_num(
        y.abs(), posinf=0.0) * 4 * U + 4 * U
