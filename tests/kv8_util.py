"""The definitions of rotary positions and of the 8-bit paged cache, in 64 bits on the CPU or wherever their inputs are,
and how far a result may be from them.

Rotation: y = a c - b s with products and sum rounded to 32 bits: off by at most 2^-24 (|a c| + |b s|) for the products
and 2^-24 |y'| for the sum, below ROT = 2.01 * 2^-24 of |a c| + |b s| together; then one rounding to the storage type,
half a step u |y| or half the smallest step.
Writing: the exponent is that of the definition unless the largest size lies within the rotation's error of a border;
a stored value is off by half a step of e4m3 at its size (2^-4 of it, 2^-10 of the scale at the least), and an older
entry by one such step more for each time that its block's scale rose.
"""
import math

import numpy as np
import torch

ROT = 2.01 * 2.0 ** -24
LIMITS = {torch.bfloat16: (-117, 119), torch.float16: (-15, 7)}
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}  # half of the smallest step


def power(e):
    """2^e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def rates(rot, base, scaling="none", factor=1.0, original=0, low=1.0, high=32.0):
    """The angles' rates by the definition, pair by pair."""
    out = []
    for i in range(rot // 2):
        w = base ** (-2.0 * i / rot)
        if scaling == "linear":
            w /= factor
        elif scaling == "base":
            w = (base * factor ** (rot / (rot - 2))) ** (-2.0 * i / rot)
        elif scaling == "ramp":
            d = [rot * math.log(original / (2 * math.pi * t)) / (2 * math.log(base)) for t in (high, low)]
            lo, hi = max(math.floor(d[0]), 0), min(math.ceil(d[1]), rot - 1)
            r = min(1.0, max(0.0, (i - lo) / (hi - lo if hi != lo else 0.001)))
            w = w * (1 - r) + w / factor * r
        elif scaling == "wave":
            s = min(1.0, max(0.0, (original * w / (2 * math.pi) - low) / (high - low)))
            w = w * s + w / factor * (1 - s)
        out.append(w)
    return np.array(out)


def angles(rows, rot, first=0, gain=1.0, **kw):
    a = (first + np.arange(rows, dtype=np.float64))[:, None] * rates(rot, kw.pop("base", 10000.0), **kw)[None]
    return torch.from_numpy(np.stack([np.cos(a), np.sin(a)], 1) * gain)


def pairs(rot, inter):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)


def rotate(x, cs, inter):
    """x [T][H][D] turned by cs [T][2][rot / 2]: (y in 64 bits, sum of the products' sizes)."""
    y, size = x.double().clone(), x.double().abs()
    a, b = pairs(2 * cs.shape[2], inter)
    c, s = cs[:, None, 0].double(), cs[:, None, 1].double()
    u, v = x[..., a].double(), x[..., b].double()
    y[..., a], y[..., b] = u * c - v * s, v * c + u * s
    size[..., a], size[..., b] = (u * c).abs() + (v * s).abs(), (v * c).abs() + (u * s).abs()
    return y, size


def rotate32(x, cs, inter):
    """The rotation with every product and sum rounded to 32 bits: what the kernels compute, bit for bit."""
    y = x.float().clone()
    if cs is None:
        return y
    a, b = pairs(2 * cs.shape[2], inter)
    c, s = cs[:, None, 0], cs[:, None, 1]
    u, v = x[..., a].float(), x[..., b].float()
    y[..., a], y[..., b] = u * c - v * s, v * c + u * s
    return y


def check_rotated(got, x, cs, inter):
    y, size = rotate(x, cs, inter)
    u = torch.finfo(x.dtype).eps / 2
    tol = (ROT * size + u * (y.abs() + ROT * size)) * 1.001 + TINY[x.dtype]
    off = (got.double() - y).abs()
    assert bool((off <= tol).all()), float((off / tol).nan_to_num(math.inf).max())
    rest = 2 * cs.shape[2]
    assert torch.equal(got[..., rest:], x[..., rest:])


def to_e4m3(x):
    """64-bit values to the nearest of e4m3, ties to even, at most 448 in size; what is not finite to NaN."""
    step = power(torch.frexp(x.abs().clamp(min=2.0 ** -6).nan_to_num(1.0, 1.0, 1.0)).exponent - 4)
    y = (torch.round(x / step) * step).clamp(-448, 448)
    return torch.where(x.isfinite(), y, torch.nan)


def exponent(x, dtype):
    """The exponent of a block's new entries x [...][block * D] by the definition (last dimension)."""
    peak = torch.where(x.isfinite(), x.abs(), 0).amax(-1) / 448
    m, e = torch.frexp(peak)
    e = e - (m == 0.5).to(e.dtype)
    lo, hi = LIMITS[dtype]
    return torch.where(peak > 0, e, lo).clamp(lo, hi)


def values(pages, scales):
    """What 8-bit pages hold, in 64 bits [P][LH][page][D]; a scale byte of 255 is NaN."""
    P, LH, page, D = pages.shape
    x = pages.view(torch.uint8).view(E4M3).float().double()
    s = scales.view(torch.uint8).long()
    f = torch.where(s == 255, torch.nan, power(s - 127))
    return (x.view(P, LH, s.shape[2], page // s.shape[2], D) * f[..., None, None]).view(P, LH, page, D)


def write(pages, scales, x, table, start, dtype):
    """Entries x [LH][n][D] (64 bits, or 32: then every product with a power of two is exact, too) of one request into
    its pages from position `start`, in place (pages [P][LH][page][D], scales [P][LH][page / block], 64-bit values:
    e4m3 values and exponents)."""
    P, LH, page, D = pages.shape
    block = page // scales.shape[2]
    done, n = 0, x.shape[1]
    while done < n:
        col, row = divmod(start + done, page)
        j, into = divmod(row, block)
        part = x[:, done:done + block - into].double()
        pg = int(table[col])
        e = exponent(part.reshape(LH, -1), dtype).long()
        rows = pages[pg, :, j * block:(j + 1) * block]
        if into:
            own = scales[pg, :, j]
            e = torch.maximum(e, own)
            up = (e > own)[:, None, None]
            rows[:, :into] = torch.where(up, to_e4m3(rows[:, :into] * power(own - e)[:, None, None]), rows[:, :into])
        rows[:, into:into + part.shape[1]] = to_e4m3(part * power(-e)[:, None, None])
        scales[pg, :, j] = e
        done += part.shape[1]


def split(pages, scales):
    """(e4m3 values in 64 bits, exponents) of a cache, as `write` takes them."""
    return pages.view(torch.uint8).view(E4M3).float().double(), scales.view(torch.uint8).long() - 127


def used_cache(rng, P, LH, page, D, block, dtype, device, spread=2):
    """A cache of normal entries whose blocks differ in size, at the exponents that these ask for."""
    nb = page // block
    x = rng.standard_normal((P, LH, nb, block, D)) * 2.0 ** rng.integers(-spread, spread + 1, (P, LH, nb, 1, 1))
    x = torch.from_numpy(x).to(device)
    e = exponent(x.reshape(P, LH, nb, -1), dtype)
    y = to_e4m3(x * power(-e)[..., None, None]).float().to(E4M3)
    return y.view(P, LH, page, D), (e + 127).to(torch.uint8).view(E8M0)
