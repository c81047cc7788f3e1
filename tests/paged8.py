"""Rows of an 8-bit cache for tests: the formula in 64 bits, pages of them."""
from __future__ import annotations

import math

import torch

from tests import paged as P

D = P.D
LEAST_E, MOST_E = -100, 120
# Probabilities times value scales are rounded to f16 (half a step of 2^-10);
# the exponent of a scale, up to 120, is added to the score in fp32: half a step
# of 2^-17 at most (the sum stays below 256 where it counts), of which ln 2 goes
# into the term, and as much when the maximum is taken off.
P_F16 = 2.0 ** -11 + 2 * math.log(2) * 2.0 ** -17


def bound(ref, mean, size, keys, most_scale=0.0):
    """P.bound, and the terms that f16 holds in steps of 2^-24: of weights times
    2^15 below 2^-14, half a step of 2^-39 of the largest weight times scale
    each, times values of up to 448 units."""
    return P.bound(ref, mean, size, keys, P_F16) + keys * 2.0 ** -40 * 448 * most_scale


def exponent(x):
    """Of rows [..., 128] (64 bits, finite where they count): the least e with max |x| <= 448 x 2^e."""
    a = torch.where(torch.isfinite(x), x.double().abs(), torch.zeros_like(x, dtype=torch.float64)).amax(-1)
    e = torch.full(a.shape, LEAST_E, dtype=torch.int32, device=x.device)
    for k in range(LEAST_E, MOST_E):
        e += (a > 448.0 * 2.0 ** k).int()
    return e


def two_to(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def e4m3(x, e):
    """x / 2^e rounded to e4m3's values, ties to even: steps of an eighth of the
    power of two below it, of 2^-9 at least. NaN for what is not finite."""
    y = x.double() * two_to(-e)[..., None]
    step = two_to(torch.frexp(y)[1].clamp_min(-5) - 4)
    r = torch.round(y / step) * step
    return torch.where(torch.isfinite(x), r, torch.full_like(r, math.nan))


def quantised(x):
    """(values in units, exponents) of rows x."""
    e = exponent(x)
    return e4m3(x, e), e


def as_fp8(units):
    y = units.float().to(torch.float8_e4m3fn)
    assert torch.equal(torch.nan_to_num(y.float(), 999.0), torch.nan_to_num(units.float(), 999.0))
    return y


def values(pages, scales):
    """The values that pages and scale bytes stand for, in 64 bits."""
    return pages.float().double() * two_to(scales.int() - 127)[..., None]


def same(a, b):
    """Equal, NaN among it."""
    return torch.equal(torch.nan_to_num(a.double(), 12345.0), torch.nan_to_num(b.double(), 12345.0))


def junk(shape, byte, order="nhd"):
    """Bytes [pages, page, n_kv, ...] all `byte`, in memory page, row, head or page, head, row."""
    if order == "hnd":
        shape = (shape[0], shape[2], shape[1], *shape[3:])
    t = torch.full(shape, byte, dtype=torch.uint8, device="cuda")
    return t.transpose(1, 2) if order == "hnd" else t


def pages_of(gen, ends, page, n_kv, order="nhd", byte=0x7f, scale_byte=255, **kw):
    """(k_pages, v_pages, k_scales, v_scales, table), every row `byte` (0x7f: NaN)."""
    _, _, table = P.pages_of(gen, ends, page, 1, **kw)
    pool = sum(-(-e // page) for e in ends) + kw.get("spare", 3)
    kv = [junk((pool, page, n_kv, D), byte, order).view(torch.float8_e4m3fn) for _ in range(2)]
    sc = [junk((pool, page, n_kv), scale_byte, order) for _ in range(2)]
    return (*kv, *sc, table)


def put(pages, at, x):
    pages.view(torch.uint8)[at] = x.view(torch.uint8)


def fill(gen, lens, page, n_kv, spread=3, **kw):
    """Pages with random rows of sequences, scales 2^-spread .. 2^spread of one
    another; the rows' values [n, n_kv, 128] in 64 bits."""
    k_pages, v_pages, k_scales, v_scales, table = pages_of(gen, lens, page, n_kv, **kw)
    rows = []
    for b, n in enumerate(lens):
        at = P.slots(table, page, b, 0, n)
        pair = []
        for pages, scales, wide in ((k_pages, k_scales, 0), (v_pages, v_scales, spread)):
            x = torch.randn(n, n_kv, D, generator=gen, device="cuda")
            x *= 2.0 ** torch.randint(-wide, wide + 1, (n, n_kv, 1), generator=gen, device="cuda")
            units, e = quantised(x)
            put(pages, at, as_fp8(units))
            scales[at] = (e + 127).to(torch.uint8)
            pair.append(units * two_to(e)[..., None])
        rows.append(tuple(pair))
    return (k_pages, v_pages, k_scales, v_scales, table), rows


def turned32(x, cs, halves):
    """Rows x [n, h, 128] turned in fp32, each product and sum rounded."""
    x = x.float()
    n = cs.shape[1]
    at = torch.arange(n, device=x.device)
    first, second = (at, at + n) if halves else (2 * at, 2 * at + 1)
    a, b, c, s = x[..., first], x[..., second], cs[:, None, :, 0], cs[:, None, :, 1]
    y = x.clone()
    y[..., first] = a * c - b * s
    y[..., second] = a * s + b * c
    return y


def turned64(x, cs, halves):
    """The same in 64 bits, and the size of the products of each dim."""
    n = cs.shape[1]
    at = torch.arange(n, device=x.device)
    first, second = (at, at + n) if halves else (2 * at, 2 * at + 1)
    x, cs = x.double(), cs.double()
    a, b, c, s = x[..., first], x[..., second], cs[:, None, :, 0], cs[:, None, :, 1]
    y, m = x.clone(), torch.zeros_like(x)
    y[..., first], y[..., second] = a * c - b * s, a * s + b * c
    m[..., first], m[..., second] = (a * c).abs() + (b * s).abs(), (a * s).abs() + (b * c).abs()
    return y, m
