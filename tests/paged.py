"""Inputs and 64-bit references of the paged serving operators (test
infrastructure: plain loops over sequences and heads)."""
from __future__ import annotations

import math

import torch

D = 128
BF16_HALF_STEP = 2.0 ** -8     # one rounding to bf16, relative to the value
# A tensor-core product adds the 16 terms of a step to the running sum; each
# of the 17 may lose what lies below 2^-23 of the largest of them.
STEP = 17 * 2.0 ** -23


def normal(gen, *shape, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).bfloat16()


def pages_of(gen, ends, page, n_kv, spare=3, columns=None, order="nhd", fill=0.0):
    """(k_pages, v_pages, block_table) for sequences of `ends` cache rows, pages
    handed out in random order; order "hnd": [pages, n_kv, page, 128] in memory."""
    need = [-(-e // page) for e in ends]
    columns = columns or max(max(need), 1)
    pool = sum(need) + spare
    perm = torch.randperm(pool, generator=gen, device="cuda").int()
    # entries that hold no position are out of range: nothing may look at them
    table = torch.full((len(ends), columns), -7, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    shape = (pool, page, n_kv, D)
    if order == "hnd":
        k, v = (torch.full((pool, n_kv, page, D), fill, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
                for _ in range(2))
    else:
        k, v = (torch.full(shape, fill, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    return k, v, table


def slots(table, page, b, first, n):
    """(page, row) of positions first .. first+n-1 of sequence b."""
    at = torch.arange(first, first + n, device="cuda")
    return table[b].long()[at // page], at % page


def write_rows(pages, table, page, b, first, rows):
    p, r = slots(table, page, b, first, rows.shape[0])
    pages[p, r] = rows


def read_rows(pages, table, page, b, n):
    p, r = slots(table, page, b, 0, n)
    return pages[p, r]


def attend64(q, k, v, first, scale=D ** -0.5):
    """q [t, H, D], k, v [s, G, D]: query i sees keys 0..first+i. The fp64
    result and the two quantities its error bounds are made of: the p-weighted
    mean of |v|, and scale x sum |q||k| (largest over the visible keys)."""
    t, H, _ = q.shape
    s, G, _ = k.shape
    q, k, v = q.double(), k.double(), v.double()
    hidden = torch.arange(s, device=q.device)[None] > first + torch.arange(t, device=q.device)[:, None]
    out, mean, size = (torch.zeros(t, H, n, dtype=torch.float64, device=q.device) for n in (D, D, 1))
    for h in range(H):
        g = h * G // H
        x = (q[:, h] @ k[:, g].T * scale).masked_fill(hidden, -math.inf)
        p = torch.softmax(x, -1)
        # hidden values take no part: 0 x inf would
        seen = (~hidden).double()
        vg = torch.nan_to_num(v[:, g], 0.0, 0.0, 0.0)
        dirty = ~torch.isfinite(v[:, g])
        out[:, h] = p @ vg
        if dirty.any():
            bad = (seen @ dirty.double()) > 0
            out[:, h][bad] = math.nan
        mean[:, h] = p @ vg.abs()
        size[:, h] = (q[:, h].abs() @ k[:, g].abs().T * scale).masked_fill(hidden, 0).amax(-1, keepdim=True)
    return out, mean, size


def bound(ref, mean, size, keys, p_error):
    """|got - ref| at most: the output's rounding, and of the weighted mean of
    |v| the share by which the probabilities may be off. p_error: their
    rounding; the score is 8 product steps and a few fp32 operations off, which
    enters numerator and denominator; the value product runs keys / 16 steps,
    as does the sum; 2^-20 covers the base-2 exponential, the last division
    and the joins of partial results."""
    share = p_error + 2 * size * (8 * STEP + 2.0 ** -20) + (keys / 16 + 2) * STEP + 2.0 ** -20
    return BF16_HALF_STEP * ref.abs() + (1 + BF16_HALF_STEP) * share * mean


def check(got, ref, tol, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - ref).abs() - tol
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} of {over.numel()} values beyond the bound, " \
                              f"by up to {float(over.max()):.3e}"


# probabilities as two bf16 terms: the upper 8 bits and a remainder below
# 2^-7 of the value, itself rounded to bf16
P_TWO_TERMS = 2.0 ** -7 * BF16_HALF_STEP
P_ONE_TERM = BF16_HALF_STEP


def rotate64(x, cs):
    """x [n, H, D] by (cos, sin) cs [n, 64, 2]: the value, and the size of its two products."""
    x = x.double().unflatten(-1, (D // 2, 2))
    a, b = x[..., 0], x[..., 1]
    c, s = (cs.double()[:, None, :, i] for i in (0, 1))
    y = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    m = torch.stack([(a * c).abs() + (b * s).abs(), (a * s).abs() + (b * c).abs()], -1).flatten(-2)
    return y, m


def check_rotated(got, x, cs, what):
    """fp32: two products and a sum, each half a step of 2^-23 off, then one rounding to bf16."""
    y, m = rotate64(x, cs)
    check(got, y, BF16_HALF_STEP * y.abs() + 2.0 ** -22 * m, what)


# Relative L2 error of a whole output, for values that are independent of the
# weights: a rounding to bf16 is even within half a step, which is 0.0015 to
# 0.0017 of what is rounded in the mean square (2^-8 / sqrt(3 x 2.16) for evenly
# spread exponents). The output's own and the probabilities' add up to 0.0023;
# losing m of n keys costs sqrt(m / n) (0.046 for 148 of 70,001), which the
# bound above, whose share grows with n, does not see.
L2_BAR = 2.0 ** -8


def check_l2(got, ref, what):
    err = float((got.double() - ref).norm() / ref.norm())
    assert err <= L2_BAR, f"{what}: off by {err:.5f} of its norm"


CODE_KEYS, CODE_WINDOW = 16, 16 * D


def coded_values(n, window, device):
    """[n, D] of zeros and ones: key j of the window of 2,048 positions shows in
    dim (j % 2048) // 16 alone. With equal weights dim d of the mean is the
    number of its keys that were summed over the number of all: one key lost or
    taken twice is a sixteenth."""
    j = torch.arange(n, device=device)
    at = (j % CODE_WINDOW) // CODE_KEYS
    v = torch.zeros(n, D, dtype=torch.bfloat16, device=device)
    v[j, at] = (j // CODE_WINDOW == window).to(v.dtype)
    return v


def check_counts(got, window, first, what):
    """got [t, H, D]: equal weights over keys 0 .. first + i of coded values."""
    t = got.shape[0]
    seen = first + 1 + torch.arange(t, device=got.device).double()[:, None]
    begin = window * CODE_WINDOW + CODE_KEYS * torch.arange(D, device=got.device).double()
    want = ((seen - begin).clamp(0, CODE_KEYS) / seen)[:, None].expand(got.shape)
    # whole numbers up to 2^24 are exact in fp32; one division, one product, one rounding
    over = (got.double() - want).abs() - (BF16_HALF_STEP + 2.0 ** -20) * want
    assert (over <= 0).all(), f"{what}, window {window}: {int((over > 0).sum())} counts are wrong"
