"""The 8-bit paged cache and the rotary layouts against the formula, at the
sizes, masks, values and layouts where they can go wrong."""
import math

import pytest
import torch

import grouped_query_attention_gemv_gb300 as G
from tests import paged as P
from tests import paged8 as Q
from tests.test_paged_gpu import LAYOUTS, ints, offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ws():
    return G.make_paged_workspace()


@pytest.fixture
def gen():
    return torch.Generator(device="cuda").manual_seed(5)


def rotary_table(rows, dim):
    return G.rope_table(max(rows, 1), dim=dim)


# ------------------------------------------------------------------ tables

@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("dim", [2, 16, 64, 96, 128])
def test_rope_table_of_a_part(dim, scaled):
    got = G.rope_table(3000, dim=dim, scaled=scaled).double()
    f = 500000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64, device="cuda") / dim)
    if scaled:   # wavelengths past 8192 by 8, below 2048 as they are, between them by their place
        wave = 2 * math.pi / f
        mu = (8192 / wave - 1) / 3
        f = torch.where(wave > 8192, f / 8, torch.where(wave < 2048, f, (1 - mu) * f / 8 + mu * f))
    a = torch.arange(3000, dtype=torch.float64, device="cuda")[:, None] * f
    want = torch.stack([a.cos(), a.sin()], -1)
    # one rounding to fp32; angles up to 3,000 in 64 bits
    assert (got - want).abs().max() <= 2.0 ** -24 + 1e-11
    if dim == 128:
        assert torch.equal(got.float(), G.rope_table(3000, scaled=scaled))


# ------------------------------------------------------------------ append

def inputs(gen, n, heads, n_kv, strided):
    if strided:
        qkv = P.normal(gen, n, heads + 2 * n_kv, P.D)
        return qkv[:, :heads], qkv[:, heads:heads + n_kv], qkv[:, heads + n_kv:]
    return tuple(P.normal(gen, n, h, P.D) for h in (heads, n_kv, n_kv))


def check_turned(got, x, cs, halves, what):
    y, m = Q.turned64(x, cs, halves)
    P.check(got, y, P.BF16_HALF_STEP * y.abs() + 2.0 ** -22 * m, what)


def run_append(gen, ws, bits, heads, n_kv, page, lens, starts, dim=128, halves=False, order="nhd", strided=True, cu=True,
               with_q=True, behind=0, in_place=False):
    n = sum(lens) + behind
    ends = [s + t if s >= 0 else 0 for s, t in zip(starts, lens)]
    if bits == 8:
        *cache, table = Q.pages_of(gen, ends, page, n_kv, order=order, byte=0x11, scale_byte=3)
    else:
        *cache, table = P.pages_of(gen, ends, page, n_kv, order=order, fill=3.0)
    q, k, v = inputs(gen, n, heads, n_kv, strided)
    q0, before = q.clone(), [x.clone() for x in cache]
    rope = rotary_table(max(ends), dim)
    q_out = q if in_place else torch.full((n, heads, P.D), 7.0, dtype=torch.bfloat16, device="cuda")
    q_before = q_out.clone()
    args = dict(cu_tokens=offsets(lens) if cu else None, q_out=q_out if with_q else None, workspace=ws, rotary_dim=dim,
                halves=halves)
    entry = G.paged_append_fp8 if bits == 8 else G.paged_append
    got = entry(q if with_q else None, k, v, ints(starts), rope, *cache, table, **args)
    assert (got is q_out) if with_q else (got is None)
    at = 0
    for b, (t, s) in enumerate(zip(lens, starts)):
        rows = slice(at, at + t)
        at += t
        if s < 0:
            assert torch.equal(q_out[rows], q_before[rows])
            continue
        if t == 0:
            continue
        cs, spot = rope[s:s + t], P.slots(table, page, b, s, t)
        if with_q:
            check_turned(q_out[rows], q0[rows], cs, halves, f"q of sequence {b}")
            assert torch.equal(q_out[rows][..., dim:], q0[rows][..., dim:])
        turned = Q.turned32(k[rows], cs, halves)
        if bits == 16:
            check_turned(cache[0][spot], k[rows], cs, halves, f"k of sequence {b}")
            assert torch.equal(cache[0][spot], turned.bfloat16())
            assert torch.equal(cache[1][spot], v[rows])
        else:
            for pages, scales, x in ((cache[0], cache[2], turned), (cache[1], cache[3], v[rows].float())):
                units, e = Q.quantised(x)
                assert torch.equal(scales[spot].int() - 127, e)
                assert Q.same(pages.view(torch.uint8)[spot].view(torch.float8_e4m3fn).float(), units)
        for x, was in zip(cache, before):
            x.view(torch.uint8)[spot] = was.view(torch.uint8)[spot]
    # every other row, of the pages and of the queries, is as it was
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(cache, before))
    assert torch.equal(q_out[at:], q_before[at:])
    assert G.device_status(ws) == 0


@pytest.mark.parametrize("heads,n_kv", LAYOUTS)
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("bits,dim,halves", [(8, 128, False), (8, 128, True), (16, 128, True), (16, 64, False)])
def test_append_layouts(gen, ws, heads, n_kv, page, bits, dim, halves):
    run_append(gen, ws, bits, heads, n_kv, page, [1, 0, 17, 33, 1], [0, 4, 15, 127, 16], dim, halves)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("dim", [16, 32, 48, 64, 80, 96, 112, 128])
def test_append_turns_a_part(gen, ws, bits, halves, dim):
    run_append(gen, ws, bits, 6, 2, 32, [3, 40], [30, 0], dim, halves)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("kw", [dict(order="hnd"), dict(strided=False), dict(with_q=False), dict(behind=9),
                                dict(strided=False, in_place=True), dict(dim=32, strided=False, in_place=True)])
def test_append_forms(gen, ws, bits, kw):
    run_append(gen, ws, bits, 8, 2, 32, [5, 40, 0, 3], [31, -1, 3, 64], halves=True, **kw)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("B", [1, 2, 33, 300])
def test_append_one_token_each(gen, ws, bits, B):
    run_append(gen, ws, bits, 8, 2, 16, [1] * B, [-1 if b % 5 == 4 else (7 * b) % 90 for b in range(B)], halves=True,
               cu=False)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("heads,n_kv,dim,halves", [(8, 2, 128, True), (28, 4, 96, False), (5, 1, 64, True)])
def test_append_many_tokens(gen, ws, bits, heads, n_kv, dim, halves):
    # a warp takes several batches of a token's rows
    run_append(gen, ws, bits, heads, n_kv, 64, [3000, 0, 1500, 1, 620], [5, 7, 0, -1, 40], dim, halves, behind=3)


def test_append_rounds_as_the_formula(gen, ws):
    """Value rows of every kind: ties, the least and the largest exponents, zero,
    one value at the border of a scale, what is not finite."""
    rows = []
    for k in (-133, -110, -92, -91, -90, -20, -1, 0, 3, 40, 100, 118, 119):
        x = torch.randn(128, generator=gen, device="cuda")
        x[0] = 1.9
        rows.append((x / x.abs().max() * 1.99).double() * 2.0 ** k)
    # multiples of a sixteenth are ties of every second step between 1 and 2, of 2^-10 below the least normal value
    rows.append(torch.arange(-64, 64, device="cuda").double() / 16)
    rows.append(torch.arange(-64, 64, device="cuda").double() * 2.0 ** -10)
    rows[-1][0] = 448.0
    for top in (448.0, 450.0, 446.0, 224.0, 225.0):
        x = torch.linspace(-1, 1, 128, device="cuda").double()
        x[77] = top
        rows.append(x)
    rows.append(torch.zeros(128, dtype=torch.float64, device="cuda"))
    x = torch.linspace(-1, 1, 128, device="cuda").double()
    x[3], x[50], x[100] = math.inf, -math.inf, math.nan
    rows.append(x)
    rows.append(torch.full((128,), math.nan, dtype=torch.float64, device="cuda"))
    v = torch.stack(rows).bfloat16()[:, None]
    n = v.shape[0]
    *cache, table = Q.pages_of(gen, [n], 64, 1)
    G.paged_append_fp8(None, torch.zeros_like(v), v, ints([0]), G.rope_table(n), *cache, table, cu_tokens=offsets([n]),
                       workspace=ws)
    assert G.device_status(ws) == 0
    spot = P.slots(table, 64, 0, 0, n)
    units, e = Q.quantised(v.double())
    assert torch.equal(cache[3][spot].int() - 127, e)
    assert Q.same(cache[1].view(torch.uint8)[spot].view(torch.float8_e4m3fn).float(), units)
    # keys of zero: the least scale
    assert (cache[2][spot] == Q.LEAST_E + 127).all() and (cache[0].view(torch.uint8)[spot] & 0x7f == 0).all()
    # within half a step: 2^-4 of the value, 2^-10 of the scale
    ok = torch.isfinite(v.double())
    back = Q.values(cache[1].view(torch.uint8)[spot].view(torch.float8_e4m3fn), cache[3][spot])
    off = (back - v.double()).abs()
    assert (off <= torch.maximum(2.0 ** -4 * v.double().abs(), 2.0 ** -10 * Q.two_to(e)[..., None]))[ok].all()


@pytest.mark.parametrize("shape,at", [((9, 2, 16, 2, 128), 1), ((9, 16, 2, 2, 128), 2), ((2, 9, 16, 2, 128), 0)])
def test_append_into_interleaved_pages(gen, ws, shape, at):
    both = torch.full(shape, 0x22, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.full(shape[:-1], 9, dtype=torch.uint8, device="cuda")
    (k_pages, v_pages), (k_scales, v_scales) = both.unbind(at), scales.unbind(at)
    table = torch.randperm(9, generator=gen, device="cuda")[:8].view(2, 4).int()
    k, v = P.normal(gen, 70, 2, P.D), P.normal(gen, 70, 2, P.D)
    rope = G.rope_table(64)
    G.paged_append_fp8(None, k, v, ints([3, 0]), rope, k_pages, v_pages, k_scales, v_scales, table,
                       cu_tokens=offsets([20, 50]), workspace=ws)
    assert G.device_status(ws) == 0
    for b, (rows, s) in enumerate(((slice(0, 20), 3), (slice(20, 70), 0))):
        spot = P.slots(table, 16, b, s, rows.stop - rows.start)
        for pages, sc, x in ((k_pages, k_scales, Q.turned32(k[rows], rope[s:s + rows.stop - rows.start], False)),
                             (v_pages, v_scales, v[rows])):
            units, e = Q.quantised(x)
            assert torch.equal(sc[spot].int() - 127, e)
            assert Q.same(pages.view(torch.uint8)[spot].view(torch.float8_e4m3fn).float(), units)
            pages.view(torch.uint8)[spot] = 0x22
            sc[spot] = 9
    assert (both.view(torch.uint8) == 0x22).all() and (scales == 9).all()


# ------------------------------------------------------------------ read

def run_read(gen, ws, n_kv, page, to_page, lens, order="nhd", to_order="nhd"):
    cache, rows = Q.fill(gen, lens, page, n_kv, spread=20, order=order)
    k_out, v_out, table = P.pages_of(gen, lens, to_page, n_kv, order=to_order, fill=5.0)
    G.paged_read_fp8(ints(lens), *cache, k_out, v_out, table, workspace=ws)
    assert G.device_status(ws) == 0
    for b, n in enumerate(lens):
        spot = P.slots(table, to_page, b, 0, n)
        for out, want in zip((k_out, v_out), rows[b]):
            assert torch.equal(out[spot].double(), want), f"sequence {b}"
            out[spot] = 5.0
    assert (k_out == 5.0).all() and (v_out == 5.0).all()


@pytest.mark.parametrize("n_kv", [1, 2, 3, 8, 32])
@pytest.mark.parametrize("page,to_page", [(16, 16), (16, 128), (256, 32), (64, 1024)])
def test_read_sizes(gen, ws, n_kv, page, to_page):
    run_read(gen, ws, n_kv, page, to_page, [1, 0, 15, 16, 17, 300, 0, 64, 65, 1000])


@pytest.mark.parametrize("order,to_order", [("hnd", "nhd"), ("nhd", "hnd"), ("hnd", "hnd")])
def test_read_orders(gen, ws, order, to_order):
    run_read(gen, ws, 4, 32, 64, [33, 700, 2], order, to_order)


@pytest.mark.parametrize("B", [1, 300, 2048])
def test_read_many_sequences(gen, ws, B):
    run_read(gen, ws, 2, 16, 32, [(29 * b) % 50 if b % 3 else 0 for b in range(B)])


def test_read_skips_and_reports(gen, ws):
    lens = [40, 40, 40]
    cache, rows = Q.fill(gen, lens, 16, 2)
    k_out, v_out, table = P.pages_of(gen, lens, 16, 2, fill=5.0)
    G.paged_read_fp8(ints([-1, 40, 0]), *cache, k_out, v_out, table, workspace=ws)
    assert G.device_status(ws) == 0
    spot = P.slots(table, 16, 1, 0, 40)
    assert torch.equal(k_out[spot].double(), rows[1][0])
    k_out[spot] = 5.0
    assert (k_out == 5.0).all()
    for bad in (-2, 49, 1 << 30):
        G.paged_read_fp8(ints([40, bad, 40]), *cache, k_out, v_out, table, workspace=ws)
        assert G.device_status(ws, clear=True) == 1
        for b in (0, 2):
            assert torch.equal(v_out[P.slots(table, 16, b, 0, 40)].double(), rows[b][1])
    for side in range(2):
        bad_tables = [cache[4].clone(), table.clone()]
        bad_tables[side][1, 1] = (-1, 1 << 20)[side]
        v_out.fill_(5.0)
        G.paged_read_fp8(ints(lens), *cache[:4], bad_tables[0], k_out, v_out, bad_tables[1], workspace=ws)
        assert G.device_status(ws, clear=True) == 3
        for b in (0, 2):
            assert torch.equal(v_out[P.slots(table, 16, b, 0, 40)].double(), rows[b][1])


# ------------------------------------------------------------------ decode

def most_scale(rows):
    """The largest value scale of a sequence's rows (of their largest values: 448 units at most, more than 224)."""
    return float(rows[1].abs().max()) / 224


def check_decode(out, q, rows, scale=P.D ** -0.5):
    for b, (k, v) in enumerate(rows):
        n = k.shape[0]
        if n == 0:
            assert torch.equal(out[b], torch.zeros_like(out[b])), f"sequence {b} sees nothing"
            continue
        ref, mean, size = P.attend64(q[b:b + 1], k, v, n - 1, scale)
        P.check(out[b:b + 1], ref, Q.bound(ref, mean, size, n, most_scale((k, v))), f"sequence {b} of {n} rows")


def run_decode(gen, ws, heads, n_kv, page, lens, scale=P.D ** -0.5, q_scale=1.5, **kw):
    cache, rows = Q.fill(gen, lens, page, n_kv, **kw)
    q = P.normal(gen, len(lens), heads, P.D, scale=q_scale)
    out = torch.full_like(q, math.nan)
    start = ints([n - 1 for n in lens])
    assert G.paged_decode_fp8(q, start, *cache, scale=scale, out=out, workspace=ws) is out
    assert G.device_status(ws) == 0
    check_decode(out, q, rows, scale)
    assert torch.equal(out, G.paged_decode_fp8(q, start, *cache, scale=scale, workspace=ws))


@pytest.mark.parametrize("heads,n_kv", LAYOUTS + [(16, 1), (9, 1), (24, 2)])
@pytest.mark.parametrize("page,order", [(16, "nhd"), (64, "hnd")])
def test_decode_layouts(gen, ws, heads, n_kv, page, order):
    run_decode(gen, ws, heads, n_kv, page, [1, 0, 15, 16, 17, 300, 31, 32, 33, 0, 63, 64, 65, 129], order=order)


@pytest.mark.parametrize("heads,n_kv", [(32, 8), (16, 1), (8, 1)])
@pytest.mark.parametrize("n", [1, 2, 16, 33, 128, 1001, 5000])
def test_decode_one_sequence(gen, ws, heads, n_kv, n):
    run_decode(gen, ws, heads, n_kv, 32, [n])


@pytest.mark.parametrize("page", [16, 32, 128, 4096])
def test_decode_page_sizes(gen, ws, page):
    run_decode(gen, ws, 8, 2, page, [page, page + 1, 2 * page - 1, 1, 40])


@pytest.mark.parametrize("B", [33, 300, 2048])
def test_decode_many_sequences(gen, ws, B):
    run_decode(gen, ws, 4, 2, 16, [(29 * b) % 70 if b % 3 else 0 for b in range(B)])


def test_decode_most_heads_per_kv_head(gen, ws):
    run_decode(gen, ws, 16, 1, 16, [(31 * b) % 40 for b in range(2048)])


def test_decode_lengths_of_every_remainder(gen, ws):
    run_decode(gen, ws, 8, 2, 16, list(range(0, 70)))


def test_decode_long(gen, ws):
    run_decode(gen, ws, 8, 2, 64, [70001, 3, 20000])


def test_decode_strided_queries_and_scale(gen, ws):
    lens = [40, 7, 200]
    cache, rows = Q.fill(gen, lens, 16, 2)
    qkv = P.normal(gen, 3, 12, P.D)
    out = G.paged_decode_fp8(qkv[:, :8], ints([n - 1 for n in lens]), *cache, scale=0.3, workspace=ws)
    check_decode(out, qkv[:, :8], rows, 0.3)


def test_decode_sharp_scores(gen, ws):
    run_decode(gen, ws, 8, 2, 16, [900, 31, 4000], q_scale=60.0)


@pytest.mark.parametrize("spread", [0, 12, 25])
def test_decode_value_scales_far_apart(gen, ws, spread):
    run_decode(gen, ws, 8, 2, 16, [1, 40, 2000], spread=spread)


@pytest.mark.parametrize("at", [2.0 ** -80, 2.0 ** -30, 2.0 ** 30, 2.0 ** 80])
def test_decode_small_and_large_queries(gen, ws, at):
    # scores do not change: keys and queries by powers of two that cancel, in the scale
    lens = [1, 40, 300]
    cache, rows = Q.fill(gen, lens, 16, 2)
    q = P.normal(gen, 3, 8, P.D)
    start = ints([n - 1 for n in lens])
    want = G.paged_decode_fp8(q, start, *cache, scale=0.25, workspace=ws)
    got = G.paged_decode_fp8((q.float() * at).bfloat16(), start, *cache, scale=0.25 / at, workspace=ws)
    assert torch.equal(got, want)
    check_decode(got, q, rows, 0.25)


def test_decode_queries_of_mixed_size(gen, ws):
    # dims down to 2^-26 of the head's largest count in full: the large one meets keys of zero
    lens = [33, 500]
    cache, _ = Q.fill(gen, lens, 16, 1)
    q = P.normal(gen, 2, 4, P.D)
    q[:, :, 5] = 2.0 ** 24
    rows = []
    for b, n in enumerate(lens):
        spot = P.slots(cache[4], 16, b, 0, n)
        cache[0].view(torch.uint8)[(*spot, slice(None), 5)] = 0
        rows.append(tuple(Q.values(cache[i].view(torch.uint8)[spot].view(torch.float8_e4m3fn), cache[2 + i][spot])
                          for i in range(2)))
    out = G.paged_decode_fp8(q, ints([n - 1 for n in lens]), *cache, workspace=ws)
    check_decode(out, q, rows)


def test_decode_nan_stays_where_it_is(gen, ws):
    lens = [50, 50, 50]
    cache, rows = Q.fill(gen, lens, 16, 2)
    q = P.normal(gen, 3, 8, P.D)
    p, r = P.slots(cache[4], 16, 1, 20, 1)
    cache[1].view(torch.uint8)[p, r, 0, 5] = 0x7f            # a value of sequence 1
    p, r = P.slots(cache[4], 16, 2, 7, 1)
    cache[0].view(torch.uint8)[p, r, 1, 9] = 0xff            # a key of sequence 2
    out = G.paged_decode_fp8(q, ints([49, 49, 49]), *cache, workspace=ws)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[1, :4, 5] = True
    hit[2, 4:] = True
    assert torch.isnan(out[hit]).all()
    for b, (k, v) in enumerate(rows):
        ref, mean, size = P.attend64(q[b:b + 1], k, v, 49)
        tol = Q.bound(ref, mean, size, 50, most_scale((k, v)))
        keep = ~hit[b:b + 1]
        P.check(out[b:b + 1][keep], ref[keep], tol[keep], f"sequence {b}")


def test_decode_infinite_and_nan_queries_stay_in_their_heads(gen, ws):
    cache, rows = Q.fill(gen, [50, 50], 16, 2)
    q = P.normal(gen, 2, 8, P.D)
    clean = q.clone()
    q[0, 1, 3], q[1, 6, 100] = math.nan, math.inf
    out = G.paged_decode_fp8(q, ints([49, 49]), *cache, workspace=ws)
    assert torch.isnan(out[0, 1]).all() and torch.isnan(out[1, 6]).all()
    want = G.paged_decode_fp8(clean, ints([49, 49]), *cache, workspace=ws)
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[0, 1], hit[1, 6] = True, True
    assert torch.equal(out[~hit], want[~hit])


def test_decode_zero_queries_average(gen, ws):
    cache, rows = Q.fill(gen, [1, 33, 4000], 32, 2)
    q = torch.zeros(3, 8, P.D, dtype=torch.bfloat16, device="cuda")
    check_decode(G.paged_decode_fp8(q, ints([0, 32, 3999]), *cache, workspace=ws), q, rows)


@pytest.mark.parametrize("heads,n_kv,page,lens", [(8, 2, 64, [70001, 3, 20000]), (32, 8, 16, [1001] * 16),
                                                  (4, 4, 32, [4100, 17, 2049])])
def test_decode_is_close_in_the_mean(gen, ws, heads, n_kv, page, lens):
    cache, rows = Q.fill(gen, lens, page, n_kv, spread=0)
    q = P.normal(gen, len(lens), heads, P.D, scale=1.5)
    out = G.paged_decode_fp8(q, ints([n - 1 for n in lens]), *cache, workspace=ws)
    for b, (k, v) in enumerate(rows):
        P.check_l2(out[b:b + 1], P.attend64(q[b:b + 1], k, v, k.shape[0] - 1)[0], f"sequence {b}")


@pytest.mark.parametrize("heads,n_kv,page,lens", [(8, 2, 64, [70001, 3, 20000]), (16, 1, 16, [9001]),
                                                  (4, 4, 32, [4100, 17, 2049])])
def test_decode_counts_every_key_once(gen, ws, heads, n_kv, page, lens):
    cache, _ = Q.fill(gen, lens, page, n_kv)
    q = torch.zeros(len(lens), heads, P.D, dtype=torch.bfloat16, device="cuda")
    start = ints([n - 1 for n in lens])
    for window in range(-(-max(lens) // P.CODE_WINDOW)):
        for b, n in enumerate(lens):
            spot = P.slots(cache[4], page, b, 0, n)
            x = P.coded_values(n, window, "cuda")[:, None].expand(-1, n_kv, -1).double()
            units, e = Q.quantised(x)
            Q.put(cache[1], spot, Q.as_fp8(units))
            cache[3][spot] = (e + 127).to(torch.uint8)
        out = G.paged_decode_fp8(q, start, *cache, workspace=ws)
        for b, n in enumerate(lens):
            P.check_counts(out[b:b + 1], window, n - 1, f"sequence {b} of {n} rows")
    assert G.device_status(ws) == 0


def test_decode_far_pages(gen, ws):
    """Pages and scales whose offsets pass 32 bits."""
    free = torch.cuda.mem_get_info()[0]
    page, n_kv, pool = 4096, 8, 700
    if free < 30 << 30:
        pytest.skip("needs 12 GB")
    small, rows = Q.fill(gen, [5000, 100], page, n_kv)
    far = [torch.empty(pool, *x.shape[1:], dtype=torch.uint8, device="cuda") for x in small[:4]]
    # 700 pages of 4 MB: 2.9 GB each of k and v, past 2^31
    table = small[4].clone()
    for old in table.unique().tolist():
        if old < 0:
            continue
        new = pool - 1 - old
        for x, y in zip(far, small[:4]):
            x[new] = y.view(torch.uint8)[old]
        table[small[4] == old] = new
    q = P.normal(gen, 2, 32, P.D)
    cache = [x.view(torch.float8_e4m3fn) for x in far[:2]] + far[2:]
    out = G.paged_decode_fp8(q, ints([4999, 99]), *cache, table, workspace=ws)
    assert G.device_status(ws) == 0
    check_decode(out, q, rows)
    k_out, v_out, to = P.pages_of(gen, [5000, 100], 64, n_kv, fill=5.0)
    G.paged_read_fp8(ints([5000, 100]), *cache, table, k_out, v_out, to, workspace=ws)
    assert torch.equal(P.read_rows(v_out, to, 64, 0, 5000).double(), rows[0][1])
    k, v = P.normal(gen, 2, n_kv, P.D), P.normal(gen, 2, n_kv, P.D)
    G.paged_append_fp8(None, k, v, ints([5000, 100]), G.rope_table(5001), *cache, table, workspace=ws)
    assert G.device_status(ws) == 0
    units, e = Q.quantised(v[0].float())
    p, r = P.slots(table, page, 0, 5000, 1)
    assert torch.equal(cache[3][p, r][0].int() - 127, e) and Q.same(far[1][p, r][0].view(torch.float8_e4m3fn).float(), units)


# ------------------------------------------------------------------ errors on the device

def test_bad_positions_are_reported_and_skipped(gen, ws):
    cache, rows = Q.fill(gen, [20, 20, 20], 16, 2)
    cap = cache[4].shape[1] * 16
    q, k, v = (P.normal(gen, 3, h, P.D) for h in (8, 2, 2))
    rope = G.rope_table(cap)
    for bad in (-2, cap, 1 << 30):
        out = G.paged_decode_fp8(q, ints([19, bad, 19]), *cache, workspace=ws)
        assert G.device_status(ws, clear=True) == 1
        assert torch.equal(out[1], torch.zeros_like(out[1]))
        check_decode(out[[0, 2]], q[[0, 2]], [rows[0], rows[2]])
        before = [x.view(torch.uint8).clone() for x in cache[:4]]
        G.paged_append_fp8(None, k, v, ints([-1, bad, -1]), rope, *cache, workspace=ws)
        assert G.device_status(ws, clear=True) == 1
        assert all(torch.equal(x.view(torch.uint8), y) for x, y in zip(cache, before))
    G.paged_append_fp8(None, k, v, ints([-1, 20, -1]), rope[:20], *cache, workspace=ws)
    assert G.device_status(ws, clear=True) == 1


@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("entry", [-1, 1 << 20])
def test_bad_pages_are_reported(gen, ws, entry, page):
    cache, rows = Q.fill(gen, [40, 40], page, 2)
    table = cache[4]
    table[0, 1] = entry
    q, k, v = (P.normal(gen, 2, h, P.D) for h in (8, 2, 2))
    out = G.paged_decode_fp8(q, ints([39, 39]), *cache, workspace=ws)
    assert G.device_status(ws, clear=True) == 3
    check_decode(out[1:], q[1:], rows[1:])
    G.paged_append_fp8(None, k, v, ints([page, -1]), G.rope_table(64), *cache, workspace=ws)
    assert G.device_status(ws, clear=True) == 3
    run_decode(gen, ws, 8, 2, 16, [300, 40])


# ------------------------------------------------------------------ as a server uses them

@pytest.mark.parametrize("dim,halves", [(128, False), (64, True)])
def test_prompts_chunks_and_decode_steps_together(gen, ws, dim, halves):
    """Prompts in, chunk by chunk (read back for the prefill attention), then
    decode steps with one slot unused: every output against the 64-bit attention
    over everything appended so far."""
    heads, n_kv, page, B = 8, 2, 16, 4
    plan = [[37, 5, 0, 64], [20, 100, 1, 3], [1, 1, 1, 1], [1, 1, 1, 1], [1, 1, 0, 1]]
    total = [sum(x) for x in zip(*plan)]
    *cache, table = Q.pages_of(gen, total, page, n_kv)
    rope = rotary_table(256, dim)
    columns = 4
    k_out, v_out = (torch.full((B * columns, 64, n_kv, P.D), math.nan, dtype=torch.bfloat16, device="cuda")
                    for _ in range(2))
    to = torch.arange(B * columns, dtype=torch.int32, device="cuda").view(B, columns)
    start = [0] * B
    for lens in plan:
        step = max(lens) == 1
        rows_of = [1] * B if step else lens
        starts = [s if t else -1 for s, t in zip(start, lens)] if step else start
        q, k, v = inputs(gen, sum(rows_of), heads, n_kv, True)
        cu, sp = offsets(rows_of), ints(starts)
        rq = G.paged_append_fp8(q, k, v, sp, rope, *cache, table, cu_tokens=None if step else cu, rotary_dim=dim,
                                halves=halves, workspace=ws)
        if step:
            out = G.paged_decode_fp8(rq, sp, *cache, table, workspace=ws)
        else:
            G.paged_read_fp8(sp + (cu[1:] - cu[:-1]), *cache, table, k_out, v_out, to, workspace=ws)
            out = G.paged_prefill(rq, cu, sp, k_out, v_out, to, workspace=ws)
        at = 0
        for b, (t, s) in enumerate(zip(rows_of, starts)):
            r = slice(at, at + t)
            at += t
            if s < 0:
                assert torch.equal(out[r], torch.zeros_like(out[r]))
                continue
            if t == 0:
                continue
            cs = rope[s:s + t]
            check_turned(rq[r], q[r], cs, halves, "turned q")
            spot = P.slots(table, page, b, 0, s + t)
            kk, vv = (Q.values(cache[i].view(torch.uint8)[spot].view(torch.float8_e4m3fn), cache[2 + i][spot])
                      for i in range(2))
            # what was appended is within its rounding of what was given
            for have, given in ((kk[s:], Q.turned64(k[r], cs, halves)[0]), (vv[s:], v[r].double())):
                off = (have - given).abs()
                assert (off <= 2.0 ** -4 * 1.001 * given.abs() + 2.0 ** -10 * given.abs().amax(-1, keepdim=True) / 200).all()
            ref, mean, size = P.attend64(rq[r], kk, vv, s)
            tol = Q.bound(ref, mean, size, s + t, most_scale((kk, vv))) if step else \
                P.bound(ref, mean, size, s + t, P.P_ONE_TERM)
            P.check(out[r], ref, tol, f"sequence {b}, {t} tokens after {s}")
        start = [s + t for s, t in zip(start, lens)]
    assert G.device_status(ws) == 0


def test_a_captured_step_replays_with_other_lengths(gen):
    heads, n_kv, page, B = 8, 2, 16, 3
    ws = G.make_paged_workspace()
    cache, _ = Q.fill(gen, [600, 600, 600], page, n_kv, byte=0)
    rope = G.rope_table(600)
    qkv = P.normal(gen, B, heads + 2 * n_kv, P.D)
    start = ints([5, 5, 5])
    q_out, out = (torch.empty(B, heads, P.D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k_out, v_out = (torch.empty(B * 10, 64, n_kv, P.D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    to = torch.arange(B * 10, dtype=torch.int32, device="cuda").view(B, 10)

    def step():
        G.paged_append_fp8(qkv[:, :heads], qkv[:, heads:heads + n_kv], qkv[:, heads + n_kv:], start, rope, *cache,
                           q_out=q_out, halves=True, workspace=ws)
        G.paged_decode_fp8(q_out, start, *cache, out=out, workspace=ws)
        G.paged_read_fp8(start, *cache, k_out, v_out, to, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        step()
        for _ in range(2):   # two graphs over one workspace
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                step()
            graphs.append(g)
    torch.cuda.current_stream().wait_stream(side)
    for i, lens in enumerate(([599, 0, 17], [-1, 300, 64], [15, 16, 500])):
        start.copy_(ints(lens))
        qkv.copy_(P.normal(gen, B, heads + 2 * n_kv, P.D))
        graphs[i % 2].replay()
        o, q = out.clone(), q_out.clone()
        assert torch.equal(o, G.paged_decode_fp8(q, start, *cache, workspace=G.make_paged_workspace()))
        rows = []
        for b, s in enumerate(lens):
            spot = P.slots(cache[4], page, b, 0, s + 1)
            rows.append(tuple(Q.values(cache[j].view(torch.uint8)[spot].view(torch.float8_e4m3fn), cache[2 + j][spot])
                              for j in range(2)))
            if s > 0:
                assert torch.equal(P.read_rows(v_out, to, 64, b, s).double(), rows[b][1][:s])
        check_decode(o, q, rows)
    assert G.device_status(ws) == 0


def test_calls_on_two_streams_and_without_workspaces(gen):
    cache, rows = Q.fill(gen, [3000, 40, 700], 32, 4)
    start = ints([2999, 39, 699])
    qs = [P.normal(gen, 3, 16, P.D) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(10):
        for i in range(2):
            outs[i].append(G.paged_decode_fp8(qs[i], start, *cache, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        check_decode(outs[i][0], qs[i], rows)
        assert all(torch.equal(o, outs[i][0]) for o in outs[i])
        assert G.device_status(G.default_paged_workspace(stream=streams[i])) == 0


def test_launch_counts_and_empty_calls(gen, ws):
    cache, rows = Q.fill(gen, [40], 16, 2)
    q = P.normal(gen, 1, 8, P.D)
    G.paged_decode_fp8(q, ints([39]), *cache, workspace=ws)
    assert G.last_launch_count() == 1
    none = q[:0]
    empty = (*cache[:4], cache[4][:0])
    assert G.paged_decode_fp8(none, ints([]), *empty, workspace=ws).shape == (0, 8, P.D)
    assert G.paged_append_fp8(None, none[:, :2], none[:, :2], ints([39]), G.rope_table(64), *cache,
                              cu_tokens=offsets([0]), workspace=ws) is None
    k_out, v_out, to = P.pages_of(gen, [40], 16, 2)
    G.paged_read_fp8(ints([]), *empty, k_out, v_out, to[:0], workspace=ws)
