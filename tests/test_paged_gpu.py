"""The paged serving operators against 64-bit references, at the sizes, masks
and layouts where they can go wrong."""
import math
import time

import pytest
import torch

import grouped_query_attention_gemv_gb300 as G
from tests import paged as P

pytestmark = pytest.mark.gpu

LAYOUTS = [(32, 8), (32, 32), (4, 1), (28, 4), (64, 4), (3, 3), (10, 2)]


@pytest.fixture(scope="module")
def ws():
    return G.make_paged_workspace()


@pytest.fixture
def gen():
    return torch.Generator(device="cuda").manual_seed(5)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def offsets(lens, first=0):
    c = [first]
    for n in lens:
        c.append(c[-1] + n)
    return ints(c)


# ------------------------------------------------------------------ append

def run_append(gen, ws, heads, n_kv, page, lens, starts, order="nhd", strided=True, cu=True, with_q=True, behind=0,
               in_place=False):
    n = sum(lens) + behind
    ends = [s + t if s >= 0 else 0 for s, t in zip(starts, lens)]
    k_pages, v_pages, table = P.pages_of(gen, ends, page, n_kv, order=order, fill=3.0)
    if strided:
        qkv = P.normal(gen, n, heads + 2 * n_kv, P.D)
        q, k, v = qkv[:, :heads], qkv[:, heads:heads + n_kv], qkv[:, heads + n_kv:]
    else:
        q, k, v = (P.normal(gen, n, h, P.D) for h in (heads, n_kv, n_kv))
    q0 = q.clone()
    rope = G.rope_table(max(max(ends), 1))
    before_k, before_v = k_pages.clone(), v_pages.clone()
    q_out = q if in_place else torch.full((n, heads, P.D), 7.0, dtype=torch.bfloat16, device="cuda")
    q_before = q_out.clone()
    got = G.paged_append(q if with_q else None, k, v, ints(starts), rope, k_pages, v_pages, table,
                         cu_tokens=offsets(lens) if cu else None, q_out=q_out if with_q else None, workspace=ws)
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
        cs = rope[s:s + t]
        if with_q:
            P.check_rotated(q_out[rows], q0[rows], cs, f"q of sequence {b}")
        p, r = P.slots(table, page, b, s, t)
        P.check_rotated(k_pages[p, r], k[rows], cs, f"k of sequence {b}")
        assert torch.equal(v_pages[p, r], v[rows])
        k_pages[p, r] = before_k[p, r]
        v_pages[p, r] = before_v[p, r]
    # every other row, of the pages and of the queries, is as it was
    assert torch.equal(k_pages, before_k) and torch.equal(v_pages, before_v)
    assert torch.equal(q_out[at:], q_before[at:])
    assert G.device_status(ws) == 0


@pytest.mark.parametrize("heads,n_kv", LAYOUTS)
@pytest.mark.parametrize("page", [16, 128])
def test_append_layouts(gen, ws, heads, n_kv, page):
    run_append(gen, ws, heads, n_kv, page, [1, 0, 17, 33, 1], [0, 4, 15, 127, 16])


@pytest.mark.parametrize("kw", [dict(order="hnd"), dict(strided=False), dict(with_q=False), dict(behind=9),
                                dict(strided=False, in_place=True)])
def test_append_forms(gen, ws, kw):
    run_append(gen, ws, 8, 2, 32, [5, 40, 0, 3], [31, -1, 3, 64], **kw)


@pytest.mark.parametrize("shape,at", [((9, 2, 16, 2, P.D), 1), ((9, 16, 2, 2, P.D), 2), ((9, 16, 2, 2, P.D), 3),
                                      ((2, 9, 16, 2, P.D), 0)])
def test_append_into_interleaved_pages(gen, ws, shape, at):
    # keys and values in one tensor, beside each other by page, row or head, or one behind the other
    both = torch.full(shape, 3.0, dtype=torch.bfloat16, device="cuda")
    k_pages, v_pages = both.unbind(at)
    table = torch.randperm(9, generator=gen, device="cuda")[:8].view(2, 4).int()
    k, v = P.normal(gen, 70, 2, P.D), P.normal(gen, 70, 2, P.D)
    rope = G.rope_table(64)
    G.paged_append(None, k, v, ints([3, 0]), rope, k_pages, v_pages, table, cu_tokens=offsets([20, 50]), workspace=ws)
    assert G.device_status(ws) == 0
    for b, (rows, s) in enumerate(((slice(0, 20), 3), (slice(20, 70), 0))):
        t = rows.stop - rows.start
        p, r = P.slots(table, 16, b, s, t)
        P.check_rotated(k_pages[p, r], k[rows], rope[s:s + t], f"k of sequence {b}")
        assert torch.equal(v_pages[p, r], v[rows])
        k_pages[p, r], v_pages[p, r] = 3.0, 3.0
    assert (both == 3.0).all()


def test_append_refuses_rows_that_lie_in_the_pages(gen, ws):
    k_pages, v_pages = (P.normal(gen, 6, 16, 2, P.D) for _ in range(2))
    before = k_pages.clone(), v_pages.clone()
    table, rope = ints([[0, 1], [2, 3]]), G.rope_table(32)
    k, v = P.normal(gen, 2, 2, P.D), P.normal(gen, 2, 2, P.D)
    for args in ((k_pages[5, :2], v), (k, k_pages[5, :2]), (v_pages[4, 3:5], v), (k, v_pages[4, 3:5])):
        with pytest.raises(G.GQAError):
            G.paged_append(None, *args, ints([3, 9]), rope, k_pages, v_pages, table, workspace=ws)
    with pytest.raises(G.GQAError):
        G.paged_append(None, k, v, ints([3, 9]), rope, k_pages, k_pages, table, workspace=ws)
    assert torch.equal(k_pages, before[0]) and torch.equal(v_pages, before[1])


@pytest.mark.parametrize("B", [1, 2, 33, 300])
def test_append_one_token_each(gen, ws, B):
    run_append(gen, ws, 4, 2, 16, [1] * B, [(37 * b) % 50 - 1 for b in range(B)], cu=False)


@pytest.mark.parametrize("B", [31, 32, 33, 65, 1025])
def test_append_finds_the_sequence(gen, ws, B):
    # lengths 0..3: empty sequences at the start, the end and between
    run_append(gen, ws, 1, 1, 16, [(b * 7 // 3) % 4 for b in range(B)], [b % 5 for b in range(B)])


# ------------------------------------------------------------------ decode

def fill_cache(gen, lens, page, n_kv, order="nhd", junk=math.nan, **kw):
    """Pages whose rows past each sequence's end hold `junk`."""
    k_pages, v_pages, table = P.pages_of(gen, lens, page, n_kv, order=order, fill=junk, **kw)
    rows = []
    for b, n in enumerate(lens):
        k, v = P.normal(gen, n, n_kv, P.D), P.normal(gen, n, n_kv, P.D)
        if n:
            P.write_rows(k_pages, table, page, b, 0, k)
            P.write_rows(v_pages, table, page, b, 0, v)
        rows.append((k, v))
    return k_pages, v_pages, table, rows


def check_decode(out, q, rows, scale=P.D ** -0.5):
    for b, (k, v) in enumerate(rows):
        n = k.shape[0]
        if n == 0:
            assert torch.equal(out[b], torch.zeros_like(out[b])), f"sequence {b} sees nothing"
            continue
        ref, mean, size = P.attend64(q[b:b + 1], k, v, n - 1, scale)
        P.check(out[b:b + 1], ref, P.bound(ref, mean, size, n, P.P_TWO_TERMS), f"sequence {b} of {n} rows")


def run_decode(gen, ws, heads, n_kv, page, lens, order="nhd", scale=P.D ** -0.5, q_scale=1.5, **kw):
    k_pages, v_pages, table, rows = fill_cache(gen, lens, page, n_kv, order, **kw)
    q = P.normal(gen, len(lens), heads, P.D, scale=q_scale)
    out = torch.full_like(q, math.nan)
    start = ints([n - 1 for n in lens])
    assert G.paged_decode(q, start, k_pages, v_pages, table, scale=scale, out=out, workspace=ws) is out
    check_decode(out, q, rows, scale)
    assert G.device_status(ws) == 0
    again = G.paged_decode(q, start, k_pages, v_pages, table, scale=scale, workspace=ws)
    assert torch.equal(out, again)


@pytest.mark.parametrize("heads,n_kv", LAYOUTS)
@pytest.mark.parametrize("page,order", [(16, "nhd"), (64, "hnd")])
def test_decode_layouts(gen, ws, heads, n_kv, page, order):
    run_decode(gen, ws, heads, n_kv, page, [1, 0, 15, 16, 17, 300, 63, 64, 65, 0, 129], order)


@pytest.mark.parametrize("heads,n_kv", [(32, 8), (16, 1), (8, 1)])
@pytest.mark.parametrize("n", [1, 2, 16, 33, 128, 1001, 5000])
def test_decode_one_sequence(gen, ws, heads, n_kv, n):
    run_decode(gen, ws, heads, n_kv, 32, [n])


@pytest.mark.parametrize("page", [16, 32, 128, 4096])
def test_decode_page_sizes(gen, ws, page):
    run_decode(gen, ws, 8, 2, page, [page, page + 1, 2 * page - 1, 1, 40], junk=math.inf)


@pytest.mark.parametrize("B", [33, 300, 2048])
def test_decode_many_sequences(gen, ws, B):
    # more sequences than CTAs, most of them short, unused slots between
    run_decode(gen, ws, 4, 2, 16, [(29 * b) % 50 if b % 3 else 0 for b in range(B)])


def test_decode_lengths_of_every_remainder(gen, ws):
    run_decode(gen, ws, 8, 2, 16, list(range(0, 70)))


def test_decode_long(gen, ws):
    run_decode(gen, ws, 8, 2, 64, [70001, 3, 20000])


def test_decode_strided_queries_and_scale(gen, ws):
    lens = [40, 7, 200]
    k_pages, v_pages, table, rows = fill_cache(gen, lens, 16, 2)
    qkv = P.normal(gen, 3, 12, P.D)
    out = G.paged_decode(qkv[:, :8], ints([n - 1 for n in lens]), k_pages, v_pages, table, scale=0.3, workspace=ws)
    check_decode(out, qkv[:, :8], rows, 0.3)


def test_decode_sharp_scores(gen, ws):
    # scores of several hundred: one key takes everything, and the maxima of the parts differ by far more than 2^8
    run_decode(gen, ws, 8, 2, 16, [900, 31, 4000], q_scale=60.0)


def test_decode_visible_infinity_and_nan_stay_where_they_are(gen, ws):
    lens = [50, 50, 50]
    k_pages, v_pages, table, rows = fill_cache(gen, lens, 16, 2)
    q = P.normal(gen, 3, 8, P.D)
    for b, value in ((0, math.inf), (1, math.nan)):
        p, r = P.slots(table, 16, b, 20, 1)
        v_pages[p, r, 0, 5] = value
    out = G.paged_decode(q, ints([49, 49, 49]), k_pages, v_pages, table, workspace=ws)
    assert (out[0, :4, 5] == math.inf).all() and torch.isnan(out[1, :4, 5]).all()
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[:2, :4, 5] = True
    for b, (k, v) in enumerate(rows):
        ref, mean, size = P.attend64(q[b:b + 1], k, v, 49)
        tol = P.bound(ref, mean, size, 50, P.P_TWO_TERMS)
        keep = ~hit[b:b + 1]
        P.check(out[b:b + 1][keep], ref[keep], tol[keep], f"sequence {b}")


@pytest.mark.parametrize("value", [math.inf, -math.inf])
def test_decode_infinity_of_little_weight(gen, ws, value):
    # an infinite value is one however little its key weighs, down to 2^-126 of the largest
    scale = math.log(2.0) * (1 - 2.0 ** -20)   # scores count powers of two, and stay above 2^-126 where rounded
    lens = [17] * 127
    k_pages, v_pages, table, rows = fill_cache(gen, lens, 32, 1, junk=0.0)
    k_pages.zero_()
    q = torch.zeros(127, 1, P.D, dtype=torch.bfloat16, device="cuda")
    q[:, 0, 0] = 1.0
    for b in range(127):
        p, r = P.slots(table, 32, b, 5, 1)
        k_pages[p, r, 0, 0] = -float(b)
        v_pages[p, r, 0, 7] = value
    out = G.paged_decode(q, ints([16] * 127), k_pages, v_pages, table, scale=scale, workspace=ws)
    assert G.device_status(ws) == 0
    assert (out[:, 0, 7] == value).all(), out[:, 0, 7].tolist()
    keep = [d for d in range(P.D) if d != 7]
    for b in range(127):
        k, v = (P.read_rows(x, table, 32, b, 17) for x in (k_pages, v_pages))
        ref, mean, size = P.attend64(q[b:b + 1], k, torch.nan_to_num(v, 0.0, 0.0, 0.0), 16, scale)
        tol = P.bound(ref, mean, size, 17, P.P_TWO_TERMS)
        P.check(out[b:b + 1, :, keep], ref[..., keep], tol[..., keep], f"weight 2^-{b}")


def test_decode_far_pages(gen, ws):
    # element offsets past 2^32
    n_kv, page = 8, 64
    pool = (1 << 32) // (page * n_kv * P.D) + 40
    k_pages, v_pages = (torch.empty(pool, page, n_kv, P.D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lens = [200, 70]
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    table[0] = ints([pool - 1, 3, pool - 7, pool - 2])
    table[1, :2] = ints([pool - 5, 0])
    rows = []
    for b, n in enumerate(lens):
        k, v = P.normal(gen, n, n_kv, P.D), P.normal(gen, n, n_kv, P.D)
        P.write_rows(k_pages, table, page, b, 0, k)
        P.write_rows(v_pages, table, page, b, 0, v)
        rows.append((k, v))
    q = P.normal(gen, 2, 32, P.D)
    start = ints([n - 1 for n in lens])
    check_decode(G.paged_decode(q, start, k_pages, v_pages, table, workspace=ws), q, rows)
    # the last rows once more, through the append, and the same attention through the prefill
    k, v = P.normal(gen, 2, n_kv, P.D), P.normal(gen, 2, n_kv, P.D)
    rope = G.rope_table(256)
    G.paged_append(None, k, v, start, rope, k_pages, v_pages, table, workspace=ws)
    for b, n in enumerate(lens):
        p, r = P.slots(table, page, b, n - 1, 1)
        P.check_rotated(k_pages[p, r], k[b:b + 1], rope[n - 1:n], "far k row")
        assert torch.equal(v_pages[p, r], v[b:b + 1])
        rows[b][0][-1], rows[b][1][-1] = k_pages[p, r][0], v[b]
    out = G.paged_prefill(q, offsets([1, 1]), start, k_pages, v_pages, table, workspace=ws)
    for b, (kk, vv) in enumerate(rows):
        ref, mean, size = P.attend64(q[b:b + 1], kk, vv, lens[b] - 1)
        P.check(out[b:b + 1], ref, P.bound(ref, mean, size, lens[b], P.P_ONE_TERM), f"sequence {b}")


# ------------------------------------------------------------------ prefill

def check_prefill(out, q, rows, lens, starts, scale=P.D ** -0.5, first=0):
    at = first
    for b, (t, s) in enumerate(zip(lens, starts)):
        o, x = out[at:at + t], q[at:at + t]
        at += t
        if t == 0:
            continue
        if s < 0:
            assert torch.equal(o, torch.zeros_like(o)), f"slot {b} is unused"
            continue
        k, v = rows[b]
        ref, mean, size = P.attend64(x, k, v, s, scale)
        fine = torch.isfinite(ref).all(-1)
        assert torch.isnan(o[~fine]).any(-1).all(), f"sequence {b}: a visible NaN was lost"
        tol = P.bound(ref, mean, size, s + t, P.P_ONE_TERM)
        P.check(o[fine], ref[fine], tol[fine], f"sequence {b}: {t} tokens after {s}")


def run_paged_prefill(gen, ws, heads, n_kv, page, lens, starts, order="nhd", behind=0, scale=P.D ** -0.5, q_scale=1.5):
    ends = [s + t if s >= 0 and t else 0 for s, t in zip(starts, lens)]
    k_pages, v_pages, table, rows = fill_cache(gen, ends, page, n_kv, order)
    n = sum(lens) + behind
    q = P.normal(gen, n, heads, P.D, scale=q_scale)
    out = torch.full_like(q, 9.0)
    args = (q, offsets(lens), ints(starts), k_pages, v_pages, table)
    assert G.paged_prefill(*args, scale=scale, out=out, workspace=ws) is out
    assert G.device_status(ws) == 0
    check_prefill(out, q, rows, lens, starts, scale)
    assert (out[sum(lens):] == 9.0).all()
    assert torch.equal(out[:sum(lens)], G.paged_prefill(*args, scale=scale, workspace=ws)[:sum(lens)])


def run_packed(gen, ws, heads, n_kv, lens, strided=True, behind=0, first=0, **kw):
    n = first + sum(lens) + behind
    if strided:
        qkv = P.normal(gen, n, heads + 2 * n_kv, P.D)
        q, k, v = qkv[:, :heads], qkv[:, heads:heads + n_kv], qkv[:, heads + n_kv:]
    else:
        q, k, v = (P.normal(gen, n, h, P.D) for h in (heads, n_kv, n_kv))
    if behind:
        k[first + sum(lens):], v[first + sum(lens):] = math.nan, math.nan
    out = torch.full((n, heads, P.D), 9.0, dtype=torch.bfloat16, device="cuda")
    G.packed_prefill(q, k, v, offsets(lens, first), out=out, workspace=ws, **kw)
    assert G.device_status(ws) == 0
    rows, at = [], first
    for t in lens:
        rows.append((k[at:at + t], v[at:at + t]))
        at += t
    check_prefill(out, q, rows, lens, [0] * len(lens), first=first, **kw)
    assert (out[:first] == 9.0).all() and (out[at:] == 9.0).all()


@pytest.mark.parametrize("heads,n_kv", LAYOUTS)
@pytest.mark.parametrize("page,order", [(16, "nhd"), (64, "hnd")])
def test_paged_prefill_layouts(gen, ws, heads, n_kv, page, order):
    run_paged_prefill(gen, ws, heads, n_kv, page, [1, 70, 0, 33, 5, 129], [0, 0, 7, 100, -1, 63], order, behind=3)


@pytest.mark.parametrize("page", [16, 32, 128, 4096])
@pytest.mark.parametrize("lens,starts", [([1], [0]), ([17], [0]), ([64], [64]), ([65], [63]), ([300], [1]),
                                         ([3, 2], [1000, 0])])
def test_paged_prefill_tile_edges(gen, ws, page, lens, starts):
    run_paged_prefill(gen, ws, 8, 2, page, lens, starts)


def test_paged_prefill_few_rows_after_a_long_prefix(gen, ws):
    run_paged_prefill(gen, ws, 8, 2, 64, [3, 40], [20000, 9000])


def test_paged_prefill_more_items_than_ctas(gen, ws):
    run_paged_prefill(gen, ws, 16, 4, 32, [700, 1, 0, 513, 64, 255], [0, 300, 3, 40, 0, 1])


def test_paged_prefill_many_sequences(gen, ws):
    run_paged_prefill(gen, ws, 4, 2, 16, [b % 4 for b in range(2048)], [b % 37 - 1 for b in range(2048)])


def test_paged_prefill_scale_and_sharp_scores(gen, ws):
    run_paged_prefill(gen, ws, 8, 2, 16, [200], [90], scale=0.02)
    run_paged_prefill(gen, ws, 8, 2, 16, [200], [90], q_scale=60.0)


@pytest.mark.parametrize("heads,n_kv", LAYOUTS)
def test_packed_prefill_layouts(gen, ws, heads, n_kv):
    run_packed(gen, ws, heads, n_kv, [1, 70, 0, 130, 5], behind=4)


@pytest.mark.parametrize("lens", [[1], [2], [63], [64], [65], [256], [257], [0, 0, 9, 0], [1] * 40, [600, 3, 900]])
@pytest.mark.parametrize("strided", [False, True])
def test_packed_prefill_lengths(gen, ws, lens, strided):
    run_packed(gen, ws, 8, 2, lens, strided=strided)


def test_packed_prefill_rows_before_the_first_sequence(gen, ws):
    run_packed(gen, ws, 8, 2, [30, 100], first=5, behind=2)


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("at", [0, 10, 63, 64, 100, 199])
def test_packed_prefill_rows_do_not_see_later_values(gen, ws, value, at):
    # a non-finite value row in the middle of a sequence: earlier rows are
    # untouched by it, also those of its own tile; later rows show it
    q, k, v = (P.normal(gen, 300, h, P.D) for h in (8, 2, 2))
    clean = v.clone()
    v[at, 1, 3] = value
    out = G.packed_prefill(q, k, v, offsets([200, 100]), workspace=ws)
    assert G.device_status(ws) == 0
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[at:200, 4:, 3] = True
    if math.isnan(value):
        assert torch.isnan(out[hit]).all()
    else:
        assert (out[hit] == value).all()
    for rows in (slice(0, 200), slice(200, 300)):
        ref, mean, size = P.attend64(q[rows], k[rows], clean[rows], 0)
        tol = P.bound(ref, mean, size, 200, P.P_ONE_TERM)
        keep = ~hit[rows]
        P.check(out[rows][keep], ref[keep], tol[keep], f"rows {rows}")


def test_packed_prefill_rows_do_not_see_later_keys(gen, ws):
    q, k, v = (P.normal(gen, 200, h, P.D) for h in (8, 2, 2))
    clean = k.clone()
    k[150:] = math.nan
    out = G.packed_prefill(q, k, v, offsets([200]), workspace=ws)
    ref, mean, size = P.attend64(q[:150], clean[:150], v[:150], 0)
    P.check(out[:150], ref, P.bound(ref, mean, size, 200, P.P_ONE_TERM), "rows before the NaN keys")
    assert torch.isnan(out[150:]).all()


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("new,prefix,at", [(100, 6000, 6050), (100, 6000, 3000), (64, 500, 563), (1, 9000, 9000)])
def test_paged_prefill_shared_items_do_not_see_later_values(gen, ws, value, new, prefix, at):
    # few items after a long prefix: their keys are split over CTAs and joined
    k_pages, v_pages, table, rows = fill_cache(gen, [prefix + new, 40], 64, 2)
    p, r = P.slots(table, 64, 0, at, 1)
    v_pages[p, r, 1, 3] = value
    q = P.normal(gen, new + 2, 8, P.D)
    out = G.paged_prefill(q, offsets([new, 2]), ints([prefix, 38]), k_pages, v_pages, table, workspace=ws)
    assert G.device_status(ws) == 0
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[max(0, at - prefix):new, 4:, 3] = True
    assert (torch.isnan(out[hit]) if math.isnan(value) else out[hit] == value).all()
    for sl, (k, v), first in ((slice(0, new), rows[0], prefix), (slice(new, new + 2), rows[1], 38)):
        ref, mean, size = P.attend64(q[sl], k, v, first)
        tol = P.bound(ref, mean, size, k.shape[0], P.P_ONE_TERM)
        keep = ~hit[sl]
        P.check(out[sl][keep], ref[keep], tol[keep], f"rows {sl}")


def test_paged_prefill_shared_items_and_unused_slots(gen, ws):
    run_paged_prefill(gen, ws, 8, 2, 64, [5, 33, 1, 0, 70, 2], [4000, -1, 12000, 100, -1, 0])


def test_paged_prefill_one_item_over_every_cta(gen, ws):
    run_paged_prefill(gen, ws, 16, 1, 128, [8], [60000])


@pytest.mark.parametrize("heads,n_kv,lens,starts", [
    (8, 2, [300], [9000]), (28, 4, [100], [5000]), (28, 4, [1, 90], [7000, 2500]), (16, 16, [130], [4000]),
    (32, 8, [600, 40], [5000, 3000]), (32, 8, [1000], [1500]), (4, 1, [2500], [0]), (16, 1, [40], [30000]),
    # around the most rows that an item can span in the join's short slices
    (8, 2, [5], [2100]), (8, 2, [40], [8000]), (8, 2, [41], [8000]), (28, 4, [18], [3000]), (28, 4, [19], [3000]),
    (28, 4, [23], [3000]), (4, 4, [129], [3000]), (4, 4, [161], [3000]), (16, 1, [9, 3], [5000, 9000])])
def test_paged_prefill_items_shared_by_few_and_many(gen, ws, heads, n_kv, lens, starts):
    run_paged_prefill(gen, ws, heads, n_kv, 64, lens, starts, behind=2)


@pytest.mark.parametrize("heads,n_kv,lens,starts", [(32, 8, [600, 40], [5000, 3000]), (32, 8, [1024], [7168])])
def test_paged_prefill_does_not_depend_on_who_is_last(gen, ws, heads, n_kv, lens, starts):
    k_pages, v_pages, table, rows = fill_cache(gen, [s + t for s, t in zip(starts, lens)], 64, n_kv)
    q = P.normal(gen, sum(lens), heads, P.D, scale=1.5)
    args = (q, offsets(lens), ints(starts), k_pages, v_pages, table)
    first = G.paged_prefill(*args, workspace=ws)
    for _ in range(40):
        assert torch.equal(first, G.paged_prefill(*args, workspace=ws))


def test_paged_prefill_joins_only_its_own_items(gen, ws):
    # the second call has none to join: what the first left stays unread
    k_pages, v_pages, table, ((k, v),) = fill_cache(gen, [9000], 64, 2)
    q = P.normal(gen, 100, 8, P.D)
    out = torch.full_like(q, 9.0)
    G.paged_prefill(q, offsets([100]), ints([8900]), k_pages, v_pages, table, out=out, workspace=ws)
    assert G.last_launch_count() == 2
    check_prefill(out, q, [(k, v)], [100], [8900])
    out.fill_(9.0)
    G.paged_prefill(q, offsets([3]), ints([0]), k_pages, v_pages, table, out=out, workspace=ws)
    assert G.device_status(ws) == 0
    check_prefill(out, q, [(k[:3], v[:3])], [3], [0])
    assert (out[3:] == 9.0).all()


# ------------------------------------------------------------------ nothing lost, nothing twice

@pytest.mark.parametrize("heads,n_kv,page,lens", [(8, 2, 64, [70001, 3, 20000]), (32, 8, 16, [1001] * 16),
                                                  (16, 1, 128, [131072]), (32, 8, 64, [8192, 1, 4000, 17, 300]),
                                                  (32, 32, 32, [1001] * 3)])
def test_decode_is_close_in_the_mean(gen, ws, heads, n_kv, page, lens):
    k_pages, v_pages, table, rows = fill_cache(gen, lens, page, n_kv)
    q = P.normal(gen, len(lens), heads, P.D, scale=1.5)
    out = G.paged_decode(q, ints([n - 1 for n in lens]), k_pages, v_pages, table, workspace=ws)
    for b, (k, v) in enumerate(rows):
        P.check_l2(out[b:b + 1], P.attend64(q[b:b + 1], k, v, lens[b] - 1)[0], f"sequence {b} of {lens[b]} rows")


SHARED = [(16, 1, 128, [8], [60000]), (32, 8, 64, [1024], [7168]), (8, 2, 64, [40, 5], [8000, 2100]),
          (32, 8, 64, [600, 40], [5000, 3000]), (28, 4, 64, [100], [5000]), (4, 1, 64, [2500], [0]),
          (8, 2, 64, [700, 1, 300], [20, 12000, 0])]


@pytest.mark.parametrize("heads,n_kv,page,lens,starts", SHARED)
def test_paged_prefill_is_close_in_the_mean(gen, ws, heads, n_kv, page, lens, starts):
    k_pages, v_pages, table, rows = fill_cache(gen, [s + t for s, t in zip(starts, lens)], page, n_kv)
    q = P.normal(gen, sum(lens), heads, P.D, scale=1.5)
    out = G.paged_prefill(q, offsets(lens), ints(starts), k_pages, v_pages, table, workspace=ws)
    at = 0
    for b, (t, s) in enumerate(zip(lens, starts)):
        ref = P.attend64(q[at:at + t], *rows[b], s)[0]
        P.check_l2(out[at:at + t], ref, f"sequence {b}: {t} tokens after {s}")
        at += t


def test_packed_prefill_is_close_in_the_mean(gen, ws):
    lens = [2048, 5, 700]
    q, k, v = (P.normal(gen, sum(lens), h, P.D, scale=1.5) for h in (32, 8, 8))
    out = G.packed_prefill(q, k, v, offsets(lens), workspace=ws)
    at = 0
    for t in lens:
        r = slice(at, at + t)
        at += t
        P.check_l2(out[r], P.attend64(q[r], k[r], v[r], 0)[0], f"{t} tokens")


def coded(k_pages, v_pages, table, page, ends, window):
    for b, n in enumerate(ends):
        if n:
            P.write_rows(v_pages, table, page, b, 0,
                         P.coded_values(n, window, "cuda")[:, None].expand(-1, v_pages.shape[2], -1))


@pytest.mark.parametrize("heads,n_kv,page,lens", [(8, 2, 64, [70001, 3, 20000]), (16, 1, 16, [9001]),
                                                  (4, 4, 32, [4100, 17, 2049])])
def test_decode_counts_every_key_once(gen, ws, heads, n_kv, page, lens):
    k_pages, v_pages, table, _ = fill_cache(gen, lens, page, n_kv)
    q = torch.zeros(len(lens), heads, P.D, dtype=torch.bfloat16, device="cuda")
    start = ints([n - 1 for n in lens])
    for window in range(-(-max(lens) // P.CODE_WINDOW)):
        coded(k_pages, v_pages, table, page, lens, window)
        out = G.paged_decode(q, start, k_pages, v_pages, table, workspace=ws)
        for b, n in enumerate(lens):
            P.check_counts(out[b:b + 1], window, n - 1, f"sequence {b} of {n} rows")


@pytest.mark.parametrize("heads,n_kv,page,lens,starts", SHARED)
def test_paged_prefill_counts_every_key_once(gen, ws, heads, n_kv, page, lens, starts):
    ends = [s + t for s, t in zip(starts, lens)]
    k_pages, v_pages, table, _ = fill_cache(gen, ends, page, n_kv)
    q = torch.zeros(sum(lens), heads, P.D, dtype=torch.bfloat16, device="cuda")
    cu, start = offsets(lens), ints(starts)
    for window in range(-(-max(ends) // P.CODE_WINDOW)):
        coded(k_pages, v_pages, table, page, ends, window)
        out = G.paged_prefill(q, cu, start, k_pages, v_pages, table, workspace=ws)
        at = 0
        for b, (t, s) in enumerate(zip(lens, starts)):
            P.check_counts(out[at:at + t], window, s, f"sequence {b}: {t} tokens after {s}")
            at += t


# ------------------------------------------------------------------ errors on the device

def test_bad_positions_are_reported_and_skipped(gen, ws):
    k_pages, v_pages, table, rows = fill_cache(gen, [20, 20, 20], 16, 2)
    cap = table.shape[1] * 16
    q, k, v = (P.normal(gen, 3, h, P.D) for h in (8, 2, 2))
    rope = G.rope_table(cap)
    for bad in (-2, cap, 1 << 30):
        start = ints([19, bad, 19])
        out = G.paged_decode(q, start, k_pages, v_pages, table, workspace=ws)
        assert G.device_status(ws, clear=True) == 1
        assert torch.equal(out[1], torch.zeros_like(out[1]))
        check_decode(out[[0, 2]], q[[0, 2]], [rows[0], rows[2]])
        out = G.paged_prefill(q, offsets([1, 1, 1]), start, k_pages, v_pages, table, workspace=ws)
        assert G.device_status(ws, clear=True) == 1
        assert torch.equal(out[1], torch.zeros_like(out[1]))
        before = k_pages.clone()
        G.paged_append(None, k, v, ints([-1, bad, -1]), rope, k_pages, v_pages, table, workspace=ws)
        assert G.device_status(ws, clear=True) == 1
        assert torch.equal(before.view(torch.int16), k_pages.view(torch.int16))
    # a position past the rope table
    G.paged_append(None, k, v, ints([-1, 20, -1]), rope[:20], k_pages, v_pages, table, workspace=ws)
    assert G.device_status(ws, clear=True) == 1


@pytest.mark.parametrize("padding", [16, 17, 18, 300])
def test_an_unused_slot_may_be_longer_than_its_table(gen, ws, padding):
    # a padded batch keeps its padding tokens in one slot without pages
    k_pages, v_pages, table, rows = fill_cache(gen, [16, 0], 16, 2)
    q, k, v = (P.normal(gen, 2 + padding, h, P.D) for h in (8, 2, 2))
    cu, start = offsets([2, padding]), ints([14, -1])
    out = torch.full_like(q, 9.0)
    G.paged_prefill(q, cu, start, k_pages, v_pages, table, out=out, workspace=ws)
    assert G.device_status(ws, clear=True) == 0
    check_prefill(out, q, rows, [2, padding], [14, -1])
    G.paged_append(q, k, v, start, G.rope_table(16), k_pages, v_pages, table, cu_tokens=cu, workspace=ws)
    assert G.device_status(ws, clear=True) == 0
    # a sequence of as many tokens is reported all the same
    G.paged_prefill(q, cu, ints([14, 0 if padding > 16 else 1]), k_pages, v_pages, table, workspace=ws)
    assert G.device_status(ws, clear=True) == 1


@pytest.mark.parametrize("entry", [-1, 1 << 20])
def test_bad_pages_are_reported(gen, ws, entry):
    k_pages, v_pages, table, rows = fill_cache(gen, [40, 40], 16, 2)
    table[0, 1] = entry
    q, k, v = (P.normal(gen, 2, h, P.D) for h in (8, 2, 2))
    start = ints([39, 39])
    out = G.paged_decode(q, start, k_pages, v_pages, table, workspace=ws)
    assert G.device_status(ws, clear=True) == 3
    check_decode(out[1:], q[1:], rows[1:])
    out = G.paged_prefill(q, offsets([1, 1]), start, k_pages, v_pages, table, workspace=ws)
    assert G.device_status(ws, clear=True) == 3
    check_prefill(out[1:], q[1:], rows[1:], [1], [39])
    G.paged_append(None, k, v, ints([20, -1]), G.rope_table(64), k_pages, v_pages, table, workspace=ws)
    assert G.device_status(ws, clear=True) == 3
    # the same workspace serves the next call
    run_decode(gen, ws, 8, 2, 16, [300, 40])


TICKETS = 256   # byte offset in the workspace: of each CTA, parts that arrived and parts that are written


def test_a_wait_that_runs_out_is_reported_and_recovered(gen):
    """Failure injected on the host: the counts of written parts are set so far
    back that the CTA that adds them up waits in vain. The call ends after the
    limit, records GQA_DEV_WAIT_TIMEOUT and touches nothing but its rows; zero-filled,
    the workspace serves the next call."""
    ws = G.make_paged_workspace()
    k_pages, v_pages, table, rows = fill_cache(gen, [8192], 64, 8)
    q = P.normal(gen, 1026, 32, P.D)
    out = torch.full_like(q, 9.0)
    args = (q, offsets([1024]), ints([7168]), k_pages, v_pages, table)
    G.paged_prefill(*args, out=out, workspace=ws)
    check_prefill(out, q, rows, [1024], [7168])
    before = [x.view(torch.int16).clone() for x in (k_pages, v_pages)]
    counts = ws[TICKETS:TICKETS + 152 * 8].view(torch.int32)
    assert int(counts.abs().sum()) == 0
    counts[1::2] = -(1 << 30)
    torch.cuda.synchronize()
    prev = G.set_wait_limit_ns(1_000_000)
    try:
        t0 = time.perf_counter()
        G.paged_prefill(*args, out=out, workspace=ws)
        torch.cuda.synchronize()
        took = time.perf_counter() - t0
    finally:
        G.set_wait_limit_ns(prev)
    assert G.device_status(ws) == 2
    assert took < 0.5, f"a limit of 1 ms ended the call after {took:.2f} s"
    assert (out[1024:] == 9.0).all()
    assert all(torch.equal(x.view(torch.int16), y) for x, y in zip((k_pages, v_pages), before))
    ws.zero_()
    G.paged_prefill(*args, out=out, workspace=ws)
    assert G.device_status(ws) == 0
    check_prefill(out, q, rows, [1024], [7168])


def test_rows_computed_again_are_no_stall(gen, ws):
    """A NaN among the values of an item's last position: its earlier rows are
    computed again one after the other (31 rows over 4,100 keys: 47 ms) while
    the rest of the CTA, with an item to come, waits under a limit of 5 ms."""
    heads, page, prefix, new = 304, 128, 4096, 32     # two items a CTA, none of them shared
    k_pages, v_pages = (P.normal(gen, 2, page, heads, P.D) for _ in range(2))
    table = ints([[0] * (prefix // page) + [1]])      # the prefix is one page over and over
    v_pages[1, new - 1, [0, 7, 303], 5] = math.nan
    q = P.normal(gen, new, heads, P.D)
    out = torch.full_like(q, 9.0)
    prev = G.set_wait_limit_ns(5_000_000)
    try:
        G.paged_prefill(q, offsets([new]), ints([prefix]), k_pages, v_pages, table, out=out, workspace=ws)
        torch.cuda.synchronize()
    finally:
        G.set_wait_limit_ns(prev)
    assert G.device_status(ws) == 0
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[new - 1, [0, 7, 303], 5] = True
    assert torch.isnan(out[hit]).all()
    for g in (0, 1, 7, 100, 152, 160, 303):   # each head by itself
        k, v = (P.read_rows(x[:, :, g:g + 1], table, page, 0, prefix + new) for x in (k_pages, v_pages))
        ref, mean, size = P.attend64(q[:, g:g + 1], k, torch.nan_to_num(v), prefix)
        tol = P.bound(ref, mean, size, prefix + new, P.P_ONE_TERM)
        keep = ~hit[:, g:g + 1]
        P.check(out[:, g:g + 1][keep], ref[keep], tol[keep], f"head {g}")


@pytest.mark.parametrize("heads,short,long", [(104, 4, 73), (79, 10, 37), (57, 3, 21), (51, 2, 33), (123, 4, 60)])
def test_rows_computed_again_before_a_shared_item_are_no_stall(gen, ws, heads, short, long):
    """Two sequences of `short` and `long` key tiles: a range ends one tile into
    the second one's first head, and the last item before that has rows to
    compute again in its second query tile alone. The CTA that adds up the
    shared item's parts must not take that CTA for arrived meanwhile."""
    k_pages, v_pages = (P.normal(gen, 5, 128, heads, P.D) for _ in range(2))
    table = torch.zeros(2, long, dtype=torch.int32, device="cuda")   # prefixes are page 0 over and over
    table[0, short - 2:short], table[1, long - 2:] = ints([1, 2]), ints([3, 4])
    v_pages[2, 100, heads - 1, 5] = math.nan
    q = P.normal(gen, 512, heads, P.D)
    starts = [128 * (short - 2), 128 * (long - 2)]
    out = torch.full_like(q, 9.0)
    prev = G.set_wait_limit_ns(500_000)
    try:
        for _ in range(10):
            G.paged_prefill(q, offsets([256, 256]), ints(starts), k_pages, v_pages, table, out=out, workspace=ws)
            assert G.device_status(ws) == 0
    finally:
        G.set_wait_limit_ns(prev)
        ws.zero_()
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[228:256, heads - 1, 5] = True
    assert torch.isnan(out[hit]).all()
    for b, s in enumerate(starts):
        rows = slice(256 * b, 256 * b + 256)
        for g in (0, 1, heads // 2, heads - 1):
            k, v = (P.read_rows(x[:, :, g:g + 1], table, 128, b, s + 256) for x in (k_pages, v_pages))
            ref, mean, size = P.attend64(q[rows, g:g + 1], k, torch.nan_to_num(v), s)
            tol = P.bound(ref, mean, size, s + 256, P.P_ONE_TERM)
            keep = ~hit[rows, g:g + 1]
            P.check(out[rows, g:g + 1][keep], ref[keep], tol[keep], f"sequence {b}, head {g}")


# ------------------------------------------------------------------ as a server uses them

def test_prompt_chunks_and_decode_steps_together(gen, ws):
    """Prompts in, chunk by chunk, then decode steps with one slot unused: every
    output against the 64-bit attention over everything appended so far."""
    heads, n_kv, page, B = 8, 2, 16, 4
    plan = [[37, 5, 0, 64], [20, 100, 1, 3], [1, 1, 1, 1], [1, 1, 1, 1], [1, 1, 0, 1]]
    total = [sum(x) for x in zip(*plan)]
    k_pages, v_pages, table = P.pages_of(gen, total, page, n_kv, fill=math.nan)
    rope = G.rope_table(256)
    start = [0] * B
    seen = [(torch.empty(0, n_kv, P.D, dtype=torch.bfloat16, device="cuda"),) * 2 for _ in range(B)]
    for lens in plan:
        step = max(lens) == 1
        if step:   # a padded batch: every sequence has a row, an unused slot start -1
            rows_of, starts = [1] * B, [s if t else -1 for s, t in zip(start, lens)]
        else:
            rows_of, starts = lens, start
        n = sum(rows_of)
        qkv = P.normal(gen, n, heads + 2 * n_kv, P.D)
        q, k, v = qkv[:, :heads], qkv[:, heads:heads + n_kv], qkv[:, heads + n_kv:]
        cu, sp = offsets(rows_of), ints(starts)
        rq = G.paged_append(q, k, v, sp, rope, k_pages, v_pages, table, cu_tokens=None if step else cu, workspace=ws)
        if step:
            out = G.paged_decode(rq, sp, k_pages, v_pages, table, workspace=ws)
        else:
            out = G.paged_prefill(rq, cu, sp, k_pages, v_pages, table, workspace=ws)
        at = 0
        for b, (t, s) in enumerate(zip(rows_of, starts)):
            r = slice(at, at + t)
            at += t
            if s < 0:
                assert torch.equal(out[r], torch.zeros_like(out[r]))
                continue
            if t == 0:
                continue
            P.check_rotated(rq[r], q[r], rope[s:s + t], "rotated q")
            p, rr = P.slots(table, page, b, s, t)
            seen[b] = (torch.cat([seen[b][0], k_pages[p, rr]]), torch.cat([seen[b][1], v[r]]))
            P.check_rotated(seen[b][0][s:], k[r], rope[s:s + t], "appended k")
            ref, mean, size = P.attend64(rq[r], *seen[b], s)
            P.check(out[r], ref, P.bound(ref, mean, size, s + t, P.P_TWO_TERMS if step else P.P_ONE_TERM),
                    f"sequence {b}, {t} tokens after {s}")
        start = [s + t for s, t in zip(start, lens)]
    assert G.device_status(ws) == 0


def test_paged_step_equals_the_dense_block():
    """The block's decode step and prefill with W_O = I against projections by
    matmul and the paged operators, on the same weights and prefix, at the
    block's own bar."""
    import gqa_inputs as I
    from tests import harness as H
    c = H.make_case(2, 33, [50, 50], 96, weights=I.draw_weights(seed=0))
    d = c.dev
    rope = H.rope_for(c)
    eye = torch.eye(4096, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    k_pages, v_pages, table = P.pages_of(gen, [96, 96], 16, 8)
    for b in range(2):
        P.write_rows(k_pages, table, 16, b, 0, d["cache_k"][b, :50])
        P.write_rows(v_pages, table, 16, b, 0, d["cache_v"][b, :50])
    ws = G.make_paged_workspace()
    w = torch.cat([d["wq"], d["wk"], d["wv"]])

    def paged(x, start):
        t = x.shape[1]
        qkv = (x.reshape(-1, 4096) @ w.T).view(-1, 48, 128)
        cu, sp = offsets([t, t]), ints([start, start])
        q = G.paged_append(qkv[:, :32], qkv[:, 32:40], qkv[:, 40:], sp, rope, k_pages, v_pages, table, cu_tokens=cu,
                           workspace=ws)
        o = G.paged_decode(q, sp, k_pages, v_pages, table, workspace=ws) if t == 1 else \
            G.paged_prefill(q, cu, sp, k_pages, v_pages, table, workspace=ws)
        return o.view(2, t, 4096)

    x = d["x"]
    for part, start in ((x, 50), (x[:, :1].contiguous(), 83)):
        dense = G.block_forward(part, start, d["wq"], d["wk"], d["wv"], eye, rope, d["cache_k"], d["cache_v"])
        got = paged(part, start)
        assert H.rel_l2(H.f64(got), H.f64(dense)) <= H.REL_L2_TOL
    for b in range(2):
        rows = P.read_rows(k_pages, table, 16, b, 84)
        assert H.rel_l2(H.f64(rows), H.f64(d["cache_k"][b, :84])) <= H.REL_L2_TOL
    assert G.device_status(ws) == 0


def test_a_captured_step_replays_with_other_lengths(gen):
    heads, n_kv, page, B = 8, 2, 16, 3
    ws = G.make_paged_workspace()
    k_pages, v_pages, table, rows = fill_cache(gen, [600, 600, 600], page, n_kv, junk=0.0)
    rope = G.rope_table(600)
    qkv = P.normal(gen, B, heads + 2 * n_kv, P.D)
    start = ints([5, 5, 5])
    q_out, out = (torch.empty(B, heads, P.D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pre = torch.empty_like(out)
    cu = offsets([1, 1, 1])

    def step():
        G.paged_append(qkv[:, :heads], qkv[:, heads:heads + n_kv], qkv[:, heads + n_kv:], start, rope, k_pages,
                       v_pages, table, q_out=q_out, workspace=ws)
        G.paged_decode(q_out, start, k_pages, v_pages, table, out=out, workspace=ws)
        G.paged_prefill(q_out, cu, start, k_pages, v_pages, table, out=pre, workspace=ws)

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
        want_ws = G.make_paged_workspace()
        graphs[i % 2].replay()
        o, p, q = out.clone(), pre.clone(), q_out.clone()
        assert torch.equal(o, G.paged_decode(q, start, k_pages, v_pages, table, workspace=want_ws))
        for b, s in enumerate(lens):
            if s < 0:
                assert torch.equal(o[b], torch.zeros_like(o[b])) and torch.equal(p[b], torch.zeros_like(p[b]))
                continue
            kk, vv = P.read_rows(k_pages, table, page, b, s + 1), P.read_rows(v_pages, table, page, b, s + 1)
            ref, mean, size = P.attend64(q[b:b + 1], kk, vv, s)
            P.check(o[b:b + 1], ref, P.bound(ref, mean, size, s + 1, P.P_TWO_TERMS), f"decode of {s}")
            P.check(p[b:b + 1], ref, P.bound(ref, mean, size, s + 1, P.P_ONE_TERM), f"prefill of {s}")
    assert G.device_status(ws) == 0


def test_a_captured_prefill_replays_between_shared_and_whole_items(gen):
    heads, n_kv, page = 8, 2, 64
    ws = G.make_paged_workspace()
    k_pages, v_pages, table, rows = fill_cache(gen, [9100, 9100], page, n_kv)
    q = P.normal(gen, 120, heads, P.D)
    cu, start = offsets([100, 20]), ints([0, 0])
    out = torch.empty_like(q)
    G.paged_prefill(q, cu, start, k_pages, v_pages, table, out=out, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        G.paged_prefill(q, cu, start, k_pages, v_pages, table, out=out, workspace=ws)
    for lens, starts in (([100, 20], [9000, 9080]), ([100, 20], [0, 3]), ([3, 60], [8000, -1]), ([1, 119], [9099, 500])):
        cu.copy_(offsets(lens))
        start.copy_(ints(starts))
        out.fill_(9.0)
        g.replay()
        ends = [(k[:s + t], v[:s + t]) for (k, v), t, s in zip(rows, lens, starts)]
        check_prefill(out, q, ends, lens, starts)
        assert (out[sum(lens):] == 9.0).all()
    assert G.device_status(ws) == 0


def test_sequences_that_share_pages(gen, ws):
    # one prompt's pages under two sequences, each with a last page of its own
    k_pages, v_pages, table, rows = fill_cache(gen, [3000, 3000], 64, 2)
    table[1, :40] = table[0, :40]
    for x, other in zip(rows[1], rows[0]):
        x[:40 * 64] = other[:40 * 64]
    q = P.normal(gen, 2, 8, P.D)
    check_decode(G.paged_decode(q, ints([2999, 2999]), k_pages, v_pages, table, workspace=ws), q, rows)
    q = P.normal(gen, 50, 8, P.D)
    out = G.paged_prefill(q, offsets([30, 20]), ints([2970, 2980]), k_pages, v_pages, table, workspace=ws)
    check_prefill(out, q, rows, [30, 20], [2970, 2980])
    assert G.device_status(ws) == 0


def test_most_sequences_and_most_heads_per_kv_head(gen, ws):
    lens = [(31 * b) % 40 for b in range(2048)]
    run_decode(gen, ws, 16, 1, 16, lens)
    run_paged_prefill(gen, ws, 16, 1, 16, [n % 2 for n in lens], [n // 2 for n in lens])


def test_calls_on_two_streams_with_their_own_workspaces(gen):
    k_pages, v_pages, table, rows = fill_cache(gen, [3000, 40, 700], 32, 4)
    start = ints([2999, 39, 699])
    qs = [P.normal(gen, 3, 16, P.D) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [G.make_paged_workspace() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i in range(2):
            outs[i].append(G.paged_decode(qs[i], start, k_pages, v_pages, table, workspace=spaces[i],
                                          stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        check_decode(outs[i][0], qs[i], rows)
        assert all(torch.equal(o, outs[i][0]) for o in outs[i])
        assert G.device_status(spaces[i]) == 0


def test_defaults_on_a_side_stream(gen):
    # no out, no workspace: both belong to the stream of the call
    k_pages, v_pages, table, rows = fill_cache(gen, [100], 32, 4)
    q = P.normal(gen, 1, 16, P.D)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = G.paged_decode(q, ints([99]), k_pages, v_pages, table, stream=side)
    side.synchronize()
    check_decode(out, q, rows)


def test_errors_of_calls_without_a_workspace_can_be_read(gen):
    k_pages, v_pages, table, rows = fill_cache(gen, [40, 40], 16, 2)
    q, start = P.normal(gen, 2, 8, P.D), ints([39, 39])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (None, side):
        mine, other = (G.default_paged_workspace(stream=s) for s in (stream, side if stream is None else None))
        assert mine is G.default_paged_workspace("cuda", stream) and mine is not other
        bad = table.clone()
        bad[0, 1] = 1 << 20
        torch.cuda.synchronize()
        out = G.paged_decode(q, start, k_pages, v_pages, bad, stream=stream)
        assert G.device_status(mine) == 3 and G.device_status(other) == 0
        check_decode(out[1:], q[1:], rows[1:])
        assert G.device_status(mine, clear=True) == 3
        G.paged_prefill(q, offsets([1, 1]), ints([39, 100]), k_pages, v_pages, table, stream=stream)
        assert G.device_status(mine, clear=True) == 1
        G.paged_append(None, q[:, :2], q[:, 2:4].contiguous(), ints([-5, -1]), G.rope_table(48), k_pages.clone(),
                       v_pages.clone(), table, stream=stream)
        assert G.device_status(mine, clear=True) == 1
        check_decode(G.paged_decode(q, start, k_pages, v_pages, table, stream=stream), q, rows)
        assert G.device_status(mine) == 0
        # none is made call by call
        at = torch.cuda.memory_allocated()
        for _ in range(3):
            G.packed_prefill(q, q[:, :2], q[:, 2:4], offsets([2]), stream=stream)
        torch.cuda.synchronize()
        assert torch.cuda.memory_allocated() == at


def test_more_streams_than_kept_workspaces(gen):
    k_pages, v_pages, table, rows = fill_cache(gen, [3000], 64, 2)
    q, start = P.normal(gen, 1, 8, P.D), ints([2999])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(11)]
    outs = [G.paged_decode(q, start, k_pages, v_pages, table, stream=s) for _ in range(3) for s in streams]
    torch.cuda.synchronize()
    for o in outs:
        check_decode(o, q, rows)


def test_a_captured_call_without_a_workspace_has_its_own(gen):
    k_pages, v_pages, table, rows = fill_cache(gen, [3000, 40], 64, 2)
    q, start = P.normal(gen, 2, 8, P.D), ints([2999, 39])
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        G.paged_decode(q, start, k_pages, v_pages, table, out=out)   # this stream's workspace is there
        kept = G.default_paged_workspace()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        G.paged_decode(q, start, k_pages, v_pages, table, out=out)
    assert G.default_paged_workspace(stream=side) is kept
    table[0, 0] = -1
    for _ in range(3):
        g.replay()
    assert G.device_status(kept) == 0    # the graph's errors are not this workspace's
    check_decode(out[1:], q[1:], rows[1:])


def test_launch_counts_and_empty_calls(gen, ws):
    k_pages, v_pages, table, rows = fill_cache(gen, [40], 16, 2)
    q = P.normal(gen, 1, 8, P.D)
    G.paged_decode(q, ints([39]), k_pages, v_pages, table, workspace=ws)
    assert G.last_launch_count() == 1
    none = q[:0]
    assert G.paged_prefill(none, offsets([0]), ints([39]), k_pages, v_pages, table, workspace=ws).shape == (0, 8, P.D)
    assert G.packed_prefill(none, none[:, :2], none[:, :2], offsets([0]), workspace=ws).shape == (0, 8, P.D)
    assert G.paged_append(None, none[:, :2], none[:, :2], ints([39]), G.rope_table(64), k_pages, v_pages, table,
                          cu_tokens=offsets([0]), workspace=ws) is None
    assert G.paged_decode(none, ints([]), k_pages, v_pages, table[:0], workspace=ws).shape == (0, 8, P.D)
