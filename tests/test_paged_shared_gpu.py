"""Decode attention of groups with shared rows against 64-bit references, at the
sizes, masks and layouts where it can go wrong."""
import math
import time

import pytest
import torch

import grouped_query_attention_gemv_gb300 as G
from tests import paged as P
from tests.test_paged_gpu import LAYOUTS, fill_cache, ints

pytestmark = pytest.mark.gpu

LEAST = 200_000   # saving as many cache rows x KV heads, a batch shares


@pytest.fixture(scope="module")
def ws():
    return G.make_paged_workspace()


@pytest.fixture
def gen():
    return torch.Generator(device="cuda").manual_seed(5)


class Batch:
    """groups: (prefix rows, start positions of its members); before, after:
    start positions of sequences in no group. A member's rows begin with its
    group's; whole pages of a prefix are one copy, or each has its own (copies)."""

    def __init__(self, gen, n_kv, page, groups, before=(), after=(), order="nhd", copies=False, junk=math.nan):
        self.page, self.n_kv = page, n_kv
        self.prefix = [p for p, _ in groups]
        self.starts = list(before) + [s for _, m in groups for s in m] + list(after)
        self.cu = [len(before)]
        for _, m in groups:
            self.cu.append(self.cu[-1] + len(m))
        ends = [s + 1 for s in self.starts]
        self.k_pages, self.v_pages, self.table = P.pages_of(gen, ends, page, n_kv, order=order, fill=junk)
        self.rows, self.shares = [None] * len(ends), [False] * len(ends)
        group_of = [-1] * len(before) + [g for g, (_, m) in enumerate(groups) for _ in m] + [-1] * len(after)
        common = [[P.normal(gen, p, n_kv, P.D) for _ in range(2)] for p in self.prefix]
        lead = {}
        for b, (n, g) in enumerate(zip(ends, group_of)):
            kv = [P.normal(gen, n, n_kv, P.D) for _ in range(2)]
            if g >= 0:
                p = self.prefix[g]
                for x, c in zip(kv, common[g]):
                    x[:p] = c[:n]
                if not copies and g in lead:
                    full = min(p, n) // page
                    self.table[b, :full] = self.table[lead[g], :full]
                elif n >= p:
                    lead.setdefault(g, b)
                self.shares[b] = n >= p > 0 and sum(s + 1 >= p for s in groups[g][1]) > 1
            self.rows[b] = tuple(kv)
            if n:
                P.write_rows(self.k_pages, self.table, page, b, 0, kv[0])
                P.write_rows(self.v_pages, self.table, page, b, 0, kv[1])
        saved = sum((sum(s + 1 >= p for s in m) - 1) * p for p, m in groups if p > 0 and any(s + 1 >= p for s in m))
        self.pays = saved * n_kv >= LEAST

    def args(self):
        return ints(self.starts), ints(self.cu), ints(self.prefix), self.k_pages, self.v_pages, self.table

    def check(self, out, q, scale=P.D ** -0.5, skip=(), shared=True):
        for b, (k, v) in enumerate(self.rows):
            n = k.shape[0]
            if b in skip:
                continue
            if n == 0:
                assert torch.equal(out[b], torch.zeros_like(out[b])), f"sequence {b} sees nothing"
                continue
            ref, mean, size = P.attend64(q[b:b + 1], k, v, n - 1, scale)
            one = shared and self.pays and self.shares[b]
            P.check(out[b:b + 1], ref, P.bound(ref, mean, size, n, P.P_ONE_TERM if one else P.P_TWO_TERMS),
                    f"sequence {b} of {n} rows")


def run(gen, ws, heads, n_kv, page, groups, pays=True, scale=P.D ** -0.5, q_scale=1.5, **kw):
    x = Batch(gen, n_kv, page, groups, **kw)
    assert x.pays == pays, "the case does not test what it says"
    q = P.normal(gen, len(x.starts), heads, P.D, scale=q_scale)
    out = torch.full_like(q, math.nan)
    assert G.paged_decode_shared(q, *x.args(), scale=scale, out=out, workspace=ws) is out
    assert G.device_status(ws) == 0
    x.check(out, q, scale)
    assert torch.equal(out, G.paged_decode_shared(q, *x.args(), scale=scale, workspace=ws))
    return x, q, out


def enough(n_kv, members):
    """A prefix for which that many members save enough."""
    return -(-LEAST // (n_kv * (members - 1)))


# beside a group that pays for sharing: prefixes at tile and page edges, members without rows of their own, with
# one, on a chunk's edge; a group of one, one without a prefix, members that see a part of it, unused slots
def edges(n_kv, members=33):
    p = enough(n_kv, members) // 16 * 16 + 27
    return [(1, [0, 5, 1]), (127, [126, 127, 300]), (0, [3, 40]), (128, [127, 128, 143, 144]),
            (p, [p - 1 + (7 * i) % 50 for i in range(members)]), (129, [128, 128]), (500, [700]), (64, [63, 20, -1, 64, 90]),
            (33, [32]), (16, [15, 16, 31, 32, 33]), (4000, [10, -1, 3999])]


@pytest.mark.parametrize("heads,n_kv", LAYOUTS + [(16, 1), (9, 1), (24, 2)])
@pytest.mark.parametrize("page,order", [(16, "nhd"), (64, "hnd")])
def test_layouts_and_edges(gen, ws, heads, n_kv, page, order):
    run(gen, ws, heads, n_kv, page, edges(n_kv), before=[40, -1, 0], after=[200], order=order)


@pytest.mark.parametrize("page", [16, 32, 256, 4096])
@pytest.mark.parametrize("copies", [False, True])
def test_page_sizes_and_copies(gen, ws, page, copies):
    run(gen, ws, 8, 2, page, edges(2), copies=copies, junk=math.inf)


@pytest.mark.parametrize("members", [2, 3, 31, 32, 33, 63, 64, 65, 130, 200])
def test_members(gen, ws, members):
    p = enough(8, members)
    run(gen, ws, 32, 8, 64, [(p, [p - 1 + (3 * i) % 5 for i in range(members)])])


@pytest.mark.parametrize("p", [20_003, 65_536])
def test_long_prefix(gen, ws, p):
    run(gen, ws, 8, 2, 128, [(p, [p + 3000 * i for i in range(8)])])


def test_many_groups(gen, ws):
    run(gen, ws, 8, 2, 16, [(270 + 3 * (i % 70), [280 + 3 * (i % 70) + j for j in range(3)]) for i in range(200)])


def test_most_groups(gen, ws):
    run(gen, ws, 4, 1, 16, [(200 + i % 7, [206 + i % 5, 207 + i % 3]) for i in range(1024)])


def test_more_groups_than_are_looked_at(gen, ws):
    run(gen, ws, 1, 1, 16, [(100, [107])] * 1025, pays=False)


def test_scale_strided_queries_and_sharp_scores(gen, ws):
    run(gen, ws, 8, 2, 16, [(3500, [3500 + 9 * i for i in range(30)])], q_scale=60.0)
    x = Batch(gen, 2, 16, [(3500, [3500 + 9 * i for i in range(30)])])
    qkv = P.normal(gen, 30, 12, P.D)
    out = G.paged_decode_shared(qkv[:, :8], *x.args(), scale=0.3, workspace=ws)
    x.check(out, qkv[:, :8], 0.3)


def test_little_to_share_is_the_plain_decode(gen, ws):
    x, q, out = run(gen, ws, 8, 2, 16, [(500, [510, 520, 530]), (33, [40])], pays=False)
    assert G.last_launch_count() == 1
    assert torch.equal(out, G.paged_decode(q, ints(x.starts), x.k_pages, x.v_pages, x.table, workspace=ws))
    # a wide table, of which little is used: the plan decides
    wide = torch.full((4, 4096), -9, dtype=torch.int32, device="cuda")
    wide[:, :x.table.shape[1]] = x.table
    args = x.args()[:-1]
    out = G.paged_decode_shared(q, *args, wide, workspace=ws)
    assert G.last_launch_count() == 2 and G.device_status(ws) == 0
    x.check(out, q)


def test_more_query_rows_than_the_workspace_holds(gen, ws):
    x = Batch(gen, 4, 16, [(100, [100 + i % 9 for i in range(520)])])
    assert x.pays
    q = P.normal(gen, 520, 64, P.D)
    out = G.paged_decode_shared(q, *x.args(), workspace=ws)
    assert G.last_launch_count() == 1
    assert torch.equal(out, G.paged_decode(q, ints(x.starts), x.k_pages, x.v_pages, x.table, workspace=ws))


def test_close_in_the_mean(gen, ws):
    x = Batch(gen, 8, 64, [(9001, [9001 + 37 * i for i in range(16)]), (300, [301, 400])])
    q = P.normal(gen, 18, 32, P.D, scale=1.5)
    out = G.paged_decode_shared(q, *x.args(), workspace=ws)
    for b, (k, v) in enumerate(x.rows):
        P.check_l2(out[b:b + 1], P.attend64(q[b:b + 1], k, v, k.shape[0] - 1)[0], f"sequence {b}")


@pytest.mark.parametrize("heads,n_kv,page,groups", [
    (8, 2, 64, [(9500, [9500 + 700 * i for i in range(12)])]),
    (32, 8, 16, [(3000, [2999 + 11 * i for i in range(10)]), (129, [128, 140, 300])]),
    (16, 1, 32, [(3450, [3449 + i for i in range(60)])])])
def test_every_key_counts_once(gen, ws, heads, n_kv, page, groups):
    x = Batch(gen, n_kv, page, groups)
    assert x.pays
    q = torch.zeros(len(x.starts), heads, P.D, dtype=torch.bfloat16, device="cuda")
    for window in range(-(-(max(x.starts) + 1) // P.CODE_WINDOW)):
        for b, s in enumerate(x.starts):
            P.write_rows(x.v_pages, x.table, page, b, 0,
                         P.coded_values(s + 1, window, "cuda")[:, None].expand(-1, n_kv, -1))
        out = G.paged_decode_shared(q, *x.args(), workspace=ws)
        for b, s in enumerate(x.starts):
            P.check_counts(out[b:b + 1], window, s, f"sequence {b}")
    assert G.device_status(ws) == 0


@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_what_is_not_finite_stays_with_who_sees_it(gen, ws, value):
    p = 6000
    x = Batch(gen, 2, 32, [(p, [p - 1 + 5 * i for i in range(18)]), (100, [120, 130])], copies=False)
    assert x.pays
    q = P.normal(gen, 20, 8, P.D)
    hit = torch.zeros(20, 8, P.D, dtype=torch.bool, device="cuda")
    page, row = P.slots(x.table, 32, 0, 1234, 1)     # of the prefix
    x.v_pages[page, row, 0, 5] = value
    hit[:18, :4, 5] = True
    page, row = P.slots(x.table, 32, 7, p + 3, 1)    # of one member's own rows
    x.v_pages[page, row, 1, 9] = value
    hit[7, 4:, 9] = True
    page, row = P.slots(x.table, 32, 18, 110, 1)     # of a member of the other group, behind its prefix
    x.k_pages[page, row, 1, 0] = math.nan
    hit[18, 4:] = True
    out = G.paged_decode_shared(q, *x.args(), workspace=ws)
    assert G.device_status(ws) == 0
    assert (~torch.isfinite(out[hit])).all()
    assert (out[:18, :4, 5] == value).all() or math.isnan(value)
    for b, (k, v) in enumerate(x.rows):
        ref, mean, size = P.attend64(q[b:b + 1], k, v, k.shape[0] - 1)
        tol = P.bound(ref, mean, size, k.shape[0], P.P_ONE_TERM)
        keep = ~hit[b:b + 1]
        P.check(out[b:b + 1][keep], ref[keep], tol[keep], f"sequence {b}")


def test_a_bad_member_leaves_the_others_alone(gen, ws):
    p = 6000
    x = Batch(gen, 2, 32, [(p, [p + 5 * i for i in range(20)])])
    assert x.pays
    cap = x.table.shape[1] * 32
    q = P.normal(gen, 20, 8, P.D)
    q[4, 2, 7], q[19, 1, 0] = math.nan, math.inf
    start, *rest = x.args()
    for bad in (-2, cap, 1 << 30):
        start[5] = bad
        out = G.paged_decode_shared(q, start, *rest, workspace=ws)
        assert G.device_status(ws, clear=True) == 1
        assert torch.equal(out[5], torch.zeros_like(out[5]))
        assert torch.isnan(out[4, 2]).all() and torch.isnan(out[19, 1]).all()
        x.check(out, q, skip=(4, 5, 19))
        assert torch.isfinite(out[4, [0, 1, 3, 4, 5, 6, 7]]).all()


@pytest.mark.parametrize("cu", [[0, 10, 5, 20], [0, 5, 10, 21], [-1, 5, 10, 20], [12, 11, 15, 20]])
def test_bad_groups_are_reported_and_not_shared(gen, ws, cu):
    x = Batch(gen, 2, 32, [(5400, [5400 + i for i in range(20)])])
    assert x.pays
    q = P.normal(gen, 20, 8, P.D)
    args = (ints(x.starts), ints(cu), ints([5400] * 3), x.k_pages, x.v_pages, x.table)
    out = G.paged_decode_shared(q, *args, workspace=ws)
    assert G.device_status(ws, clear=True) == 1
    x.check(out, q, shared=False)   # to the bits that the decode attention keeps


@pytest.mark.parametrize("prefix", [-5, -(1 << 31), (1 << 31) - 1, 1 << 30])
def test_a_prefix_out_of_range_is_not_shared(gen, ws, prefix):
    x = Batch(gen, 2, 32, [(5400, [5400 + i for i in range(20)]), (70, [80, 90])])
    assert x.pays
    q = P.normal(gen, 22, 8, P.D)
    start, cu, p, *rest = x.args()
    p[1] = prefix
    out = G.paged_decode_shared(q, start, cu, p, *rest, workspace=ws)
    assert G.device_status(ws) == 0
    x.check(out, q)


@pytest.mark.parametrize("entry", [-1, 1 << 20])
def test_bad_pages_are_reported(gen, ws, entry):
    x = Batch(gen, 2, 32, [(5400, [5400 + i for i in range(20)]), (2000, [2100, 2300, 2500])])
    assert x.pays
    x.table[:20, 40] = entry
    q = P.normal(gen, 23, 8, P.D)
    out = G.paged_decode_shared(q, *x.args(), workspace=ws)
    assert G.device_status(ws, clear=True) == 3
    x.check(out, q, skip=range(20))
    # the same workspace serves the next call
    run(gen, ws, 8, 2, 16, edges(2))


def test_waits_that_run_out_are_reported_and_recovered(gen):
    """A limit no wait keeps: the call ends, records GQA_DEV_WAIT_TIMEOUT and
    writes nothing but its rows; zero-filled, the workspace serves the next call."""
    ws = G.make_paged_workspace()
    x = Batch(gen, 8, 64, [(8000, [8000 + 30 * i for i in range(16)])])
    q = P.normal(gen, 16, 32, P.D)
    before = [t.view(torch.int16).clone() for t in (x.k_pages, x.v_pages)]
    guard = torch.full((18, 32, P.D), 9.0, dtype=torch.bfloat16, device="cuda")
    prev = G.set_wait_limit_ns(1)
    try:
        t0 = time.perf_counter()
        G.paged_decode_shared(q, *x.args(), out=guard[1:17], workspace=ws)
        torch.cuda.synchronize()
        took = time.perf_counter() - t0
    finally:
        G.set_wait_limit_ns(prev)
    assert G.device_status(ws, clear=True) in (0, 2) and took < 0.5
    assert (guard[[0, 17]] == 9.0).all()
    assert all(torch.equal(t.view(torch.int16), y) for t, y in zip((x.k_pages, x.v_pages), before))
    ws.zero_()
    out = G.paged_decode_shared(q, *x.args(), workspace=ws)
    assert G.device_status(ws) == 0
    x.check(out, q)


def test_a_captured_step_replays_with_other_groups(gen):
    ws = G.make_paged_workspace()
    heads, n_kv, page, B = 16, 4, 16, 24
    k_pages, v_pages, table, rows = fill_cache(gen, [6000] * B, page, n_kv)
    # all prefixes up to 4,096 rows are sequence 0's
    table[:, :256] = table[:1, :256]
    q = P.normal(gen, B, heads, P.D)
    start, cu, prefix = ints([4100] * B), ints([0, B, B, B]), ints([4096, 0, 0])
    out = torch.empty_like(q)
    args = (q, start, cu, prefix, k_pages, v_pages, table)
    G.paged_decode_shared(*args, out=out, workspace=ws)
    graphs = []
    for _ in range(2):   # two graphs over one workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            G.paged_decode_shared(*args, out=out, workspace=ws)
        graphs.append(g)
    rows0 = rows[0]
    for i, (starts, groups, p) in enumerate((
            ([4095 + 80 * b for b in range(B)], [0, B, B, B], [4096, 0, 0]),
            ([(331 * b) % 5900 for b in range(B)], [0, 8, 16, 24], [2500, 0, 17]),
            ([4096 + b if b % 3 else -1 for b in range(B)], [3, 10, 10, 22], [4096, 77, 4001]),
            ([b for b in range(B)], [0, 8, 16, 24], [1, 2, 3]),
            ([5999] * B, [0, 1, 2, 24], [4000, 4000, 4096]))):
        for t, x in ((start, starts), (cu, groups), (prefix, p)):
            t.copy_(ints(x))
        out.fill_(9.0)
        graphs[i % 2].replay()
        o = out.clone()
        for b, s in enumerate(starts):
            if s < 0:
                assert torch.equal(o[b], torch.zeros_like(o[b]))
                continue
            k, v = (torch.cat([x0[:4096], x[4096:]])[:s + 1] for x0, x in zip(rows0, rows[b]))
            ref, mean, size = P.attend64(q[b:b + 1], k, v, s)
            P.check(o[b:b + 1], ref, P.bound(ref, mean, size, s + 1, P.P_ONE_TERM), f"sequence {b} at {s}")
    assert G.device_status(ws) == 0


def test_between_other_calls_on_one_workspace(gen, ws):
    x = Batch(gen, 4, 32, [(3000, [3000 + 40 * i for i in range(20)])])
    assert x.pays
    q = P.normal(gen, 20, 16, P.D)
    args = x.args()
    want = G.paged_decode_shared(q, *args, workspace=G.make_paged_workspace())
    x.check(want, q)
    plain = G.paged_decode(q, args[0], *args[3:], workspace=G.make_paged_workspace())
    cu = ints(list(range(21)))
    pre = G.paged_prefill(q, cu, args[0], *args[3:], workspace=G.make_paged_workspace())
    for _ in range(10):
        assert torch.equal(G.paged_decode(q, args[0], *args[3:], workspace=ws), plain)
        assert torch.equal(G.paged_decode_shared(q, *args, workspace=ws), want)
        assert torch.equal(G.paged_prefill(q, cu, args[0], *args[3:], workspace=ws), pre)
        assert torch.equal(G.paged_decode_shared(q, *args, workspace=ws), want)
    assert G.device_status(ws) == 0


def test_calls_on_two_streams_and_without_workspaces(gen):
    x = Batch(gen, 4, 32, [(3000, [3000 + 40 * i for i in range(20)])])
    assert x.pays
    qs = [P.normal(gen, 20, 16, P.D) for _ in range(2)]
    args = x.args()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(10):
        for i in range(2):
            outs[i].append(G.paged_decode_shared(qs[i], *args, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        x.check(outs[i][0], qs[i])
        assert all(torch.equal(o, outs[i][0]) for o in outs[i])
        assert G.device_status(G.default_paged_workspace(stream=streams[i])) == 0


def test_no_sequences_and_no_groups(gen, ws):
    x = Batch(gen, 2, 16, [], before=[40, 3])
    q = P.normal(gen, 2, 8, P.D)
    x.check(G.paged_decode_shared(q, *x.args(), workspace=ws), q)
    start, cu, prefix, *rest = x.args()
    none = G.paged_decode_shared(q[:0], start[:0], ints([0, 0]), ints([7]), *rest[:2], rest[2][:0], workspace=ws)
    assert none.shape == (0, 8, P.D)
