"""The paged operators' refusals (argument checks of the binding and of the C
ABI; nothing is launched) and the arithmetic of their work split, on the CPU."""
import ctypes
import random

import pytest
import torch

import grouped_query_attention_gemv_gb300 as G
from grouped_query_attention_gemv_gb300 import build as gbuild

FAKE = 1 << 20   # aligned, never dereferenced
WS = 64 << 20


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return G.lib()


class Pages(ctypes.Structure):
    """gqa_pages of include/gqa.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_stride", ctypes.c_longlong),
                ("row_stride", ctypes.c_longlong), ("head_stride", ctypes.c_longlong),
                ("block_table", ctypes.c_void_p), ("num_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("table_stride", ctypes.c_int), ("columns", ctypes.c_int)]


def pages(**kw):
    a = dict(k=FAKE, v=FAKE, page_stride=16 * 8 * 128, row_stride=8 * 128, head_stride=128, block_table=FAKE,
             num_pages=4, page_size=16, n_kv_heads=8, table_stride=4, columns=4)
    a.update(kw)
    p = Pages(**a)
    return ctypes.addressof(p), p   # the structure is kept by the caller


def append(lib, p=None, **kw):
    a = dict(q=FAKE, qs=4096, k=FAKE, ks=1024, v=FAKE, vs=1024, N=5, heads=32, cu=FAKE, B=2, start=FAKE, rope=FAKE,
             rows=64, out=FAKE * 2, ws=FAKE, n=WS)
    a.update(kw)
    g, keep = pages() if p is None else p
    return lib.gqa_paged_append(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["N"], a["heads"], a["cu"], a["B"],
                                a["start"], a["rope"], a["rows"], g, a["out"], a["ws"], a["n"], None)


def decode(lib, p=None, **kw):
    a = dict(q=FAKE, qs=4096, B=2, heads=32, start=FAKE, scale=0.1, out=FAKE, ws=FAKE, n=WS)
    a.update(kw)
    g, keep = pages() if p is None else p
    return lib.gqa_paged_decode(a["q"], a["qs"], a["B"], a["heads"], a["start"], g, a["scale"], a["out"], a["ws"],
                                a["n"], None)


def prefill(lib, p=None, **kw):
    a = dict(q=FAKE, qs=4096, N=5, heads=32, cu=FAKE, B=2, start=FAKE, scale=0.1, out=FAKE, ws=FAKE, n=WS)
    a.update(kw)
    g, keep = pages() if p is None else p
    return lib.gqa_paged_prefill(a["q"], a["qs"], a["N"], a["heads"], a["cu"], a["B"], a["start"], g, a["scale"],
                                 a["out"], a["ws"], a["n"], None)


def packed(lib, **kw):
    a = dict(q=FAKE, qs=4096, k=FAKE, ks=1024, v=FAKE, vs=1024, N=5, heads=32, kv=8, cu=FAKE, B=2, scale=0.1, out=FAKE,
             ws=FAKE, n=WS)
    a.update(kw)
    return lib.gqa_packed_prefill(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["N"], a["heads"], a["kv"],
                                  a["cu"], a["B"], a["scale"], a["out"], a["ws"], a["n"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(block_table=None), -1), (dict(num_pages=0), -1), (dict(columns=0), -1),
    (dict(table_stride=3), -1), (dict(page_size=8), -1), (dict(page_size=48), -1), (dict(page_size=1 << 17), -1),
    (dict(columns=1 << 27, table_stride=1 << 27), -1), (dict(page_stride=100), -1), (dict(row_stride=1028), -1),
    (dict(head_stride=64), -1), (dict(head_stride=-128), -1), (dict(page_stride=1 << 39), -1), (dict(n_kv_heads=0), -1),
    (dict(k=FAKE + 8), -2), (dict(v=FAKE + 2), -2), (dict(block_table=FAKE + 2), -2),
])
def test_bad_pages_are_refused_by_every_entry(lib, kw, code):
    for call in (append, decode, prefill):
        assert call(lib, pages(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(start=None), -1), (dict(rope=None), -1), (dict(rows=0), -1),
    (dict(q=None), -1), (dict(out=None), -1), (dict(N=-1), -1), (dict(N=(1 << 24) + 1), -1), (dict(B=0), -1),
    (dict(cu=None), -1), (dict(heads=33), -1), (dict(heads=8 * 17), -1), (dict(heads=0), -1), (dict(qs=4000), -1),
    (dict(ks=1023), -1), (dict(vs=512), -1), (dict(q=FAKE, out=FAKE, qs=6144), -1), (dict(ws=None), -1),
    (dict(k=FAKE + 2), -2), (dict(q=FAKE + 8), -2), (dict(rope=FAKE + 4), -2), (dict(start=FAKE + 2), -2),
    (dict(cu=FAKE + 1), -2), (dict(ws=FAKE + 8), -2), (dict(n=WS - 1), -3),
])
def test_append_refuses(lib, kw, code):
    assert append(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(out=None), -1), (dict(start=None), -1), (dict(B=0), -1), (dict(B=2049), -1),
    (dict(heads=30), -1), (dict(heads=0), -1), (dict(qs=4088), -1), (dict(scale=0.0), -1), (dict(scale=-1.0), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(q=FAKE + 8), -2), (dict(out=FAKE + 8), -2),
    (dict(start=FAKE + 2), -2), (dict(n=100), -3),
])
def test_decode_refuses(lib, kw, code):
    assert decode(lib, **kw) == code


def test_decode_refuses_more_chunks_than_it_can_count(lib):
    p = pages(columns=1 << 21, table_stride=1 << 21)
    assert decode(lib, p, B=128) == -1


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(out=None), -1), (dict(cu=None), -1), (dict(N=-1), -1), (dict(B=0), -1), (dict(B=2049), -1),
    (dict(heads=30), -1), (dict(qs=4088), -1), (dict(scale=0.0), -1), (dict(cu=FAKE + 2), -2), (dict(out=FAKE + 8), -2),
    (dict(ws=None), -1), (dict(n=0), -3),
])
def test_prefill_refuses(lib, kw, code):
    assert prefill(lib, **kw) == code
    assert packed(lib, **kw) == code


def test_prefill_refuses_its_own_arguments(lib):
    assert prefill(lib, start=None) == -1
    assert prefill(lib, start=FAKE + 2) == -2
    assert packed(lib, k=None) == -1 and packed(lib, v=None) == -1
    assert packed(lib, ks=1000) == -1 and packed(lib, vs=1028) == -1 and packed(lib, kv=0) == -1
    assert packed(lib, k=FAKE + 8) == -2


def test_prefill_refuses_more_key_tiles_than_it_can_count(lib):
    p = pages(columns=1 << 23, table_stride=1 << 23)    # 2^27 positions, 8 KV heads
    assert prefill(lib, p) == -1


A = 1 << 30   # an address space of its own for these


@pytest.mark.parametrize("call,kw", [
    (append, dict(out=A + 256)),                                      # part of q
    (append, dict(out=FAKE)), (append, dict(q=4 * A, out=A - 4096)),  # the pages; k
    (append, dict(q=4 * A, k=8 * A, out=2 * A + 4 * 2048 + 2032)),    # the end of v
    (decode, dict(out=A)), (decode, dict(out=A - 16)), (decode, dict(out=FAKE + 130000)),
    (prefill, dict(out=A)), (prefill, dict(out=A + 4 * 8192 + 8176)), (prefill, dict(out=FAKE + 130000)),
    (packed, dict(out=A)), (packed, dict(q=4 * A, out=A + 16)), (packed, dict(q=4 * A, k=8 * A, out=2 * A))])
def test_outputs_that_overlap_inputs_are_refused(lib, call, kw):
    a = dict(q=A, out=16 * A)
    if call in (append, packed):
        a.update(k=A, v=2 * A)
    a.update(kw)
    assert call(lib, **a) == -1


def test_an_append_refuses_inputs_in_the_pages(lib):
    # the pages (8 heads, 4 pages of 16 rows: 131,072 bytes each) are outputs too
    def call(k=4 * A, v=5 * A, **kw):
        p = Pages(A, 2 * A, 16 * 1024, 1024, 128, 3 * A, 4, 16, 8, 4, 4)
        a = dict(q=6 * A, k=k, v=v, cu=7 * A, start=8 * A, rope=9 * A, out=10 * A, ws=11 * A)
        a.update(kw)
        return append(lib, (ctypes.addressof(p), p), **a)
    end = 131072
    assert call(k=A) == -1 and call(k=A + end - 16) == -1 and call(k=2 * A + 4096) == -1
    assert call(v=A) == -1 and call(v=2 * A) == -1 and call(v=2 * A - 1024) == -1
    assert call(q=A + 256, ks=1024) == -1 and call(q=2 * A + 256) == -1
    # without queries as well
    for kw in (dict(k=A), dict(v=2 * A + end - 16), dict(start=A), dict(cu=2 * A), dict(rope=A + 16), dict(ws=A)):
        assert call(q=None, out=None, **kw) == -1
    # the queries on other inputs
    assert call(out=8 * A) == -1 and call(out=7 * A) == -1 and call(out=9 * A) == -1 and call(out=11 * A + 4096) == -1


@pytest.mark.parametrize("between,strides,meet", [
    (0, (16384, 1024, 128), True), (8, (16384, 1024, 128), True), (-120, (16384, 1024, 128), True),
    (16384 * 3 + 1024 * 15, (16384, 1024, 128), True), (-16384 * 3, (16384, 1024, 128), True),
    (16384 * 2 - 1024 * 5 + 128 * 7 + 64, (16384, 1024, 128), True), (16384 * 4, (16384, 1024, 128), False),
    # interleaved by page, by row, by head
    (16384, (32768, 1024, 128), False), (-16384, (32768, 1024, 128), False), (16376, (32768, 1024, 128), True),
    (1024, (32768, 2048, 128), False), (1016, (32768, 2048, 128), True), (-1032, (32768, 2048, 128), True),
    (128, (32768, 2048, 256), False), (120, (32768, 2048, 256), True),
    # head-major pages: one head further on, and side by side
    (2048, (16384, 128, 2048), True), (-128 * 15, (16384, 128, 2048), True), (16384, (32768, 128, 2048), False),
    (128, (32768, 256, 4096), False), (136, (32768, 256, 4096), True)])
def test_an_append_refuses_key_and_value_rows_that_meet(lib, between, strides, meet):
    p = Pages(A, A + 2 * between, *strides, 3 * A, 4, 16, 8, 4, 4)
    k, v = ({x * strides[0] + y * strides[1] + z * strides[2] + o for x in range(4) for y in range(16) for z in range(8)}
            for o in (0, between))
    assert meet == any(r + d in v for r in k for d in range(-120, 128, 8))
    if meet or not torch.cuda.is_available():   # accepted, the call reaches the launch, which needs a device
        got = append(lib, (ctypes.addressof(p), p), q=None, out=None, k=4 * A, v=5 * A, cu=7 * A, start=8 * A,
                     rope=9 * A, ws=11 * A)
        assert got == (-1 if meet else -4)


@pytest.mark.parametrize("call", [decode, prefill])
def test_attention_outputs_on_index_inputs_are_refused(lib, call):
    p = Pages(A, 2 * A, 16 * 1024, 1024, 128, 3 * A, 4, 16, 8, 4, 4)
    a = dict(q=6 * A, start=8 * A, ws=11 * A)
    if call is prefill:
        a["cu"] = 7 * A
        assert call(lib, (ctypes.addressof(p), p), out=7 * A, **a) == -1
    assert call(lib, (ctypes.addressof(p), p), out=8 * A, **a) == -1
    assert call(lib, (ctypes.addressof(p), p), out=3 * A + 16, **a) == -1
    assert call(lib, (ctypes.addressof(p), p), out=11 * A + 65536, **a) == -1
    if call is prefill:
        assert packed(lib, q=6 * A, k=4 * A, v=5 * A, cu=7 * A, ws=11 * A, out=7 * A) == -1
        assert packed(lib, q=6 * A, k=4 * A, v=5 * A, cu=7 * A, ws=11 * A, out=11 * A) == -1


def test_no_tokens_is_no_launch(lib):
    assert append(lib, N=0) == 0 and lib.gqa_last_launch_count() == 0
    assert prefill(lib, N=0) == 0 and packed(lib, N=0) == 0 and lib.gqa_last_launch_count() == 0


def test_binding_refuses_host_tensors():
    bf = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    kp = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        G.paged_decode(bf, i, kp, kp, t)
    with pytest.raises(ValueError, match="CUDA tensor"):
        G.paged_append(None, bf[:, :2], bf[:, :2], i, torch.zeros(4, 64, 2), kp, kp, t)
    with pytest.raises(TypeError, match="torch.Tensor"):
        G.packed_prefill(None, bf, bf, i)


@pytest.mark.parametrize("workspace", [None, torch.zeros(8, dtype=torch.uint8)])
def test_binding_refuses_an_output_without_queries(workspace):
    a = good()
    a.update(q=None, workspace=workspace)
    with pytest.raises(ValueError, match="q_out needs q"):
        G.paged_append(**a)


def good():
    """Arguments of paged_append that only their device is wrong with."""
    x = torch.zeros(6, 12, 128, dtype=torch.bfloat16)
    kp = torch.zeros(5, 16, 2, 128, dtype=torch.bfloat16)
    return dict(q=x[:, :8], k=x[:, 8:10], v=x[:, 10:], start_pos=torch.zeros(3, dtype=torch.int32),
                rope=torch.zeros(80, 64, 2), k_pages=kp, v_pages=kp.clone(),
                block_table=torch.zeros(3, 7, dtype=torch.int32), cu_tokens=torch.zeros(4, dtype=torch.int32),
                q_out=torch.zeros(6, 8, 128, dtype=torch.bfloat16), workspace=torch.zeros(8, dtype=torch.uint8))


def calls(a):
    """The four entries on the arguments `a` (a name each takes)."""
    pages = (a["k_pages"], a["v_pages"], a["block_table"])
    one = dict(out=a["q_out"], workspace=a["workspace"])
    return {
        "append": lambda: G.paged_append(**a),
        "decode": lambda: G.paged_decode(a["q"][:3] if isinstance(a["q"], torch.Tensor) else a["q"], a["start_pos"],
                                         *pages, out=a["q_out"][:3], workspace=a["workspace"]),
        "prefill": lambda: G.paged_prefill(a["q"], a["cu_tokens"], a["start_pos"], *pages, **one),
        "packed": lambda: G.packed_prefill(a["q"], a["k"], a["v"], a["cu_tokens"], **one),
    }


def test_binding_reaches_the_device_check():
    for call in calls(good()).values():
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


HND = torch.zeros(5, 2, 16, 128, dtype=torch.bfloat16).transpose(1, 2)
ALL = ("append", "decode", "prefill", "packed")
PAGED = ("append", "decode", "prefill")


@pytest.mark.parametrize("name,change,error,match,who", [
    ("q", lambda t: t.float(), TypeError, "q must be torch.bfloat16", ALL),
    ("q", lambda t: "q", TypeError, "q must be a torch.Tensor", ALL),
    ("q", lambda t: t[..., :64], ValueError, "q must be", ALL),
    ("q", lambda t: t[:, ::2], ValueError, "one after the other", ALL),
    ("q", lambda t: t[0], ValueError, "q must be", ("append", "packed", "prefill")),
    ("q", lambda t: t.transpose(1, 2).contiguous().transpose(1, 2), ValueError, "one after the other", ALL),
    ("q", lambda t: None, ValueError, "q_out needs q", ("append",)),
    ("k", lambda t: t[:5], ValueError, "must be", ("append", "packed")),
    ("k", lambda t: t[:, :1], ValueError, "must be", ("append",)),
    ("v", lambda t: t[:, :1], ValueError, r"v must be \[6, 2, 128\]", ("append", "packed")),
    ("v", lambda t: t.half(), TypeError, "v must be torch.bfloat16", ("append", "packed")),
    ("start_pos", lambda t: t.long(), TypeError, "start_pos must be torch.int32", PAGED),
    ("start_pos", lambda t: [0, 0, 0], TypeError, "start_pos must be a torch.Tensor", PAGED),
    ("start_pos", lambda t: t[:2], ValueError, "must be", PAGED),
    ("start_pos", lambda t: torch.zeros(6, dtype=torch.int32)[::2], ValueError, "start_pos must be", PAGED),
    ("cu_tokens", lambda t: t[:3], ValueError, r"cu_tokens must be a contiguous \[4\]", ("append", "prefill")),
    ("cu_tokens", lambda t: t[:1], ValueError, "cu_tokens must", ("append", "prefill", "packed")),
    ("cu_tokens", lambda t: t.long(), TypeError, "cu_tokens must be torch.int32", ("append", "prefill", "packed")),
    ("cu_tokens", lambda t: None, ValueError, "one value per token", ("append",)),
    ("rope", lambda t: t.double(), TypeError, "rope must be torch.float32", ("append",)),
    ("rope", lambda t: t[:, :32], ValueError, "rope must be", ("append",)),
    ("k_pages", lambda t: t[0], ValueError, "k_pages must be", PAGED),
    ("k_pages", lambda t: t.float(), TypeError, "k_pages must be torch.bfloat16", PAGED),
    ("k_pages", lambda t: HND, ValueError, "strides of k_pages", PAGED),
    ("v_pages", lambda t: t[:4], ValueError, "shape and the strides", PAGED),
    ("block_table", lambda t: t.long(), TypeError, "block_table must be torch.int32", PAGED),
    ("block_table", lambda t: t[:2], ValueError, r"block_table must be \[3, columns\]", PAGED),
    ("block_table", lambda t: t.repeat(1, 2)[:, ::2], ValueError, "adjacent columns", PAGED),
    ("block_table", lambda t: None, TypeError, "block_table must be a torch.Tensor", PAGED),
    ("q_out", lambda t: t.float(), TypeError, "must be torch.bfloat16", ALL),
    ("q_out", lambda t: t[:, :4], ValueError, "must be a contiguous", ALL),
    ("q_out", lambda t: t.repeat(1, 1, 2)[..., ::2], ValueError, "must be a contiguous", ALL),
    ("q_out", lambda t: t[:2], ValueError, "must be a contiguous", ALL),
])
def test_binding_refuses(name, change, error, match, who):
    a = good()
    a[name] = change(a[name])
    for entry in who:
        with pytest.raises(error, match=match):
            calls(a)[entry]()


def test_binding_is_required(monkeypatch, tmp_path):
    monkeypatch.setattr(G, "_BINDING_PATH", str(tmp_path / "missing.so"))
    monkeypatch.setattr(G, "_paged", None)
    with pytest.raises(ImportError, match="gqa_binding"):
        G._binding()


# ------------------------------------------------------------------ work split of the decode attention

class Split:
    """`total` chunks over `parts` ranges, the first `more` of them one longer."""

    def __init__(self, total, parts):
        self.each, self.more = divmod(total, parts)

    def start(self, c):
        return c * self.each + min(c, self.more)

    def holder(self, u):
        x = self.more * (self.each + 1)
        return u // (self.each + 1) if u < x else self.more + (u - x) // self.each


@pytest.mark.parametrize("lens", [[1], [16], [17], [1000] * 16, [131072], [0, 5, 0, 300, 1], list(range(70)), [1] * 2000])
@pytest.mark.parametrize("n_kv", [1, 2, 8, 32])
@pytest.mark.parametrize("warps", [6, 8])
def test_decode_ranges_cover_every_chunk_once_and_tickets_count(lens, n_kv, warps):
    """Every chunk lies in one warp's range; a segment that several CTAs hold is
    written by exactly the CTAs its ticket expects, one part each, its first
    CTA's behind-slot and the others' before-slot, at most one of each per CTA."""
    chunks = [-(-n // 16) for n in lens]
    total = sum(chunks) * n_kv
    ctas = min(152, -(-total // warps))
    assert total >= ctas
    split = Split(total, ctas)
    seg_ends, at = [], 0
    for n in chunks:
        for _ in range(n_kv if n else 0):
            seg_ends.append((at, at + n))
            at += n
    assert at == total
    slots, tickets, covered, k = {}, {}, 0, 0
    for c in range(ctas):
        c0, c1 = split.start(c), split.start(c + 1)
        assert c1 > c0 == covered
        covered = c1
        w0 = c0
        for w in range(warps):
            a0, a1 = c0 + (c1 - c0) * w // warps, c0 + (c1 - c0) * (w + 1) // warps
            assert a1 >= a0 == w0
            w0 = a1
        assert w0 == c1
        for u in (c0, c1 - 1):
            assert split.holder(u) == c
        while seg_ends[k][1] <= c0:
            k += 1
        j = k
        while j < len(seg_ends) and seg_ends[j][0] < c1:
            first, end = seg_ends[j]
            if not (first >= c0 and end <= c1):
                side = 0 if first < c0 else 1
                assert (c, side) not in slots
                slots[c, side] = j
                lo, hi = split.holder(first), split.holder(end - 1)
                assert side == (1 if c == lo else 0)
                tickets.setdefault(lo, []).append((j, hi - lo + 1))
            j += 1
    assert covered == total
    for arrivals in tickets.values():
        assert len(set(arrivals)) == 1 and len(arrivals) == arrivals[0][1]


ITEM_UNITS = 2


@pytest.mark.parametrize("tiles", [[64] * 4, [57, 58, 59, 60, 61, 62, 63, 64], [157, 1, 0, 3], [469], [1, 1, 20]])
@pytest.mark.parametrize("n_kv", [1, 2, 8])
def test_prefill_ranges_cover_every_key_tile_once(tiles, n_kv):
    """Equal ranges of units (an item: its key tiles and two units before
    them): every tile of every item in one part; the parts of an item come from
    the CTAs that its first and last tile lie in, one each, at most two shared
    items per CTA, begun before it and going on behind; the item of a range's
    last unit is the one that goes on."""
    cum = [0]
    for n in tiles:
        cum.append(cum[-1] + (n + ITEM_UNITS if n else 0))
    units = cum[-1] * n_kv
    parts = min(152, units // 3)
    if parts < 2:
        return
    split = Split(units, parts)

    def item(u, end):
        e = max(i for i in range(len(tiles)) if cum[i] * n_kv <= u)
        w = cum[e + 1] - cum[e]
        assert w > 0
        g = (u - cum[e] * n_kv) // w
        base = cum[e] * n_kv + g * w + ITEM_UNITS
        j1, j0 = min(w - ITEM_UNITS, end - base), max(0, u - base)
        return e, g, j0, j1, split.holder(base), split.holder(base + w - ITEM_UNITS - 1), min(end, base + w - ITEM_UNITS)

    seen, slots = {}, set()
    for c in range(parts):
        u, end = split.start(c), split.start(c + 1)
        assert end > u
        goes_on = None
        while u < end:
            e, g, j0, j1, first, last, after = item(u, end)
            assert after > u
            u = after
            if j1 <= j0:
                continue
            assert first <= c <= last and (j0 == 0) == (c == first)
            if first != last:
                slot = 2 * c + (c == first)
                assert slot not in slots
                slots.add(slot)
                if c == first:
                    goes_on = e, g, last
            seen.setdefault((e, g), []).append((j0, j1, c, first, last))
        e, g, _, _, first, last, _ = item(end - 1, end)
        assert goes_on == ((e, g, last) if first == c and last > c else None)
    for (e, g), got in seen.items():
        at = 0
        for j0, j1, c, first, last in got:
            assert j0 == at and j1 > j0
            at = j1
        assert at == tiles[e] and [x[2] for x in got] == list(range(got[0][3], got[0][4] + 1))
    assert len(seen) == n_kv * sum(n > 0 for n in tiles)


@pytest.mark.parametrize("n_kv", [1, 2, 8, 32])
@pytest.mark.parametrize("few", [True, False])
def test_prefill_ranges_bound_the_parts_of_an_item(n_kv, few):
    """Ranges of half the longest item: three parts at most; shorter ones: no
    more than the second kernel has room for."""
    rng = random.Random(n_kv)
    for _ in range(300):
        top = rng.choice([4, 20, 300, 8192])
        tiles = [rng.randint(0, top) for _ in range(rng.randint(1, 320))]
        cum = [0]
        for n in tiles:
            cum.append(cum[-1] + (n + ITEM_UNITS if n else 0))
        units, longest = cum[-1] * n_kv, max(tiles) + ITEM_UNITS
        if units < 6:
            continue
        mean = max((units + 151) // 152, 3)
        size = max(mean, (longest + 1) // 2 if few else (longest + 61) // 62)
        parts = min(152, max(1, units // size))
        split = Split(units, parts)
        for e, n in enumerate(tiles):
            for g in range(n_kv if n else 0):
                base = cum[e] * n_kv + g * (n + ITEM_UNITS) + ITEM_UNITS
                assert split.holder(base + n - 1) - split.holder(base) < (3 if few else 64)


def sequence_of(cu, B, m):
    lo, size = 0, B
    while size > 0:
        step = (size + 31) // 32
        n = sum(1 for lane in range(32) if (lane + 1) * step <= size and cu[lo + (lane + 1) * step] <= m)
        lo += n * step
        size = min(step - 1, size - n * step)
    return lo


@pytest.mark.parametrize("B", [1, 2, 31, 32, 33, 64, 100, 1023, 1025])
def test_sequence_search_passes_over_empty_sequences(B):
    lens = [(b * 7 // 3) % 4 for b in range(B)]
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    owner = [b for b, n in enumerate(lens) for _ in range(n)]
    for m, b in enumerate(owner):
        assert sequence_of(cu, B, m) == b
    assert sequence_of(cu, B, cu[-1]) == B
