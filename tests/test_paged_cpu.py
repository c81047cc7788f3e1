"""The paged operators' refusals (argument checks of the binding and of the C
ABI; nothing is launched) and the arithmetic of their work split, on the CPU."""
import ctypes

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


def pages(**kw):
    a = dict(k=FAKE, v=FAKE, page_stride=16 * 8 * 128, row_stride=8 * 128, head_stride=128, block_table=FAKE,
             num_pages=4, page_size=16, n_kv_heads=8, table_stride=4, columns=4)
    a.update(kw)
    p = G._Pages(**a)
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
    p = pages(columns=1 << 25, table_stride=1 << 25, page_size=32)
    assert decode(lib, p, B=2048) == -1


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


CPU = torch.device("cpu")


def test_binding_checks_rows():
    x = torch.zeros(6, 12, 128, dtype=torch.bfloat16)
    assert G._rows(x[:, :8], "q", 6, 8, CPU) == 12 * 128
    assert G._rows(x[:1, :8], "q", 1, 8, CPU) == 8 * 128
    for bad, err in ((x.float(), TypeError), (x[:, ::2], ValueError), (x.transpose(0, 1), ValueError),
                     (x[..., :64], ValueError), ("x", TypeError)):
        with pytest.raises(err):
            G._rows(bad, "q", 6, 6, CPU)


def test_binding_checks_pages():
    k = torch.zeros(5, 16, 2, 128, dtype=torch.bfloat16)
    t = torch.zeros(3, 7, dtype=torch.int32)
    p = G._pages(k, k, t[:, :4], 3, CPU)
    assert (p.page_stride, p.row_stride, p.head_stride) == (16 * 256, 256, 128)
    assert (p.num_pages, p.page_size, p.n_kv_heads, p.table_stride, p.columns) == (5, 16, 2, 7, 4)
    h = torch.zeros(5, 2, 16, 128, dtype=torch.bfloat16).transpose(1, 2)
    p = G._pages(h, h, t, 3, CPU)
    assert (p.row_stride, p.head_stride) == (128, 16 * 128)
    one = torch.zeros(1, 16, 1, 128, dtype=torch.bfloat16)
    assert G._pages(one, one, t, 3, CPU).head_stride == 128
    for bad in ((k, k[:4], t, 3), (k, h, t, 3), (k, k, t, 2), (k, k, t.t(), 7), (k[0], k[0], t, 3),
                (k[..., :64], k[..., :64], t, 3)):
        with pytest.raises(ValueError):
            G._pages(*bad, CPU)
    for bad in ((k.float(), k.float(), t, 3), (k, k, t.long(), 3), (k, k, None, 3)):
        with pytest.raises(TypeError):
            G._pages(*bad, CPU)


def test_binding_checks_integers_and_outputs():
    i = torch.zeros(4, dtype=torch.int32)
    assert G._ints(i, "start_pos", 4, CPU) == i.data_ptr()
    for bad, err in ((i.long(), TypeError), (i[:3], ValueError), (torch.zeros(8, dtype=torch.int32)[::2], ValueError),
                     ([0] * 4, TypeError)):
        with pytest.raises(err):
            G._ints(bad, "start_pos", 4, CPU)
    o = torch.zeros(4, 12, 128, dtype=torch.bfloat16)
    assert G._dense_out(o, 4, 12, CPU, None) is o
    with pytest.raises(ValueError):
        G._dense_out(o[:, :8], 4, 8, CPU, None)
    with pytest.raises(TypeError):
        G._dense_out(o.float(), 4, 12, CPU, None)
    with pytest.raises(ValueError):
        G._paged_ws(torch.zeros(8), CPU, None)


# ------------------------------------------------------------------ work split of the decode attention

def range_start(c, total, parts):
    return total * c // parts


def part_of(u, total, parts):
    return ((u + 1) * parts - 1) // total


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
    seg_ends, at = [], 0
    for n in chunks:
        for _ in range(n_kv if n else 0):
            seg_ends.append((at, at + n))
            at += n
    assert at == total
    slots, tickets, covered, k = {}, {}, 0, 0
    for c in range(ctas):
        c0, c1 = range_start(c, total, ctas), range_start(c + 1, total, ctas)
        assert c1 > c0 == covered
        covered = c1
        w0 = c0
        for w in range(warps):
            a0, a1 = c0 + range_start(w, c1 - c0, warps), c0 + range_start(w + 1, c1 - c0, warps)
            assert a0 == w0 and a1 >= a0
            w0 = a1
        assert w0 == c1
        for u in (c0, c1 - 1):
            assert part_of(u, total, ctas) == c
        while seg_ends[k][1] <= c0:
            k += 1
        j = k
        while j < len(seg_ends) and seg_ends[j][0] < c1:
            first, end = seg_ends[j]
            if not (first >= c0 and end <= c1):
                side = 0 if first < c0 else 1
                assert (c, side) not in slots
                slots[c, side] = j
                lo, hi = part_of(first, total, ctas), part_of(end - 1, total, ctas)
                assert side == (1 if c == lo else 0)
                tickets.setdefault(lo, []).append((j, hi - lo + 1))
            j += 1
    assert covered == total
    for arrivals in tickets.values():
        assert len(set(arrivals)) == 1 and len(arrivals) == arrivals[0][1]


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
