"""Refusals of the 8-bit cache's operators and of the rotary layouts (argument
checks of the binding and of the C ABI; nothing is launched), on the CPU."""
import ctypes

import pytest
import torch

import grouped_query_attention_gemv_gb300 as G
from grouped_query_attention_gemv_gb300 import build as gbuild
from tests.test_paged_cpu import FAKE, WS, pages

EINVAL, EALIGN, EWORKSPACE = -1, -2, -3
# tensors of a call lie this far apart
K, V, KS, VS, TABLE, OUT = (FAKE * n for n in (64, 128, 192, 256, 320, 384))


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return G.lib()


class Pages8(ctypes.Structure):
    """gqa_fp8_pages of include/gqa.h."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")] + \
        [(n, ctypes.c_longlong) for n in ("page_stride", "row_stride", "head_stride", "scale_page_stride",
                                          "scale_row_stride", "scale_head_stride")] + \
        [("block_table", ctypes.c_void_p)] + \
        [(n, ctypes.c_int) for n in ("num_pages", "page_size", "n_kv_heads", "table_stride", "columns")]


def pages8(**kw):
    a = dict(k=K, v=V, k_scale=KS, v_scale=VS, page_stride=16 * 8 * 128, row_stride=8 * 128, head_stride=128,
             scale_page_stride=16 * 8, scale_row_stride=8, scale_head_stride=1, block_table=TABLE, num_pages=4,
             page_size=16, n_kv_heads=8, table_stride=4, columns=4)
    a.update(kw)
    p = Pages8(**a)
    return ctypes.addressof(p), p


def append(lib, p=None, fn=None, **kw):
    a = dict(q=FAKE, qs=4096, k=FAKE * 2, ks=1024, v=FAKE * 3, vs=1024, N=5, heads=32, cu=FAKE * 4, B=2, start=FAKE * 5,
             rope=FAKE * 6, rows=64, dim=128, halves=0, out=OUT, ws=OUT * 2, n=WS)
    a.update(kw)
    g, keep = pages8() if p is None else p
    return (fn or lib.gqa_paged_append_fp8)(
        a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["N"], a["heads"], a["cu"], a["B"], a["start"], a["rope"],
        a["rows"], a["dim"], a["halves"], g, a["out"], a["ws"], a["n"], None)


def decode(lib, p=None, **kw):
    a = dict(q=FAKE, qs=4096, B=2, heads=32, start=FAKE * 5, scale=0.1, out=OUT, ws=OUT * 2, n=WS)
    a.update(kw)
    g, keep = pages8() if p is None else p
    return lib.gqa_paged_decode_fp8(a["q"], a["qs"], a["B"], a["heads"], a["start"], g, a["scale"], a["out"], a["ws"],
                                    a["n"], None)


def read(lib, p=None, to=None, **kw):
    a = dict(rows=FAKE * 5, B=2, ws=OUT * 2, n=WS)
    a.update(kw)
    g, keep = pages8() if p is None else p
    t, keep2 = pages(k=OUT, v=OUT + FAKE, block_table=FAKE * 6) if to is None else to
    return lib.gqa_paged_read_fp8(a["rows"], a["B"], g, t, a["ws"], a["n"], None)


REFUSED_LATE = EWORKSPACE   # arguments that only the workspace's size is wrong with


def test_good_arguments_reach_the_last_check(lib):
    for call in (append, decode, read):
        assert call(lib, n=WS - 1) == REFUSED_LATE
    assert append(lib, pages(k=K, v=V), lib.gqa_paged_append_rotary, n=WS - 1) == REFUSED_LATE


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(k_scale=None), EINVAL), (dict(v_scale=None), EINVAL),
    (dict(block_table=None), EINVAL), (dict(num_pages=0), EINVAL), (dict(page_size=8), EINVAL),
    (dict(page_size=48), EINVAL), (dict(page_size=131072), EINVAL), (dict(columns=0), EINVAL),
    (dict(table_stride=3), EINVAL), (dict(n_kv_heads=0), EINVAL), (dict(n_kv_heads=5), EINVAL),
    (dict(page_stride=16 * 8 * 128 + 8), EINVAL), (dict(row_stride=1032), EINVAL), (dict(head_stride=136), EINVAL),
    (dict(head_stride=64), EINVAL), (dict(row_stride=-1024), EINVAL), (dict(page_stride=1 << 38), EINVAL),
    (dict(scale_page_stride=0), EINVAL), (dict(scale_row_stride=0), EINVAL), (dict(scale_head_stride=-1), EINVAL),
    (dict(scale_row_stride=1 << 38), EINVAL), (dict(columns=1 << 27, table_stride=1 << 27), EINVAL),
    (dict(k=K + 8), EALIGN), (dict(v=V + 1), EALIGN), (dict(block_table=TABLE + 2), EALIGN),
])
def test_bad_pages_are_refused_by_every_entry(lib, kw, code):
    for call in (append, decode):
        assert call(lib, pages8(**kw)) == code
    if "n_kv_heads" not in kw:
        assert read(lib, pages8(**kw)) == code


def test_scales_may_lie_anywhere(lib):
    for call in (append, decode, read):
        assert call(lib, pages8(k_scale=KS + 1, v_scale=VS + 3, scale_row_stride=9, scale_page_stride=1), n=0) == REFUSED_LATE


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("kw,code", [
    (dict(dim=0), EINVAL), (dict(dim=8), EINVAL), (dict(dim=24), EINVAL), (dict(dim=144), EINVAL), (dict(dim=-128), EINVAL),
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(start=None), EINVAL), (dict(rope=None), EINVAL),
    (dict(rows=0), EINVAL), (dict(q=None), EINVAL), (dict(out=None), EINVAL), (dict(N=-1), EINVAL),
    (dict(N=(1 << 24) + 1), EINVAL), (dict(B=0), EINVAL), (dict(cu=None), EINVAL), (dict(heads=33), EINVAL),
    (dict(heads=8 * 17), EINVAL), (dict(ks=1016), EINVAL), (dict(vs=1028), EINVAL), (dict(qs=4088), EINVAL),
    (dict(out=FAKE, qs=4104), EINVAL), (dict(k=FAKE * 2 + 8), EALIGN), (dict(rope=FAKE * 6 + 8), EALIGN),
    (dict(out=OUT + 2), EALIGN), (dict(start=FAKE * 5 + 1), EALIGN), (dict(ws=None), EINVAL), (dict(ws=OUT * 2 + 8), EALIGN),
    (dict(n=0), EWORKSPACE),
])
def test_appends_refuse(lib, fp8, kw, code):
    if fp8:
        assert append(lib, **kw) == code
    else:
        assert append(lib, pages(k=K, v=V, block_table=TABLE), lib.gqa_paged_append_rotary, **kw) == code


PAGES = 4 * 16 * 8   # rows


@pytest.mark.parametrize("kw", [
    dict(k=K), dict(v=V + PAGES * 128 - 16), dict(q=VS - VS % 16, out=OUT), dict(k=(KS + PAGES - 1) // 16 * 16),
    dict(start=KS), dict(cu=VS), dict(rope=K + 128), dict(out=V), dict(out=KS // 16 * 16), dict(out=FAKE * 2), dict(ws=K),
    dict(ws=VS // 16 * 16), dict(out=TABLE),
])
def test_an_append_refuses_shared_memory(lib, kw):
    assert append(lib, **kw) == EINVAL


@pytest.mark.parametrize("kw", [dict(v=K), dict(v=K + 64 * 16), dict(v_scale=KS), dict(v_scale=KS + 5), dict(k_scale=K),
                                dict(v_scale=V + 100), dict(k_scale=V + PAGES * 128 - 1), dict(block_table=K),
                                dict(block_table=VS)])
def test_an_append_refuses_pages_that_meet(lib, kw):
    assert append(lib, pages8(**kw)) == EINVAL


def test_pages_may_interleave(lib):
    # [pages, 2, page, head, 128] and [pages, 2, page, head]
    p = pages8(v=K + 16 * 8 * 128, page_stride=2 * 16 * 8 * 128, v_scale=KS + 16 * 8, scale_page_stride=2 * 16 * 8)
    assert append(lib, p, N=0) == 0
    # [pages, page, head, 2]: scales side by side
    p = pages8(v_scale=KS + 1, scale_page_stride=256, scale_row_stride=16, scale_head_stride=2)
    assert append(lib, p, N=0) == 0
    assert append(lib, pages8(v_scale=KS + 2, scale_page_stride=256, scale_row_stride=16, scale_head_stride=2)) == EINVAL


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), EINVAL), (dict(start=None), EINVAL), (dict(out=None), EINVAL), (dict(B=0), EINVAL), (dict(B=2049), EINVAL),
    (dict(heads=0), EINVAL), (dict(heads=12), EINVAL), (dict(heads=136), EINVAL), (dict(scale=0.0), EINVAL),
    (dict(scale=float("nan")), EINVAL), (dict(scale=-1.0), EINVAL), (dict(qs=4095), EINVAL), (dict(qs=1024), EINVAL),
    (dict(q=FAKE + 8), EALIGN), (dict(out=OUT + 8), EALIGN), (dict(start=FAKE + 2), EALIGN), (dict(ws=None), EINVAL),
    (dict(n=0), EWORKSPACE), (dict(out=FAKE), EINVAL), (dict(out=K), EINVAL), (dict(out=KS), EINVAL), (dict(out=VS), EINVAL),
    (dict(out=TABLE), EINVAL), (dict(start=OUT), EINVAL), (dict(ws=OUT), EINVAL),
])
def test_decode_refuses(lib, kw, code):
    assert decode(lib, **kw) == code


def test_decode_refuses_more_chunks_than_it_can_count(lib):
    wide = dict(columns=1 << 20, table_stride=1 << 20, page_size=1024)
    assert decode(lib, pages8(**wide), B=7, n=0) == REFUSED_LATE
    assert decode(lib, pages8(**wide), B=8) == EINVAL


@pytest.mark.parametrize("kw,to,code", [
    (dict(rows=None), {}, EINVAL), (dict(B=0), {}, EINVAL), (dict(B=2049), {}, EINVAL), (dict(rows=FAKE + 2), {}, EALIGN),
    (dict(ws=None), {}, EINVAL), (dict(n=0), {}, EWORKSPACE), ({}, dict(n_kv_heads=4), EINVAL),
    ({}, dict(page_size=24), EINVAL), ({}, dict(k=None), EINVAL), ({}, dict(k=OUT + 2), EALIGN), ({}, dict(v=OUT), EINVAL),
    ({}, dict(k=K), EINVAL), ({}, dict(v=VS), EINVAL), ({}, dict(block_table=OUT), EINVAL),
    (dict(rows=OUT + 64), {}, EINVAL), (dict(ws=OUT), {}, EINVAL), ({}, dict(k=TABLE), EINVAL),
])
def test_read_refuses(lib, kw, to, code):
    assert read(lib, to=pages(**{**dict(k=OUT, v=OUT + FAKE, block_table=FAKE * 6), **to}), **kw) == code


def test_read_refuses_more_units_than_it_can_count(lib):
    wide = dict(columns=1 << 20, table_stride=1 << 20, page_size=1024)
    far = dict(k=OUT, v=OUT + FAKE, block_table=FAKE * 6)
    # FAKE apart, tables this wide would meet the pages: only the narrower side counts
    assert read(lib, pages8(**wide), pages(**far), B=2, n=0) == REFUSED_LATE
    assert read(lib, pages8(**wide), pages(**{**far, **wide}), B=33) == EINVAL


def test_rope_table_refuses(lib):
    f = lib.gqa_rope_table_dim
    for dim in (0, 1, 3, 130, -2):
        assert f(FAKE, 4, dim, 1e4, 0, 8.0, 1.0, 4.0, 8192.0, None) == EINVAL
        with pytest.raises(ValueError, match="dim must be even"):
            G.rope_table(4, dim=dim, device="cpu")
    assert f(FAKE + 8, 4, 64, 1e4, 0, 8.0, 1.0, 4.0, 8192.0, None) == EALIGN
    assert f(FAKE, 4, 64, 0.5, 0, 8.0, 1.0, 4.0, 8192.0, None) == EINVAL


# ------------------------------------------------------------------ the binding

def good():
    """Arguments that only their device is wrong with."""
    x = torch.zeros(6, 12, 128, dtype=torch.bfloat16)
    kp = torch.zeros(5, 16, 2, 128, dtype=torch.float8_e4m3fn)
    sc = torch.zeros(5, 16, 2, dtype=torch.uint8)
    out = torch.zeros(7, 32, 2, 128, dtype=torch.bfloat16)
    return dict(q=x[:, :8], k=x[:, 8:10], v=x[:, 10:], start_pos=torch.zeros(3, dtype=torch.int32),
                rope=torch.zeros(80, 32, 2), k_pages=kp, v_pages=kp.clone(), k_scales=sc, v_scales=sc.clone(),
                block_table=torch.zeros(3, 7, dtype=torch.int32), cu_tokens=torch.zeros(4, dtype=torch.int32),
                q_out=torch.zeros(6, 8, 128, dtype=torch.bfloat16), rotary_dim=64, halves=True,
                workspace=torch.zeros(8, dtype=torch.uint8), k_out=out, v_out=out.clone(),
                out_table=torch.zeros(3, 4, dtype=torch.int32))


def calls(a):
    cache = tuple(a[n] for n in ("k_pages", "v_pages", "k_scales", "v_scales", "block_table"))
    append_args = {n: a[n] for n in ("q", "k", "v", "start_pos", "rope", "cu_tokens", "q_out", "rotary_dim", "halves",
                                     "workspace", "block_table", "k_pages", "v_pages")}
    bf = {**append_args, "k_pages": torch.zeros(5, 16, 2, 128, dtype=torch.bfloat16)}
    bf["v_pages"] = bf["k_pages"].clone()
    return {
        "append8": lambda: G.paged_append_fp8(**append_args, k_scales=a["k_scales"], v_scales=a["v_scales"]),
        "append": lambda: G.paged_append(**bf),
        "decode": lambda: G.paged_decode_fp8(a["q"][:3] if isinstance(a["q"], torch.Tensor) else a["q"], a["start_pos"],
                                             *cache, out=a["q_out"][:3], workspace=a["workspace"]),
        "read": lambda: G.paged_read_fp8(a["start_pos"], *cache, a["k_out"], a["v_out"], a["out_table"],
                                         workspace=a["workspace"]),
    }


def test_binding_reaches_the_device_check():
    for call in calls(good()).values():
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()


APPENDS, CACHE, ALL = ("append8", "append"), ("append8", "decode", "read"), ("append8", "append", "decode", "read")


@pytest.mark.parametrize("name,change,error,match,who", [
    ("q", lambda t: t.float(), TypeError, "q must be torch.bfloat16", APPENDS + ("decode",)),
    ("q", lambda t: t[:, ::2], ValueError, "one after the other", APPENDS + ("decode",)),
    ("q", lambda t: None, ValueError, "q_out needs q", APPENDS),
    ("k", lambda t: t[:, :1], ValueError, "must be", APPENDS),
    ("v", lambda t: t.half(), TypeError, "v must be torch.bfloat16", APPENDS),
    ("start_pos", lambda t: t.long(), TypeError, "must be torch.int32", ALL),
    ("start_pos", lambda t: t[:2], ValueError, "must be", ALL),
    ("cu_tokens", lambda t: None, ValueError, "one value per token", APPENDS),
    ("rope", lambda t: t.double(), TypeError, "rope must be torch.float32", APPENDS),
    ("rope", lambda t: torch.zeros(80, 64, 2), ValueError, r"rope must be a contiguous \[rows, 32, 2\]", APPENDS),
    ("rotary_dim", lambda t: 0, ValueError, "rotary_dim must be a multiple of 16", APPENDS),
    ("rotary_dim", lambda t: 40, ValueError, "rotary_dim must be a multiple of 16", APPENDS),
    ("rotary_dim", lambda t: 256, ValueError, "rotary_dim must be a multiple of 16", APPENDS),
    ("rotary_dim", lambda t: 1 << 40, ValueError, "rotary_dim is out of range", APPENDS),
    ("rotary_dim", lambda t: "64", TypeError, "int", APPENDS),
    ("rotary_dim", lambda t: 128, ValueError, r"rope must be a contiguous \[rows, 64, 2\]", APPENDS),
    ("k_pages", lambda t: t.float(), TypeError, "k_pages must be torch.float8_e4m3fn", CACHE),
    ("k_pages", lambda t: t.view(torch.uint8), TypeError, "k_pages must be torch.float8_e4m3fn", CACHE),
    ("k_pages", lambda t: t[0], ValueError, "k_pages must be", CACHE),
    ("v_pages", lambda t: t[:4], ValueError, "shape and the strides of k_pages", CACHE),
    ("k_scales", lambda t: t.int(), TypeError, "k_scales must be torch.uint8", CACHE),
    ("k_scales", lambda t: t[..., 0], ValueError, "k_scales must be", CACHE),
    ("k_scales", lambda t: t[:, :8], ValueError, "k_scales must be", CACHE),
    ("v_scales", lambda t: t[:, :, :1], ValueError, "v_scales must have the shape", CACHE),
    ("v_scales", lambda t: t.transpose(1, 2).contiguous().transpose(1, 2), ValueError, "strides of k_scales", CACHE),
    ("v_scales", lambda t: None, TypeError, "v_scales must be a torch.Tensor", CACHE),
    ("block_table", lambda t: t.long(), TypeError, "block_table must be torch.int32", ALL),
    ("block_table", lambda t: t[:2], ValueError, r"block_table must be \[3, columns\]", ALL),
    ("q_out", lambda t: t[:, :4], ValueError, "must be a contiguous", APPENDS + ("decode",)),
    ("k_out", lambda t: t.float(), TypeError, "k_out must be torch.bfloat16", ("read",)),
    ("k_out", lambda t: t[..., :64], ValueError, "k_out must be", ("read",)),
    ("v_out", lambda t: t[:3], ValueError, "v_out must have the shape and the strides of k_out", ("read",)),
    ("out_table", lambda t: t[:2], ValueError, r"out_table must be \[3, columns\]", ("read",)),
    ("out_table", lambda t: t.long(), TypeError, "out_table must be torch.int32", ("read",)),
])
def test_binding_refuses(name, change, error, match, who):
    a = good()
    a[name] = change(a[name])
    for entry in who:
        if entry == "append" and name in ("k_pages", "v_pages"):
            continue
        with pytest.raises(error, match=match):
            calls(a)[entry]()


def test_other_kv_heads_are_refused():
    a = good()
    a["k_out"], a["v_out"] = (torch.zeros(7, 32, 3, 128, dtype=torch.bfloat16) for _ in range(2))
    with pytest.raises(ValueError, match="k_out must have the KV heads of k_pages"):
        calls(a)["read"]()


def test_missing_tensors_are_refused():
    a = good()
    a["workspace"] = None
    with pytest.raises(ValueError, match="CUDA tensor"):
        calls(a)["read"]()
    a["start_pos"] = None
    with pytest.raises(TypeError, match="rows must be a torch.Tensor"):
        calls(a)["read"]()
    with pytest.raises(ValueError, match="q_out needs q"):
        G.paged_append_fp8(None, *[None] * 9, q_out=torch.zeros(1))
