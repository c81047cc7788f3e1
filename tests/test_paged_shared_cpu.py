"""Refusals of the decode attention with shared rows (argument checks of the
binding and of the C ABI; nothing is launched), on the CPU."""
import pytest
import torch

import grouped_query_attention_gemv_gb300 as G
from grouped_query_attention_gemv_gb300 import build as gbuild
from tests.test_paged_cpu import FAKE, WS, pages

EINVAL, EALIGN, EWORKSPACE = -1, -2, -3
K, V, TABLE, OUT = (FAKE * n for n in (64, 128, 192, 256))


@pytest.fixture(scope="module")
def lib():
    gbuild.build()
    return G.lib()


def shared(lib, p=None, **kw):
    a = dict(q=FAKE, qs=4096, B=2, heads=32, start=FAKE * 5, cu=FAKE * 6, G=1, prefix=FAKE * 7, scale=0.1, out=OUT,
             ws=OUT * 2, n=WS)
    a.update(kw)
    g, keep = pages(k=K, v=V, block_table=TABLE) if p is None else p
    return lib.gqa_paged_decode_shared(a["q"], a["qs"], a["B"], a["heads"], a["start"], a["cu"], a["G"], a["prefix"], g,
                                       a["scale"], a["out"], a["ws"], a["n"], None)


def test_good_arguments_reach_the_last_check(lib):
    assert shared(lib, n=WS - 1) == EWORKSPACE


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), EINVAL), (dict(start=None), EINVAL), (dict(out=None), EINVAL), (dict(cu=None), EINVAL),
    (dict(prefix=None), EINVAL), (dict(G=0), EINVAL), (dict(G=-1), EINVAL), (dict(G=2049), EINVAL), (dict(B=0), EINVAL),
    (dict(B=2049), EINVAL), (dict(heads=12), EINVAL), (dict(heads=136), EINVAL), (dict(scale=0.0), EINVAL),
    (dict(scale=float("inf")), EINVAL), (dict(qs=4095), EINVAL), (dict(q=FAKE + 8), EALIGN), (dict(out=OUT + 8), EALIGN),
    (dict(start=FAKE * 5 + 2), EALIGN), (dict(cu=FAKE * 6 + 2), EALIGN), (dict(prefix=FAKE * 7 + 1), EALIGN),
    (dict(ws=None), EINVAL), (dict(ws=OUT * 2 + 4), EALIGN), (dict(n=0), EWORKSPACE), (dict(out=FAKE), EINVAL),
    (dict(out=K), EINVAL), (dict(out=V), EINVAL), (dict(out=TABLE), EINVAL), (dict(start=OUT), EINVAL),
    (dict(cu=OUT + 64), EINVAL), (dict(prefix=OUT), EINVAL), (dict(ws=OUT), EINVAL),
])
def test_refusals(lib, kw, code):
    assert shared(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), EINVAL), (dict(block_table=None), EINVAL), (dict(page_size=24), EINVAL), (dict(num_pages=0), EINVAL),
    (dict(row_stride=1028), EINVAL), (dict(k=K + 2), EALIGN), (dict(columns=1 << 27, table_stride=1 << 27), EINVAL),
])
def test_bad_pages_are_refused(lib, kw, code):
    assert shared(lib, pages(**{**dict(k=K, v=V, block_table=TABLE), **kw})) == code


def good():
    x = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    kp = torch.zeros(5, 16, 2, 128, dtype=torch.bfloat16)
    return dict(q=x, start_pos=torch.zeros(3, dtype=torch.int32), cu_groups=torch.zeros(3, dtype=torch.int32),
                prefix_rows=torch.zeros(2, dtype=torch.int32), k_pages=kp, v_pages=kp.clone(),
                block_table=torch.zeros(3, 7, dtype=torch.int32), out=x.clone(),
                workspace=torch.zeros(8, dtype=torch.uint8))


@pytest.mark.parametrize("name,change,error,match", [
    ("q", lambda t: t, ValueError, "q must be a CUDA tensor"),
    ("q", lambda t: t.float(), TypeError, "q must be torch.bfloat16"),
    ("q", lambda t: None, TypeError, "q must be a torch.Tensor"),
    ("q", lambda t: t[:, ::2], ValueError, "one after the other"),
    ("start_pos", lambda t: t[:2], ValueError, r"start_pos must be a contiguous \[3\]"),
    ("cu_groups", lambda t: t[:2], ValueError, r"cu_groups must be a contiguous \[3\]"),
    ("cu_groups", lambda t: t.long(), TypeError, "cu_groups must be torch.int32"),
    ("cu_groups", lambda t: None, TypeError, "cu_groups must be a torch.Tensor"),
    ("prefix_rows", lambda t: t[:1], ValueError, r"cu_groups must be a contiguous \[2\]"),
    ("prefix_rows", lambda t: t.long(), TypeError, "prefix_rows must be torch.int32"),
    ("prefix_rows", lambda t: t[None], ValueError, "prefix_rows must be a contiguous one-dimensional"),
    ("prefix_rows", lambda t: 7, TypeError, "prefix_rows must be a torch.Tensor"),
    ("k_pages", lambda t: t.float(), TypeError, "k_pages must be torch.bfloat16"),
    ("v_pages", lambda t: t[:4], ValueError, "shape and the strides"),
    ("block_table", lambda t: t[:2], ValueError, r"block_table must be \[3, columns\]"),
    ("out", lambda t: t[:, :4], ValueError, "out must be a contiguous"),
])
def test_binding_refuses(name, change, error, match):
    a = good()
    a[name] = change(a[name])
    with pytest.raises(error, match=match):
        G.paged_decode_shared(**a)
