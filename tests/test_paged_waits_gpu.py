"""Waits that run out: the call ends soon, says so, and writes nothing but its
rows; the workspace serves again once it is zero-filled."""
import time

import pytest
import torch

import grouped_query_attention_gemv_gb300 as G
from tests import paged as P
from tests import paged8 as Q
from tests.test_paged_fp8_gpu import check_decode
from tests.test_paged_gpu import ints
from tests.test_paged_shared_gpu import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture
def gen():
    return torch.Generator(device="cuda").manual_seed(5)


def given_up(call, memory):
    """`call` under a limit that no wait keeps; `memory` is left as it was."""
    before = [t.view(torch.uint8).clone() for t in memory]
    prev = G.set_wait_limit_ns(1)
    try:
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        call()
        torch.cuda.synchronize()
        took = time.perf_counter() - t0
    finally:
        G.set_wait_limit_ns(prev)
    assert took < 0.5, f"a limit of 1 ns ended the call after {took:.2f} s"
    assert all(torch.equal(t.view(torch.uint8), x) for t, x in zip(memory, before))


# With 16 query heads per KV head, and rows in L2, copies land beside the work:
# nothing need be left to wait for, and the call may be as good as any.
@pytest.mark.parametrize("heads,n_kv,page,lens,waits", [(32, 8, 64, [60_000], True),
                                                        (32, 2, 16, [20_000, 1, 30_000, 700], False)])
def test_waits_of_the_8_bit_decode(gen, heads, n_kv, page, lens, waits):
    ws = G.make_paged_workspace()
    cache, rows = Q.fill(gen, lens, page, n_kv)
    B = len(lens)
    q = P.normal(gen, B, heads, P.D, scale=1.5)
    start = ints([n - 1 for n in lens])
    guard = torch.full((B + 2, heads, P.D), 9.0, dtype=torch.bfloat16, device="cuda")
    out = guard[1:-1]
    for _ in range(3):
        given_up(lambda: G.paged_decode_fp8(q, start, *cache, out=out, workspace=ws), cache)
        status = G.device_status(ws, clear=True)
        assert status == 2 or (status == 0 and not waits)
        if status == 0:
            check_decode(out, q, rows)
        assert (guard[[0, -1]] == 9.0).all()
        ws.zero_()
        G.paged_decode_fp8(q, start, *cache, out=out, workspace=ws)
        assert G.device_status(ws) == 0
        check_decode(out, q, rows)
    assert (guard[[0, -1]] == 9.0).all()


@pytest.mark.parametrize("heads,n_kv,prefix,members", [(32, 8, 40_000, 16), (16, 1, 100_000, 40)])
def test_waits_of_shared_rows(gen, heads, n_kv, prefix, members):
    """A prefix of many tiles a CTA: its products, softmaxes and copies wait for one another at each."""
    ws = G.make_paged_workspace()
    x = Batch(gen, n_kv, 64, [(prefix, [prefix + 30 * i for i in range(members)])])
    assert x.pays
    q = P.normal(gen, members, heads, P.D)
    guard = torch.full((members + 2, heads, P.D), 9.0, dtype=torch.bfloat16, device="cuda")
    out = guard[1:-1]
    for _ in range(3):
        given_up(lambda: G.paged_decode_shared(q, *x.args(), out=out, workspace=ws), (x.k_pages, x.v_pages))
        assert G.device_status(ws, clear=True) == 2
        assert (guard[[0, -1]] == 9.0).all()
        ws.zero_()
        G.paged_decode_shared(q, *x.args(), out=out, workspace=ws)
        assert G.device_status(ws) == 0
        x.check(out, q)
    assert (guard[[0, -1]] == 9.0).all()
