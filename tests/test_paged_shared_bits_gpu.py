"""Decode attention with shared rows: shared rows count with the bits that the
decode attention keeps, whoever the neighbours of a sequence are."""
import math

import pytest
import torch

import grouped_query_attention_gemv_gb300 as G
from tests import paged as P
from tests.test_paged_gpu import LAYOUTS, ints
from tests.test_paged_shared_gpu import Batch, enough

pytestmark = pytest.mark.gpu

# What is off by a share e of the output's size before its rounding to bf16 (a
# step is 2^-7 of a value at most) is rounded to another neighbour with
# probability e x size / step, and is then off by a step: in the mean square by
# 2^-7 e + e^2 at most. Probabilities as two bf16 terms are off by 2^-15 each,
# independent of one another, scores and sums by less: e <= 2^-13 leaves four
# times that and gives 2^-10. One term (0.0015 in the mean square) gives 0.0023.
BAR = 2.0 ** -10


@pytest.fixture(scope="module")
def ws():
    return G.make_paged_workspace()


@pytest.fixture
def gen():
    return torch.Generator(device="cuda").manual_seed(5)


def off(got, refs):
    """Of whole outputs, how far they are from the rounded references."""
    d = sum(float((g.double() - r.bfloat16().double()).square().sum()) for g, r in zip(got, refs))
    return math.sqrt(d / sum(float(r.square().sum()) for r in refs))


@pytest.mark.parametrize("heads,n_kv", LAYOUTS + [(16, 1), (9, 1), (24, 2)])
@pytest.mark.parametrize("prefix,members", [(5000, 20), (8191, 70)])
def test_shared_rows_keep_the_bits_of_the_decode(gen, ws, heads, n_kv, prefix, members):
    if n_kv == 32:
        members = 8
    prefix = max(prefix, enough(n_kv, members))
    x = Batch(gen, n_kv, 64, [(prefix, [prefix - 1 + 5 * i for i in range(members)])])
    assert x.pays
    q = P.normal(gen, members, heads, P.D, scale=1.5)
    refs = [P.attend64(q[b:b + 1], k, v, k.shape[0] - 1)[0] for b, (k, v) in enumerate(x.rows)]
    args = x.args()
    plain = G.paged_decode(q, args[0], *args[3:], workspace=ws)
    assert off(plain.split(1), refs) <= BAR
    shared = G.paged_decode_shared(q, *args, workspace=ws)
    assert G.last_launch_count() == 2 and G.device_status(ws) == 0
    assert off(shared.split(1), refs) <= BAR


@pytest.mark.parametrize("below", [0, 7, 60, 100, 104, 112, 120, 124])
def test_an_infinite_value_of_little_weight_is_an_infinity(gen, ws, below):
    """A shared row whose score is that many powers of two below the largest, and
    with values of plus and minus infinity: they show as in the decode attention."""
    p, B = 5440, 20
    x = Batch(gen, 2, 64, [(p, [p + 3 * i for i in range(B)])])
    assert x.pays
    q = torch.zeros(B, 8, P.D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    scale = math.log(2.0)   # scores in powers of two
    x.k_pages.copy_(torch.nan_to_num(x.k_pages))
    x.k_pages[..., 0] = -16.0
    page, row = P.slots(x.table, 64, 0, 5, 1)
    x.k_pages[page, row, :, 0] = 0.0        # the largest score, in the first tile of keys
    for at, value, dim in ((700, math.inf, 9), (701, -math.inf, 60)):
        page, row = P.slots(x.table, 64, 0, at, 1)
        x.k_pages[page, row, :, 0] = float(-below)
        x.v_pages[page, row, 1, dim] = value
    args = x.args()
    plain = G.paged_decode(q, args[0], *args[3:], scale=scale, workspace=ws)
    out = G.paged_decode_shared(q, *args, scale=scale, workspace=ws)
    assert G.last_launch_count() == 2 and G.device_status(ws) == 0
    for o in (plain, out):
        assert (o[:, 4:, 9] == math.inf).all() and (o[:, 4:, 60] == -math.inf).all()
        o[:, 4:, [9, 60]] = 0.0
        assert torch.isfinite(o).all()


@pytest.mark.parametrize("size", [2.0 ** 8, 2.0 ** 12, 2.0 ** 14, 2.0 ** 15, 2.0 ** 20, 2.0 ** 50])
def test_scores_of_any_size(gen, ws, size):
    """Queries and keys of up to 2^50: one key has all the weight, its values come
    back as they are, but where the second is near: a score is 8 product steps of
    17 x 2^-23 of its terms off, in sum some twice the largest score, below 2^-10 of it."""
    p = 6000
    x = Batch(gen, 2, 64, [(p, [p + 5 * i for i in range(18)])])
    assert x.pays
    q = P.normal(gen, 18, 8, P.D, scale=size)
    k_pages = (x.k_pages.float() * size).bfloat16()
    start, cu, prefix, _, *rest = x.args()
    out = G.paged_decode_shared(q, start, cu, prefix, k_pages, *rest, workspace=ws)
    assert G.last_launch_count() == 2 and G.device_status(ws) == 0
    for b, (k, v) in enumerate(x.rows):
        for h in range(8):
            s = (k[:, h // 4].double() * size) @ q[b, h].double() * P.D ** -0.5
            top = s.topk(2)
            if float(top.values[0] - top.values[1]) > 40 + float(top.values[0]) * 2.0 ** -10:
                assert torch.equal(out[b, h], v[int(top.indices[0]), h // 4]), f"sequence {b}, head {h}"
    assert torch.isfinite(out).all()
