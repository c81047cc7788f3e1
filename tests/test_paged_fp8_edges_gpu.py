"""The 8-bit cache at the upper end of its range."""
import math

import pytest
import torch

import grouped_query_attention_gemv_gb300 as G
from tests import paged as P
from tests import paged8 as Q
from tests.test_paged_gpu import ints, offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ws():
    return G.make_paged_workspace()


@pytest.fixture
def gen():
    return torch.Generator(device="cuda").manual_seed(5)


def largest_rows(gen):
    """bf16 rows with their largest value from 2^120 to the type's own, 255 x 2^120."""
    tops = [m * 2.0 ** k for k in (120, 121, 124, 125, 126) for m in (1.0, 1.75, 1.7578125, 1.9921875)]
    tops += [m * 2.0 ** 120 for m in (128, 223, 224, 225, 239, 240, 241, 247, 248, 249, 254, 255)]
    rows = []
    for top in tops:
        x = torch.randn(128, generator=gen, device="cuda").double()
        x = x / x.abs().max() * top
        x[5], x[77], x[9] = top, -top, top * 0.97
        rows.append(x)
    return torch.stack(rows).bfloat16()[:, None]


def test_the_largest_values_stay_finite(gen, ws):
    """Every finite value is held within 2^-4 of itself, and what is held is a
    bf16: reading back is exact and finite."""
    v = largest_rows(gen)
    n = v.shape[0]
    assert torch.isfinite(v).all() and float(v.max()) == 255 * 2.0 ** 120
    *cache, table = Q.pages_of(gen, [n], 64, 1)
    still = torch.tensor([1.0, 0.0], device="cuda").expand(n, 64, 2).contiguous()   # keys stay as they are
    G.paged_append_fp8(None, v, v, ints([0]), still, *cache, table, cu_tokens=offsets([n]), workspace=ws)
    assert G.device_status(ws) == 0
    spot = P.slots(table, 64, 0, 0, n)
    e = Q.exponent(v.double())
    assert int(e.max()) == 120 and int(e.min()) <= 112
    units = Q.e4m3(v.double(), e)
    # 256 x 2^120 is past the largest float: the next value below is kept instead
    units = torch.where((e[..., None] == 120) & (units.abs() > 240), units.sign() * 240, units)
    k_out, v_out, to = P.pages_of(gen, [n], 16, 1)
    G.paged_read_fp8(ints([n]), *cache, table, k_out, v_out, to, workspace=ws)
    for pages, scales, out in ((cache[0], cache[2], k_out), (cache[1], cache[3], v_out)):
        assert torch.equal(scales[spot].int() - 127, e)
        held = pages.view(torch.uint8)[spot].view(torch.float8_e4m3fn)
        assert Q.same(held.float(), units)
        back = Q.values(held, scales[spot])
        assert ((back - v.double()).abs() <= torch.maximum(2.0 ** -4 * v.double().abs(),
                                                           2.0 ** -10 * Q.two_to(e)[..., None])).all()
        got = P.read_rows(out, to, 16, 0, n)
        assert torch.isfinite(got).all() and torch.equal(got.double(), back)


def test_rotated_keys_up_to_the_largest_float(gen, ws):
    """A rotation may take a key near 2^128 and past it: held as 240 x 2^120, and as NaN."""
    k = torch.zeros(3, 1, 128, dtype=torch.bfloat16, device="cuda")
    k[:, 0, 0] = 255 * 2.0 ** 120
    rope = torch.zeros(3, 64, 2, device="cuda")
    rope[..., 0] = 1.0
    rope[1, 0, 0] = 1.0039
    rope[2, 0, 0] = 1.01
    *cache, table = Q.pages_of(gen, [3], 16, 1)
    G.paged_append_fp8(None, k, torch.zeros_like(k), ints([0]), rope, *cache, table, cu_tokens=offsets([3]), workspace=ws)
    assert G.device_status(ws) == 0
    turned = Q.turned32(k, rope, False)[:, 0, 0]
    assert math.isfinite(turned[1]) and float(turned[1]) >= 255.9 * 2.0 ** 120 and turned[2] == math.inf
    spot = P.slots(table, 16, 0, 0, 3)
    held = cache[0].view(torch.uint8)[spot].view(torch.float8_e4m3fn).float()[:, 0, 0]
    assert held[:2].tolist() == [240.0, 240.0] and math.isnan(held[2])
    assert (cache[2][spot][:2].int() == 120 + 127).all()


@pytest.mark.parametrize("n", [1, 40])
def test_decode_over_the_largest_values(gen, ws, n):
    """Keys that count alike: the mean of the values, 240 x 2^120 at most."""
    heads = 4
    v = torch.zeros(n, 1, 128, dtype=torch.bfloat16, device="cuda")
    v[0, 0, :64], v[0, 0, 64:] = 255 * 2.0 ** 120, -250 * 2.0 ** 120
    *cache, table = Q.pages_of(gen, [n], 16, 1)
    G.paged_append_fp8(None, torch.zeros_like(v), v, ints([0]), G.rope_table(n), *cache, table, cu_tokens=offsets([n]),
                       workspace=ws)
    out = G.paged_decode_fp8(P.normal(gen, 1, heads, 128), ints([n - 1]), *cache, table, workspace=ws)
    assert G.device_status(ws) == 0
    want = 240 * 2.0 ** 120 / n
    assert torch.isfinite(out).all()
    assert ((out.double().abs() - want).abs() <= (P.BF16_HALF_STEP + 2.0 ** -10) * want).all()
    assert (out[..., :64] > 0).all() and (out[..., 64:] < 0).all()


@pytest.mark.parametrize("size", [1, 2 ** 4, 2 ** 6, 2 ** 8, 2 ** 10, 2 ** 12, 2 ** 20, 2 ** 50])
@pytest.mark.parametrize("heads,n_kv", [(8, 2), (16, 1)])
def test_scores_of_any_size(gen, ws, size, heads, n_kv):
    """Queries and keys of up to 2^50, values on scales 2^-3 to 2^3 of one another.
    Where one key has all the weight, its values come back as they are, but where
    the second is near: a score is 8 product steps of 17 x 2^-23 of its terms off,
    in sum some twice the largest score, below 2^-10 of it."""
    lens = [1, 40, 300, 5000, 2999, 17]
    (k_pages, v_pages, k_scales, v_scales, table), rows = Q.fill(gen, lens, 16, n_kv)
    k_scales.copy_((k_scales.int() + int(math.log2(size))).clamp(max=255).to(torch.uint8))
    q = P.normal(gen, len(lens), heads, P.D, scale=1.5 * size)
    out = G.paged_decode_fp8(q, ints([n - 1 for n in lens]), k_pages, v_pages, k_scales, v_scales, table, workspace=ws)
    assert G.device_status(ws) == 0 and torch.isfinite(out).all()
    alone = 0
    for b, (k, v) in enumerate(rows):
        for h in range(heads):
            g = h * n_kv // heads
            s = torch.sort((k[:, g] * size) @ q[b, h].double() * P.D ** -0.5, descending=True)
            top, second = float(s.values[0]), float(s.values[1]) if len(s.values) > 1 else -math.inf
            if top - second > 40 + abs(top) * 2.0 ** -10:
                # the others weigh e^-40 each at most: nothing beside a value, but not nothing beside 0
                tol = len(s.values) * math.exp(-40) * float(v.abs().max())
                assert float((out[b, h].double() - v[int(s.indices[0]), g]).abs().max()) <= tol, f"sequence {b}, head {h}"
                alone += 1
    assert alone >= heads and (size < 2 ** 6 or alone > 3 * heads)
