"""Which batches share: the rows that sharing saves are those that it really does
not read, and the limits stand where they are documented."""
import pytest
import torch

import grouped_query_attention_gemv_gb300 as G
from tests import paged as P
from tests.test_paged_gpu import ints
from tests.test_paged_shared_gpu import Batch

pytestmark = pytest.mark.gpu

LEAST = 150_000   # saving as many cache rows x KV heads, a batch shares


@pytest.fixture(scope="module")
def ws():
    return G.make_paged_workspace()


@pytest.fixture
def gen():
    return torch.Generator(device="cuda").manual_seed(5)


def shares(gen, ws, x, heads, n_kv, plain_prefix):
    """Whether the batch gives other bits than with the prefixes `plain_prefix`."""
    q = P.normal(gen, len(x.starts), heads, P.D, scale=1.5)
    start, cu, prefix, *rest = x.args()
    out = G.paged_decode_shared(q, start, cu, prefix, *rest, workspace=ws)
    assert G.last_launch_count() == 2 and G.device_status(ws) == 0, "the host must not decide it"
    x.check(out, q)
    alone = G.paged_decode_shared(q, start, cu, ints(plain_prefix), *rest, workspace=ws)
    assert G.last_launch_count() == 2 and G.device_status(ws) == 0
    return not torch.equal(out, alone)


def spread(slots, members, start):
    """Start positions of a group of `slots`, of which `members` are in use."""
    s = [-1] * slots
    for i, at in enumerate(members):
        s[at] = start + 3 * i
    return s


@pytest.mark.parametrize("heads,n_kv,slots,members,prefix", [
    (32, 8, 2048 * 14 // 32, [0, 895], 20_000),      # 14 pairs of Q tiles would read what two sequences read
    (4, 4, 2048, [0, 2047], 40_000),
    (16, 1, 64, [0, 30, 63], 80_000),                # 16 sequences in a pair: four reads for three
    (16, 1, 64, [0, 20, 40, 63], 60_000),            # four for four: nothing is saved
    (8, 2, 300, list(range(0, 300, 64)), 30_000)])
def test_few_members_in_a_large_group_do_not_share(gen, ws, heads, n_kv, slots, members, prefix):
    x = Batch(gen, n_kv, 64, [(prefix, spread(slots, members, prefix))])
    assert not shares(gen, ws, x, heads, n_kv, [0])


@pytest.mark.parametrize("heads,n_kv,slots,members,prefix", [
    (32, 8, 896, range(500, 520), 2000),             # side by side: one pair of Q tiles
    (32, 8, 896, range(876, 896), 2000),
    (16, 1, 64, range(23, 39), 15_000),              # 16: one pair, although they lie in two of the group's
    (16, 1, 64, [3, 40, 41, 42, 63, 5], 90_000),     # four reads for six
    (8, 2, 300, [0, 299] + list(range(100, 160)), 8000)])
def test_members_side_by_side_share(gen, ws, heads, n_kv, slots, members, prefix):
    x = Batch(gen, n_kv, 64, [(prefix, spread(slots, members, prefix))])
    assert shares(gen, ws, x, heads, n_kv, [0])


def test_each_group_by_itself(gen, ws):
    """A group that pays beside ones that do not: those are attended one by one."""
    groups = [(9000, spread(130, [1, 66, 129], 9000)), (6000, [6000 + 5 * i for i in range(20)]),
              (7000, spread(70, [0, 69], 7001)), (4000, [4100, -1, 30])]
    x = Batch(gen, 2, 64, groups)
    assert shares(gen, ws, x, 8, 2, [0, 0, 0, 0])
    assert not shares(gen, ws, x, 8, 2, [0, 6000, 0, 0])
    # two read side by side: one of them is saved
    groups[2] = (7000, spread(70, [30, 31], 7001))
    assert shares(gen, ws, Batch(gen, 2, 64, groups), 8, 2, [0, 6000, 0, 0])


@pytest.mark.parametrize("n_kv,members,prefix", [(2, 16, 5000), (1, 2, 150_000), (8, 11, 1875)])
def test_the_threshold_lies_where_it_is_documented(gen, ws, n_kv, members, prefix):
    assert prefix * (members - 1) * n_kv == LEAST
    for p, shared in ((prefix, True), (prefix - 1, False)):
        x = Batch(gen, n_kv, 64, [(p, [p + 7 * i for i in range(members)])])
        assert shares(gen, ws, x, 4 * n_kv, n_kv, [0]) == shared


def test_more_groups_than_are_looked_at_although_they_would_pay(gen, ws):
    """1,024 groups share, of 1,025 none does: the batch is past the host's first look in both."""
    groups = [(200, [203, 207])] * 1023
    x = Batch(gen, 1, 16, groups + [(200, [204])])
    assert shares(gen, ws, x, 1, 1, [0] * 1024)
    x = Batch(gen, 1, 16, groups + [(200, [204]), (200, [205])])
    q = P.normal(gen, 2048, 1, P.D)
    out = G.paged_decode_shared(q, *x.args(), workspace=ws)
    assert G.last_launch_count() == 1 and G.device_status(ws) == 0
    assert torch.equal(out, G.paged_decode(q, ints(x.starts), x.k_pages, x.v_pages, x.table, workspace=ws))
