"""The checks of the paged operators' tests see a part that is lost or taken
twice (planted in the reference, on the CPU)."""
import pytest
import torch

from tests import paged as P


def cache(n, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return [torch.randn(m, h, P.D, generator=gen).bfloat16() for m, h in ((1, 2), (n, 1), (n, 1))]


@pytest.mark.parametrize("n,at,lost", [(70001, 30000, 148), (70001, 69853, 148), (60008, 128 * 100, 128), (4000, 16, 16)])
def test_mean_error_sees_a_lost_part(n, at, lost):
    q, k, v = cache(n)
    ref = P.attend64(q, k, v, n - 1)[0]
    P.check_l2(ref.bfloat16(), ref, "all of it")
    keep = [i for i in range(n) if not at <= i < at + lost]
    with pytest.raises(AssertionError, match="off by"):
        P.check_l2(P.attend64(q, k[keep], v[keep], len(keep) - 1)[0].bfloat16(), ref, "a part less")


@pytest.mark.parametrize("n", [1, 16, 2048, 2049, 9001, 70001])
def test_counts_see_one_key(n):
    weights = torch.full((n,), 1.0 / n, dtype=torch.float64)
    for window in {0, (n - 1) // 4096, (n - 1) // P.CODE_WINDOW}:
        v = P.coded_values(n, window, "cpu").double()
        P.check_counts((weights @ v).bfloat16()[None, None], window, n - 1, "all of them")
        at = window * P.CODE_WINDOW
        for key in {at, min(n, at + 17) - 1, min(n, at + P.CODE_WINDOW) - 1}:
            for factor in (0.0, 2.0):
                w = weights.clone()
                w[key] *= factor
                with pytest.raises(AssertionError, match="counts are wrong"):
                    P.check_counts((w @ v).bfloat16()[None, None], window, n - 1, "one of them")


def test_counts_of_causal_rows():
    first, t = 2040, 30
    for window in (0, 1):
        v = P.coded_values(first + t, window, "cpu").double()
        rows = [v[:first + i + 1].mean(0) for i in range(t)]
        P.check_counts(torch.stack(rows)[:, None].bfloat16(), window, first, "each row")
        rows[7] = v[:first + 9].mean(0)
        if window == 1:
            with pytest.raises(AssertionError, match="counts are wrong"):
                P.check_counts(torch.stack(rows)[:, None].bfloat16(), window, first, "one key early")
