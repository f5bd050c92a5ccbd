"""The weight gradient's bound tells a sum that lost rows from one that did not."""
import pytest
import torch

from tests import feature_ref as ref
from tests.feature_bounds import weight_grad_bound


def _terms(rows, c):
    g = torch.Generator().manual_seed(rows + c)
    h, dy = (torch.randn(rows, c, generator=g, dtype=torch.float64) for _ in range(2))
    return dy * h * ref.rms_norm(h, None, 1e-6)[1][:, None]


@pytest.mark.parametrize("rows,c", [(300_000, 16), (40_001, 128), (9_001, 1000), (5_003, 500), (2_500, 7)])
def test_bound_sees_lost_rows(rows, c):
    """One thread's rows (a 1024th), a round of 1024 parts counted twice, and up to 40001 rows the last row
    alone (of 300000 one row is as large as the roundings of the rest): each is seen in some channel."""
    t = _terms(rows, c)
    want, bound = t.sum(0), weight_grad_bound(t.abs().sum(0), rows)
    each = -(-rows // 1024)
    wrong = [want - t[:each].sum(0), want - t[-each:].sum(0), want + t[:1024].sum(0)]
    if rows <= 40_001:
        wrong.append(want - t[-1])
    for sums in wrong:
        assert bool(((sums - want).abs() > bound).any())


@pytest.mark.parametrize("rows,c", [(300_000, 16), (5_003, 64)])
def test_bound_holds_for_a_sum_in_parts(rows, c):
    """1024 parts of a float sum each, then the parts in slices of 32."""
    t = _terms(rows, c)
    pad = -rows % 1024
    f = torch.cat([t.float(), torch.zeros(pad, c)]).view(-1, 1024, c)
    acc = torch.zeros(1024, c)
    for row in f:
        acc += row
    slices = torch.zeros(32, c)
    for part in acc.view(32, 32, c):
        slices += part
    got = torch.zeros(c)
    for s in slices:
        got += s
    assert bool(((got.double() - t.sum(0)).abs() <= weight_grad_bound(t.abs().sum(0), rows)).all())
