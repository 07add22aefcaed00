"""The balance loss and its gradient on rows at any address and stride: the same values give the same bits."""
import pytest
import torch

from gpu_util import note
from test_gpu_9_balance import DT, case, check, run

pytestmark = pytest.mark.gpu


def rows_at(x, skip, gap):
    """x's values in rows `gap` elements apart, the first one `skip` elements past an aligned address."""
    T, E = x.shape
    whole = torch.full((T * (E + gap) + skip + 8,), 9.0, device="cuda", dtype=x.dtype)
    rows = whole[skip:skip + T * (E + gap)].view(T, E + gap)[:, :E]
    rows.copy_(x)
    return whole, rows


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("T,E,K", [(300, 512, 10), (65, 128, 4), (40, 96, 3), (33, 2048, 8), (50, 130, 2),
                                   (7, 1000, 5), (90, 8, 2)])
def test_bits_do_not_depend_on_addresses_or_strides(T, E, K, dtype):
    """Sums are in an order that depends on the sizes alone, so every output of rows with gaps and odd
    addresses, and the gradient into such rows or over the logits, is that of contiguous ones bit for bit."""
    x, idx, v = case(T, E, K, "some", 5 * E, spread=3.0)
    xt = torch.from_numpy(x).cuda().to(DT[dtype])
    want = run(xt, idx, v, 3.0)
    check(xt, idx, v, dtype, 3.0, want)
    for skip, gap in ((1, 0), (0, 1), (1, 3), (2, 6), (3, 8), (4, 4)):
        note(f"rows {skip} past, {gap} apart")
        whole, rows = rows_at(xt, skip, gap)
        gwhole, grad = rows_at(torch.zeros_like(xt), gap, skip)
        got = run(rows, idx, v, 3.0, grad)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), (skip, gap)
        before = whole.clone()
        got = run(rows, idx, v, 3.0, rows)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), ("in place", skip, gap)
        for w, r, old in ((whole, rows, before), (gwhole, grad, torch.full_like(gwhole, 9.0))):
            keep = w.clone()                                    # what is not a row keeps its values
            keep[r.storage_offset():r.storage_offset() + T * r.stride(0)].view(T, -1)[:, :E] = 0
            r0 = old.clone()
            r0[r.storage_offset():r.storage_offset() + T * r.stride(0)].view(T, -1)[:, :E] = 0
            assert torch.equal(keep, r0)
    # the gradient's own layout alone
    for skip, gap in ((1, 0), (3, 5)):
        _, grad = rows_at(torch.zeros_like(xt), skip, gap)
        assert torch.equal(run(xt, idx, v, 3.0, grad)[3], want[3])
