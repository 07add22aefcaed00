"""Routes at int32's ends through the MXFP4 product: what names no activation row reads the nearest one."""
import numpy as np
import pytest
import torch

import mxref
from gpu_util import dev, note
from quantized_expert_grouped_amd import abi

pytestmark = pytest.mark.gpu

STRAYS = [2 ** 31 - 1, 2 ** 30, 2 ** 30 - 1, -1, -2 ** 31, 7, 0, 2 ** 31 - 2, 1]


@pytest.mark.parametrize("K", [1, 3, 32, 64])
@pytest.mark.parametrize("rows,E,N", [(9, 1, 32), (400, 1, 2048), (9000, 1, 2048), (5000, 100, 2048), (6000, 40, 2048)])
def test_strays_of_every_size_read_the_nearest_row(rows, E, N, K):
    """The same bits as the product of the rows laid out one by one: the few-rows kernel and each tile."""
    k, n_act = 256, 5
    rng = np.random.default_rng(rows + K)
    g = torch.Generator(device="cuda").manual_seed(rows + K)
    wc = torch.randint(0, 256, (E, N, k // 2), dtype=torch.uint8, device="cuda", generator=g)
    ws = torch.randint(120, 126, (E, N, k // 32), dtype=torch.uint8, device="cuda", generator=g)
    ac, as_ = (dev(v) for v in mxref.encode(rng.standard_normal((n_act, k))))
    offsets = dev(np.linspace(0, rows, E + 1).astype(np.int32))
    route = np.resize(np.array(STRAYS, np.int64), rows)
    route[::5] = rng.integers(0, n_act * K, len(route[::5]))
    row = dev(np.clip(route, 0, None) // K).clamp(max=n_act - 1)
    note(f"mxfp4 strays rows={rows} E={E} N={N} K={K}")
    want, got = (torch.full((rows, N), 7.0, device="cuda") for _ in range(2))
    abi.mxfp4_mm_grouped(wc, ws, offsets, ac[row].contiguous(), as_[row].contiguous(), want)
    abi.mxfp4_mm_grouped(wc, ws, offsets, ac, as_, got, src=dev(route.astype(np.int32)), K=K)
    assert torch.equal(got, want) and bool(want.isfinite().all()) and not bool((want == 7.0).all())
