"""Gradients where a pool's tables on the device name fewer rows than the pool has."""
import pytest
import torch

import synthetic
from tests.gpu_helpers import f32_dev
from tests.requests_helpers import Batch

pytestmark = pytest.mark.gpu

q4 = pytest.importorskip("parameter_efficient_fine_nf4_b200")


def _poison(b):
    """Leaves NaN in the memory that the next tensors of these sizes get."""
    t = [torch.full((b.pool.rows, c), float("nan"), device="cuda") for c in (b.k, b.d)]
    torch.cuda.synchronize()
    del t


@pytest.mark.parametrize("layer", [False, True])
@pytest.mark.parametrize("lens", [[5, 9, 3], [150, 90, 40]])
def test_new_gradients_are_zero_in_rows_of_no_adapter(layer, lens):
    """Adapter 1 gets a smaller rank, adapter 2 an entry outside the pool: their other rows are nobody's."""
    k, d = 256, 192
    b = Batch(k, d, [8, 100, 40], lens, [0, 1, 2], seed=3)
    if layer:
        qw = q4.qlora_nf4_quantize(f32_dev(synthetic.custom_layer(seed=3, d=d, k=k, r=4, T=1, alpha=8.0).W0))
    b.pool.rank[1], b.pool.first[2] = 20, b.pool.rows
    U = torch.ones(b.T, b.pool.width, device="cuda")
    given = [torch.full((b.pool.rows, c), 7.0, device="cuda") for c in (k, d)]
    _poison(b)
    if layer:
        _, dA, dBt = q4.qlora_bwd_requests(qw, b.pool, b.plan, b.X, U, b.dY)
        q4.qlora_bwd_requests(qw, b.pool, b.plan, b.X, U, b.dY, dA=given[0], dBt=given[1])
    else:
        _, dA, dBt = q4.lora_requests_bwd(b.pool, b.plan, b.X, U, b.dY)
        q4.lora_requests_bwd(b.pool, b.plan, b.X, U, b.dY, dA=given[0], dBt=given[1])
    first = b.pool.firsts
    for g, left in zip((dA, dBt), given):
        for rows in (slice(first[0], first[0] + 8), slice(first[1], first[1] + 20)):
            assert bool(g[rows].any()) and torch.equal(g[rows], left[rows])
        assert not g[first[1] + 20:].any()
        assert not left[first[1] + 20:first[1] + 32].any()      # up to the next multiple of 16 they are the adapter's
        assert bool((left[first[1] + 32:] == 7.0).all())        # the caller's own arrays keep the rest
