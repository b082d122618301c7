"""The sums of U and G over the long side in the few-token kernels: exchanged
among the CTAs of a cluster, and their accuracy."""
import pytest
import torch

from tests.requests_helpers import Batch

pytestmark = pytest.mark.gpu

q4 = pytest.importorskip("parameter_efficient_fine_nf4_b200")


# the CTAs that share a tile follow from the number of tiles: one token each, so 16, 8, 4, 2 and 1 of them
@pytest.mark.parametrize("n", [4, 40, 100, 200, 300])
def test_sums_of_a_cluster_repeat_and_hold(n):
    """One token per adapter at a real width: every repeat of a chain of calls
    gives the same bits, and these hold the oracle's bounds."""
    b = Batch(k=4096, d=264, ranks=[(3, 8, 16, 21, 64)[a % 5] for a in range(n)], lens=[1] * n, ids=list(range(n)), seed=n,
              alphas=[16.0] * n)
    ws = q4.workspace(max(q4.lora_requests_fwd_workspace_bytes(b.pool, b.plan),
                          q4.lora_requests_bwd_workspace_bytes(b.pool, b.plan)))
    runs = []
    for _ in range(20):
        Y, U = q4.lora_requests_fwd(b.pool, b.plan, b.X, b.base_y, save=True, ws=ws)
        runs.append((Y, U) + q4.lora_requests_bwd(b.pool, b.plan, b.X, U, b.dY, b.base_x, ws=ws))
    torch.cuda.synchronize()
    assert q4.qlora_get_device_status() == 0
    for r in runs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(r, runs[0]))
    b.check_forward(*runs[0][:2])
    b.check_backward(*runs[0][2:], runs[0][1])
