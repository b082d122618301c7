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


def _one_sided(a, b, rows):
    """Mean of (a - b) / b over all entries, and the largest, in float64."""
    e = (a.double() - b)[rows] / b[rows]
    return abs(float(e.mean())), float(e.abs().max())


@pytest.mark.parametrize("wide", ["k", "d"])
def test_long_sums_do_not_drift(wide):
    """Sums of one sign over 65536 columns, one CTA per tile (so one CTA adds all
    of them): U, and through G the gradient dA, stay within a few 1e-6.

    The tensor core may cut each of the 32 additions of a piece of 32 columns by
    a whole step of 32 bits: 32 * 2^-23 = 3.8e-6, always towards zero.  Between
    the pieces the additions round to nearest, which is centred: 256 a warp and
    7 of the warps, each off by at most 2^-24 of what was added up so far.  Their
    mean over more than 250 entries is below 263 * 2^-24 / 250^0.5 = 1.0e-6
    (the roots of independent errors add up to less), their worst below
    263 * 2^-24 = 1.6e-5."""
    n, K, N = 280, 65536, 64
    k, d = (K, N) if wide == "k" else (N, K)
    pool = q4.AdapterPool(k, d, [1] * n, [1.0] * n)
    gen = torch.Generator(device="cuda").manual_seed(5)

    def positive(*shape):
        return (torch.rand(*shape, generator=gen, device="cuda") + 0.5).to(torch.bfloat16)

    pool.A[::16], pool.Bt[::16] = positive(n, k), positive(n, d)
    X, dY = positive(n, k), positive(n, d)
    lens = torch.ones(n, dtype=torch.int32, device="cuda")
    ids = torch.arange(n, dtype=torch.int32, device="cuda")
    plan = q4.lora_requests_plan(lens, ids, q4.RequestPlan(n, n, n))
    Y, U = q4.lora_requests_fwd(pool, plan, X, save=True)
    dX, dA, dBt = q4.lora_requests_bwd(pool, plan, X, U, dY)
    torch.cuda.synchronize()
    assert q4.qlora_get_device_status() == 0
    want_u = (X.double() * pool.A[::16].double()).sum(1, keepdim=True)
    want_g = (dY.double() * pool.Bt[::16].double()).sum(1, keepdim=True)
    every = slice(None)
    got = {"k": [(U[:, :1], want_u)], "d": [(dA[::16], want_g * X.double())]}[wide]
    for value, exact in got:
        mean, worst = _one_sided(value, exact, every)
        assert mean <= 3.8e-6 + 1.0e-6 and worst <= 3.8e-6 + 1.6e-5, (mean, worst)
    # the other sums of the same calls: 64 columns, then one product
    mean, worst = _one_sided(U[:, :1], want_u, every)
    assert worst <= 3.8e-6 + 1.6e-5
    mean, worst = _one_sided(dBt[::16], U[:, :1].double() * dY.double(), every)
    assert worst <= 2.0 ** -23
