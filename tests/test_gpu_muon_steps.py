"""The orthogonalised step on momenta with fewer directions than rows, at the
largest number of steps that the entry point takes."""
import numpy as np
import pytest
import torch

from oracle import muon

pytestmark = pytest.mark.gpu

q4 = pytest.importorskip("parameter_efficient_fine_nf4_b200")

USUAL, STEEP = muon.COEFS, (4.0848, -6.8946, 2.9270)


def _deficient(kind, r, long, seed):
    gen = np.random.Generator(np.random.Philox(key=seed))
    v = gen.standard_normal((r, long))
    if kind == "rank 1":
        v = np.outer(v[:, 0], v[0])
    elif kind == "rank 3":
        v = v[:, :3] @ v[:3]
    elif kind == "rows repeated":
        v[r // 2:] = v[:r - r // 2]
    elif kind == "zero rows":
        v[2:] = 0.0
    return v.astype(np.float32)


@pytest.mark.parametrize("kind", ["rank 1", "rank 3", "rows repeated", "zero rows"])
@pytest.mark.parametrize("r,long,tall", [(16, 4096, False), (40, 300, True), (64, 1024, False), (96, 520, True), (200, 400, False)])
@pytest.mark.parametrize("coefs,steps", [(USUAL, 5), (USUAL, 8), (STEEP, 7)])
def test_fewer_directions_than_rows(kind, r, long, tall, coefs, steps):
    """momentum = 0 and no Nesterov term: u is the gradient itself, without a
    rounding, so all that is left is the 64-bit arithmetic of r x r matrices and
    one rounding each of x and of the master."""
    g = _deficient(kind, r, long, r + steps)
    g = np.ascontiguousarray(g.T) if tall else g
    W = torch.zeros(g.shape, device="cuda")
    w16 = W.to(torch.bfloat16)
    q4.lora_muon_step(W, w16, torch.zeros_like(W), torch.from_numpy(g).cuda(), lr=1.0, momentum=0.0, nesterov=False,
                      coefs=coefs, steps=steps)
    torch.cuda.synchronize()
    assert q4.qlora_get_device_status() == 0
    co = tuple(float(np.float32(c)) for c in coefs)
    want = muon.orthogonalise(g, steps, co, float(np.float32(1e-7)))
    # x and the master are rounded to 32 bits (2^-24 each); beyond that, what the limit on the steps promises: the
    # recursion on the Gram matrix, in numpy and 64 bits, is at most 2e-9 from the iteration on the matrix itself at
    # these steps, and 1e-4 to 1e76 at more of them
    err = np.abs(-W.double().cpu().numpy() - want)
    assert np.all(err <= 2 * 2.0 ** -24 * np.abs(want) + 2.0 ** -26), float(err.max())
