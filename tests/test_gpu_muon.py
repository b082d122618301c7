"""GPU parity of the orthogonalised optimiser step with the float64 oracle."""
import numpy as np
import pytest
import torch

from oracle import muon

pytestmark = pytest.mark.gpu

q4 = pytest.importorskip("parameter_efficient_fine_nf4_b200")

F32, BF16 = 2.0 ** -24, 2.0 ** -8


def _inputs(n, rows, cols, seed, spread=30.0):
    """Gradients whose singular values fall from 1 to 1 / spread."""
    gen = np.random.Generator(np.random.Philox(key=seed))
    r, long = min(rows, cols), max(rows, cols)
    fall = np.geomspace(1.0, 1.0 / spread, r)
    g = np.stack([(gen.standard_normal((r, r)) * fall) @ gen.standard_normal((r, long)) for _ in range(n)]) * 1e-3
    g = g.transpose(0, 2, 1) if rows > cols else g
    m = g * gen.standard_normal((n, 1, 1)) + 1e-4 * gen.standard_normal((n, rows, cols))
    W = 0.02 * gen.standard_normal((n, rows, cols))
    return [np.ascontiguousarray(v, dtype=np.float32) for v in (W, m, g)]


def _run(W, m, g, **kw):
    d = [torch.from_numpy(v.copy()).cuda() for v in (W, m, g)]
    w16 = torch.zeros(W.shape, dtype=torch.bfloat16, device="cuda")
    q4.lora_muon_step(d[0], w16, d[1], d[2], **kw)
    torch.cuda.synchronize()
    assert torch.equal(d[2].cpu().view(torch.int32), torch.from_numpy(g).view(torch.int32))
    return d[0].double().cpu().numpy(), d[1].double().cpu().numpy(), w16


def _check(n, rows, cols, seed=0, **kw):
    kw = dict(dict(lr=0.05, momentum=0.9, nesterov=True, scale=0.3, weight_decay=0.1), **kw)
    W, m, g = _inputs(n, rows, cols, seed)
    got, gm, w16 = _run(W, m, g, **kw)
    f = {k: float(np.float32(v)) for k, v in kw.items() if isinstance(v, float)}
    for i in range(n):
        rW, rm, x = muon.step(W[i], m[i], g[i], **{**kw, **f})
        # m: one multiply-add
        assert np.all(np.abs(gm[i] - rm) <= 2 * F32 * np.abs(rm) + 1e-40)
        # x: u is rounded to 32 bits (two multiply-adds, 2^-23 of |u| in the Frobenius norm), which the iterations
        # raise by at most the product of the quintic's slope at zero, 3.4445^steps; then one rounding of x and two of
        # the master
        raised = abs((kw.get("coefs") or muon.COEFS)[0]) ** kw.get("steps", 5)
        tol = f["lr"] * abs(f["scale"]) * (2 * raised * 2.0 ** -23) + 4 * F32 * (np.abs(rW) + np.abs(W[i]))
        assert np.all(np.abs(got[i] - rW) <= tol), float((np.abs(got[i] - rW) / tol).max())
    master = torch.from_numpy(got).float()
    assert torch.equal(w16.cpu(), master.to(torch.bfloat16))


@pytest.mark.parametrize("n,rows,cols", [
    (1, 1, 1), (1, 1, 300), (1, 300, 1), (2, 8, 8), (3, 5, 77), (1, 16, 4096), (2, 64, 1000), (1, 64, 64), (2, 1000, 64),
    (1, 65, 130), (1, 130, 65), (1, 100, 2001), (3, 2001, 17), (1, 256, 300), (1, 300, 256), (1, 256, 256), (20, 8, 256)])
def test_against_the_oracle(n, rows, cols):
    _check(n, rows, cols, seed=rows + cols)


@pytest.mark.parametrize("kw", [dict(nesterov=False), dict(weight_decay=0.0), dict(momentum=0.0), dict(steps=1),
                                dict(steps=3, coefs=(3.0, -16.0 / 5.0, 6.0 / 5.0)), dict(lr=0.0), dict(scale=-2.0)])
def test_options(kw):
    _check(2, 24, 200, seed=3, **kw)


def test_matrices_of_a_stack_do_not_mix():
    W, m, g = _inputs(3, 16, 500, 5)
    m[1], g[1] = 0.0, 0.0                    # a zero update only decays
    kw = dict(lr=0.05, weight_decay=0.1, scale=0.3)
    got, gm, _ = _run(W, m, g, **kw)
    keep = np.float32(1.0 - float(np.float32(0.05)) * float(np.float32(0.1)))
    assert np.array_equal(got[1], (W[1] * keep).astype(np.float32).astype(np.float64)) and not gm[1].any()
    g[1] = np.nan
    bad, _, _ = _run(W, m, g, **kw)
    assert np.array_equal(bad[[0, 2]], got[[0, 2]])
    for i in (0, 2):                         # alone, up to the order of the long side's sums
        one, _, _ = _run(W[i], m[i], g[i], **kw)
        assert np.allclose(one, got[i], rtol=0, atol=1e-6)


def test_orthogonal_result_and_repeats():
    """On a well-conditioned matrix the step's direction has singular values
    near 1, whatever the gradient's size; repeats are bit-identical."""
    for size in (1e-20, 1.0, 1e15):
        W, m, g = _inputs(1, 32, 700, 9, spread=3.0)
        W[:], m[:] = 0.0, 0.0
        g = (g * size).astype(np.float32)
        runs = [_run(W, m, g, lr=1.0, momentum=0.0, eps=1e-30) for _ in range(2)]
        assert np.array_equal(runs[0][0], runs[1][0])
        sv = np.linalg.svd(runs[0][0][0], compute_uv=False)
        assert np.all((sv > 0.6) & (sv < 1.3))


def test_captured_beside_another_shape():
    W, m, g = _inputs(2, 16, 640, 21)
    d = [torch.from_numpy(v.copy()).cuda() for v in (W, m, g)]
    w16 = torch.zeros(W.shape, dtype=torch.bfloat16, device="cuda")
    ws = q4.workspace(q4.lora_muon_workspace_bytes(2, 16, 640))
    q4.lora_muon_step(d[0], w16, d[1], d[2], lr=0.1, ws=ws)
    for t, v in zip(d, (W, m, g)):
        t.copy_(torch.from_numpy(v))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q4.lora_muon_step(d[0], w16, d[1], d[2], lr=0.1, ws=ws)
    for t, v in zip(d, (W, m, g)):
        t.copy_(torch.from_numpy(v))
    graph.replay()
    torch.cuda.synchronize()
    ref, rm, _ = _run(W, m, g, lr=0.1)
    assert np.array_equal(d[0].double().cpu().numpy(), ref) and np.array_equal(d[1].double().cpu().numpy(), rm)


def test_an_empty_stack_is_nothing_to_do():
    W = torch.zeros(0, 4, 64, device="cuda")
    q4.lora_muon_step(W, W.to(torch.bfloat16), W, W, lr=0.1)


def test_refusals_of_the_binding():
    W = torch.zeros(4, 64, device="cuda")
    w16 = W.to(torch.bfloat16)
    with pytest.raises(TypeError):
        q4.lora_muon_step(W.double(), w16, W, W, lr=0.1)
    with pytest.raises(ValueError):
        q4.lora_muon_step(W, w16[:2], W, W, lr=0.1)
    with pytest.raises(ValueError):
        q4.lora_muon_step(W.cpu(), w16, W, W, lr=0.1)
    with pytest.raises(ValueError):
        q4.lora_muon_step(W, w16, W, W, lr=0.1, coefs=(1.0, 2.0))
    with pytest.raises(q4.QloraError):
        q4.lora_muon_step(W, w16, W, W, lr=-0.1)
    with pytest.raises(q4.QloraError):
        big = torch.zeros(300, 300, device="cuda")
        q4.lora_muon_step(big, big.to(torch.bfloat16), big, big, lr=0.1)
