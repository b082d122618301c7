"""Pins of the many-adapter and orthogonalised-step oracles (CPU), and the
refusals of their entry points, which need no device."""
import ctypes

import numpy as np
import pytest

from oracle import lora, muon
from oracle import requests as req

rng = np.random.Generator(np.random.Philox(key=20))


def _stack(k, d, ranks):
    return ([rng.standard_normal((r, k)) for r in ranks], [rng.standard_normal((d, r)) for r in ranks],
            [0.5 + i for i in range(len(ranks))])


def test_plan_by_hand():
    p = req.plan([2, 0, 3, -4, 1], [1, 0, 0, 1, 7], 2, 8)
    assert p["starts"].tolist() == [0, 2, 2, 5, 5, 6]
    assert p["idx"].tolist() == [1, 1, 0, 0, 0, -1, -1, -1]
    assert p["order"].tolist() == [2, 3, 4, 0, 1, 5, -1, -1]
    assert p["seg"].tolist() == [0, 3, 5, 6]
    cut = req.plan([5, 5], [0, 1], 2, 7)
    assert cut["starts"].tolist() == [0, 5, 7] and cut["seg"].tolist() == [0, 5, 7, 7]


def test_equal_ranks_reduce_to_the_stacked_oracle():
    k, d, r, n, T = 24, 16, 3, 4, 19
    A, B, s = _stack(k, d, [r] * n)
    idx = rng.integers(0, n, T).astype(np.int32)
    X, dY = rng.standard_normal((T, k)), rng.standard_normal((T, d))
    W = rng.standard_normal((d, k))
    fw = req.forward(X, A, B, s, idx, X @ W.T)
    ref = lora.forward_multi(X, W, np.stack(A), np.stack(B), np.array(s), idx)
    assert np.allclose(fw["Y"], ref["Y"]) and np.allclose(fw["U"], ref["U"])
    bw = req.backward(X, A, B, s, idx, fw["U"], dY, dY @ W)
    rb = lora.backward_multi(X, W, np.stack(A), np.stack(B), np.array(s), idx, dY)
    assert np.allclose(bw["dX"], rb["dX"])
    assert np.allclose(np.stack(bw["dA"]), rb["dA"]) and np.allclose(np.stack(bw["dB"]), rb["dB"])


def test_gradients_against_differences():
    k, d, T = 11, 7, 9
    A, B, s = _stack(k, d, [2, 5])
    idx = np.array([0, 1, 1, -1, 0, 1, 0, -1, 1], np.int32)
    X, dY = rng.standard_normal((T, k)), rng.standard_normal((T, d))

    def loss(X, A, B):
        return float((req.forward(X, A, B, s, idx)["Y"] * dY).sum())

    bw = req.backward(X, A, B, s, idx, req.forward(X, A, B, s, idx)["U"], dY)
    h = 1e-6
    V = rng.standard_normal(X.shape)
    assert np.isclose((loss(X + h * V, A, B) - loss(X - h * V, A, B)) / (2 * h), (bw["dX"] * V).sum(), rtol=1e-6)
    for i in range(2):
        for which, grad in ((A, bw["dA"][i]), (B, bw["dB"][i])):
            V = rng.standard_normal(grad.shape)
            up, down = [v.copy() for v in which], [v.copy() for v in which]
            up[i], down[i] = up[i] + h * V, down[i] - h * V
            args = ((up, B), (down, B)) if which is A else ((A, up), (A, down))
            diff = (loss(X, *args[0]) - loss(X, *args[1])) / (2 * h)
            assert np.isclose(diff, (grad * V).sum(), rtol=1e-6)


@pytest.mark.parametrize("shape", [(4, 9), (9, 4), (5, 5), (1, 7)])
def test_orthogonalise_acts_on_singular_values_alone(shape):
    u = rng.standard_normal(shape)
    U, sv, Vh = np.linalg.svd(u, full_matrices=False)
    sv = sv / (np.linalg.norm(u) + 1e-7)
    a, b, c = muon.COEFS
    for _ in range(5):
        sv = a * sv + b * sv ** 3 + c * sv ** 5
    assert np.allclose(muon.orthogonalise(u), (U * sv) @ Vh, atol=1e-12)
    assert np.all((sv > 0.6) & (sv < 1.3))        # where the quintic drives values that are not tiny


def test_zero_momentum_only_decays():
    W, m, x = muon.step(np.ones((3, 5)), np.zeros((3, 5)), np.zeros((3, 5)), 0.1, weight_decay=0.5)
    assert np.allclose(W, 0.95) and not m.any() and not x.any()


# ------------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def q4():
    import parameter_efficient_fine_nf4_b200 as q4
    from parameter_efficient_fine_nf4_b200 import build
    build.build()
    return q4


def _pool(q4, **v):
    f = dict(A=16, Bt=16, first=16, rank=16, scale=16, rows=64, k=256, d=256, n=4, width=16)
    f.update(v)
    return q4._Pool(*(f[name] for name, _ in q4._Pool._fields_))


def _req(q4, **v):
    f = dict(starts=16, idx=16, order=16, seg=16, tile_first=16, tiles=16, T=8, n_req=2, n=4)
    f.update(v)
    return q4._Requests(*(f[name] for name, _ in q4._Requests._fields_))


@pytest.mark.parametrize("over,status", [
    (dict(k=100), 2), (dict(d=12), 2), (dict(width=24), 2), (dict(width=272), 2), (dict(width=0), 2), (dict(rows=8), 2),
    (dict(rows=24), 2), (dict(n=5), 1), (dict(A=None), 1), (dict(Bt=None), 1), (dict(first=None), 1), (dict(rank=None), 1),
    (dict(scale=None), 1), (dict(A=18), 3), (dict(Bt=24), 3), (dict(k=0), 2), (dict(d=1 << 25), 2)])
def test_pool_refusals(q4, over, status):
    p, r = _pool(q4, **over), _req(q4)
    L = q4.lib()
    assert L.lora_requests_fwd(ctypes.byref(p), ctypes.byref(r), 16, 16, 16, 16, 16, 1 << 30, None) == status
    assert L.lora_requests_bwd(ctypes.byref(p), ctypes.byref(r), 16, 16, 16, 16, 16, 16, 16, 16, 1 << 30, None) == status


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), 1), (dict(n_req=-1), 1), (dict(n=0), 1), (dict(T=(1 << 22) + 1), 2), (dict(n_req=4097), 2),
    (dict(n=4097), 2), (dict(order=None), 1), (dict(tiles=None), 1), (dict(seg=20), 3)])
def test_plan_refusals(q4, over, status):
    r = _req(q4, **over)
    assert q4.lib().lora_requests_plan(16, 16, ctypes.byref(r), None) == status


def test_call_refusals(q4):
    L, p, r = q4.lib(), _pool(q4), _req(q4)
    P, R = ctypes.byref(p), ctypes.byref(r)
    assert L.lora_requests_plan(None, 16, R, None) == 1 and L.lora_requests_plan(16, None, R, None) == 1
    assert L.lora_requests_plan(16, 16, None, None) == 1
    assert L.lora_requests_fwd(P, R, None, 16, 16, 16, 16, 1 << 30, None) == 1      # X
    assert L.lora_requests_fwd(P, R, 16, 16, None, 16, 16, 1 << 30, None) == 1      # Y
    assert L.lora_requests_fwd(P, R, 16, 16, 16, 16, None, 1 << 30, None) == 1      # workspace
    assert L.lora_requests_fwd(P, R, 17, 16, 16, 16, 16, 1 << 30, None) == 3
    assert L.lora_requests_fwd(P, R, 16, 18, 16, 16, 16, 1 << 30, None) == 3
    assert L.lora_requests_fwd(P, R, 16, 16, 16, 20, 16, 1 << 30, None) == 3
    assert L.lora_requests_fwd(P, R, 16, 16, 16, 16, 16, 16, None) == 4
    assert L.lora_requests_bwd(P, R, 16, 16, 16, 16, 16, None, 16, 16, 1 << 30, None) == 1
    assert L.lora_requests_bwd(P, R, 16, None, 16, 16, 16, 16, 16, 16, 1 << 30, None) == 1
    assert L.lora_requests_bwd(P, R, 16, 16, 16, 16, 16, 16, 24, 16, 1 << 30, None) == 3
    assert L.lora_requests_bwd(P, R, 16, 16, 16, 16, 16, 16, 16, 16, 16, None) == 4
    # outputs that are inputs read beside them
    for Y, refused in ((16, True), (32, False)):
        assert (L.lora_requests_fwd(P, R, 16, 16, Y, 16, 16, 1 << 30, None) == 1) == refused
    for X, dY, dX, refused in ((16, 32, 16, True), (32, 16, 16, True), (32, 32, 16, False)):
        got = L.lora_requests_bwd(P, R, X, 16, dY, dX, dX, 16, 16, 16, 1 << 30, None)
        assert (got == 1) == refused
    assert L.lora_requests_max_tiles(4097, 1, 1) == 0 and L.lora_requests_max_tiles(1, 0, 1) == 0
    assert L.lora_requests_max_tiles(3, 2, 100) > 0


def test_muon_refusals(q4):
    L = q4.lib()

    def call(master=16, w=16, m=16, g=16, n=1, rows=8, cols=64, lr=0.1, mu=0.9, nesterov=1, scale=1.0, wd=0.0, eps=1e-7,
             steps=5, coefs=None, ws=16, size=1 << 30):
        return L.lora_muon_step(master, w, m, g, n, rows, cols, lr, mu, nesterov, scale, wd, eps, steps, coefs, ws, size, None)

    nan, inf = float("nan"), float("inf")
    for v in (dict(master=None), dict(w=None), dict(m=None), dict(g=None), dict(ws=None), dict(n=-1), dict(lr=-1.0),
              dict(lr=nan), dict(lr=inf), dict(mu=1.0), dict(mu=-0.1), dict(mu=nan), dict(scale=nan), dict(wd=-1.0),
              dict(eps=0.0), dict(eps=nan), dict(steps=0), dict(steps=17)):
        assert call(**v) == 1, v
    assert call(rows=257, cols=300) == 2 and call(rows=0) == 2 and call(cols=(1 << 24) + 1) == 2 and call(n=20000) == 2
    assert call(w=18) == 3 and call(ws=17) == 3
    assert call(size=16) == 4
    assert call(n=0) == 0
    bad = (ctypes.c_float * 3)(1.0, nan, 0.0)
    assert call(coefs=ctypes.addressof(bad)) == 1
    assert q4.lora_muon_workspace_bytes(1, 257, 300) == 0 and q4.lora_muon_workspace_bytes(2, 64, 4096) > 0
