"""The layer on an NF4 base with an adapter per request, and a training step of
several tenants as they run together: maps, forward, backward, optimiser."""
import numpy as np
import pytest
import torch

import synthetic
from oracle import muon, nf4
from oracle import requests as oracle
from tests.gpu_helpers import bf16_host_f64, f32_dev, f32_host_f64, rows_within
from tests.requests_helpers import Batch

pytestmark = pytest.mark.gpu

q4 = pytest.importorskip("parameter_efficient_fine_nf4_b200")


def _weight(d, k, seed):
    lay = synthetic.custom_layer(seed=seed, d=d, k=k, r=4, T=1, alpha=8.0)
    return q4.qlora_nf4_quantize(f32_dev(lay.W0)), nf4.bf16_to_f64(nf4.dequantize(nf4.quantize(lay.W0)))


@pytest.mark.parametrize("lens,ids,T", [
    ([1] * 13, [i % 4 - 1 for i in range(13)], 16),         # decoding, padded
    ([30, 34], [2, 0], 64),                                 # the most tokens of the few-token base GEMM
    ([30, 35, 9], [2, -1, 0], 74),                          # few tokens for the adapters only
    ([150, 3, 260, 90], [1, 0, 2, -1], 510),
])
def test_layer_against_the_oracle(lens, ids, T):
    k, d = 256, 384
    b = Batch(k=k, d=d, ranks=[8, 20, 16], lens=lens, ids=ids, T=T, seed=T)
    qw, W = _weight(d, k, T)
    Y, U = q4.qlora_fwd_requests(qw, b.pool, b.plan, b.X, save=True)
    dX, dA, dBt = q4.qlora_bwd_requests(qw, b.pool, b.plan, b.X, U, b.dY)
    torch.cuda.synchronize()
    assert q4.qlora_get_device_status() == 0
    idx = b.maps["idx"]
    fw = oracle.forward(b.Xf, b.A, b.B, b.s, idx, b.Xf @ W.T)
    bw = oracle.backward(b.Xf, b.A, b.B, b.s, idx, f32_host_f64(U), b.dYf, b.dYf @ W)
    # the layer's own bound, rows behind the last request among them (the base product)
    rows_within(bf16_host_f64(Y), fw["Y"], what="Y")
    rows_within(bf16_host_f64(dX), bw["dX"], what="dX")
    for a in range(b.n):
        rows_within(f32_host_f64(dA[b.pool.rows_of(a)]), bw["dA"][a], tol=1e-4, what="dA")
        rows_within(f32_host_f64(dBt[b.pool.rows_of(a)]), bw["dB"][a].T, tol=1e-4, what="dBt")
    # the same as the base and the term one after the other, bit for bit
    none = q4.RequestPlan(1, b.n, T)
    q4.lora_requests_plan(torch.tensor([T], dtype=torch.int32).cuda(), torch.tensor([-1], dtype=torch.int32).cuda(), none)
    base, _ = q4.qlora_fwd_requests(qw, b.pool, none, b.X)
    rows_within(bf16_host_f64(base), b.Xf @ W.T, what="base")
    two, _ = q4.lora_requests_fwd(b.pool, b.plan, b.X, base, Y=base.clone())
    assert torch.equal(two, Y)


def test_layer_refusals():
    b = Batch(k=256, d=384, ranks=[8], lens=[5], ids=[0])
    qw, _ = _weight(256, 256, 1)
    with pytest.raises(ValueError):
        q4.qlora_fwd_requests(qw, b.pool, b.plan, b.X)
    qw, _ = _weight(384, 256, 1)
    with pytest.raises(q4.QloraError):
        q4.qlora_fwd_requests(qw, b.pool, b.plan, b.X, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("captured", [False, True])
def test_training_step_of_several_tenants(captured):
    """Two steps of maps -> forward -> backward -> optimiser on the factors of
    every tenant, against the same steps of the oracles (the bf16 factors of
    the second step are the GPU's own)."""
    k, d, ranks = 256, 320, [8, 16, 24]
    b = Batch(k=k, d=d, ranks=ranks, lens=[60, 90, 33, 70], ids=[0, 2, 1, 0], seed=5)
    qw, W = _weight(d, k, 5)
    dev = "cuda"
    masters = {"A": b.pool.A.float(), "Bt": b.pool.Bt.float()}
    ms = {n: torch.zeros_like(v) for n, v in masters.items()}
    lr, scale = 0.02, 0.5
    dims = {"A": k, "Bt": d}
    wsm = {(n, r): q4.workspace(q4.lora_muon_workspace_bytes(1, r, dims[n])) for n in dims for r in ranks}
    U = torch.zeros(b.T, b.pool.width, device=dev)
    Y, dX = torch.zeros(b.T, d, dtype=torch.bfloat16, device=dev), torch.zeros(b.T, k, dtype=torch.bfloat16, device=dev)
    dA, dBt = torch.zeros(b.pool.rows, k, device=dev), torch.zeros(b.pool.rows, d, device=dev)
    wf = q4.workspace(q4.qlora_fwd_requests_workspace_bytes(qw, b.pool, b.plan))
    wb = q4.workspace(q4.qlora_bwd_requests_workspace_bytes(qw, b.pool, b.plan))

    def step():
        q4.lora_requests_plan(b.dev_lens, b.dev_ids, b.plan)
        q4.qlora_fwd_requests(qw, b.pool, b.plan, b.X, Y=Y, U_save=U, ws=wf)
        q4.qlora_bwd_requests(qw, b.pool, b.plan, b.X, U, b.dY, dX=dX, dA=dA, dBt=dBt, ws=wb)
        for a in range(b.n):
            rows = b.pool.rows_of(a)
            for n, w16, g in (("A", b.pool.A, dA), ("Bt", b.pool.Bt, dBt)):
                q4.lora_muon_step(masters[n][rows], w16[rows], ms[n][rows], g[rows], lr=lr, momentum=0.9, scale=scale,
                                  ws=wsm[n, ranks[a]])

    def factors():
        A = [b.pool.A[b.pool.rows_of(a)].double().cpu().numpy() for a in range(b.n)]
        return A, [b.pool.Bt[b.pool.rows_of(a)].double().cpu().numpy().T for a in range(b.n)]

    ref_w = {n: v.double().cpu().numpy() for n, v in masters.items()}
    ref_m = {n: np.zeros_like(v) for n, v in ref_w.items()}
    idx = b.maps["idx"]
    run = step
    if captured:
        keep = [t.clone() for t in (b.pool.A, b.pool.Bt, *masters.values(), *ms.values())]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for t, v in zip((b.pool.A, b.pool.Bt, *masters.values(), *ms.values()), keep):
            t.copy_(v)
        torch.cuda.synchronize()
        run = graph.replay
    for _ in range(2):
        A, B = factors()
        run()
        torch.cuda.synchronize()
        fw = oracle.forward(b.Xf, A, B, b.s, idx, b.Xf @ W.T)
        rows_within(bf16_host_f64(Y), fw["Y"], what="Y")
        bw = oracle.backward(b.Xf, A, B, b.s, idx, f32_host_f64(U), b.dYf, b.dYf @ W)
        rows_within(bf16_host_f64(dX), bw["dX"], what="dX")
        for a in range(b.n):
            rows = b.pool.rows_of(a)
            for n, g in (("A", bw["dA"][a]), ("Bt", bw["dB"][a].T)):
                got = (dA if n == "A" else dBt)[rows]
                rows_within(f32_host_f64(got), g, tol=1e-4, what="d" + n)
                # the optimiser is held to the gradient it was given
                ref_w[n][rows], ref_m[n][rows], _ = muon.step(ref_w[n][rows], ref_m[n][rows], f32_host_f64(got),
                                                              float(np.float32(lr)), float(np.float32(0.9)), True, scale)
                # u is rounded to 32 bits, which the iterations raise at most 3.4445^5 times
                tol = lr * scale * 2 * 3.4445 ** 5 * 2.0 ** -23 + 1e-6
                assert np.abs(f32_host_f64(masters[n][rows]) - ref_w[n][rows]).max() <= tol
                ref_w[n][rows] = f32_host_f64(masters[n][rows])
                ref_m[n][rows] = f32_host_f64(ms[n][rows])
                w16 = (b.pool.A if n == "A" else b.pool.Bt)[rows]
                assert torch.equal(w16, masters[n][rows].to(torch.bfloat16))
