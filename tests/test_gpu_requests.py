"""GPU parity of the many-adapter operators with the float64 oracle: the maps,
the adapter term and its gradients, at the lengths, ranks and groups where they
can go wrong."""
import numpy as np
import pytest
import torch

from tests.requests_helpers import Batch

pytestmark = pytest.mark.gpu

q4 = pytest.importorskip("parameter_efficient_fine_nf4_b200")

CASES = {
    "one token": dict(k=64, d=64, ranks=[8], lens=[1], ids=[0]),
    "one token, no adapter": dict(k=64, d=64, ranks=[8], lens=[1], ids=[-1]),
    "smallest sizes": dict(k=8, d=8, ranks=[1], lens=[3], ids=[0]),
    "decoding": dict(k=256, d=512, ranks=[8, 16, 5, 64], lens=[1] * 19, ids=[i % 5 - 1 for i in range(19)]),
    "decoding, one adapter": dict(k=512, d=256, ranks=[16, 16], lens=[1] * 40, ids=[1] * 40),
    "decoding, two blocks a tile": dict(k=1000, d=640, ranks=[24, 3], lens=[1] * 11, ids=[0, 1, 1, 0, 0, 0, 1, 1, 1, 1, -1]),
    "decoding, wide": dict(k=4104, d=1032, ranks=[64, 12, 33], lens=[1, 2, 3, 1, 5, 1, 8], ids=[0, 1, 2, 0, 1, -1, 2]),
    "decoding, wide output": dict(k=264, d=8192, ranks=[16, 40], lens=[2, 1, 4, 9], ids=[1, 0, 0, 1]),
    "one token, wide": dict(k=8192, d=4096, ranks=[48], lens=[1], ids=[0]),
    "few tokens, rank 256": dict(k=2048, d=2056, ranks=[256, 100], lens=[3, 9, 1], ids=[0, 1, 0]),
    "few tokens, rank 128": dict(k=4096, d=512, ranks=[128], lens=[2], ids=[0]),
    "the most few tokens": dict(k=520, d=4096, ranks=[20, 9], lens=[100, 28], ids=[1, 0]),
    "padded batch": dict(k=256, d=264, ranks=[12, 4], lens=[3, 0, 5, -2, 1], ids=[1, 0, 0, 1, 9], T=21),
    "cut batch": dict(k=136, d=72, ranks=[3, 30], lens=[9, 30, 2000000000, 2000000000], ids=[0, 1, 0, 1], T=70),
    "empty requests only": dict(k=64, d=64, ranks=[8], lens=[0, 0], ids=[0, 0], T=5),
    "no requests": dict(k=64, d=64, ranks=[8], lens=[], ids=[], T=5),
    "one more than few tokens": dict(k=520, d=512, ranks=[20, 9], lens=[100, 29], ids=[1, 0]),
    "decoding, many": dict(k=512, d=1032, ranks=[8, 24, 64] * 40, lens=[1] * 300, ids=[(7 * i) % 121 - 1 for i in range(300)],
                           T=311),
    "decoding, more than tokens for it": dict(k=136, d=72, ranks=[8, 24], lens=[1] * 1030, ids=[i % 3 - 1 for i in range(1030)]),
    "tiles end inside": dict(k=320, d=192, ranks=[16, 40, 7], lens=[127, 1, 128, 129, 8, 7, 9],
                             ids=[0, 1, 1, 2, 0, 2, 1]),
    "rank 256": dict(k=200, d=328, ranks=[256, 17], lens=[70, 65, 30], ids=[0, 1, 0]),
    "ranks past 64": dict(k=512, d=640, ranks=[65, 96, 128, 130], lens=[40, 200, 100, 33, 140], ids=[0, 1, 2, 3, 1]),
    "many adapters": dict(k=128, d=128, ranks=[1 + i % 9 for i in range(200)], lens=[1 + i % 3 for i in range(150)],
                          ids=[(7 * i) % 200 for i in range(150)]),
    "eight tokens per adapter": dict(k=72, d=136, ranks=[1 + i % 20 for i in range(255)], lens=[8] * 256,
                                     ids=[i - 1 for i in range(256)]),
    "one more than eight per adapter": dict(k=72, d=136, ranks=[1 + i % 20 for i in range(149)], lens=[9] + [8] * 149,
                                            ids=[i - 1 for i in range(150)]),
    "many adapters, nine tokens each": dict(k=264, d=136, ranks=[16, 70, 3] * 40, lens=[9] * 120, ids=list(range(120))),
    "many adapters, one in use": dict(k=136, d=264, ranks=[24] * 100, lens=[5] * 100, ids=[42] * 100),
    "more than 2048 tokens": dict(k=64, d=72, ranks=[8] * 300, lens=[7] * 300, ids=[(7 * i) % 301 - 1 for i in range(300)]),
    "one adapter, long": dict(k=1032, d=520, ranks=[24], lens=[700, 333], ids=[0, 0]),
    "training batch": dict(k=768, d=1024, ranks=[16, 64, 8], lens=[100, 250, 61, 300, 19, 77], ids=[0, 1, 2, 1, -1, 0]),
    "unused adapters": dict(k=256, d=256, ranks=[8, 16, 32, 8], lens=[90, 170], ids=[2, -1]),
}


@pytest.mark.parametrize("name", list(CASES))
def test_against_the_oracle(name):
    b = Batch(seed=len(name), **CASES[name])
    b.check_maps()
    Y0, dX0 = torch.full_like(b.base_y, 7.0), torch.full_like(b.base_x, 7.0)
    U0 = torch.full((b.T, b.pool.width), 7.0, device="cuda")
    Y, U = q4.lora_requests_fwd(b.pool, b.plan, b.X, b.base_y, Y=Y0, U_save=U0)
    dX, dA, dBt = q4.lora_requests_bwd(b.pool, b.plan, b.X, U, b.dY, b.base_x, dX=dX0,
                                       dA=torch.full((b.pool.rows, b.k), float("nan"), device="cuda"),
                                       dBt=torch.full((b.pool.rows, b.d), float("nan"), device="cuda"))
    torch.cuda.synchronize()
    assert q4.qlora_get_device_status() == 0
    b.check_forward(Y, U)
    b.check_backward(dX, dA, dBt, U)
    for t in (Y, U, dX):          # rows behind the last request are left as they were
        assert bool((t[b.total:] == 7.0).all())


@pytest.mark.parametrize("name", ["decoding", "training batch"])
def test_without_base_and_in_place(name):
    b = Batch(seed=3, **CASES[name])
    Y, U = q4.lora_requests_fwd(b.pool, b.plan, b.X, save=True)
    dX, dA, dBt = q4.lora_requests_bwd(b.pool, b.plan, b.X, U, b.dY)
    b.check_forward(Y, U, base=False)
    b.check_backward(dX, dA, dBt, U, base=False)
    y, x = b.base_y.clone(), b.base_x.clone()
    ref = q4.lora_requests_fwd(b.pool, b.plan, b.X, b.base_y)[0]
    got, none = q4.lora_requests_fwd(b.pool, b.plan, b.X, y, Y=y)
    assert none is None and got is y and torch.equal(y, ref)
    ref = q4.lora_requests_bwd(b.pool, b.plan, b.X, U, b.dY, b.base_x)
    got = q4.lora_requests_bwd(b.pool, b.plan, b.X, U, b.dY, x, dX=x)
    assert all(torch.equal(p, q) for p, q in zip(ref, got))


@pytest.mark.parametrize("name", ["decoding", "training batch", "ranks past 64"])
def test_repeats_are_bit_identical(name):
    b = Batch(seed=4, **CASES[name])
    runs = []
    for _ in range(2):
        Y, U = q4.lora_requests_fwd(b.pool, b.plan, b.X, b.base_y, save=True)
        runs.append((Y, U) + q4.lora_requests_bwd(b.pool, b.plan, b.X, U, b.dY, b.base_x))
    assert all(torch.equal(p, q) for p, q in zip(*runs))


@pytest.mark.parametrize("name", ["decoding", "training batch"])
def test_values_do_not_leak_between_rows(name):
    """NaN in one token and in one adapter's factors stays with that token's
    and that adapter's rows."""
    b = Batch(seed=6, **CASES[name])
    clean = q4.lora_requests_fwd(b.pool, b.plan, b.X, b.base_y, save=True)
    cg = q4.lora_requests_bwd(b.pool, b.plan, b.X, clean[1], b.dY, b.base_x)
    idx = b.plan.idx.cpu().numpy()
    t = int(np.flatnonzero(idx == 0)[1])
    b.X[t] = float("nan")
    b.dY[t] = float("inf")
    b.pool.A[b.pool.rows_of(1)] = float("nan")
    b.pool.Bt[b.pool.rows_of(1)] = float("inf")
    Y, U = q4.lora_requests_fwd(b.pool, b.plan, b.X, b.base_y, save=True)
    dX, dA, dBt = q4.lora_requests_bwd(b.pool, b.plan, b.X, clean[1], b.dY, b.base_x)
    keep = torch.from_numpy((idx != 1) & (np.arange(b.T) != t)).cuda()
    assert torch.equal(Y[keep], clean[0][keep]) and torch.equal(U[keep], clean[1][keep])
    assert torch.equal(dX[keep], cg[0][keep])
    for a in range(2, b.n):
        rows = b.pool.rows_of(a)
        assert torch.equal(dA[rows], cg[1][rows]) and torch.equal(dBt[rows], cg[2][rows])


@pytest.mark.parametrize("lens", [[5, 9, 3], [150, 90, 40]])
def test_infinite_tokens_leave_the_padding_rows_zero(lens):
    b = Batch(72, 136, [5, 20], lens, [0, 1, -1], seed=9)
    _, U = q4.lora_requests_fwd(b.pool, b.plan, b.X, b.base_y, save=True)
    b.X[1, 3], b.dY[2, 7], b.X[lens[0] + 1, 70] = float("inf"), float("-inf"), float("nan")
    _, dA, dBt = q4.lora_requests_bwd(b.pool, b.plan, b.X, U, b.dY)
    assert not dA[:5].isfinite().all() and not dBt[:5].isfinite().all()
    for pad in (slice(5, 16), slice(16 + 20, 16 + 32)):
        assert not dA[pad].any() and not dBt[pad].any()


def test_most_adapters_of_the_widest_rank():
    ranks = [1] * 4095 + [256]
    b = Batch(8, 16, ranks, [2, 3, 1], [4095, 7, 4094], seed=3, alphas=[float(r) for r in ranks])
    Y, U = q4.lora_requests_fwd(b.pool, b.plan, b.X, b.base_y, save=True)
    dX, dA, dBt = q4.lora_requests_bwd(b.pool, b.plan, b.X, U, b.dY, b.base_x)
    b.check_forward(Y, U)
    b.check_backward(dX, dA, dBt, U)


def test_a_table_that_leaves_the_pool_counts_as_no_adapter():
    b = Batch(k=256, d=256, ranks=[8, 16], lens=[5, 200, 4], ids=[0, 1, 1], seed=8)
    want = q4.lora_requests_fwd(b.pool, b.plan, b.X, b.base_y)[0]
    for first, rank in ((b.pool.rows, 16), (-16, 16), (16, 0), (16, -3), (16, 17), (2 ** 31 - 1, 16), (24, 16)):
        b.pool.first[1], b.pool.rank[1] = first, rank
        Y, U = q4.lora_requests_fwd(b.pool, b.plan, b.X, b.base_y, save=True)
        assert torch.equal(Y[:5], want[:5]) and torch.equal(Y[5:], b.base_y[5:]) and not U[5:].any()


def test_maps_feed_the_stacked_entry_points():
    """idx is what qlora_fwd_multi takes: the same layer both ways."""
    import synthetic
    from tests.gpu_helpers import f32_dev
    k, d, r, n = 256, 256, 8, 3
    b = Batch(k=k, d=d, ranks=[r] * n, lens=[70, 33, 50], ids=[2, 0, -1], seed=9)
    lay = synthetic.custom_layer(seed=9, d=d, k=k, r=r, T=4, alpha=16.0)
    qw = q4.qlora_nf4_quantize(f32_dev(lay.W0))
    As = torch.stack([b.pool.A[b.pool.rows_of(a)] for a in range(n)])
    Bs = torch.stack([b.pool.Bt[b.pool.rows_of(a)].t().contiguous() for a in range(n)])
    alphas = [s * r for s in b.s]
    Ym, Um = q4.qlora_fwd_multi(qw, As, Bs, alphas, b.plan.idx, b.X)
    none = torch.full_like(b.plan.idx, -1)
    base, _ = q4.qlora_fwd_multi(qw, As, Bs, alphas, none, b.X)
    Y, U = q4.lora_requests_fwd(b.pool, b.plan, b.X, base, save=True)
    # two roundings of Y here, and s U in one bf16 term there: 2^-8 each
    tol = 3 * 2.0 ** -8 * (Ym.float().abs().amax(1, keepdim=True))
    assert bool(((Y.float() - Ym.float()).abs() <= tol).all())
    assert torch.allclose(U[:, :r], Um, rtol=0, atol=1e-4 * float(Um.abs().max()))


def test_refusals_of_the_binding():
    b = Batch(seed=1, **CASES["decoding"])
    with pytest.raises(ValueError):
        q4.lora_requests_fwd(b.pool, b.plan, b.X[:-1])
    with pytest.raises(TypeError):
        q4.lora_requests_fwd(b.pool, b.plan, b.X.float())
    with pytest.raises(ValueError):
        q4.lora_requests_fwd(b.pool, b.plan, b.X.cpu())
    with pytest.raises(ValueError):
        q4.lora_requests_fwd(b.pool, b.plan, b.X.t().contiguous().t())
    with pytest.raises(ValueError):
        q4.lora_requests_fwd(b.pool, q4.RequestPlan(3, 9, b.T), b.X)
    with pytest.raises(q4.QloraError):
        q4.lora_requests_bwd(b.pool, b.plan, b.X, torch.zeros(b.T, b.pool.width, device="cuda"), b.dY,
                             ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        q4.lora_requests_plan(b.dev_lens[:-1], b.dev_ids, b.plan)
    with pytest.raises(TypeError):
        q4.lora_requests_plan(b.dev_lens.long(), b.dev_ids, b.plan)
    for bad in (dict(ranks=[0]), dict(ranks=[257]), dict(alphas=[-1.0]), dict(k=60), dict(alphas=[1.0, 2.0])):
        with pytest.raises(ValueError):
            q4.AdapterPool(**{**dict(k=64, d=64, ranks=[8], alphas=[16.0]), **bad})
    with pytest.raises(ValueError):
        q4.RequestPlan(5000, 1, 8)
    with pytest.raises(IndexError):
        b.pool.rows_of(b.n)
    for held, name in ((b.pool, "A"), (b.pool, "scale"), (b.plan, "order")):
        with pytest.raises(AttributeError):       # the addresses are in a C struct
            setattr(held, name, getattr(held, name).clone())
    with pytest.raises(ValueError):
        b.pool.load(0, b.pool.A[:4], b.pool.Bt[:8].t())


@pytest.mark.parametrize("name", ["decoding", "training batch"])
def test_captured_and_replayed_with_other_requests(name):
    """A captured batch follows the lengths and adapters in its buffers, beside
    a second captured batch with its own plan and workspace."""
    kw = CASES[name]
    b = Batch(seed=11, T=sum(kw["lens"]) + 3, **kw)
    ws = q4.workspace(max(q4.lora_requests_fwd_workspace_bytes(b.pool, b.plan),
                          q4.lora_requests_bwd_workspace_bytes(b.pool, b.plan)))
    out = {}

    def step():
        q4.lora_requests_plan(b.dev_lens, b.dev_ids, b.plan)
        out["Y"], out["U"] = q4.lora_requests_fwd(b.pool, b.plan, b.X, b.base_y, Y=out.get("Y"), U_save=out.get("U"),
                                                  save=True, ws=ws)
        out["dX"], out["dA"], out["dBt"] = q4.lora_requests_bwd(
            b.pool, b.plan, b.X, out["U"], b.dY, b.base_x, dX=out.get("dX"), dA=out.get("dA"), dBt=out.get("dBt"), ws=ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    lens = list(reversed(kw["lens"]))
    ids = [(i + 1) % b.n for i in range(len(lens))]
    b.dev_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    b.dev_ids.copy_(torch.tensor(ids, dtype=torch.int32))
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    from oracle import requests as oracle
    b.maps = oracle.plan(lens, ids, b.n, b.T)
    b.total = int(b.maps["starts"][-1])
    b.check_maps()
    b.check_forward(out["Y"], out["U"])
    b.check_backward(out["dX"], out["dA"], out["dBt"], out["U"])


def test_on_another_stream():
    b = Batch(seed=12, **CASES["training batch"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = []
    for _ in range(4):
        # temporaries of earlier calls may be reused while these still run
        Y, U = q4.lora_requests_fwd(b.pool, b.plan, b.X, b.base_y, save=True, stream=s)
        got.append((Y, U) + q4.lora_requests_bwd(b.pool, b.plan, b.X, U, b.dY, b.base_x, stream=s))
        junk = torch.full((1 << 22,), float("nan"), device="cuda")
        del junk
    s.synchronize()
    for r in got:
        b.check_forward(r[0], r[1])
        b.check_backward(r[2], r[3], r[4], r[1])


def test_calls_on_several_streams_at_once():
    """Chains on three streams, each with its own outputs and workspaces, give
    what each gives alone."""
    batches = [Batch(seed=20 + i, **CASES[n]) for i, n in enumerate(("training batch", "decoding, wide", "ranks past 64"))]

    def chain(b, ws, stream=None):
        got = []
        for _ in range(6):
            q4.lora_requests_plan(b.dev_lens, b.dev_ids, b.plan, stream=stream)
            Y, U = q4.lora_requests_fwd(b.pool, b.plan, b.X, b.base_y, save=True, ws=ws, stream=stream)
            got = [Y, U, *q4.lora_requests_bwd(b.pool, b.plan, b.X, U, b.dY, b.base_x, ws=ws, stream=stream)]
        return got

    wss = [q4.workspace(max(q4.lora_requests_fwd_workspace_bytes(b.pool, b.plan),
                            q4.lora_requests_bwd_workspace_bytes(b.pool, b.plan))) for b in batches]
    alone = [chain(b, ws) for b, ws in zip(batches, wss)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in batches]
    for _ in range(3):
        both = [chain(b, ws, s) for b, ws, s in zip(batches, wss, streams)]
    torch.cuda.synchronize()
    assert q4.qlora_get_device_status() == 0
    for x, y in zip(alone, both):
        assert all(torch.equal(p, q) for p, q in zip(x, y))


def test_gradients_against_differences():
    """dA and dBt against differences of the fp32-valued loss sum(Y dY) formed
    from U and the factors: a directional derivative along the gradient."""
    b = Batch(seed=13, **CASES["training batch"])
    Y, U = q4.lora_requests_fwd(b.pool, b.plan, b.X, save=True)
    dX, dA, dBt = q4.lora_requests_bwd(b.pool, b.plan, b.X, U, b.dY)
    from oracle import requests as oracle
    idx, h = b.maps["idx"], 1e-4
    for a in range(b.n):
        gA = dA[b.pool.rows_of(a)].double().cpu().numpy()
        gB = dBt[b.pool.rows_of(a)].double().cpu().numpy().T
        up = [[m.copy() for m in b.A], [m.copy() for m in b.B]]
        dn = [[m.copy() for m in b.A], [m.copy() for m in b.B]]
        nA, nB = np.linalg.norm(gA), np.linalg.norm(gB)
        up[0][a] += h * gA / nA
        dn[0][a] -= h * gA / nA
        loss = lambda f: float((oracle.forward(b.Xf, f[0], f[1], b.s, idx)["Y"] * b.dYf).sum())  # noqa: E731
        assert np.isclose((loss(up) - loss(dn)) / (2 * h), nA, rtol=1e-4)
        up[0][a], dn[0][a] = b.A[a], b.A[a]
        up[1][a] += h * gB / nB
        dn[1][a] -= h * gB / nB
        assert np.isclose((loss(up) - loss(dn)) / (2 * h), nB, rtol=1e-4)
