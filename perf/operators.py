"""What the operators for many adapters cost: the calls that are measured, their plain forms and their exact values.

Four operators of a base model that serves or trains many low-rank adapters at once:

* ``plan``: the maps from request lengths to tokens that the other calls of a batch share (first row of each request,
  adapter of each token, the tokens grouped by adapter, where each group starts);
* ``fwd``: the adapters' term beside a shared projection, Y = base + s_a (X A_a^T) B_a^T, token by token with the
  adapter a of its request;
* ``bwd``: its gradients, dX = base + s_a (dY B_a) A_a, dA_a = s_a sum (dY B_a)^T X, dB_a = s_a sum dY^T U;
* ``muon``: the optimiser step that orthogonalises a factor's momentum by Newton-Schulz products.

An adapter's factors are rows of two matrices, A (rows x k) and B transposed (rows x d); its rank is padded to a
multiple of 16 rows, the added rows are zero.
"""
import math

import numpy as np
import torch

own = False

COEFS = (3.4445, -4.7750, 2.0315)      # the quintic of the orthogonalisation
STEPS = 5
MOMENTUM, LR, DECAY, EPS = 0.95, 2e-3, 0.01, 1e-7


def _case(name, op, **v):
    return dict({"name": name} if name else {}, op=op, **v)


def _tokens(name, op, k, d, ranks, n, req, T, pad=0, none=0):
    """A batch of `req` requests and T rows, the last `pad` of them behind the last request; every `none`-th request
    runs on the bare base."""
    return _case(name, op, k=k, d=d, ranks=ranks, n=n, req=req, T=T, pad=pad, none=none)


def listed():
    return [
        # one decoding step of 64 requests over 32 adapters
        _case("plan decode", "plan", n=32, req=64, T=64, pad=0, none=8),
        # a prefill of 300 ragged prompts, the batch padded to a fixed length
        _case("plan prefill", "plan", n=100, req=300, T=16384, pad=200, none=10),
        # the smallest layer, 16 requests of one token each: latency
        _tokens("fwd small", "fwd", 256, 256, "8", 4, 16, 16),
        # decoding, 64 requests with ranks of their own, a few without an adapter, padded rows
        _tokens("fwd decode", "fwd", 4096, 4096, "8,16,64,32,12", 48, 60, 64, pad=4, none=12),
        # prompts of many tenants through the projection 4096 -> 11008
        _tokens("fwd prefill", "fwd", 4096, 11008, "16", 8, 24, 8192, pad=77, none=9),
        # the largest projection, few tenants with long inputs
        _tokens("fwd large", "fwd", 8192, 22016, "64", 4, 9, 16384),
        # fine-tuning on a handful of short samples
        _tokens("bwd small", "bwd", 4096, 4096, "8", 6, 6, 48),
        # a training batch of several tenants, ranks of their own
        _tokens("bwd train", "bwd", 4096, 4096, "16,64,8,40", 4, 13, 4096, pad=33, none=7),
        # the largest projection, a full batch
        _tokens("bwd large", "bwd", 8192, 22016, "64", 3, 8, 16384),
        # one factor A of a 4096-wide layer
        _case("muon one", "muon", n=1, rows=64, cols=4096, nesterov=True),
        # the A factors of several tenants at once
        _case("muon stack", "muon", n=8, rows=16, cols=11008, nesterov=True),
        # B of the largest projection: more rows than columns
        _case("muon tall", "muon", n=2, rows=22016, cols=64, nesterov=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "fwd", "fwd", "bwd", "bwd", "muon"])
    if op == "plan":
        decode = rng.random() < 0.4
        req = _log(rng, 1, 1024)
        T = req if decode else min(32768, max(req, _log(rng, 16, 32768)))
        pad = rng.randrange(1, 64) if rng.random() < 0.5 else 0
        return _case(None, op, n=_log(rng, 1, 512), req=req, T=T + pad, pad=pad, none=rng.choice([0, 5, 11]))
    if op == "muon":
        r, long = _log(rng, 4, 128), _log(rng, 256, 22016)
        r = min(r, long)
        n = max(1, min(_log(rng, 1, 16), 2 * 22016 * 64 // (r * long)))
        tall = rng.random() < 0.5
        return _case(None, op, n=n, rows=long if tall else r, cols=r if tall else long, nesterov=rng.random() < 0.5)
    k, d = (8 * _log(rng, 32, 1024), 8 * _log(rng, 32, 2048)) if rng.random() < 0.5 else (64 * _log(rng, 4, 128), 64 * _log(rng, 4, 256))
    ranks = ",".join(str(_log(rng, 1, 96)) for _ in range(rng.randint(1, 4)))
    if rng.random() < 0.4:        # decoding, or samples of a few tokens
        T = _log(rng, 1, 256)
        req = T if rng.random() < 0.6 else rng.randint(1, T)
    else:
        T = _log(rng, 256, min(16384, 16384 * 30208 // (k + d)))
        req = rng.randint(1, min(64, T))
    n = rng.randint(1, min(req, 64 if op == "fwd" else 16))
    return _tokens(None, op, k, d, ranks, n, req, T, pad=rng.choice([0, 0, T // 9]) if req < T // 2 else 0,
                   none=rng.choice([0, 0, 6]))


def _ranks(case):
    got = [int(v) for v in case["ranks"].split(",")]
    return [got[a % len(got)] for a in range(case["n"])]


def _requests(case, seed):
    """Lengths (their sum is T - pad) and adapters of the requests: every adapter is used where there are requests
    enough, some more than once."""
    g = np.random.RandomState(seed % (1 << 31))
    req, total = case["req"], case["T"] - case["pad"]
    w = np.exp(1.2 * g.randn(req))
    lens = 1 + np.floor(w / w.sum() * (total - req)).astype(np.int64) if total > req else np.ones(req, np.int64)
    lens[int(g.randint(req))] += total - lens.sum()
    ids = np.concatenate([g.permutation(case["n"]), g.randint(0, case["n"], max(0, req - case["n"]))])[:req]
    ids = ids[g.permutation(req)]
    if case["none"]:
        ids[case["none"] - 1::case["none"]] = -1
    return lens, ids


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, sigma=1.0, dtype=torch.float32):
        out = torch.empty(*shape, dtype=dtype, device=dev)
        for a in range(0, shape[0], 4096):
            part = out[a:a + 4096]
            part.copy_(torch.randn(part.shape, generator=gen, device=dev) * sigma)
        return out

    if case["op"] == "muon":
        n, rows, cols, r = case["n"], case["rows"], case["cols"], min(case["rows"], case["cols"])
        long = max(rows, cols)
        # a gradient's spectrum falls off: directions of size 1, 1/2, 1/3, ...
        fall = 1.0 / torch.arange(1, r + 1, device=dev, dtype=torch.float32)
        g = normal(n, r, r) * fall @ normal(n, r, long) * (1e-3 / math.sqrt(r))
        g = g.transpose(1, 2).contiguous() if rows > cols else g
        m = g * normal(n, 1, 1) + normal(n, rows, cols, sigma=1e-5)
        master = normal(n, rows, cols, sigma=0.01 if rows > cols else 1.0 / r)
        s = {"case": case, "grad": g, "m": m, "master": master, "w": master.to(torch.bfloat16)}
        s["scale"] = 0.2 * math.sqrt(long)
        if own:
            import parameter_efficient_fine_nf4_b200 as q4
            s["ws"] = q4.workspace(q4.lora_muon_workspace_bytes(n, rows, cols), dev)
        return s

    lens, ids = _requests(case, seed)
    s = {"case": case, "total": int(lens.sum()), "n": case["n"], "T": case["T"],
         "lens": torch.tensor(lens, dtype=torch.int32, device=dev), "ids": torch.tensor(ids, dtype=torch.int32, device=dev)}
    if own:
        import parameter_efficient_fine_nf4_b200 as q4
        s["plan"] = q4.RequestPlan(case["req"], case["n"], case["T"], dev)
    if case["op"] == "plan":
        return s
    k, d, T = case["k"], case["d"], case["T"]
    ranks = _ranks(case)
    bf = torch.bfloat16
    first, rows = [], 0
    for r in ranks:
        first.append(rows)
        rows += -(-r // 16) * 16
    A, Bt = torch.zeros(rows, k, dtype=bf, device=dev), torch.zeros(rows, d, dtype=bf, device=dev)
    owner = torch.full((rows,), -2, dtype=torch.int32, device=dev)
    scale = torch.zeros(rows, device=dev)
    for a, (f, r) in enumerate(zip(first, ranks)):
        A[f:f + r] = normal(r, k, sigma=1.0 / r, dtype=bf)
        Bt[f:f + r] = normal(r, d, sigma=0.01, dtype=bf)
        owner[f:f + r] = a
        scale[f:f + r] = 2.0
    s |= {"A": A, "Bt": Bt, "owner": owner, "scale": scale, "X": normal(T, k, dtype=bf)}
    s["idx"] = torch.cat([torch.repeat_interleave(s["ids"], s["lens"].long()),
                          torch.full((case["pad"],), -1, dtype=torch.int32, device=dev)])
    out = d if case["op"] == "fwd" else k
    s["base"] = normal(T, out, sigma=0.02 * math.sqrt(k), dtype=bf)
    s["out"] = torch.zeros(T, out, dtype=bf, device=dev)
    if case["op"] == "bwd":
        s["dY"] = normal(T, d, dtype=bf)
        # what the forward saved: each token's own U, as wide as the largest rank
        wide = max(-(-r // 16) * 16 for r in ranks)
        U = torch.zeros(T, wide, device=dev)
        for a, (f, r) in enumerate(zip(first, ranks)):
            at = torch.nonzero(s["idx"] == a).flatten()
            U[at, :r] = s["X"][at].float() @ A[f:f + r].float().t()
        s["U"] = U
        s["column"] = torch.arange(rows, device=dev) - torch.tensor(first, device=dev)[owner.clamp(min=0).long()]
        s["column"].clamp_(0, wide - 1)
    if own:
        pool = q4.AdapterPool(k, d, ranks, [2.0 * r for r in ranks], dev)
        pool.A.copy_(A)
        pool.Bt.copy_(Bt)
        s["pool"] = pool
        q4.lora_requests_plan(s["lens"], s["ids"], s["plan"])
        query = q4.lora_requests_fwd_workspace_bytes if case["op"] == "fwd" else q4.lora_requests_bwd_workspace_bytes
        s["ws"] = q4.workspace(query(pool, s["plan"]), dev)
        if case["op"] == "bwd":
            s["dA"], s["dBt"] = torch.empty(rows, k, device=dev), torch.empty(rows, d, device=dev)
    return s


def _plain_plan(s):
    n, T = s["n"], s["T"]
    ends = s["lens"].long().clamp(min=0).cumsum(0).clamp(max=T)
    starts = torch.cat([torch.zeros_like(ends[:1]), ends])
    t = torch.arange(T, device=ends.device)
    req = torch.searchsorted(ends, t, right=True)
    behind = req >= ends.numel()
    a = s["ids"].long()[req.clamp(max=ends.numel() - 1)]
    none = (a < 0) | (a >= n)
    idx = torch.where(behind | none, -1, a)
    key = torch.where(behind, n + 1, torch.where(none, n, a))
    order = torch.where(t < ends[-1], torch.argsort(key, stable=True), -1)
    seg = torch.cat([torch.zeros_like(ends[:1]), torch.bincount(key, minlength=n + 2)[:n + 1].cumsum(0)])
    return {"starts": starts.int(), "idx": idx.int(), "order": order.int(), "seg": seg.int()}


def _plain_mask(s, rows):
    """What each row of the pool is worth to each token: its adapter's scale, or zero."""
    return (s["idx"][:rows, None] == s["owner"][None, :]).float() * s["scale"]


def _plain_fwd(s):
    m = s["total"]
    low = s["X"][:m].float() @ s["A"].float().t() * _plain_mask(s, m)
    s["out"][:m] = (s["base"][:m].float() + low @ s["Bt"].float()).to(torch.bfloat16)
    return s["out"]


def _plain_bwd(s):
    m = s["total"]
    mask = _plain_mask(s, m)
    X, dY = s["X"][:m].float(), s["dY"][:m].float()
    G = dY @ s["Bt"].float().t() * mask
    s["out"][:m] = (s["base"][:m].float() + G @ s["A"].float()).to(torch.bfloat16)
    U = s["U"][:m][:, s["column"]] * mask
    return {"dX": s["out"], "dA": G.t() @ X, "dBt": U.t() @ dY}


def _plain_muon(s):
    case, (a, b, c) = s["case"], COEFS
    m = s["m"].mul_(MOMENTUM).add_(s["grad"])
    u = s["grad"] + MOMENTUM * m if case["nesterov"] else m
    x = u.transpose(1, 2) if case["rows"] > case["cols"] else u
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    g = x @ x.transpose(1, 2)
    x1 = a * x + (b * g + c * (g @ g)) @ x
    g = x1 @ x1.transpose(1, 2)
    x2 = a * x1 + (b * g + c * (g @ g)) @ x1
    g = x2 @ x2.transpose(1, 2)
    x3 = a * x2 + (b * g + c * (g @ g)) @ x2
    g = x3 @ x3.transpose(1, 2)
    x4 = a * x3 + (b * g + c * (g @ g)) @ x3
    g = x4 @ x4.transpose(1, 2)
    x5 = a * x4 + (b * g + c * (g @ g)) @ x4
    o = x5.transpose(1, 2) if case["rows"] > case["cols"] else x5
    s["master"].mul_(1 - LR * DECAY).sub_(LR * s["scale"] * o)
    s["w"].copy_(s["master"])
    return {"master": s["master"], "w": s["w"], "m": m}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"plan": _plain_plan, "fwd": _plain_fwd, "bwd": _plain_bwd, "muon": _plain_muon}[op](s)
    import parameter_efficient_fine_nf4_b200 as q4
    if op == "plan":
        p = q4.lora_requests_plan(s["lens"], s["ids"], s["plan"])
        return {"starts": p.starts, "idx": p.idx, "order": p.order, "seg": p.seg}
    if op == "fwd":
        return q4.lora_requests_fwd(s["pool"], s["plan"], s["X"], s["base"], Y=s["out"], ws=s["ws"])[0]
    if op == "bwd":
        dX, dA, dBt = q4.lora_requests_bwd(s["pool"], s["plan"], s["X"], s["U"], s["dY"], s["base"], dX=s["out"],
                                           dA=s["dA"], dBt=s["dBt"], ws=s["ws"])
        return {"dX": dX, "dA": dA, "dBt": dBt}
    q4.lora_muon_step(s["master"], s["w"], s["m"], s["grad"], lr=LR, momentum=MOMENTUM, nesterov=s["case"]["nesterov"],
                      scale=s["scale"], weight_decay=DECAY, ws=s["ws"])
    return {"master": s["master"], "w": s["w"], "m": s["m"]}


def work(case):
    T, n = case.get("T", 0), case["n"]
    if case["op"] == "plan":
        return {"bytes": 4.0 * (3 * case["req"] + 1 + 2 * T + n + 2), "flops": 0.0}
    if case["op"] == "muon":
        r, size = min(case["rows"], case["cols"]), n * case["rows"] * case["cols"]
        # gradient, momentum and master read, momentum, master and the 16-bit copy written; the Gram matrix, its
        # polynomial (17 products of r x r) and one product with the momentum
        return {"bytes": 22.0 * size, "flops": 4.0 * size * r + n * 17 * 2.0 * r ** 3}
    m = T - case["pad"]
    k, d, ranks = case["k"], case["d"], _ranks(case)
    bare = m // case["none"] if case["none"] else 0
    r = sum(ranks) / n
    factors = 2.0 * sum(ranks) * (k + d)
    if case["op"] == "fwd":
        return {"bytes": 2.0 * ((m - bare) * k + 2 * m * d) + factors, "flops": 2.0 * (m - bare) * r * (k + d)}
    return {"bytes": 2.0 * ((m - bare) * (k + d) + 2 * m * k) + 4.0 * (m - bare) * r + factors + 2 * factors,
            "flops": 4.0 * (m - bare) * r * (k + d)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        starts, idx, groups = [0], [-1] * case["T"], [[] for _ in range(case["n"] + 1)]
        for size, a in zip(s["lens"].tolist(), s["ids"].tolist()):
            at = range(starts[-1], min(case["T"], starts[-1] + max(0, size)))
            a = a if 0 <= a < case["n"] else -1
            groups[a].extend(at)          # the last group is the bare base's
            for t in at:
                idx[t] = a
            starts.append(at.stop)
        order = [t for g in groups for t in g]
        seg = np.cumsum([0] + [len(g) for g in groups])
        maps = {"starts": starts, "idx": idx, "order": order + [-1] * (case["T"] - len(order)), "seg": seg}
        return {name: torch.tensor(np.asarray(v), dtype=torch.int32) for name, v in maps.items()}
    if case["op"] == "muon":
        master, m, g = s["master"].double(), s["m"].double(), s["grad"].double()
        m = MOMENTUM * m + g
        out = master * (1 - LR * DECAY)
        for i in range(case["n"]):
            u = g[i] + MOMENTUM * m[i] if case["nesterov"] else m[i]
            # the quintic acts on each singular value alone
            U, sv, Vh = torch.linalg.svd(u, full_matrices=False)
            sv = sv / (torch.linalg.vector_norm(u) + EPS)
            for _ in range(STEPS):
                sv = COEFS[0] * sv + COEFS[1] * sv ** 3 + COEFS[2] * sv ** 5
            out[i] -= LR * s["scale"] * ((U * sv) @ Vh)
        return {"master": out, "w": out.clone(), "m": m}
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["X"].device)
    m = s["total"]
    out[:m] = s["base"][:m].double()
    dA = torch.zeros(s["A"].shape, dtype=torch.float64, device=out.device)
    dBt = torch.zeros(s["Bt"].shape, dtype=torch.float64, device=out.device)
    for a in range(case["n"]):
        rows = torch.nonzero(s["owner"] == a).flatten()
        at = torch.nonzero(s["idx"] == a).flatten()
        A, Bt, X = s["A"][rows].double(), s["Bt"][rows].double(), s["X"][at].double()
        if case["op"] == "fwd":
            out[at] += 2.0 * (X @ A.t()) @ Bt
            continue
        dY = s["dY"][at].double()
        G = 2.0 * dY @ Bt.t()
        out[at] += G @ A
        dA[rows] = G.t() @ X
        dBt[rows] = 2.0 * s["U"][at][:, :rows.numel()].double().t() @ dY
    return out if case["op"] == "fwd" else {"dX": out, "dA": dA, "dBt": dBt}
