"""Inputs, oracle values and derived tolerances of the many-adapter tests."""
import numpy as np
import torch

import parameter_efficient_fine_nf4_b200 as q4
from oracle import requests as oracle
from tests.gpu_helpers import bf16_host_f64, f32_host_f64

# A rounding is off by at most half a step: bf16 2^-8, fp32 2^-24 (tensor
# cores may cut instead of round: a whole step, 2^-23, per fp32 addition).
BF16, F32 = 2.0 ** -8, 2.0 ** -23


def bf16_values(gen, shape, sigma):
    t = torch.from_numpy((gen.standard_normal(shape) * sigma).astype(np.float32)).to(torch.bfloat16)
    return t, t.double().numpy()


class Batch:
    """A pool, a batch of requests and their data, with the float64 oracle's
    values and, in `abs`, the same sums over absolute values (what errors are
    relative to)."""

    def __init__(self, k, d, ranks, lens, ids, T=None, seed=0, alphas=None):
        gen = np.random.Generator(np.random.Philox(key=seed))
        self.k, self.d, self.ranks, self.n = k, d, list(ranks), len(ranks)
        self.lens, self.ids = list(lens), list(ids)
        self.T = T = int(sum(max(0, v) for v in lens)) if T is None else T
        alphas = [r * (0.5 + 0.25 * i) for i, r in enumerate(ranks)] if alphas is None else alphas
        self.s = [float(np.float32(a / r)) for a, r in zip(alphas, ranks)]
        self.maps = oracle.plan(lens, ids, self.n, T)
        self.total = int(self.maps["starts"][-1])
        self.pool = q4.AdapterPool(k, d, ranks, alphas)
        self.A, self.B = [], []
        for a, r in enumerate(ranks):
            A, Af = bf16_values(gen, (r, k), 1.0 / r)
            B, Bf = bf16_values(gen, (d, r), 0.05)
            self.pool.load(a, A.cuda(), B.cuda())
            self.A.append(Af)
            self.B.append(Bf)
        (X, self.Xf), (dY, self.dYf) = bf16_values(gen, (T, k), 1.0), bf16_values(gen, (T, d), 1.0)
        (by, self.byf), (bx, self.bxf) = bf16_values(gen, (T, d), 1.0), bf16_values(gen, (T, k), 1.0)
        self.X, self.dY, self.base_y, self.base_x = X.cuda(), dY.cuda(), by.cuda(), bx.cuda()
        self.plan = q4.RequestPlan(len(self.lens), self.n, T)
        self.dev_lens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.dev_ids = torch.tensor(self.ids, dtype=torch.int32).cuda()
        q4.lora_requests_plan(self.dev_lens, self.dev_ids, self.plan)

    def check_maps(self):
        for name in ("starts", "idx", "order", "seg"):
            got = getattr(self.plan, name).cpu().numpy()
            assert np.array_equal(got, self.maps[name]), name

    def check_forward(self, Y, U, base=True):
        idx, m = self.maps["idx"], self.total
        ref = oracle.forward(self.Xf, self.A, self.B, self.s, idx, self.byf if base else None)
        ab = oracle.forward(abs(self.Xf), [abs(a) for a in self.A], [abs(b) for b in self.B], self.s, idx,
                            abs(self.byf) if base else None)
        # U: k products and sums in fp32
        self._within(f32_host_f64(U)[:m, :ref["U"].shape[1]], ref["U"][:m], (self.k + 2) * F32 * ab["U"][:m], "U")
        assert not U[:m, ref["U"].shape[1]:].any()
        for a, r in enumerate(self.ranks):
            assert not U[torch.from_numpy(np.flatnonzero(idx == a)).cuda(), r:].any()
        # Y: the sums above, U as at least two bf16 terms (2^-16), one rounding
        tol = BF16 * abs(ref["Y"]) + ((self.k + max(self.ranks) + 8) * F32 + BF16 ** 2) * ab["Y"] * (1 + BF16)
        self._within(bf16_host_f64(Y)[:m], ref["Y"][:m], tol[:m], "Y")

    def check_backward(self, dX, dA, dBt, U, base=True):
        idx, m = self.maps["idx"], self.total
        Uf = f32_host_f64(U)
        ref = oracle.backward(self.Xf, self.A, self.B, self.s, idx, Uf, self.dYf, self.bxf if base else None)
        ab = oracle.backward(abs(self.Xf), [abs(a) for a in self.A], [abs(b) for b in self.B], self.s, idx, abs(Uf),
                             abs(self.dYf), abs(self.bxf) if base else None)
        tol = BF16 * abs(ref["dX"]) + ((self.d + max(self.ranks) + 8) * F32 + BF16 ** 2) * ab["dX"] * (1 + BF16)
        self._within(bf16_host_f64(dX)[:m], ref["dX"][:m], tol[:m], "dX")
        for a, r in enumerate(self.ranks):
            rows, pad = self.pool.rows_of(a), slice(self.pool.firsts[a] + r, self.pool.firsts[a] + (r + 15) // 16 * 16)
            c = int((idx == a).sum())
            # G (d sums) or the given U, then c sums over the tokens; three bf16
            # terms hold a 32-bit value to 2^-24, counted with the roundings of s
            self._within(f32_host_f64(dA[rows]), ref["dA"][a], (self.d + 3 * c + 8) * F32 * ab["dA"][a], f"dA[{a}]")
            self._within(f32_host_f64(dBt[rows]), ref["dB"][a].T, (3 * c + 8) * F32 * ab["dB"][a].T, f"dBt[{a}]")
            assert not dA[pad].any() and not dBt[pad].any()

    @staticmethod
    def _within(got, ref, tol, what):
        assert np.all(np.isfinite(got)), f"{what}: non-finite"
        bad = np.abs(got - ref) > tol
        assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} values beyond the bound, worst " \
                              f"{float((np.abs(got - ref) / np.maximum(tol, 1e-300)).max()):.3g} of it"
