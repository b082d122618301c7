"""Float64 oracle of the many-adapter operators: the maps of a batch of
requests, the adapter term and its gradients ([P2] "The LoRA hypothesis": one
base in memory, a small adapter chosen per request).  Plain loops over requests
and adapters; adapter a is the pair A_a (r_a x k), B_a (d x r_a)."""
from __future__ import annotations

import numpy as np


def plan(lens, ids, n: int, T: int) -> dict:
    """starts, idx, order, seg of requests of lens[i] rows each with adapter
    ids[i] (outside [0, n): none), cut at T rows."""
    starts, idx = [0], np.full(T, -1, np.int32)
    groups = [[] for _ in range(n + 1)]
    for size, a in zip(lens, ids):
        lo = starts[-1]
        hi = min(T, lo + max(0, int(size)))
        a = int(a) if 0 <= a < n else -1
        idx[lo:hi] = a
        groups[a].extend(range(lo, hi))
        starts.append(hi)
    order = [t for g in groups for t in g]
    order = np.array(order + [-1] * (T - len(order)), np.int32)
    seg = np.cumsum([0] + [len(g) for g in groups]).astype(np.int32)
    return {"starts": np.array(starts, np.int32), "idx": idx, "order": order, "seg": seg}


def forward(X, A, B, s, idx, base=None) -> dict:
    """Y = base + s_a U B_a^T and U = X A_a^T, row by row of idx (lists A, B, s
    by adapter; rows with idx < 0 keep the base and have U = 0)."""
    T, d = X.shape[0], B[0].shape[0]
    Y = np.zeros((T, d)) if base is None else base.astype(np.float64).copy()
    U = np.zeros((T, max(a.shape[0] for a in A)))
    for a in range(len(A)):
        at = np.flatnonzero(idx == a)
        U[at, :A[a].shape[0]] = X[at] @ A[a].T
        Y[at] += s[a] * (U[at, :A[a].shape[0]] @ B[a].T)
    return {"Y": Y, "U": U}


def backward(X, A, B, s, idx, U, dY, base=None) -> dict:
    """dX (from `base`), and dA_a, dB_a of every adapter."""
    dX = np.zeros_like(X) if base is None else base.astype(np.float64).copy()
    dA, dB = [], []
    for a in range(len(A)):
        at = np.flatnonzero(idx == a)
        G = s[a] * (dY[at] @ B[a])
        dX[at] += G @ A[a]
        dA.append(G.T @ X[at])
        dB.append(s[a] * (dY[at].T @ U[at, :A[a].shape[0]]))
    return {"dX": dX, "dA": dA, "dB": dB}
