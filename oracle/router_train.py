"""Oracle of the training router in 64 bits: the forward with its counts and
losses, and the backward pass by its formulas (test infrastructure only)."""
from __future__ import annotations

import numpy as np

from . import router as RT


def forward(x, w, k, mask=None):
    """x [T, H], w [E, H]; mask [T] of truth values (None: every token
    counts).  Returns a dict as the library's, in 64 bits."""
    T, E = x.shape[0], w.shape[0]
    on = np.ones(T, bool) if mask is None else np.asarray(mask).astype(bool)
    ids, vals = np.full((T, k), -1), np.zeros((T, k))
    probs, lse = np.zeros((T, E)), np.zeros(T)
    logits = np.zeros((T, E))
    if on.any():
        logits[on] = RT.router_logits(x[on], w)
        probs[on] = RT.softmax(logits[on])
        top = logits[on].max(1)
        lse[on] = top + np.log(np.exp(logits[on] - top[:, None]).sum(1))
        # the order of the logits themselves: exact where they are
        order = np.argsort(-logits[on], axis=1, kind="stable")[:, :k]
        ids[on], vals[on] = order, np.take_along_axis(probs[on], order, 1)
    counts = np.concatenate((np.bincount(ids[on].reshape(-1), minlength=E), [on.sum()]))
    n = int(on.sum())
    balance = E / (k * n) * (counts[:E] * probs[on].mean(0)).sum() if n else 0.0
    z = (lse[on] ** 2).mean() if n else 0.0
    return {"ids": ids, "vals": vals, "probs": probs, "lse": lse, "counts": counts, "losses": np.array([balance, z]),
            "logits": logits}


def dlogits(probs, lse, ids, counts, g, dlosses, mask=None):
    """dl [T, E] from the routed weights' gradients g [T, k] and the losses'."""
    T, E = probs.shape
    k, n = ids.shape[1], int(counts[E])
    on = np.ones(T, bool) if mask is None else np.asarray(mask).astype(bool)
    a, b = (0.0, 0.0) if dlosses is None or n == 0 else dlosses
    dl = np.zeros((T, E))
    for t in np.flatnonzero(on):
        dp = a * E * np.asarray(counts[:E], np.float64) / (k * max(n, 1) ** 2)
        for j in range(k):
            if 0 <= ids[t, j] < E:
                dp[ids[t, j]] += g[t, j]
        dl[t] = probs[t] * (dp - (probs[t] * dp).sum()) + 2 * b * lse[t] * probs[t] / max(n, 1)
    return dl


def backward(x, w, dl, mask=None):
    """(dx, dw) from dl."""
    on = np.ones(x.shape[0], bool) if mask is None else np.asarray(mask).astype(bool)
    return dl @ w, dl[on].T @ x[on]
