"""Oracle of the routed FFN's training pass, in 64 bits on whatever device
its tensors live: the forward of one expert's rows, and the gradients from
their formulas, row group by row group."""
from __future__ import annotations

import torch


def forward(x, wg, wu, wd, w):
    """out [n, H] of rows x [n, H], weights wg, wu [I, H], wd [H, I], routed
    weights w [n]."""
    g, u = x @ wg.T, x @ wu.T
    return ((g * torch.sigmoid(g) * u) @ wd.T) * w[:, None]


def hidden_grads(dy, wd, w, g, u):
    """(b, dgate, dup, whidden, drw) from the output gradient and the
    pre-activations."""
    s = torch.sigmoid(g)
    h = g * s * u
    b = dy @ wd
    dh = b * w[:, None]
    return b, dh * u * (s + g * s * (1 - s)), dh * g * s, w[:, None] * h, (b * h).sum(1)


def backward(x, dy, wg, wu, wd, w):
    """Gradients of sum(forward * dy): (dx, dwg, dwu, dwd, dw)."""
    g, u = x @ wg.T, x @ wu.T
    _, dg, du, hw, dw = hidden_grads(dy, wd, w, g, u)
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dy.T @ hw, dw
