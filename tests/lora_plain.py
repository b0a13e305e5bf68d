"""The low-rank adapters' products and gradients in numpy, 64 bits, token by token of each adapter."""
import numpy as np


def forward(x, idx, a, b, scales, ranks, base):
    """x [T, K], a [n, r, K], b [n, N, r], base [T, N]; the parts of a and b past an adapter's rank may hold NaN."""
    y = base.copy()
    h = np.zeros((x.shape[0], a.shape[1]))
    for i in range(a.shape[0]):
        at = np.flatnonzero(idx == i)
        r = ranks[i]
        h[at, :r] = (x[at] @ a[i, :r].T) * scales[i]
        y[at] += h[at, :r] @ b[i, :, :r].T
    return y, h


def backward(x, dy, idx, a, b, scales, ranks, dx_base):
    dx = dx_base.copy()
    da, db = np.zeros(a.shape), np.zeros(b.shape)
    _, h = forward(x, idx, a, b, scales, ranks, np.zeros((x.shape[0], b.shape[1])))
    for i in range(a.shape[0]):
        at = np.flatnonzero(idx == i)
        r = ranks[i]
        g = (dy[at] @ b[i, :, :r]) * scales[i]
        dx[at] += g @ a[i, :r]
        da[i, :r] = g.T @ x[at]
        db[i, :, :r] = dy[at].T @ h[at, :r]
    return dx, da, db
