"""Float64 restatement of the operators around the linear: the RMS norm, 8-bit activation
checkpoints, the adapter gradient read from one, and the loss over a frozen head.

Only the checkpoint's codes are defined in float32 (amax, 127 / amax and the product that is
rounded); everything else is the plain formula in float64.
"""

import numpy as np

BLOCK = 128
TINY = np.float32(2.0 ** -116)


def act8_quantize(x):
    """(codes int8 [M, K], scales float32 [M, ceil(K / 128)]) of a float32 array of finite values."""
    x = np.asarray(x, dtype=np.float32)
    M, K = x.shape
    nb = -(-K // BLOCK)
    v = np.zeros((M, nb * BLOCK), dtype=np.float32)
    v[:, :K] = x
    v = v.reshape(M, nb, BLOCK)
    amax = np.abs(v).max(axis=2)
    live = amax >= TINY
    safe = np.where(live, amax, np.float32(1))
    inv = np.where(live, np.float32(127) / safe, np.float32(0))
    codes = np.rint(v * inv[:, :, None]).astype(np.int8).reshape(M, nb * BLOCK)[:, :K]
    return codes, np.where(live, safe / np.float32(127), np.float32(0)).astype(np.float32)


def act8_values(codes, scales):
    """The values the codes stand for, in float64 (code * scale is then exact)."""
    s = np.repeat(np.asarray(scales, dtype=np.float64), BLOCK, axis=1)[:, :codes.shape[1]]
    return np.asarray(codes, dtype=np.float64) * s


def grad_a(G, x, s):
    """dA = s G^T x."""
    return s * (np.asarray(G, dtype=np.float64).T @ x)


def rms_norm_fwd(x, residual, weight, eps):
    """(y, h, rstd, n)."""
    h = np.asarray(x, dtype=np.float64)
    if residual is not None:
        h = h + np.asarray(residual, dtype=np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    n = h * rstd[:, None]
    return n * np.asarray(weight, dtype=np.float64), h, rstd, n


def rms_norm_bwd(dy, n, rstd, weight, dresidual):
    """(dx, dweight) from the normalised rows n."""
    dy = np.asarray(dy, dtype=np.float64)
    d = dy * np.asarray(weight, dtype=np.float64)
    dx = np.asarray(rstd, dtype=np.float64)[:, None] * (d - n * (d * n).mean(axis=1, keepdims=True))
    if dresidual is not None:
        dx = dx + dresidual
    return dx, (dy * n).sum(axis=0)


def lm_loss(x, W, targets, g=1.0, ignore_index=-100):
    """dict(loss, lse, dx): softmax cross entropy of x W^T and its gradient times g (a number or
    one for each token); tokens with target ignore_index give zeros.  `others`: the softmax with
    the target's own entry left out (what dx's sum runs over)."""
    x, W = np.asarray(x, dtype=np.float64), np.asarray(W, dtype=np.float64)
    targets = np.asarray(targets)
    live = targets != ignore_index
    y = np.where(live, targets, 0)
    rows = np.arange(x.shape[0])
    z = x @ W.T
    top = z.max(axis=1, keepdims=True)
    e = np.exp(z - top)
    lse = np.log(e.sum(axis=1)) + top[:, 0]
    p = e / e.sum(axis=1, keepdims=True)
    p[rows, y] = 0.0
    rest = p.sum(axis=1)                    # 1 - p[target] without the cancellation
    own = np.exp(z[rows, y] - lse)
    loss = np.where(own > 0.5, np.log1p(rest / np.where(own > 0.5, own, 1.0)), lse - z[rows, y])
    scale = np.broadcast_to(np.asarray(g, dtype=np.float64), live.shape) * live
    dx = scale[:, None] * (p @ W - rest[:, None] * W[y])
    return dict(loss=loss * live, lse=lse * live, dx=dx, others=p, rest=rest, scale=scale)
