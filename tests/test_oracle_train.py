"""Pins of the float64 oracle of the norm, the 8-bit checkpoints and the loss (CPU): hand-worked
values, closed forms and finite differences."""

import numpy as np
import pytest

from oracle import train as ot


def _rng(i):
    return np.random.Generator(np.random.PCG64(71 + i))


def test_act8_by_hand():
    x = np.zeros((2, 130), np.float32)
    x[0, :4] = [127.0, -63.5, 0.5, 1.5]       # scale 1: ties to even
    x[0, 128:] = [-2.0, 1.0]                  # the ragged block has its own scale
    x[1, 0] = 2.0 ** -120                     # below the smallest amax: zeros
    codes, scales = ot.act8_quantize(x)
    assert codes[0, :4].tolist() == [127, -64, 0, 2]
    assert codes[0, 128:].tolist() == [-127, 64]
    assert scales[0, 0] == 1.0 and scales[0, 1] == np.float32(2) / np.float32(127)
    assert not codes[1].any() and not scales[1].any()
    assert ot.act8_values(codes, scales)[0, 0] == 127.0


@pytest.mark.parametrize("K", [1, 127, 128, 300])
def test_act8_error_is_half_a_step(K):
    x = _rng(K).standard_normal((5, K)).astype(np.float32)
    codes, scales = ot.act8_quantize(x)
    step = np.repeat(scales, ot.BLOCK, axis=1)[:, :K]
    assert np.all(np.abs(ot.act8_values(codes, scales) - x) <= 0.5 * step * (1 + 2.0 ** -15))
    assert np.abs(codes.astype(int)).max() == 127


def test_norm_gradient_by_differences():
    g = _rng(1)
    x, r, w, dy = g.standard_normal((3, 7)), g.standard_normal((3, 7)), g.standard_normal(7), g.standard_normal((3, 7))
    dres = g.standard_normal((3, 7))
    eps = 1e-5
    _, h, rstd, n = ot.rms_norm_fwd(x, r, w, eps)
    dx, dw = ot.rms_norm_bwd(dy, n, rstd, w, dres)

    def value(x, w):   # the loss whose gradient reaches h by the norm (dy) and by the residual (dres)
        y, h, _, _ = ot.rms_norm_fwd(x, r, w, eps)
        return (y * dy).sum() + (h * dres).sum()

    for _ in range(5):
        vx, vw = g.standard_normal(x.shape), g.standard_normal(w.shape)
        t = 1e-5
        num = (value(x + t * vx, w + t * vw) - value(x - t * vx, w - t * vw)) / (2 * t)
        # central differences: a third-derivative term of order t^2 and 1e-16 / t of rounding
        assert abs(num - ((dx * vx).sum() + (dw * vw).sum())) <= 1e-7 * (1 + abs(num))


def test_norm_of_constant_rows():
    y, _, rstd, n = ot.rms_norm_fwd(np.full((2, 9), -3.0), None, np.full(9, 2.0), 0.0)
    assert np.allclose(n, -1.0) and np.allclose(y, -2.0) and np.allclose(rstd, 1 / 3)


def test_loss_closed_forms():
    V, D = 11, 4
    out = ot.lm_loss(np.zeros((2, D)), _rng(2).standard_normal((V, D)), [3, -100])
    assert np.allclose(out["loss"], [np.log(V), 0]) and np.allclose(out["lse"], [np.log(V), 0])
    assert not out["dx"][1].any()
    one = ot.lm_loss(np.ones((1, D)), np.ones((1, D)), [0])     # a vocabulary of one: sure
    assert one["loss"][0] == 0 and not one["dx"].any()


def test_loss_gradient_by_differences():
    g = _rng(3)
    x, W, t = g.standard_normal((4, 6)), g.standard_normal((9, 6)), np.array([0, 8, -100, 4])
    scale = g.standard_normal(4)
    dx = ot.lm_loss(x, W, t, scale)["dx"]
    for _ in range(5):
        v = g.standard_normal(x.shape)
        h = 1e-5
        num = ((ot.lm_loss(x + h * v, W, t)["loss"] - ot.lm_loss(x - h * v, W, t)["loss"]) * scale).sum() / (2 * h)
        assert abs(num - (dx * v).sum()) <= 1e-7 * (1 + abs(num))


def test_loss_of_a_sure_token_keeps_its_digits():
    x = np.array([[40.0, 0.0]])
    W = np.array([[1.0, 0.0], [0.0, 1.0], [0.0, 2.0]])
    out = ot.lm_loss(x, W, [0])
    want = 2 * np.exp(-40.0)
    assert abs(out["loss"][0] - want) <= 1e-12 * want
    assert abs(out["rest"][0] - want) <= 1e-12 * want


def test_grad_a_by_loops():
    g = _rng(4)
    G, x = g.standard_normal((5, 2)), g.standard_normal((5, 3))
    want = [[0.5 * sum(G[m, j] * x[m, k] for m in range(5)) for k in range(3)] for j in range(2)]
    assert np.allclose(ot.grad_a(G, x, 0.5), want, rtol=1e-14, atol=0)
