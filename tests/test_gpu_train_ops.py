"""GPU checks of the norm, the 8-bit checkpoints, the adapter gradient from one and the loss,
against the float64 oracle on the same (already rounded) inputs.

Bounds, with u = 2^-24 and u_out the rounding of the output (2^-8 bf16, 2^-11 half, 2^-24
float32; half outputs also 2^-25, half the smallest step):

  norm     a sum of K squares in fp32 by at most 64 sequential terms and a tree, a root and a
           quotient, and a product or two: 100 u relative on rstd, n and y; h one rounding
  norm bwd the same relative error on each term: 2^-16 of rstd (|d| + |n| mean |d n|)
  sums over M tokens (dweight, dA): (M + 64) u of the sum of magnitudes; dA's operands may be
           split in two halves of 11 bits: 2^-21 of the magnitudes more
  loss     a logit of D products, added to an fp32 sum 16 at a time by the tensor cores, each
           step losing up to 2^-23: e_z = (D / 16 + 2) 2^-23 of the largest sum of magnitudes;
           loss and lse: 2 e_z and 2^-20 (1 + |value|)
  dx       16-bit exponentials (u_op = 2^-8 or 2^-11 of each term's magnitude, the target's own
           excepted; half ones also 2^-25 of the largest possible term), relative errors
           2 e_z + 2^-20 of every exponential, fp32 sums over V 16 at a time, and u_out
"""

import numpy as np
import pytest
import torch

from bit_nf4_quantized_gb300 import binding as b
from oracle import nf4 as onf4
from oracle import qlora
from oracle import train as ot

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U_OUT = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
FLOOR = {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -25}


def _rng(*ids):
    return np.random.Generator(np.random.PCG64([71, *ids]))


def _dev(a, dt=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(dt)


def _np(t):
    return t.double().cpu().numpy()


def _within(got, want, bound, what):
    got = _np(got)
    assert got.shape == want.shape
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside; worst ratio " \
                          f"{np.nanmax(np.abs(got - want) / np.maximum(bound, 1e-300)):.3g}"


def _ok():
    assert b.device_status(clear=True) == b.NF4_OK


def _stream_values(rng, M, K):
    x = rng.standard_normal((M, K)) * np.exp(0.4 * rng.standard_normal(K))
    x[:, rng.random(K) < 1 / 64] *= 6
    return x.astype(np.float32)


# ---- 8-bit checkpoints ----------------------------------------------------------------------

SIZES = [(1, 1), (3, 7), (1, 128), (5, 129), (2, 8), (33, 577), (64, 1000), (17, 4096), (2, 20000), (1, 33000)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K", SIZES)
def test_act8_bits(lib, dtype, M, K):
    x = _dev(_stream_values(_rng(1, M, K), M, K), DT[dtype])
    if M > 2:
        x[1, :min(K, 200)] = 0                       # a block of zeros
        x[2, :min(K, 64)] = 127 * x[2, 0].sign()     # values on the grid's ties
    codes, scales = ot.act8_quantize(x.float().cpu().numpy())
    c = b.qlora_act8_quantize(x)
    assert np.array_equal(c.codes.cpu().numpy(), codes)
    assert np.array_equal(c.scales.cpu().numpy().view(np.uint32), scales.view(np.uint32))
    w = _dev(_rng(2, K).standard_normal(K))
    for out in DT.values():
        want = torch.from_numpy(codes.astype(np.float32) * np.repeat(scales, 128, axis=1)[:, :K])
        assert torch.equal(b.qlora_act8_dequantize(c, out).cpu(), want.to(out))
        got = b.qlora_act8_dequantize(c, out, weight=w)
        assert torch.equal(got.cpu(), (want * w.cpu()).to(out))
    _ok()


def test_act8_extremes(lib):
    x = torch.zeros(4, 300, device=DEV)
    x[0, 0] = 2.0 ** -117                            # under the smallest amax: zeros
    x[1, 0], x[1, 1] = 3.4e38, -3.4e38               # the largest finite values
    x[2, 5] = 2.0 ** -116
    c = b.qlora_act8_quantize(x)
    _ok()
    assert not c.codes[0].any() and not c.scales[0].any()
    assert c.codes[1, :2].tolist() == [127, -127] and torch.isfinite(c.scales).all()
    assert c.codes[2, 5] == 127
    x[3, 130], x[2, 299] = float("nan"), float("inf")
    c = b.qlora_act8_quantize(x)
    assert b.device_status(clear=True) == b.NF4_ERR_NONFINITE
    v = b.qlora_act8_dequantize(c, torch.float32)
    assert torch.isnan(v[3, 128:256]).all() and torch.isnan(v[2, 256:]).all()
    assert torch.isfinite(v[3, :128]).all() and torch.isfinite(v[3, 256:]).all() and torch.isfinite(v[:2]).all()


# ---- dA from a checkpoint -----------------------------------------------------------------------

def _grad_bound(G, x, s, M):
    return s * (2.0 ** -21 + (M + 64) * U) * (np.abs(G).T @ np.abs(x)) * 1.01


@pytest.mark.parametrize("M,K,r", [(1, 1, 1), (1, 128, 16), (2, 7, 3), (15, 130, 16), (64, 576, 16), (65, 577, 8),
                                   (129, 200, 17), (500, 1000, 64), (1000, 136, 256), (4097, 640, 16), (300, 4096, 33)])
@pytest.mark.parametrize("weight", [False, True])
def test_grad_a(lib, M, K, r, weight):
    rng = _rng(3, M, K, r)
    codes, scales = ot.act8_quantize(_stream_values(rng, M, K))
    G = (rng.standard_normal((M, r)) * np.exp(2 * rng.standard_normal((M, 1))) * 1e-4).astype(np.float32)
    w = rng.standard_normal(K).astype(np.float32) if weight else None
    c = b.Act8(torch.from_numpy(codes).to(DEV), _dev(scales))
    dA = b.qlora_act8_grad_a(_dev(G), c, 32.0, weight=None if w is None else _dev(w))
    x = ot.act8_values(codes, scales) * (1.0 if w is None else w)
    s = 32.0 / r
    want = ot.grad_a(G, x, s)
    _within(dA, want, _grad_bound(G, x, s, M), "dA")
    assert qlora.rel_frobenius(_np(dA), want) <= 1e-5
    again = b.qlora_act8_grad_a(_dev(G), c, 32.0, weight=None if w is None else _dev(w))
    assert torch.equal(dA, again)
    rs = b.qlora_act8_grad_a(_dev(G), c, 32.0, mode=b.SCALE_RSLORA)
    assert qlora.rel_frobenius(_np(rs), ot.grad_a(G, ot.act8_values(codes, scales), 32.0 / np.sqrt(r))) <= 1e-5
    _ok()


@pytest.mark.parametrize("gmag,smag", [(1e-30, 1.0), (1e30, 1e-3), (1.0, 1e-30), (1e-20, 1e20), (0.0, 1.0)])
def test_grad_a_ranges(lib, gmag, smag):
    """G and the scales anywhere in float32's range keep their relative accuracy."""
    rng = _rng(4)
    M, K, r = 70, 300, 16
    G = (rng.standard_normal((M, r)) * gmag).astype(np.float32)
    codes, scales = ot.act8_quantize(rng.standard_normal((M, K)).astype(np.float32))
    scales = (scales * np.float32(smag)).astype(np.float32)
    dA = b.qlora_act8_grad_a(_dev(G), b.Act8(torch.from_numpy(codes).to(DEV), _dev(scales)), 16.0)
    x = ot.act8_values(codes, scales)
    _within(dA, ot.grad_a(G, x, 1.0), _grad_bound(G, x, 1.0, M) + 2.0 ** -140, "dA")


@pytest.mark.parametrize("M,K,r", [(8192, 14336, 64), (30000, 1024, 16), (5000, 777, 20)])
def test_grad_a_of_long_batches(lib, M, K, r):
    """More tokens than a slice adds up in the tensor cores: the same bound, in norm 1e-5 (float32)."""
    gen = torch.Generator(device=DEV).manual_seed(M)
    c = b.qlora_act8_quantize(torch.randn(M, K, generator=gen, device=DEV))
    G = torch.randn(M, r, generator=gen, device=DEV) * 1e-3
    dA = b.qlora_act8_grad_a(G, c, float(r)).double()
    x = c.codes.double() * c.scales.double().repeat_interleave(128, 1)[:, :K]
    want, mag = G.double().T @ x, G.double().abs().T @ x.abs()
    assert ((dA - want).abs() <= (2.0 ** -21 + (M + 64) * U) * mag).all()
    assert (dA - want).norm() <= 1e-5 * want.norm()
    _ok()


def test_grad_a_no_tokens_and_nan(lib):
    c = b.Act8.empty(0, 256)
    assert not b.qlora_act8_grad_a(torch.empty(0, 4, device=DEV), c, 1.0).any()
    x = torch.randn(40, 256, device=DEV)
    x[3, 200] = float("nan")
    c = b.qlora_act8_quantize(x)
    b.device_status(clear=True)
    dA = b.qlora_act8_grad_a(torch.randn(40, 4, device=DEV), c, 1.0)
    assert torch.isnan(dA[:, 128:]).all() and torch.isfinite(dA[:, :128]).all()


@pytest.mark.parametrize("compute,M,N,K", [("bf16", 40, 136, 192), ("f16", 300, 1024, 640), ("bf16", 5, 64, 1024),
                                           ("f32", 33, 100, 70)])
@pytest.mark.parametrize("decoded", [False, True])
def test_linear_backward_from_checkpoint(lib, compute, M, N, K, decoded):
    if decoded and compute == "f32":
        return
    rng = _rng(5, M, N)
    r, alpha = 16, 32.0
    dt = DT[compute]
    wq = b.nf4_quantize(_dev(rng.standard_normal((N, K)) * 0.02))
    x = _dev(_stream_values(rng, M, K), dt)
    A, B = _dev(rng.standard_normal((r, K)) / r), _dev(rng.standard_normal((N, r)) * 0.01)
    dy = _dev(rng.standard_normal((M, N)), dt)
    gain = _dev(1 + 0.1 * rng.standard_normal(K))
    c = b.qlora_act8_quantize(x)
    T = (b.qlora_act8_dequantize(c, torch.float32, weight=gain) @ A.T).contiguous()
    W = b.nf4_dequantize(wq, dt) if decoded else wq
    dx, dA, dB = b.qlora_linear_bwd_act8(dy, c, T, W, A, B, alpha, weight=gain)
    xv = ot.act8_values(c.codes.cpu().numpy(), c.scales.cpu().numpy()) * _np(gain)
    s = qlora.lora_scale(alpha, r)
    wd = _np(b.nf4_dequantize(wq, dt))
    A64, B64, dy64 = _np(A), _np(B), _np(dy)
    tol = 1e-5 if compute == "f32" else 2e-2          # the linear's stated tolerances
    assert qlora.rel_frobenius(_np(dx), dy64 @ wd + s * (dy64 @ B64) @ A64) <= tol
    assert qlora.rel_frobenius(_np(dA), s * (dy64 @ B64).T @ xv) <= tol
    assert qlora.rel_frobenius(_np(dB), s * dy64.T @ _np(T)) <= tol
    _ok()


# ---- the norm -------------------------------------------------------------------------------------

NORM_SIZES = [(1, 1), (2, 5), (1, 4096), (5, 129), (9, 576), (300, 64), (33, 1531), (8, 6000), (3, 14336), (2, 16384),
              (2, 16392), (2, 20001)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K", NORM_SIZES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm_forward(lib, dtype, M, K, residual):
    rng = _rng(6, M, K)
    x = _dev(_stream_values(rng, M, K), DT[dtype])
    r = _dev(_stream_values(rng, M, K), DT[dtype]) if residual else None
    w = _dev(1 + 0.2 * rng.standard_normal(K))
    y, h, rstd, c = b.qlora_rms_norm_fwd(x, w, 1e-5, residual=r, checkpoint=True)
    wy, wh, wr, wn = ot.rms_norm_fwd(_np(x), None if r is None else _np(r), _np(w), 1e-5)
    e = 100 * U
    _within(rstd, wr, e * wr, "rstd")
    _within(y, wy, (U_OUT[dtype] + e) * np.abs(wy) * 1.01 + FLOOR[dtype] + 2 * U * wr[:, None] * np.abs(_np(w)) * (
        np.abs(_np(x)) + (0 if r is None else np.abs(_np(r)))), "y")
    if residual:
        _within(h, wh, (U_OUT[dtype] + U) * np.abs(wh) * 1.01 + FLOOR[dtype], "h")
    else:
        assert h.data_ptr() == x.data_ptr()
    step = np.repeat(_np(c.scales), 128, axis=1)[:, :K]
    got = ot.act8_values(c.codes.cpu().numpy(), c.scales.cpu().numpy())
    slack = 2 * e * np.abs(wn) + 2 * U * wr[:, None] * (np.abs(_np(x)) + (0 if r is None else np.abs(_np(r))))
    assert np.all(np.abs(got - wn) <= 0.5 * step * (1 + 2.0 ** -14) + slack)
    top = np.array([[np.abs(row[i:i + 128]).max() for i in range(0, K, 128)] for row in wn])
    assert np.all(np.abs(_np(c.scales) * 127 - top) <= 1e-5 * top + 1e-30)
    y2, _, rstd2, none = b.qlora_rms_norm_fwd(x, w, 1e-5, residual=r)
    assert none is None and torch.equal(y, y2) and torch.equal(rstd, rstd2)
    _ok()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K", NORM_SIZES)
@pytest.mark.parametrize("saved", ["h", "checkpoint"])
@pytest.mark.parametrize("full", [False, True])
def test_norm_backward(lib, dtype, M, K, saved, full):
    rng = _rng(7, M, K)
    h = _dev(_stream_values(rng, M, K), DT[dtype])
    w = _dev(1 + 0.2 * rng.standard_normal(K))
    dy = _dev(rng.standard_normal((M, K)), DT[dtype])
    dres = _dev(rng.standard_normal((M, K)), DT[dtype]) if full else None
    _, _, rstd, c = b.qlora_rms_norm_fwd(h, w, 1e-5, checkpoint=True)
    n = _np(h) * _np(rstd)[:, None] if saved == "h" else ot.act8_values(c.codes.cpu().numpy(), c.scales.cpu().numpy())
    dx, dw = b.qlora_rms_norm_bwd(dy, h if saved == "h" else c, rstd, w, dresidual=dres, dweight=full)
    wdx, wdw = ot.rms_norm_bwd(_np(dy), n, _np(rstd), _np(w), None if dres is None else _np(dres))
    d = np.abs(_np(dy) * _np(w))
    mag = _np(rstd)[:, None] * (d + np.abs(n) * (d * np.abs(n)).mean(axis=1, keepdims=True))
    if full:
        mag = mag + np.abs(_np(dres))
    _within(dx, wdx, U_OUT[dtype] * np.abs(wdx) * 1.01 + 2.0 ** -16 * mag + FLOOR[dtype], "dx")
    if full:
        _within(dw, wdw, (M + 64) * U * (np.abs(_np(dy)) * np.abs(n)).sum(axis=0), "dweight")
        _, dw2 = b.qlora_rms_norm_bwd(dy, h if saved == "h" else c, rstd, w, dresidual=dres, dweight=True)
        assert torch.equal(dw, dw2)
    else:
        assert dw is None


@pytest.mark.parametrize("K", [576, 577])
def test_norm_backward_many_rows(lib, K):
    """More rows than the grid holds at once: every group walks over several."""
    rng = _rng(8, K)
    M = 9001
    h, dy = _dev(rng.standard_normal((M, K)), torch.bfloat16), _dev(rng.standard_normal((M, K)), torch.bfloat16)
    w = _dev(1 + 0.2 * rng.standard_normal(K))
    _, _, rstd, _ = b.qlora_rms_norm_fwd(h, w)
    dx, dw = b.qlora_rms_norm_bwd(dy, h, rstd, w, dweight=True)
    n = _np(h) * _np(rstd)[:, None]
    wdx, wdw = ot.rms_norm_bwd(_np(dy), n, _np(rstd), _np(w), None)
    _within(dw, wdw, (M + 64) * U * (np.abs(_np(dy)) * np.abs(n)).sum(axis=0), "dweight")
    assert qlora.rel_frobenius(_np(dx), wdx) <= 2.0 ** -8


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,K", [(2503, 1025), (1201, 2050), (1600, 1533), (631, 4097), (700, 8195), (331, 10001)])
def test_norm_rows_off_their_alignment(lib, dtype, M, K):
    """Rows that start and end inside a 16-byte piece, several a worker: values, in place, and nothing
    written past the tensors' ends."""
    rng = _rng(9, M, K)
    dt, pad = DT[dtype], 64

    def tail(like, n=M * K):
        flat = torch.full((n + pad,), 77, dtype=like, device=DEV)
        return flat, flat[:n]

    x, r, dy = (_dev(rng.standard_normal((M, K)), dt) for _ in range(3))
    w = _dev(1 + 0.2 * rng.standard_normal(K))
    bufs = {k: tail(dt) for k in ("y", "h", "dx")}
    y, h, dx = (bufs[k][1].view(M, K) for k in ("y", "h", "dx"))
    cf, cv = tail(torch.int8)
    c = b.Act8(cv.view(M, K), torch.empty(M, (K + 127) // 128, device=DEV))
    _, _, rstd, _ = b.qlora_rms_norm_fwd(x, w, 1e-5, residual=r, y=y, h=h, checkpoint=c)
    wy, wh, wr, wn = ot.rms_norm_fwd(_np(x), _np(r), _np(w), 1e-5)
    e = 100 * U
    near = 2 * U * wr[:, None] * (np.abs(_np(x)) + np.abs(_np(r)))
    _within(rstd, wr, e * wr, "rstd")
    _within(y, wy, (U_OUT[dtype] + e) * np.abs(wy) * 1.01 + FLOOR[dtype] + near * np.abs(_np(w)), "y")
    _within(h, wh, (U_OUT[dtype] + U) * np.abs(wh) * 1.01 + FLOOR[dtype], "h")
    got = ot.act8_values(c.codes.cpu().numpy(), c.scales.cpu().numpy())
    step = np.repeat(_np(c.scales), 128, axis=1)[:, :K]
    assert np.all(np.abs(got - wn) <= 0.5 * step * (1 + 2.0 ** -14) + 2 * e * np.abs(wn) + near)
    x2, r2 = x.clone(), r.clone()
    b.qlora_rms_norm_fwd(x2, w, 1e-5, residual=r2, y=x2, h=r2)
    assert torch.equal(x2, y) and torch.equal(r2, h)
    for saved, n in ((h, _np(h) * _np(rstd)[:, None]), (c, got)):
        _, dw = b.qlora_rms_norm_bwd(dy, saved, rstd, w, dresidual=r, dweight=True, dx=dx)
        wdx, wdw = ot.rms_norm_bwd(_np(dy), n, _np(rstd), _np(w), _np(r))
        d = np.abs(_np(dy) * _np(w))
        mag = _np(rstd)[:, None] * (d + np.abs(n) * (d * np.abs(n)).mean(axis=1, keepdims=True)) + np.abs(_np(r))
        _within(dx, wdx, U_OUT[dtype] * np.abs(wdx) * 1.01 + 2.0 ** -16 * mag + FLOOR[dtype], "dx")
        _within(dw, wdw, (M + 64) * U * (np.abs(_np(dy)) * np.abs(n)).sum(axis=0), "dweight")
        once = dx.clone()
        b.qlora_rms_norm_bwd(dy, saved, rstd, w, dresidual=r, dx=dx)      # a frozen weight's form
        assert qlora.rel_frobenius(_np(dx), _np(once)) <= U_OUT[dtype]
    for flat, _ in (*bufs.values(), (cf, cv)):
        assert (flat[M * K:] == 77).all()
    _ok()


def test_norm_zero_rows_and_in_place(lib):
    w = torch.ones(200, device=DEV)
    x = torch.zeros(3, 200, device=DEV)
    y, _, rstd, c = b.qlora_rms_norm_fwd(x, w, 1e-6, checkpoint=True)
    assert not y.any() and not c.codes.any() and torch.isfinite(rstd).all()
    _ok()
    x, r = torch.randn(5, 200, device=DEV), torch.randn(5, 200, device=DEV)
    y, h, _, _ = b.qlora_rms_norm_fwd(x, w, residual=r)
    x2, r2 = x.clone(), r.clone()
    b.qlora_rms_norm_fwd(x2, w, residual=r2, y=x2, h=r2)
    assert torch.equal(x2, y) and torch.equal(r2, h)
    e = b.qlora_rms_norm_fwd(torch.empty(0, 64, device=DEV), torch.ones(64, device=DEV), checkpoint=True)
    assert e[0].shape == (0, 64)
    _, dw = b.qlora_rms_norm_bwd(torch.empty(0, 64, device=DEV), torch.empty(0, 64, device=DEV),
                                 torch.empty(0, device=DEV), torch.ones(64, device=DEV), dweight=True)
    assert not dw.any()


# ---- the loss ---------------------------------------------------------------------------------------

def _loss_case(M, V, D, dtype, seed, lean=12.0, ignore=0.2):
    rng = _rng(9, M, V, D, seed)
    W = _dev(rng.standard_normal((V, D)) * 0.05, DT[dtype])
    t = rng.integers(0, V, M)
    w = _np(W)[t]
    x = rng.standard_normal((M, D)) + rng.random((M, 1)) * lean * w / np.maximum(np.linalg.norm(w, axis=1, keepdims=True), 1e-9)
    if M > 1:
        t = np.where(rng.random(M) < ignore, -100, t)
    return _dev(x, DT[dtype]), W, t


def _check_loss(x, W, t, g, dtype, loss, lse, dx, ref=None):
    X, Wn = _np(x), _np(W)
    D, V = X.shape[1], Wn.shape[0]
    ref = ot.lm_loss(X, Wn, t, 1.0 if g is None else g) if ref is None else ref
    live = ref["scale"] != 0
    mag = (np.abs(X) @ np.abs(Wn).T).max(axis=1)
    ez = (D / 16 + 2) * 2.0 ** -23 * mag
    _within(loss, ref["loss"], 2 * ez + 2.0 ** -20 * (1 + np.abs(ref["loss"])), "loss")
    _within(lse, ref["lse"], 2 * ez + 2.0 ** -20 * (1 + np.abs(ref["lse"])), "lse")
    assert not _np(loss)[~live].any() and not _np(lse)[~live].any()
    if dx is None:
        return
    aw = np.abs(Wn)
    terms = ref["others"] @ aw
    y = np.where(live, t, 0)
    own = ref["rest"][:, None] * aw[y]
    u_op = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    rel = (2 * ez + 2.0 ** -20)[:, None] + (V / 16 + 8) * 2.0 ** -23
    small = 0.0 if dtype == "bf16" else 2.0 ** -25 * aw.sum(axis=0)[None, :]
    bound = np.abs(ref["scale"])[:, None] * (u_op * terms + rel * (terms + own) + small)
    _within(dx, ref["dx"], (bound + U_OUT[dtype] * np.abs(ref["dx"])) * 1.01 + FLOOR[dtype], "dx")
    assert not _np(dx)[~live].any()


LOSS_SIZES = [(1, 1, 64), (1, 300, 64), (2, 2, 72), (3, 257, 64), (17, 256, 576), (130, 1000, 200), (257, 513, 576),
              (300, 5000, 136), (64, 12001, 1000), (600, 300, 1096),
              # few tokens: the pass over the vocabulary's bytes, its limits and just past them
              (8, 1000, 4096), (5, 333, 1000), (1, 5000, 2048), (8, 40, 64), (4, 700, 4104), (9, 700, 576)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,V,D", LOSS_SIZES)
def test_loss(lib, dtype, M, V, D):
    x, W, t = _loss_case(M, V, D, dtype, 0)
    g = _rng(10, M).standard_normal(M).astype(np.float32)
    g[g == 0] = 1
    loss, lse, dx = b.qlora_lm_loss(x, W, torch.from_numpy(t).to(DEV), grad_scale=_dev(g))
    _check_loss(x, W, t, g.astype(np.float64), dtype, loss, lse, dx)
    again = b.qlora_lm_loss(x, W, torch.from_numpy(t).to(DEV), grad_scale=_dev(g))
    assert all(torch.equal(p, q) for p, q in zip((loss, lse, dx), again))
    l2, e2, none = b.qlora_lm_loss(x, W, torch.from_numpy(t).to(DEV), need_dx=False)
    assert none is None
    _check_loss(x, W, t, None, dtype, l2, e2, None)
    one = torch.full((1,), 0.25, device=DEV)
    _, _, d3 = b.qlora_lm_loss(x, W, torch.from_numpy(t).to(DEV), grad_scale=one)
    _, _, d4 = b.qlora_lm_loss(x, W, torch.from_numpy(t).to(DEV))
    _check_loss(x, W, t, 0.25, dtype, loss, lse, d3)
    _check_loss(x, W, t, None, dtype, loss, lse, d4)
    _ok()


# one launch, or several: either side of where one takes less time; hidden sizes around the one
# launch's groups of 32, 64, 128, 256 and 512; tokens and entries around its 16
LOSS_EDGES = [(15, 15, 64), (16, 16, 72), (17, 17, 88), (33, 1500, 120), (1, 31, 128), (40, 129, 136), (100, 900, 256),
              (20, 500, 264), (50, 300, 512), (6, 170, 520), (3, 100, 1024), (700, 600, 64), (3000, 90, 80),
              (300, 30000, 136), (7, 60000, 72), (100, 20000, 576), (1, 40000, 256), (500, 9000, 1024)]
# few tokens over a vocabulary that every SM takes a part of
LOSS_PARTS = [(2, 9000, 1616), (16, 9001, 512), (17, 5000, 256), (33, 7001, 136), (9, 3000, 1032), (1, 9000, 2048),
              (12, 20000, 64), (3, 700, 216)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,V,D", LOSS_EDGES + LOSS_PARTS)
def test_loss_in_one_launch_or_several(lib, dtype, M, V, D):
    x, W, t = _loss_case(M, V, D, dtype, 7)
    tt = torch.from_numpy(t).to(DEV)
    g = _rng(12, M).random(M).astype(np.float32) + 0.5
    loss, lse, dx = b.qlora_lm_loss(x, W, tt, grad_scale=_dev(g))
    _check_loss(x, W, t, g.astype(np.float64), dtype, loss, lse, dx)
    again = b.qlora_lm_loss(x, W, tt, grad_scale=_dev(g))
    assert all(torch.equal(p, q) for p, q in zip((loss, lse, dx), again))
    l2, e2, _ = b.qlora_lm_loss(x, W, tt, need_dx=False)
    _check_loss(x, W, t, None, dtype, l2, e2, None)
    _ok()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("above", [5.0, 70.0, 200.0])
@pytest.mark.parametrize("M,V", [(600, 30000), (8, 60000), (40, 400)])
def test_loss_spikes_in_every_form(lib, dtype, above, M, V):
    """An entry far above the target's logit, and one far below all others."""
    D = 64
    rng = _rng(13, M)
    W = rng.standard_normal((V, D)) * 0.05
    x = rng.standard_normal((M, D))
    W[:, 0], x[:, 0] = 0.0, 0.0
    W[[V // 2, V - 1], 0] = 1.0
    W[V // 3, 0] = -1.0
    x[5, 0] = x[M // 2, 0] = x[M - 1, 0] = above
    t = rng.integers(0, V // 4, M)
    t[6] = -100
    t[0], x[0, 0] = V - 1, above                  # a sure token
    W, x = _dev(W, DT[dtype]), _dev(x, DT[dtype])
    loss, lse, dx = b.qlora_lm_loss(x, W, torch.from_numpy(t).to(DEV))
    _check_loss(x, W, t, None, dtype, loss, lse, dx)
    _ok()


@pytest.mark.parametrize("dq", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,V,D", [(5, 300, 64), (140, 1025, 576)])
def test_loss_of_a_stored_head(lib, dtype, dq, M, V, D):
    x, W, t = _loss_case(M, V, D, dtype, 1)
    q = b.nf4_quantize(W.float(), double_quant=dq)
    w16 = b.nf4_dequantize(q, DT[dtype])
    tt = torch.from_numpy(t).to(DEV)
    got = b.qlora_lm_loss(x, q, tt)
    want = b.qlora_lm_loss(x, w16, tt)
    for p, r in zip(got, want):
        assert torch.equal(p, r)
    _check_loss(x, w16, t, None, dtype, *got)
    l2, _, _ = b.qlora_lm_loss(x, q, tt, need_dx=False)
    assert torch.equal(l2, b.qlora_lm_loss(x, w16, tt, need_dx=False)[0])
    _ok()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("above", [5.0, 30.0, 70.0, 200.0])
@pytest.mark.parametrize("M", [600, 8])
def test_loss_spikes_far_above_the_target(lib, dtype, above, M):
    """One vocabulary entry `above` the target's logit, for some tokens of some tiles."""
    V, D = 1500, 64
    rng = _rng(11)
    W = rng.standard_normal((V, D)) * 0.05
    x = rng.standard_normal((M, D))
    W[:, 0], x[:, 0] = 0.0, 0.0
    spike = [700, 1400]
    W[spike, 0] = 1.0
    x[5, 0] = x[M // 2, 0] = x[M - 1, 0] = above
    t = rng.integers(0, 256, M)
    t[6] = -100
    W, x = _dev(W, DT[dtype]), _dev(x, DT[dtype])
    loss, lse, dx = b.qlora_lm_loss(x, W, torch.from_numpy(t).to(DEV))
    _check_loss(x, W, t, None, dtype, loss, lse, dx)
    _ok()


def _big_reference(x, W, t):
    """The float64 loss on the device, for sizes that numpy would take long over."""
    X, Wd = x.double(), W.double()
    tt = torch.from_numpy(t).to(DEV)
    live = tt != -100
    y = torch.where(live, tt, 0)[:, None]
    z = X @ Wd.T
    lse = torch.logsumexp(z, 1)
    zt = z.gather(1, y)[:, 0]
    p = torch.exp(z - lse[:, None])
    p.scatter_(1, y, 0.0)
    rest = p.sum(1)
    dx = (p @ Wd - rest[:, None] * Wd[y[:, 0]]) * live[:, None]
    return (lse - zt) * live, lse * live, dx


@pytest.mark.parametrize("M,V,D,spike", [(4096, 40000, 64, False), (4096, 40000, 64, True), (9000, 700, 72, False),
                                         (2000, 70001, 64, True)])
def test_loss_in_pieces(lib, M, V, D, spike):
    """More vocabulary than one piece holds, and more tokens than one pass takes; with spikes the
    reference rises in a later piece."""
    x, W, t = _loss_case(M, V, D, "bf16", 2, lean=4.0)
    if spike:
        W[:, 0] = 0
        x[:, 0] = 0
        W[V - 100, 0], W[V // 2, 0] = 2.0, 1.0
        x[::97, 0] = 64.0
    loss, lse, dx = b.qlora_lm_loss(x, W, torch.from_numpy(t).to(DEV))
    wl, we, wd = _big_reference(x, W, t)
    # the same terms as _check_loss, in norms: 2^-8 for the exponentials and 2^-8 for dx
    assert qlora.rel_frobenius(_np(loss), wl.cpu().numpy()) <= 1e-5
    assert qlora.rel_frobenius(_np(lse), we.cpu().numpy()) <= 1e-5
    assert qlora.rel_frobenius(_np(dx), wd.cpu().numpy()) <= 2.0 ** -7
    rows = (dx.double() - wd).norm(dim=1) / wd.norm(dim=1).clamp(min=1e-6)
    assert rows.max().item() <= 2.0 ** -6
    _ok()


def test_loss_tokens_that_do_not_count(lib):
    x, W, t = _loss_case(70, 400, 64, "bf16", 3)
    tt = torch.from_numpy(t).to(DEV)
    x[np.flatnonzero(t == -100)[0]] = float("nan")       # what an ignored token holds does not matter
    loss, lse, dx = b.qlora_lm_loss(x, W, tt)
    assert torch.isfinite(loss).all() and torch.isfinite(lse).all() and torch.isfinite(dx).all()
    for grad in (True, False):
        out = b.qlora_lm_loss(x, W, torch.full_like(tt, -100), need_dx=grad)
        assert not any(o.any() for o in out if o is not None)
    out = b.qlora_lm_loss(x[:5], W, torch.full_like(tt[:5], 7), ignore_index=7)
    assert not any(o.any() for o in out)
    _ok()
    bad = torch.full((3,), 1, device=DEV)
    bad[1] = 400
    loss, _, dx = b.qlora_lm_loss(x[20:23].nan_to_num(), W, bad)
    assert b.device_status(clear=True) == b.NF4_ERR_ARG
    assert loss[1] == 0 and not dx[1].any() and (loss[[0, 2]] > 0).all()
    assert b.qlora_lm_loss(x[:0], W, tt[:0])[2].shape == (0, 64)


def test_loss_nan_stays_in_its_row(lib):
    x, W, t = _loss_case(300, 700, 64, "bf16", 4, ignore=0.0)
    clean = b.qlora_lm_loss(x, W, torch.from_numpy(t).to(DEV))
    x[150, 3] = float("nan")
    got = b.qlora_lm_loss(x, W, torch.from_numpy(t).to(DEV))
    keep = torch.arange(300, device=DEV) != 150
    for c, g in zip(clean, got):
        assert torch.equal(c[keep], g[keep]) and torch.isnan(g[150]).all()


def test_loss_timeout_is_reported(lib):
    x, W, t = _loss_case(40, 300, 128, "bf16", 5)
    tt = torch.from_numpy(t).to(DEV)
    want = b.qlora_lm_loss(x, W, tt)
    b.debug_wait_timeout(True)
    b.qlora_lm_loss(x, W, tt)
    assert b.device_status(clear=True) == b.NF4_ERR_TIMEOUT
    got = b.qlora_lm_loss(x, W, tt)
    _ok()
    for p, r in zip(want, got):
        assert torch.equal(p, r)


# ---- strides, streams, refusals ------------------------------------------------------------------------

def test_strided_inputs_and_another_stream(lib):
    x, W, t = _loss_case(50, 300, 64, "bf16", 6)
    tt = torch.from_numpy(t).to(DEV)
    w = torch.rand(64, device=DEV) + 0.5
    res = torch.randn_like(x)
    want = b.qlora_lm_loss(x, W, tt)
    wn = b.qlora_rms_norm_fwd(x, w, residual=res, checkpoint=True)
    wide = torch.zeros(50, 200, dtype=x.dtype, device=DEV)
    wide[:, 3:67] = x
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = b.qlora_lm_loss(wide[:, 3:67], W.T.contiguous().T, tt, stream=side)
    gn = b.qlora_rms_norm_fwd(wide[:, 3:67], w, residual=res, checkpoint=True, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for p, r in zip(want, got):
        assert torch.equal(p, r)
    assert all(torch.equal(p, r) for p, r in zip(wn[:3], gn[:3])) and torch.equal(wn[3].codes, gn[3].codes)
    dA = b.qlora_act8_grad_a(torch.randn(4, 50, device=DEV).T, wn[3], 4.0)
    assert dA.shape == (4, 64)


def test_refusals_of_the_binding(lib):
    x = torch.randn(4, 64, device=DEV)
    w = torch.ones(64, device=DEV)
    c = b.qlora_act8_quantize(x)
    bad = [
        lambda: b.qlora_rms_norm_fwd(x.cpu(), w),
        lambda: b.qlora_rms_norm_fwd(x, w[:32]),
        lambda: b.qlora_rms_norm_fwd(x, w.half()),
        lambda: b.qlora_rms_norm_fwd(x, w, residual=x.half()),
        lambda: b.qlora_rms_norm_fwd(x, w, y=torch.empty(64, 4, device=DEV).T),
        lambda: b.qlora_rms_norm_bwd(x, c, torch.ones(3, device=DEV), w),
        lambda: b.qlora_act8_quantize(x[0]),
        lambda: b.qlora_act8_quantize(x, out=b.Act8.empty(4, 65)),
        lambda: b.qlora_act8_grad_a(torch.ones(5, 2, device=DEV), c, 1.0),
        lambda: b.qlora_act8_dequantize(c, torch.float32, weight=w[:5]),
        lambda: b.qlora_lm_loss(x.bfloat16(), x.half(), torch.zeros(4, dtype=torch.int64, device=DEV)),
        lambda: b.qlora_lm_loss(x.bfloat16(), x.bfloat16(), torch.zeros(4, dtype=torch.int32, device=DEV)),
        lambda: b.qlora_lm_loss(x.bfloat16(), x.bfloat16(), torch.zeros(4, dtype=torch.int64, device=DEV),
                                grad_scale=torch.ones(3, device=DEV)),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    t = torch.zeros(4, dtype=torch.int64, device=DEV)
    with pytest.raises(TypeError):
        b.qlora_act8_quantize(x.double())
    for f, status in [
        (lambda: b.qlora_lm_loss(x, x, t), b.NF4_ERR_DTYPE),
        (lambda: b.qlora_lm_loss(x[:, :40].bfloat16(), x[:, :40].bfloat16(), t), b.NF4_ERR_SHAPE),
        (lambda: b.qlora_rms_norm_fwd(x, w, eps=float("nan")), b.NF4_ERR_ARG),
        (lambda: b.qlora_act8_grad_a(torch.ones(4, 257, device=DEV), c, 1.0), b.NF4_ERR_ARG),
        (lambda: b.qlora_act8_grad_a(torch.ones(4, 2, device=DEV), c, float("inf")), b.NF4_ERR_ARG),
        (lambda: b.qlora_lm_loss(x.bfloat16(), x.bfloat16(), t, workspace=torch.empty(64, dtype=torch.uint8, device=DEV)),
         b.NF4_ERR_WORKSPACE),
    ]:
        with pytest.raises(b.Nf4Error) as e:
            f()
        assert e.value.status == status
