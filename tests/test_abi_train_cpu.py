"""C-ABI checks of the norm, the 8-bit checkpoints and the loss that need no GPU: sizes, and
invalid arguments refused before any device work."""

import ctypes

import pytest

from bit_nf4_quantized_gb300 import binding, build

P = 0x50000000           # addresses that are never read: every call here is refused first
ODD = 0x50000008
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def _act8(rows=4, cols=256, codes=P, scales=P):
    return ctypes.byref(binding._Act8(rows, cols, codes, scales))


def _nf4(numel):
    t = binding._Nf4Tensor()
    t.numel, t.double_quant, t.reserved = numel, 1, 0
    t.packed, t.absmax, t.nested_absmax, t.offset = P, P, P, P
    return ctypes.byref(t)


def test_sizes(lib):
    assert lib.qlora_act8_scales(3, 256) == 6 and lib.qlora_act8_scales(3, 257) == 9
    assert lib.qlora_act8_scales(0, 5) == 0 and lib.qlora_act8_scales(-1, 5) == 0 and lib.qlora_act8_scales(5, 0) == 0
    assert lib.qlora_act8_grad_a_workspace_bytes(4, 256, 0) == 0
    assert lib.qlora_act8_grad_a_workspace_bytes(4, 256, 257) == 0
    assert lib.qlora_rms_norm_bwd_workspace_bytes(0, 64) == 0
    assert lib.qlora_rms_norm_bwd_workspace_bytes(5, 64) >= 5 * 64 * 4 // 8
    assert lib.qlora_lm_loss_workspace_bytes(0, 10, 64, 0, 1) == 0
    # the gradient's workspace holds a piece of the vocabulary, not all of it
    M, V, D = 8192, 1 << 20, 4096
    score, grad = (lib.qlora_lm_loss_workspace_bytes(M, V, D, 0, g) for g in (0, 1))
    assert 0 < score < grad < 2 * M * V // 4
    # a stored head's decoded copy is a piece too
    assert lib.qlora_lm_loss_workspace_bytes(8, V, D, 1, 0) < 2 * V * D // 8
    # a block of tokens bounds it whatever the batch
    assert lib.qlora_lm_loss_workspace_bytes(1 << 20, V, D, 0, 1) == grad


def test_act8_refusals(lib):
    q, d = lib.qlora_act8_quantize, lib.qlora_act8_dequantize
    assert q(P, 1, None, None) == binding.NF4_ERR_ARG
    assert q(P, 9, _act8(), None) == binding.NF4_ERR_DTYPE
    assert q(P, 1, _act8(rows=-1), None) == binding.NF4_ERR_ARG
    assert q(P, 1, _act8(cols=0), None) == binding.NF4_ERR_ARG
    assert q(P, 1, _act8(rows=BIG, cols=BIG), None) == binding.NF4_ERR_SHAPE
    assert q(P, 1, _act8(codes=None), None) == binding.NF4_ERR_ARG
    assert q(P, 1, _act8(scales=ODD), None) == binding.NF4_ERR_ALIGN
    assert q(None, 1, _act8(), None) == binding.NF4_ERR_ARG
    assert q(ODD, 1, _act8(), None) == binding.NF4_ERR_ALIGN
    assert q(None, 1, _act8(rows=0, codes=None, scales=None), None) == binding.NF4_OK
    assert d(None, None, P, 1, None) == binding.NF4_ERR_ARG
    assert d(_act8(), None, P, 3, None) == binding.NF4_ERR_DTYPE
    assert d(_act8(), ODD, P, 1, None) == binding.NF4_ERR_ALIGN
    assert d(_act8(), None, None, 1, None) == binding.NF4_ERR_ARG
    assert d(_act8(rows=0), None, None, 1, None) == binding.NF4_OK


def test_grad_a_refusals(lib):
    def g(rank=8, alpha=1.0, mode=0, G=P, c=None, w=None, dA=P, ws=P, n=1 << 30):
        return lib.qlora_act8_grad_a(rank, alpha, mode, G, _act8() if c is None else c, w, dA, ws, n, None)
    assert g(rank=0) == binding.NF4_ERR_ARG and g(rank=257) == binding.NF4_ERR_ARG
    assert g(alpha=float("nan")) == binding.NF4_ERR_ARG and g(mode=2) == binding.NF4_ERR_ARG
    assert g(G=None) == binding.NF4_ERR_ARG and g(dA=None) == binding.NF4_ERR_ARG
    assert g(G=ODD) == binding.NF4_ERR_ALIGN and g(w=ODD) == binding.NF4_ERR_ALIGN and g(ws=ODD) == binding.NF4_ERR_ALIGN
    assert lib.qlora_act8_grad_a(8, 1.0, 0, P, None, None, P, P, 1 << 30, None) == binding.NF4_ERR_ARG


def test_linear_backward_refusals(lib):
    def f(M=4, N=64, K=256, r=8, cd=1, dy=P, c=None, xw=None, T=P, W=None, w16=P, dx=P, ws=P, n=1 << 40):
        return lib.qlora_linear_bwd_act8(M, N, K, r, 16.0, 0, cd, dy, _act8() if c is None else c, xw, T, W, w16, P, P, dx,
                                         P, P, ws, n, None)
    assert f(r=0) == binding.NF4_ERR_ARG and f(cd=9) == binding.NF4_ERR_DTYPE
    assert f(cd=binding.NF4_F32) == binding.NF4_ERR_DTYPE                   # a decoded weight is 16-bit
    assert f(c=_act8(rows=5)) == binding.NF4_ERR_SHAPE and f(c=_act8(cols=128)) == binding.NF4_ERR_SHAPE
    assert f(N=60) == binding.NF4_ERR_SHAPE                                 # N % 8
    assert f(w16=None) == binding.NF4_ERR_ARG                               # neither weight
    assert f(w16=None, W=_nf4(63 * 256)) == binding.NF4_ERR_CORRUPT
    assert f(dy=None) == binding.NF4_ERR_ARG and f(c=_act8(codes=None)) == binding.NF4_ERR_ARG
    assert f(xw=ODD) == binding.NF4_ERR_ALIGN and f(dx=ODD) == binding.NF4_ERR_ALIGN
    assert f(n=8) == binding.NF4_ERR_WORKSPACE and f(ws=None) == binding.NF4_ERR_WORKSPACE


def test_norm_refusals(lib):
    def f(M=4, K=256, eps=1e-5, dt=1, x=P, res=None, w=P, y=P, h=None, rstd=P, c=None):
        return lib.qlora_rms_norm_fwd(M, K, eps, dt, x, res, w, y, h, rstd, c, None)
    assert f(M=-1) == binding.NF4_ERR_ARG and f(K=0) == binding.NF4_ERR_ARG and f(M=BIG, K=BIG) == binding.NF4_ERR_SHAPE
    assert f(dt=3) == binding.NF4_ERR_DTYPE
    assert f(eps=-1.0) == binding.NF4_ERR_ARG and f(eps=float("inf")) == binding.NF4_ERR_ARG
    assert f(x=None) == binding.NF4_ERR_ARG and f(w=None) == binding.NF4_ERR_ARG and f(rstd=None) == binding.NF4_ERR_ARG
    assert f(res=ODD) == binding.NF4_ERR_ALIGN and f(h=ODD) == binding.NF4_ERR_ALIGN
    assert f(c=_act8(rows=3)) == binding.NF4_ERR_SHAPE
    assert f(M=0, x=None, y=None, rstd=None) == binding.NF4_OK

    def g(M=4, K=256, dt=1, dy=P, h=P, c=None, rstd=P, w=P, dres=None, dx=P, dw=None, ws=None, n=0):
        return lib.qlora_rms_norm_bwd(M, K, dt, dy, h, c, rstd, w, dres, dx, dw, ws, n, None)
    assert g(dt=5) == binding.NF4_ERR_DTYPE
    assert g(c=_act8()) == binding.NF4_ERR_ARG                              # both h and a checkpoint
    assert g(h=None) == binding.NF4_ERR_ARG                                 # neither
    assert g(h=None, c=_act8(cols=255)) == binding.NF4_ERR_SHAPE
    assert g(dy=None) == binding.NF4_ERR_ARG and g(dx=ODD) == binding.NF4_ERR_ALIGN
    assert g(dw=P) == binding.NF4_ERR_WORKSPACE
    assert g(dw=P, ws=ODD, n=1 << 40) == binding.NF4_ERR_ALIGN


def test_loss_refusals(lib):
    def f(M=4, V=100, D=128, cd=1, x=P, W=None, w16=P, t=P, gs=None, loss=P, lse=None, dx=P, ws=P, n=1 << 40):
        return lib.qlora_lm_loss(M, V, D, cd, x, W, w16, t, -100, gs, 0, loss, lse, dx, ws, n, None)
    assert f(M=-1) == binding.NF4_ERR_ARG and f(V=0) == binding.NF4_ERR_ARG and f(D=0) == binding.NF4_ERR_ARG
    assert f(cd=binding.NF4_F32) == binding.NF4_ERR_DTYPE
    assert f(D=56) == binding.NF4_ERR_SHAPE and f(D=132) == binding.NF4_ERR_SHAPE
    assert f(V=1 << 31) == binding.NF4_ERR_SHAPE
    assert f(w16=None) == binding.NF4_ERR_ARG
    assert f(w16=None, W=_nf4(99 * 128)) == binding.NF4_ERR_CORRUPT
    assert f(w16=None, W=_nf4(100 * 72), D=72) == binding.NF4_ERR_SHAPE     # a stored head needs D % 64
    assert f(x=None) == binding.NF4_ERR_ARG and f(t=None) == binding.NF4_ERR_ARG and f(loss=None) == binding.NF4_ERR_ARG
    assert f(gs=ODD) == binding.NF4_ERR_ALIGN and f(lse=ODD) == binding.NF4_ERR_ALIGN and f(dx=ODD) == binding.NF4_ERR_ALIGN
    assert f(ws=None) == binding.NF4_ERR_WORKSPACE and f(n=64) == binding.NF4_ERR_WORKSPACE
    assert f(ws=ODD) == binding.NF4_ERR_ALIGN
    assert f(M=0, x=None, t=None, loss=None, dx=None, ws=None, n=0) == binding.NF4_OK
