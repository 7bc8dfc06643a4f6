"""The training step of bit_nf4_quantized_gb300.example_step on a GPU: its loss and gradients
against the same model in float64 torch autograd on the decoded weights, and its training.

The step multiplies 16-bit operands and keeps its activations in 8 bits, so the comparison is in
norm: the linear's stated 2e-2 for each of the chained 16-bit products, and a checkpoint's error of
half a step, amax / 254 over values of about amax / 3, 0.6 % of its norm.  Over three blocks
forward and back that stays within 5e-2."""

import pytest
import torch

from bit_nf4_quantized_gb300 import binding as b
from bit_nf4_quantized_gb300 import example_step as ex

pytestmark = pytest.mark.gpu


def _float64(model, ids, targets):
    dec = lambda q: b.nf4_dequantize(q, torch.float32).double()  # noqa: E731
    table = dec(model.table)
    params = {n: p.double().requires_grad_() for n, p in model.parameters()}

    def linear(i, k, x):
        p = model.blocks[i][k]
        A, B = params[f"{i}.{k}.A"], params[f"{i}.{k}.B"]
        return x @ dec(p.W).T + p.alpha / A.shape[0] * (x @ A.T) @ B.T

    def norm(h, w):
        return h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-5) * w.double()

    h = table[ids]
    for i, blk in enumerate(model.blocks):
        y = norm(h, blk["norm"])
        h = h + linear(i, "down", torch.nn.functional.silu(linear(i, "gate", y)) * linear(i, "up", y))
    z = norm(h, model.last_norm) @ table.T
    loss = torch.nn.functional.cross_entropy(z, targets, ignore_index=-100)
    loss.backward()
    return loss.item(), {n: p.grad for n, p in params.items()}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_step_gradients(lib, dtype):
    torch.manual_seed(0)
    model = ex.Model(vocab=500, hidden=192, inner=320, blocks=3, dtype=dtype)
    for name, p in model.parameters():
        if name.endswith("B"):
            p.normal_(0, 0.02)
    model.blocks[1]["norm"].normal_(1, 0.2)
    ids = torch.randint(0, 500, (150,), device="cuda")
    targets = torch.randint(0, 500, (150,), device="cuda")
    targets[::5] = -100
    loss, grads = model.loss_and_gradients(ids, targets)
    want, wgrads = _float64(model, ids, targets)
    assert abs(loss.item() - want) <= 1e-2 * want
    for name, g in grads.items():
        rel = (g.double() - wgrads[name]).norm() / wgrads[name].norm()
        assert rel <= 5e-2, f"{name}: {rel:.3g}"
    assert b.device_status(clear=True) == b.NF4_OK


def test_training_lowers_the_loss(lib):
    model = ex.Model(blocks=2)
    ids = torch.arange(0, 200, device="cuda")
    targets = (ids * 7 + 3) % 1000
    opt = torch.optim.Adam([p for _, p in model.parameters()], lr=5e-3)
    losses = []
    for _ in range(30):
        loss, grads = model.loss_and_gradients(ids, targets)
        for name, p in model.parameters():
            p.grad = grads[name]
        opt.step()
        losses.append(loss.item())
    assert losses[-1] < 0.5 * losses[0]
