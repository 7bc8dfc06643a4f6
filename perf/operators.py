"""The operators around the frozen-base linear in a training step, as measured cases.

What a step runs between and after its QLoRA linears:

  norm_fwd  h = x + residual, n = h / rms(h), y = n * weight; optionally n kept in 8 bits, the
            checkpoint that the backward pass of the norm and of the linears behind it reads
  norm_bwd  dx (the residual branch's gradient added) and dweight, from h or from the checkpoint
  act8      an activation stored as int8 codes with one float32 scale for each token and block of
            128 features, and read back
  grad_a    dA = s G^T x of a LoRA adapter, x being an 8-bit checkpoint (optionally times the
            norm's weight)
  loss      softmax cross entropy of x W^T against target tokens, and its gradient dx, over the
            whole vocabulary (W, the head, is frozen); tokens with target -100 do not count

`run` computes each in plain torch operations in 32 bits, or with the library's entry points
where `own` is set.  `exact` computes them from the definitions in 64 bits.
"""

import math

import torch

own = False

BLOCK = 128        # features that share a scale of an 8-bit checkpoint
TINY = 2.0 ** -116  # a block whose largest magnitude is below this is stored as zeros
EPS = 1e-5
ALPHA = 32.0       # LoRA alpha: s = alpha / rank
IGNORE = -100

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def listed():
    return [
        # the norm in front of a projection while one token is decoded: latency alone
        dict(name="norm_fwd_1x4096", op="norm_fwd", dtype="bf16", M=1, K=4096, residual=True, checkpoint=False),
        # a Llama-3-8B-shaped layer's norm in training (2 x 2048 tokens), keeping the checkpoint
        dict(name="norm_fwd_4096x4096_ckpt", op="norm_fwd", dtype="bf16", M=4096, K=4096, residual=True,
             checkpoint=True),
        # its backward pass from the residual stream, with a frozen weight
        dict(name="norm_bwd_4096x4096", op="norm_bwd", dtype="bf16", M=4096, K=4096, residual=True,
             checkpoint=False, dweight=False),
        # the backward pass from the checkpoint with a trained weight, at odd sizes
        dict(name="norm_bwd_777x1531_ckpt", op="norm_bwd", dtype="f16", M=777, K=1531, residual=True,
             checkpoint=True, dweight=True),
        # the MLP activation (down's input) of the same layer, stored and read back
        dict(name="act8_4096x14336", op="act8", dtype="bf16", M=4096, K=14336),
        # a short ragged prompt in the float32 profile
        dict(name="act8_33x577_f32", op="act8", dtype="f32", M=33, K=577),
        # a SmolLM2-135M-shaped q or v adapter (512 tokens) behind a norm's checkpoint
        dict(name="grad_a_512x576", op="grad_a", M=512, K=576, r=16, weight=True),
        # down's adapter in the Llama-3-8B-shaped layer
        dict(name="grad_a_4096x14336", op="grad_a", M=4096, K=14336, r=16, weight=False),
        # scoring one token with the Llama-3-8B-shaped head: no gradient
        dict(name="loss_1x128256x4096_score", op="loss", dtype="bf16", M=1, V=128256, D=4096, grad=False),
        # one step's loss with the SmolLM2-135M-shaped head
        dict(name="loss_512x49152x576", op="loss", dtype="bf16", M=512, V=49152, D=576, grad=True),
        # a ragged batch over a vocabulary and a width that no tile divides
        dict(name="loss_1021x50257x1000_f16", op="loss", dtype="f16", M=1021, V=50257, D=1000, grad=True),
        # one step's loss with the Llama-3-8B-shaped head (2 x 2048 tokens)
        dict(name="loss_4096x128256x4096", op="loss", dtype="bf16", M=4096, V=128256, D=4096, grad=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "act8", "grad_a", "loss", "loss"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "loss":
        V, D, grad = _log(rng, 300, 128256), 8 * _log(rng, 8, 512), rng.random() < 0.75
        most = max(1, min(4096, (4096 * 128256 * 4096) // (V * D)))
        return dict(op=op, dtype=dtype, M=_log(rng, 1, most), V=V, D=D, grad=grad)
    M, K = _log(rng, 1, 8192), _log(rng, 48, 14336)
    if rng.random() < 0.5:
        K = (K + 63) // 64 * 64
    if op == "grad_a":
        return dict(op=op, M=M, K=K, r=rng.choice([1, 4, 8, 16, 16, 32, 64]), weight=rng.random() < 0.5)
    dtype = rng.choice([dtype, dtype, dtype, "f32"])
    if op == "act8":
        return dict(op=op, dtype=dtype, M=M, K=K)
    case = dict(op=op, dtype=dtype, M=M, K=K, residual=rng.random() < 0.75, checkpoint=rng.random() < 0.5)
    if op == "norm_bwd":
        case["dweight"] = rng.random() < 0.5
    return case


def work(case):
    if case["op"] == "loss":
        M, V, D = case["M"], case["V"], case["D"]
        # x, W, targets once; loss and lse out; dx out.  Products: logits, and dx where asked
        moved = 2 * (M * D + V * D) + 8 * M + 8 * M + (2 * M * D if case["grad"] else 0)
        return {"bytes": moved, "flops": (4 if case["grad"] else 2) * M * V * D}
    M, K = case["M"], case["K"]
    ckpt = M * K + 4 * M * -(-K // BLOCK)          # codes and scales
    if case["op"] == "grad_a":
        r = case["r"]
        return {"bytes": ckpt + 4 * M * r + 4 * r * K + (4 * K if case["weight"] else 0), "flops": 2 * M * K * r}
    b = BYTES[case["dtype"]]
    if case["op"] == "act8":                       # the activation in, the codes out and in, the values out
        return {"bytes": 2 * b * M * K + 2 * ckpt, "flops": 4 * M * K}
    if case["op"] == "norm_fwd":
        streams = 4 if case["residual"] else 2     # x, residual in; h, y out
        return {"bytes": (streams * b) * M * K + 4 * K + 4 * M + ((2 * ckpt + b * M * K) if case["checkpoint"] else 0),
                "flops": 6 * M * K}
    saved = ckpt if case["checkpoint"] else b * M * K
    streams = 3 if case["residual"] else 2         # dy, the residual branch's gradient in; dx out
    return {"bytes": streams * b * M * K + saved + 4 * K + 4 * M + (4 * K if case["dweight"] else 0),
            "flops": 8 * M * K}


# ---- inputs -----------------------------------------------------------------------------

def _activations(gen, M, K):
    """Residual-stream-like values: channels of different gain, one in 64 of them large."""
    gain = torch.exp(0.4 * torch.randn(K, generator=gen, device="cuda"))
    gain = torch.where(torch.rand(K, generator=gen, device="cuda") < 1 / 64, gain * 6, gain)
    return torch.randn(M, K, generator=gen, device="cuda") * gain


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    M, op = case["M"], case["op"]
    s = dict(case=case)
    if op == "loss":
        V, D, dt = case["V"], case["D"], DTYPES[case["dtype"]]
        s["W"] = (torch.randn(V, D, generator=gen, device="cuda") * 0.02).to(dt)
        t = torch.randint(0, V, (M,), generator=gen, device="cuda")
        # hidden states lean towards their target by a random amount: from a guess to a sure token
        lean = torch.rand(M, 1, generator=gen, device="cuda") * 12
        w = s["W"][t].float()
        s["x"] = (torch.randn(M, D, generator=gen, device="cuda") + lean * w / w.norm(dim=1, keepdim=True)).to(dt)
        if M > 1:                                  # prompt tokens do not count
            t = torch.where(torch.rand(M, generator=gen, device="cuda") < 0.2, torch.full_like(t, IGNORE), t)
        s["targets"] = t
        s["grad_scale"] = 1 / (t != IGNORE).sum().clamp(min=1).float().reshape(1)
        return s
    K = case["K"]
    x = _activations(gen, M, K)
    weight = 1 + 0.1 * torch.randn(K, generator=gen, device="cuda")
    if op == "grad_a":
        s["codes"], s["scales"] = _store(x)
        s["G"] = torch.randn(M, case["r"], generator=gen, device="cuda") * 1e-3
        s["weight"] = weight if case["weight"] else None
        return s
    dt = DTYPES[case["dtype"]]
    if op == "act8":
        s["x"] = x.to(dt)
        return s
    s["weight"] = weight
    if op == "norm_fwd":
        s["x"] = x.to(dt)
        s["residual"] = _activations(gen, M, K).to(dt) if case["residual"] else None
        return s
    h = x.to(dt)
    s["rstd"] = torch.rsqrt(h.float().square().mean(1) + EPS)
    s["codes"], s["scales"] = _store(h.float() * s["rstd"][:, None]) if case["checkpoint"] else (None, None)
    s["h"] = None if case["checkpoint"] else h
    s["dy"] = (torch.randn(M, K, generator=gen, device="cuda") * 1e-2).to(dt)
    s["dres"] = (torch.randn(M, K, generator=gen, device="cuda") * 1e-2).to(dt) if case["residual"] else None
    return s


# ---- the plain forms ----------------------------------------------------------------------

def _store(x):
    """int8 codes [M, K] and scales [M, ceil(K / 128)] of x: scale = amax / 127 over a token's block,
    code = rint(x * (127 / amax)), ties to even."""
    M, K = x.shape
    nb = -(-K // BLOCK)
    v = torch.nn.functional.pad(x, (0, nb * BLOCK - K)).view(M, nb, BLOCK)
    amax = v.abs().amax(2)
    live = amax >= TINY
    inv = torch.where(live, 127.0 / amax, torch.zeros_like(amax))
    codes = torch.round(v * inv[:, :, None]).to(torch.int8).view(M, nb * BLOCK)[:, :K].contiguous()
    return codes, torch.where(live, amax / 127.0, torch.zeros_like(amax)).float()


def _values(codes, scales, dt):
    return codes.to(dt) * scales.to(dt).repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def _norm_fwd(s, f):
    h = s["x"].to(f) + s["residual"].to(f) if s["residual"] is not None else s["x"].to(f)
    rstd = 1 / torch.sqrt(h.square().mean(1) + EPS)
    n = h * rstd[:, None]
    out = dict(y=n * s["weight"].to(f), rstd=rstd)
    if s["residual"] is not None:
        out["h"] = h
    if s["case"]["checkpoint"]:
        out["n"] = _values(*_store(n), f)
    return out


def _norm_bwd(s, f):
    rstd = s["rstd"].to(f)[:, None]
    n = _values(s["codes"], s["scales"], f) if s["h"] is None else s["h"].to(f) * rstd
    dy = s["dy"].to(f)
    g = dy * s["weight"].to(f)
    dx = rstd * (g - n * (g * n).mean(1, keepdim=True))
    out = dict(dx=dx + s["dres"].to(f) if s["dres"] is not None else dx)
    if s["case"]["dweight"]:
        out["dweight"] = (dy * n).sum(0)
    return out


def _loss(s, f):
    x, W, t = s["x"].to(f), s["W"].to(f), s["targets"]
    live = t != IGNORE
    at = torch.where(live, t, torch.zeros_like(t))[:, None]
    z = x @ W.T
    top = z.amax(1, keepdim=True)
    zt = z.gather(1, at)[:, 0]
    z = z.sub_(top).exp_()
    total = z.sum(1, keepdim=True)
    lse = torch.log(total[:, 0]) + top[:, 0]
    zero = torch.zeros_like(lse)
    out = dict(loss=torch.where(live, lse - zt, zero), lse=torch.where(live, lse, zero))
    if s["case"]["grad"]:
        z = z.div_(total)
        z.scatter_add_(1, at, -torch.ones_like(total))
        z.mul_((live.to(f) * s["grad_scale"].to(f))[:, None])
        out["dx"] = z @ W
    return out


def _plain(s, f):
    case = s["case"]
    op = case["op"]
    if op == "norm_fwd":
        return _norm_fwd(s, f)
    if op == "norm_bwd":
        return _norm_bwd(s, f)
    if op == "act8":
        return dict(values=_values(*_store(s["x"].to(f)), f))
    if op == "grad_a":
        x = _values(s["codes"], s["scales"], f)
        dA = (ALPHA / case["r"]) * (s["G"].to(f).T @ x)
        return dict(dA=dA * s["weight"].to(f) if s["weight"] is not None else dA)
    return _loss(s, f)


def _read_back(dt):
    """The type a norm's checkpoint is read back in: a 16-bit one, as the linears behind it take it."""
    return torch.bfloat16 if dt == torch.float32 else dt


# ---- one pass -----------------------------------------------------------------------------

def run(s):
    case = s["case"]
    op = case["op"]
    dt = DTYPES[case.get("dtype", "f32")]
    if not own:
        out = _plain(s, torch.float32)
        kinds = {"n": _read_back(dt), **dict.fromkeys(("rstd", "dweight", "dA", "loss", "lse"), torch.float32)}
        return {k: v.to(kinds.get(k, dt)) for k, v in out.items()}
    from bit_nf4_quantized_gb300 import binding as b
    if op == "norm_fwd":
        y, h, rstd, ckpt = b.qlora_rms_norm_fwd(s["x"], s["weight"], EPS, residual=s["residual"],
                                                checkpoint=case["checkpoint"])
        out = dict(y=y, rstd=rstd)
        if case["residual"]:
            out["h"] = h
        if case["checkpoint"]:
            out["n"] = b.qlora_act8_dequantize(ckpt, _read_back(dt))
        return out
    if op == "norm_bwd":
        saved = b.Act8(s["codes"], s["scales"]) if s["h"] is None else s["h"]
        dx, dweight = b.qlora_rms_norm_bwd(s["dy"], saved, s["rstd"], s["weight"], dresidual=s["dres"],
                                           dweight=case["dweight"])
        return dict(dx=dx, dweight=dweight) if case["dweight"] else dict(dx=dx)
    if op == "act8":
        return dict(values=b.qlora_act8_dequantize(b.qlora_act8_quantize(s["x"]), dt))
    if op == "grad_a":
        return dict(dA=b.qlora_act8_grad_a(s["G"], b.Act8(s["codes"], s["scales"]), ALPHA, weight=s["weight"]))
    loss, lse, dx = b.qlora_lm_loss(s["x"], s["W"], s["targets"], grad_scale=s["grad_scale"], ignore_index=IGNORE,
                                    need_dx=case["grad"])
    return dict(loss=loss, lse=lse, dx=dx) if case["grad"] else dict(loss=loss, lse=lse)


# ---- 64 bits, from the definitions ----------------------------------------------------------

def _exact_values(x):
    """What the 8-bit codes of x stand for: each token's blocks of 128 on a grid of 255 steps."""
    parts = []
    for b in torch.split(x, BLOCK, dim=1):
        step = b.abs().max(dim=1, keepdim=True).values / 127
        parts.append(torch.where(step * 127 >= TINY, torch.round(b / step) * step, torch.zeros_like(b)))
    return torch.cat(parts, dim=1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and k not in ("targets", "codes")}
    if "codes" in s and s["codes"] is not None:
        stored = s["codes"].double()
        for j in range(d["scales"].shape[1]):
            stored[:, j * BLOCK:(j + 1) * BLOCK] *= d["scales"][:, j:j + 1]
    if op == "act8":
        return dict(values=_exact_values(d["x"]))
    if op == "grad_a":
        dA = torch.einsum("mr,mk->rk", d["G"], stored) * (ALPHA / case["r"])
        return dict(dA=dA if s["weight"] is None else dA * d["weight"])
    if op == "norm_fwd":
        h = d["x"] if s["residual"] is None else d["x"] + d["residual"]
        rms = torch.sqrt((h * h).sum(dim=1) / case["K"] + EPS)
        n = h / rms[:, None]
        out = dict(y=n * d["weight"], rstd=1 / rms)
        if s["residual"] is not None:
            out["h"] = h
        if case["checkpoint"]:
            out["n"] = _exact_values(n)
        return out
    if op == "norm_bwd":
        n = stored if case["checkpoint"] else d["h"] * d["rstd"][:, None]
        dn = d["dy"] * d["weight"]
        along = torch.einsum("mk,mk->m", dn, n) / case["K"]
        dx = (dn - along[:, None] * n) * d["rstd"][:, None]
        out = dict(dx=dx if s["dres"] is None else dx + d["dres"])
        if case["dweight"]:
            out["dweight"] = torch.einsum("mk,mk->k", d["dy"], n)
        return out
    t = s["targets"]
    logp = torch.log_softmax(torch.mm(d["x"], d["W"].t()), dim=1)
    counts = t >= 0
    rows = torch.arange(case["M"], device="cuda")
    safe = t.clamp(min=0)
    own_logp = logp[rows, safe]
    zt = (d["x"] * d["W"][safe]).sum(dim=1)
    out = dict(loss=-own_logp * counts, lse=(zt - own_logp) * counts)
    if case["grad"]:
        p = logp.exp_()
        p[rows, safe] -= 1
        p *= (counts * d["grad_scale"])[:, None]
        out["dx"] = torch.mm(p, d["W"])
    return out
