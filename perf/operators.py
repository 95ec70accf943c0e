"""The feed-forward operators on group-quantised INT4 weights: their measured cases and plain forms.

A quantised linear layer holds packed [N, K/8] int32 (8 four-bit codes per word, the lowest k in the
lowest nibble), scales [N, K/128] fp16 and zeros [N, K/128] uint8; its weight is
W[n, k] = (q[n, k] - zeros[n, k/128]) * scales[n, k/128].  Activations and gradients are fp16.

    fused         Y = act(X W^T + bias) + residual, optionally with Z = X W^T + bias for the backward pass
    gated         H = act(X Wg^T) * (X Wu^T), optionally with G = X Wg^T and U = X Wu^T
    dx            dX = dY W (+ dY2 W2): the gradient of one or two layers' common input
    dx_gated      dH = dY W; dG = dH * U * act'(G), dU = dH * act(G): the down projection's input
                  gradient carried through the gate
    act_backward  dZ = dY * act'(Z), dbias = column sums of dZ; with a second factor U:
                  dG = dH * U * act'(G), dU = dH * act(G)
"""
import math

import torch

own = False

_ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
_GROUP = 128


def listed():
    return [
        # token-by-token decode of a 7B-class block: the down projection with the residual stream added
        dict(name="fused_decode_down", op="fused", M=1, N=4096, K=11008, act="none", bias=False, residual=True, pre=False),
        # 32 requests decoded together through a 70B-class down projection
        dict(name="fused_batch32_down", op="fused", M=32, N=8192, K=28672, act="none", bias=False, residual=True, pre=False),
        # a training step's biased GELU layer, an odd number of tokens, pre-activations kept
        dict(name="fused_train_gelu", op="fused", M=1999, N=11008, K=4096, act="gelu", bias=True, residual=False, pre=True),
        # token-by-token decode: both projections of the gate
        dict(name="gated_decode", op="gated", M=1, N=11008, K=4096, act="silu", pre=False),
        # a training step's forward pass, gate and up kept for the backward pass
        dict(name="gated_train", op="gated", M=2048, N=11008, K=4096, act="silu", pre=True),
        # prefill of 4096 tokens through a 70B-class block
        dict(name="gated_prefill", op="gated", M=4096, N=28672, K=8192, act="silu", pre=False),
        # the gated block's input gradient: both projections' products added
        dict(name="dx_train_pair", op="dx", M=2048, N=11008, K=4096, pair=True),
        # a short ragged batch through one narrow layer
        dict(name="dx_ragged", op="dx", M=333, N=1000, K=1152, pair=False),
        # the down projection's input gradient carried through the gate
        dict(name="dx_gated_train", op="dx_gated", M=2048, N=4096, K=11008, act="silu"),
        # the same for a few tokens of a small block
        dict(name="dx_gated_small", op="dx_gated", M=24, N=520, K=384, act="gelu_tanh"),
        # the gate's backward pass alone (the gradient of H came from another layer)
        dict(name="act_backward_gated", op="act_backward", M=2048, N=11008, act="silu", gated=True, dbias=False),
        # a biased GELU layer's activation and bias gradient, ragged
        dict(name="act_backward_bias", op="act_backward", M=1999, N=11000, act="gelu", gated=False, dbias=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("fused", "gated", "dx", "dx_gated", "act_backward"))
    while True:
        M = _log_uniform(rng, 1, 4096)
        N = 8 * _log_uniform(rng, 1, 3584)
        K = 128 * _log_uniform(rng, 1, 224)
        if N * K <= 28672 * 8192:
            break
    case = dict(op=op, M=M, N=N, K=K)
    if op == "fused":
        case.update(act=rng.choice(_ACTS), bias=rng.random() < 0.5, residual=rng.random() < 0.5, pre=rng.random() < 0.3)
    elif op == "gated":
        case.update(act=rng.choice(_ACTS), pre=rng.random() < 0.5)
    elif op == "dx":
        case.update(pair=rng.random() < 0.5)
    elif op == "dx_gated":
        case.update(act=rng.choice(_ACTS))
    else:
        del case["K"]
        gated = rng.random() < 0.5
        case.update(act=rng.choice(_ACTS[1:]), gated=gated, dbias=not gated and rng.random() < 0.5)
    return case


def _quantised_layer(gen, N, K):
    """Round-to-nearest INT4 codes of an N(0, 0.02) weight matrix, one fp16 scale and one zero point
    per group of 128."""
    W = torch.randn(N, K // _GROUP, _GROUP, device="cuda", dtype=torch.float16, generator=gen) * 0.02
    lo = W.amin(2).float().clamp(max=0.0)
    hi = W.amax(2).float().clamp(min=0.0)
    scales = ((hi - lo) / 15.0).half()
    scales = torch.where(scales > 0, scales, torch.ones_like(scales))
    zeros = (-lo / scales.float()).round().clamp(0, 15)
    codes = (W / scales[..., None]).round_().add_(zeros[..., None]).clamp_(0, 15).to(torch.uint8)
    codes = codes.view(N, K // 2, 2)
    packed = (codes[..., 0] | (codes[..., 1] << 4)).contiguous().view(torch.int32)
    return packed.view(N, K // 8), scales, zeros.to(torch.uint8)


def _activations(gen, M, K):
    """N(0, 1) with 1 % of the channels twenty times larger."""
    X = torch.randn(M, K, device="cuda", generator=gen)
    loud = torch.randperm(K, device="cuda", generator=gen)[: max(1, K // 100)]
    X[:, loud] *= 20.0
    return X.half()


def _normal(gen, M, N, std):
    return (torch.randn(M, N, device="cuda", generator=gen) * std).half()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    M, N, K, op = case["M"], case["N"], case.get("K"), case["op"]
    s = dict(op=op, act=case.get("act", "none"))
    if op != "act_backward":
        s["W"] = _quantised_layer(gen, N, K)
    if op == "fused":
        s["X"] = _activations(gen, M, K)
        s["bias"] = _normal(gen, 1, N, 0.5)[0].contiguous() if case["bias"] else None
        s["residual"] = _normal(gen, M, N, 2.0) if case["residual"] else None
        s["pre"] = case["pre"]
    elif op == "gated":
        s["X"] = _activations(gen, M, K)
        s["W2"] = _quantised_layer(gen, N, K)
        s["pre"] = case["pre"]
    elif op == "dx":
        s["dY"] = _normal(gen, M, N, 0.05)
        s["W2"] = _quantised_layer(gen, N, K) if case["pair"] else None
        s["dY2"] = _normal(gen, M, N, 0.05) if case["pair"] else None
    elif op == "dx_gated":
        s["dY"] = _normal(gen, M, N, 0.05)
        s["G"] = _normal(gen, M, K, 1.5)
        s["U"] = _normal(gen, M, K, 1.5)
    else:
        s["dY"] = _normal(gen, M, N, 0.05)
        s["Z"] = _normal(gen, M, N, 1.5)
        s["U"] = _normal(gen, M, N, 1.5) if case["gated"] else None
        s["dbias"] = case["dbias"]
    return s


# ------------------------------------------------------------------------------------ plain forms
def _weight(W):
    """[N, K] fp32, exactly (q - z) * s (15 significant bits)."""
    packed, scales, zeros = W
    N, G = scales.shape
    shifts = torch.arange(0, 32, 4, device=packed.device, dtype=torch.int32)
    q = ((packed[..., None] >> shifts) & 15).view(N, G, _GROUP)
    w = (q.float() - zeros.float()[..., None]) * scales.float()[..., None]
    return w.view(N, G * _GROUP)


def _act(x, act):
    if act == "relu":
        return torch.where(x < 0, torch.zeros_like(x), x)
    if act == "gelu":
        return 0.5 * x * torch.erfc(x * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return x / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    return x


def _act_grad(x, act):
    if act == "relu":
        return (x > 0).to(x.dtype)
    if act == "gelu":
        return 0.5 * torch.erfc(x * -math.sqrt(0.5)) + x * torch.exp(-0.5 * x * x) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        c = 2.0 * math.sqrt(2.0 / math.pi)
        t = 1.0 / (1.0 + torch.exp(-c * (x + 0.044715 * x * x * x)))
        return t + x * t * (1.0 - t) * c * (1.0 + 3.0 * 0.044715 * x * x)
    if act == "silu":
        t = 1.0 / (1.0 + torch.exp(-x))
        return t * (1.0 + x * (1.0 - t))
    return torch.ones_like(x)


def _plain(s):
    op, act = s["op"], s["act"]
    if op == "fused":
        z = s["X"].float() @ _weight(s["W"]).t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _act(z, act)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return (y.half(), z.half()) if s["pre"] else (y.half(),)
    if op == "gated":
        x = s["X"].float()
        g, u = x @ _weight(s["W"]).t(), x @ _weight(s["W2"]).t()
        h = (_act(g, act) * u).half()
        return (h, g.half(), u.half()) if s["pre"] else (h,)
    if op == "dx":
        dx = s["dY"].float() @ _weight(s["W"])
        if s["W2"] is not None:
            dx = dx + s["dY2"].float() @ _weight(s["W2"])
        return (dx.half(),)
    if op == "dx_gated":
        dh = s["dY"].float() @ _weight(s["W"])
        g, u = s["G"].float(), s["U"].float()
        return (dh * u * _act_grad(g, act)).half(), (dh * _act(g, act)).half()
    dy, z = s["dY"].float(), s["Z"].float()
    if s["U"] is not None:
        return (dy * s["U"].float() * _act_grad(z, act)).half(), (dy * _act(z, act)).half()
    dz = dy * _act_grad(z, act)
    return (dz.half(), dz.double().sum(0).float()) if s["dbias"] else (dz.half(),)


def _own(s):
    from weight_only_int4_06_b200 import w4a16 as W4

    op, act = s["op"], W4.ACTIVATIONS[s["act"]]
    if op == "fused":
        out = W4.w4_gemm_fused(s["X"], *s["W"], bias=s["bias"], activation=act, residual=s["residual"], save_pre=s["pre"])
        return out if s["pre"] else (out,)
    if op == "gated":
        out = W4.w4_gemm_gated(s["X"], s["W"], s["W2"], activation=act, save_pre=s["pre"])
        return out if s["pre"] else (out,)
    if op == "dx":
        return (W4.w4_gemm_dx(s["dY"], *s["W"], dY2=s["dY2"], weights2=s["W2"]),)
    if op == "dx_gated":
        return W4.w4_gemm_dx_gated(s["dY"], *s["W"], s["G"], s["U"], activation=act)
    out = W4.w4_act_backward(s["dY"], s["Z"], U=s["U"], activation=act, bias_grad=s["dbias"])
    return out if isinstance(out, tuple) else (out,)


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ------------------------------------------------------------------------------------ 64-bit values
def _weight64(W):
    packed, scales, zeros = W
    N, G = scales.shape
    b = packed.view(torch.uint8).view(N, G, _GROUP // 2)
    w = torch.empty(N, G, _GROUP, dtype=torch.float64, device=b.device)
    w[..., 0::2] = (b & 15).double()
    w[..., 1::2] = (b >> 4).double()
    w -= zeros.double().unsqueeze(2)
    w *= scales.double().unsqueeze(2)
    return w.reshape(N, G * _GROUP)


def _act64(x, act):
    """(act(x), act'(x)) in 64 bits."""
    if act == "relu":
        return x.clamp(min=0.0), torch.heaviside(x, torch.zeros((), dtype=x.dtype, device=x.device))
    if act == "gelu":
        cdf = torch.special.ndtr(x)
        return x * cdf, cdf + x * torch.exp(-x.square() / 2.0) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (x + 0.044715 * x.pow(3)))
        return 0.5 * x * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * c * (1.0 + 0.134145 * x.square())
    if act == "silu":
        t = torch.sigmoid(x)
        return x * t, t + x * t * (1.0 - t)
    return x, torch.ones_like(x)


def exact(case, seed):
    s = prepare(case, seed)
    op, act = s["op"], s["act"]
    if op == "fused":
        z = torch.mm(s["X"].double(), _weight64(s["W"]).t())
        if s["bias"] is not None:
            z += s["bias"].double()
        y = _act64(z, act)[0]
        if s["residual"] is not None:
            y = y + s["residual"].double()
        return (y, z) if s["pre"] else (y,)
    if op == "gated":
        g = torch.mm(s["X"].double(), _weight64(s["W"]).t())
        u = torch.mm(s["X"].double(), _weight64(s["W2"]).t())
        h = _act64(g, act)[0].mul_(u)
        return (h, g, u) if s["pre"] else (h,)
    if op == "dx":
        dx = torch.mm(s["dY"].double(), _weight64(s["W"]))
        if s["W2"] is not None:
            dx += torch.mm(s["dY2"].double(), _weight64(s["W2"]))
        return (dx,)
    if op == "dx_gated":
        dh = torch.mm(s["dY"].double(), _weight64(s["W"]))
        a, da = _act64(s["G"].double(), act)
        return dh * s["U"].double() * da, dh * a
    a, da = _act64(s["Z"].double(), act)
    if s["U"] is not None:
        return s["dY"].double() * s["U"].double() * da, s["dY"].double() * a
    dz = s["dY"].double() * da
    return (dz, dz.sum(0)) if s["dbias"] else (dz,)


def work(case):
    """Bytes: each input read once, each output written once.  Operations: two per multiply-add of the
    products, and about ten per element of what follows them."""
    M, N, K, op = case["M"], case["N"], case.get("K", 0), case["op"]
    layer = N * K // 2 + 3 * N * (K // _GROUP)  # codes, scales and zero points
    product = 2.0 * M * N * K
    if op == "fused":
        planes = 1 + int(case["residual"]) + int(case["pre"])
        return {"bytes": 2 * M * K + layer + 2 * M * N * planes + (2 * N if case["bias"] else 0), "flops": product + 10.0 * M * N}
    if op == "gated":
        return {"bytes": 2 * M * K + 2 * layer + 2 * M * N * (3 if case["pre"] else 1), "flops": 2 * product + 10.0 * M * N}
    if op == "dx":
        n = 2 if case["pair"] else 1
        return {"bytes": n * (2 * M * N + layer) + 2 * M * K, "flops": n * product}
    if op == "dx_gated":
        return {"bytes": 2 * M * N + layer + 8 * M * K, "flops": product + 10.0 * M * K}
    return {"bytes": 2 * M * N * (5 if case["gated"] else 3) + (4 * N if case["dbias"] else 0), "flops": 10.0 * M * N}
