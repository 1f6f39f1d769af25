"""The training and serving operators around the linear layer: cases to time, and their plain forms.

Four kinds of case:

- ``gated``: the gated feed-forward block h = act(x Wg^T) * (x Wu^T), for serving (h alone)
  and for training (the two projections are kept as well);
- ``gated_backward``: its gradients dx, dWg, dWu from dh and the kept projections;
- ``linear_backward``: the linear layer's gradients dx, dW and db from dy;
- ``clip``: the global gradient norm over many tensors, and the gradients scaled by it.

``own`` chooses between elementary torch operations in 32 bits and the library's calls.
"""
import math

import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_MAX_NORM = 1.0


def listed():
    return [
        # one token through the feed-forward block of the 4096 / 14336 layers (decode)
        {"name": "gated_token", "kind": "gated", "M": 1, "N": 14336, "K": 4096, "type": "f16", "act": "silu", "keep": False},
        # one token through a small block: the call's latency
        {"name": "gated_token_small", "kind": "gated", "M": 1, "N": 1024, "K": 768, "type": "bf16", "act": "gelu_tanh", "keep": False},
        # a decode batch of 16
        {"name": "gated_batch16", "kind": "gated", "M": 16, "N": 14336, "K": 4096, "type": "bf16", "act": "silu", "keep": False},
        # prefill of 4096 tokens
        {"name": "gated_prefill", "kind": "gated", "M": 4096, "N": 14336, "K": 4096, "type": "f16", "act": "silu", "keep": False},
        # the forward half of a training step on a ragged batch: the projections are kept for the gradients
        {"name": "gated_train_ragged", "kind": "gated", "M": 2000, "N": 4000, "K": 4096, "type": "bf16", "act": "gelu_erf", "keep": True},
        # the backward half of a training step at the full width
        {"name": "gated_backward_full", "kind": "gated_backward", "M": 4096, "N": 14336, "K": 4096, "type": "bf16", "act": "silu"},
        # a short ragged batch through a small block
        {"name": "gated_backward_ragged", "kind": "gated_backward", "M": 517, "N": 2720, "K": 1024, "type": "f16", "act": "gelu_tanh"},
        # gradients of an attention projection over 8192 tokens, bias among them
        {"name": "linear_backward_attn", "kind": "linear_backward", "M": 8192, "N": 4096, "K": 4096, "type": "bf16", "bias": True, "wide": False},
        # gradients of a ragged down projection, the weight's kept in 32 bits
        {"name": "linear_backward_down", "kind": "linear_backward", "M": 2000, "N": 4000, "K": 14336, "type": "f16", "bias": False, "wide": True},
        # the toy layer's gradients: the call's latency
        {"name": "linear_backward_toy", "kind": "linear_backward", "M": 1024, "N": 1024, "K": 768, "type": "f16", "bias": True, "wide": False},
        # the gradients of four 4096 / 14336 layers: attention projections, feed-forward weights, vectors
        {"name": "clip_layers", "kind": "clip", "type": "bf16", "layers": 4, "width": 4096, "inner": 14336, "odd": 0},
        # a small model's 32-bit gradients, a few values past whole vectors: launches count
        {"name": "clip_small", "kind": "clip", "type": "f32", "layers": 7, "width": 257, "inner": 515, "odd": 1},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _dims(rng):
    """Widths of a layer: most are multiples of 8, as weights are stored; one in six is any number."""
    n, k = _spread(rng, 64, 14336), _spread(rng, 64, 4096)
    if rng.random() < 5 / 6:
        n, k = max(64, n // 8 * 8), max(64, k // 8 * 8)
    return n, k


def draw(rng):
    kind = rng.choice(["gated", "gated_backward", "linear_backward", "clip"])
    if kind == "clip":
        width, t = _spread(rng, 33, 4096), rng.choice(["f16", "bf16", "f32"])
        return {"kind": kind, "type": t, "layers": rng.randint(1, 2 if t == "f32" else 4), "width": width,
                "inner": rng.randint(2 * width, 7 * width // 2), "odd": rng.randint(0, 3)}
    n, k = _dims(rng)
    case = {"kind": kind, "M": _spread(rng, 1, 4096), "N": n, "K": k, "type": rng.choice(["f16", "bf16"])}
    if kind == "linear_backward":
        return {**case, "bias": rng.random() < 0.5, "wide": rng.random() < 0.5}
    case["act"] = rng.choice(["silu", "gelu_tanh", "gelu_erf"])
    return {**case, "keep": rng.random() < 0.5} if kind == "gated" else case


def _shapes(case):
    """The gradients' shapes of a stack of layers: four attention projections, three feed-forward weights, two vectors each."""
    w, i, odd = case["width"], case["inner"], case["odd"]
    return ([(w, w)] * 4 + [(i, w)] * 3 + [(w,), (w + odd,)]) * case["layers"]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = _TYPES[case["type"]]

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(t)

    def weight(n, k):
        return ((torch.rand(n, k, generator=gen, device="cuda") * 2 - 1) / math.sqrt(k)).to(t)

    if case["kind"] == "clip":
        grads = [normal(*s, scale=0.01) for s in _shapes(case)]
        return {"case": case, "grads": grads, "out": [torch.empty_like(g) for g in grads]}
    M, N, K = case["M"], case["N"], case["K"]
    state = {"case": case, "x": normal(M, K)}
    if case["kind"] == "linear_backward":
        state["w"] = weight(N, K)
        state["dy"] = normal(M, N, scale=0.1)
        return state
    state["wg"], state["wu"] = weight(N, K), weight(N, K)
    if case["kind"] == "gated_backward":
        state["dh"] = normal(M, N, scale=0.1)
        state["g"] = (state["x"].float() @ state["wg"].float().t()).to(t)
        state["u"] = (state["x"].float() @ state["wu"].float().t()).to(t)
    return state


# ---- the library's calls -------------------------------------------------------------

def _run_own(s):
    import linear_amd as la
    case = s["case"]
    if case["kind"] == "clip":
        norm = la.linear_grad_norm(s["grads"])
        return {"norm": norm, "grads": la.linear_grad_clip(s["grads"], norm, _MAX_NORM, out=s["out"])}
    f16 = case["type"] == "f16"
    if case["kind"] == "linear_backward":
        dx = (la.linear_f16_backward_input if f16 else la.linear_bf16_backward_input)(s["dy"], s["w"])
        if case["wide"]:
            weight = la.linear_f16_backward_weight_f32out if f16 else la.linear_bf16_backward_weight_f32out
        else:
            weight = la.linear_f16_backward_weight if f16 else la.linear_bf16_backward_weight
        dw, db = weight(s["dy"], s["x"], bias=case["bias"])
        return {"dx": dx, "dw": dw, "db": db} if case["bias"] else {"dx": dx, "dw": dw}
    act = {"silu": la.EPI_SILU, "gelu_tanh": la.EPI_GELU_TANH, "gelu_erf": la.EPI_GELU_ERF}[case["act"]]
    if case["kind"] == "gated":
        gated = la.linear_f16_gated if f16 else la.linear_bf16_gated
        if not case["keep"]:
            return {"h": gated(s["x"], s["wg"], s["wu"], act)}
        h, g, u = gated(s["x"], s["wg"], s["wu"], act, keep=True)
        return {"h": h, "g": g, "u": u}
    backward = la.linear_f16_gated_backward if f16 else la.linear_bf16_gated_backward
    dx, dwg, dwu = backward(s["dh"], s["x"], s["wg"], s["wu"], s["g"], s["u"], act)
    return {"dx": dx, "dwg": dwg, "dwu": dwu}


# ---- the plain forms -----------------------------------------------------------------

_GELU_A = 2 * math.sqrt(2 / math.pi)
_GELU_B = 0.044715


def _act(name, g):
    """The activation, and its derivative."""
    if name == "gelu_erf":
        p = 0.5 * torch.erfc(g * -math.sqrt(0.5))
        return g * p, p + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    if name == "gelu_tanh":
        s = 1 / (1 + torch.exp(-_GELU_A * (g + _GELU_B * g * g * g)))
        return g * s, s + g * s * (1 - s) * _GELU_A * (1 + 3 * _GELU_B * g * g)
    s = 1 / (1 + torch.exp(-g))
    return g * s, s + g * s * (1 - s)


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    t = _TYPES[case["type"]]
    if case["kind"] == "clip":
        squares = torch.stack([g.double().square().sum() for g in state["grads"]])
        norm = squares.sum().sqrt().float().reshape(1)
        scale = torch.clamp(_MAX_NORM / (norm + 1e-6), max=1.0)
        return {"norm": norm, "grads": [(g.float() * scale).to(t) for g in state["grads"]]}
    x = state["x"].float()
    if case["kind"] == "linear_backward":
        dy = state["dy"].float()
        wide = torch.float32 if case["wide"] else t
        out = {"dx": (dy @ state["w"].float()).to(t), "dw": (dy.t() @ x).to(wide)}
        if case["bias"]:
            out["db"] = dy.sum(0).to(wide)
        return out
    wg, wu = state["wg"].float(), state["wu"].float()
    if case["kind"] == "gated":
        g, u = x @ wg.t(), x @ wu.t()
        h = (_act(case["act"], g)[0] * u).to(t)
        return {"h": h, "g": g.to(t), "u": u.to(t)} if case["keep"] else {"h": h}
    dh, g, u = state["dh"].float(), state["g"].float(), state["u"].float()
    a, d = _act(case["act"], g)
    dg, du = dh * u * d, dh * a
    return {"dx": (dg @ wg + du @ wu).to(t), "dwg": (dg.t() @ x).to(t), "dwu": (du.t() @ x).to(t)}


# ---- the work, and the values in 64 bits ---------------------------------------------

def work(case):
    b = 4 if case["type"] == "f32" else 2
    if case["kind"] == "clip":
        n = sum(math.prod(s) for s in _shapes(case))
        # read for the norm, read again to be scaled once the norm is known, written
        return {"bytes": 3 * n * b + 4, "flops": 3 * n}
    M, N, K = case["M"], case["N"], case["K"]
    if case["kind"] == "gated":
        return {"bytes": b * (M * K + 2 * N * K + (3 if case["keep"] else 1) * M * N), "flops": 4 * M * N * K + 8 * M * N}
    if case["kind"] == "gated_backward":
        return {"bytes": b * (3 * M * N + 2 * M * K + 4 * N * K), "flops": 8 * M * N * K + 16 * M * N}
    wide = 4 if case["wide"] else 2
    return {"bytes": b * (M * N + 2 * M * K + N * K) + wide * (N * K + (N if case["bias"] else 0)),
            "flops": 4 * M * N * K + (M * N if case["bias"] else 0)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "clip":
        total = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g, dtype=torch.float64)) ** 2 for g in s["grads"]))
        scale = min(1.0, _MAX_NORM / (total + 1e-6))
        return {"norm": torch.tensor([total], dtype=torch.float64), "grads": [g.double() * scale for g in s["grads"]]}
    x = s["x"].double()
    if case["kind"] == "linear_backward":
        dy = s["dy"].double()
        out = {"dx": torch.matmul(dy, s["w"].double()), "dw": torch.matmul(dy.t(), x)}
        if case["bias"]:
            out["db"] = torch.matmul(torch.ones(1, dy.shape[0], dtype=torch.float64, device=dy.device), dy)[0]
        return out
    act = {"silu": torch.nn.functional.silu, "gelu_erf": torch.nn.functional.gelu,
           "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[case["act"]]
    wg, wu = s["wg"].double(), s["wu"].double()
    if case["kind"] == "gated":
        g, u = torch.matmul(x, wg.t()), torch.matmul(x, wu.t())
        h = act(g) * u
        return {"h": h, "g": g, "u": u} if case["keep"] else {"h": h}
    with torch.enable_grad():
        g, u = s["g"].double().requires_grad_(), s["u"].double().requires_grad_()
        dg, du = torch.autograd.grad(act(g) * u, (g, u), s["dh"].double())
    return {"dx": torch.matmul(dg, wg) + torch.matmul(du, wu), "dwg": torch.matmul(dg.t(), x), "dwu": torch.matmul(du.t(), x)}
