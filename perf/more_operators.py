"""The two ends of a training step, the loss and the update: cases to time, and their plain forms.

Three kinds of case:

- ``score``: the softmax cross entropy of a linear head, loss[m] = lse[m] - z[m, target[m]] with
  z = x W^T (+ b), and lse; a target outside [0, N) (-100 here) marks a row that does not count;
- ``train``: the same, then its gradients dx, dW (and db) from the rows' dloss, and dlse where
  lse itself is penalised (``z``: the penalty's weight);
- ``adamw``: an AdamW step over many tensors, clipped by the gradients' norm, with the two
  moments in 32 bits or in 8.

8-bit moments.  A state of n values is n codes, then one byte k + 127 for each block of 32 values,
which share the factor 2^k.  The first moment's codes are a sign and 4 bits of exponent, 3 of
mantissa (code 127: NaN), the second's 5 bits of exponent, 3 of mantissa (codes 248, 255:
infinity, NaN); exponent field 0 holds the subnormals, as in IEEE formats.  k is the smallest,
from -100 on, for which the block's largest finite value is under 464 * 2^k (first moment) or
63488 * 2^k (second): then none rounds past the last code.  Values are rounded to nearest even,
a second moment over zero to the first code at least.  Every value that a state stands for is
a bfloat16 number: that is how states are returned.

The tensors of an ``adamw`` case lie in arenas, one for the weights, one for the gradients and
so on, each starting at a multiple of 256 values; what a pass returns is the arenas.

``own`` chooses between elementary torch operations in 32 bits and the library's calls.
"""
import math

import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_MAX_NORM = 1.0
_LR, _BETA1, _BETA2, _EPS, _DECAY, _STEP = 1e-3, 0.9, 0.95, 1e-8, 0.1, 10


def listed():
    return [
        # the log probability of one token: decode, with the vocabulary-sized projection of the tests
        {"name": "score_token", "kind": "score", "M": 1, "N": 128259, "K": 4096, "type": "f16", "bias": False},
        # a few tokens through a small head: the call's latency
        {"name": "score_small", "kind": "score", "M": 16, "N": 8000, "K": 768, "type": "bf16", "bias": True},
        # perplexity of a prompt of 4096 tokens
        {"name": "score_prompt", "kind": "score", "M": 4096, "N": 128259, "K": 4096, "type": "bf16", "bias": False},
        # a training step's loss and gradients at the full vocabulary
        {"name": "train_full", "kind": "train", "M": 4096, "N": 128259, "K": 4096, "type": "bf16", "bias": False, "z": 0.0},
        # a ragged batch in binary16 (the loss scaled up, as that type's small gradients need), bias, penalised lse
        {"name": "train_ragged", "kind": "train", "M": 1999, "N": 32001, "K": 2048, "type": "f16", "bias": True, "z": 1e-3},
        # a few rows: fine tuning on short answers
        {"name": "train_few", "kind": "train", "M": 20, "N": 32000, "K": 4096, "type": "bf16", "bias": False, "z": 0.0},
        # the toy layer as a head: the calls' latency
        {"name": "train_toy", "kind": "train", "M": 1024, "N": 1024, "K": 768, "type": "bf16", "bias": True, "z": 0.0},
        # the weights of two 4096 / 14336 layers, 32-bit moments
        {"name": "adamw_layers", "kind": "adamw", "param": "bf16", "grad": "bf16", "copy": False, "bits": 32, "layers": 2, "width": 4096, "inner": 14336, "odd": 0},
        # the same with 8-bit moments: what a card's memory is short of
        {"name": "adamw_layers_8", "kind": "adamw", "param": "bf16", "grad": "bf16", "copy": False, "bits": 8, "layers": 2, "width": 4096, "inner": 14336, "odd": 0},
        # 32-bit weights with the 16-bit copy that the next forward pass reads, widths that fill no vector
        {"name": "adamw_copy", "kind": "adamw", "param": "f32", "grad": "f16", "copy": True, "bits": 32, "layers": 2, "width": 1023, "inner": 3581, "odd": 2},
        # a small model in 32 bits, many tensors: launches count
        {"name": "adamw_small", "kind": "adamw", "param": "f32", "grad": "f32", "copy": False, "bits": 32, "layers": 7, "width": 257, "inner": 515, "odd": 1},
        # the same with 8-bit moments
        {"name": "adamw_small_8", "kind": "adamw", "param": "f32", "grad": "f32", "copy": False, "bits": 8, "layers": 7, "width": 257, "inner": 515, "odd": 1},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["score", "train", "train", "adamw"])
    if kind == "adamw":
        width, param = _spread(rng, 33, 4096), rng.choice(["f16", "bf16", "f32"])
        return {"kind": kind, "param": param, "grad": rng.choice(["f16", "bf16", "f32"]),
                "copy": param == "f32" and rng.random() < 0.5, "bits": rng.choice([8, 32]),
                "layers": 1 if width > 2048 else rng.randint(1, 4), "width": width,
                "inner": rng.randint(2 * width, 7 * width // 2), "odd": rng.randint(0, 3)}
    # most heads have rows of whole vectors, as weights are stored; one in six has any length.  A vocabulary has any size
    k = _spread(rng, 64, 4096)
    case = {"kind": kind, "M": _spread(rng, 1, 4096), "N": _spread(rng, 512, 128259),
            "K": max(64, k // 8 * 8) if rng.random() < 5 / 6 else k, "type": rng.choice(["f16", "bf16"]),
            "bias": rng.random() < 0.5}
    return {**case, "z": rng.choice([0.0, 1e-3])} if kind == "train" else case


def _shapes(case):
    """A stack of layers' weights: four attention projections, three feed-forward weights, two vectors each."""
    w, i, odd = case["width"], case["inner"], case["odd"]
    return ([(w, w)] * 4 + [(i, w)] * 3 + [(w,), (w + odd,)]) * case["layers"]


def _arena(shapes, t):
    """Zeros for tensors of these shapes in one tensor, and the tensors as views of it."""
    sizes = [-(-math.prod(s) // 256) * 256 for s in shapes]
    whole = torch.zeros(sum(sizes), dtype=t, device="cuda")
    return whole, [part[:math.prod(s)].view(s) for part, s in zip(whole.split(sizes), shapes)]


def _loss_scale(case):
    return 65536.0 if case["type"] == "f16" else 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, scale, t):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(t)

    if case["kind"] == "adamw":
        shapes, eight = _shapes(case), case["bits"] == 8
        held = [(math.prod(s) + -(-math.prod(s) // 32),) for s in shapes] if eight else shapes
        state = {"case": case, "norm": torch.tensor([2.5], device="cuda")}
        kinds = [("params", shapes, _TYPES[case["param"]]), ("grads", shapes, _TYPES[case["grad"]]),
                 ("m", held, torch.uint8 if eight else torch.float32), ("v", held, torch.uint8 if eight else torch.float32)]
        if case["copy"]:
            kinds.append(("copies", shapes, torch.float16 if case["grad"] == "f16" else torch.bfloat16))
        if eight:
            kinds += [("m_values", shapes, torch.bfloat16), ("v_values", shapes, torch.bfloat16)]
        for name, sizes, t in kinds:
            state["all_" + name], state[name] = _arena(sizes, t)
        for i, s in enumerate(shapes):
            state["params"][i].copy_(normal(s, 0.02, torch.float32))
            state["grads"][i].copy_(normal(s, 0.01, torch.float32))
            # the moments after some steps of gradients of this size
            m, v = normal(s, 0.002, torch.float32), normal(s, 0.004, torch.float32).square_()
            state["m"][i].copy_(_encode(m, True) if eight else m)
            state["v"][i].copy_(_encode(v, False) if eight else v)
        return state
    M, N, K = case["M"], case["N"], case["K"]
    t = _TYPES[case["type"]]
    state = {"case": case, "x": normal((M, K), 1.0, t), "w": normal((N, K), 2 / math.sqrt(K), t),
             "b": normal((N,), 0.5, t) if case["bias"] else None}
    target = torch.randint(0, N, (M,), generator=gen, device="cuda")
    if M > 4:      # one row in eight is padding
        target[torch.rand(M, generator=gen, device="cuda") < 0.125] = -100
    state["target"] = target
    if case["kind"] == "train":    # of the mean over the rows that count
        state["dloss"] = torch.where(target >= 0, _loss_scale(case) / (target >= 0).sum().clamp(min=1), 0.0).float()
    return state


# ---- the library's calls -------------------------------------------------------------

def _run_own(s):
    import linear_amd as la
    case = s["case"]
    if case["kind"] == "adamw":
        la.linear_adamw(s["params"], s["grads"], s["m"], s["v"], lr=_LR, beta1=_BETA1, beta2=_BETA2, eps=_EPS,
                        weight_decay=_DECAY, step=_STEP, norm=s["norm"], max_norm=_MAX_NORM, copies=s.get("copies"))
        if case["bits"] == 8:
            la.linear_adamw_values(s["m"], second=False, out=s["m_values"])
            la.linear_adamw_values(s["v"], second=True, out=s["v_values"])
        return _returned(s)
    f16 = case["type"] == "f16"
    loss, lse = (la.linear_f16_cross_entropy if f16 else la.linear_bf16_cross_entropy)(s["x"], s["w"], s["target"], s["b"])
    out = {"loss": loss, "lse": lse}
    if case["kind"] == "train":
        backward = la.linear_f16_cross_entropy_backward if f16 else la.linear_bf16_cross_entropy_backward
        dlse = lse * s["dloss"] * (2 * case["z"]) if case["z"] else None
        out["dx"], out["dw"], db = backward(s["dloss"], s["x"], s["w"], s["target"], lse, s["b"], dlse=dlse)
        if case["bias"]:
            out["db"] = db
    return out


def _returned(s):
    """What a training step hands back: weights, moments and, where there are any, the weights' copies."""
    eight = "_values" if s["case"]["bits"] == 8 else ""
    out = {"params": s["all_params"], "m": s["all_m" + eight], "v": s["all_v" + eight]}
    return {**out, "copies": s["all_copies"]} if s["case"]["copy"] else out


# ---- the plain forms -----------------------------------------------------------------

def _decode(state, n, signed):
    """The n values of an 8-bit state, in 32 bits."""
    code = state[:n].int()
    magnitude = code & 127 if signed else code
    e, f = magnitude >> 3, (magnitude & 7).float()
    bias = 7 if signed else 15
    value = torch.where(e == 0, f, f + 8) * torch.exp2((e.clamp(min=1) - (bias + 3)).float())
    if signed:
        value = torch.where(magnitude == 127, math.nan, value) * torch.where(code > 127, -1.0, 1.0)
    else:
        value = torch.where(code == 248, math.inf, torch.where(code > 248, math.nan, value))
    k = torch.exp2(state[n:].float() - 127)
    return value * k.repeat_interleave(32)[:n]


def _encode(x, signed):
    """The 8-bit state of x."""
    x = x.reshape(-1)
    n = x.numel()
    low, top, most = (-6, 8, 1.8125) if signed else (-14, 15, 1.9375)    # 464 = 1.8125 * 2^8, 63488 = 1.9375 * 2^15
    a = torch.nn.functional.pad(x.abs(), (0, -n % 32)).reshape(-1, 32)
    f, e = torch.frexp(torch.where(a.isfinite(), a, 0.0).amax(1))   # f in [1/2, 1), or 0
    k = torch.where(f > 0, e - 1 + (2 * f >= most).int() - top, -100).clamp(min=-100)
    y = (a * torch.exp2(-k.to(a.dtype))[:, None]).reshape(-1)[:n]
    e = (torch.frexp(y)[1] - 1).clamp(min=low)
    q = torch.round(y * torch.exp2((3 - e).to(y.dtype)))            # in eighths of 2^e: 16 is 8 of the next
    code = torch.where(y.isfinite(), q.nan_to_num(0, 0, 0).int() + 8 * (e - low), 0)
    if signed:
        code = torch.where(y.isfinite(), code, 127) + 128 * torch.signbit(x).int()
    else:
        code = torch.where(y > 0, code.clamp(min=1), code)
        code = torch.where(y.isinf(), 248, torch.where(y.isnan(), 255, code))
    return torch.cat([code.to(torch.uint8), (k + 127).to(torch.uint8)])


def _plain_adamw(s):
    case = s["case"]
    eight = case["bits"] == 8
    # 8-bit moments in 64 bits: sums of few-bit numbers lie on borders between codes, or within 32 bits' error of one
    wide = torch.float64 if eight else torch.float32
    scale = torch.clamp(_MAX_NORM / (s["norm"].to(wide) + 1e-6), max=1.0)
    a, r = _LR / (1 - _BETA1 ** _STEP), 1 / math.sqrt(1 - _BETA2 ** _STEP)
    for i, (p, grad) in enumerate(zip(s["params"], s["grads"])):
        g = grad.to(wide) * scale
        m, v = s["m"][i], s["v"][i]
        if eight:
            m, v = (_decode(t, p.numel(), signed).to(wide).reshape(p.shape) for t, signed in ((m, True), (v, False)))
        m, v = m * _BETA1 + g * (1 - _BETA1), v * _BETA2 + g * g * (1 - _BETA2)
        new = p.float() * (1 - _LR * _DECAY) - a * m.float() / (v.float().sqrt() * r + _EPS)
        p.copy_(new)
        if case["copy"]:
            s["copies"][i].copy_(new)
        for name, t in (("m", m), ("v", v)):
            s[name][i].copy_(_encode(t, name == "m") if eight else t)
            if eight:
                s[name + "_values"][i].copy_(_decode(s[name][i], p.numel(), name == "m").reshape(p.shape))
    return _returned(s)


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    if case["kind"] == "adamw":
        return _plain_adamw(state)
    t = _TYPES[case["type"]]
    x, w, target = state["x"].float(), state["w"].float(), state["target"]
    z = x @ w.t()
    if case["bias"]:
        z += state["b"].float()
    top = z.amax(1, keepdim=True)
    lse = (top + torch.exp(z - top).sum(1, keepdim=True).log())[:, 0]
    counts = (target >= 0) & (target < case["N"])
    at = torch.where(counts, target, 0)[:, None]
    out = {"loss": torch.where(counts, lse - z.gather(1, at)[:, 0], 0.0), "lse": lse}
    if case["kind"] == "score":
        return out
    dloss = torch.where(counts, state["dloss"], 0.0)
    rows = dloss + lse * state["dloss"] * (2 * case["z"]) if case["z"] else dloss
    dz = torch.exp(z - lse[:, None]) * rows[:, None]
    dz.scatter_add_(1, at, -dloss[:, None])
    out["dx"], out["dw"] = (dz @ w).to(t), (dz.t() @ x).to(t)
    if case["bias"]:
        out["db"] = dz.sum(0).to(t)
    return out


# ---- the work, and the values in 64 bits ---------------------------------------------

def work(case):
    if case["kind"] == "adamw":
        n = sum(math.prod(s) for s in _shapes(case))
        size = {"f16": 2, "bf16": 2, "f32": 4}
        p, g = size[case["param"]], size[case["grad"]]
        # weights and moments read and written, gradients read; 8-bit moments are returned as values too
        moments = 16 if case["bits"] == 32 else 2 * (2 + 2 / 32) + 2 * 2
        return {"bytes": n * (2 * p + g + moments + (g if case["copy"] else 0)), "flops": 16 * n}
    M, N, K = case["M"], case["N"], case["K"]
    read = 2 * (M * K + N * K + (N if case["bias"] else 0)) + 8 * M
    if case["kind"] == "score":
        return {"bytes": read + 8 * M, "flops": 2 * M * N * K + 3 * M * N}
    # the logits are not kept: they are formed for the loss, and again for the gradients
    return {"bytes": 2 * read + 16 * M + 2 * (M * K + N * K + (N if case["bias"] else 0)), "flops": 8 * M * N * K + 8 * M * N}


def _levels(signed):
    """The values of the codes 0, 1, .. that are finite and not negative, in 64 bits."""
    count, bias = (127, 7) if signed else (248, 15)
    return torch.tensor([(c % 8) * 2.0 ** (-bias - 2) if c < 8 else (8 + c % 8) * 2.0 ** (c // 8 - bias - 3) for c in range(count)],
                        dtype=torch.float64)


def _levels_of(state, n, signed):
    levels = _levels(signed).to(state.device)
    code = state[:n].long()
    value = levels[code % 128] * torch.where(code >= 128, -1.0, 1.0).double() if signed else levels[code]
    return value * torch.pow(2.0, state[n:].double() - 127).repeat_interleave(32)[:n]


def _nearest(x, signed):
    """What the 8-bit state of x (finite) stands for: in each block the nearest level, of two as near the even code's."""
    n = x.numel()
    levels = _levels(signed).to(x.device)
    middles = (levels[1:] + levels[:-1]) / 2
    a = torch.zeros(-(-n // 32) * 32, dtype=torch.float64, device=x.device)
    a[:n] = x.reshape(-1).abs()
    a = a.reshape(-1, 32)
    # the smallest k for which the largest is under the middle past the last level
    border = 464.0 if signed else 63488.0
    k = torch.ceil(torch.log2(torch.clamp(a.amax(1), min=1e-300) / border))
    k = torch.where(a.amax(1) >= border * torch.pow(2.0, k), k + 1, k).clamp(min=-100.0)
    y = a / torch.pow(2.0, k)[:, None]
    code = torch.searchsorted(middles, y)                    # the lower of two as near
    tie = (y == middles[code.clamp(max=middles.numel() - 1)]) & (code % 2 == 1) & (code < middles.numel())
    code = code + tie
    if not signed:
        code = torch.where((y > 0) & (code == 0), 1, code)
    value = (levels[code] * torch.pow(2.0, k)[:, None]).reshape(-1)[:n].reshape(x.shape)
    return torch.where(x < 0, -value, value)


def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "adamw":
        scale = min(1.0, _MAX_NORM / (float(s["norm"]) + 1e-6))
        names = ["params", "m", "v"] + (["copies"] if case["copy"] else [])
        out = {n: _arena(_shapes(case), torch.float64) for n in names}
        for i, (p, g, m, v) in enumerate(zip(s["params"], s["grads"], s["m"], s["v"])):
            g = g.double() * scale
            if case["bits"] == 8:
                m, v = (_levels_of(t, p.numel(), signed).reshape(p.shape) for t, signed in ((m, True), (v, False)))
            m = torch.lerp(g, m.double(), _BETA1)
            v = torch.lerp(g.square(), v.double(), _BETA2)
            hat = m / (1 - _BETA1 ** _STEP), v / (1 - _BETA2 ** _STEP)
            p = p.double()
            p = p - _LR * (hat[0] / (hat[1].sqrt() + _EPS) + _DECAY * p)
            if case["bits"] == 8:
                m, v = _nearest(m, True), _nearest(v, False)
            for name, value in zip(names, (p, m, v, p)):
                out[name][1][i].copy_(value)
        return {n: whole for n, (whole, _) in out.items()}
    x, w = s["x"].double().requires_grad_(), s["w"].double().requires_grad_()
    b = s["b"].double().requires_grad_() if case["bias"] else None
    with torch.enable_grad():
        z = torch.nn.functional.linear(x, w, b)
        lse = torch.logsumexp(z, 1)
        loss = torch.nn.functional.cross_entropy(z, s["target"], reduction="none", ignore_index=-100)
        out = {"loss": loss.detach(), "lse": lse.detach()}
        if case["kind"] == "train":
            total = (loss * s["dloss"].double()).sum() + case["z"] * (lse.square() * s["dloss"].double()).sum()
            wanted = [x, w] + ([b] if case["bias"] else [])
            grads = torch.autograd.grad(total, wanted)
            out.update(zip(["dx", "dw", "db"], grads))
    return out
