"""Plain 64-bit forms of the AdamW step and of 8-bit moments, and the bounds that the kernels' outputs
are held to.  Test infrastructure only.

Bounds, in half steps of FP32 (H = 2^-24).  32-bit moments: the factors beta and 1 - beta, the scale
and each product and sum are rounded, so m is off by at most 6 H (|beta1 m| + |(1 - beta1) g|) and v by
10 H of its (positive) terms.  The update rate * m / (sqrt(v) * root + eps) takes m's error over the
denominator, half of v's relative error, 4 H for the square root (2 steps), 2 H each for the
reciprocal, its rounded factors and the products: 16 H in all; p's product and difference are two more
roundings, and its own.  Codes of 8-bit moments are computed in FP64 in the order written here, so
they are equal.
"""
import torch

from train_refs import half_step, tiny

H = 2.0 ** -24
BLOCK = 32


def levels(second):
    """The values of the codes 0, 1, .. (no sign), in units of the block."""
    count, bias = (248, 15) if second else (127, 7)
    return torch.tensor([(c % 8) * 2.0 ** (-bias - 2) if c < 8 else (8 + c % 8) * 2.0 ** (c // 8 - bias - 3) for c in range(count)],
                        dtype=torch.float64)


def power(k):
    """2^k for whole k, exactly (torch.ldexp goes through a power that may be a step off)."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def decode(state, n, second):
    """The n values of a state, in 64 bits."""
    lv = torch.cat([levels(second), torch.tensor([float("inf")] if second else [], dtype=torch.float64),
                    torch.full((7 if second else 1,), float("nan"), dtype=torch.float64)]).to(state.device)
    code = state[:n].long()
    value = lv[code] if second else lv[code % 128] * (1 - 2 * (code // 128)).double()
    unit = torch.where(state[n:] == 0, 0.0, power(state[n:].int() - 127))
    return value * unit.repeat_interleave(BLOCK)[:n]


def encode(x, second):
    """The state of the 64-bit values x: the nearest code, of two as near the even one."""
    x = x.reshape(-1).double()
    n = x.numel()
    lv = levels(second).to(x.device)
    middle = (lv[1:] + lv[:-1]) / 2
    border, nan = (63488.0, 255) if second else (464.0, 127)
    held = x.float().abs()                            # magnitudes are judged as FP32 holds them
    odd = ~(held < 1.9375 * 2.0 ** 127)
    held = torch.nn.functional.pad(torch.where(odd, 0.0, held), (0, -n % BLOCK)).reshape(-1, BLOCK).amax(1).double()
    a = torch.nn.functional.pad(torch.where(odd, 0.0, x.abs()), (0, -n % BLOCK)).reshape(-1, BLOCK)
    k = torch.full((a.shape[0],), -100, dtype=torch.int32, device=x.device)
    for _ in range(230):                              # the smallest k from -100 on that the largest fits under
        k += (held >= border * power(k)).int()
    y = (a * power(-k)[:, None]).reshape(-1)[:n]
    code = torch.searchsorted(middle, y)              # the lower of two as near
    code += ((code % 2 == 1) & (code < middle.numel()) & (y == middle[code.clamp(max=middle.numel() - 1)])).long()
    if second:
        code = torch.where((y > 0) & (code == 0), 1, code)
        code = torch.where(odd, torch.where(x.isnan(), 255, 248), code)
    else:
        code = torch.where(odd, 127, code) + 128 * torch.signbit(x).long()
    return torch.cat([code.to(torch.uint8), (k + 127).to(torch.uint8)])


def same_state(a, b, n, second):
    """The same units, and codes that stand for the same numbers (a zero's sign, and which of the codes
    for NaN, are not told apart)."""
    x, y = decode(a, n, second), decode(b, n, second)
    return torch.equal(a[n:], b[n:]) and bool(((x == y) | (x.isnan() & y.isnan())).all())


def clip_scale(norm, max_norm):
    if norm is None:
        return 1.0
    s = max_norm / (float(norm) + 1e-6)
    return 1.0 if s >= 1.0 else s


def step64(p, g, m, v, o, step, scale=1.0):
    """(p, m, v) after a step and the bounds of each; m and v the 64-bit values before it."""
    p, g = p.double(), g.double() * scale
    b1, b2 = o["beta1"], o["beta2"]
    am, av = (m * b1).abs() + (g * (1 - b1)).abs(), v * b2 + g * g * (1 - b2)
    m, v = m * b1 + g * (1 - b1), v * b2 + g * g * (1 - b2)
    em, ev = 6 * H * am + 2.0 ** -149, 10 * H * av + 2.0 ** -149
    c1, c2 = 1 - b1 ** step, 1 - b2 ** step
    den = (v / c2).sqrt() + o["eps"]
    u = o["lr"] / c1 * m / den
    eu = o["lr"] / c1 * em / den + u.abs() * (((v + ev) / c2).sqrt() - ((v - ev).clamp(min=0) / c2).sqrt()) / den + 16 * H * u.abs()
    new = p * (1 - o["lr"] * o["weight_decay"]) - u
    return (new, m, v), (eu + 4 * H * (p.abs() + u.abs()), em, ev)


def stored(value, bound, t):
    return bound + half_step(t) * (value.abs() + bound) + tiny(t) if t != torch.float32 else bound + tiny(t)
