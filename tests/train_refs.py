"""Plain 64-bit forms of the gated block, its gradients and the layer's gradients, and the bounds
that the kernels' outputs are held to.  Test infrastructure only.

Bounds.  S = the step of one FP32 ulp, 2^-23 relative; u = half a step of the output type,
finfo.eps / 2.  A matrix-core step adds 16 or more products to an accumulator with an error under
one FP32 ulp of its largest term, so a sum of L products of total magnitude A is off by at most
(L / 16 + 48) S A (48: the additions of partial sums over waves, segments and splits, each an
FP32 addition).  A rounding to the output type adds u times the value, or half the spacing of the
subnormals (tiny).  The activations' FP32 evaluation: exp(z) is off by a relative S (|z| + 8)
(the rounding of its scaled argument, and the instruction), erfc(v) by S (2 v^2 + 8) (the
argument's rounding times |v erfc'(v) / erfc(v)| <= 2 v^2 + 2, and the function), the few other
operations by S / 2 each.  Where exp overflows FP32 (z below -88) the kernel has 0 for a sigmoid
under 2^-126; FLOOR covers what is then lost, times the factors it is multiplied with.
"""
import math

import torch

import linear_amd as la

S = 2.0 ** -23
FLOOR = 2.0 ** -118          # |g| 2^-126 for |g| <= 2^8
ACTS = {la.EPI_SILU: "silu", la.EPI_GELU_TANH: "gelu_tanh", la.EPI_GELU_ERF: "gelu_erf"}
A_TANH, B_TANH = 2 * math.sqrt(2 / math.pi), 0.044715


def half_step(t):
    return torch.finfo(t).eps / 2


def tiny(t):
    return torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2


def rounded(v, e, t):
    """The bound of a value v, known to e, after rounding to t."""
    return e + half_step(t) * (v.abs() + e) + tiny(t) if t != torch.float32 else e + tiny(t)


def acc(L, A):
    return (L / 16 + 48) * S * A


def act64(act, g):
    """act(g), act'(g), and the relative bounds of their FP32 evaluation (the derivative's as an
    absolute bound)."""
    if act == la.EPI_GELU_ERF:
        p = 0.5 * torch.special.erfc(-g / math.sqrt(2))
        q = g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
        r = S * (g * g + 12)
        return g * p, p + q, r, 2 * r * (p + q.abs()) + FLOOR
    z, dz = g, torch.ones_like(g)
    if act == la.EPI_GELU_TANH:
        z, dz = A_TANH * (g + B_TANH * g ** 3), A_TANH * (1 + 3 * B_TANH * g * g)
    s = torch.sigmoid(z)
    c = torch.sigmoid(-z)
    r = S * (4 * z.abs() + 12)
    return g * s, s + g * s * c * dz, r, 2 * r * (s + (g * s * c * dz).abs()) + FLOOR * (1 + dz.abs())


def gated64(x, wg, wu, act, t):
    """(h, g, u) and their bounds for operands of type t."""
    x, wg, wu = x.double(), wg.double(), wu.double()
    K = x.shape[1]
    g, u = x @ wg.t(), x @ wu.t()
    eg, eu = acc(K, x.abs() @ wg.abs().t()), acc(K, x.abs() @ wu.abs().t())
    a, _, r, _ = act64(act, g)
    h = a * u
    # |act'| <= 1.13 for all three
    ea = 1.13 * eg + r * (a.abs() + 1.13 * eg) + FLOOR
    eh = ea * (u.abs() + eu) + a.abs() * eu + S * h.abs()
    return (h, g, u), (rounded(h, eh, t), rounded(g, eg, t), rounded(u, eu, t))


def gated_backward64(dh, x, wg, wu, g, u, act, t):
    """(dx, dwg, dwu), their bounds, and dg and du."""
    dh, x, wg, wu, g, u = (v.double() for v in (dh, x, wg, wu, g, u))
    M, N = dh.shape
    a, d, r, ed = act64(act, g)
    dg, du = dh * u * d, dh * a
    eg = rounded(dg, (dh * u).abs() * ed + 2 * S * dg.abs(), t)
    eu = rounded(du, (r + S) * du.abs() + dh.abs() * FLOOR, t)
    dx = dg @ wg + du @ wu
    bg, bu = dg.abs() + eg, du.abs() + eu
    ex = eg @ wg.abs() + eu @ wu.abs() + acc(2 * N, bg @ wg.abs() + bu @ wu.abs())
    dwg, dwu = dg.t() @ x, du.t() @ x
    ewg = eg.t() @ x.abs() + acc(M, bg.t() @ x.abs())
    ewu = eu.t() @ x.abs() + acc(M, bu.t() @ x.abs())
    return (dx, dwg, dwu), (rounded(dx, ex, t), rounded(dwg, ewg, t), rounded(dwu, ewu, t)), (dg, du)


def linear_backward64(dy, x, w, t, wide):
    """(dx, dw, db) and their bounds; dw and db in FP32 when wide."""
    dy, x, w = dy.double(), x.double(), w.double()
    M, N = dy.shape
    o = torch.float32 if wide else t
    dx, dw, db = dy @ w, dy.t() @ x, dy.sum(0)
    ax, aw, ab = dy.abs() @ w.abs(), dy.abs().t() @ x.abs(), dy.abs().sum(0)
    # db: a chain of at most M additions in all (rows of a split, then the splits)
    return (dx, dw, db), (rounded(dx, acc(N, ax), t), rounded(dw, acc(M, aw), o), rounded(db, (M + 2) * S / 2 * ab, o))


def inside(got, want, bound, what):
    """Every value within its bound; a value at or past the type's overflow threshold (its largest
    value plus half of the spacing there: 65520 in binary16) rounds to the infinity of its sign."""
    d = (got.double() - want).abs()
    top = torch.finfo(got.dtype).max * (1 + half_step(got.dtype) / 2)
    over = got.isinf() & (want.sign() == got.double().sign()) & (want.abs() + bound >= top)
    bad = ~((d <= bound) | over)
    if bool(bad.any()):
        i = int(torch.argmax((d / bound).nan_to_num(nan=float("inf")).flatten()))
        raise AssertionError("%s: %d of %d outside, worst at %d: got %r want %r bound %r" % (
            what, int(bad.sum()), bad.numel(), i, float(got.flatten()[i]), float(want.flatten()[i]),
            float(bound.flatten()[i])))
