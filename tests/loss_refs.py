"""Plain 64-bit forms of a linear head's cross entropy and its gradients, and the bounds that the
kernels' outputs are held to.  Test infrastructure only; the notation and the bound of a matrix-core
sum (acc) are train_refs'.

Bounds.  z is a sum of K products plus the bias: ez = acc(K, |x||w|) + S (|z| + |b|).  An FP32
exp(y) of a rounded difference is off by a relative S (|y| + 8).  A row's sum of exponentials is
taken relative to a tile's, a workgroup's and the row's largest z, three factors whose arguments lie
between 0 and z - top, and added in a chain of at most 64 values a lane, 16 steps over lanes and
waves, N / 8192 + 1 statistics a thread (tiles of 32 columns, 256 threads) and 8 more: a relative
(90 + N / 8192) S.  Each term's error counts by its share p of the sum, so lse is off by
sum_n p (ez + 3 S (|z - top| + 8)) + (90 + N / 8192) S, doubled for second-order terms, and the
logarithm and the addition by 2 S (|lse - top| + |lse|).  dz follows by the same rules, is rounded to the
type (binary16: after a scaling that puts the largest row weight above 2^14, so its subnormals'
half spacing is 2^-25 / 2^14 of that weight), and dx, dw, db are sums of its products.
"""
import torch

from train_refs import S, acc, half_step, rounded


def counted(target, N):
    return (target >= 0) & (target < N)


def forward64(x, w, target, b=None):
    """(loss, lse, z) in 64 bits and the bounds of each."""
    x, w = x.double(), w.double()
    (M, K), N = x.shape, w.shape[0]
    z, ez = x @ w.t(), acc(K, x.abs() @ w.abs().t())
    if b is not None:
        z = z + b.double()
        ez = ez + S * (z.abs() + b.double().abs()).nan_to_num(0, posinf=0, neginf=0)
    if N == 0:
        lse = torch.full((M,), float("-inf"), dtype=torch.float64, device=x.device)
        return (torch.zeros_like(lse), lse, z), (torch.zeros_like(lse),) * 2 + (ez,)
    top = z.amax(1, keepdim=True)
    lse = torch.logsumexp(z, 1)
    p = torch.exp(z - lse[:, None])
    far = (top - z).nan_to_num(0, posinf=0, neginf=0)
    el = 2 * ((p * (ez + 3 * S * (far + 8))).sum(1) + (90 + N / 8192) * S) + 2 * S * ((lse - top[:, 0]).abs() + lse.abs())
    ok = counted(target, N)
    at = torch.where(ok, target, 0)[:, None]
    loss = torch.where(ok, lse - z.gather(1, at)[:, 0], 0.0)
    eo = torch.where(ok, el + ez.gather(1, at)[:, 0] + S * loss.abs(), 0.0)
    return (loss, lse, z), (eo, el, ez)


def backward64(dloss, dlse, x, w, target, b, t, f32=False):
    """(dx, dw, db) and their bounds."""
    (_, lse, z), (_, el, ez) = forward64(x, w, target, b)
    x, w = x.double(), w.double()
    (M, K), N = x.shape, w.shape[0]
    ok = counted(target, N)
    one = torch.where(ok, dloss.double(), 0.0)[:, None]
    rows = one if dlse is None else one + dlse.double()[:, None]
    y = z - lse[:, None]
    p = torch.exp(y)
    hot = torch.zeros_like(z)
    if M and N:
        hot.scatter_(1, torch.where(ok, target, 0)[:, None], ok.double()[:, None])
    dz = rows * p - one * hot
    far = y.abs().nan_to_num(0, posinf=0)
    e = rows.abs() * p * (2 * (ez + el[:, None]) + S * (far + 10)) + S * (rows.abs() * p + one.abs() * hot)
    least = 0.0
    if t == torch.float16 and M:
        least = 2.0 ** -39 * float((rows.abs() + one.abs()).max())
    e = e + half_step(t) * (dz.abs() + e) + least
    # the matrix unit takes a binary16 subnormal for a number of 2^-14 where it aligns a product's sum
    size = dz.abs() + e + (2.0 ** 11 * least if t == torch.float16 else 0)
    ax = x.abs().clamp(min=2.0 ** -14) if t == torch.float16 else x.abs()
    aw = w.abs().clamp(min=2.0 ** -14) if t == torch.float16 else w.abs()
    o = torch.float32 if f32 else t
    dx, dw, db = dz @ w, dz.t() @ x, dz.sum(0)
    return (dx, dw, db), (rounded(dx, e @ w.abs() + acc(N, size @ aw), t),
                          rounded(dw, e.t() @ x.abs() + acc(M, size.t() @ ax), o),
                          rounded(db, e.sum(0) + (M + 2) * S / 2 * size.sum(0), o))
