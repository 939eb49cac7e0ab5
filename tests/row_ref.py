"""Plain 64-bit forms of the row operators and the tolerances their FP32
kernels are held to.

A rounding to a type t is off by at most finfo(t).eps / 2 relative to the
value.  U = 2^-24 is FP32's.  A sum of n FP32 terms is off by at most
depth * U * sum |terms|, depth the longest chain of additions that a term
goes through; the kernels' chains are written beside each use."""
import torch

U = 2.0 ** -24
# A thread adds at most 128 values of a row in a chain (long rows: N / 1024),
# then 5 shuffles and at most 32 warps: under 170 roundings.
ROW = 170


def half_ulp(t: torch.dtype) -> float:
    return torch.finfo(t).eps / 2


def assert_within(got, ref, bound, what):
    """|got - ref| <= bound, element by element; the subnormal step of got's
    type is allowed too, since a rounding there is absolute."""
    assert got.shape == ref.shape, f"{what}: shape {tuple(got.shape)}"
    tiny = torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps
    over = (got.double() - ref).abs() - (bound + tiny)
    assert not torch.isnan(over).any(), f"{what}: NaN"
    worst = over.max().item() if over.numel() else -1.0
    assert worst <= 0.0, f"{what}: off by {worst:.3e} beyond the bound"


def layernorm(x, gamma, beta, eps):
    """y, mean, rstd and y's bound.  The centred value carries the mean's error
    (ROW * U * avg|x - mean|, under ROW * U / rstd, after the kernel's second
    pass), rstd half of the variance's, and a few roundings follow."""
    x = x.double()
    g = torch.ones(x.shape[1], dtype=torch.float64, device=x.device) if gamma is None else gamma.double()
    b = torch.zeros_like(g) if beta is None else beta.double()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / torch.sqrt(d.square().mean(1) + eps)
    xh = d * rstd[:, None]
    y = xh * g + b
    return y, mean, rstd, (ROW + 8) * U * ((xh.abs() + 1.0) * g.abs() + b.abs())


def norm_backward(dy, x, mean, rstd, gamma, dres):
    """dx, dgamma, dbeta and their bounds (mean None: RMSNorm).  The averages
    carry ROW roundings of their absolute terms, the rest a few each.  dgamma
    and dbeta: a block adds its rows one after another (at most M / blocks + 8
    groups), the blocks' sums in chains of at most 40, 16 warps after that."""
    dy, x, rstd = dy.double(), x.double(), rstd.double()[:, None]
    g = dy * (1.0 if gamma is None else gamma.double())
    xh = (x if mean is None else x - mean.double()[:, None]) * rstd
    c1 = torch.zeros_like(rstd) if mean is None else g.mean(1, keepdim=True)
    c2 = (g * xh).mean(1, keepdim=True)
    dx = rstd * (g - c1 - xh * c2)
    a1 = torch.zeros_like(rstd) if mean is None else g.abs().mean(1, keepdim=True)
    a2 = (g * xh).abs().mean(1, keepdim=True)
    bound = rstd * (8 * U * (g.abs() + c1.abs() + (xh * c2).abs()) + ROW * U * (a1 + xh.abs() * a2))
    # (x - mean) is rounded once relative to itself: within the 8
    if dres is not None:
        dx = dx + dres.double()
        bound = bound + U * dx.abs()
    depth = x.shape[0] / 64 + 80
    return (dx, bound), ((dy * xh).sum(0), depth * U * (dy * xh).abs().sum(0) + 1e-300), \
        (dy.sum(0), depth * U * dy.abs().sum(0) + 1e-300)


def embedding_backward(dy, ids, vocab, scale, padding, old=None):
    """dw and its bound: a row of n tokens is a chain of at most n additions,
    and the scale and an old value cost one rounding each."""
    dy, ids = dy.double().reshape(ids.numel(), -1), ids.reshape(-1).long()
    keep = (ids >= 0) & (ids < vocab)
    if padding is not None:
        keep &= ids != padding
    dw = torch.zeros(vocab, dy.shape[1], dtype=torch.float64, device=dy.device)
    size = torch.zeros_like(dw)
    dw.index_add_(0, ids[keep], dy[keep] * scale)
    size.index_add_(0, ids[keep], (dy[keep] * scale).abs())
    n = torch.bincount(ids[keep], minlength=vocab).double()[:, None]
    bound = (n + 2) * U * size
    if old is not None:
        dw = dw + old.double()
        bound = bound + U * dw.abs()
    return dw, bound


def padded(rows, cols, ld, dtype, fill, device="cuda"):
    """A [rows, cols] view of leading dimension ld inside a buffer of `fill`."""
    buf = torch.full((rows, ld), fill, dtype=dtype, device=device)
    return buf, buf[:, :cols]
