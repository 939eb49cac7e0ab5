"""GPU tests of the row operators where sizes, magnitudes and orders reach their
limits: rows at the ends of their buffers, values near the ends of FP32's range,
NaN and infinities, rows longer than a grid's dimension, failures of two kinds."""
import pytest
import torch

import blockwise_fp8_linear_fp8bq_b200 as fp
from row_ref import U, assert_within, half_ulp, layernorm, norm_backward

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def gen_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def inside(t, by):
    """t's values `by` elements into a buffer of NaN that ends with them."""
    flat = torch.full((by + t.numel(),), float("nan"), dtype=t.dtype, device="cuda")
    view = flat[by:].view(t.shape)
    view.copy_(t)
    return view


def backward(kind, dy, x, mean, rstd, gamma=None, dres=None, **kw):
    if kind == "ln":
        return fp.layernorm_backward(dy, x, mean, rstd, gamma, dres, **kw)
    return (*fp.rmsnorm_backward(dy, x, rstd, gamma, dres, **kw), None)


@pytest.mark.parametrize("kind", ["ln", "rms"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N", [(1, 1), (1, 3), (1, 9), (2, 5), (3, 17), (40, 333)])
def test_values_at_the_ends_of_unaligned_tensors(M, N, dtype, kind):
    """Rows whose first and last values are copied into their stage one by one,
    each tensor's by another lane (of the smallest tensors nothing else is), call
    after call into memory that held other rows."""
    gen = gen_of(M * 100 + N)
    for by in range(1, 9):
        x = inside(torch.randn(M, N, generator=gen, device="cuda").to(dtype), by)
        dy = inside((torch.randn(M, N, generator=gen, device="cuda") * 0.01).to(dtype), by + 1)
        dres = inside((torch.randn(M, N, generator=gen, device="cuda") * 0.01).to(dtype), by + 2)
        mean = x.double().mean(1).float() if kind == "ln" else None
        rstd = torch.rand(M, generator=gen, device="cuda") + 0.5
        (ref, bound), _, _ = norm_backward(dy, x, mean, rstd, None, dres)
        y = fp.layernorm_forward(x)[0]
        ry, _, _, by_ = layernorm(x, None, None, 1e-5)
        assert_within(y, ry, by_ + half_ulp(dtype) * (ry.abs() + by_), "y")
        for _ in range(20):
            dx = backward(kind, dy, x, mean, rstd, None, dres)[0]
            assert_within(dx, ref, bound + half_ulp(dtype) * (ref.abs() + bound), "dx")
    fp.check()


def test_table_gradient_of_rows_longer_than_a_grids_second_dimension():
    """Rows of an odd length of which a grid of 65535 x 256 threads does not reach
    the end, in two chunks of tokens that one id's run spans."""
    T, V, D = 9, 2, 65535 * 256 + 300001
    ids = torch.tensor([0, 1, 1, 1, 1, 1, 1, 1, 1], device="cuda")  # the last of them is the second chunk
    dy = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
    for t in range(T):
        dy[t] = t + 1.0
        dy[t, -1] = -1.0 - t
    dw = fp.embedding_backward(dy, ids, V, scale=0.5)
    for v, s in ((0, 0.5), (1, 22.0)):
        assert (dw[v, :-1] == s).all() and dw[v, -1] == -s
    fp.embedding_backward(dy, ids, V, scale=0.5, out=dw, accumulate=True)
    for v, s in ((0, 1.0), (1, 44.0)):
        assert (dw[v, :-1] == s).all() and dw[v, -1] == -s
    fp.check()
    torch.cuda.synchronize()


# (rows, columns): one warp's, 8 lanes', several warps', few rows', unaligned and long rows
LAYOUTS = [(1100, 640), (1100, 64), (1100, 100), (1050, 4096), (1100, 641), (40, 2048), (40, 77), (20, 20001)]


@pytest.mark.parametrize("M,N", LAYOUTS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_layernorm_statistics_of_rows_with_nan_and_infinities(dtype, M, N):
    """Such a row's rstd is NaN as the definition has it, not that of a row of no
    variance, its mean is not finite, and the other rows keep their bits."""
    x = torch.randn(M, N, generator=gen_of(N), device="cuda").to(dtype)
    clean = fp.layernorm_forward(x)
    x[3, N - 1] = float("nan")
    x[7, 0] = float("inf")
    x[8, N // 2] = -float("inf")
    x[11, 1], x[11, N - 2] = float("inf"), -float("inf")
    y, mean, rstd = fp.layernorm_forward(x)
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    bad[[3, 7, 8, 11]] = True
    assert torch.isnan(rstd[bad]).all() and torch.isnan(y[bad]).all() and not torch.isfinite(mean[bad]).any()
    for got, want in zip((y, mean, rstd), clean):
        assert torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("kind", ["ln", "rms", "rms64"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N", LAYOUTS + [(1030, 2047), (1100, 2048), (300, 12288)])
def test_norm_backward_of_tiny_and_huge_rows(M, N, dtype, kind):
    """Rows whose rstd is in FP32's range and whose rstd^2 is not (eps = 0 for the
    tiny ones); dy goes along with x, so that the projection is as large as dy.
    rms64: a float64 rstd."""
    gen = gen_of(M + N)
    x0 = torch.randn(M, N, generator=gen, device="cuda") + 0.3
    dy0 = 0.5 * x0 + torch.randn(M, N, generator=gen, device="cuda")
    gamma = (1 + 0.1 * torch.randn(N, generator=gen, device="cuda")).to(dtype)
    dres0 = torch.randn(M, N, generator=gen, device="cuda") if N % 2 or M == 1100 else None
    for size in (1e-37, 1e-25, 1e-18, 1e15, 1e17, 1e20, 1e25, 1e30, 1e37):
        x = (x0.double() * size).to(dtype)
        at = min(max(size * 1e-20, 1e-10), 1e10)
        dy = (dy0.double() * at).to(dtype)
        dres = None if dres0 is None else (dres0.double() * (at / size)).to(dtype)
        x64 = x.double()
        mean = x64.mean(1).float() if kind == "ln" else None
        rstd = 1.0 / (x64 if mean is None else x64 - mean.double()[:, None]).square().mean(1).sqrt()
        rstd = rstd if kind == "rms64" else rstd.float()
        (ref, bound), (rdg, bdg), (rdb, bdb) = norm_backward(dy, x, mean, rstd, gamma, dres)
        dx, dgamma, dbeta = backward(kind, dy, x, mean, rstd, gamma, dres)
        assert_within(dx, ref, bound + half_ulp(dtype) * (ref.abs() + bound), f"dx at {size}")
        assert_within(dgamma, rdg, bdg + 8 * U * rdg.abs(), f"dgamma at {size}")
        if kind == "ln":
            assert_within(dbeta, rdb, bdb + U * rdb.abs(), f"dbeta at {size}")


@pytest.mark.parametrize("kind", ["ln", "rms"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N", LAYOUTS + [(1500, 2047)])
def test_dx_over_the_residuals_gradient(M, N, dtype, kind):
    """The same bits, and the same sums, as into memory of its own."""
    gen = gen_of(M + N)
    x = torch.randn(M, N, generator=gen, device="cuda").to(dtype)
    dy = (torch.randn(M, N, generator=gen, device="cuda") * 0.01).to(dtype)
    dres = (torch.randn(M, N, generator=gen, device="cuda") * 0.01).to(dtype)
    mean = x.double().mean(1).float() if kind == "ln" else None
    rstd = torch.rand(M, generator=gen, device="cuda") + 0.5
    want = backward(kind, dy, x, mean, rstd, None, dres)
    over = dres.clone()
    got = backward(kind, dy, x, mean, rstd, None, over, out=(over, None, None) if kind == "ln" else (over, None))
    assert got[0] is over or got[0].data_ptr() == over.data_ptr()
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("kind", ["ln", "rms"])
@pytest.mark.parametrize("M,N", LAYOUTS)
def test_norm_backward_with_nan_and_infinities(M, N, kind):
    """They reach dx in their rows alone, dgamma and dbeta in their columns alone."""
    gen = gen_of(M * 3 + N)
    x = torch.randn(M, N, generator=gen, device="cuda")
    dy = torch.randn(M, N, generator=gen, device="cuda") * 0.01
    mean = x.mean(1) if kind == "ln" else None
    rstd = torch.rand(M, generator=gen, device="cuda") + 0.5
    clean = backward(kind, dy, x, mean, rstd)
    x[3, N - 1] = float("nan")
    dy[7, 0] = float("nan")
    dy[11, N // 2] = float("inf")
    dx, dgamma, dbeta = backward(kind, dy, x, mean, rstd)
    rows = torch.zeros(M, dtype=torch.bool, device="cuda")
    rows[[3, 7, 11]] = True
    assert torch.equal(dx[~rows], clean[0][~rows])
    assert torch.isnan(dx[3]).all() and torch.isnan(dx[7]).all() and not torch.isfinite(dx[11]).any()
    cols = torch.zeros(N, dtype=torch.bool, device="cuda")
    cols[[N - 1, 0, N // 2]] = True
    assert torch.equal(dgamma[~cols], clean[1][~cols]) and not torch.isfinite(dgamma[cols]).any()
    if kind == "ln":
        assert torch.isnan(dbeta[0]) and dbeta[N // 2] == float("inf") and torch.equal(dbeta[1:N // 2], clean[2][1:N // 2])


@pytest.mark.parametrize("D", [64, 77])
@pytest.mark.parametrize("T", [300, 3000])
def test_table_gradient_with_nan_and_infinities(T, D):
    """They reach their own token's row; those of tokens that add nothing reach none."""
    gen = gen_of(T)
    V = 90
    ids = torch.randint(1, V - 2, (T,), generator=gen, device="cuda")
    ids[10], ids[20], ids[30], ids[40] = 0, V, V - 1, V - 2
    dy = torch.randn(T, D, generator=gen, device="cuda")
    clean = fp.embedding_backward(dy, ids, V, padding_id=0)
    dy[10], dy[20] = float("nan"), float("inf")  # padding and an id outside the table
    dy[30, 3], dy[40, 5] = float("nan"), -float("inf")
    dw = fp.embedding_backward(dy, ids, V, padding_id=0)
    assert torch.equal(dw[:V - 2], clean[:V - 2])
    assert torch.isnan(dw[V - 1, 3]) and dw[V - 1].isnan().sum() == 1
    assert dw[V - 2, 5] == -float("inf") and (~dw[V - 2].isfinite()).sum() == 1
    with pytest.raises(fp.Fp8bqError):
        fp.check()


@pytest.mark.parametrize("most", [1.0, 1e-6, 1e-30, 1e-38])
@pytest.mark.parametrize("n", [1, 5000, 300001, 6000000])
def test_clipping_gradients_that_blew_up(n, most):
    """A limit so far below the norm that their quotient is below FP32's normal
    range; the clipped values are not."""
    g = torch.randn(n, generator=gen_of(n), device="cuda").clamp_(-3, 3) * 1e38
    g64 = g.double()
    norm = g64.square().sum().sqrt().item()
    factor = most / (norm + 1e-6)
    ref = g64 * factor
    for out in (torch.float32, torch.bfloat16):
        o = torch.empty(n, dtype=out, device="cuda")
        fp.clip_grads([g], most, out=[o])
        # the norm's error, the factor's rounding, the product's, then the type's
        assert_within(o, ref, (8 * U + half_ulp(out) * (1 + 4 * U)) * ref.abs(), "clipped")
    over = g.clone()
    fp.clip_grads([over], most)
    assert_within(over, ref, (8 * U + half_ulp(torch.float32) * (1 + 4 * U)) * ref.abs(), "clipped in place")


def test_a_small_factor_whose_bits_round_to_one_is_not_one():
    """In place: a factor of 2^-146 (1 - 2^-27) scales, though FP32 rounds its bits up to 1."""
    g = torch.tensor([2.0 ** 126], device="cuda")
    fp.clip_grads([g], 2.0 ** -20 * (1 - 2.0 ** -27))
    assert abs(g.item() - 2.0 ** -20) <= 2.0 ** -20 * 2.0 ** -22
