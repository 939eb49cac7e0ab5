"""GPU tests of LayerNorm's two passes and RMSNorm's backward pass against the
64-bit forms, at the sizes where the kernels change shape: rows of one value,
rows of a warp, of a block, longer than a block's registers, odd lengths and
leading dimensions, one row to many."""
import pytest
import torch

import blockwise_fp8_linear_fp8bq_b200 as fp
from row_ref import U, assert_within, half_ulp, layernorm, norm_backward, padded

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
# (rows, columns, extra leading dimension)
SIZES = [(1, 1, 0), (3, 7, 0), (5, 64, 8), (1, 640, 0), (200, 1283, 0), (130, 1280, 3), (509, 2048, 0), (33, 4100, 0),
         (300, 4096, 16), (40, 6144, 0), (7, 8192, 0), (3, 8200, 0), (5, 16384, 0), (3, 20001, 0), (2, 70000, 0),
         (2000, 64, 0), (2001, 128, 8), (3000, 77, 0), (1500, 120, 1), (1100, 256, 0), (1027, 250, 0), (1025, 320, 0),
         (1200, 1000, 24), (1100, 1048, 0), (1030, 2047, 0), (1030, 2100, 0), (1026, 5000, 0), (1025, 12288, 0),
         (600, 12287, 0), (300, 14000, 0)]


def draw(gen, rows, cols, dtype, ld=0, std=1.0, mean=0.0):
    x = (torch.randn(rows, cols, generator=gen, device="cuda") * std + mean).to(dtype)
    if ld:
        buf, view = padded(rows, cols, cols + ld, dtype, float("nan"))
        view.copy_(x)
        return view
    return x


def gen_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def params(gen, n, dtype, mode):
    if mode == "none":
        return None, None
    dt = torch.float32 if mode == "fp32" else dtype
    return (1 + 0.1 * torch.randn(n, generator=gen, device="cuda")).to(dt), torch.randn(n, generator=gen,
                                                                                        device="cuda").to(dt)


@pytest.mark.parametrize("mode", ["same", "fp32", "none"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,pad", SIZES)
def test_layernorm_forward(M, N, pad, dtype, mode):
    gen = gen_of(M * 1000 + N)
    x = draw(gen, M, N, dtype, pad, mean=0.5)
    gamma, beta = params(gen, N, dtype, mode)
    buf, out = padded(M, N, N + pad, dtype, 7.0)
    y, mean, rstd = fp.layernorm_forward(x, gamma, beta, 1e-5, out=(out, None, None))
    ry, rmean, rrstd, bound = layernorm(x, gamma, beta, 1e-5)
    assert_within(y, ry, bound + half_ulp(dtype) * (ry.abs() + bound), "y")
    spread = 1.0 / rrstd
    assert_within(mean, rmean, U * rmean.abs() + 178 * U * spread, "mean")
    assert_within(rstd, rrstd, 100 * U * rrstd, "rstd")
    assert (buf[:, N:] == 7.0).all()  # columns past the row are left alone
    # in place, in the same layout (another one may be summed in another order)
    x2 = torch.empty_strided(x.shape, x.stride(), dtype=dtype, device="cuda")
    x2.copy_(x)
    y2, _, _ = fp.layernorm_forward(x2, gamma, beta, 1e-5, out=(x2, None, None))
    assert torch.equal(y2, y)


def shifted(t, by, fill=float("nan")):
    """t's values `by` elements into a buffer: rows that start anywhere."""
    flat = torch.full((t.numel() + by + 9,), fill, dtype=t.dtype, device="cuda")
    view = flat[by:by + t.numel()].view(t.shape)
    view.copy_(t)
    return flat, view


@pytest.mark.parametrize("by", [1, 3, 4, 7])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N", [(1, 1), (2, 3), (5, 64), (2100, 64), (70, 333), (400, 640), (3, 5000), (1, 9)])
def test_rows_that_start_anywhere(M, N, dtype, by):
    """Tensors whose first value is at no multiple of 16 bytes, in a buffer of
    NaN, every one of them at another offset."""
    gen = gen_of(M + N + by)
    _, x = shifted(draw(gen, M, N, dtype, mean=0.5), by)
    _, dy = shifted(draw(gen, M, N, dtype, std=0.01), by + 1)
    _, dres = shifted(draw(gen, M, N, dtype, std=0.01), by + 2)
    gamma, beta = params(gen, N, dtype, "same")
    _, gamma = shifted(gamma, by)
    ybuf, y = shifted(torch.zeros_like(x), by + 3, 7.0)
    got, mean, rstd = fp.layernorm_forward(x, gamma, beta, 1e-5, out=(y, None, None))
    ry, _, _, bound = layernorm(x, gamma, beta, 1e-5)
    assert_within(got, ry, bound + half_ulp(dtype) * (ry.abs() + bound), "y")
    assert (ybuf[:by + 3] == 7.0).all() and (ybuf[by + 3 + M * N:] == 7.0).all()
    for kind in ("ln", "rms"):
        mean, rstd = statistics(x, kind)
        dbuf, dx = shifted(torch.zeros_like(x), by, 7.0)
        out = (dx, None, None) if kind == "ln" else (dx, None)
        check_backward(kind, dy, x, mean, rstd, gamma, dres, run_backward(kind, dy, x, mean, rstd, gamma, dres, out=out))
        assert (dbuf[:by] == 7.0).all() and (dbuf[by + M * N:] == 7.0).all()


@pytest.mark.parametrize("M,N", [(40, 2048), (1500, 2048), (1500, 77)])
def test_two_backward_passes_at_once(M, N):
    """On two streams at the same time, each with its own workspace, and dx
    written over x as well as over dy."""
    gen = gen_of(21)
    x, dy = draw(gen, M, N, torch.bfloat16), draw(gen, M, N, torch.bfloat16, std=0.01)
    gamma, _ = params(gen, N, torch.bfloat16, "same")
    mean, rstd = statistics(x, "ln")
    want = fp.layernorm_backward(dy, x, mean, rstd, gamma)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(fp.layernorm_backward(dy, x, mean, rstd, gamma))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
    over = x.clone()
    got = fp.layernorm_backward(dy, over, mean, rstd, gamma, out=(over, None, None))
    assert torch.equal(got[0], want[0])
    check_backward("ln", dy, x, mean, rstd, gamma, None, got)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N", [(8, 1280), (1500, 100), (1500, 1280), (1500, 1277), (700, 5000), (9, 16384), (8, 20001)])
def test_layernorm_forward_far_from_zero(M, N, dtype):
    """Rows whose mean is far larger than their spread, constant rows and a
    zero row: y is right to the spread, not to the mean."""
    gen = gen_of(3)
    x = draw(gen, M, N, dtype, mean=200.0, std=2.0)
    x[5] = 3.0
    x[6] = 0.0
    y, mean, rstd = fp.layernorm_forward(x, eps=1e-5)
    ry, rmean, rrstd, bound = layernorm(x, None, None, 1e-5)
    # each centred value is exact up to a rounding of the mean-free value plus
    # the rounding of x - m, half an ulp of 256 at most: 2^-17
    assert_within(y, ry, bound + half_ulp(dtype) * ry.abs() + 2.0 ** -17 * rrstd[:, None], "y")
    assert (y[5] == 0).all() and (y[6] == 0).all()


def test_layernorm_nan_stays_in_its_row():
    x = draw(gen_of(4), 20, 640, torch.bfloat16)
    clean, _, _ = fp.layernorm_forward(x)
    x[7, 3] = float("nan")
    x[9, 5] = float("inf")
    y, _, _ = fp.layernorm_forward(x)
    keep = [i for i in range(20) if i not in (7, 9)]
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[7]).all() and torch.isnan(y[9]).any()


def run_backward(kind, dy, x, mean, rstd, gamma, dres, **kw):
    if kind == "ln":
        return fp.layernorm_backward(dy, x, mean, rstd, gamma, dres, **kw)
    return (*fp.rmsnorm_backward(dy, x, rstd, gamma, dres, **kw), None)


def statistics(x, kind):
    x64 = x.double()
    mean = x64.mean(1) if kind == "ln" else torch.zeros(x.shape[0], dtype=torch.float64, device=x.device)
    rstd = torch.rsqrt((x64 - mean[:, None]).square().mean(1) + 1e-5)
    return (mean.float() if kind == "ln" else None), rstd.float()


def check_backward(kind, dy, x, mean, rstd, gamma, dres, got, old=None):
    dtype = x.dtype
    (rdx, bdx), (rdg, bdg), (rdb, bdb) = norm_backward(dy, x, mean, rstd, gamma, dres)
    dx, dgamma, dbeta = got
    assert_within(dx, rdx, bdx + half_ulp(dtype) * (rdx.abs() + bdx), "dx")
    if old is not None:
        rdg, bdg = rdg + old.double(), bdg + 2 * U * (old.double().abs() + rdg.abs())
        rdb, bdb = rdb + old.double(), bdb + 2 * U * (old.double().abs() + rdb.abs())
    assert_within(dgamma, rdg, bdg + 8 * U * rdg.abs(), "dgamma")
    if kind == "ln":
        assert_within(dbeta, rdb, bdb + U * rdb.abs(), "dbeta")


@pytest.mark.parametrize("kind", ["ln", "rms"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N,pad", SIZES)
def test_norm_backward(M, N, pad, dtype, kind):
    gen = gen_of(M * 1000 + N + 1)
    x = draw(gen, M, N, dtype, pad, mean=0.5)
    dy = draw(gen, M, N, dtype, pad, std=0.01)
    dres = draw(gen, M, N, dtype, pad, std=0.01) if (M + N) % 2 else None
    gamma, _ = params(gen, N, dtype, ["same", "fp32", "none"][(M + N) % 3])
    mean, rstd = statistics(x, kind)
    buf, out = padded(M, N, N + pad, dtype, 7.0)
    got = run_backward(kind, dy, x, mean, rstd, gamma, dres, out=(out, None, None) if kind == "ln" else (out, None))
    check_backward(kind, dy, x, mean, rstd, gamma, dres, got)
    assert (buf[:, N:] == 7.0).all()
    # dx written over dy; the sums added into what is there
    old = torch.randn(N, generator=gen, device="cuda")
    d2 = torch.empty_strided(dy.shape, dy.stride(), dtype=dtype, device="cuda")
    d2.copy_(dy)
    o2 = (d2, old.clone(), old.clone()) if kind == "ln" else (d2, old.clone())
    got2 = run_backward(kind, d2, x, mean, rstd, gamma, dres, out=o2, accumulate=True)
    assert torch.equal(got2[0], got[0])
    check_backward(kind, dy, x, mean, rstd, gamma, dres, got2, old)
    # without the parameters' gradients
    got3 = run_backward(kind, dy, x, mean, rstd, gamma, dres, params=False)
    assert got3[1] is None and got3[2] is None and torch.equal(got3[0], got[0])


@pytest.mark.parametrize("kind", ["ln", "rms"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_backward_full_size(kind, dtype):
    gen = gen_of(11)
    x, dy = draw(gen, 16384, 2048, dtype), draw(gen, 16384, 2048, dtype, std=1e-3)
    dres = draw(gen, 16384, 2048, dtype, std=1e-3)
    gamma, _ = params(gen, 2048, dtype, "same")
    mean, rstd = statistics(x, kind)
    got = run_backward(kind, dy, x, mean, rstd, gamma, dres)
    check_backward(kind, dy, x, mean, rstd, gamma, dres, got)
    again = run_backward(kind, dy, x, mean, rstd, gamma, dres)
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, again))  # the same bits


@pytest.mark.parametrize("kind", ["ln", "rms"])
def test_norm_backward_against_differences(kind):
    """dx, dgamma and dbeta in FP32 against central differences of the 64-bit
    forward form.  A difference over 2h is off by h^2 / 6 times the third
    derivative and by 64-bit cancellation: under 1e-7 here."""
    gen = gen_of(5)
    M, N = 3, 10
    x = torch.randn(M, N, generator=gen, device="cuda")
    dy = torch.randn(M, N, generator=gen, device="cuda")
    gamma = 1 + 0.2 * torch.randn(N, generator=gen, device="cuda")
    beta = torch.randn(N, generator=gen, device="cuda")
    mean, rstd = statistics(x, kind)
    dx, dg, db = run_backward(kind, dy, x, mean, rstd, gamma, None)

    def loss(x64, g64, b64):
        d = x64 - x64.mean(1, keepdim=True) if kind == "ln" else x64
        y = d / torch.sqrt(d.square().mean(1, keepdim=True) + 1e-5) * g64 + (b64 if kind == "ln" else 0.0)
        return (y * dy.double()).sum()
    args = [x.double(), gamma.double(), beta.double()]
    h = 1e-5
    for which, got in ((0, dx), (1, dg), (2, db)):
        if got is None:
            continue
        flat = args[which].reshape(-1)
        for i in range(flat.numel()):
            keep = flat[i].item()
            flat[i] = keep + h
            up = loss(*args)
            flat[i] = keep - h
            down = loss(*args)
            flat[i] = keep
            assert abs((up - down).item() / (2 * h) - got.reshape(-1)[i].item()) < 2e-5 * (1 + abs(got).max().item())


@pytest.mark.parametrize("exact", [False, True])
def test_rmsnorm_backward_takes_the_producers_rstd(exact):
    gen = gen_of(6)
    x, dy = draw(gen, 256, 640, torch.bfloat16), draw(gen, 256, 640, torch.bfloat16, std=0.01)
    gamma, _ = params(gen, 640, torch.bfloat16, "same")
    _, _, _, _, _, rstd = fp.rmsnorm_quantize(x, gamma, 1e-6, exact=exact)
    assert rstd.dtype == (torch.float64 if exact else torch.float32)
    got = fp.rmsnorm_backward(dy, x, rstd, gamma)
    check_backward("rms", dy, x, None, rstd, gamma, None, (*got, None))


def test_statistics_are_optional():
    """The C call without mean and rstd to write."""
    x = draw(gen_of(30), 70, 640, torch.bfloat16)
    want, _, _ = fp.layernorm_forward(x)
    y = torch.empty_like(x)
    st = fp.lib().fp8bq_layernorm_forward(x.data_ptr(), 70, 640, 640, None, None, 1e-5, y.data_ptr(), 640, None, None, 1, 1,
                                          torch.cuda.current_stream().cuda_stream)
    assert st == 0 and torch.equal(y, want)


def test_more_values_than_32_bits_count():
    """2.25e9 BF16 values (4.5 GB a tensor): the last rows."""
    M, N = 1100000, 2048
    x = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    tail = draw(gen_of(31), 300, N, torch.bfloat16)
    x[-300:] = tail
    y, mean, rstd = fp.layernorm_forward(x)
    ry, _, _, bound = layernorm(tail, None, None, 1e-5)
    assert_within(y[-300:], ry, bound + half_ulp(torch.bfloat16) * (ry.abs() + bound), "y")
    del y
    dx, dgamma, dbeta = fp.layernorm_backward(x, x, mean, rstd)  # zero rows add nothing
    (rdx, bdx), (rdg, bdg), (rdb, bdb) = norm_backward(tail, tail, mean[-300:], rstd[-300:], None, None)
    assert_within(dx[-300:], rdx, bdx + half_ulp(torch.bfloat16) * (rdx.abs() + bdx), "dx")
    assert_within(dgamma, rdg, bdg + 8 * U * rdg.abs(), "dgamma")
    assert_within(dbeta, rdb, bdb + U * rdb.abs(), "dbeta")


def test_norm_no_rows():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    stat = torch.empty(0, device="cuda")
    y, mean, rstd = fp.layernorm_forward(x)
    assert y.shape == (0, 64) and mean.shape == (0,)
    dx, dg, db = fp.layernorm_backward(x, x, stat, stat)
    assert dx.shape == (0, 64) and (dg == 0).all() and (db == 0).all()
    old = torch.ones(64, device="cuda")
    _, dg, db = fp.layernorm_backward(x, x, stat, stat, out=(None, old, old.clone()), accumulate=True)
    assert (dg == 1).all() and (db == 1).all()
    e = torch.empty(5, 0, device="cuda")
    assert fp.layernorm_forward(e)[0].shape == (5, 0)


def test_norm_captured_and_on_another_stream():
    """The two passes captured into a graph and replayed on new inputs, and on
    a side stream, give the eager calls' bits."""
    gen = gen_of(7)
    x, dy = draw(gen, 300, 2048, torch.bfloat16), draw(gen, 300, 2048, torch.bfloat16, std=0.01)
    gamma, beta = params(gen, 2048, torch.bfloat16, "same")

    def both():
        y, mean, rstd = fp.layernorm_forward(x, gamma, beta)
        return (y, mean, rstd, *fp.layernorm_backward(dy, x, mean, rstd, gamma))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = both()
    torch.cuda.current_stream().wait_stream(side)
    want = both()
    assert all(torch.equal(a, b) for a, b in zip(on_side, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for seed in (8, 9):
        x.copy_(draw(gen_of(seed), 300, 2048, torch.bfloat16))
        graph.replay()
        want = both()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_norm_refusals():
    x = torch.zeros(4, 64, device="cuda")
    s = torch.zeros(4, device="cuda")
    for bad in (lambda: fp.layernorm_forward(x, gamma=torch.zeros(63, device="cuda")),
                lambda: fp.layernorm_forward(x, gamma=torch.zeros(64, device="cuda", dtype=torch.bfloat16)),
                lambda: fp.layernorm_forward(x, gamma=torch.zeros(64)),
                lambda: fp.layernorm_backward(x.half(), x, s, s),
                lambda: fp.layernorm_backward(x[:, :63], x, s, s),
                lambda: fp.layernorm_backward(x, x, s[:3], s),
                lambda: fp.layernorm_backward(x, x, None, s),
                lambda: fp.layernorm_backward(x, x, s, s, accumulate=True),
                lambda: fp.rmsnorm_backward(x, x, s.half()),
                lambda: fp.rmsnorm_backward(x, x, s, out=(x.half(), None))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(fp.Fp8bqError) as e:
        fp.layernorm_forward(x[:1].expand(4, 64))  # rows that share memory
    assert e.value.status == -2
    with pytest.raises(fp.Fp8bqError) as e:
        fp.layernorm_forward(x, eps=-1.0)
    assert e.value.status == -1
