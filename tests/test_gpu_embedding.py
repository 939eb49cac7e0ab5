"""GPU tests of the embedding lookup and its gradient against the 64-bit
forms: one token to many, ids all alike, ids outside the table, padding,
odd and strided rows, every pair of types."""
import pytest
import torch

import blockwise_fp8_linear_fp8bq_b200 as fp
from row_ref import U, assert_within, embedding_backward, half_ulp, padded

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def gen_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ids_of(gen, T, V, kind, wide=True):
    if kind == "uniform":
        ids = torch.randint(0, V, (T,), generator=gen, device="cuda")
    elif kind == "alike":
        ids = torch.full((T,), V - 1, dtype=torch.int64, device="cuda")
    else:  # as texts have them: about 1 / rank
        u = torch.rand(T, generator=gen, device="cuda", dtype=torch.float64)
        ids = ((V + 1.0) ** u).long().sub_(1).clamp_(0, V - 1)
    return ids if wide else ids.int()


@pytest.mark.parametrize("w_dtype", DTYPES)
@pytest.mark.parametrize("y_dtype", DTYPES)
@pytest.mark.parametrize("T,V,D,pad", [(1, 1, 1, 0), (7, 1031, 64, 0), (33, 500, 640, 8), (200, 151936, 77, 3),
                                       (509, 1031, 2048, 0), (3, 40, 8192, 0)])
def test_lookup(T, V, D, pad, w_dtype, y_dtype):
    gen = gen_of(T + D)
    _, w = padded(V, D, D + pad, w_dtype, float("nan"))
    w.copy_(torch.randn(V, D, generator=gen, device="cuda") * 0.02)
    ids = ids_of(gen, T, V, "uniform", wide=T % 2 == 1)
    scale = float(D) ** 0.5
    buf, out = padded(T, D, D + pad, y_dtype, 7.0)
    y = fp.embedding_forward(w, ids, scale, out=out, dtype=y_dtype)
    ref = w.double()[ids.long()] * scale
    # the scale's and the product's roundings, then the type's
    assert_within(y, ref, (2 * U + half_ulp(y_dtype) * (1 + 2 * U)) * ref.abs(), "y")
    assert (buf[:, D:] == 7.0).all()
    if w_dtype == y_dtype:
        assert torch.equal(fp.embedding_forward(w, ids), w[ids.long()])  # scale 1: the table's own bits
    fp.check()


def test_lookup_shapes_and_empty():
    w = torch.randn(10, 16, device="cuda")
    ids = torch.arange(6, device="cuda").view(2, 3)
    assert torch.equal(fp.embedding_forward(w, ids), w[ids])
    assert fp.embedding_forward(w, ids[:0]).shape == (0, 3, 16)
    assert fp.embedding_forward(w[:, :0], ids).shape == (2, 3, 0)


@pytest.mark.parametrize("bad", [-1, 10, 2 ** 40, -2 ** 62])
def test_ids_outside_the_table(bad):
    w = torch.randn(10, 16, device="cuda")
    ids = torch.tensor([3, bad, 9], device="cuda")
    y = fp.embedding_forward(w, ids)
    assert torch.equal(y[0], w[3]) and (y[1] == 0).all() and torch.equal(y[2], w[9])
    with pytest.raises(fp.Fp8bqError) as e:
        fp.check()
    assert e.value.status == -7
    fp.check()  # reported once
    dy = torch.randn(3, 16, device="cuda")
    dw = fp.embedding_backward(dy, ids, 10)
    with pytest.raises(fp.Fp8bqError) as e:
        fp.check()
    assert e.value.status == -7
    assert torch.equal(dw[3], dy[0]) and torch.equal(dw[9], dy[2])
    assert (dw[[0, 1, 2, 4, 5, 6, 7, 8]] == 0).all()


@pytest.mark.parametrize("dtype,grad", [(t, g) for t in DTYPES for g in {t, torch.float32}])
@pytest.mark.parametrize("T,V,D,pad,kind", [
    (1, 1, 1, 0, "alike"), (2, 3, 64, 0, "alike"), (9, 1031, 640, 8, "uniform"), (100, 7, 77, 1, "uniform"),
    (509, 1031, 640, 0, "text"), (4096, 20, 8, 0, "text"), (4097, 600, 130, 0, "text"), (5000, 2, 48, 0, "alike"),
    (20000, 151936, 64, 0, "text"), (40000, 100000, 16, 0, "text"), (40001, 3, 24, 8, "alike"),
    (300, 50, 4104, 0, "text"), (33, 500, 8192, 0, "uniform"),
    (1500, 50, 4104, 0, "text"), (3000, 600000, 8, 0, "uniform"), (6000, 600001, 6, 2, "text"),
    (1024, 70, 96, 0, "text"), (1025, 70, 96, 0, "text"), (9000, 33, 2050, 0, "text")])
def test_gradient(T, V, D, pad, kind, dtype, grad):
    gen = gen_of(T + V + D)
    ids = ids_of(gen, T, V, kind, wide=T % 2 == 0)
    _, dy = padded(T, D, D + pad, dtype, float("nan"))
    dy.copy_(torch.randn(T, D, generator=gen, device="cuda") * 0.01)
    buf, out = padded(V, D, D + pad, grad, 7.0)
    scale = 1.0 if V % 2 else float(D) ** 0.5
    padding = None if T % 3 else 0
    dw = fp.embedding_backward(dy, ids, V, scale, padding, out=out)
    ref, bound = embedding_backward(dy, ids, V, scale, padding)
    assert_within(dw, ref, bound + half_ulp(grad) * (ref.abs() + bound), "dw")
    assert (buf[:, D:] == 7.0).all()
    named = torch.zeros(V, dtype=torch.bool, device="cuda")
    named[ids.long()] = True
    assert (dw[~named] == 0).all()
    # the same bits again
    assert torch.equal(fp.embedding_backward(dy, ids, V, scale, padding, dtype=grad), dw)
    # added into a gradient: the rows no id names are left as they are
    buf2, old = padded(V, D, D + pad, grad, 7.0)
    old.copy_(torch.randn(V, D, generator=gen, device="cuda") * 0.01)
    before = old.clone()
    got = fp.embedding_backward(dy, ids, V, scale, padding, out=old, accumulate=True)
    ref, bound = embedding_backward(dy, ids, V, scale, padding, before)
    assert_within(got, ref, bound + half_ulp(grad) * (ref.abs() + bound), "dw added")
    assert torch.equal(got[~named], before[~named]) and (buf2[:, D:] == 7.0).all()
    fp.check()


@pytest.mark.parametrize("T", [300, 2000, 9000])
@pytest.mark.parametrize("wide", [False, True])
def test_padding_and_ids_outside_among_many(T, wide):
    """Few tokens, the sort: ids below 0, at the
    vocabulary's end and beyond add nothing and are reported, the padding id
    adds nothing and is not; a padding id outside the table is none."""
    gen = gen_of(T)
    V, D = 100, 72
    ids = torch.randint(0, V, (T,), generator=gen, device="cuda", dtype=torch.int64 if wide else torch.int32)
    dy = torch.randn(T, D, generator=gen, device="cuda")
    dw = fp.embedding_backward(dy, ids, V, padding_id=5)
    ref, bound = embedding_backward(dy, ids, V, 1.0, 5)
    assert_within(dw, ref, bound + U * ref.abs(), "dw")
    assert (dw[5] == 0).all()
    fp.check()
    ids[::7], ids[3::7], ids[5::7] = -1, V, V + 1000
    for padding in (5, V, -3):
        dw = fp.embedding_backward(dy, ids, V, padding_id=padding)
        ref, bound = embedding_backward(dy, ids, V, 1.0, padding if padding == 5 else None)
        assert_within(dw, ref, bound + U * ref.abs(), "dw")
        with pytest.raises(fp.Fp8bqError) as e:
            fp.check()
        assert e.value.status == -7


def test_more_values_than_32_bits_count():
    """A BF16 table of 2.5e9 values (5 GB): rows at its end, and the dense
    gradient's zeros up to there."""
    V, D = 151936, 16384
    w = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([V - 1, 0, 131072, V - 2, V - 1], device="cuda")
    for k, i in enumerate(ids.tolist()):
        w[i] = k + 1.0
    assert torch.equal(fp.embedding_forward(w, ids), w[ids])
    dy = torch.ones(5, D, dtype=torch.bfloat16, device="cuda")
    w.fill_(3.0)
    dw = fp.embedding_backward(dy, ids, V, out=w)
    sums = dw[:, 0].float() + dw[:, D - 1].float()
    want = torch.zeros(V, device="cuda").index_add_(0, ids, torch.full((5,), 2.0, device="cuda"))
    assert torch.equal(sums, want)
    assert sum(dw[v0:v0 + 16384].count_nonzero().item() for v0 in range(0, V, 16384)) == 4 * D


def test_gradient_full_size():
    """A training step's table gradient: 16384 tokens, vocabulary 151936."""
    gen = gen_of(1)
    ids = ids_of(gen, 16384, 151936, "text")
    dy = (torch.randn(16384, 2048, generator=gen, device="cuda") * 1e-3).bfloat16()
    dw = fp.embedding_backward(dy, ids, 151936)
    rows = torch.unique(ids)
    back = torch.searchsorted(rows, ids)
    ref, bound = embedding_backward(dy, back, rows.numel(), 1.0, None)
    assert_within(dw[rows], ref, bound + half_ulp(torch.float32) * ref.abs(), "dw")
    dw[rows] = 0
    assert not dw.any()


@pytest.mark.parametrize("by", [1, 2, 5])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V,D", [(50, 11, 30), (1500, 300, 64), (5000, 40, 129)])
def test_rows_that_start_anywhere(T, V, D, dtype, by):
    """Tables, rows and gradients whose first value is at no multiple of 16 bytes."""
    gen = gen_of(T + by)
    place = lambda n: torch.full((n + 20,), float("nan"), dtype=dtype, device="cuda")
    w = place(V * D)[by:by + V * D].view(V, D)
    w.copy_(torch.randn(V, D, generator=gen, device="cuda"))
    dy = place(T * D)[by + 1:by + 1 + T * D].view(T, D)
    dy.copy_(torch.randn(T, D, generator=gen, device="cuda") * 0.01)
    ids = ids_of(gen, T, V, "text")
    ybuf = torch.full((T * D + 20,), 7.0, dtype=dtype, device="cuda")
    y = fp.embedding_forward(w, ids, out=ybuf[by:by + T * D].view(T, D))
    assert torch.equal(y, w[ids]) and (ybuf[:by] == 7.0).all() and (ybuf[by + T * D:] == 7.0).all()
    for grad in {dtype, torch.float32}:
        buf = torch.full((V * D + 20,), 7.0, dtype=grad, device="cuda")
        dw = fp.embedding_backward(dy, ids, V, out=buf[by:by + V * D].view(V, D))
        ref, bound = embedding_backward(dy, ids, V, 1.0, None)
        assert_within(dw, ref, bound + half_ulp(grad) * (ref.abs() + bound), "dw")
        assert (buf[:by] == 7.0).all() and (buf[by + V * D:] == 7.0).all()


def test_gradient_of_no_tokens():
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    dy = torch.empty(0, 64, device="cuda")
    out = torch.full((50, 64), 3.0, device="cuda")
    assert (fp.embedding_backward(dy, ids, 50, out=out, accumulate=True) == 3.0).all()
    assert (fp.embedding_backward(dy, ids, 50, out=out) == 0.0).all()


def test_gradient_against_differences():
    """The loss sum(c * scale * W[ids]) is linear in W, so a difference equals
    the gradient up to 64-bit rounding."""
    gen = gen_of(2)
    w = torch.randn(5, 4, generator=gen, device="cuda", dtype=torch.float64)
    ids = torch.tensor([4, 1, 1, 0, 4, 4], device="cuda")
    c = torch.randn(6, 4, generator=gen, device="cuda")
    dw = fp.embedding_backward(c, ids, 5, scale=2.0)
    loss = lambda t: (c.double() * 2.0 * t[ids]).sum().item()
    for v in range(5):
        for d in range(4):
            up, down = w.clone(), w.clone()
            up[v, d] += 0.5
            down[v, d] -= 0.5
            assert abs(loss(up) - loss(down) - dw[v, d].item()) < 1e-5


def test_captured_and_concurrent():
    """Captured and replayed with new ids and gradients, and two calls on two
    streams at once, give the eager calls' bits."""
    gen = gen_of(3)
    ids = ids_of(gen, 6000, 1031, "text")
    dy = (torch.randn(6000, 640, generator=gen, device="cuda") * 0.01).bfloat16()
    w = torch.randn(1031, 640, generator=gen, device="cuda").bfloat16()
    run = lambda: (fp.embedding_forward(w, ids, 2.0), fp.embedding_backward(dy, ids, 1031, 2.0, 0))
    want = run()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(run())
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for seed in (4, 5):
        ids.copy_(ids_of(gen_of(seed), 6000, 1031, "text"))
        graph.replay()
        want = run()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    fp.check()


def test_refusals():
    w = torch.zeros(10, 16, device="cuda")
    ids = torch.zeros(3, dtype=torch.int64, device="cuda")
    dy = torch.zeros(3, 16, device="cuda")
    for bad in (lambda: fp.embedding_forward(w.double(), ids),
                lambda: fp.embedding_forward(w, ids.float()),
                lambda: fp.embedding_forward(w, ids.cpu()),
                lambda: fp.embedding_forward(w, torch.zeros(6, dtype=torch.int64, device="cuda")[::2]),
                lambda: fp.embedding_forward(w, ids, out=torch.zeros(2, 16, device="cuda")),
                lambda: fp.embedding_backward(dy, ids[:2], 10),
                lambda: fp.embedding_backward(dy, ids, 10, accumulate=True),
                lambda: fp.embedding_backward(dy, ids, 10, out=torch.zeros(9, 16, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: fp.embedding_forward(w, ids, scale=float("nan")),
                lambda: fp.embedding_backward(dy, ids, 10, dtype=torch.bfloat16)):
        with pytest.raises(fp.Fp8bqError) as e:
            bad()
        assert e.value.status == -1
