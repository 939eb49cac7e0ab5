"""GPU tests of the global gradient norm and clipping against the 64-bit
forms: many tensors of every type and alignment, values whose squares leave
FP32's range, infinities and NaN."""
import math

import pytest
import torch

import blockwise_fp8_linear_fp8bq_b200 as fp
from row_ref import U, assert_within, half_ulp

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
# FP32 sums of eight squares (8 roundings, halved by the root), then 64 bits and one rounding
NORM = 6 * U


def ref_norm(grads):
    return math.sqrt(math.fsum(g.double().square().sum().item() for g in grads))


def check(grads, norm, outs, most):
    n = ref_norm(grads)
    assert abs(norm.item() - n) <= NORM * n
    f = min(1.0, most / (n + 1e-6))
    for g, o in zip(grads, outs):
        ref = g.double() * f
        # the factor's error, its rounding and the product's, then the type's
        assert_within(o, ref, (NORM + 2 * U + half_ulp(o.dtype) * (1 + 4 * U)) * ref.abs(), "clipped")


def draw(gen, n, dtype, std=1e-2, offset=0):
    return (torch.randn(n + offset, generator=gen, device="cuda") * std).to(dtype)[offset:]


def gen_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("most", [0.05, 1e9])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sizes", [(1,), (7, 0, 300), (16384, 16385, 1, 16383), (509, 1283 * 640, 3, 77777),
                                   tuple(range(1, 300))])
def test_clip(sizes, dtype, most):
    gen = gen_of(len(sizes))
    grads = [draw(gen, n, dtype) for n in sizes]
    norm = fp.grad_norm(grads)
    outs = [torch.empty_like(g) for g in grads]
    got = fp.clip_grads(grads, most, out=outs)
    assert torch.equal(norm, got)
    check(grads, norm, outs, most)
    kept = [g.clone() for g in grads]
    got = fp.clip_grads(grads, most)  # in place: the same bits
    assert torch.equal(got, norm) and all(torch.equal(a, b) for a, b in zip(grads, outs))
    if most > 1e6:
        assert all(torch.equal(a, b) for a, b in zip(grads, kept))


@pytest.mark.parametrize("out", DTYPES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_clip_mixed_types_and_alignments(dtype, out):
    gen = gen_of(5)
    grads = [draw(gen, 20000 + k, DTYPES[k % 3] if k % 2 else dtype, offset=k) for k in range(6)]
    outs = [torch.full((g.numel() + 9,), 7.0, dtype=out, device="cuda")[k % 2:][:g.numel()] for k, g in enumerate(grads)]
    norm = fp.clip_grads(grads, 0.5, out=outs)
    check(grads, norm, outs, 0.5)
    for k, (g, o) in enumerate(zip(grads, outs)):
        whole = o._base if o._base is not None else o
        assert (whole[k % 2 + g.numel():] == 7.0).all()


def test_weight_shapes():
    """2-D gradients, and a transposed one (its elements fill one span)."""
    gen = gen_of(6)
    a = torch.randn(64, 33, generator=gen, device="cuda")
    b = torch.randn(48, 20, generator=gen, device="cuda").t()
    kept = [a.clone(), b.clone()]
    norm = fp.clip_grads([a, b], 1.0)
    check(kept, norm, [a, b], 1.0)


@pytest.mark.parametrize("std", [1e-30, 1e-42, 1e30])
def test_squares_outside_fp32(std):
    g = (torch.randn(5000, generator=gen_of(7), device="cuda", dtype=torch.float64) * std).float()
    norm = fp.grad_norm([g])
    n = ref_norm([g])
    assert n > 0 and abs(norm.item() - n) <= NORM * n + 2.0 ** -149
    assert fp.grad_norm([torch.zeros(5000, device="cuda")]).item() == 0.0


def test_one_large_among_tiny():
    g = torch.full((100000,), 1e-25, device="cuda")
    g[77777] = 1e25
    assert abs(fp.grad_norm([g]).item() - 1e25) <= 4 * U * 1e25


def test_infinities_and_nan():
    a, b = torch.ones(3000, device="cuda"), torch.ones(40000, device="cuda")
    b[123] = float("inf")
    outs = [torch.empty_like(a), torch.empty_like(b)]
    assert fp.clip_grads([a, b], 1.0, out=outs).item() == float("inf")
    assert (outs[0] == 0).all() and torch.isnan(outs[1][123]) and outs[1].isnan().sum() == 1
    b[123] = float("nan")
    assert math.isnan(fp.clip_grads([a, b], 1.0, out=outs).item())
    assert outs[0].isnan().all() and outs[1].isnan().all()


def test_infinite_limit():
    a, b = torch.ones(3000, device="cuda"), torch.ones(40000, device="cuda")
    b[7] = float("inf")
    out = [torch.empty_like(a), torch.empty_like(b)]
    assert fp.clip_grads([a, b], float("inf"), out=out).item() == float("inf")
    assert torch.equal(out[0], a) and torch.equal(out[1], b)
    a[3] = float("nan")
    fp.clip_grads([a, b], float("inf"), out=out)
    assert out[0].isnan().all() and out[1].isnan().all()


@pytest.mark.parametrize("count,n", [(200, 20000), (129, 1), (128, 5000)])
def test_more_tensors_than_a_launch_takes(count, n):
    gen = gen_of(count)
    grads = [draw(gen, n + k % 7, DTYPES[k % 3]) for k in range(count)]
    outs = [torch.empty_like(g) for g in grads]
    norm = fp.clip_grads(grads, 0.3, out=outs)
    check(grads, norm, outs, 0.3)


def test_zero_limit_and_zero_gradients():
    a = torch.ones(1000, device="cuda")
    out = [torch.empty_like(a)]
    fp.clip_grads([a], 0.0, out=out)
    assert (out[0] == 0).all()
    z = torch.zeros(1000, device="cuda")
    assert fp.clip_grads([z], 1.0).item() == 0.0 and not z.any()


def test_full_size_and_repeatable():
    gen = gen_of(8)
    grads = [torch.randn(s, generator=gen, device="cuda") * 1e-3
             for s in ((4096, 2048), (2048, 2048), (12288, 2048), (2048, 6144), (2048,), (2048,))]
    outs = [torch.empty_like(g) for g in grads]
    norm = fp.clip_grads(grads, 1.0, out=outs)
    check(grads, norm, outs, 1.0)
    assert torch.equal(fp.grad_norm(grads), norm)


def test_captured_and_concurrent():
    gen = gen_of(9)
    grads = [draw(gen, n, torch.float32) for n in (100000, 77, 20001)]
    outs = [torch.empty_like(g) for g in grads]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        n_side = fp.grad_norm(grads)
    n_main = fp.clip_grads(grads, 0.1, out=outs)
    torch.cuda.synchronize()
    assert torch.equal(n_side, n_main)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = fp.clip_grads(grads, 0.1, out=outs)
    for seed in (10, 11):
        for k, g in enumerate(grads):
            g.copy_(draw(gen_of(seed + k), g.numel(), torch.float32))
        graph.replay()
        check(grads, norm, outs, 0.1)


def test_refusals():
    a = torch.ones(10, 10, device="cuda")
    for bad in (lambda: fp.clip_grads([a[:, :5]], 1.0), lambda: fp.clip_grads([a.double()], 1.0),
                lambda: fp.clip_grads([a], 1.0, out=[]), lambda: fp.clip_grads([a], 1.0, out=[a.t()]),
                lambda: fp.clip_grads([a], 1.0, out=[a[:5]])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: fp.clip_grads([a, a], 1.0), lambda: fp.clip_grads([a[:6], a[5:]], 1.0),
                lambda: fp.clip_grads([a], -1.0), lambda: fp.clip_grads([a], float("nan"))):
        with pytest.raises(fp.Fp8bqError) as e:
            bad()
        assert e.value.status == -1
    assert (a == 1).all()
