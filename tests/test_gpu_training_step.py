"""The row operators and the blockwise-FP8 linears run together, as a training
step uses them: lookup, LayerNorm, an FP8 linear, RMSNorm's producer and a
second FP8 linear, their backward passes with the residual stream's gradient,
the table's gradient, FP32 master gradients, and the clipping of all of them.
Every row operator is held to its 64-bit form on the inputs it was given; the
whole step runs twice, eagerly and from a captured graph, to the same bits."""
import math

import pytest
import torch

import blockwise_fp8_linear_fp8bq_b200 as fp
from blockwise_fp8_linear_fp8bq_b200 import synth
from row_ref import U, assert_within, embedding_backward, half_ulp, layernorm, norm_backward

pytestmark = pytest.mark.gpu

T, V, D = 512, 1031, 640
FMT = fp.SCALE_UE8M0
BF = torch.bfloat16


def step(s):
    """One step's every intermediate, and the clipped gradients."""
    r = {}
    x0 = fp.embedding_forward(s["table"], s["ids"], scale=D ** 0.5)
    h1, mean, rstd1 = fp.layernorm_forward(x0, s["g1"], s["b1"])
    q1, s1, qt1, st1 = fp.quantize_act_dual(h1, FMT)
    qw1, sw1 = fp.quantize_weight(s["w1"], FMT)
    y1 = fp.gemm(fp.row_operand(q1, s1, FMT), fp.block_operand(qw1, sw1, FMT))
    x1 = x0 + y1
    q2, s2, qt2, st2, _, rstd2 = fp.rmsnorm_quantize(x1, s["g2"], 1e-6, FMT)
    qw2, sw2 = fp.quantize_weight(s["w2"], FMT)
    y2 = fp.gemm(fp.row_operand(q2, s2, FMT), fp.block_operand(qw2, sw2, FMT))
    dy2 = (y2.float() - s["target"]).to(BF)  # the gradient of half the squared distance
    dq, ds, dqt, dst = fp.quantize_act_dual(dy2, FMT)
    dw2, dw1 = torch.zeros_like(s["w2"], dtype=torch.float32), torch.zeros_like(s["w1"], dtype=torch.float32)
    fp.gemm(fp.row_operand(dqt, dst, FMT), fp.row_operand(qt2, st2, FMT), out=dw2, accumulate=True)
    dh2 = fp.gemm(fp.row_operand(dq, ds, FMT), fp.block_operand(qw2, sw2, FMT, transposed=True))
    dx1, dg2 = fp.rmsnorm_backward(dh2, x1, rstd2, s["g2"], dres=dy2)
    dq, ds, dqt, dst = fp.quantize_act_dual(dx1, FMT)
    fp.gemm(fp.row_operand(dqt, dst, FMT), fp.row_operand(qt1, st1, FMT), out=dw1, accumulate=True)
    dh1 = fp.gemm(fp.row_operand(dq, ds, FMT), fp.block_operand(qw1, sw1, FMT, transposed=True))
    dx0, dg1, db1 = fp.layernorm_backward(dh1, x0, mean, rstd1, s["g1"], dres=dx1)
    dtable = fp.embedding_backward(dx0, s["ids"], V, scale=D ** 0.5, padding_id=0)
    grads = [dtable, dg1, db1, dw1, dg2, dw2]
    clipped = [torch.empty_like(g) for g in grads]
    norm = fp.clip_grads(grads, 1.0, out=clipped)
    r.update(x0=x0, h1=h1, mean=mean, rstd1=rstd1, x1=x1, rstd2=rstd2, dh2=dh2, dy2=dy2, dx1=dx1, dg2=dg2, dh1=dh1, dx0=dx0,
             dg1=dg1, db1=db1, dtable=dtable, grads=grads, clipped=clipped, norm=norm)
    return r


def test_training_step():
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    s = dict(table=synth.normal_bf16((V, D), 0.02, 1, "cuda"), w1=synth.weights_bf16(D, D, 2, "cuda"),
             w2=synth.weights_bf16(D, D, 3, "cuda"), g1=(1 + 0.1 * synth.normal_bf16((D,), 1.0, 4, "cuda").float()).to(BF),
             b1=synth.normal_bf16((D,), 0.1, 5, "cuda"), g2=(1 + 0.1 * synth.normal_bf16((D,), 1.0, 6, "cuda").float()).to(BF),
             ids=torch.randint(0, V, (T,), generator=gen, device="cuda"),
             target=torch.randn(T, D, generator=gen, device="cuda"))
    r = step(s)
    fp.check()
    ref = s["table"].double()[s["ids"]] * D ** 0.5
    assert_within(r["x0"], ref, (2 * U + half_ulp(BF)) * 1.001 * ref.abs(), "lookup")
    ry, _, _, bound = layernorm(r["x0"], s["g1"], s["b1"], 1e-5)
    assert_within(r["h1"], ry, bound + half_ulp(BF) * (ry.abs() + bound), "layernorm")
    (dx, bx), (dg, bg), _ = norm_backward(r["dh2"], r["x1"], None, r["rstd2"], s["g2"], r["dy2"])
    assert_within(r["dx1"], dx, bx + half_ulp(BF) * (dx.abs() + bx), "rmsnorm dx")
    assert_within(r["dg2"], dg, bg + 8 * U * dg.abs(), "rmsnorm dgamma")
    (dx, bx), (dg, bg), (db, bb) = norm_backward(r["dh1"], r["x0"], r["mean"], r["rstd1"], s["g1"], r["dx1"])
    assert_within(r["dx0"], dx, bx + half_ulp(BF) * (dx.abs() + bx), "layernorm dx")
    assert_within(r["dg1"], dg, bg + 8 * U * dg.abs(), "layernorm dgamma")
    assert_within(r["db1"], db, bb + U * db.abs(), "layernorm dbeta")
    dt, bt = embedding_backward(r["dx0"], s["ids"], V, D ** 0.5, 0)
    assert_within(r["dtable"], dt, bt + U * dt.abs(), "table gradient")
    n = math.sqrt(math.fsum(g.double().square().sum().item() for g in r["grads"]))
    assert n > 1.0 and abs(r["norm"].item() - n) <= 6 * U * n
    for g, c in zip(r["grads"], r["clipped"]):
        ref = g.double() / (n + 1e-6)
        assert_within(c, ref, 9 * U * ref.abs(), "clipped")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(s)
    graph.replay()
    fp.check()
    assert torch.equal(captured["norm"], r["norm"])
    assert all(torch.equal(a, b) for a, b in zip(captured["clipped"], r["clipped"]))


def test_behind_copies_and_fills():
    """Each operator right behind a host copy, a fill and another operator that
    writes its inputs, eagerly, on a side stream and captured: none reads or
    writes ahead of what comes before it on the stream."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    M, N, V = 3000, 1024, 700
    sources = [torch.randn(M, N, generator=gen, device="cuda").to(BF).cpu().pin_memory() for _ in range(3)]
    id_sources = [torch.randint(0, V, (M,), generator=gen, device="cuda").cpu().pin_memory() for _ in range(3)]
    x, ids = torch.empty(M, N, dtype=BF, device="cuda"), torch.empty(M, dtype=torch.int64, device="cuda")
    host_x, host_ids = torch.empty(M, N, dtype=BF).pin_memory(), torch.empty(M, dtype=torch.int64).pin_memory()
    dw, dx = torch.empty(V, N, device="cuda"), torch.empty(M, N, dtype=BF, device="cuda")
    big = torch.empty(64 << 20, device="cuda")

    def run():
        big.fill_(1.0)  # work that is still running when the rest is queued
        x.copy_(host_x, non_blocking=True)
        y, mean, rstd = fp.layernorm_forward(x)
        dx.fill_(7.0)
        fp.layernorm_backward(y, x, mean, rstd, out=(dx, None, None), params=False)
        ids.copy_(host_ids, non_blocking=True)
        dw.fill_(7.0)
        fp.embedding_backward(dx, ids, V, out=dw)
        t = fp.embedding_forward(dw, ids)
        dw.mul_(0.5)
        fp.embedding_backward(dx, ids, V, out=dw, accumulate=True)
        norm = fp.clip_grads([dw, t], 1.0)
        return y, dx.clone(), t, norm, dw.clone()

    def plain():
        y, mean, rstd = fp.layernorm_forward(x)
        torch.cuda.synchronize()
        a = fp.layernorm_backward(y, x, mean, rstd, params=False)[0]
        torch.cuda.synchronize()
        w = fp.embedding_backward(a, ids, V)
        torch.cuda.synchronize()
        t = fp.embedding_forward(w, ids)
        w = w * 0.5
        torch.cuda.synchronize()
        fp.embedding_backward(a, ids, V, out=w, accumulate=True)
        torch.cuda.synchronize()
        norm = fp.clip_grads([w, t], 1.0)
        torch.cuda.synchronize()
        return y, a, t, norm, w

    def fill(k):
        torch.cuda.synchronize()
        host_x.copy_(sources[k])
        host_ids.copy_(id_sources[k])

    fill(0)
    got = run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, plain()))
    fill(1)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, plain()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for k in (2, 0):
        fill(k)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, plain()))


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs a second GPU")
def test_on_a_device_that_is_not_current():
    """Tensors of another device than the current one: the calls run there."""
    with torch.cuda.device(1):
        x = torch.randn(300, 640, device="cuda").to(BF)
        ids = torch.randint(0, 50, (300,), device="cuda")
        y, mean, rstd = fp.layernorm_forward(x)
        want = (y, mean, rstd, *fp.layernorm_backward(x, x, mean, rstd), fp.embedding_backward(x, ids, 50), fp.grad_norm([x]))
    y, mean, rstd = fp.layernorm_forward(x)
    got = (y, mean, rstd, *fp.layernorm_backward(x, x, mean, rstd), fp.embedding_backward(x, ids, 50), fp.grad_norm([x]))
    assert torch.cuda.current_device() == 0
    torch.cuda.synchronize(1)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
