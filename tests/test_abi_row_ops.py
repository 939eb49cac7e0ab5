"""The row operators' C ABI on the CPU (embedding, norms, gradient clipping):
bad arguments give the documented status codes before a device is touched
(fake pointers are never dereferenced), and the Python binding refuses what
it documents."""
import ctypes

import pytest
import torch

OK, INVALID, SHAPE, ALIGN, UNSUPPORTED, CUDA = 0, -1, -2, -3, -4, -5
P = 1 << 20
# With a device, an accepted call would launch on the fake pointers.
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="fake device pointers: only where there is no GPU")
NODEV = (CUDA, UNSUPPORTED)  # every argument accepted: no device here
BF16, FP16, FP32 = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    from blockwise_fp8_linear_fp8bq_b200 import build
    build.build()
    import blockwise_fp8_linear_fp8bq_b200 as fp
    return fp.lib()


def test_index_status_text(L):
    assert L.fp8bq_status_string(-7).decode() not in ("", "unknown status")


def test_embedding_forward_arguments(L):
    def f(w=P, V=100, D=64, ldw=64, ids=P, i64=1, T=5, scale=1.0, y=P, ldy=64, dt=BF16, out=BF16):
        return L.fp8bq_embedding_forward(w, V, D, ldw, ids, i64, T, scale, y, ldy, dt, out, None)
    assert f() in NODEV
    assert f(w=None) == INVALID and f(ids=None) == INVALID and f(y=None) == INVALID
    assert f(dt=0) == INVALID and f(out=0) == INVALID and f(dt=4) == INVALID
    assert f(i64=2) == INVALID
    assert f(scale=float("nan")) == INVALID and f(scale=float("inf")) == INVALID
    assert f(V=-1) == SHAPE and f(D=-1) == SHAPE and f(T=-1) == SHAPE
    assert f(ldw=63) == SHAPE and f(ldy=63) == SHAPE
    assert f(V=2 ** 31) == SHAPE and f(T=2 ** 31) == SHAPE
    assert f(w=P + 1) == ALIGN and f(ids=P + 4) == ALIGN and f(y=P + 1) == ALIGN
    assert f(w=P + 2, dt=FP32) == ALIGN and f(y=P + 2, out=FP32) == ALIGN
    assert f(w=P + 2, ids=P + 4, i64=0, y=P + 6) in NODEV  # element alignment suffices
    assert f(T=0) == OK and f(D=0, ldw=0, ldy=0) == OK


def test_embedding_backward_arguments(L):
    n = L.fp8bq_embedding_workspace_bytes(5000, 64, 100)
    assert n > 0
    assert L.fp8bq_embedding_workspace_bytes(0, 64, 100) == 0
    assert L.fp8bq_embedding_workspace_bytes(-1, 64, 100) == -1 and L.fp8bq_embedding_workspace_bytes(5, -1, 100) == -1
    assert L.fp8bq_embedding_workspace_bytes(5, 64, -1) == -1
    assert L.fp8bq_embedding_workspace_bytes(5, 64, 100) == 0  # few tokens: none

    def f(dy=P, T=5000, D=64, lddy=64, ids=P, i64=1, V=100, scale=1.0, pad=-1, dw=P, lddw=64, dt=BF16, dwt=FP32, flags=0,
          ws=P, nbytes=n):
        return L.fp8bq_embedding_backward(dy, T, D, lddy, ids, i64, V, scale, pad, dw, lddw, dt, dwt, flags, ws, nbytes,
                                          None)
    assert f() in NODEV and f(dwt=BF16) in NODEV and f(flags=1) in NODEV and f(pad=7) in NODEV
    assert f(dy=None) == INVALID and f(ids=None) == INVALID and f(dw=None) == INVALID and f(ws=None) == INVALID
    assert f(nbytes=n - 1) == INVALID
    assert f(dwt=FP16) == INVALID and f(dt=FP32, dwt=BF16) == INVALID and f(dt=0) == INVALID
    assert f(flags=2) == INVALID and f(i64=-1) == INVALID and f(scale=float("nan")) == INVALID
    assert f(lddy=63) == SHAPE and f(lddw=63) == SHAPE and f(V=-1) == SHAPE and f(V=2 ** 31 - 1) == SHAPE
    assert f(dy=P + 1) == ALIGN and f(dw=P + 2) == ALIGN and f(ids=P + 4) == ALIGN and f(ws=P + 8) == ALIGN
    assert f(D=0, lddy=0, lddw=0) == OK
    assert f(T=0, flags=1) == OK                            # nothing to add
    assert f(T=0, dy=None, ids=None, ws=None, nbytes=0) in NODEV  # the gradient is all zeros
    assert f(T=5, ws=None, nbytes=0) in NODEV


def test_layernorm_forward_arguments(L):
    def f(x=P, M=4, N=64, ldx=64, g=P, b=P, eps=1e-5, y=P, ldy=64, mean=P, rstd=P, dt=BF16, pdt=BF16):
        return L.fp8bq_layernorm_forward(x, M, N, ldx, g, b, eps, y, ldy, mean, rstd, dt, pdt, None)
    assert f() in NODEV and f(g=None, b=None, mean=None, rstd=None) in NODEV and f(pdt=FP32) in NODEV
    assert f(x=None) == INVALID and f(y=None) == INVALID
    assert f(eps=-1.0) == INVALID and f(eps=float("nan")) == INVALID and f(eps=float("inf")) == INVALID
    assert f(dt=0) == INVALID and f(pdt=FP16) == INVALID and f(dt=FP32, pdt=BF16) == INVALID
    assert f(M=-1) == SHAPE and f(N=-1) == SHAPE and f(ldx=63) == SHAPE and f(ldy=63) == SHAPE and f(M=2 ** 31) == SHAPE
    assert f(x=P + 1) == ALIGN and f(y=P + 1) == ALIGN and f(g=P + 1) == ALIGN and f(b=P + 2, pdt=FP32) == ALIGN
    assert f(mean=P + 2) == ALIGN and f(rstd=P + 1) == ALIGN
    assert f(M=0) == OK and f(N=0, ldx=0, ldy=0) == OK


@pytest.mark.parametrize("what", ["fp8bq_layernorm_backward", "fp8bq_rmsnorm_backward"])
def test_norm_backward_arguments(L, what):
    import blockwise_fp8_linear_fp8bq_b200 as fp
    layernorm = what == "fp8bq_layernorm_backward"

    def f(**kw):
        d = dict(dy=P, x=P, dres=None, dx=P, M=4, N=64, lddy=64, ldx=64, lddres=0, lddx=64, gamma=P, mean=P, rstd=P,
                 dgamma=P, dbeta=P, workspace=P, workspace_bytes=1 << 30, dtype=BF16, param_dtype=BF16, flags=0, reserved=0)
        d.update(kw)
        return getattr(L, what)(ctypes.byref(fp._CNormGrad(**d)), None)
    assert getattr(L, what)(None, None) == INVALID
    assert f() in NODEV and f(gamma=None) in NODEV and f(dgamma=None, dbeta=None, workspace=None) in NODEV
    assert f(flags=3) in NODEV and f(dres=P, lddres=64) in NODEV and f(param_dtype=FP32) in NODEV
    for name in ("dy", "x", "dx", "rstd"):
        assert f(**{name: None}) == INVALID
    assert f(mean=None) == INVALID if layernorm else f(mean=None) in NODEV
    assert f(dtype=0) == INVALID and f(param_dtype=FP16) == INVALID and f(flags=4) == INVALID
    assert f(M=-1) == SHAPE and f(N=-1) == SHAPE and f(M=2 ** 31) == SHAPE
    for name in ("lddy", "ldx", "lddx"):
        assert f(**{name: 63}) == SHAPE
    assert f(dres=P, lddres=63) == SHAPE
    for name in ("dy", "x", "dx", "gamma"):
        assert f(**{name: P + 1}) == ALIGN
    assert f(dres=P + 1, lddres=64) == ALIGN and f(gamma=P + 2, param_dtype=FP32) == ALIGN
    assert f(rstd=P + 2) == ALIGN and f(rstd=P + 4, flags=2) == ALIGN and f(mean=P + 2) == ALIGN
    assert f(dgamma=P + 2) == ALIGN and f(dbeta=P + 1) == ALIGN and f(workspace=P + 8) == ALIGN
    assert f(N=0, lddy=0, ldx=0, lddx=0) == OK
    assert f(M=0, dgamma=None, dbeta=None) == OK
    assert L.fp8bq_norm_workspace_bytes(4, 64) == -1  # no usable device here


def test_grad_list_arguments(L):
    import blockwise_fp8_linear_fp8bq_b200 as fp

    def f(*grads, count=None, most=1.0, norm=P, ws=P, nbytes=1 << 30, clip=True):
        table = (fp._CGrad * max(1, len(grads)))(*grads)
        n = len(grads) if count is None else count
        if clip:
            return L.fp8bq_grad_clip(table, n, most, norm, ws, nbytes, None)
        return L.fp8bq_grad_norm(table, n, norm, ws, nbytes, None)
    G = lambda g=P, out=P, n=100, dt=BF16, odt=BF16: fp._CGrad(g, out, n, dt, odt)
    assert f(G()) in NODEV and f() in NODEV and f(G(), clip=False) in NODEV
    assert f(G(out=None, odt=0), clip=False) in NODEV          # the norm reads no output
    assert L.fp8bq_grad_clip(None, 1, 1.0, P, P, 1 << 30, None) == INVALID
    assert f(G(g=None)) == INVALID and f(G(out=None)) == INVALID
    assert f(G(n=0, g=None, out=None)) in NODEV
    assert f(G(dt=0)) == INVALID and f(G(odt=0)) == INVALID
    assert f(G(odt=FP32)) == INVALID                           # in place with another type
    assert f(G(), most=-1.0) == INVALID and f(G(), most=float("nan")) == INVALID
    assert f(G(), norm=None) == INVALID
    assert f(G(n=-1)) == SHAPE and f(G(n=2 ** 35 + 1)) == SHAPE and f(G(), count=-1) == SHAPE
    assert f(G(g=P + 1)) == ALIGN and f(G(out=P + 1)) == ALIGN and f(G(g=P + 4096, out=P + 2, odt=FP32)) == ALIGN
    assert f(G(), norm=P + 2) == ALIGN and f(G(), ws=P + 8) == ALIGN
    # overlaps: a tensor listed twice, an output over another input, and neighbours that touch
    assert f(G(), G()) == INVALID
    assert f(G(), G(g=P + 100, out=P + 4096)) == INVALID
    assert f(G(), G(g=P + 200, out=P + 200)) in NODEV
    assert f(G(out=P + 4096), G(out=P + 8192)) in NODEV        # one input read twice
    assert f(G(out=P + 4096), G(g=P + 2048, out=P + 4196)) == INVALID
    assert f(G(), G(), clip=False) in NODEV
    assert L.fp8bq_grad_workspace_bytes(-1) == -1


def test_binding_refuses():
    import blockwise_fp8_linear_fp8bq_b200 as fp
    x, ids = torch.zeros(4, 64), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        fp.embedding_forward(x, ids)                            # no CPU path
    with pytest.raises(ValueError):
        fp.embedding_backward(x, ids, 10)
    with pytest.raises(ValueError):
        fp.layernorm_forward(x)
    with pytest.raises(ValueError):
        fp.layernorm_backward(x, x, x[:, 0], x[:, 0])
    with pytest.raises(ValueError):
        fp.rmsnorm_backward(x, x, x[:, 0])
    with pytest.raises(ValueError):
        fp.clip_grads([x], 1.0)
    with pytest.raises(ValueError):
        fp.clip_grads([], 1.0)
    with pytest.raises(ValueError):
        fp.grad_norm([])
    with pytest.raises(ValueError):
        fp.layernorm_forward(x.double())
    with pytest.raises(ValueError):
        fp.layernorm_forward(x.t())
