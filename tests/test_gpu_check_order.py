"""Two kinds of failure between two checks: an id outside its table, recorded
first, does not hide a wait that ran out after it.  The wait is the split-tile
GEMM's, on flags that one CTA pair is made to withhold, limited to 1 ms."""
import ctypes

import pytest
import torch

import blockwise_fp8_linear_fp8bq_b200 as fp
from blockwise_fp8_linear_fp8bq_b200 import synth
from test_gpu_timeout import OK, TIMEOUT, _check_status, _hook, mid_tile_pairs

pytestmark = pytest.mark.gpu
INDEX = -7


@pytest.mark.parametrize("first", ["id", "wait"])
def test_each_kind_is_reported(first):
    M, N, K = 6400, 1280, 4096
    C = torch.cuda.get_device_properties(0).multi_processor_count // 2
    pairs = mid_tile_pairs(((N + 255) // 256) * ((K + 255) // 256) % C, M // 128)
    fmt = fp.SCALE_FP32
    dy = synth.grads_bf16(M, N, seed=811, device="cuda")
    x = synth.activations_bf16(M, K, seed=812, device="cuda")
    A = fp.row_operand(*fp.quantize_act_t(dy, fmt), fmt)
    B = fp.row_operand(*fp.quantize_act_t(x, fmt), fmt)
    ws = fp.gemm_workspace()
    w = torch.randn(10, 16, device="cuda")
    bad = torch.tensor([3, 10], device="cuda")
    assert _check_status() == OK
    ca, cb = A._c(), B._c()
    D = torch.empty(N, K, dtype=torch.bfloat16, device="cuda")

    def lookup():
        assert (fp.embedding_forward(w, bad)[1] == 0).all()

    def wait():
        assert _hook()(ctypes.byref(ca), ctypes.byref(cb), D.data_ptr(), N, K, M, K, 0, ws.data_ptr(), ws.numel(), pairs[0],
                       1000000, torch.cuda.current_stream().cuda_stream) == OK

    for f in (lookup, wait) if first == "id" else (wait, lookup):
        f()
    # the wait's first: what its kernel wrote is undefined
    assert _check_status() == TIMEOUT
    assert _check_status() == INDEX
    assert _check_status() == OK
    # one kind alone, and a check that raises nothing after it
    lookup()
    assert _check_status() == INDEX and _check_status() == OK
    ws.zero_()
    fp.gemm(A, B, workspace=ws)
    assert _check_status() == OK
