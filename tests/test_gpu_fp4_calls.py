"""What calls of the microscaled 4-bit operators leave behind, accept and
launch, on the GPU."""

import ctypes

import pytest
import torch

from test_gpu_fp4 import BF16, FMTS, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("call", ["quantize", "dequantize", "linear", "linear of many", "codes", "codes of many"])
def test_a_refused_launch_leaves_no_error_behind(mq, cuda, fmt, call):
    # launches into a stream whose capture is no longer valid are refused by
    # the runtime; this library's other launches look at the last error and
    # must not find that one
    M = 200 if "many" in call else 20
    W, X = values(300, 512, BF16, 1), values(M, 512, BF16, 2).to(cuda)
    w, other = mq.Fp4Weight.pack(W.to(cuda), fmt), mq.Weight.pack(W.float().numpy() * 0.05, 0.01)
    want = other.linear(X, path="prefill")
    q, Y = mq.fp4_quantize(X, fmt), torch.empty(M, 300, dtype=BF16, device=cuda)
    V, ws = torch.empty(M, 512, dtype=BF16, device=cuda), torch.empty(1 << 22, dtype=torch.uint8, device=cuda)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    lib, cu, s, f = mq.lib(), ctypes.CDLL("libcuda.so.1"), side.cuda_stream, mq.FP4_FORMATS[fmt]
    calls = {
        "quantize": lambda: lib.mq_fp4_quantize(X.data_ptr(), 0, M, 512, 512, None, M, f, *q._at, s),
        "dequantize": lambda: lib.mq_fp4_dequantize(*q._at, M, 512, f, V.data_ptr(), 0, 512, s),
        "linear": lambda: lib.mq_fp4_linear(w.handle, X.data_ptr(), 0, M, 512, Y.data_ptr(), 300, ws.data_ptr(), ws.numel(), s),
        "codes": lambda: lib.mq_fp4_linear_codes(w.handle, *q._at, M, Y.data_ptr(), 0, 300, s),
    }
    run = calls[call.split(" of ")[0]]
    graph, code = ctypes.c_void_p(), ctypes.c_int32()
    assert cu.cuStreamBeginCapture_v2(ctypes.c_void_p(s), 2) == 0  # relaxed: this stream alone
    waited = lib.mq_fp4_device_error(w.handle, s, ctypes.byref(code))  # a wait makes the capture invalid
    status = run()
    ended = cu.cuStreamEndCapture(ctypes.c_void_p(s), ctypes.byref(graph))
    assert (waited, status) == (mq.CUDA, mq.CUDA) and ended != 0
    got = other.linear(X, path="prefill")
    assert torch.equal(got, want)
    assert run() == 0  # the stream takes launches again
    torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("E,N,K", [(1, 200, 96), (1, 1024, 4096), (1, 11007, 4100), (8, 1000, 640), (40, 384, 512),
                                   (300, 72, 192)])
def test_a_workspace_for_the_largest_batch_serves_the_smaller_ones(mq, cuda, fmt, E, N, K):
    w = mq.Fp4Weight.pack(values(E * N, K, BF16, 1).view(E, N, K).to(cuda), fmt)
    need = [w.workspace_bytes(r) for r in range(1, 4001)]
    assert need == sorted(need)
    for most in (17, 65, 129, 225, 257, 385, 2369):
        ws = torch.full((need[most - 1] + 64,), 9, dtype=torch.uint8, device=cuda)
        for M in (most, most - 1, most // 2, 1):
            X = values(M, K, BF16, M, spread=0.3).to(cuda)
            offsets = torch.linspace(0, M, E + 1).int().to(cuda)
            Y = w.linear_grouped(X, offsets, None, ws[:-64])
            assert torch.equal(Y, w.linear_grouped(mq.fp4_quantize(X, fmt), offsets))
            assert E > 1 or torch.equal(Y, w.linear(X, None, ws[:-64]))
        assert (ws[-64:] == 9).all()
    assert w.device_error() == 0
