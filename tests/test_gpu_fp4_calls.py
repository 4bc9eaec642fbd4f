"""What calls of the microscaled 4-bit operators leave behind, accept and
launch, on the GPU."""

import ctypes

import numpy as np
import pytest
import torch

from test_gpu_fp4 import BF16, FMTS, held, values

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


class KernelNode(ctypes.Structure):  # CUDA_KERNEL_NODE_PARAMS
    _fields_ = [("func", ctypes.c_void_p), ("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3),
                ("smem", ctypes.c_uint), ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p),
                ("kern", ctypes.c_void_p), ("ctx", ctypes.c_void_p)]


class Attribute(ctypes.Structure):  # CUlaunchAttribute
    _fields_ = [("id", ctypes.c_int), ("pad", ctypes.c_int), ("value", ctypes.c_uint * 16)]


class Config(ctypes.Structure):  # CUlaunchConfig
    _fields_ = [("grid", ctypes.c_uint * 3), ("block", ctypes.c_uint * 3), ("smem", ctypes.c_uint),
                ("stream", ctypes.c_void_p), ("attrs", ctypes.POINTER(Attribute)), ("count", ctypes.c_uint)]


def launches(cu, stream, call):
    """(kernel's name, CTAs of the launch, CTAs that the device holds at once)
    of what a call launches, from the graph it leaves in a capture.

    The runtime's own count of clusters takes an SM for one CTA of a kernel with
    tensor memory. So many CTAs as an SM has registers and shared memory for
    (228 KB, of which a CTA takes 1 KB more than it asks for) hold so many
    clusters as that at least."""
    ptr, CLUSTER = ctypes.c_void_p, 4
    graph, count = ptr(), ctypes.c_size_t()
    assert cu.cuStreamBeginCapture_v2(ptr(stream), 2) == 0
    status = call()
    assert cu.cuStreamEndCapture(ptr(stream), ctypes.byref(graph)) == 0 and status == 0
    assert cu.cuGraphGetNodes(graph, None, ctypes.byref(count)) == 0
    nodes = (ptr * count.value)()
    assert cu.cuGraphGetNodes(graph, nodes, ctypes.byref(count)) == 0
    out = []
    for node in nodes:
        k, cluster, name, room = KernelNode(), (ctypes.c_uint * 16)(), ctypes.c_char_p(), ctypes.c_int()
        assert cu.cuGraphKernelNodeGetParams_v2(ptr(node), ctypes.byref(k)) == 0
        func = ptr(k.func)
        if not k.func:
            assert cu.cuKernelGetFunction(ctypes.byref(func), ptr(k.kern)) == 0
        assert cu.cuFuncGetName(ctypes.byref(name), func) == 0
        assert cu.cuGraphKernelNodeGetAttribute(ptr(node), CLUSTER, cluster) == 0
        size = max(1, cluster[0])
        a = Attribute(id=CLUSTER)
        a.value[:3] = [size, 1, 1]
        c = Config(grid=k.grid, block=k.block, smem=k.smem, stream=None, attrs=ctypes.pointer(a), count=1)
        assert cu.cuOccupancyMaxActiveClusters(ctypes.byref(room), func, ctypes.byref(c)) == 0
        regs = ctypes.c_int()
        assert cu.cuFuncGetAttribute(ctypes.byref(regs), 4, func) == 0
        share = min(228 * 1024 // (k.smem + 1024), 65536 // (regs.value * k.block[0])) if k.smem else 1
        out.append((name.value.decode(), k.grid[0], room.value * size * share))
    assert cu.cuGraphDestroy(graph) == 0
    return out


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("N,K", [(1024, 4096), (1920, 2048), (2048, 2048), (2816, 8192), (4096, 11008), (9500, 1024),
                                 (11008, 4096), (20480, 512), (28672, 2048), (37888, 512)])
def test_products_of_few_tokens_run_in_one_wave(mq, cuda, fmt, N, K):
    # clusters that find no room wait for all of the first ones to end
    w = mq.Fp4Weight.pack(torch.zeros(N, K, dtype=BF16, device=cuda), fmt)
    lib, cu, s = mq.lib(), ctypes.CDLL("libcuda.so.1"), torch.cuda.Stream().cuda_stream
    X, Y = torch.zeros(128, K, dtype=BF16, device=cuda), torch.empty(128, N, dtype=BF16, device=cuda)
    ws = torch.empty(max(16, w.workspace_bytes(128)), dtype=torch.uint8, device=cuda)
    for M in (1, 8, 16, 17, 24, 32, 33, 48, 64, 65, 100, 128):
        def call():
            return lib.mq_fp4_linear(w.handle, X.data_ptr(), 0, M, K, Y.data_ptr(), N, ws.data_ptr(), ws.numel(), s)

        assert call() == 0  # sets the kernel up
        torch.cuda.synchronize()
        got = [x for x in launches(cu, s, call) if "quantize" not in x[0]]
        assert len(got) == 1
        name, ctas, room = got[0]
        assert "fp4_narrow" in name or "fp4_wide" in name
        assert ctas <= room, (M, name, ctas, room)


@pytest.mark.parametrize("fmt", FMTS)
def test_clusters_fill_the_device_once(mq, cuda, fmt):
    # every number of row tiles around what the device holds of clusters of 2
    # to 8 CTAs, whatever its SMs' groups are like
    lib, cu, s, K = mq.lib(), ctypes.CDLL("libcuda.so.1"), torch.cuda.Stream().cuda_stream, 6144
    X, most = torch.zeros(48, K, dtype=BF16, device=cuda), 0
    for tiles in [*range(1, 40), *range(42, 52), *range(70, 80)]:
        N = 128 * tiles
        w = mq.Fp4Weight.pack(torch.zeros(N, K, dtype=BF16, device=cuda), fmt)
        Y = torch.empty(48, N, dtype=BF16, device=cuda)
        ws = torch.empty(max(16, w.workspace_bytes(48)), dtype=torch.uint8, device=cuda)
        for M in (24, 48):
            def call():
                return lib.mq_fp4_linear(w.handle, X.data_ptr(), 0, M, K, Y.data_ptr(), N, ws.data_ptr(), ws.numel(), s)

            assert call() == 0
            torch.cuda.synchronize()
            name, ctas, room = [x for x in launches(cu, s, call) if "quantize" not in x[0]][0]
            assert ctas <= room, (M, tiles, name, ctas, room)
            most = max(most, ctas)
    assert most > 0.9 * torch.cuda.get_device_properties(cuda).multi_processor_count


def exact_values(q):
    """The values held, in 64 bits on the device (exact: 2, 4 and 24 bits)."""
    c = torch.stack([q.codes & 15, q.codes >> 4], -1).flatten(-2)[:, :q.K].long()
    half = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=c.device)
    v = half[c & 7] * (1 - 2 * (c >> 3))
    if q.fmt == "mxfp4":
        s = torch.exp2(q.scales.double() - 127)
    else:
        s = q.scales.view(torch.float8_e4m3fn).double() * q.row_scale.double()[:, None]
    return v * s.repeat_interleave(32 if q.fmt == "mxfp4" else 16, dim=1)[:, :q.K]


def test_exact_values(mq, cuda):
    for fmt in FMTS:
        X = values(50, 333, BF16, 1)
        assert np.array_equal(exact_values(mq.fp4_quantize(X.to(cuda), fmt)).cpu().numpy(), held(X, fmt))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, torch.float16])
@pytest.mark.parametrize("M,N,K", [(1, 8192, 11008), (16, 14336, 4096), (24, 20480, 4100), (60, 4096, 11008),
                                   (96, 4096, 4096), (1000, 4096, 2048), (2048, 2560, 4096), (2000, 9001, 11008),
                                   (4096, 4096, 11008)])
def test_every_output_of_large_products(mq, cuda, fmt, dtype, M, N, K):
    # all of them against 64 bits, within the bound of a single output: a block
    # of 16 columns left out of such products is beyond it in most outputs (two
    # of three at K = 11008, nine of ten at 4096)
    X = values(M, K, dtype, M, spread=0.3).to(cuda)
    w = mq.Fp4Weight.pack((values(N, K, torch.float32, N, spread=0.3) * 0.05).to(cuda), fmt)
    x64, w64 = exact_values(mq.fp4_quantize(X, fmt)), exact_values(w.export())
    y64, S = x64 @ w64.T, x64.abs() @ w64.abs().T
    # as `bound`, with the 64-bit products' own error, 2^-53 of S for each of K terms
    tol = ((torch.finfo(dtype).eps / 2 + 2**-22) * y64.abs() + (K / 16 + 16) * 2.0**-23 * S * 1.01 + K * 2.0**-52 * S +
           2.0**-25)
    off = (w.linear(X).double() - y64).abs()
    assert (off <= tol).all()
    assert w.device_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, torch.float16])
@pytest.mark.parametrize("K", [999, 4096])
def test_dequantised_values_are_rounded_as_documented(mq, cuda, fmt, dtype, K):
    # to 32 bits by the row factor (not at all for mxfp4), then to the type
    q = mq.fp4_quantize(values(700, K, BF16, 1).to(cuda), fmt)
    whole, once = q.dequantize(), exact_values(q).float()
    assert torch.equal(whole, once)
    assert torch.equal(q.dequantize(dtype), once.to(dtype))
