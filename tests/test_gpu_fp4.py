"""Microscaled 4-bit floating point on the GPU against the fp64 oracle
(oracle/fp4.py): codes and scales byte for byte, values and products within
bounds derived below.

A product's bound: products of codes and scales are exact, so an output is off
by the fp32 accumulation, at most 2^-23 of the sum of the terms' magnitudes S
for each of its additions (one for every 16 terms at the finest, a few more to
join shares of K), by two products with the row factors (2^-24 of |y| each)
and by its own rounding, half a step: eps / 2 of |y|, and half of the smallest
fp16 step (2^-25) where |y| is below its normal range.
"""

import numpy as np
import pytest
import torch

from oracle import fp4

pytestmark = pytest.mark.gpu

FMTS = ["mxfp4", "nvfp4"]
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def values(M, K, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * torch.exp(spread * torch.randn(M, 1, generator=g))
    x[:, torch.randint(0, K, (2,), generator=g)] *= 12
    return x.to(dtype)


def held(X, fmt):
    return fp4.dequantize(*fp4.quantize(X.float().cpu().numpy(), fmt), fmt)


def same_bits(q, X, fmt):
    c, s, r = fp4.quantize(X.float().cpu().numpy(), fmt)
    cb, sb = fp4.pack(c, s, fmt)
    assert np.array_equal(q.codes.cpu().numpy(), cb)
    assert np.array_equal(q.scales.cpu().numpy(), sb)
    if r is None:
        assert q.row_scale is None
    else:
        got = q.row_scale.cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(r))
        assert np.array_equal(got[~np.isnan(r)], r[~np.isnan(r)])


def bound(y64, S, K, dtype):
    adds = K / 16 + 16
    return (torch.finfo(dtype).eps / 2 + 2**-22) * np.abs(y64) + adds * 2.0**-23 * S * 1.01 + 2.0**-25


def check_product(Y, x64, w64, dtype):
    y64, S = fp4.linear(x64, w64)
    got = Y.double().cpu().numpy()
    off = np.abs(got - y64) - bound(y64, S, x64.shape[1], dtype)
    assert np.isfinite(got).all() and off.max() <= 0, (off.max(), np.unravel_index(off.argmax(), off.shape))


# ---------------------------------------------------------------- quantise
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 16), (3, 31), (2, 33), (1, 4096), (5, 1000), (70, 255), (33, 513),
                                 (2, 11008), (700, 2048), (2501, 99), (1, 33000)])
def test_quantize_bits(mq, cuda, fmt, dtype, M, K):
    X = values(M, K, dtype, M * 7 + K, spread=2.0 if dtype != FP16 else 1.0)
    q = mq.fp4_quantize(X.to(cuda), fmt)
    same_bits(q, X, fmt)
    v = held(X, fmt)
    got = q.dequantize().double().cpu().numpy()
    # mxfp4's values are exact in fp32; nvfp4's product with the row factor rounds once
    assert (np.abs(got - v) <= (0 if fmt == "mxfp4" else 2.0**-24) * np.abs(v)).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("left,ld", [(0, 640), (8, 616), (1, 601), (3, 611), (7, 613), (5, 608)])
def test_quantize_views(mq, cuda, fmt, dtype, left, ld):
    # rows that start at any element, columns around them that must not count
    M, K = 37, 595
    big = torch.full((M, ld), 1000.0)
    big[:, left:left + K] = values(M, K, FP32, left)
    X = big.to(dtype).to(cuda)[:, left:left + K]
    assert X.stride(0) == ld
    same_bits(mq.fp4_quantize(X, fmt), X, fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 2, 9])
def test_quantize_inside_a_tight_buffer(mq, cuda, fmt, M):
    # X up to the first and last element of its memory, at an odd start
    K = 333
    flat = values(1, M * K + 1, BF16, M).to(cuda).flatten()
    X = flat[1:].view(M, K)
    same_bits(mq.fp4_quantize(X, fmt), X, fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_special_values(mq, cuda, fmt):
    X = torch.zeros(9, 96)
    X[1, 5] = float("inf")
    X[2, 40] = float("nan")
    X[3, 70] = -float("inf")
    X[4] = torch.finfo(BF16).max
    X[5] = -torch.finfo(BF16).tiny / 64  # subnormal
    X[6, ::2] = 1e-30
    X[7] = torch.linspace(-6, 6, 96)
    X[8, 3] = -0.0
    X = X.to(BF16)
    q = mq.fp4_quantize(X.to(cuda), fmt)
    same_bits(q, X, fmt)
    got, v = q.dequantize().cpu().double().numpy(), held(X, fmt)
    assert np.array_equal(np.isnan(got), np.isnan(v))
    ok = np.isfinite(v)
    assert (np.abs(got - v)[ok] <= 2.0**-24 * np.abs(v)[ok]).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_rows(mq, cuda, fmt):
    X = values(20, 300, FP16, 5).to(cuda)
    rows = torch.tensor([3, 3, 19, 0, -1, 20, 7, 2**31 - 1, 3], device=cuda)
    want = torch.stack([X[r] if 0 <= r < 20 else torch.zeros_like(X[0]) for r in rows.tolist()])
    for t in (torch.int32, torch.int64):
        same_bits(mq.fp4_quantize(X, fmt, rows=rows.to(t)), want, fmt)
    same_bits(mq.fp4_quantize(X, fmt, rows=torch.tensor([2**32 + 1], device=cuda)), torch.zeros_like(want[:1]), fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("M,K", [(1, 1), (4, 77), (9, 1024), (3, 2051)])
def test_dequantize_types_and_strides(mq, cuda, fmt, dtype, M, K):
    X = values(M, K, FP32, K, spread=0.5)
    q = mq.fp4_quantize(X.to(cuda), fmt)
    v = held(X, fmt)
    half = torch.finfo(dtype).eps / 2 + (0 if fmt == "mxfp4" else 2.0**-24)
    got = q.dequantize(dtype)
    assert got.dtype == dtype
    assert (np.abs(got.cpu().double().numpy() - v) <= half * 1.01 * np.abs(v) + 2.0**-25).all()
    # into a strided buffer through the C ABI: what lies around the rows stays
    ld = K + 5
    Y = torch.full((M, ld), 7.0, dtype=dtype, device=cuda)
    lib = mq.lib()
    r = q.row_scale
    st = lib.mq_fp4_dequantize(q.codes.data_ptr(), q.scales.data_ptr(), None if r is None else r.data_ptr(), M, K,
                               mq.FP4_FORMATS[fmt], Y[:, 2:].data_ptr(), {BF16: 0, FP16: 1, FP32: 2}[dtype], ld,
                               torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert torch.equal(Y[:, 2:2 + K], got) and (Y[:, :2] == 7).all() and (Y[:, 2 + K:] == 7).all()


# ---------------------------------------------------------------- linear
LINEAR = [(1, 1, 1), (1, 128, 256), (1, 4096, 512), (2, 130, 64), (16, 128, 2048), (17, 300, 1001), (7, 1111, 32),
          (33, 257, 4100), (64, 640, 768), (65, 127, 300), (128, 128, 256), (129, 384, 1280), (250, 260, 515),
          (513, 200, 96), (1025, 512, 512), (3, 300, 1536), (5, 260, 1792), (40, 200, 1280), (50, 256, 1792),
          (12, 512, 700), (16, 384, 5000), (80, 200, 11008), (81, 1100, 4200), (100, 130, 5003), (113, 140, 11111),
          (128, 390, 6144), (65, 700, 9000)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("M,N,K", LINEAR)
def test_linear(mq, cuda, fmt, dtype, M, N, K):
    X, W = values(M, K, dtype, M + N, spread=0.3), values(N, K, FP32, K, spread=0.3) * 0.05
    w = mq.Fp4Weight.pack(W.to(cuda), fmt)
    Y = w.linear(X.to(cuda))
    assert Y.dtype == dtype and Y.shape == (M, N)
    check_product(Y, held(X, fmt), held(W, fmt), dtype)
    assert torch.equal(w.linear(X.to(cuda)), Y)  # no dependence on timing
    q = mq.fp4_quantize(X.to(cuda), fmt)
    assert torch.equal(w.linear(q, dtype=dtype), Y)
    assert torch.equal(w.linear(q, torch.empty_like(Y)), Y)
    assert w.device_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(1, 8192, 11008), (16, 14336, 4096), (96, 4096, 4096), (1000, 4096, 2048),
                                   (2048, 2560, 4096), (4096, 4096, 11008), (2000, 9001, 11008), (4000, 4096, 11008)])
def test_linear_large(mq, cuda, fmt, M, N, K):
    # sampled rows of W and of X: the whole range of tiles, the rest by columns
    X, W = values(M, K, BF16, M, spread=0.3), values(N, K, BF16, N, spread=0.3) * 0.05
    w = mq.Fp4Weight.pack(W.to(cuda), fmt)
    Y = w.linear(X.to(cuda))
    g = np.random.default_rng(M)
    rows = np.unique(np.concatenate([g.integers(0, M, 40), [0, M - 1]]))
    cols = np.unique(np.concatenate([g.integers(0, N, 40), [0, 127, 128, N - 1]]))
    check_product(Y[rows][:, cols], held(X[rows], fmt), held(W[cols], fmt), BF16)
    # every output, against the product of the same held values in fp32
    q = mq.fp4_quantize(X.to(cuda), fmt).dequantize()
    e = w.export()
    full = q @ e.dequantize().T
    S = q.abs() @ e.dequantize().abs().T
    # both sides' accumulations, the product's as `bound` has it; rounding to
    # bf16 (8 significant bits) is off by half a step, eps / 2 = 2^-8 of |y|
    tol = (torch.finfo(BF16).eps / 2 + 2**-21) * full.abs() + (K / 16 + K + 16) * 2.0**-23 * S + 2.0**-25
    assert ((Y.float() - full).abs() <= tol * 1.01).all()
    # tokens quantised before, whose scales are row-major: the same bits
    assert torch.equal(w.linear(mq.fp4_quantize(X.to(cuda), fmt)), Y)
    assert w.device_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 40, 300])
def test_linear_strides_and_canaries(mq, cuda, fmt, M):
    N, K = 203, 333
    X, W = values(M, K, BF16, M, spread=0.3), values(N, K, BF16, 1, spread=0.3)
    w = mq.Fp4Weight.pack(W.to(cuda), fmt)
    want = w.linear(X.to(cuda))
    wide = torch.zeros(M, K + 7, dtype=BF16)
    wide[:, 3:3 + K] = X
    out = torch.full((M + 2, N + 9), 5.0, dtype=BF16, device=cuda)
    ws = torch.full((w.workspace_bytes(M) + 64,), 9, dtype=torch.uint8, device=cuda)
    Y = w.linear(wide.to(cuda)[:, 3:3 + K], out[1:M + 1, 4:4 + N], ws[:w.workspace_bytes(M)])
    assert torch.equal(Y, want) and Y.data_ptr() == out[1:, 4:].data_ptr()
    out[1:M + 1, 4:4 + N] = 5.0
    assert (out == 5.0).all() and (ws[-64:] == 9).all()
    check_product(want, held(X, fmt), held(W, fmt), BF16)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(5, 300, 512), (6, 200, 2048), (50, 200, 1792), (300, 260, 512)])
def test_linear_largest_and_smallest(mq, cuda, fmt, M, N, K):
    # whatever the rows' sizes, an output is finite and right where it and the
    # sums on the way to it are
    X, W = values(M, K, FP32, M, spread=0.3), values(N, K, FP32, N, spread=0.3)
    X = (X * torch.tensor([1e35, 1e-25, 1.0, 1e20, 1e-12])[torch.arange(M) % 5][:, None]).to(BF16)
    W = W * torch.tensor([1e-25, 1e34, 1e-3, 1e10, 1e-12, 1e18, 1.0])[torch.arange(N) % 7][:, None]
    w = mq.Fp4Weight.pack(W.to(cuda), fmt)
    x64, w64 = held(X, fmt), held(W, fmt)
    y64, S = fp4.linear(x64, w64)
    got = w.linear(X.to(cuda)).double().cpu().numpy()
    ok = S < 2.0**126
    # as `bound`, but no fp16: bf16 and fp32 are normal down to 2^-126, where an
    # fp32 step is 2^-149; the smallest S here are 2^-150 or so
    tol = ((torch.finfo(BF16).eps / 2 + 2**-22) * np.abs(y64) + (K / 16 + 16) * 2.0**-23 * S * 1.01 +
           (K / 16 + 16) * 2.0**-126)
    assert np.isfinite(got[ok]).all() and (np.abs(got - y64)[ok] <= tol[ok]).all()
    assert 0.7 < ok.mean() < 1
    assert w.device_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [5, 200])
def test_linear_non_finite_rows(mq, cuda, fmt, M):
    N, K = 150, 400
    X, W = values(M, K, BF16, 2, spread=0.3), values(N, K, BF16, 3, spread=0.3)
    w = mq.Fp4Weight.pack(W.to(cuda), fmt)
    want = w.linear(X.to(cuda))
    X[1, 17], X[3, 399] = float("nan"), float("inf")
    Y = w.linear(X.to(cuda))
    bad = torch.zeros(M, dtype=torch.bool)
    bad[[1, 3]] = True
    assert torch.isnan(Y[bad.to(cuda)]).all()
    assert torch.equal(Y[~bad.to(cuda)], want[~bad.to(cuda)])
    W[5, 0] = float("nan")
    Y = mq.Fp4Weight.pack(W.to(cuda), fmt).linear(X[2:3].to(cuda))
    assert torch.isnan(Y[0, 5]) and torch.isfinite(Y[0, :5]).all() and torch.isfinite(Y[0, 6:]).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_offsets_past_32_bits(mq, cuda, fmt):
    # 2^32 outputs, 2^31 inputs: the same rows again and again
    rows, times, N, K = 4099, 16384, 64, 32
    X, W = values(rows, K, BF16, 1, spread=0.3), values(N, K, BF16, 2, spread=0.3)
    w = mq.Fp4Weight.pack(W.to(cuda), fmt)
    big = X.to(cuda).repeat(times, 1)
    Y = w.linear(big)
    check_product(Y[:rows], held(X, fmt), held(W, fmt), BF16)
    assert (Y.view(times, rows, N) == Y[:rows]).all()
    del Y
    q = mq.fp4_quantize(big, fmt)
    same_bits(mq.Fp4Tensor(*(None if t is None else t[-rows:] for t in (q.codes, q.scales, q.row_scale)), K, fmt), X, fmt)
    v = q.dequantize(BF16)
    assert (v.view(times, rows, K) == v[:rows]).all()


# the same name is defined once more below: this one is collected under its own
test_more_than_2_32_outputs = test_offsets_past_32_bits


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [2, 70])
def test_longest_rows(mq, cuda, fmt, M):
    # K = 2^24: every stage's place, with few values that are not zero and sums that are exact
    K, N = 1 << 24, 3
    X, W = torch.zeros(M, K, dtype=BF16, device=cuda), torch.zeros(N, K, dtype=BF16, device=cuda)
    at = torch.arange(0, K, 65521, device=cuda)
    X[:, at] = 1.0
    X[:, -1] = 1.0
    W[:, at] = (torch.arange(len(at), device=cuda) % 2 * 2 - 1).to(BF16)
    W[1], W[2, -1] = 2 * W[0], 4.0
    Y = mq.Fp4Weight.pack(W, fmt).linear(X)
    x64, w64 = (held(t[:, torch.cat([at, at.new_tensor([K - 1])])], "mxfp4") for t in (X, W))
    # both formats hold these values, nvfp4 but for the roundings of the row
    # factors, and the sums of codes are exact; half a step of bf16 remains
    want = x64 @ w64.T
    assert (np.abs(Y.double().cpu().numpy() - want) <= (2.0**-8 + 2.0**-20) * np.abs(want)).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_no_rows(mq, cuda, fmt):
    w = mq.Fp4Weight.pack(values(64, 64, BF16, 1).to(cuda), fmt)
    X = torch.empty(0, 64, dtype=BF16, device=cuda)
    assert w.linear(X).shape == (0, 64)
    q = mq.fp4_quantize(X, fmt)
    assert q.rows == 0 and w.linear(q).shape == (0, 64) and q.dequantize().shape == (0, 64)
    assert w.linear_grouped(X, torch.zeros(2, dtype=torch.int32, device=cuda)).shape == (0, 64)


@pytest.mark.parametrize("fmt", FMTS)
def test_pack_and_export(mq, cuda, fmt):
    W = values(2 * 131, 340, FP32, 6).view(2, 131, 340)
    w = mq.Fp4Weight.pack(W.to(cuda), fmt)
    assert (w.E, w.N, w.K, w.fmt) == (2, 131, 340, fmt)
    e = w.export()
    same_bits(e, W.view(-1, 340), fmt)
    lead = lambda t: None if t is None else t.view(2, 131, *t.shape[1:])  # noqa: E731
    again = mq.Fp4Weight.pack_codes(lead(e.codes), lead(e.scales), lead(e.row_scale), 340, fmt).export()
    assert torch.equal(again.codes, e.codes) and torch.equal(again.scales, e.scales)
    assert fmt == "mxfp4" or torch.equal(again.row_scale, e.row_scale)


@pytest.mark.parametrize("fmt", FMTS)
def test_pack_too_large_for_the_device(mq, cuda, fmt):
    # refused before anything is read; no error is left behind for the next launch to find
    buf = torch.zeros(1024, dtype=torch.uint8, device=cuda)
    h = mq.ctypes.c_void_p()
    at, s = buf.data_ptr(), torch.cuda.current_stream().cuda_stream
    lib, f = mq.lib(), mq.FP4_FORMATS[fmt]
    assert lib.mq_fp4_pack_codes(at, at, at, 1, 1 << 30, 1 << 24, f, s, mq.ctypes.byref(h)) == mq.OUT_OF_MEMORY
    assert lib.mq_fp4_pack(at, 0, 1, 1 << 30, 1 << 24, f, s, mq.ctypes.byref(h)) == mq.OUT_OF_MEMORY
    assert not h.value
    assert (buf + 1).sum().item() == 1024
    W = values(40, 64, BF16, 1)
    same_bits(mq.Fp4Weight.pack(W.to(cuda), fmt).export(), W, fmt)


# ---------------------------------------------------------------- grouped
def grouped_check(mq, cuda, fmt, dtype, N, K, counts, lead=0, tail=0, index=None, x_rows=None, seed=0):
    E, R = len(counts), lead + sum(counts) + tail
    x_rows = R if index is None else x_rows
    X = values(x_rows, K, dtype, seed + 1, spread=0.3)
    W = values(E * N, K, BF16, seed + 2, spread=0.3).view(E, N, K)
    w = mq.Fp4Weight.pack(W.to(cuda), fmt)
    at = lead + np.concatenate([[0], np.cumsum(counts)])
    offsets = torch.tensor(at, dtype=torch.int32, device=cuda)
    Y = torch.full((R, N), 3.0, dtype=dtype, device=cuda)
    rows = None if index is None else torch.tensor(index, device=cuda)
    assert w.linear_grouped(X.to(cuda), offsets, Y, rows=rows) is Y
    assert (Y[:lead] == 3).all() and (Y[R - tail:] == 3).all()
    x64 = held(X, fmt)
    if index is not None:
        x64 = np.stack([x64[i] if 0 <= i < x_rows else np.zeros(K) for i in index])
    for e, c in enumerate(counts):
        if c:
            check_product(Y[at[e]:at[e + 1]], x64[at[e]:at[e + 1]], held(W[e], fmt), dtype)
    # rows quantised apart, the same bits
    q = mq.fp4_quantize(X.to(cuda), fmt, rows=rows)
    assert torch.equal(w.linear_grouped(q, offsets, torch.full_like(Y, 3.0), dtype=dtype), Y)
    assert w.device_error() == 0
    return w, X, offsets, Y


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("N,K,counts,lead,tail", [
    (128, 256, [1], 0, 0),
    (200, 100, [0, 3, 0, 1, 0], 0, 0),
    (130, 300, [5, 16, 17, 0, 1, 33], 2, 3),
    (64, 512, [0, 0, 0], 1, 2),
    (257, 64, [300, 0, 1, 129], 0, 1),
    (96, 768, [1] * 40, 0, 0),
    (384, 640, [64, 250, 7], 0, 0),
    (130, 260, [0] * 70 + [2, 0, 150] + [1] * 30, 4, 4),
    (256, 11008, [150, 30], 3, 1),
    (130, 8200, [0, 270, 20], 0, 5),
])
def test_grouped(mq, cuda, fmt, dtype, N, K, counts, lead, tail):
    grouped_check(mq, cuda, fmt, dtype, N, K, counts, lead, tail, seed=N)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("E,rows", [(300, 700), (2, 9000), (33, 5000)])
def test_grouped_many(mq, cuda, fmt, E, rows):
    # shares drawn at random, some of them empty, one of them half of all rows
    g = np.random.default_rng(E)
    cut = np.sort(g.integers(0, rows, E - 1))
    counts = np.diff(np.concatenate([[0], cut, [rows]]))
    counts[E // 2] += rows
    grouped_check(mq, cuda, fmt, BF16, 72, 192, counts.tolist(), lead=5, tail=7, seed=E)


@pytest.mark.parametrize("fmt", FMTS)
def test_grouped_index(mq, cuda, fmt):
    g = np.random.default_rng(1)
    index = g.integers(0, 30, 60)
    index[[4, 50]] = [-1, 30]  # rows of zeros
    grouped_check(mq, cuda, fmt, BF16, 140, 288, [10, 0, 35, 15], index=index.tolist(), x_rows=30)


@pytest.mark.parametrize("fmt", FMTS)
def test_grouped_equals_linear(mq, cuda, fmt):
    # one matrix with every row is the plain product
    X, W = values(70, 512, BF16, 1), values(300, 512, BF16, 2)
    w = mq.Fp4Weight.pack(W.to(cuda), fmt)
    Y = w.linear_grouped(X.to(cuda), torch.tensor([0, 70], device=cuda))
    check_product(Y, held(X, fmt), held(W, fmt), BF16)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("offsets", [[0, 50, 20, 60], [-5, 10, 10**6, 2**31 - 1], [60, 0, 0, 0], [70, 80, 90, 100],
                                     [0, -1, -1, 40]])
def test_grouped_bad_offsets_stay_inside(mq, cuda, fmt, offsets):
    # clamped on the device: no row of Y outside the clamped ranges is written
    R, N, K = 60, 96, 128
    w = mq.Fp4Weight.pack(values(3 * N, K, BF16, 1).view(3, N, K).to(cuda), fmt)
    out = torch.full((R + 8, N), 3.0, dtype=BF16, device=cuda)
    w.linear_grouped(values(R, K, BF16, 2).to(cuda), torch.tensor(offsets, dtype=torch.int32, device=cuda),
                     out[4:4 + R])
    torch.cuda.synchronize()
    mine = torch.zeros(R, dtype=torch.bool)
    for a, b in zip(offsets, offsets[1:]):
        a = min(max(a, 0), R)
        mine[a:min(max(b, a), R)] = True
    assert (out[:4] == 3).all() and (out[4 + R:] == 3).all()
    assert (out[4:4 + R][~mine.to(cuda)] == 3).all()
    assert w.device_error() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R", [9, 60, 900])
@pytest.mark.parametrize("E", [4, 70])
def test_grouped_descending_offsets(mq, cuda, fmt, R, E):
    # an entry below an earlier one counts as that one: no row belongs to two matrices
    N, K = 96, 300
    w = mq.Fp4Weight.pack(values(E * N, K, BF16, 1).view(E, N, K).to(cuda), fmt)
    X = values(R, K, BF16, 2).to(cuda)
    g = torch.Generator().manual_seed(R + E)
    offsets = torch.randint(-R // 4, R + R // 4, (E + 1,), generator=g).sort().values
    swap = torch.randint(0, E + 1, (E // 2,), generator=g)
    offsets[swap] = offsets[swap.flip(0)]
    offsets[0] = 0
    ascending = offsets.clamp(0, R).cummax(0).values
    want = torch.full((R, N), 3.0, dtype=BF16, device=cuda)
    w.linear_grouped(X, ascending.int().to(cuda), want)
    for x in (X, mq.fp4_quantize(X, fmt)):
        Y = torch.full_like(want, 3.0)
        w.linear_grouped(x, offsets.int().to(cuda), Y)
        assert torch.equal(Y, want)
    assert w.device_error() == 0


# ---------------------------------------------------------------- refusals on the device's side
def test_refusals(mq, cuda):
    w1 = mq.Fp4Weight.pack(values(64, 64, BF16, 1).to(cuda), "nvfp4")
    w2 = mq.Fp4Weight.pack(values(128, 64, BF16, 1).view(2, 64, 64).to(cuda), "nvfp4")
    M = 40  # enough that the product needs its workspace
    X = values(M, 64, BF16, 2).to(cuda)
    off = torch.tensor([0, 1, M], dtype=torch.int32, device=cuda)
    Y = torch.empty(M, 64, dtype=BF16, device=cuda)
    with pytest.raises(mq.MQError):
        w2.linear(X)                               # several matrices
    for call in (lambda: w1.linear(X.float()), lambda: w1.linear(X[:, :63]), lambda: w1.linear(X.cpu()),
                 lambda: w1.linear(X, Y[:3]), lambda: w1.linear(X, Y.half()), lambda: w1.linear(X, Y.t()),
                 lambda: w1.linear(X, dtype=FP16), lambda: w1.linear(mq.fp4_quantize(X, "mxfp4")),
                 lambda: w1.linear(mq.fp4_quantize(X), dtype=FP32),
                 lambda: w2.linear_grouped(X, off[:2]), lambda: w2.linear_grouped(X, off.float()),
                 lambda: w2.linear_grouped(X, off.cpu()), lambda: w2.linear_grouped(X, off, rows=off.cpu()),
                 lambda: w2.linear_grouped(mq.fp4_quantize(X), off, rows=off)):
        with pytest.raises(ValueError):
            call()
    small = torch.empty(w1.workspace_bytes(M) - 16, dtype=torch.uint8, device=cuda)
    with pytest.raises(mq.MQError):
        w1.linear(X, Y, small)
    with pytest.raises(mq.MQError):
        w1.linear(X, Y, torch.empty(w1.workspace_bytes(M) + 16, dtype=torch.uint8, device=cuda)[1:])
    lib = mq.lib()
    s = torch.cuda.current_stream().cuda_stream
    ws = torch.empty(w2.workspace_bytes(M), dtype=torch.uint8, device=cuda)
    args = [w2.handle, X.data_ptr(), 0, M, 64, None, M, off.data_ptr(), Y.data_ptr(), 64, ws.data_ptr(), ws.numel(), s]
    for k, bad, status in ((2, 2, 2), (4, 63, 1), (6, 3, 1), (7, None, 1), (7, off.data_ptr() + 1, 1), (8, None, 1),
                           (8, Y.data_ptr() + 1, 1), (9, 63, 1), (10, None, 1), (11, ws.numel() - 1, 1)):
        a = list(args)
        a[k] = bad
        assert lib.mq_fp4_linear_grouped(*a) == status, (k, bad)
    assert lib.mq_fp4_linear_grouped(*args) == 0
    torch.cuda.synchronize()


# ---------------------------------------------------------------- sizes past 32 bits
@pytest.mark.parametrize("fmt", FMTS)
def test_offsets_past_32_bits(mq, cuda, fmt):
    # X and Y of more than 2^32 bytes and 2^31 elements; only some rows are
    # not zeros
    M, N, K = 66000, 33000, 64
    X = torch.zeros(M, K, dtype=BF16, device=cuda)
    rows = torch.tensor([0, 40000, M - 1])
    X[rows] = values(3, K, BF16, 1, spread=0.3).to(cuda)
    W = values(N, K, BF16, 2, spread=0.3)
    w = mq.Fp4Weight.pack(W.to(cuda), fmt)
    Y = w.linear(X)
    assert Y.numel() > 2**31
    check_product(Y[rows.to(cuda)], held(X[rows.to(cuda)], fmt), held(W, fmt), BF16)
    live = torch.zeros(M, dtype=torch.bool, device=cuda)
    live[rows.to(cuda)] = True
    assert not Y[~live].any() and w.device_error() == 0
    del X, Y, live
    M, K = 140000, 32768
    X = torch.zeros(M, K, dtype=BF16, device=cuda)
    rows = torch.tensor([0, 65537, 131075, M - 1], device=cuda)
    X[rows] = values(4, K, BF16, 3).to(cuda)
    q = mq.fp4_quantize(X, fmt)
    assert X.numel() * 2 > 2**32 and q.codes.numel() > 2**31
    c, s, r = fp4.quantize(X[rows].float().cpu().numpy(), fmt)
    cb, sb = fp4.pack(c, s, fmt)
    assert np.array_equal(q.codes[rows].cpu().numpy(), cb) and np.array_equal(q.scales[rows].cpu().numpy(), sb)
    Y = q.dequantize(BF16)
    assert torch.equal(Y[rows], mq.fp4_quantize(X[rows], fmt).dequantize(BF16))


# ---------------------------------------------------------------- streams, graphs, layers
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 9, 40, 300])
def test_chain_without_waits(mq, cuda, fmt, M):
    # layers whose launches overlap: the same bits as one launch at a time,
    # with inputs that torch kernels write right before and overwrite right after
    D = 512
    ws = [mq.Fp4Weight.pack((values(D, D, BF16, k, spread=0.1) * 0.05).to(cuda), fmt) for k in range(6)]
    experts = mq.Fp4Weight.pack((values(4 * D, D, BF16, 9, spread=0.1) * 0.05).view(4, D, D).to(cuda), fmt)
    offsets = torch.tensor([0, M // 3, M // 3, M, M], dtype=torch.int32, device=cuda)
    start = values(M, D, BF16, 7, spread=0.2).to(cuda)

    def run(wait):
        sync = torch.cuda.synchronize if wait else (lambda: None)
        x, seen = start.clone(), []
        for step in range(8):
            for w in ws:
                y = w.linear(x)
                sync()
                x.copy_(y)
                sync()
            off = offsets.clone()
            y = experts.linear_grouped(x, off)
            sync()
            off.zero_()
            q = mq.fp4_quantize(y, fmt)
            sync()
            y.zero_()
            y = ws[0].linear(q)
            sync()
            seen.append(q.dequantize(BF16))
            x.copy_(y).mul_(0.5).add_(start)
            sync()
        torch.cuda.synchronize()
        return seen + [x]

    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", FMTS)
def test_beside_the_other_linears(mq, cuda, fmt):
    # this library's other products before and after on one stream, whose
    # launches overlap with these
    W = values(512, 512, FP32, 1, spread=0.1) * 0.05
    a, b = mq.Weight.pack(W.numpy(), 0.01), mq.Fp4Weight.pack(W.to(cuda), fmt)
    X = values(8, 512, BF16, 2, spread=0.2).to(cuda)

    def run(sync):
        x = X
        for _ in range(6):
            for f in (a.linear, b.linear, a.linear_w4a4, b.linear, b.linear):
                x = f(x)
                sync()
        torch.cuda.synchronize()
        return x

    assert torch.equal(run(torch.cuda.synchronize), run(lambda: None))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 9, 90, 300])
def test_chain_in_a_graph(mq, cuda, fmt, M):
    # launches that overlap, copies and fills between them, captured and
    # replayed with other inputs: the same bits as call by call
    D = 1024
    ws = [mq.Fp4Weight.pack((values(D, D, BF16, k, spread=0.1) * 0.04).to(cuda), fmt) for k in range(3)]
    experts = mq.Fp4Weight.pack((values(4 * D, D, BF16, 9, spread=0.1) * 0.04).view(4, D, D).to(cuda), fmt)
    given = values(M, D, BF16, 7, spread=0.2).to(cuda)
    cut = torch.tensor([0, M // 3, M // 3, M, M], dtype=torch.int32, device=cuda)
    x, y, off = torch.empty_like(given), torch.empty_like(given), torch.empty_like(cut)

    def step():
        x.copy_(given)
        off.copy_(cut)
        for w in ws:
            w.linear(x, y)
            x.copy_(y)
            y.zero_()
        experts.linear_grouped(x, off, y)
        off.zero_()
        x.zero_()
        q = mq.fp4_quantize(y, fmt)
        y.zero_()
        return ws[0].linear(q), q.dequantize(BF16)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for k in range(3):
        given.copy_(values(M, D, BF16, 20 + k, spread=0.2))
        cut.copy_(torch.tensor([0, M // 2, M, M, M] if k == 1 else [0, 0, M // 4, M // 2, M], dtype=torch.int32))
        g.replay()
        g.replay()
        have = [t.clone() for t in got]
        assert all(torch.equal(a, b) for a, b in zip(have, step()))
    assert all(w.device_error() == 0 for w in ws + [experts])


@pytest.mark.parametrize("fmt", FMTS)
def test_other_stream(mq, cuda, fmt):
    w = mq.Fp4Weight.pack(values(300, 256, BF16, 1).to(cuda), fmt)
    X = values(20, 256, BF16, 2).to(cuda)
    want = w.linear(X)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    Y = w.linear(X, stream=side)
    Z = w.linear(X.t().contiguous().t(), stream=side.cuda_stream)  # converted on that stream
    q = mq.fp4_quantize(X, fmt, stream=side)
    assert torch.cuda.current_stream() != side
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(Y, want) and torch.equal(Z, want) and torch.equal(q.codes, mq.fp4_quantize(X, fmt).codes)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 48, 700])
def test_two_streams_at_once(mq, cuda, fmt, M):
    w = mq.Fp4Weight.pack(values(2000, 1024, BF16, 1).to(cuda), fmt)
    Xs = [values(M, 1024, BF16, k).to(cuda) for k in range(2)]
    want = [w.linear(X) for X in Xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in Xs]
    got = [[], []]
    for _ in range(10):
        for k in range(2):
            got[k].append(w.linear(Xs[k], stream=streams[k]))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[k]) for k in range(2) for y in got[k])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [1, 30])
def test_graphs_that_share_a_workspace(mq, cuda, fmt, T):
    E, N, K = 4, 200, 320
    w = mq.Fp4Weight.pack(values(E * N, K, BF16, 1).view(E, N, K).to(cuda), fmt)
    lin = mq.Fp4Weight.pack(values(N, K, BF16, 3).to(cuda), fmt)
    ws = torch.empty(max(16, w.workspace_bytes(T), lin.workspace_bytes(T)), dtype=torch.uint8, device=cuda)
    X = values(T, K, BF16, 4).to(cuda)
    offsets = torch.tensor([0, 0, T, T, T], dtype=torch.int32, device=cuda)
    Y = [torch.zeros(T, N, dtype=BF16, device=cuda) for _ in range(2)]
    w.linear_grouped(X, offsets, Y[0], ws)
    lin.linear(X, Y[1], ws)
    torch.cuda.synchronize()
    graphs = []
    for call in (lambda: w.linear_grouped(X, offsets, Y[0], ws), lambda: lin.linear(X, Y[1], ws)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for k in range(3):
        X.copy_(values(T, K, BF16, 10 + k).to(cuda))
        offsets.copy_(torch.tensor([0, 0, T // 2, T, T] if k else [0, T, T, T, T], dtype=torch.int32))
        for g in graphs:
            g.replay()
        got = [y.clone() for y in Y]
        assert torch.equal(got[0], w.linear_grouped(X, offsets))
        assert torch.equal(got[1], lin.linear(X))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [1, 9, 200])
def test_experts_feed_forward(mq, cuda, fmt, T):
    # a layer of experts as a model runs it: route, up product of the gathered
    # rows, activation, down product, weighted sum back to the tokens
    E, top, D, H = 8, 2, 384, 640
    g = torch.Generator().manual_seed(T)
    X = values(T, D, BF16, T, spread=0.2).to(cuda)
    up = values(E * 2 * H, D, BF16, 1, spread=0.1).view(E, 2 * H, D) * 0.04
    down = values(E * D, H, BF16, 2, spread=0.1).view(E, D, H) * 0.04
    wu, wd = mq.Fp4Weight.pack(up.to(cuda), fmt), mq.Fp4Weight.pack(down.to(cuda), fmt)
    p, chosen = torch.randn(T, E, generator=g).softmax(-1).topk(top, dim=1)
    flat = chosen.flatten()
    order = torch.sort(flat, stable=True).indices
    offsets = torch.nn.functional.pad(torch.bincount(flat, minlength=E).cumsum(0), (1, 0)).to(cuda)
    rows = (order // top).to(cuda)
    h = wu.linear_grouped(X, offsets, rows=rows)
    a = torch.nn.functional.silu(h[:, :H].float()) * h[:, H:].float()
    a = a.to(BF16)
    y = wd.linear_grouped(a, offsets)
    out = torch.zeros(T, D, device=cuda)
    out.index_add_(0, rows, y.float() * p.flatten()[order].to(cuda)[:, None])
    # stage by stage, each from the bf16 input that its kernel had
    x64, a64 = held(X, fmt), held(a, fmt)
    at = offsets.tolist()
    want = np.zeros((T, D))
    for e in range(E):
        r = slice(at[e], at[e + 1])
        if at[e] == at[e + 1]:
            continue
        check_product(h[r], x64[rows.cpu().numpy()[r]], held(up[e], fmt), BF16)
        check_product(y[r], a64[r], held(down[e], fmt), BF16)
    np.add.at(want, rows.cpu().numpy(), y.double().cpu().numpy() * p.flatten()[order].double().numpy()[:, None])
    # index_add in fp32: two terms a token, each product and sum rounded once
    assert np.abs(out.cpu().double().numpy() - want).max() <= 4 * 2.0**-24 * np.abs(y.double().cpu().numpy()).max() * 2
