// C ABI of the microscaled 4-bit floating point calls (include/mosaicq.h,
// mq_fp4_*): validation, packing, workspaces and dispatch.

#include <cuda_runtime.h>

#include <new>
#include <string>

#include "fp4.h"
#include "kernels.h"

struct mq_fp4_weight {
    int device = -1;
    mq::Fp4Device d;
    int64_t device_bytes = 0;
    void *allocations[3];  // the first `allocated` of them
    int allocated = 0;
};

namespace mq {

mq_status fp4_cuda_fail(cudaError_t e, const char *what) {
    cudaGetLastError();
    return fail(e == cudaErrorMemoryAllocation ? MQ_ERR_OUT_OF_MEMORY : MQ_ERR_CUDA,
                std::string(what) + ": " + cudaGetErrorString(e));
}

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 30;  // rows, N, E * N
constexpr int64_t kMaxK = int64_t(1) << 24;

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

mq_status check_format(int fmt) {
    return fmt == MQ_FP4_MX || fmt == MQ_FP4_NV ? MQ_OK : fail(MQ_ERR_INVALID_ARG, "unknown fp4 format");
}

mq_status check_dtype(int dtype, bool fp32) {
    if (dtype == MQ_BF16 || dtype == MQ_FP16 || (fp32 && dtype == MQ_FP32)) return MQ_OK;
    if (dtype == MQ_FP32) return fail(MQ_ERR_UNSUPPORTED, "fp32 is served by mq_fp4_quantize and mq_fp4_dequantize only");
    return fail(MQ_ERR_INVALID_ARG, "unknown dtype");
}

mq_status check_k(int64_t K) {
    return K > 0 && K <= kMaxK ? MQ_OK : fail(MQ_ERR_INVALID_ARG, "K must be in [1, 2^24]");
}

// X of x_rows rows with stride ldx, `rows` of them taken (by index or in order)
mq_status check_input(const void *X, int dtype, int64_t rows, int64_t K, int64_t ldx, const int32_t *index,
                      int64_t x_rows) {
    if (rows < 0 || x_rows < 0) return fail(MQ_ERR_INVALID_ARG, "row counts must be >= 0");
    if (rows > kMaxRows || x_rows > kMaxRows) return fail(MQ_ERR_UNSUPPORTED, "more than 2^30 rows");
    if (ldx < K) return fail(MQ_ERR_INVALID_ARG, "ldx is smaller than K");
    if (ldx > (int64_t(1) << 40)) return fail(MQ_ERR_INVALID_ARG, "ldx too large");
    if (!index && rows != x_rows) return fail(MQ_ERR_INVALID_ARG, "without an index the row counts are the same");
    if (rows > 0 && !X && x_rows > 0) return fail(MQ_ERR_INVALID_ARG, "X is NULL");
    const uintptr_t mask = dtype == MQ_FP32 ? 3 : 1;
    if ((reinterpret_cast<uintptr_t>(X) & mask) || (reinterpret_cast<uintptr_t>(index) & 3))
        return fail(MQ_ERR_INVALID_ARG, "X or the index is not aligned to its elements");
    return MQ_OK;
}

mq_status check_quantized(const void *codes, const void *scales, const void *row_scale, int fmt) {
    if (!codes || !scales) return fail(MQ_ERR_INVALID_ARG, "codes or scales is NULL");
    if (fmt == MQ_FP4_NV && !row_scale) return fail(MQ_ERR_INVALID_ARG, "row_scale is NULL");
    if (!aligned16(codes) || !aligned16(scales)) return fail(MQ_ERR_INVALID_ARG, "codes and scales must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(row_scale) & 3) return fail(MQ_ERR_INVALID_ARG, "row_scale must be 4-byte aligned");
    return MQ_OK;
}

mq_status check_shape_fp4(int64_t E, int64_t N, int64_t K, int fmt) {
    if (mq_status st = check_format(fmt)) return st;
    if (mq_status st = check_k(K)) return st;
    if (E <= 0 || N <= 0) return fail(MQ_ERR_INVALID_ARG, "E and N must be positive");
    if (E > 65535 || N > kMaxRows || E * N > kMaxRows)
        return fail(MQ_ERR_UNSUPPORTED, "more than 65535 matrices or 2^30 rows");
    return MQ_OK;
}

// The weight's device buffers, left unwritten.
mq_status allocate(mq_fp4_weight *w, int64_t E, int64_t N, int64_t K, int fmt) {
    Fp4Device &d = w->d;
    d.E = E;
    d.N = N;
    d.K = K;
    d.fmt = fmt;
    d.device = w->device;
    d.sms = sm_count();
    d.KS = static_cast<int>((K + kFp4StageK - 1) / kFp4StageK);
    d.NT = (N + 127) / 128;
    if (mq_status st = fp4_count_clusters(d)) return st;
    auto get = [&](void **p, int64_t bytes) {
        const cudaError_t e = cudaMalloc(p, static_cast<size_t>(bytes));
        if (e != cudaSuccess) return fp4_cuda_fail(e, "cudaMalloc");
        w->allocations[w->allocated++] = *p;
        w->device_bytes += bytes;
        return MQ_OK;
    };
    const int64_t bytes = E * d.NT * d.KS * fp4_piece(fmt);
    if (mq_status st = get(reinterpret_cast<void **>(&d.pieces), bytes)) return st;
    if (fmt == MQ_FP4_NV)
        if (mq_status st = get(reinterpret_cast<void **>(&d.row_scale), E * N * 4)) return st;
    if (mq_status st = get(reinterpret_cast<void **>(&d.err), 4)) return st;
    if (!encode_bytes_map(&d.map, d.pieces, 128, bytes / 128, fp4_piece(fmt) / 128, false))
        return fail(MQ_ERR_CUDA, "cuTensorMapEncodeTiled failed for the weight");
    return MQ_OK;
}

mq_status new_weight(mq_fp4_weight **out) {
    int dev = -1;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fp4_cuda_fail(e, "no usable CUDA device");
    if (dev < 0 || dev >= 64) return fail(MQ_ERR_UNSUPPORTED, "device ordinal above 63");
    mq_fp4_weight *w = new (std::nothrow) mq_fp4_weight();
    if (!w) return fail(MQ_ERR_OUT_OF_MEMORY, "host allocation failed");
    w->device = dev;
    *out = w;
    return MQ_OK;
}

// The buffers of R quantised rows inside a workspace, whose size grows with R:
// one for a program's largest batch serves the smaller ones.
struct Workspace {
    int64_t factors, scales, total;
    Workspace(const Fp4Device &d, int64_t R) {
        factors = R * fp4_code_pitch(d.K);
        scales = factors + (d.fmt == MQ_FP4_NV ? (R * 4 + 127) / 128 * 128 : 0);
        total = scales + fp4_token_scale_bytes(d, R);
    }
};

mq_status check_device(const mq_fp4_weight *w) {
    int dev = -1;
    if (const cudaError_t e = cudaGetDevice(&dev)) return fp4_cuda_fail(e, "no usable CUDA device");
    if (dev != w->device)
        return fail(MQ_ERR_INVALID_ARG, "the current device is not the device that packed the weight");
    return MQ_OK;
}

mq_status check_output(const mq_fp4_weight *w, const void *Y, int dtype, int64_t ldy) {
    if (mq_status st = check_dtype(dtype, false)) return st;
    if (!Y) return fail(MQ_ERR_INVALID_ARG, "Y is NULL");
    if (reinterpret_cast<uintptr_t>(Y) & 1) return fail(MQ_ERR_INVALID_ARG, "Y is not aligned to its elements");
    if (ldy < w->d.N || ldy > (int64_t(1) << 40)) return fail(MQ_ERR_INVALID_ARG, "ldy is smaller than N or too large");
    return MQ_OK;
}

mq_status quantize_and_multiply(const mq_fp4_weight *w, const void *X, int dtype, int64_t x_rows, int64_t ldx,
                                const int32_t *index, int64_t R, const int32_t *offsets, void *Y, int64_t ldy,
                                void *workspace, size_t workspace_bytes, mq_stream stream) {
    const Fp4Device &d = w->d;
    if (mq_status st = check_dtype(dtype, false)) return st;
    if (mq_status st = check_input(X, dtype, R, d.K, ldx, index, x_rows)) return st;
    if (R == 0) return MQ_OK;
    if (mq_status st = check_output(w, Y, dtype, ldy)) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (fp4_linear_quantises(d, R)) {
        if (mq_status st = check_device(w)) return st;
        return launch_fp4_linear_direct(d, X, static_cast<mq_dtype>(dtype), R, ldx, index, x_rows, offsets, Y, ldy, s);
    }
    const Fp4Order order = fp4_token_order(d, R, offsets);
    const Workspace ws(d, R);
    if (!workspace || !aligned16(workspace)) return fail(MQ_ERR_INVALID_ARG, "the workspace is NULL or not 16-byte aligned");
    if (workspace_bytes < static_cast<size_t>(ws.total))
        return fail(MQ_ERR_INVALID_ARG, "workspace smaller than mq_fp4_workspace_bytes");
    if (mq_status st = check_device(w)) return st;
    uint8_t *base = static_cast<uint8_t *>(workspace);
    float *factors = d.fmt == MQ_FP4_NV ? reinterpret_cast<float *>(base + ws.factors) : nullptr;
    if (mq_status st = launch_fp4_quantize(X, static_cast<mq_dtype>(dtype), R, d.K, ldx, index, x_rows, d.fmt, base,
                                           base + ws.scales, factors, order, offsets == nullptr, s))
        return st;
    const Fp4Rows x{base, base + ws.scales, factors, R, order};
    return launch_fp4_linear(d, x, offsets, Y, static_cast<mq_dtype>(dtype), ldy, true, s);
}

mq_status multiply(const mq_fp4_weight *w, const void *codes, const void *scales, const float *row_scale, int64_t R,
                   const int32_t *offsets, void *Y, int dtype, int64_t ldy, mq_stream stream) {
    if (R < 0) return fail(MQ_ERR_INVALID_ARG, "row counts must be >= 0");
    if (R > kMaxRows) return fail(MQ_ERR_UNSUPPORTED, "more than 2^30 rows");
    if (R == 0) return MQ_OK;
    if (mq_status st = check_quantized(codes, scales, row_scale, w->d.fmt)) return st;
    if (mq_status st = check_output(w, Y, dtype, ldy)) return st;
    if (mq_status st = check_device(w)) return st;
    const Fp4Rows x{static_cast<const uint8_t *>(codes), static_cast<const uint8_t *>(scales), row_scale, R, {}};
    return launch_fp4_linear(w->d, x, offsets, Y, static_cast<mq_dtype>(dtype), ldy, false,
                             reinterpret_cast<cudaStream_t>(stream));
}

mq_status check_offsets(const int32_t *offsets) {
    if (!offsets) return fail(MQ_ERR_INVALID_ARG, "offsets is NULL");
    if (reinterpret_cast<uintptr_t>(offsets) & 3) return fail(MQ_ERR_INVALID_ARG, "offsets must be 4-byte aligned");
    return MQ_OK;
}

}  // namespace
}  // namespace mq

using namespace mq;

extern "C" {

int64_t mq_fp4_code_bytes(int64_t K) { return K > 0 && K <= kMaxK ? fp4_code_pitch(K) : 0; }

int64_t mq_fp4_scale_bytes(mq_fp4_format fmt, int64_t K) {
    return (fmt == MQ_FP4_MX || fmt == MQ_FP4_NV) && K > 0 && K <= kMaxK ? fp4_scale_pitch(fmt, K) : 0;
}

mq_status mq_fp4_quantize(const void *X, mq_dtype dtype, int64_t rows, int64_t K, int64_t ldx, const int32_t *index,
                          int64_t x_rows, mq_fp4_format fmt, void *codes, void *scales, float *row_scale,
                          mq_stream stream) {
    if (mq_status st = check_format(fmt)) return st;
    if (mq_status st = check_dtype(dtype, true)) return st;
    if (mq_status st = check_k(K)) return st;
    if (mq_status st = check_input(X, dtype, rows, K, ldx, index, x_rows)) return st;
    if (rows == 0) return MQ_OK;
    if (mq_status st = check_quantized(codes, scales, row_scale, fmt)) return st;
    return launch_fp4_quantize(X, dtype, rows, K, ldx, index, x_rows, fmt, static_cast<uint8_t *>(codes),
                               static_cast<uint8_t *>(scales), row_scale, {}, true, reinterpret_cast<cudaStream_t>(stream));
}

mq_status mq_fp4_dequantize(const void *codes, const void *scales, const float *row_scale, int64_t rows, int64_t K,
                            mq_fp4_format fmt, void *Y, mq_dtype dtype, int64_t ldy, mq_stream stream) {
    if (mq_status st = check_format(fmt)) return st;
    if (mq_status st = check_dtype(dtype, true)) return st;
    if (mq_status st = check_k(K)) return st;
    if (rows < 0) return fail(MQ_ERR_INVALID_ARG, "row counts must be >= 0");
    if (rows > kMaxRows) return fail(MQ_ERR_UNSUPPORTED, "more than 2^30 rows");
    if (rows == 0) return MQ_OK;
    if (mq_status st = check_quantized(codes, scales, row_scale, fmt)) return st;
    if (!Y) return fail(MQ_ERR_INVALID_ARG, "Y is NULL");
    if (reinterpret_cast<uintptr_t>(Y) & (dtype == MQ_FP32 ? 3 : 1))
        return fail(MQ_ERR_INVALID_ARG, "Y is not aligned to its elements");
    if (ldy < K || ldy > (int64_t(1) << 40)) return fail(MQ_ERR_INVALID_ARG, "ldy is smaller than K or too large");
    const Fp4Rows x{static_cast<const uint8_t *>(codes), static_cast<const uint8_t *>(scales), row_scale, rows, {}};
    return launch_fp4_dequantize(x, K, fmt, Y, dtype, ldy, reinterpret_cast<cudaStream_t>(stream));
}

void mq_fp4_free(mq_fp4_weight *w) {
    if (!w) return;
    int prev = -1;
    bool switched = false;
    if (w->device >= 0 && cudaGetDevice(&prev) == cudaSuccess && prev != w->device)
        switched = cudaSetDevice(w->device) == cudaSuccess;
    for (int i = 0; i < w->allocated; ++i) cudaFree(w->allocations[i]);
    if (switched) cudaSetDevice(prev);
    cudaGetLastError();  // nothing is reported from here, nothing is left behind
    delete w;
}

mq_status mq_fp4_pack_codes(const void *codes, const void *scales, const float *row_scale, int64_t E, int64_t N,
                            int64_t K, mq_fp4_format fmt, mq_stream stream, mq_fp4_weight **out) {
    if (!out) return fail(MQ_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    if (mq_status st = check_shape_fp4(E, N, K, fmt)) return st;
    if (mq_status st = check_quantized(codes, scales, row_scale, fmt)) return st;
    mq_fp4_weight *w = nullptr;
    if (mq_status st = new_weight(&w)) return st;
    mq_status st = allocate(w, E, N, K, fmt);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (!st) {
        const Fp4Device &d = w->d;
        if (d.row_scale)
            e = cudaMemcpyAsync(d.row_scale, row_scale, E * N * 4, cudaMemcpyDeviceToDevice, s);
        if (e == cudaSuccess) e = cudaMemsetAsync(d.err, 0, 4, s);
        if (e != cudaSuccess) st = fp4_cuda_fail(e, "mq_fp4_pack_codes");
    }
    if (!st)
        st = launch_fp4_order(w->d, static_cast<uint8_t *>(const_cast<void *>(codes)),
                              static_cast<uint8_t *>(const_cast<void *>(scales)), false, s);
    if (!st && (e = cudaStreamSynchronize(s)) != cudaSuccess) st = fp4_cuda_fail(e, "mq_fp4_pack_codes");
    if (st) {
        mq_fp4_free(w);
        return st;
    }
    *out = w;
    return MQ_OK;
}

mq_status mq_fp4_pack(const void *W, mq_dtype dtype, int64_t E, int64_t N, int64_t K, mq_fp4_format fmt,
                      mq_stream stream, mq_fp4_weight **out) {
    if (!out) return fail(MQ_ERR_INVALID_ARG, "out is NULL");
    *out = nullptr;
    if (mq_status st = check_shape_fp4(E, N, K, fmt)) return st;
    if (mq_status st = check_dtype(dtype, true)) return st;
    if (!W) return fail(MQ_ERR_INVALID_ARG, "W is NULL");
    if (mq_status st = check_input(W, dtype, E * N, K, K, nullptr, E * N)) return st;
    mq_fp4_weight *w = nullptr;
    if (mq_status st = new_weight(&w)) return st;
    mq_status st = allocate(w, E, N, K, fmt);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // codes and scales row by row, on the way to their order
    uint8_t *rows = nullptr;
    const int64_t code_bytes = E * N * fp4_code_pitch(K);
    cudaError_t e = cudaSuccess;
    if (!st) {
        e = cudaMalloc(reinterpret_cast<void **>(&rows),
                       static_cast<size_t>(code_bytes + E * N * fp4_scale_pitch(fmt, K)));
        if (e == cudaSuccess) e = cudaMemsetAsync(w->d.err, 0, 4, s);
        if (e != cudaSuccess) st = fp4_cuda_fail(e, "mq_fp4_pack");
    }
    if (!st)
        st = launch_fp4_quantize(W, dtype, E * N, K, K, nullptr, E * N, fmt, rows, rows + code_bytes, w->d.row_scale,
                                 {}, false, s);
    if (!st) st = launch_fp4_order(w->d, rows, rows + code_bytes, false, s);
    if (rows) {
        e = cudaStreamSynchronize(s);
        if (!st && e != cudaSuccess) st = fp4_cuda_fail(e, "mq_fp4_pack");
        cudaFree(rows);
        cudaGetLastError();
    }
    if (st) {
        mq_fp4_free(w);
        return st;
    }
    *out = w;
    return MQ_OK;
}

mq_status mq_fp4_get_info(const mq_fp4_weight *w, mq_fp4_info *out) {
    if (!w || !out) return fail(MQ_ERR_INVALID_ARG, "NULL pointer");
    out->E = w->d.E;
    out->N = w->d.N;
    out->K = w->d.K;
    out->format = w->d.fmt;
    out->device = w->device;
    out->device_bytes = w->device_bytes;
    return MQ_OK;
}

mq_status mq_fp4_export(const mq_fp4_weight *w, void *codes, void *scales, float *row_scale, mq_stream stream) {
    if (!w) return fail(MQ_ERR_INVALID_ARG, "weight handle is NULL");
    const Fp4Device &d = w->d;
    if (mq_status st = check_quantized(codes, scales, row_scale, d.fmt)) return st;
    if (mq_status st = check_device(w)) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // the scales' padding past the last stage has no place in the pieces
    cudaError_t e = cudaMemsetAsync(scales, 0, d.E * d.N * fp4_scale_pitch(d.fmt, d.K), s);
    if (e == cudaSuccess && d.row_scale)
        e = cudaMemcpyAsync(row_scale, d.row_scale, d.E * d.N * 4, cudaMemcpyDeviceToDevice, s);
    if (e != cudaSuccess) return fp4_cuda_fail(e, "mq_fp4_export");
    return launch_fp4_order(d, static_cast<uint8_t *>(codes), static_cast<uint8_t *>(scales), true, s);
}

int64_t mq_fp4_workspace_bytes(const mq_fp4_weight *w, int64_t rows) {
    if (!w || rows <= 0 || rows > kMaxRows || fp4_linear_quantises(w->d, rows)) return 0;
    return Workspace(w->d, rows).total;
}

mq_status mq_fp4_linear(const mq_fp4_weight *w, const void *X, mq_dtype dtype, int64_t M, int64_t ldx, void *Y,
                        int64_t ldy, void *workspace, size_t workspace_bytes, mq_stream stream) {
    if (!w) return fail(MQ_ERR_INVALID_ARG, "weight handle is NULL");
    if (w->d.E != 1) return fail(MQ_ERR_INVALID_ARG, "the weight holds several matrices: use mq_fp4_linear_grouped");
    return quantize_and_multiply(w, X, dtype, M, ldx, nullptr, M, nullptr, Y, ldy, workspace, workspace_bytes, stream);
}

mq_status mq_fp4_linear_codes(const mq_fp4_weight *w, const void *codes, const void *scales, const float *row_scale,
                              int64_t M, void *Y, mq_dtype dtype, int64_t ldy, mq_stream stream) {
    if (!w) return fail(MQ_ERR_INVALID_ARG, "weight handle is NULL");
    if (w->d.E != 1) return fail(MQ_ERR_INVALID_ARG, "the weight holds several matrices: use mq_fp4_linear_grouped_codes");
    return multiply(w, codes, scales, row_scale, M, nullptr, Y, dtype, ldy, stream);
}

mq_status mq_fp4_linear_grouped(const mq_fp4_weight *w, const void *X, mq_dtype dtype, int64_t x_rows, int64_t ldx,
                                const int32_t *index, int64_t R, const int32_t *offsets, void *Y, int64_t ldy,
                                void *workspace, size_t workspace_bytes, mq_stream stream) {
    if (!w) return fail(MQ_ERR_INVALID_ARG, "weight handle is NULL");
    if (mq_status st = check_offsets(offsets)) return st;
    return quantize_and_multiply(w, X, dtype, x_rows, ldx, index, R, offsets, Y, ldy, workspace, workspace_bytes,
                                 stream);
}

mq_status mq_fp4_linear_grouped_codes(const mq_fp4_weight *w, const void *codes, const void *scales,
                                      const float *row_scale, int64_t R, const int32_t *offsets, void *Y,
                                      mq_dtype dtype, int64_t ldy, mq_stream stream) {
    if (!w) return fail(MQ_ERR_INVALID_ARG, "weight handle is NULL");
    if (mq_status st = check_offsets(offsets)) return st;
    return multiply(w, codes, scales, row_scale, R, offsets, Y, dtype, ldy, stream);
}

mq_status mq_fp4_device_error(const mq_fp4_weight *w, mq_stream stream, int32_t *code) {
    if (!w || !code) return fail(MQ_ERR_INVALID_ARG, "NULL pointer");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaStreamSynchronize(s);
    int v = 0;
    if (e == cudaSuccess) e = cudaMemcpy(&v, w->d.err, 4, cudaMemcpyDeviceToHost);
    if (e == cudaSuccess && v) e = cudaMemset(w->d.err, 0, 4);
    if (e != cudaSuccess) return fp4_cuda_fail(e, "mq_fp4_device_error");
    *code = v;
    return v ? fail(MQ_ERR_DEVICE_TIMEOUT, "a kernel gave up a bounded wait") : MQ_OK;
}

}  // extern "C"
