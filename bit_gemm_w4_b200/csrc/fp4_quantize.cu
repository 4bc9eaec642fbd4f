// Microscaled 4-bit floating point: quantisation of activations and weights,
// the way back, and the order of scales that the tensor cores take.
//
// A block of B columns shares one scale: MQ_FP4_MX has B = 32 and scale
// 2^(s - 127), MQ_FP4_NV has B = 16, an e4m3 scale and a 32-bit factor for
// the row. Both are decided in 32 bits with the roundings the header states,
// so that the codes are a function of the input alone.
//
// Both directions are bound by memory: quantising 16-bit X reads 2 bytes and
// writes 0.53 to 0.56 bytes an element.

#include <algorithm>

#include "common.cuh"
#include "fp4.h"
#include "fp4_convert.cuh"
#include "fp4_device.cuh"

namespace mq {
namespace {

struct QuantArgs {
    const void *X;
    long long ldx, x_rows;
    const int32_t *index;
    uint8_t *codes, *scales;
    float *row_scale;
    long long rows;
    long long cpitch, spitch;  // bytes of a row of codes, of scales
    RowSource from;
};

// ---------------------------------------------------------------- quantise
// blockDim = (bx, by): bx threads share a row, by rows side by side, kRows
// rows one after another in each thread's registers (their loads are issued
// together). A thread holds kChunks chunks of a row; wider rows are read
// twice by MQ_FP4_NV, whose row factor needs the whole row first.
template <class T, bool NV, int kChunks, int kRows>
__global__ void __launch_bounds__(512) fp4_quantize_kernel(const QuantArgs a) {
    // The launch after this one may start once the launches before are over.
    pdl_wait();
    pdl_launch_dependents();
    constexpr int kMaxWarps = 32;
    __shared__ uint32_t wmax[NV ? kRows * kMaxWarps : 1];
    const int bx = blockDim.x, tx = threadIdx.x, ty = threadIdx.y;
    const long long chunks = NV ? a.spitch : a.spitch * 2;  // the scales' padding included
    const long long step = static_cast<long long>(bx) * kChunks;
    const long long r0 = (static_cast<long long>(blockIdx.x) * blockDim.y + ty) * kRows;

    const T *src[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const long long r = r0 + i;
        src[i] = nullptr;
        if (r < a.rows) {
            const long long x = a.index ? static_cast<long long>(load_i32(a.index + r)) : r;
            if (x >= 0 && x < a.x_rows) src[i] = static_cast<const T *>(a.X) + x * a.ldx;
        }
    }
    Raw<T> raw[kRows][kChunks];
    auto load = [&](long long base) {
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
            for (int j = 0; j < kChunks; ++j) {
                const long long c = (base + tx + static_cast<long long>(j) * bx) * kChunk;
                if (src[i])
                    load_chunk(raw[i][j], a.from, src[i], c);
                else
                    raw[i][j].clear();
            }
    };
    load(0);

    float factor[kRows], inv_factor[kRows];
    if constexpr (NV) {
        uint32_t m[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            m[i] = 0;
#pragma unroll
            for (int j = 0; j < kChunks; ++j) m[i] = max(m[i], raw[i][j].max_bits());
        }
        for (long long base = step; base < chunks; base += step) {
#pragma unroll
            for (int i = 0; i < kRows; ++i)
#pragma unroll
                for (int j = 0; j < kChunks; ++j) {
                    Raw<T> t;
                    if (src[i])
                        load_chunk(t, a.from, src[i], (base + tx + static_cast<long long>(j) * bx) * kChunk);
                    else
                        t.clear();
                    m[i] = max(m[i], t.max_bits());
                }
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) m[i] = __reduce_max_sync(0xffffffffu, m[i]);
        if (bx > 32) {
            const int warps = bx >> 5, w0 = ty * warps;
            if ((tx & 31) == 0)
#pragma unroll
                for (int i = 0; i < kRows; ++i) wmax[i * kMaxWarps + w0 + (tx >> 5)] = m[i];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                const int l = tx & 31;
                m[i] = __reduce_max_sync(0xffffffffu, l < warps ? wmax[i * kMaxWarps + w0 + l] : 0u);
            }
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            factor[i] = nv_factor<T>(m[i], inv_factor[i]);
            if (tx == 0 && r0 + i < a.rows) a.row_scale[r0 + i] = factor[i];
        }
    }

    for (long long base = 0; base < chunks; base += step) {
        if (base > 0) load(base);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const long long r = r0 + i;
#pragma unroll
            for (int j = 0; j < kChunks; ++j) {
                const long long ch = base + tx + static_cast<long long>(j) * bx;
                uint32_t top = raw[i][j].max_bits();
                float inv;
                uint32_t sbits;
                if constexpr (NV) {
                    sbits = nv_scale<T>(top, factor[i], inv_factor[i], inv);
                } else {
                    // lanes 2i and 2i + 1 hold the two halves of a block
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    sbits = mx_scale<T>(top, inv);
                }
                if (r >= a.rows || ch >= chunks) continue;
                if (ch * 8 < a.cpitch)
                    *reinterpret_cast<uint2 *>(a.codes + r * a.cpitch + ch * 8) = codes_of(raw[i][j], inv);
                if (ch * kChunk >= a.from.K) sbits = 0;
                if constexpr (NV)
                    a.scales[r * a.spitch + ch] = static_cast<uint8_t>(sbits);
                else if ((ch & 1) == 0)
                    a.scales[r * a.spitch + (ch >> 1)] = static_cast<uint8_t>(sbits);
            }
        }
    }
}

template <class T, bool NV, int kChunks, int kRows>
mq_status run_quantize(const QuantArgs &a, int bx, int by, cudaStream_t stream) {
    const long long per = static_cast<long long>(by) * kRows;
    const long long grid = (a.rows + per - 1) / per;
    if (grid > 0x7FFFFFFFll) return fail(MQ_ERR_UNSUPPORTED, "fp4 quantisation: too many rows");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(bx, by);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fp4_quantize_kernel<T, NV, kChunks, kRows>, a);
    if (e != cudaSuccess)
        return fail(MQ_ERR_CUDA, std::string("fp4 quantisation launch: ") + cudaGetErrorString(e));
    return MQ_OK;
}

template <class T, bool NV>
mq_status pick_quantize(const QuantArgs &a, cudaStream_t stream) {
    const long long chunks = NV ? a.spitch : a.spitch * 2;
    int bx = 32;
    while (bx < 128 && bx < chunks) bx *= 2;
    const int by = 256 / std::max(bx, 128) * (bx < 128 ? 128 / bx : 1);
    if (chunks <= 128) return run_quantize<T, NV, 1, 1>(a, bx, by, stream);
    auto threads = [&](int per) {
        const long long n = (chunks + per - 1) / per;
        return static_cast<int>(std::min<long long>(512, (n + 31) / 32 * 32));
    };
    if (chunks <= 512) {
        if (a.rows >= 4ll * 4 * sm_count()) return run_quantize<T, NV, 1, 4>(a, threads(1), 1, stream);
        return run_quantize<T, NV, 1, 1>(a, threads(1), 1, stream);
    }
    if (chunks <= 1024) {
        if (a.rows >= 4ll * 2 * sm_count()) return run_quantize<T, NV, 2, 2>(a, threads(2), 1, stream);
        return run_quantize<T, NV, 2, 1>(a, threads(2), 1, stream);
    }
    return run_quantize<T, NV, 4, 1>(a, threads(4), 1, stream);
}

// ---------------------------------------------------------------- dequantise
struct DequantArgs {
    const uint8_t *codes, *scales;
    const float *row_scale;
    void *Y;
    long long ldy, rows, K, cpitch, spitch;
};

// A thread writes aligned 16-byte units of Y, whatever the row's start: the
// unit's columns are any run of 8 (16-bit types) or 4 (fp32), whose codes
// come out of two words and whose scales are at most two.
template <class T, bool NV>
__global__ void __launch_bounds__(256) fp4_dequantize_kernel(const DequantArgs a) {
    constexpr int kUnit = 16 / static_cast<int>(sizeof(T));
    constexpr int kBlock = NV ? 16 : 32;
    const long long r = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (r >= a.rows) return;
    T *row = static_cast<T *>(a.Y) + r * a.ldy;
    const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    const uint32_t *words = reinterpret_cast<const uint32_t *>(a.codes + r * a.cpitch);
    const long long nwords = a.cpitch / 4;
    const uint8_t *sc = a.scales + r * a.spitch;
    const float factor = NV ? __ldg(a.row_scale + r) : 1.0f;
    const long long units = (a.K + lead + kUnit - 1) / kUnit;
    auto scale = [&](long long b) {
        const uint32_t s = __ldg(sc + b);
        return NV ? e4m3_value(s) : e8m0_value(s);
    };
    for (long long u = static_cast<long long>(blockIdx.y) * blockDim.x + threadIdx.x; u < units;
         u += static_cast<long long>(gridDim.y) * blockDim.x) {
        const long long c0 = u * kUnit - lead;  // negative in the first unit of a row with a lead
        const long long w = c0 >> 3;
        const int sh = static_cast<int>(c0 & 7) * 4;
        const uint32_t lo = w >= 0 ? __ldg(words + w) : 0u;
        const uint32_t hi = sh && w + 1 < nwords ? __ldg(words + w + 1) : 0u;
        uint32_t h[4];
        e2m1_values(__funnelshift_r(lo, hi, sh), h);
        const long long first = max(c0, 0ll), last = min(c0 + kUnit, a.K) - 1;
        const long long b0 = first / kBlock, b1 = last / kBlock;
        const float s0 = scale(b0), s1 = b1 != b0 ? scale(b1) : s0;
        T out[kUnit];
#pragma unroll
        for (int i = 0; i < kUnit; ++i) {
            const __half2 p = *reinterpret_cast<const __half2 *>(&h[i >> 1]);
            float v = i & 1 ? __high2float(p) : __low2float(p);
            v = __fmul_rn(v, (c0 + i) / kBlock > b0 ? s1 : s0);
            if constexpr (NV) v = __fmul_rn(v, factor);
            if constexpr (std::is_same<T, float>::value)
                out[i] = v;
            else if constexpr (std::is_same<T, __half>::value)
                out[i] = __float2half_rn(v);
            else
                out[i] = __float2bfloat16_rn(v);
        }
        if (c0 >= 0 && c0 + kUnit <= a.K) {
            *reinterpret_cast<uint4 *>(row + c0) = *reinterpret_cast<const uint4 *>(out);
        } else {
#pragma unroll
            for (int i = 0; i < kUnit; ++i)
                if (c0 + i >= 0 && c0 + i < a.K) row[c0 + i] = out[i];
        }
    }
}

template <class T, bool NV>
mq_status run_dequantize(const DequantArgs &a, cudaStream_t stream) {
    const long long units = (a.K * static_cast<long long>(sizeof(T)) + 15) / 16 + 1;
    int bx = 32;
    while (bx < 256 && bx < units) bx *= 2;
    const int by = 256 / bx;
    const long long gx = (a.rows + by - 1) / by;
    // two units a thread, so that short rows and few rows still spread out
    const long long gy = std::max<long long>(1, std::min<long long>(64, units / (2 * bx)));
    if (gx > 0x7FFFFFFFll) return fail(MQ_ERR_UNSUPPORTED, "fp4 dequantisation: too many rows");
    fp4_dequantize_kernel<T, NV><<<dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), dim3(bx, by), 0,
                                   stream>>>(a);
    const cudaError_t e = cudaPeekAtLastError();
    if (e != cudaSuccess)
        return fail(MQ_ERR_CUDA, std::string("fp4 dequantisation launch: ") + cudaGetErrorString(e));
    return MQ_OK;
}

// ---------------------------------------------------------------- order
// Between row-major codes and scales and a weight's pieces: one thread for
// every (piece, row, 16-byte unit), eight codes units and the row's scale
// words by the unit's number.
__global__ void __launch_bounds__(256) fp4_order_kernel(uint8_t *pieces, uint8_t *codes, uint8_t *scales,
                                                        long long total, long long N, long long NT, int KS,
                                                        int units, long long cpitch, long long spitch, bool back) {
    const int piece_bytes = kFp4CodePiece + units * 512;
    for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
         i += static_cast<long long>(gridDim.x) * blockDim.x) {
        const int u = static_cast<int>(i & 7), row = static_cast<int>(i >> 3) & 127;
        long long k = i >> 10;  // piece
        uint8_t *piece = pieces + k * piece_bytes;
        const int ks = static_cast<int>(k % KS);
        k /= KS;
        const long long n = (k % NT) * 128 + row, e = k / NT;
        const long long col = static_cast<long long>(ks) * 128 + u * 16;
        uint4 *at = reinterpret_cast<uint4 *>(piece + row * 128 + ((u ^ (row & 7)) * 16));
        uint4 *from = reinterpret_cast<uint4 *>(codes + (e * N + n) * cpitch + col);
        const bool live = n < N && col < cpitch;
        if (!back)
            *at = live ? *from : make_uint4(0, 0, 0, 0);
        else if (live)
            *from = *at;
        if (u < units) {
            const long long scol = (static_cast<long long>(ks) * units + u) * 4;
            uint32_t *sat = reinterpret_cast<uint32_t *>(piece + kFp4CodePiece + u * 512 + (row & 31) * 16 + (row >> 5) * 4);
            uint32_t *sfrom = reinterpret_cast<uint32_t *>(scales + (e * N + n) * spitch + scol);
            const bool slive = n < N && scol < spitch;
            if (!back)
                *sat = slive ? *sfrom : 0u;
            else if (slive)
                *sfrom = *sat;
        }
    }
}

}  // namespace

mq_status launch_fp4_quantize(const void *X, mq_dtype dtype, int64_t rows, int64_t K, int64_t ldx,
                              const int32_t *index, int64_t x_rows, int fmt, uint8_t *codes,
                              uint8_t *scales, float *row_scale, cudaStream_t stream) {
    if (rows <= 0) return MQ_OK;
    const int64_t size = dtype == MQ_FP32 ? 4 : 2;
    QuantArgs a{X, ldx, x_rows, index, codes, scales, row_scale, rows, fp4_code_pitch(K), fp4_scale_pitch(fmt, K),
                {K, static_cast<const char *>(X), static_cast<const char *>(X) + ((x_rows - 1) * ldx + K) * size}};
    const bool nv = fmt == MQ_FP4_NV;
    switch (dtype) {
        case MQ_BF16: return nv ? pick_quantize<__nv_bfloat16, true>(a, stream) : pick_quantize<__nv_bfloat16, false>(a, stream);
        case MQ_FP16: return nv ? pick_quantize<__half, true>(a, stream) : pick_quantize<__half, false>(a, stream);
        case MQ_FP32: return nv ? pick_quantize<float, true>(a, stream) : pick_quantize<float, false>(a, stream);
    }
    return fail(MQ_ERR_INVALID_ARG, "unknown dtype");
}

mq_status launch_fp4_dequantize(const Fp4Rows &x, int64_t K, int fmt, void *Y, mq_dtype dtype,
                                int64_t ldy, cudaStream_t stream) {
    if (x.rows <= 0) return MQ_OK;
    DequantArgs a{x.codes, x.scales, x.row_scale, Y, ldy, x.rows, K, fp4_code_pitch(K),
                  fp4_scale_pitch(fmt, K)};
    const bool nv = fmt == MQ_FP4_NV;
    switch (dtype) {
        case MQ_BF16: return nv ? run_dequantize<__nv_bfloat16, true>(a, stream) : run_dequantize<__nv_bfloat16, false>(a, stream);
        case MQ_FP16: return nv ? run_dequantize<__half, true>(a, stream) : run_dequantize<__half, false>(a, stream);
        case MQ_FP32: return nv ? run_dequantize<float, true>(a, stream) : run_dequantize<float, false>(a, stream);
    }
    return fail(MQ_ERR_INVALID_ARG, "unknown dtype");
}

mq_status launch_fp4_order(const Fp4Device &d, uint8_t *codes, uint8_t *scales, bool to_rows, cudaStream_t stream) {
    const int units = fp4_stage_scales(d.fmt) / 4;
    const long long total = d.E * d.NT * d.KS * 1024;
    const long long blocks = std::min<long long>((total + 255) / 256, 32ll * sm_count());
    fp4_order_kernel<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(
        d.pieces, codes, scales, total, d.N, d.NT, d.KS, units, fp4_code_pitch(d.K), fp4_scale_pitch(d.fmt, d.K),
        to_rows);
    const cudaError_t e = cudaPeekAtLastError();
    if (e != cudaSuccess)
        return fail(MQ_ERR_CUDA, std::string("fp4 order launch: ") + cudaGetErrorString(e));
    return MQ_OK;
}

}  // namespace mq
