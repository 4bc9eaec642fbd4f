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
    Fp4Order order;
    bool open;
};

// A launch that may start while the one before it ends; its kernel waits for
// that one itself (pdl_wait).
template <class A>
cudaError_t launch_after(void (*kernel)(A), const A &args, dim3 grid, dim3 block, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args);
}

// ---------------------------------------------------------------- quantise
// blockDim = (bx, by): bx threads share a row, by rows side by side. A thread
// holds kChunks chunks of its row, all on their way from memory at once;
// wider rows are read twice by MQ_FP4_NV, whose row factor needs the whole row
// first.
template <class T, bool NV, int kChunks, bool kOrdered>
__global__ void __launch_bounds__(512) fp4_quantize_kernel(QuantArgs a) {
    // The launch after this one starts early: at once when all it looks at
    // before its own wait is a packed weight, else when the launches before
    // this one are over.
    if (a.open) pdl_launch_dependents();
    pdl_wait();
    if (!a.open) pdl_launch_dependents();
    __shared__ uint32_t wmax[16];
    const int bx = blockDim.x, tx = threadIdx.x, ty = threadIdx.y;
    const int chunks = static_cast<int>(NV ? a.spitch : a.spitch * 2);  // the scales' padding included
    const int code_chunks = static_cast<int>(a.cpitch / 8), real_chunks = static_cast<int>((a.from.K + kChunk - 1) / kChunk);
    const int whole_chunks = static_cast<int>(a.from.K / kChunk);
    const int step = bx * kChunks;
    const long long r = static_cast<long long>(blockIdx.x) * blockDim.y + ty;
    const bool real = r < a.rows;
    const T *src = nullptr;
    if (real) {
        const long long x = a.index ? static_cast<long long>(load_i32(a.index + r)) : r;
        if (x >= 0 && x < a.x_rows) src = static_cast<const T *>(a.X) + x * a.ldx;
    }
    const bool aligned = (reinterpret_cast<uintptr_t>(src) & 31) == 0;
    // where the row's scales go
    uint8_t *scales = a.scales + r * a.spitch;
    if constexpr (kOrdered) {
        long long slot = r / a.order.HT, x = r % a.order.HT;
        if (a.order.offsets && real) {
            // the last matrix that begins at or before the row; an entry below
            // an earlier one counts as that one
            int e = -1, first = 0;
            for (int base = 0; base < a.order.E; base += 32) {
                const int i = base + (tx & 31);
                const int at = i < a.order.E ? min(max(load_i32(a.order.offsets + i), 0), static_cast<int>(a.rows)) : 0;
                const uint32_t after = __ballot_sync(0xffffffffu, i >= a.order.E || at > r);
                const int n = after ? __ffs(after) - 1 : 32;
                e += n;
                first = max(first, __reduce_max_sync(0xffffffffu, (tx & 31) < n ? at : 0));
                if (n < 32) break;
            }
            slot = e < 0 ? -1 : first / a.order.HT + e + (r - first) / a.order.HT;
            x = (r - first) % a.order.HT;
        }
        scales = !real || slot < 0 ? nullptr
                                   : a.scales + slot * a.order.KS * (NV ? 4 : 2) * a.order.unit + (x >> 7) * 512 +
                                         (x & 31) * 16 + ((x >> 5) & 3) * 4;
    }
    auto load_one = [&](Raw<T> &t, int ch) {
        if (src && aligned && ch < whole_chunks)
            load_whole_chunk(t, src + ch * kChunk);
        else if (src && ch < real_chunks)
            load_chunk(t, a.from, src, static_cast<long long>(ch) * kChunk);
        else
            t.clear();
    };
    Raw<T> raw[kChunks];
    auto load = [&](int base) {
#pragma unroll
        for (int j = 0; j < kChunks; ++j) load_one(raw[j], base + tx + j * bx);
    };
    load(0);

    float factor = 0.0f, inverse = 0.0f;
    if constexpr (NV) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < kChunks; ++j) m = max(m, raw[j].max_bits());
        for (int base = step; base < chunks; base += step) {
#pragma unroll
            for (int j = 0; j < kChunks; ++j) {
                Raw<T> t;
                load_one(t, base + tx + j * bx);
                m = max(m, t.max_bits());
            }
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if (bx > 32) {
            const int warps = bx >> 5, lane = tx & 31;
            if (lane == 0) wmax[ty * warps + (tx >> 5)] = m;
            __syncthreads();
            m = __reduce_max_sync(0xffffffffu, lane < warps ? wmax[ty * warps + lane] : 0u);
        }
        factor = nv_factor<T>(m, inverse);
        if (tx == 0 && real) a.row_scale[r] = factor;
    }

    uint8_t *codes = a.codes + r * a.cpitch;
    for (int base = 0; base < chunks; base += step) {
        if (base > 0) load(base);
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
            const int ch = base + tx + j * bx;
            uint32_t top = raw[j].max_bits(), scale;
            float inv;
            if constexpr (NV) {
                scale = nv_scale<T>(top, factor, inverse, inv);
            } else {
                // lanes 2i and 2i + 1 hold the two halves of a block
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                scale = mx_scale<T>(top, inv);
            }
            if (ch >= real_chunks) scale = 0;
            if constexpr (kOrdered) {
                // four scales of a row are a word: 4 lanes' (8 lanes' of MQ_FP4_MX)
                constexpr int kLanes = NV ? 4 : 8;
                uint32_t word = scale << (8 * (NV ? tx & 3 : (tx >> 1) & 3));
                word |= __shfl_xor_sync(0xffffffffu, word, kLanes / 4);
                word |= __shfl_xor_sync(0xffffffffu, word, kLanes / 2);
                const int unit = ch / kLanes;  // units of a stage follow one another
                if (scales && (tx & (kLanes - 1)) == 0 && unit < a.order.KS * (NV ? 4 : 2))
                    *reinterpret_cast<uint32_t *>(scales + static_cast<long long>(unit) * a.order.unit) = word;
            }
            if (!real || ch >= chunks) continue;
            if (ch < code_chunks) *reinterpret_cast<uint2 *>(codes + ch * 8) = codes_of(raw[j], inv);
            if constexpr (kOrdered)
                continue;
            else if constexpr (NV)
                scales[ch] = static_cast<uint8_t>(scale);
            else if ((ch & 1) == 0)
                scales[ch >> 1] = static_cast<uint8_t>(scale);
        }
    }
}

template <class T, bool NV, int kChunks>
mq_status run_quantize(const QuantArgs &a, int bx, cudaStream_t stream) {
    const int by = std::max(1, 128 / bx);
    const long long grid = (a.rows + by - 1) / by;
    if (grid > 0x7FFFFFFFll) return fail(MQ_ERR_UNSUPPORTED, "fp4 quantisation: too many rows");
    cudaError_t e = cudaSuccess;
    if constexpr (sizeof(T) == 2)  // the products' types
        if (a.order.HT)
            e = launch_after(fp4_quantize_kernel<T, NV, kChunks, true>, a, dim3(static_cast<unsigned>(grid)), dim3(bx, by),
                             stream);
    if (!a.order.HT)
        e = launch_after(fp4_quantize_kernel<T, NV, kChunks, false>, a, dim3(static_cast<unsigned>(grid)), dim3(bx, by),
                         stream);
    if (e != cudaSuccess) return fp4_cuda_fail(e, "fp4 quantisation launch");
    return MQ_OK;
}

template <class T, bool NV>
mq_status pick_quantize(const QuantArgs &a, cudaStream_t stream) {
    const long long chunks = NV ? a.spitch : a.spitch * 2;
    auto threads = [&](int per) {
        return static_cast<int>(std::min<long long>(512, ((chunks + per - 1) / per + 31) / 32 * 32));
    };
    // Chunks a thread: one while all of them find a thread at once, two up to
    // some waves of that, then four (nvfp4, one / two / four: 999 x 2891 4.5 /
    // 5.1 / 6.7 us, 2048 x 4096 7.2 / 6.1 / 6.8 us, 8192 x 4096 23.0 / 17.8 /
    // 17.1 us); no more than a row has for a warp.
    const long long total = a.rows * chunks;
    if (chunks <= 32 || (chunks <= 512 && total <= 1350ll * sm_count())) return run_quantize<T, NV, 1>(a, threads(1), stream);
    if (chunks <= 64 || (chunks <= 1024 && total <= 7000ll * sm_count())) return run_quantize<T, NV, 2>(a, threads(2), stream);
    return run_quantize<T, NV, 4>(a, threads(4), stream);
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
// come out of two words and whose scales are at most two. Four units a thread
// (a block's width apart) are on their way at once.
template <class T, bool NV>
__global__ void __launch_bounds__(256) fp4_dequantize_kernel(DequantArgs a) {
    pdl_launch_dependents();
    pdl_wait();
    constexpr int kUnit = 16 / static_cast<int>(sizeof(T));
    constexpr int kShift = NV ? 4 : 5;  // log2 of the columns of a block
    constexpr int kUnits = 4;
    const long long r = static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (r >= a.rows) return;
    T *row = static_cast<T *>(a.Y) + r * a.ldy;
    const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    const uint32_t *words = reinterpret_cast<const uint32_t *>(a.codes + r * a.cpitch);
    const int nwords = static_cast<int>(a.cpitch / 4), K = static_cast<int>(a.K);
    const uint8_t *sc = a.scales + r * a.spitch;
    const float factor = NV ? load_f32(a.row_scale + r) : 1.0f;
    const int units = (K + lead + kUnit - 1) / kUnit;
    const int u0 = blockIdx.y * (blockDim.x * kUnits) + threadIdx.x;
    // Two codes' values as fp32 pairs: exact in f16, the products with an e4m3
    // scale too (6 of 11 bits), so that only the row's factor rounds.
    auto pair = [&](uint32_t byte, uint32_t scale_f16x2, float scale) {
        uint32_t h = e2m1_values(byte);
        if constexpr (NV) asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(h) : "r"(h), "r"(scale_f16x2));
        const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        uint64_t d;
        const float f = NV ? factor : scale;
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pack2(v.x, v.y)), "l"(pack2(f, f)));
        return make_float2(__uint_as_float(static_cast<uint32_t>(d)), __uint_as_float(static_cast<uint32_t>(d >> 32)));
    };
    auto twice = [](uint32_t s) {  // an e4m3 scale as f16x2
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<unsigned short>(s | s << 8)));
        return h;
    };
    if (lead == 0) {
        uint32_t code[kUnits], scale[kUnits];
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int u = min(u0 + i * static_cast<int>(blockDim.x), units - 1);
            const uint32_t w = load_word(words + u / (8 / kUnit));
            code[i] = kUnit == 8 ? w : w >> (16 * (u & 1));
            scale[i] = load_byte(sc + ((u * kUnit) >> kShift));
        }
#pragma unroll
        for (int i = 0; i < kUnits; ++i) {
            const int u = u0 + i * static_cast<int>(blockDim.x);
            if (u >= units) break;
            const uint32_t s2 = NV ? twice(scale[i]) : 0u;
            const float s = NV ? 0.0f : e8m0_value(scale[i]);
            uint32_t out[4];
#pragma unroll
            for (int k = 0; k < kUnit / 2; ++k) {
                const float2 v = pair(code[i] >> (8 * k), s2, s);
                if constexpr (std::is_same<T, float>::value) {
                    out[2 * k] = __float_as_uint(v.x);
                    out[2 * k + 1] = __float_as_uint(v.y);
                } else {
                    out[k] = std::is_same<T, __half>::value ? pack_f16(v.x, v.y) : pack_bf16(v.x, v.y);
                }
            }
            if ((u + 1) * kUnit <= K) {
                *reinterpret_cast<uint4 *>(row + u * kUnit) = make_uint4(out[0], out[1], out[2], out[3]);
            } else {
                const T *o = reinterpret_cast<const T *>(out);
#pragma unroll
                for (int k = 0; k < kUnit; ++k)
                    if (u * kUnit + k < K) row[u * kUnit + k] = o[k];
            }
        }
        return;
    }
    uint32_t code[kUnits], s0[kUnits], s1[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int u = min(u0 + i * static_cast<int>(blockDim.x), units - 1);
        const int c0 = u * kUnit - lead;  // negative in the first unit of a row with a lead
        const int w = c0 >> 3, sh = (c0 & 7) * 4;
        const uint32_t lo = w >= 0 ? load_word(words + w) : 0u;
        const uint32_t hi = sh && w + 1 < nwords ? load_word(words + w + 1) : 0u;
        code[i] = __funnelshift_r(lo, hi, sh);
        s0[i] = load_byte(sc + (max(c0, 0) >> kShift));
        s1[i] = load_byte(sc + ((min(c0 + kUnit, K) - 1) >> kShift));
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int u = u0 + i * static_cast<int>(blockDim.x);
        if (u >= units) break;
        const int c0 = u * kUnit - lead;
        // the second scale begins at this of the unit's columns, if at all
        const int edge = ((((max(c0, 0)) >> kShift) + 1) << kShift) - c0;
        const uint32_t a2 = NV ? twice(s0[i]) : 0u, b2 = NV ? twice(s1[i]) : 0u;
        const float af = NV ? 0.0f : e8m0_value(s0[i]), bf = NV ? 0.0f : e8m0_value(s1[i]);
        uint32_t out[4];
#pragma unroll
        for (int k = 0; k < kUnit / 2; ++k) {
            const uint32_t byte = code[i] >> (8 * k);
            // an odd lead lets the edge fall between the two
            float2 v = pair(byte, 2 * k < edge ? a2 : b2, 2 * k < edge ? af : bf);
            if (2 * k + 1 == edge) v.y = pair(byte, b2, bf).y;
            if constexpr (std::is_same<T, float>::value) {
                out[2 * k] = __float_as_uint(v.x);
                out[2 * k + 1] = __float_as_uint(v.y);
            } else {
                out[k] = std::is_same<T, __half>::value ? pack_f16(v.x, v.y) : pack_bf16(v.x, v.y);
            }
        }
        if (c0 >= 0 && c0 + kUnit <= K) {
            *reinterpret_cast<uint4 *>(row + c0) = make_uint4(out[0], out[1], out[2], out[3]);
        } else {
            const T *o = reinterpret_cast<const T *>(out);
#pragma unroll
            for (int k = 0; k < kUnit; ++k)
                if (c0 + k >= 0 && c0 + k < K) row[c0 + k] = o[k];
        }
    }
}

template <class T, bool NV>
mq_status run_dequantize(const DequantArgs &a, cudaStream_t stream) {
    const long long units = (a.K * static_cast<long long>(sizeof(T)) + 15) / 16 + 1;
    int bx = 32;
    while (bx < 256 && bx * 4 < units) bx *= 2;
    const int by = 256 / bx;
    const long long gx = (a.rows + by - 1) / by, gy = (units + bx * 4 - 1) / (bx * 4);
    if (gx > 0x7FFFFFFFll || gy > 65535) return fail(MQ_ERR_UNSUPPORTED, "fp4 dequantisation: too large");
    const cudaError_t e = launch_after(fp4_dequantize_kernel<T, NV>, a,
                                       dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), dim3(bx, by), stream);
    if (e != cudaSuccess) return fp4_cuda_fail(e, "fp4 dequantisation launch");
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
                              uint8_t *scales, float *row_scale, const Fp4Order &order, bool open,
                              cudaStream_t stream) {
    if (rows <= 0) return MQ_OK;
    const int64_t size = dtype == MQ_FP32 ? 4 : 2;
    QuantArgs a{X, ldx, x_rows, index, codes, scales, row_scale, rows, fp4_code_pitch(K), fp4_scale_pitch(fmt, K),
                {K, static_cast<const char *>(X), static_cast<const char *>(X) + ((x_rows - 1) * ldx + K) * size}, order,
                open};
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fp4_order_kernel, d.pieces, codes, scales, total,
                                             static_cast<long long>(d.N), static_cast<long long>(d.NT), d.KS, units,
                                             static_cast<long long>(fp4_code_pitch(d.K)),
                                             static_cast<long long>(fp4_scale_pitch(d.fmt, d.K)), to_rows);
    if (e != cudaSuccess) return fp4_cuda_fail(e, "fp4 order launch");
    return MQ_OK;
}

}  // namespace mq
