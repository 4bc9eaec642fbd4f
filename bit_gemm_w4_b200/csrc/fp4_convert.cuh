// Device side of the microscaled 4-bit formats: conversions, and sixteen
// elements of a row at a time from memory to codes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"

namespace mq {

constexpr int kChunk = 16;  // columns a thread holds at a time

// Where rows are read from: K columns, and the bytes the whole matrix occupies.
struct RowSource {
    long long K;
    const char *begin, *end;
};

// ---------------------------------------------------------------- conversions
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}

// Eight values to eight E2M1 codes, the first in the low nibble; rounded to
// nearest even, saturating at 6.
__device__ __forceinline__ uint32_t e2m1_x8(const float *v) {
    uint32_t d;
    asm("{\n\t.reg .b8 a, b, c, e;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 e, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, e};\n\t}"
        : "=r"(d)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return d;
}

// The two E2M1 codes of a byte (the low eight bits) to their values as f16x2
// (exact).
__device__ __forceinline__ uint32_t e2m1_values(uint32_t byte) {
    uint32_t h;
    asm("{\n\t.reg .b8 a;\n\tcvt.u8.u32 a, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(h) : "r"(byte));
    return h;
}

__device__ __forceinline__ uint32_t e4m3_bits(float v) {
    unsigned short d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(0.0f), "f"(v));
    return d & 0xFFu;
}

__device__ __forceinline__ float e4m3_value(uint32_t bits) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<unsigned short>(bits)));
    return __low2float(*reinterpret_cast<__half2 *>(&h));
}

// 2^(s - 127); 255 is NaN.
__device__ __forceinline__ float e8m0_value(uint32_t s) {
    return __uint_as_float(s == 0 ? 0x00400000u : s == 255 ? 0x7FC00000u : s << 23);
}

// ---------------------------------------------------------------- input
// Sixteen consecutive elements as raw words: 8 for the 16-bit types, 16 for
// fp32.
template <class T>
struct Raw {
    static constexpr int kWords = kChunk * static_cast<int>(sizeof(T)) / 4;
    uint32_t w[kWords];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    // The largest magnitude's bits, a NaN's where there is one (the order of
    // non-negative floats is the order of their bits).
    __device__ __forceinline__ uint32_t max_bits() const {
        if constexpr (sizeof(T) == 2) {
            uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
            for (int i = 1; i < kWords; ++i) m = max_abs2(m, w[i]);
            return max(m & 0xFFFFu, m >> 16);
        } else {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < kWords; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
            return m;
        }
    }
    // max(m, |v|) of two 16-bit elements, NaN if either is.
    static __device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t v) {
        uint32_t d;
        if constexpr (std::is_same<T, __nv_bfloat16>::value)
            asm("{\n\t.reg .b32 a;\n\tabs.bf16x2 a, %2;\n\tmax.NaN.bf16x2 %0, %1, a;\n\t}" : "=r"(d) : "r"(m), "r"(v));
        else
            asm("{\n\t.reg .b32 a;\n\tabs.f16x2 a, %2;\n\tmax.NaN.f16x2 %0, %1, a;\n\t}" : "=r"(d) : "r"(m), "r"(v));
        return d;
    }
    __device__ __forceinline__ float value(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        const uint32_t h = i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xFFFFu;
        return of_bits(h);
    }
    // An element's bits (as max_bits gives them) as fp32.
    static __device__ __forceinline__ float of_bits(uint32_t h) {
        if constexpr (sizeof(T) == 4) return __uint_as_float(h);
        if constexpr (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(h << 16);
        return half_bits_to_f32(h);
    }
};

// Plain loads, not the read-only ones: a launch that started before the one
// that writes X was over may not take X for read-only.
__device__ __forceinline__ uint4 ldg128(const char *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Columns c .. c + 15 of the row at `row`, zeros past K. Rows on 16-byte
// boundaries are read as they are. Others (a 16-bit type with an odd stride,
// a view) are read in the aligned 16-byte units that cover the chunk, which
// lie inside X, and shifted into place; the units that stick out of X at
// either end, and the last partial chunk, go element by element.
template <class T>
__device__ __forceinline__ void load_chunk(Raw<T> &r, const RowSource &a, const T *row, long long c) {
    if (c >= a.K) {
        r.clear();
        return;
    }
    const char *p = reinterpret_cast<const char *>(row + c);
    if (c + kChunk <= a.K) {
        const uint32_t phase = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15);
        if (phase == 0) {
#pragma unroll
            for (int i = 0; i < Raw<T>::kWords / 4; ++i) {
                const uint4 v = ldg128(p + 16 * i);
                r.w[4 * i] = v.x;
                r.w[4 * i + 1] = v.y;
                r.w[4 * i + 2] = v.z;
                r.w[4 * i + 3] = v.w;
            }
            return;
        }
        if constexpr (sizeof(T) == 2) {
            const char *q = p - phase;
            if (q >= a.begin && q + 48 <= a.end) {
                uint32_t t[12];
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    uint4 v;
                    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                 : "l"(q + 16 * i));
                    t[4 * i] = v.x;
                    t[4 * i + 1] = v.y;
                    t[4 * i + 2] = v.z;
                    t[4 * i + 3] = v.w;
                }
                // whole words, then half a word
                if (phase & 8) {
#pragma unroll
                    for (int i = 0; i < 10; ++i) t[i] = t[i + 2];
                }
                if (phase & 4) {
#pragma unroll
                    for (int i = 0; i < 9; ++i) t[i] = t[i + 1];
                }
                const uint32_t sh = (phase & 2) * 8;
#pragma unroll
                for (int i = 0; i < 8; ++i) r.w[i] = __funnelshift_r(t[i], t[i + 1], sh);
                return;
            }
        }
    }
    r.clear();
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
        if (c + i >= a.K) break;
        if constexpr (sizeof(T) == 4) {
            asm volatile("ld.global.b32 %0, [%1];" : "=r"(r.w[i]) : "l"(row + c + i));
        } else {
            unsigned short h;
            asm volatile("ld.global.b16 %0, [%1];" : "=h"(h) : "l"(row + c + i));
            r.w[i >> 1] |= static_cast<uint32_t>(h) << (16 * (i & 1));
        }
    }
}

// The same for a whole chunk on a 32-byte boundary.
template <class T>
__device__ __forceinline__ void load_whole_chunk(Raw<T> &r, const T *p) {
#pragma unroll
    for (int i = 0; i < Raw<T>::kWords / 8; ++i)
        asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r.w[8 * i]), "=r"(r.w[8 * i + 1]), "=r"(r.w[8 * i + 2]), "=r"(r.w[8 * i + 3]),
                       "=r"(r.w[8 * i + 4]), "=r"(r.w[8 * i + 5]), "=r"(r.w[8 * i + 6]), "=r"(r.w[8 * i + 7])
                     : "l"(p + i * (32 / sizeof(T))));
}

// ---------------------------------------------------------------- decisions
// All in 32 bits, one rounding an operation, in the order the header states.

// MQ_FP4_NV: a row's factor from the bits of its largest magnitude; NaN for a
// row that is not finite, whose reciprocal then reads as 0.
template <class T>
__device__ __forceinline__ float nv_factor(uint32_t top_bits, float &inverse) {
    const float top = Raw<T>::of_bits(top_bits);
    const bool finite = top <= 3.402823466e38f;
    const float f = fmaxf(__fmul_rn(top, static_cast<float>(1.0 / 2688.0)), 0x1p-100f);
    inverse = finite ? __frcp_rn(f) : 0.0f;
    return finite ? f : __uint_as_float(0x7FC00000u);
}

// The scale byte of a block from its largest magnitude's bits, and what its
// elements are multiplied by (0: codes 0).
template <class T>
__device__ __forceinline__ uint32_t nv_scale(uint32_t top_bits, float factor, float inverse, float &inv) {
    const float t = __fmul_rn(__fmul_rn(Raw<T>::of_bits(top_bits), static_cast<float>(1.0 / 6.0)), inverse);
    const uint32_t s = inverse > 0.0f ? e4m3_bits(t) : 0u;
    inv = s ? __frcp_rn(__fmul_rn(e4m3_value(s), factor)) : 0.0f;
    return s;
}
template <class T>
__device__ __forceinline__ uint32_t mx_scale(uint32_t top_bits, float &inv) {
    const uint32_t e = __float_as_uint(Raw<T>::of_bits(top_bits)) >> 23;
    const bool finite = e < 255;
    const uint32_t s = e > 2 ? e - 2 : 0;
    inv = finite ? __uint_as_float((254u - s) << 23) : 0.0f;
    return finite ? s : 255u;
}

// Sixteen codes, the first in the low nibble; zeros where inv is 0 (which
// also keeps what an infinity or a NaN times 0 gives out).
template <class T>
__device__ __forceinline__ uint2 codes_of(const Raw<T> &raw, float inv) {
    float v[kChunk];
    const uint64_t i2 = pack2(inv, inv);
#pragma unroll
    for (int k = 0; k < kChunk; k += 2) {
        uint64_t d;
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pack2(raw.value(k), raw.value(k + 1))), "l"(i2));
        v[k] = __uint_as_float(static_cast<uint32_t>(d));
        v[k + 1] = __uint_as_float(static_cast<uint32_t>(d >> 32));
    }
    const uint32_t keep = inv == 0.0f ? 0u : 0xFFFFFFFFu;
    return make_uint2(e2m1_x8(v) & keep, e2m1_x8(v + 8) & keep);
}

}  // namespace mq
