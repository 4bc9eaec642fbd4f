// Device helpers that the fp4 products share: where a tile lies, the store of
// an output, waits and arrivals across a cluster.
#pragma once

#include "common.cuh"
#include "fp4_convert.cuh"
#include "tc5.cuh"

namespace mq {

// ~1 ms, far beyond any copy's time: what a block that gave up a wait leaves
// its copies in flight to land before it hands its shared memory back.
constexpr long long kDrainCycles = 1 << 21;

__device__ __forceinline__ void drain_after_abort(const int *abort_flag) {
    if (!*reinterpret_cast<const volatile int *>(abort_flag)) return;
    const long long t0 = clock64();
    while (clock64() - t0 < kDrainCycles) {
    }
}

// An integer that an earlier launch may have written: the volatile load stays
// behind the wait for that launch.
__device__ __forceinline__ int load_i32(const int32_t *p) {
    int v;
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ float load_f32(const float *p) {
    float v;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t load_word(const uint32_t *p) {
    uint32_t v;
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t load_byte(const uint8_t *p) {
    uint32_t v;
    asm volatile("{\n\t.reg .u8 b;\n\tld.global.u8 b, [%1];\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ uint4 load_u128(const void *p) {
    uint4 v;
    asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint2 load_u64(const void *p) {
    uint2 v;
    asm volatile("ld.global.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
    return v;
}

// Tiles in order: matrix by matrix, each with ceil(rows / TT) token tiles for
// each of its NT row tiles; the token tiles of one row tile are neighbours,
// so that its codes come from L2 again. Each warp walks for itself (all lanes
// together) over ascending tile indices.
struct Tile {
    int e, m0, tokens, nt;
    int first;  // the matrix's first row
};

struct TileWalk {
    const int32_t *offsets;  // NULL: one matrix with all R rows
    int E, R, TT, NT;
    int base = 0;            // matrices [base, base + 32) hold the next tile, or later ones do
    int top = 0;             // where the matrices below base end
    long long before = 0;    // tiles of the matrices below base

    __device__ __forceinline__ TileWalk(const int32_t *o, int e, int r, int tt, int nt)
        : offsets(o), E(e), R(r), TT(tt), NT(nt) {}

    __device__ __forceinline__ bool find(long long t, Tile &out) {
        if (!offsets) {
            const int tiles = (R + TT - 1) / TT;
            if (t >= static_cast<long long>(tiles) * NT) return false;
            const int tt = static_cast<int>(t % tiles);
            out = {0, tt * TT, min(TT, R - tt * TT), static_cast<int>(t / tiles), 0};
            return true;
        }
        const int lane = threadIdx.x & 31;
        while (base < E) {
            const int e = base + lane;
            int a = R, b = R;
            if (e < E) {
                // entries out of range are clamped, never followed
                a = min(max(load_i32(offsets + e), 0), R);
                b = min(max(load_i32(offsets + e + 1), 0), R);
            }
            if (__any_sync(0xffffffffu, b < a || a < top)) {
                // out of order: an entry below an earlier one counts as that one
                a = max(a, top);
#pragma unroll
                for (int d = 1; d < 32; d *= 2) {
                    const int o = __shfl_up_sync(0xffffffffu, a, d);
                    if (lane >= d) a = max(a, o);
                }
                b = max(a, b);
            }
            const long long mine = static_cast<long long>((b - a + TT - 1) / TT) * NT;
            long long sum = mine;
#pragma unroll
            for (int d = 1; d < 32; d *= 2) {
                const long long o = __shfl_up_sync(0xffffffffu, sum, d);
                if (lane >= d) sum += o;
            }
            const uint32_t hit = __ballot_sync(0xffffffffu, t - before < sum);
            if (hit) {
                const int l = __ffs(hit) - 1;
                a = __shfl_sync(0xffffffffu, a, l);
                b = __shfl_sync(0xffffffffu, b, l);
                const long long within = t - before - __shfl_sync(0xffffffffu, sum - mine, l);
                const int tiles = (b - a + TT - 1) / TT;
                const int tt = static_cast<int>(within % tiles);
                out = {base + l, a + tt * TT, min(TT, b - a - tt * TT), static_cast<int>(within / tiles), a};
                return true;
            }
            before += __shfl_sync(0xffffffffu, sum, 31);
            top = __shfl_sync(0xffffffffu, b, 31);
            base += 32;
        }
        return false;
    }
};

__device__ __forceinline__ void store_output(void *Y, long long at, float y, bool fp16) {
    if (fp16)
        static_cast<__half *>(Y)[at] = __float2half_rn(y);
    else
        static_cast<__nv_bfloat16 *>(Y)[at] = __float2bfloat16_rn(y);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// v * f * w with a token's and a weight row's factor (at least 2^-100), two
// roundings: by the weight's first where that is at most 1, else last, so that
// nothing between overflows or underflows that the result does not.
__device__ __forceinline__ float apply_factor(float v, float f, float w) {
    return w <= 1.0f ? v * w * f : v * f * w;
}

// apply_factor for sixteen tokens; f: 16 bytes aligned.
__device__ __forceinline__ void apply_factors(float (&v)[16], const float *f, float w) {
    const bool small = w <= 1.0f;
    const uint64_t w2 = pack2(small ? w : 1.0f, small ? w : 1.0f);
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
        const ulonglong2 g = *reinterpret_cast<const ulonglong2 *>(f + j);
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            uint64_t d;
            asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pack2(v[j + i], v[j + i + 1])), "l"(w2));
            asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(d) : "l"(i ? g.y : g.x));
            v[j + i] = __uint_as_float(static_cast<uint32_t>(d));
            v[j + i + 1] = __uint_as_float(static_cast<uint32_t>(d >> 32));
        }
    }
    if (!small) {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] *= w;
    }
}

// Sixteen tokens' outputs of this lane's weight row, as 16-bit words ready to
// be stored. With `paired` (N, ldy and Y's address even) neighbouring lanes
// trade halves: even lanes then hold two rows of the even tokens, odd lanes
// two rows of the odd ones, 4 bytes a lane and two tokens a warp's store;
// without, a word holds two tokens of the lane's own row. Called by whole warps.
__device__ __forceinline__ void pack_chunk(const float (&v)[16], uint32_t (&w)[8], bool paired, bool fp16) {
    const uint32_t pick = threadIdx.x & 1 ? 0x3276u : 0x5410u;
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
        const uint32_t mine = fp16 ? pack_f16(v[j], v[j + 1]) : pack_bf16(v[j], v[j + 1]);
        w[j / 2] = paired ? __byte_perm(mine, __shfl_xor_sync(0xffffffffu, mine, 1), pick) : mine;
    }
}

// pack_chunk's words into Y [tokens][ldy]: tokens m .. m + 15, of which `left`
// are real, for row n (live: n < N).
__device__ __forceinline__ void store_packed(const uint32_t (&w)[8], void *Y, long long ldy, long long m, long long n,
                                             int left, bool live, bool paired) {
    if (!live) return;
    if (paired) {
        const int odd = threadIdx.x & 1;
        // ldy words of 4 bytes: two rows of 16-bit values
        uint32_t *y = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(Y) + (m + odd) * ldy + (n - odd));
        if (left >= 16) {
#pragma unroll
            for (int j = 0; j < 8; ++j, y += ldy) *y = w[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j, y += ldy)
                if (2 * j + odd < left) *y = w[j];
        }
        return;
    }
    uint16_t *y = static_cast<uint16_t *>(Y) + m * ldy + n;
#pragma unroll
    for (int j = 0; j < 16; ++j, y += ldy)
        if (j < left) *y = static_cast<uint16_t>(j & 1 ? w[j / 2] >> 16 : w[j / 2]);
}

__device__ __forceinline__ void store_chunk(const float (&v)[16], void *Y, long long ldy, long long m, long long n,
                                            int left, bool live, bool paired, bool fp16) {
    uint32_t w[8];
    pack_chunk(v, w, paired, fp16);
    store_packed(w, Y, ldy, m, n, left, live, paired);
}

// Bulk copy of `bytes` (a multiple of 16) into shared memory, completing on `bar`.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// The address, in the cluster's shared memory, of this CTA's `p` in CTA `rank`.
__device__ __forceinline__ uint32_t in_cta(const void *p, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}

// Arrives on a barrier given by in_cta. What this thread wrote for the tensor
// core in its own shared memory has to be fenced (fence_proxy_async) before.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Tiled load into this CTA's shared memory that completes on a barrier of
// either CTA of a pair (given by in_cta).
__device__ __forceinline__ void tma_pair_load_2d(void *dst, const CUtensorMap *map, uint32_t bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}

}  // namespace mq
