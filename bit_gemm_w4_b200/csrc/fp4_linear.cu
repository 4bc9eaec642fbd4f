// Products with a microscaled 4-bit weight, narrow form: few tokens, where
// the weight's bytes from HBM and the latency of a launch are the bound.
//
//   Y[r][n] = fx[r] * fw[n] * sum_k (cx[r][k] sx[r][k / B]) (cw[n][k] sw[n][k / B])
//
// The weight is the MMA's A operand (128 rows a tile), the tokens its B
// operand (16 to 128 columns), so that a single token fills a tile of the
// tensor core; block scales are applied inside the MMA and the 32-bit row
// factors (MQ_FP4_NV) when Y is stored. One CTA computes one tile over a share
// of K; the CTAs of a cluster share a tile, push their partial sums into the
// shared memory of the CTA that owns the rows, and each owner adds them in
// rank order, so that results do not depend on timing.
//
// Warp 0 copies codes and weight scales (TMA), warp 1 issues scale copies to
// tensor memory and MMAs, warps 2 to 9 bring what the tokens need and are the
// epilogue. The tokens come in two forms: quantised before (their codes by
// TMA, their row-major scales placed in the tensor core's order by warps 2 to
// 9), or as they are, quantised by warps 2 to 9 on the way into shared memory,
// which saves a launch and the round through memory where few tokens would be
// quantised by every CTA alike.

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "fp4.h"
#include "fp4_convert.cuh"
#include "fp4_device.cuh"
#include "tc5.cuh"

namespace mq {
namespace {

constexpr int kThreads = 320;
constexpr int kFeeders = 256;  // threads of warps 2 to 9
constexpr int kMaxStages = 8;
constexpr int kBoxRows = 16;   // tokens of one copy
constexpr int kMaxTT = 128;  // what a scale unit holds

struct NarrowParams {
    CUtensorMap tx;
    const uint8_t *pieces;
    const float *wfactor;
    const uint8_t *xscales;  // quantised tokens
    const float *xfactor;
    long long xspitch;
    const void *X;           // tokens as they are
    long long ldx, x_rows;
    const int32_t *index;
    RowSource from;
    const int32_t *offsets;
    void *Y;
    long long ldy;
    int *err;
    long long N;
    int NT, KS, E, R;
    int TT;      // tokens of a tile, a multiple of 16
    int split;   // CTAs that share a tile (the cluster)
    int stages;  // ring slots
    int fp16;    // Y's type
    int paired;  // N, the stride and Y's address are even: 4-byte stores
    int wait_first;
};

// Shared memory: the ring (a piece of the weight, the tokens' codes and scales
// in each slot), partial sums from the cluster, factors, barriers.
template <bool NV>
struct NarrowSmem {
    static constexpr int kUnits = NV ? 4 : 2;  // 512-byte scale units of 128 rows in a stage
    static constexpr int kScales = kUnits * 512;
    static constexpr int kPiece = kFp4CodePiece + kScales;
    __host__ __device__ static int slot(int TT) { return kPiece + TT * 128 + kScales; }
    __host__ __device__ static int width(int split) { return (128 + split - 1) / split; }
    __host__ __device__ static int recv(int TT, int split) {
        return split > 1 ? (split * width(split) * TT * 4 + 127) / 128 * 128 : 0;
    }
    // Partial sums of up to 32 tokens have room of their own; more go where
    // the ring was, once every CTA of the cluster is done with it.
    __host__ __device__ static bool apart(int TT) { return TT <= 32; }
    __host__ __device__ static int fixed(int TT, int split) {
        return (apart(TT) ? recv(TT, split) : 0) + kMaxTT * 12 + 512 + 256 + 1024;
    }
    __host__ __device__ static int total(int TT, int split, int stages) { return slot(TT) * stages + fixed(TT, split); }
};

// T: void for tokens quantised before, else their type.
template <bool NV, class T>
__global__ void __launch_bounds__(kThreads, 2) fp4_narrow_kernel(const __grid_constant__ NarrowParams p) {
    using S = NarrowSmem<NV>;
    constexpr bool kQuantise = !std::is_same<T, void>::value;
    constexpr int kUnits = S::kUnits;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int TT = p.TT, stages = p.stages, slot = S::slot(TT);
    const int split = p.split, rank = split > 1 ? static_cast<int>(cluster_rank()) : 0;
    const int at_b = S::kPiece, at_sb = at_b + TT * 128;
    float *recv = reinterpret_cast<float *>(smem + (S::apart(TT) ? slot * stages : 0));
    float *factors =
        reinterpret_cast<float *>(smem + slot * stages + (S::apart(TT) ? S::recv(TT, split) : 0));  // [TT]
    uint32_t *tops = reinterpret_cast<uint32_t *>(factors + kMaxTT);                        // [TT]
    int *sources = reinterpret_cast<int *>(tops + kMaxTT);                                  // [TT]
    float *wfactors = reinterpret_cast<float *>(sources + kMaxTT);                          // [128]
    uint64_t *full = reinterpret_cast<uint64_t *>(wfactors + 128);
    uint64_t *empty = full + kMaxStages, *done = empty + kMaxStages;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
    int *abort_flag = reinterpret_cast<int *>(tmem_slot + 1);

    if (split > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], 1 + kFeeders / 32);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_mbar_init();
        if constexpr (!kQuantise) prefetch_tensormap(&p.tx);
    }
    if constexpr (kQuantise)
        if (threadIdx.x >= 64)
            for (int i = threadIdx.x - 64; i < TT; i += kFeeders) tops[i] = 0;
    if (p.wait_first) pdl_wait();  // the offsets may come from the launch just before
    // Tensor memory for the accumulator and both operands' scales (two CTAs of
    // an SM share 512 columns). Only with it in hand may whatever follows on the
    // stream start: that waits for this launch before it reads anything but
    // packed weights, and may take the rest of the tensor memory before. (The
    // allocation takes 330 cycles; chains of calls of 3.4 to 8.5 us take -0.2 to
    // 0.2 us more than with a start ahead of it.)
    const uint32_t tmem_cols = TT + 8 * kUnits <= 128 ? 128 : 256;
    if (warp == 1) {
        tc5::alloc<1>(tmem_slot, tmem_cols);
        if (lane == 0) pdl_launch_dependents();
        __syncwarp();
    }
    Tile t{0, 0, 0, 0, 0};
    TileWalk walk(p.offsets, p.E, p.R, TT, p.NT);
    const bool live = walk.find(blockIdx.x / split, t);  // the same in every CTA of a cluster
    const int m0 = t.m0, tokens = t.tokens, n0 = t.nt * 128;
    const int nb = (tokens + kBoxRows - 1) / kBoxRows;
    const int k0 = static_cast<int>(static_cast<long long>(p.KS) * rank / split);
    const int nk = static_cast<int>(static_cast<long long>(p.KS) * (rank + 1) / split) - k0;
    const int ahead = min(stages, nk);  // stages that fill the ring without waiting
    auto weight = [&](int i, int s) {
        mbar_arrive_expect_tx(&full[s], S::kPiece + (kQuantise ? 0 : nb * kBoxRows * 128));
        bulk_load(smem + s * slot,
                  p.pieces + ((static_cast<long long>(t.e) * p.NT + t.nt) * p.KS + k0 + i) * S::kPiece, S::kPiece,
                  &full[s]);
    };
    // the weight does not depend on the launch before: its first stages go ahead
    if (warp == 0) {
        __syncwarp();
        if (live && tc5::elect())
            for (int i = 0; i < ahead; ++i) weight(i, i);
        __syncwarp();
    }
    if constexpr (NV)
        if (threadIdx.x >= 64 && threadIdx.x < 64 + 128 && live) {
            const int row = threadIdx.x - 64;
            wfactors[row] = n0 + row < p.N ? __ldg(p.wfactor + static_cast<long long>(t.e) * p.N + n0 + row) : 0.0f;
        }
    tc5::fence_before();
    __syncthreads();
    tc5::fence_after();
    const uint32_t tmem = *tmem_slot;

    if (!live) {
        // nothing to do
    } else if (warp == 0) {
        auto tokens_in = [&](int i, int s) {
            for (int b = 0; b < nb; ++b)
                tma_load_2d(smem + s * slot + at_b + b * kBoxRows * 128, &p.tx, &full[s], (k0 + i) * 128,
                            m0 + b * kBoxRows);
        };
        pdl_wait();  // the launch before may take its time: no wait with a limit before this
        if constexpr (!kQuantise) {
            if (tc5::elect())
                for (int i = 0; i < ahead; ++i) tokens_in(i, i);
            __syncwarp();
        }
        bool ok = true;
        for (int i = ahead, s = 0, ph = 0; i < nk && ok; ++i) {
            ok = mbar_wait(&empty[s], ph, p.err, kErrWaitEmpty, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (tc5::elect()) {
                weight(i, s);
                if constexpr (!kQuantise) tokens_in(i, s);
            }
            __syncwarp();
            if (++s == stages) s = 0, ph ^= 1;
        }
    } else if (warp == 1) {
        const uint32_t desc = tc5::idesc(128, nb * kBoxRows, !NV);
        const uint32_t sfa = tmem + TT, sfb = sfa + 4 * kUnits;
        bool ok = true;
        pdl_wait();  // as above
        for (int i = 0, s = 0, ph = 0; i < nk && ok; ++i) {
            ok = mbar_wait(&full[s], ph, p.err, kErrWaitFull, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc5::fence_after();
            const uint32_t at = smem_u32(smem) + s * slot;
            const uint32_t sa = at + kFp4CodePiece, sb = at + at_sb;
            const uint64_t da = tc5::operand_desc(at), db = tc5::operand_desc(at + at_b);
            if (tc5::elect()) {
#pragma unroll
                for (int u = 0; u < kUnits; ++u) {
                    tc5::copy_scales<1>(sfa + 4 * u, tc5::scale_desc(sa + 512 * u));
                    tc5::copy_scales<1>(sfb + 4 * u, tc5::scale_desc(sb + 512 * u));
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int u = NV ? k : k >> 1;
                    const uint32_t byte = NV ? 0 : (k & 1) * 2;
                    tc5::mma<1, NV>(tmem, da + 2 * k, db + 2 * k, desc | tc5::idesc_scale_byte(byte), sfa + 4 * u,
                                    sfb + 4 * u, i > 0 || k > 0);
                }
                tc5::commit(&empty[s]);
            }
            __syncwarp();
            if (++s == stages) s = 0, ph ^= 1;
        }
        if (tc5::elect()) tc5::commit(done);
        __syncwarp();
    } else {
        const int tid = threadIdx.x - 64;
        // a stage's tokens are written: order that before the tensor core's reads
        auto hand_over = [&](int s) {
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[s]);
        };
        pdl_wait();
        if constexpr (kQuantise) {
            if (tid < tokens) sources[tid] = p.index ? load_i32(p.index + m0 + tid) : m0 + tid;
            asm volatile("bar.sync 1, %0;" ::"n"(kFeeders) : "memory");
            auto chunk = [&](int r, long long c) {
                Raw<T> raw;
                const long long x = sources[r];
                const T *row = static_cast<const T *>(p.X) + x * p.ldx;
                if (x < 0 || x >= p.x_rows)
                    raw.clear();
                else if ((reinterpret_cast<uintptr_t>(row) & 31) == 0 && c + kChunk <= p.from.K)
                    load_whole_chunk(raw, row + c);
                else
                    load_chunk(raw, p.from, row, c);
                return raw;
            };
            if constexpr (NV) {
                // the rows' largest magnitudes over all of K, a warp a row, or
                // the warps shared out over a few rows
                const int chunks = static_cast<int>((p.from.K + kChunk - 1) / kChunk);
                const int parts = tokens == 1 ? 8 : tokens == 2 ? 4 : tokens <= 4 ? 2 : 1;
                for (int x = warp - 2; x < tokens * parts; x += kFeeders / 32) {
                    const int r = x / parts;
                    uint32_t m = 0;
#pragma unroll 8
                    for (int c = (x - r * parts) * 32 + lane; c < chunks; c += 32 * parts)
                        m = max(m, chunk(r, static_cast<long long>(c) * kChunk).max_bits());
                    m = __reduce_max_sync(0xffffffffu, m);
                    if (lane == 0) atomicMax(&tops[r], m);
                }
                asm volatile("bar.sync 1, %0;" ::"n"(kFeeders) : "memory");
                if (tid < tokens) {
                    float inverse;
                    factors[tid] = nv_factor<T>(tops[tid], inverse);
                }
            }
            const int per = tokens * 16;  // chunks of a stage
            auto read = [&](int i, int w) {
                Raw<T> raw;
                raw.clear();
                if (w < per) raw = chunk(w >> 4, static_cast<long long>(k0 + i) * kFp4StageK + (w & 15) * kChunk);
                return raw;
            };
            // chunk w of a stage into slot s; called by whole warps, w >= per does nothing
            auto place = [&](const Raw<T> &raw, int s, int w) {
                const int r = w < per ? w >> 4 : 0, c = w & 15;
                uint8_t *at = smem + s * slot;
                uint32_t top = raw.max_bits(), scale;
                int unit = c >> 2, byte = c & 3;
                float inv;
                if constexpr (NV) {
                    float inverse;
                    const float factor = nv_factor<T>(tops[r], inverse);
                    scale = nv_scale<T>(top, factor, inverse, inv);
                } else {
                    // lanes 2i and 2i + 1 hold the two halves of a block
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    scale = mx_scale<T>(top, inv);
                    unit = c >> 3, byte = (c >> 1) & 3;
                }
                if (w >= per) return;
                at[at_sb + unit * 512 + r * 16 + byte] = static_cast<uint8_t>(scale);
                // 16-byte unit c / 2 of the row, under the 128-byte swizzle
                *reinterpret_cast<uint2 *>(at + at_b + r * 128 + (((c >> 1) ^ (r & 7)) * 16) + (c & 1) * 8) =
                    codes_of(raw, inv);
            };
            // stages that need no slot to be given back: all their chunks at once
            for (int x = tid; x - lane < ahead * per; x += kFeeders) {
                const int i = min(x / per, ahead), w = i < ahead ? x - i * per : per + (x & 1);
                place(read(i, w), i < ahead ? i : 0, w);
            }
            for (int i = 0; i < ahead; ++i) hand_over(i);
            // the others one by one, a stage's elements read ahead of its turn;
            // a thread has at most one chunk of up to 16 tokens
            Raw<T> next;
            if (ahead < nk) next = read(ahead, tid);
            for (int i = ahead, s = 0, ph = 0; i < nk; ++i) {
                const Raw<T> now = next;
                if (i + 1 < nk) next = read(i + 1, tid);
                if (!mbar_wait_warp(&empty[s], ph, p.err, kErrWaitEmpty, abort_flag)) break;
                place(now, s, tid);
                hand_over(s);
                if (++s == stages) s = 0, ph ^= 1;
            }
        } else {
            if constexpr (NV)
                for (int r = tid; r < tokens; r += kFeeders) factors[r] = load_f32(p.xfactor + m0 + r);
            // scales: a row's of four stages (64 or 32 bytes) are read in one
            // go, one group of stages ahead of their turn
            constexpr int kGroup = 4, kVecs = NV ? 4 : 2;
            uint4 next[kVecs];
            auto fetch = [&](int i) {
                if (tid >= tokens) return;
                const uint8_t *src = p.xscales + (m0 + tid) * p.xspitch + static_cast<long long>(k0 + i) * (4 * kUnits);
                if constexpr (NV) {
#pragma unroll
                    for (int v = 0; v < kVecs; ++v)
                        if (i + v < nk) next[v] = load_u128(src + 16 * v);
                } else {
                    // an 8-byte step: two stages may lie across 16-byte units
#pragma unroll
                    for (int v = 0; v < kGroup; ++v)
                        if (i + v < nk) {
                            const uint2 w = load_u64(src + 8 * v);
                            if (v & 1)
                                next[v >> 1].z = w.x, next[v >> 1].w = w.y;
                            else
                                next[v >> 1].x = w.x, next[v >> 1].y = w.y;
                        }
                }
            };
            fetch(0);
            int s = 0, ph = 1;
            bool ok = true;
            for (int i = 0; i < nk && ok; i += kGroup) {
                uint4 now[kVecs];
#pragma unroll
                for (int v = 0; v < kVecs; ++v) now[v] = next[v];
                if (i + kGroup < nk) fetch(i + kGroup);
#pragma unroll
                for (int j = 0; j < kGroup; ++j) {
                    if (i + j >= nk) break;
                    ok = mbar_wait_warp(&empty[s], ph, p.err, kErrWaitEmpty, abort_flag);
                    if (!ok) break;
                    if (tid < tokens) {
                        uint32_t *dst =
                            reinterpret_cast<uint32_t *>(smem + s * slot + at_sb + (tid & 31) * 16 + (tid >> 5) * 4);
                        if constexpr (NV) {
                            dst[0] = now[j].x;
                            dst[128] = now[j].y;
                            dst[256] = now[j].z;
                            dst[384] = now[j].w;
                        } else {
                            dst[0] = j & 1 ? now[j >> 1].z : now[j >> 1].x;
                            dst[128] = j & 1 ? now[j >> 1].w : now[j >> 1].y;
                        }
                    }
                    hand_over(s);
                    if (++s == stages) s = 0, ph ^= 1;
                }
            }
        }
    }
    __syncwarp();

    // ------------------------------------------------------------ epilogue
    if (split > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // every CTA has started
    const int first = 128 * rank / split, width = 128 * (rank + 1) / split - first;  // the rows this CTA adds up
    const int W = S::width(split);
    if (live && warp >= 2) {
        asm volatile("bar.sync 1, %0;" ::"n"(kFeeders) : "memory");  // the factors are written
        mbar_wait_warp(done, 0, p.err, kErrWaitMma, abort_flag);
        tc5::fence_after();
    }
    if (split > 1 && !S::apart(TT)) {
        __syncwarp();
        cluster_sync();
    }
    if (live && warp >= 2) {
        const int quad = warp & 3, row = quad * 32 + lane;
        const long long n = n0 + row;
        const int owner = ((row + 1) * split - 1) / 128;
        uint32_t to = 0;
        if (split > 1) to = in_cta(recv + rank * TT * W + row - 128 * owner / split, owner);
        // two warps share a quarter of the lanes: every other chunk of tokens each
        for (int c = 16 * ((warp - 2) >> 2); c < tokens; c += 32) {
            uint32_t bits[16];
            tc5::load16(tmem + (static_cast<uint32_t>(quad) << 21) + c, bits);
            tc5::load_wait();
            const int left = tokens - c;
            if (split > 1) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (j < left)
                        asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(to + (c + j) * W * 4), "r"(bits[j])
                                     : "memory");
                continue;
            }
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(bits[j]);
            if constexpr (NV) apply_factors(v, factors + c, wfactors[row]);
            store_chunk(v, p.Y, p.ldy, m0 + c, n, left, n < p.N, p.paired, p.fp16);
        }
    }
    drain_after_abort(abort_flag);
    __syncwarp();
    if (split > 1) {
        cluster_sync();  // every partial sum has arrived; nobody reaches into another CTA after this
        if (live && warp >= 2) {
            for (int i = threadIdx.x - 64; i < tokens * width; i += kFeeders) {
                const int m = i / width, w = i - m * width;
                const long long n = n0 + first + w;
                float part[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) part[r] = r < split ? recv[(r * TT + m) * W + w] : 0.0f;
                float y = part[0];
#pragma unroll
                for (int r = 1; r < 8; ++r) y += part[r];  // those past `split` are zeros
                if constexpr (NV) y = apply_factor(y, factors[m], wfactors[first + w]);
                if (n < p.N) store_output(p.Y, (m0 + m) * p.ldy + n, y, p.fp16);
            }
        }
    }
    pdl_wait();  // a launch is not over before the one it was chained to
    tc5::fence_before();
    __syncthreads();
    if (warp == 1) {
        tc5::fence_after();
        tc5::dealloc<1>(tmem, tmem_cols);
    }
}

// Ring slots of a CTA that shares its SM with `each` - 1 others.
int narrow_stages(int fmt, int TT, int split, int each) {
    const int room = (each == 2 ? 113 : 227) * 1024;
    return std::min(kMaxStages, fmt == MQ_FP4_NV
                                    ? (room - NarrowSmem<true>::fixed(TT, split)) / NarrowSmem<true>::slot(TT)
                                    : (room - NarrowSmem<false>::fixed(TT, split)) / NarrowSmem<false>::slot(TT));
}

// How a product is run, from its sizes alone (the rows of each matrix are not
// known to the host: `per` is their average).
struct Choice {
    int TT;          // tokens of a narrow tile; 0: the wide form
    int split;       // CTAs that share a narrow tile
    int each;        // narrow CTAs that share an SM
    int64_t likely;  // narrow tiles of the matrices that have rows
    int64_t per;     // rows of a matrix that has some
};

Choice choose(const Fp4Device &d, int64_t rows, bool grouped) {
    const int64_t mats = grouped ? std::min<int64_t>(d.E, rows) : 1, per = (rows + mats - 1) / mats;
    const int64_t sms = d.sms;
    const int64_t likely = mats * d.NT;
    const int TT = per <= 16 ? 16 : per <= 32 ? 32 : per <= 64 ? 64 : static_cast<int>((per + 15) / 16 * 16);
    // Times below: us on the device, calls in a row over weights that L2 does not
    // hold, quantisation included, nvfp4 unless another format is named.
    // K is split as far as that gives every SM at most one CTA (1 x 4096 x 4096,
    // 32 tiles: 7.6, 6.3, 6.5 and 6.8 with 2, 4, 6 and 8). For one token of 75 to
    // 148 tiles that is less than would be best: 1 x 11008 x 4096 (86 tiles) takes
    // 10.9, 9.5, 8.8 and 13.6 with 1 to 4.
    int split = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({8, d.KS, sms / likely})));
    // CTAs of up to 16 tokens share an SM, so that the next launch's may start
    // beside them. More tokens leave a CTA its SM, and a ring of up to eight
    // slots, as long as all clusters run at once that way: the SMs' groups hold
    // only so many (148, 74, 45, 33, 26, 22, 15, 15 of 1 to 8 CTAs), and the others
    // wait for the first to end (24 x 2048 x 2048, 16 tiles: 9.4 with 8 CTAs a
    // cluster, 6.3 with 6). Where they do not, up to 32 tokens two share an SM if
    // each then has four slots, which nvfp4 with partial sums has not; else K is
    // split less. One an SM and two: 24 x 11008 x 4096 (86 tiles) 10.2 and 11.8, 24
    // x 28672 x 8192 (224) 32.2 and 25.9; mxfp4 24 x 11008 x 4096 8.9 and 10.4, 48
    // x 8192 x 8192 13.8 and 16.1. (Up to 16 tokens too a lone CTA would be better
    // for large layers, 1 x 16384 x 8192 16.1 and 18.5, and worse for small ones,
    // 1 x 4096 x 4096 6.8 and 6.3.)
    int each = per <= 16 ? 2 : 1;
    while (each == 1 && likely > d.clusters[split]) {
        if (per <= 32 && narrow_stages(d.fmt, TT, split, 2) >= 4)
            each = 2;
        else if (split > 1)
            --split;
        else
            break;
    }
    // Up to 32 tokens: narrow, as long as its tiles run in one wave of two CTAs
    // an SM (mxfp4 16 x 28672 x 8192, 224 tiles: 23.5, wide 28.0; 192 rows over 64
    // experts of 2048 x 2048, 1024 tiles: 34.2, wide 32.1). Up to 128: where
    // splitting K, which the wide form does not do, takes enough stages off a
    // CTA to pay for the sum, whose time goes with the tokens. Narrow and wide:
    // 80 x 4096 x 11008 (43 stages, 11 a CTA) 13.7 and 19.0, 128 tokens 16.0 and
    // 20.5; 80 x 1024 x 4096 (16, 2) 8.1 and 9.3, 128 tokens 9.7 and 9.8; 48 x 4096
    // x 4096 (16, 4) 8.8 and 9.7, 80 tokens 10.4 and 10.2. Not with a second tile
    // of tokens, whose clusters find no room (192 x 4096 x 11008 27.3 and 21.0).
    const int64_t saved = d.KS - (d.KS + split - 1) / split;
    const bool narrow = per <= 32 ? likely <= 2 * sms : per <= kMaxTT && 6 * saved >= per;
    return {narrow ? TT : 0, split, each, likely, per};
}

template <bool NV, class T>
mq_status run_narrow(const Fp4Device &d, NarrowParams &p, int64_t rows, const Choice &c, bool chained,
                     cudaStream_t stream) {
    using S = NarrowSmem<NV>;
    p.TT = c.TT;
    // the most tiles that any split of the rows into matrices makes
    const int64_t tiles = (p.offsets ? std::min<int64_t>(d.E, rows) + rows / p.TT : (rows + p.TT - 1) / p.TT) * d.NT;
    p.split = c.split;
    if (tiles * p.split > 0x7FFFFFFFll) return fail(MQ_ERR_UNSUPPORTED, "fp4 linear: too many tiles");
    p.stages = narrow_stages(d.fmt, p.TT, p.split, c.each);
    const int smem = S::total(p.TT, p.split, p.stages);
    p.pieces = d.pieces;
    p.wfactor = d.row_scale;
    p.err = d.err;
    p.N = d.N;
    p.NT = static_cast<int>(d.NT);
    p.KS = d.KS;
    p.E = static_cast<int>(d.E);
    p.R = static_cast<int>(rows);
    p.wait_first = p.offsets && !chained;
    p.paired = d.N % 2 == 0 && p.ldy % 2 == 0 && (reinterpret_cast<uintptr_t>(p.Y) & 3) == 0;
    static bool configured[64] = {};
    if (!configured[d.device]) {
        if (const cudaError_t e = cudaFuncSetAttribute(fp4_narrow_kernel<NV, T>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024))
            return fp4_cuda_fail(e, "fp4 linear: device setup");
        configured[d.device] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * p.split));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int na = 0;
    if (p.split > 1) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = p.split;
        attr[na].val.clusterDim.y = 1;
        attr[na].val.clusterDim.z = 1;
        ++na;
    }
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
    cfg.attrs = attr;
    cfg.numAttrs = na;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fp4_narrow_kernel<NV, T>, p);
    if (e != cudaSuccess) return fp4_cuda_fail(e, "fp4 linear launch");
    return MQ_OK;
}

}  // namespace

mq_status launch_fp4_linear(const Fp4Device &d, const Fp4Rows &x, const int32_t *offsets, void *Y,
                            mq_dtype dtype, int64_t ldy, bool chained, cudaStream_t stream) {
    if (x.rows <= 0) return MQ_OK;
    const Choice c = choose(d, x.rows, d.E > 1);
    if (!c.TT) return launch_fp4_wide(d, x, offsets, Y, dtype, ldy, chained, stream);
    NarrowParams p{};
    if (!encode_bytes_map(&p.tx, x.codes, fp4_code_pitch(d.K), x.rows, kBoxRows, true))
        return fail(MQ_ERR_CUDA, "cuTensorMapEncodeTiled failed for the activations");
    p.xscales = x.scales;
    p.xfactor = x.row_scale;
    p.xspitch = fp4_scale_pitch(d.fmt, d.K);
    p.offsets = offsets;
    p.Y = Y;
    p.ldy = ldy;
    p.fp16 = dtype == MQ_FP16;
    return d.fmt == MQ_FP4_NV ? run_narrow<true, void>(d, p, x.rows, c, chained, stream)
                              : run_narrow<false, void>(d, p, x.rows, c, chained, stream);
}

template <bool NV>
static mq_status count_clusters(Fp4Device &d) {
    // asked for once a device: it does not change
    static std::mutex lock;
    static int counts[64][9] = {};
    const std::lock_guard<std::mutex> hold(lock);
    int *of = counts[d.device];
    if (!of[1]) {
        const auto kernel = fp4_narrow_kernel<NV, void>;
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        for (int size = 8; size > 0 && e == cudaSuccess; --size) {
            cudaLaunchAttribute attr = {};
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = size;
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(size * d.sms);
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = 227 * 1024;  // one CTA an SM
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&of[size], kernel, &cfg);
        }
        if (e != cudaSuccess) {
            of[1] = 0;
            return fp4_cuda_fail(e, "fp4 weight: device setup");
        }
    }
    std::copy(of, of + 9, d.clusters);
    return MQ_OK;
}

mq_status fp4_count_clusters(Fp4Device &d) {
    return d.fmt == MQ_FP4_NV ? count_clusters<true>(d) : count_clusters<false>(d);
}

// Ordered for the wide form, whose four loader warps then have nothing to
// place: 2048 x 14336 x 4096 nvfp4 takes 62 us instead of 76 us, 4096 x 4096 x
// 11008 mxfp4 98 us instead of 102 us (with the quantisation). Not for many
// matrices with few rows each, whose slots would be mostly empty.
static bool ordered(const Fp4Device &d, int64_t rows, int HT) { return d.E <= 8 * (rows / HT) + 256; }

static Fp4Order token_order(const Fp4Device &d, int64_t rows, int HT) {
    Fp4Order o;
    o.HT = HT;
    o.unit = fp4_scale_unit(HT);
    o.KS = d.KS;
    o.slots = rows / HT + d.E + 1;
    o.E = static_cast<int>(d.E);
    return o;
}

Fp4Order fp4_token_order(const Fp4Device &d, int64_t rows, const int32_t *offsets) {
    if (choose(d, rows, d.E > 1).TT) return {};
    const Fp4WidePlan plan = fp4_wide_plan(d, rows);
    const int HT = plan.TT / plan.halves;
    if (!ordered(d, rows, HT)) return {};
    Fp4Order o = token_order(d, rows, HT);
    o.offsets = offsets;
    return o;
}

int64_t fp4_token_scale_bytes(const Fp4Device &d, int64_t rows) {
    int64_t most = rows * fp4_scale_pitch(d.fmt, d.K);
    // narrow tiles of up to 32 tokens: fewer rows take them too
    const Choice c = choose(d, rows, d.E > 1);
    if (c.TT && c.per <= 32) return most;
    int i = 0;
    for (int TT : kFp4WideTiles) {
        if (!fp4_wide_may_take(d, rows, i++)) break;
        const int HT = TT / fp4_wide_halves(TT);
        if (ordered(d, rows, HT)) most = std::max(most, token_order(d, rows, HT).bytes(d.fmt));
    }
    return most;
}

// Whether the product quantises its tokens itself: the launch and the round
// through memory saved against every CTA's own quantisation, which for
// MQ_FP4_NV includes a look at the whole of each row. It is taken where it
// costs the device at most 2 us more (nvfp4 4096 x 4096, 1 / 4 / 8 / 16 rows:
// 6.3 / 7.3 / 9.0 / 12.9 us against 6.5 / 6.6 / 7.0 / 7.3 us; mxfp4 4.7 / 5.0 /
// 5.9 / 7.5 against 5.9 / 6.0 / 6.3 / 6.5 us): the host's share of a launch is
// 3 us. (In a captured graph the host has none, and those up to 2 us are lost.) A
// CTA with more stages than its ring (11008 x 4096) quantises while
// its loads wait, and large weights leave no time to hide it in.
bool fp4_linear_quantises(const Fp4Device &d, int64_t rows) {
    const Choice c = choose(d, rows, d.E > 1);
    if (c.TT != 16 || c.likely * d.KS * fp4_piece(d.fmt) > (int64_t(40) << 20)) return false;
    const int64_t stages = (d.KS + c.split - 1) / c.split;
    if (d.fmt == MQ_FP4_MX) return stages <= 5 || c.per <= 8;
    return c.per * d.K <= (stages <= 5 ? 32768 : 0);
}

mq_status launch_fp4_linear_direct(const Fp4Device &d, const void *X, mq_dtype dtype, int64_t rows, int64_t ldx,
                                   const int32_t *index, int64_t x_rows, const int32_t *offsets, void *Y,
                                   int64_t ldy, cudaStream_t stream) {
    if (rows <= 0) return MQ_OK;
    const Choice c = choose(d, rows, d.E > 1);
    NarrowParams p{};
    p.X = X;
    p.ldx = ldx;
    p.x_rows = x_rows;
    p.index = index;
    p.from = {d.K, static_cast<const char *>(X), static_cast<const char *>(X) + ((x_rows - 1) * ldx + d.K) * 2};
    p.offsets = offsets;
    p.Y = Y;
    p.ldy = ldy;
    p.fp16 = dtype == MQ_FP16;
    if (dtype == MQ_FP16)
        return d.fmt == MQ_FP4_NV ? run_narrow<true, __half>(d, p, rows, c, false, stream)
                                  : run_narrow<false, __half>(d, p, rows, c, false, stream);
    return d.fmt == MQ_FP4_NV ? run_narrow<true, __nv_bfloat16>(d, p, rows, c, false, stream)
                              : run_narrow<false, __nv_bfloat16>(d, p, rows, c, false, stream);
}

}  // namespace mq
