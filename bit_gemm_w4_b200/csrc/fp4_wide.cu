// Products with a microscaled 4-bit weight, wide form: many tokens, where the
// tensor cores and the way into them are the bound.
//
// A pair of CTAs (two SMs) computes a tile of 256 weight rows x up to 224
// tokens with cta_group::2 MMAs: each CTA brings its own 128 rows of the
// weight and half of the tokens, so that a byte in shared memory feeds twice
// the products of a single CTA's tile. At the 4-bit rate a lone CTA would
// have to write and read 192 bytes of shared memory a cycle, a pair 128.
// Persistent: one pair for every two SMs walks over the tiles.
//
// Two shapes of tile. Up to 224 tokens (kHalves 1): two accumulators let a
// tile's outputs be stored while the next tile is computed (2 x 256 columns
// would leave none for the scales). Up to 384 tokens (kHalves 2): both
// accumulators belong to one tile, whose weight piece is multiplied with two
// halves of up to 192 tokens; what has to come from L2 for a product falls by
// 30 %, and the epilogue packs its outputs into registers first, so that the
// next tile waits for that alone and not for the stores.
//
// Each CTA fills its own ring: warp 0 copies codes and scales (TMA). Token
// scales that lie row by row in memory (tokens the caller quantised) are
// placed in the tensor core's order by warps 2 to 5 instead. Both report to
// the first CTA's barriers, whose warp 1 issues scale copies to tensor memory
// and MMAs for the pair. Warps 6 to 13 are the epilogue.

#include <algorithm>
#include <cmath>
#include <iterator>

#include "common.cuh"
#include "fp4.h"
#include "fp4_device.cuh"
#include "tc5.cuh"

namespace mq {
namespace {

constexpr int kThreads = 448;
constexpr int kStorers = 8;    // epilogue warps, two for each quarter of the lanes
constexpr int kMaxStages = 8;
constexpr int kBoxRows = 16;   // tokens of one copy in a tile that is not full
constexpr int kLoaders = 4;

struct WideParams {
    CUtensorMap tw, tx, tx_small;  // boxes of a piece of the weight, half a MMA's tokens, 16 tokens
    CUtensorMap tsx;               // ordered token scales, a slot's stage a box
    const float *wfactor;
    const uint8_t *xscales;
    const float *xfactor;
    const int32_t *offsets;
    void *Y;
    long long ldy, xspitch;
    int *err;
    long long N;
    int NT;   // pairs of 128-row tiles
    int NT1;  // 128-row tiles
    int KS, E, R;
    int TT;   // tokens of a tile, kHalves times a multiple of 32
    int stages;
    int fp16;
    int paired;  // N, the stride and Y's address are even: 4-byte stores
    int wait_first;
    int ordered;
};

template <bool NV, int kHalves>
struct WideSmem {
    static constexpr int kUnits = NV ? 4 : 2;
    static constexpr int kCols = kHalves == 1 ? 224 : 192;  // columns of an accumulator
    // scales in tensor memory: the weight's, then each half's, in one or two sets
    static constexpr uint32_t kScaleCols = 2 * kCols, kScaleSet = (4 + 8 * kHalves) * kUnits;
    static constexpr int kSets = kScaleCols + 2 * kScaleSet <= 512 ? 2 : 1;
    static_assert(kScaleCols + kSets * kScaleSet <= 512, "tensor memory");
    static constexpr int kPiece = kFp4CodePiece + kUnits * 512;
    static constexpr int kFactors = NV ? kStorers * kCols * 4 : 0;
    // bytes of a unit of one half's scales
    __host__ __device__ static int unit(int TT) { return TT / kHalves > 128 ? 1024 : 512; }
    __host__ __device__ static int slot(int TT) { return kPiece + TT * 64 + kHalves * kUnits * unit(TT); }
    __host__ __device__ static int total(int TT, int stages) { return slot(TT) * stages + 1024 + 256 + kFactors; }
};

template <bool NV, int kHalves>
__global__ void __launch_bounds__(kThreads, 1) fp4_wide_kernel(const __grid_constant__ WideParams p) {
    using S = WideSmem<NV, kHalves>;
    constexpr int kUnits = S::kUnits, kBuffers = 3 - kHalves;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int TT = p.TT, stages = p.stages, slot = S::slot(TT), KS = p.KS;
    const int at_b = S::kPiece, at_sb = at_b + TT * 64, unit = S::unit(TT), HT = TT / kHalves;
    // tokens of half h of a tile, and the MMA's columns for them
    auto tokens_of = [&](const Tile &t, int h) { return min(max(t.tokens - h * HT, 0), HT); };
    auto cols_of = [&](const Tile &t, int h) { return (tokens_of(t, h) + 31) / 32 * 32; };
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + slot * stages);
    uint64_t *full = bars, *empty = bars + kMaxStages, *acc_full = bars + 2 * kMaxStages, *acc_empty = acc_full + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_empty + 2);
    int *abort_flag = reinterpret_cast<int *>(tmem_slot + 1);
    const uint32_t rank = cluster_rank();

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&full[s], p.ordered ? 1 : 1 + 2 * kLoaders);  // the first CTA's producer, both CTAs' loaders
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 2 * kStorers);  // the epilogue warps of both CTAs
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) tc5::alloc<2>(tmem_slot, 512);
    tc5::fence_before();
    __syncthreads();
    cluster_sync();
    tc5::fence_after();
    const uint32_t tmem = *tmem_slot;

    // Whatever follows on the stream may start: it waits for this launch
    // before it reads anything but packed weights.
    pdl_launch_dependents();
    if (p.wait_first) pdl_wait();  // the offsets may come from the launch just before
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    TileWalk walk(p.offsets, p.E, p.R, TT, p.NT);
    Tile t;

    if (warp == 0) {
        int s = 0, ph = 1, first = 1;
        bool ok = true;
        for (long long ti = pair; ok && walk.find(ti, t); ti += pairs) {
            uint32_t bytes = 2 * S::kPiece;  // both CTAs' copies
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
                const int n = cols_of(t, h);
                bytes += n * 128 + (p.ordered && n ? 2 * kUnits * unit : 0);
            }
            const int token_slot = (p.offsets ? t.first / HT + t.e : 0) + (t.m0 - t.first) / HT;
            // past the last row tile (an odd count) that tile again: rows that are not stored
            const int nt1 = min(t.nt * 2 + static_cast<int>(rank), p.NT1 - 1);
            const int piece = (t.e * p.NT1 + nt1) * KS;
            auto weight = [&](int k, int slot_i) {
                const uint32_t bar = in_cta(&full[slot_i], 0);
                if (rank == 0) mbar_arrive_expect_tx(&full[slot_i], bytes);
                tma_pair_load_2d(smem + slot_i * slot, &p.tw, bar, 0, (piece + k) * (S::kPiece / 128));
            };
            auto tokens_in = [&](int k, int slot_i) {
                const uint32_t bar = in_cta(&full[slot_i], 0);
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
                    uint8_t *at = smem + slot_i * slot + at_b + h * HT * 64;
                    const int half = cols_of(t, h) / 2, m = t.m0 + h * HT + rank * half;
                    if (half == 0) break;
                    if (p.ordered)
                        tma_pair_load_2d(smem + slot_i * slot + at_sb + h * kUnits * unit, &p.tsx, bar, 0,
                                         ((token_slot + h) * KS + k) * (kUnits * unit / 128));
                    if (half == HT / 2)
                        tma_pair_load_2d(at, &p.tx, bar, k * 128, m);
                    else
                        for (int b = 0; b < half; b += kBoxRows)
                            tma_pair_load_2d(at + b * 128, &p.tx_small, bar, k * 128, m + b);
                }
            };
            int k = 0;
            if (first) {
                // the weight does not depend on the launch before: its first stages go ahead
                const int ahead = min(stages, KS);
                if (tc5::elect())
                    for (int i = 0; i < ahead; ++i) weight(i, i);
                __syncwarp();
                pdl_wait();
                if (tc5::elect())
                    for (int i = 0; i < ahead; ++i) tokens_in(i, i);
                __syncwarp();
                k = ahead;
                s = ahead == stages ? 0 : ahead;
                if (ahead == stages) ph ^= 1;
                first = 0;
            }
            for (; k < KS && ok; ++k) {
                ok = mbar_wait(&empty[s], ph, p.err, kErrWaitEmpty, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (tc5::elect()) {
                    weight(k, s);
                    tokens_in(k, s);
                }
                __syncwarp();
                if (++s == stages) s = 0, ph ^= 1;
            }
        }
    } else if (warp == 1 && rank == 1) {
        // the first CTA's warp 1 issues for both
    } else if (warp == 1) {
        int s = 0, ph = 0, b = 0, bph = 1, set = 0;
        bool ok = true;
        pdl_wait();  // before any wait with a limit: the launch before may take its time
        for (long long ti = pair; ok && walk.find(ti, t); ti += pairs) {
            ok = mbar_wait(&acc_empty[b], bph, p.err, kErrWaitEmpty, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            for (int k = 0; k < KS && ok; ++k) {
                ok = mbar_wait(&full[s], ph, p.err, kErrWaitFull, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc5::fence_after();
                const uint32_t at = smem_u32(smem) + s * slot;
                const uint32_t sfa = tmem + S::kScaleCols + set * S::kScaleSet;
                const uint64_t da = tc5::operand_desc(at);
                if (tc5::elect()) {
#pragma unroll
                    for (int u = 0; u < kUnits; ++u)
                        tc5::copy_scales<2>(sfa + 4 * u, tc5::scale_desc(at + kFp4CodePiece + 512 * u));
#pragma unroll
                    for (int h = 0; h < kHalves; ++h) {
                        const int n = cols_of(t, h);
                        if (n == 0) break;
                        const uint32_t sfb = sfa + (4 + 8 * h) * kUnits, sb = at + at_sb + h * kUnits * unit;
                        const uint32_t d = tmem + (kHalves == 2 ? h : b) * S::kCols, desc = tc5::idesc(256, n, !NV);
                        const uint64_t db = tc5::operand_desc(at + at_b + h * HT * 64);
#pragma unroll
                        for (int u = 0; u < kUnits; ++u) {
                            tc5::copy_scales<2>(sfb + 8 * u, tc5::scale_desc(sb + unit * u));
                            if (n > 128) tc5::copy_scales<2>(sfb + 8 * u + 4, tc5::scale_desc(sb + unit * u + 512));
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int u = NV ? q : q >> 1;
                            const uint32_t byte = NV ? 0 : (q & 1) * 2;
                            tc5::mma<2, NV>(d, da + 2 * q, db + 2 * q, desc | tc5::idesc_scale_byte(byte), sfa + 4 * u,
                                            sfb + 8 * u, k > 0 || q > 0);
                        }
                    }
                    tc5::commit_pair(&empty[s]);
                }
                __syncwarp();
                if (S::kSets == 2) set ^= 1;
                if (++s == stages) s = 0, ph ^= 1;
            }
            if (tc5::elect()) tc5::commit_pair(&acc_full[b]);
            __syncwarp();
            ok = __all_sync(0xffffffffu, ok);
            if (++b == kBuffers) b = 0, bph ^= 1;
        }
    } else if (warp < 6 && p.ordered) {
        // nothing to place
    } else if (warp < 6) {
        // the tokens' scales, two stages at a time: a row's 32 (MQ_FP4_MX: 16)
        // bytes are read in one go, one pair of stages ahead of their turn
        pdl_wait();
        constexpr int kVec = NV ? 2 : 1, kLoadRows = (kHalves * S::kCols + 32 * kLoaders - 1) / (32 * kLoaders);
        uint4 next[kLoadRows][kVec];
        const int t0 = threadIdx.x - 64;
        auto read = [&](const Tile &tile, int k) {
#pragma unroll
            for (int i = 0; i < kLoadRows; ++i) {
                const int r = t0 + i * 32 * kLoaders;
                if (r < tile.tokens) {
                    const uint8_t *src = p.xscales + (tile.m0 + r) * p.xspitch + static_cast<long long>(k) * (4 * kUnits);
#pragma unroll
                    for (int v = 0; v < kVec; ++v)
                        if (NV ? k + v < KS : true)
                            asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                                         : "=r"(next[i][v].x), "=r"(next[i][v].y), "=r"(next[i][v].z),
                                           "=r"(next[i][v].w)
                                         : "l"(src + 16 * v));
                }
            }
        };
        int s = 0, ph = 1;
        bool ok = true;
        bool have = walk.find(pair, t);
        if (have) read(t, 0);
        for (long long ti = pair; have && ok;) {
            const Tile cur = t;
            ti += pairs;
            have = walk.find(ti, t);
            for (int k = 0; k < KS && ok; k += 2) {
                uint4 now[kLoadRows][kVec];
#pragma unroll
                for (int i = 0; i < kLoadRows; ++i)
#pragma unroll
                    for (int v = 0; v < kVec; ++v) now[i][v] = next[i][v];
                if (k + 2 < KS)
                    read(cur, k + 2);
                else if (have)
                    read(t, 0);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (k + j >= KS) break;
                    ok = mbar_wait_warp(&empty[s], ph, p.err, kErrWaitEmpty, abort_flag);
                    if (!ok) break;
                    uint8_t *at = smem + s * slot + at_sb;
#pragma unroll
                    for (int i = 0; i < kLoadRows; ++i) {
                        const int r = t0 + i * 32 * kLoaders;
                        if (r < cur.tokens) {
                            const int h = kHalves == 2 && r >= HT, x = r - h * HT;
                            uint32_t *dst = reinterpret_cast<uint32_t *>(at + h * kUnits * unit + (x >> 7) * 512 +
                                                                         (x & 31) * 16 + ((x >> 5) & 3) * 4);
                            const uint4 v = now[i][NV ? j : 0];
                            const int next_unit = unit / 4;
                            if constexpr (NV) {
                                dst[0] = v.x;
                                dst[next_unit] = v.y;
                                dst[2 * next_unit] = v.z;
                                dst[3 * next_unit] = v.w;
                            } else {
                                dst[0] = j ? v.z : v.x;
                                dst[next_unit] = j ? v.w : v.y;
                            }
                        }
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(in_cta(&full[s], 0));
                    if (++s == stages) s = 0, ph ^= 1;
                }
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        pdl_wait();
        const int quad = warp & 3, row = quad * 32 + lane, which = (warp - 6) >> 2;
        float *factors = reinterpret_cast<float *>(smem + slot * stages + 256) + (warp - 6) * S::kCols;
        int b = 0, bph = 0;
        for (long long ti = pair; walk.find(ti, t); ti += pairs) {
            const long long n = (t.nt * 2 + static_cast<int>(rank)) * 128ll + row;
            const bool live = n < p.N;
            const float fw = NV && live ? __ldg(p.wfactor + static_cast<long long>(t.e) * p.N + n) : 1.0f;
            // the two warps of a quarter take every other 16 tokens of a tile, or a half each
            const int tokens = kHalves == 2 ? tokens_of(t, which) : t.tokens;
            const int m0 = t.m0 + (kHalves == 2 ? which * HT : 0);
            if constexpr (NV) {
                __syncwarp();
                for (int m = lane; m < tokens; m += 32) factors[m] = load_f32(p.xfactor + m0 + m);
                __syncwarp();
            }
            auto outputs = [&](const uint32_t (&bits)[16], int c, float (&v)[16]) {
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(bits[j]);
                if constexpr (NV) apply_factors(v, factors + c, fw);
            };
            auto release = [&] {
                tc5::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(in_cta(&acc_empty[b], 0));
            };
            if (!mbar_wait_warp(&acc_full[b], bph, p.err, kErrWaitMma, abort_flag)) break;
            tc5::fence_after();
            const uint32_t d = tmem + (kHalves == 2 ? which : b) * S::kCols + (static_cast<uint32_t>(quad) << 21);
            if constexpr (kHalves == 1) {
                // the next 16 tokens on their way meanwhile
                uint32_t next[16];
                int c = 16 * which;
                if (c < tokens) tc5::load16(d + c, next);
                for (; c < tokens; c += 32) {
                    float v[16];
                    tc5::load_wait();
                    outputs(next, c, v);
                    if (c + 32 < tokens) tc5::load16(d + c + 32, next);
                    store_chunk(v, p.Y, p.ldy, m0 + c, n, tokens - c, live, p.paired, p.fp16);
                }
                release();
            } else {
                constexpr int kSteps = S::kCols / 16;
                uint32_t packed[kSteps][8];
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    if (i * 16 < tokens) {
                        uint32_t bits[16];
                        float v[16];
                        tc5::load16(d + i * 16, bits);
                        tc5::load_wait();
                        outputs(bits, i * 16, v);
                        pack_chunk(v, packed[i], p.paired, p.fp16);
                    }
                }
                release();
#pragma unroll
                for (int i = 0; i < kSteps; ++i)
                    if (i * 16 < tokens)
                        store_packed(packed[i], p.Y, p.ldy, m0 + i * 16, n, tokens - i * 16, live, p.paired);
            }
            if (++b == kBuffers) b = 0, bph ^= 1;
        }
    }
    __syncwarp();
    drain_after_abort(abort_flag);
    __syncwarp();
    pdl_wait();  // a launch is not over before the one it was chained to
    tc5::fence_before();
    __syncthreads();
    cluster_sync();  // neither CTA leaves while the other may still reach it
    if (warp == 1) {
        tc5::fence_after();
        tc5::dealloc<2>(tmem, 512);
    }
}

}  // namespace

template <bool NV, int kHalves>
static mq_status run_wide(const Fp4Device &d, const Fp4Rows &x, const int32_t *offsets, void *Y, mq_dtype dtype,
                          int64_t ldy, bool chained, cudaStream_t stream, int TT) {
    using S = WideSmem<NV, kHalves>;
    WideParams p{};
    p.TT = TT;
    p.NT1 = static_cast<int>(d.NT);
    p.NT = static_cast<int>((d.NT + 1) / 2);
    // the most tiles that any split of the rows into matrices makes
    const int64_t tiles = (offsets ? std::min<int64_t>(d.E, x.rows) + x.rows / TT : (x.rows + TT - 1) / TT) * p.NT;
    p.stages = std::min(kMaxStages, (227 * 1024 - S::total(TT, 0)) / S::slot(TT));
    p.tw = d.map;
    if (!encode_bytes_map(&p.tx, x.codes, fp4_code_pitch(d.K), x.rows, TT / kHalves / 2, true) ||
        !encode_bytes_map(&p.tx_small, x.codes, fp4_code_pitch(d.K), x.rows, kBoxRows, true))
        return fail(MQ_ERR_CUDA, "cuTensorMapEncodeTiled failed for the activations");
    p.paired = d.N % 2 == 0 && ldy % 2 == 0 && (reinterpret_cast<uintptr_t>(Y) & 3) == 0;
    p.wfactor = d.row_scale;
    p.ordered = x.order.HT != 0;
    if (p.ordered && !encode_bytes_map(&p.tsx, x.scales, 128, x.order.bytes(d.fmt) / 128, S::kUnits * x.order.unit / 128, false))
        return fail(MQ_ERR_CUDA, "cuTensorMapEncodeTiled failed for the activations' scales");
    p.xscales = x.scales;
    p.xfactor = x.row_scale;
    p.offsets = offsets;
    p.Y = Y;
    p.ldy = ldy;
    p.xspitch = fp4_scale_pitch(d.fmt, d.K);
    p.err = d.err;
    p.N = d.N;
    p.KS = d.KS;
    p.E = static_cast<int>(d.E);
    p.R = static_cast<int>(x.rows);
    p.fp16 = dtype == MQ_FP16;
    p.wait_first = offsets && !chained;
    static bool configured[64] = {};
    if (!configured[d.device]) {
        if (const cudaError_t e = cudaFuncSetAttribute(fp4_wide_kernel<NV, kHalves>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024))
            return fp4_cuda_fail(e, "fp4 linear: device setup");
        configured[d.device] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min<int64_t>(tiles, d.sms / 2)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::total(TT, p.stages);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fp4_wide_kernel<NV, kHalves>, p);
    if (e != cudaSuccess) return fp4_cuda_fail(e, "fp4 linear launch");
    return MQ_OK;
}

Fp4WidePlan fp4_wide_plan(const Fp4Device &d, int64_t rows) {
    // Tokens of a tile: the choice that leaves the least time over the waves of
    // tiles. A stage takes a time that does not depend on the tokens plus one
    // for each of them; the constants (ns) fit 8192^3, 4096 x 4096 x 11008 and
    // 2048 x 14336 x 4096 at 128 to 384 tokens, all of which run at the power
    // limit. Two halves move less and pay 1 us a tile, for which K has to be
    // long: 8192^3 mxfp4 takes 253 us with 384 tokens and 275 us with 224, 2048
    // x 14336 x 4096 nvfp4 80 and 63 us (both with the quantisation).
    // Matrices of a ragged batch end half a tile early on average.
    const bool nv = d.fmt == MQ_FP4_NV;
    const int64_t NT = (d.NT + 1) / 2, pairs = d.sms / 2, mats = std::min<int64_t>(d.E, rows);
    int best = 0;
    double least = 0;
    for (int i = std::size(kFp4WideTiles); i-- > 0;) {
        const int TT = kFp4WideTiles[i];
        const bool two = fp4_wide_halves(TT) == 2;
        const double even = static_cast<double>((rows + mats * TT - 1) / (mats * TT)) * mats;
        const double tiles = (mats == 1 ? even : std::max<double>(mats, static_cast<double>(rows) / TT + 0.5 * mats)) * NT;
        double waves = tiles / pairs;
        if (mats == 1 || waves < 1) waves = std::ceil(waves);
        const double stage = nv ? (two ? 200 + 1.67 * TT : 210 + 1.35 * TT) : (two ? 240 + 0.9 * TT : 245 + 0.66 * TT);
        const double cost = waves * (d.KS * stage + (two ? 1000 : 0));
        if (!best || cost < least) least = cost, best = TT;
    }
    return {best, fp4_wide_halves(best)};
}

mq_status launch_fp4_wide(const Fp4Device &d, const Fp4Rows &x, const int32_t *offsets, void *Y, mq_dtype dtype,
                          int64_t ldy, bool chained, cudaStream_t stream) {
    const Fp4WidePlan plan = fp4_wide_plan(d, x.rows);
    const bool nv = d.fmt == MQ_FP4_NV;
    if (plan.halves == 2) return nv ? run_wide<true, 2>(d, x, offsets, Y, dtype, ldy, chained, stream, plan.TT)
                                    : run_wide<false, 2>(d, x, offsets, Y, dtype, ldy, chained, stream, plan.TT);
    return nv ? run_wide<true, 1>(d, x, offsets, Y, dtype, ldy, chained, stream, plan.TT)
              : run_wide<false, 1>(d, x, offsets, Y, dtype, ldy, chained, stream, plan.TT);
}

}  // namespace mq
