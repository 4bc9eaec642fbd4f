// Products with a microscaled 4-bit weight, narrow form: few tokens, where
// the weight's bytes from HBM are the bound.
//
//   Y[r][n] = fx[r] * fw[n] * sum_k (cx[r][k] sx[r][k / B]) (cw[n][k] sw[n][k / B])
//
// The weight is the MMA's A operand (128 rows a tile), the tokens its B
// operand (16, 32, 64 or 128 columns), so that a single token fills a tile of
// the tensor core; block scales are applied inside the MMA and the 32-bit row
// factors (MQ_FP4_NV) when Y is stored. One CTA computes one tile over a share
// of K; the CTAs of a cluster share a tile and add their partial sums through
// distributed shared memory in rank order, so that results do not depend on
// timing.
//
// Warp 0 copies codes and weight scales (TMA), warp 1 issues scale copies to
// tensor memory and MMAs, warps 2 and 3 place the tokens' scales (row-major in
// memory) in the order the tensor core takes, and warps 2 to 5 are the
// epilogue.

#include <algorithm>

#include "common.cuh"
#include "fp4.h"
#include "fp4_device.cuh"
#include "tc5.cuh"

namespace mq {
namespace {

constexpr int kThreads = 192;
constexpr int kMaxStages = 8;
constexpr int kBoxRows = 16;  // tokens of one copy
constexpr int kATile = 128 * 128;

struct NarrowParams {
    CUtensorMap tw, tx;
    const uint8_t *wscales;
    const float *wfactor;
    const uint8_t *xscales;
    const float *xfactor;
    const int32_t *offsets;
    void *Y;
    long long ldy, xspitch;
    int *err;
    long long N;
    int NT, KS, E, R;
    int TT;      // tokens of a tile: 16, 32, 64 or 128
    int split;   // CTAs that share a tile (the cluster)
    int stages;  // ring slots
    int fp16;
    int chained;
};

// Shared memory: the ring (codes of A and B, scales of A and B in each slot),
// then barriers.
template <bool NV>
struct NarrowSmem {
    static constexpr int kUnits = NV ? 4 : 2;      // 512-byte scale units of 128 rows in a stage
    static constexpr int kScales = kUnits * 512;
    __host__ __device__ static int slot(int TT) { return kATile + TT * 128 + 2 * kScales; }
    __host__ __device__ static int total(int TT, int stages) { return slot(TT) * stages + 1024 + 256; }
};

template <bool NV>
__global__ void __launch_bounds__(kThreads) fp4_narrow_kernel(const __grid_constant__ NarrowParams p) {
    using S = NarrowSmem<NV>;
    constexpr int kUnits = S::kUnits;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int TT = p.TT, stages = p.stages, slot = S::slot(TT);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + slot * stages);
    uint64_t *full = bars, *empty = bars + kMaxStages, *done = bars + 2 * kMaxStages;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
    int *abort_flag = reinterpret_cast<int *>(tmem_slot + 1);
    int *info = abort_flag + 1;  // expert, token begin, tokens, row tile, live

    const int split = p.split, rank = split > 1 ? static_cast<int>(cluster_rank()) : 0;
    if (warp == 0) {
        Tile t{0, 0, 0, 0};
        TileWalk walk(p.offsets, p.E, p.R, TT, p.NT);
        const bool live = walk.find(blockIdx.x / split, t);
        if (lane == 0) {
            info[0] = t.e;
            info[1] = t.m0;
            info[2] = t.tokens;
            info[3] = t.nt;
            info[4] = live ? 1 : 0;
            for (int s = 0; s < stages; ++s) {
                mbar_init(&full[s], 3);
                mbar_init(&empty[s], 1);
            }
            mbar_init(done, 1);
            *abort_flag = 0;
            fence_mbar_init();
        }
    }
    const uint32_t tmem_cols = TT <= 64 ? 128 : 256;
    if (warp == 1) tc5::alloc<1>(tmem_slot, tmem_cols);
    tc5::fence_before();
    __syncthreads();
    tc5::fence_after();
    const uint32_t tmem = *tmem_slot;
    const int expert = info[0], m0 = info[1], tokens = info[2], n0 = info[3] * 128;
    const bool live = info[4] != 0;  // the same in every CTA of a cluster
    const int nb = (tokens + kBoxRows - 1) / kBoxRows;
    const int k0 = static_cast<int>(static_cast<long long>(p.KS) * rank / split);
    const int nk = static_cast<int>(static_cast<long long>(p.KS) * (rank + 1) / split) - k0;

    if (!live) {
        // nothing to do
    } else if (warp == 0) {
        const uint32_t bytes = kATile + S::kScales + nb * kBoxRows * 128;
        const uint8_t *ws = p.wscales + ((static_cast<long long>(expert) * p.NT + info[3]) * p.KS + k0) * S::kScales;
        auto weight = [&](int i, int s) {
            uint8_t *at = smem + s * slot;
            mbar_arrive_expect_tx(&full[s], bytes);
            tma_load_3d(at, &p.tw, &full[s], (k0 + i) * 128, n0, expert);
            bulk_load(at + kATile + TT * 128, ws + static_cast<long long>(i) * S::kScales, S::kScales, &full[s]);
        };
        auto tokens_in = [&](int i, int s) {
            for (int b = 0; b < nb; ++b)
                tma_load_2d(smem + s * slot + kATile + b * kBoxRows * 128, &p.tx, &full[s], (k0 + i) * 128,
                            m0 + b * kBoxRows);
        };
        // the weight does not depend on the launch before: its first stages go ahead
        const int ahead = min(stages, nk);
        if (tc5::elect())
            for (int i = 0; i < ahead; ++i) weight(i, i);
        __syncwarp();
        pdl_wait();
        if (tc5::elect())
            for (int i = 0; i < ahead; ++i) tokens_in(i, i);
        __syncwarp();
        bool ok = true;
        for (int i = ahead, s = 0, ph = 0; i < nk && ok; ++i) {
            ok = mbar_wait(&empty[s], ph, p.err, kErrWaitEmpty, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (tc5::elect()) {
                weight(i, s);
                tokens_in(i, s);
            }
            __syncwarp();
            if (++s == stages) s = 0, ph ^= 1;
        }
    } else if (warp == 1) {
        const uint32_t desc = tc5::idesc(128, nb * kBoxRows, !NV);
        const uint32_t sfa = tmem + TT, sfb = sfa + 4 * kUnits;
        bool ok = true;
        for (int i = 0, s = 0, ph = 0; i < nk && ok; ++i) {
            ok = mbar_wait(&full[s], ph, p.err, kErrWaitFull, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc5::fence_after();
            const uint32_t at = smem_u32(smem) + s * slot;
            const uint32_t sa = at + kATile + TT * 128, sb = sa + S::kScales;
            const uint64_t da = tc5::operand_desc(at), db = tc5::operand_desc(at + kATile);
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
    } else if (warp < 4) {
        // the tokens' scales: 4-byte pieces into the tensor core's order. A
        // stage is handed over two iterations after its copies were issued.
        pdl_wait();
        auto place = [&](int i, int s) {
            uint8_t *at = smem + s * slot + kATile + TT * 128 + S::kScales;
            for (int r = threadIdx.x - 64; r < tokens; r += 64) {
                const uint8_t *src = p.xscales + (m0 + r) * p.xspitch + static_cast<long long>(k0 + i) * (4 * kUnits);
                uint8_t *dst = at + (r & 31) * 16 + (r >> 5) * 4;
#pragma unroll
                for (int u = 0; u < kUnits; ++u) cp_async4(dst + 512 * u, src + 4 * u);
            }
            cp_async_commit();
        };
        auto hand_over = [&](int s) {
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[s]);
        };
        int s = 0, ph = 1, hs = 0;
        for (int i = 0; i < nk; ++i) {
            if (!mbar_wait_warp(&empty[s], ph, p.err, kErrWaitEmpty, abort_flag)) break;
            place(i, s);
            if (++s == stages) s = 0, ph ^= 1;
            if (i >= 2) {
                cp_async_wait_group<2>();
                hand_over(hs);
                if (++hs == stages) hs = 0;
            }
        }
        if (nk >= 2) {
            cp_async_wait_group<1>();
            hand_over(hs);
            if (++hs == stages) hs = 0;
        }
        cp_async_wait_group<0>();
        hand_over(hs);
    }

    __syncwarp();

    // ------------------------------------------------------------ epilogue
    if (live && warp >= 2) {
        const int quad = warp & 3, row = quad * 32 + lane;
        pdl_wait();
        __syncwarp();
        mbar_wait_warp(done, 0, p.err, kErrWaitMma, abort_flag);
        tc5::fence_after();
        const long long n = n0 + row;
        const float fw = NV && n < p.N ? __ldg(p.wfactor + static_cast<long long>(expert) * p.N + n) : 1.0f;
        float *part = reinterpret_cast<float *>(smem);  // [tokens][128], the ring is drained
        for (int c = 0; c < nb * kBoxRows; c += 16) {
            uint32_t bits[16];
            tc5::load16(tmem + (static_cast<uint32_t>(quad) << 21) + c, bits);
            tc5::load_wait();
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(bits[j]);
            if (split > 1) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (c + j < tokens) part[(c + j) * 128 + row] = v[j];
            } else if (n < p.N) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int t = c + j;
                    if (t >= tokens) break;
                    float y = v[j];
                    if constexpr (NV) y = y * p.xfactor[m0 + t] * fw;
                    store_output(p.Y, (m0 + t) * p.ldy + n, y, p.fp16);
                }
            }
        }
    }
    drain_after_abort(abort_flag);
    __syncwarp();
    if (live && split > 1) {
        cluster_sync();
        if (warp >= 2) {
            // rank r adds the elements [r, r + 1) / split of the tile
            const float *part = reinterpret_cast<const float *>(smem);
            const int total = tokens * 128;
            const int lo = static_cast<int>(static_cast<long long>(total) * rank / split);
            const int hi = static_cast<int>(static_cast<long long>(total) * (rank + 1) / split);
            for (int i = lo + threadIdx.x - 64; i < hi; i += 128) {
                const int t = i >> 7;
                const long long n = n0 + (i & 127);
                float y = 0.0f;
                for (int r = 0; r < split; ++r) y += ld_dsmem_f32(part + i, r);
                if (n >= p.N) continue;
                if constexpr (NV)
                    y = y * p.xfactor[m0 + t] * __ldg(p.wfactor + static_cast<long long>(expert) * p.N + n);
                store_output(p.Y, (m0 + t) * p.ldy + n, y, p.fp16);
            }
        }
        cluster_sync();
    }
    tc5::fence_before();
    __syncthreads();
    if (warp == 1) {
        tc5::fence_after();
        tc5::dealloc<1>(tmem, tmem_cols);
    }
}

template <bool NV>
mq_status run_narrow(const Fp4Device &d, const Fp4Rows &x, const int32_t *offsets, void *Y, mq_dtype dtype,
                     int64_t ldy, bool chained, cudaStream_t stream) {
    using S = NarrowSmem<NV>;
    NarrowParams p{};
    const int64_t per = offsets ? (x.rows + d.E - 1) / d.E : x.rows;  // rows of an average matrix
    p.TT = per <= 16 ? 16 : per <= 32 ? 32 : per <= 64 ? 64 : 128;
    // the most tiles that any split of the rows into matrices makes
    const int64_t tiles = (offsets ? std::min<int64_t>(d.E, x.rows) + x.rows / p.TT : (x.rows + p.TT - 1) / p.TT) * d.NT;
    const int64_t likely = (offsets ? std::min<int64_t>(d.E, x.rows) * ((per + p.TT - 1) / p.TT)
                                    : (x.rows + p.TT - 1) / p.TT) * d.NT;
    p.split = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({8, d.KS, 2 * sm_count() / std::max<int64_t>(1, likely)})));
    if (tiles * p.split > 0x7FFFFFFFll) return fail(MQ_ERR_UNSUPPORTED, "fp4 linear: too many tiles");
    p.stages = std::min(kMaxStages, std::max(3, (112 * 1024 - 1280) / S::slot(p.TT)));
    const int smem = S::total(p.TT, p.stages);
    p.tw = d.map;
    if (!encode_bytes_map(&p.tx, x.codes, d.pitch, x.rows, 0, kBoxRows))
        return fail(MQ_ERR_CUDA, "cuTensorMapEncodeTiled failed for the activations");
    p.wscales = d.scales;
    p.wfactor = d.row_scale;
    p.xscales = x.scales;
    p.xfactor = x.row_scale;
    p.offsets = offsets;
    p.Y = Y;
    p.ldy = ldy;
    p.xspitch = fp4_scale_pitch(d.fmt, d.K);
    p.err = d.err;
    p.N = d.N;
    p.NT = static_cast<int>(d.NT);
    p.KS = d.KS;
    p.E = static_cast<int>(d.E);
    p.R = static_cast<int>(x.rows);
    p.fp16 = dtype == MQ_FP16;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return fail(MQ_ERR_CUDA, "cudaGetDevice failed");
    if (dev < 0 || dev >= 64) return fail(MQ_ERR_UNSUPPORTED, "device ordinal above 63");
    static bool configured[64] = {};
    if (!configured[dev]) {
        if (cudaFuncSetAttribute(fp4_narrow_kernel<NV>, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) !=
            cudaSuccess)
            return fail(MQ_ERR_CUDA, "fp4 linear: device setup failed");
        configured[dev] = true;
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
    if (chained) {
        attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[na].val.programmaticStreamSerializationAllowed = 1;
        ++na;
    }
    cfg.attrs = attr;
    cfg.numAttrs = na;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fp4_narrow_kernel<NV>, p);
    if (e != cudaSuccess) return fail(MQ_ERR_CUDA, std::string("fp4 linear launch: ") + cudaGetErrorString(e));
    return MQ_OK;
}

}  // namespace

mq_status launch_fp4_linear(const Fp4Device &d, const Fp4Rows &x, const int32_t *offsets, void *Y,
                            mq_dtype dtype, int64_t ldy, bool chained, cudaStream_t stream) {
    if (x.rows <= 0) return MQ_OK;
    const int64_t per = offsets ? x.rows / std::min<int64_t>(d.E, x.rows) : x.rows;  // rows of a matrix
    if (per > 128) return launch_fp4_wide(d, x, offsets, Y, dtype, ldy, chained, stream);
    return d.fmt == MQ_FP4_NV ? run_narrow<true>(d, x, offsets, Y, dtype, ldy, chained, stream)
                              : run_narrow<false>(d, x, offsets, Y, dtype, ldy, chained, stream);
}

}  // namespace mq
