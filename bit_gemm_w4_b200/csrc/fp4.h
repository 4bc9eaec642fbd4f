// Microscaled 4-bit floating point: declarations shared by the C ABI
// (fp4_api.cpp) and the kernels (fp4_quantize.cu, fp4_linear.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"

namespace mq {

// What a CUDA call that failed is reported as. It clears the last error, which
// other launches of this library look at and would take for their own.
mq_status fp4_cuda_fail(cudaError_t e, const char *what);

// One K stage of the products: 256 columns, 128 bytes of codes in a row (the
// 128-byte swizzle's span), 16 (MQ_FP4_NV) or 8 (MQ_FP4_MX) scale bytes.
constexpr int kFp4StageK = 256;

constexpr int fp4_block(int fmt) { return fmt == MQ_FP4_NV ? 16 : 32; }
// scale bytes of one row in one K stage
constexpr int fp4_stage_scales(int fmt) { return kFp4StageK / fp4_block(fmt); }
// Bytes of a row of codes and of a row of scales: whole 16-byte units, so
// that rows are readable by TMA and in 16-byte pieces; what lies past K is 0.
constexpr int64_t fp4_code_pitch(int64_t K) { return (K + 31) / 32 * 16; }
constexpr int64_t fp4_scale_pitch(int fmt, int64_t K) {
    const int64_t cols = 16 * fp4_block(fmt);
    return (K + cols - 1) / cols * 16;
}

// Token scales in the order the wide form takes them: slots of HT tokens of
// one matrix, [slots][KS][units of four scale columns][unit bytes], a token's
// four bytes at (x / 128) * 512 + (x % 32) * 16 + (x / 32 % 4) * 4 of each
// unit for the slot's token x. Matrix e's tokens begin at row a = offsets[e],
// and at slot a / HT + e: past every slot of the matrices before it, since
// ceil(c / HT) <= floor((a + c) / HT) - floor(a / HT) + 1.
struct Fp4Order {
    int HT = 0;  // 0: row-major scales
    int unit = 0;
    int KS = 0;
    int64_t slots = 0;
    const int32_t *offsets = nullptr;  // NULL: one matrix with every row
    int E = 1;
    int64_t bytes(int fmt) const { return slots * KS * (fp4_stage_scales(fmt) / 4) * unit; }
};

// A quantised matrix in caller memory (row-major codes; scales row-major or
// ordered).
struct Fp4Rows {
    const uint8_t *codes;
    const uint8_t *scales;
    const float *row_scale;  // NULL for MQ_FP4_MX
    int64_t rows;
    Fp4Order order;
};

// Device side of a packed weight: E matrices [N][K] of one format. A matrix is
// held in pieces of 128 rows x one K stage, in the order the products read
// them, [E][NT][KS]: a piece is what a CTA copies to shared memory in one go,
// byte for byte as the tensor core takes it from there (a row-major matrix
// would be read in 128-byte bits of 128 rows, which costs HBM a third of its
// rate). Rows and columns past N and K are zeros.
//   codes   16 KB: row r's 16-byte unit u at r * 128 + (u ^ r % 8) * 16 (the
//           128-byte swizzle)
//   scales  512-byte units of four scale columns: row r's column c at
//           (c / 4) * 512 + (r % 32) * 16 + (r / 32) * 4 + c % 4
struct Fp4Device {
    int64_t E = 0, N = 0, K = 0;
    int fmt = 0;
    int device = 0, sms = 0;
    int clusters[9] = {};  // clusters of 1 to 8 narrow CTAs that the device holds at once, one CTA an SM
    int KS = 0;      // K stages
    int64_t NT = 0;  // 128-row tiles of one matrix
    uint8_t *pieces = nullptr;
    float *row_scale = nullptr;  // [E][N], NULL for MQ_FP4_MX
    int *err = nullptr;
    CUtensorMap map;  // pieces as rows of 128 bytes, a piece a box
};

constexpr int kFp4CodePiece = 128 * 128;
constexpr int fp4_scale_piece(int fmt) { return 128 * fp4_stage_scales(fmt); }
constexpr int fp4_piece(int fmt) { return kFp4CodePiece + fp4_scale_piece(fmt); }

// X (dtype, row stride ldx elements) to codes, scales and (MQ_FP4_NV) row
// factors, `rows` output rows; output row r is X row index[r] (index NULL: r),
// and a row of zeros where index[r] is outside [0, x_rows). `open`: the launch
// that follows may start at once (it waits for this one before it reads
// anything but packed weights).
mq_status launch_fp4_quantize(const void *X, mq_dtype dtype, int64_t rows, int64_t K, int64_t ldx,
                              const int32_t *index, int64_t x_rows, int fmt, uint8_t *codes,
                              uint8_t *scales, float *row_scale, const Fp4Order &order, bool open,
                              cudaStream_t stream);

mq_status launch_fp4_dequantize(const Fp4Rows &x, int64_t K, int fmt, void *Y, mq_dtype dtype,
                                int64_t ldy, cudaStream_t stream);

// Row-major codes and scales ([E * N] rows) to a weight's pieces, or back.
mq_status launch_fp4_order(const Fp4Device &d, uint8_t *codes, uint8_t *scales, bool to_rows, cudaStream_t stream);

// Y[r] = x[r] * W[e]^T for the rows offsets[e] <= r < offsets[e + 1] of every
// e (offsets NULL: E is 1 and every row belongs to it). `chained`: x was
// written by the launch just before on this stream, which started after the
// offsets were there.
mq_status launch_fp4_linear(const Fp4Device &d, const Fp4Rows &x, const int32_t *offsets, void *Y,
                            mq_dtype dtype, int64_t ldy, bool chained, cudaStream_t stream);

// Fills in d.clusters for d's format and device (the current one).
mq_status fp4_count_clusters(Fp4Device &d);

// The same from X as it is (as for launch_fp4_quantize), quantised by the
// product itself, where fp4_linear_quantises says that this is the faster way.
bool fp4_linear_quantises(const Fp4Device &d, int64_t rows);
mq_status launch_fp4_linear_direct(const Fp4Device &d, const void *X, mq_dtype dtype, int64_t rows, int64_t ldx,
                                   const int32_t *index, int64_t x_rows, const int32_t *offsets, void *Y,
                                   int64_t ldy, cudaStream_t stream);

// The order in which launch_fp4_linear wants the scales of `rows` rows that
// are quantised for it.
Fp4Order fp4_token_order(const Fp4Device &d, int64_t rows, const int32_t *offsets);

// Bytes that the scales of up to `rows` rows quantised for launch_fp4_linear
// take at most, in whichever order: no less for more rows.
int64_t fp4_token_scale_bytes(const Fp4Device &d, int64_t rows);

// The form of launch_fp4_linear for many tokens (fp4_wide.cu): the tokens of
// a tile and the halves they come in.
struct Fp4WidePlan {
    int TT, halves;
};
Fp4WidePlan fp4_wide_plan(const Fp4Device &d, int64_t rows);
// Its tiles, the smallest first, and whether up to `rows` rows may take tile i:
// not where they make no more of the tile before it, which takes less time (one
// for a single matrix; for several the plan counts half a tile each, one at least).
constexpr int kFp4WideTiles[] = {32, 64, 96, 128, 160, 192, 224, 256, 320, 384};
inline int fp4_wide_halves(int TT) { return TT > 224 ? 2 : 1; }
inline int fp4_scale_unit(int HT) { return HT > 128 ? 1024 : 512; }
inline bool fp4_wide_may_take(const Fp4Device &d, int64_t rows, int i) {
    return i == 0 || rows > (d.E == 1 ? kFp4WideTiles[i - 1] : d.E * kFp4WideTiles[i - 1] / 2);
}
mq_status launch_fp4_wide(const Fp4Device &d, const Fp4Rows &x, const int32_t *offsets, void *Y,
                          mq_dtype dtype, int64_t ldy, bool chained, cudaStream_t stream);

// Rows of `pitch` bytes as a tensor map with boxes of box_rows x 128 bytes
// (zeros past the end), with or without the 128-byte swizzle.
bool encode_bytes_map(CUtensorMap *map, const void *base, int64_t pitch, int64_t rows, int box_rows, bool swizzle);

}  // namespace mq
