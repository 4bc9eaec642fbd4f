// Microscaled 4-bit floating point: declarations shared by the C ABI
// (fp4_api.cpp) and the kernels (fp4_quantize.cu, fp4_linear.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"

namespace mq {

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

// A quantised matrix in caller memory (row-major codes and scales).
struct Fp4Rows {
    const uint8_t *codes;
    const uint8_t *scales;
    const float *row_scale;  // NULL for MQ_FP4_MX
    int64_t rows;
};

// Device side of a packed weight: E matrices [N][K] of one format.
struct Fp4Device {
    int64_t E = 0, N = 0, K = 0;
    int fmt = 0;
    int64_t pitch = 0;  // bytes of a row of codes
    int KS = 0;         // K stages
    int64_t NT = 0;     // 128-row tiles of one matrix
    // codes [E][N][pitch]
    uint8_t *codes = nullptr;
    // scales in the order the tensor core takes them: [E][NT][KS] pieces of
    // 128 rows x one stage, each a run of 512-byte units of four scale
    // columns; byte (row % 32) * 16 + (row / 32) * 4 + column % 4 of a unit
    uint8_t *scales = nullptr;
    float *row_scale = nullptr;  // [E][N], NULL for MQ_FP4_MX
    int *err = nullptr;
    CUtensorMap map;        // codes as [E][N][pitch] bytes, boxes of 128 rows x 128 bytes
    CUtensorMap scale_map;  // scales as rows of 256 bytes, boxes of one piece
};

// Bytes of one piece of `scales` above.
constexpr int fp4_piece_bytes(int fmt) { return 128 * fp4_stage_scales(fmt); }

// X (dtype, row stride ldx elements) to codes, scales and (MQ_FP4_NV) row
// factors, `rows` output rows; output row r is X row index[r] (index NULL: r),
// and a row of zeros where index[r] is outside [0, x_rows).
mq_status launch_fp4_quantize(const void *X, mq_dtype dtype, int64_t rows, int64_t K, int64_t ldx,
                              const int32_t *index, int64_t x_rows, int fmt, uint8_t *codes,
                              uint8_t *scales, float *row_scale, cudaStream_t stream);

mq_status launch_fp4_dequantize(const Fp4Rows &x, int64_t K, int fmt, void *Y, mq_dtype dtype,
                                int64_t ldy, cudaStream_t stream);

// Row-major scales [E][N][scale pitch] to the order of Fp4Device::scales, or back.
mq_status launch_fp4_scale_order(const Fp4Device &d, uint8_t *row_major, bool to_row_major,
                                 cudaStream_t stream);

// Y[r] = x[r] * W[e]^T for the rows offsets[e] <= r < offsets[e + 1] of every
// e (offsets NULL: E is 1 and every row belongs to it). `chained`: x was
// written by the launch just before on this stream, which lets this one start
// early.
mq_status launch_fp4_linear(const Fp4Device &d, const Fp4Rows &x, const int32_t *offsets, void *Y,
                            mq_dtype dtype, int64_t ldy, bool chained, cudaStream_t stream);

// The form of launch_fp4_linear for many tokens (fp4_wide.cu).
mq_status launch_fp4_wide(const Fp4Device &d, const Fp4Rows &x, const int32_t *offsets, void *Y,
                          mq_dtype dtype, int64_t ldy, bool chained, cudaStream_t stream);

// Byte matrix [outer][rows][pitch] (outer = 0: [rows][pitch], two coordinates)
// as a tensor map with boxes of box_rows x 128 bytes, 128-byte swizzle, zero
// fill.
bool encode_bytes_map(CUtensorMap *map, const void *base, int64_t pitch, int64_t rows, int64_t outer,
                      int box_rows);

// `bytes` (a multiple of 256) as a tensor map of rows of 256 bytes with boxes
// of box_bytes, in their order in memory.
bool encode_pieces_map(CUtensorMap *map, const void *base, int64_t bytes, int box_bytes);

}  // namespace mq
