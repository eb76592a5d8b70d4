// dense.hpp -- launch interfaces of the dense 8-bit path: norm, quantisation and 8-bit products.
#pragma once

#include "common.hpp"
#include "mxmoe.h"

namespace mxmoe {

// moe_norm, or (norm = false) the quantisation of x's rows alone.
hipError_t launch_norm(const moe_norm_args &a, bool norm, hipStream_t st);
hipError_t launch_dequantise(const int8_t *codes, int64_t ldc, const float *scales, int32_t T, int32_t K, uint16_t *out,
                             int64_t ldo, hipStream_t st);

// Packed 8-bit weights: N rows (gate and up rows alternating per 16 when glu) padded to 16, K padded to
// I8_STAGE, in 1 KiB blocks of 16 rows x 64 codes. Lane l's 16 bytes of a block are its operand of the
// 16x16x64 8-bit matrix-core instruction: row l % 16, codes 16 (l / 16) .. +15. Blocks are ordered
// by 128-wide K stage, then row block, then 64-wide half: workgroups that go through K together sweep
// one contiguous range (chunks of 4 or 8 stages per row block, or whole rows, were slower by 0 to 15%
// in every few-token product, and equal in the others).
constexpr int I8_BLOCK_BYTES = 1024;
constexpr int I8_STAGE = 128;
constexpr int I8_STAGE_BYTES = 2 * I8_BLOCK_BYTES;   // of one row block

__host__ __device__ inline int64_t i8_row_blocks(int64_t n, bool glu) { return (n + 15) / 16 * (glu ? 2 : 1); }
__host__ __device__ inline int64_t i8_stages(int64_t k) { return (k + I8_STAGE - 1) / I8_STAGE; }

struct I8Args {
    const int8_t *x;       // codes [T, K]
    int64_t ldx;
    const float *sx;       // [T]
    const uint8_t *w;      // packed blocks
    const float *sw;       // [16 * row blocks], packed row order
    const float *bias;     // [N] padded to 16, or null
    void *out;
    int64_t ldo;
    int T, N, K;           // N output columns
    int nblk;              // row blocks of w
    int glu, out_type;
    int direct;            // rows at 16-byte steps and K in whole 16-byte chunks
};
// Whether the product of these sizes takes rows that are not `direct`; else they have to be restaged.
bool i8_takes_any_rows(const I8Args &g);
hipError_t launch_i8_product(const I8Args &g, hipStream_t st);
// Codes [T, K] with any row alignment -> [T, I8_STAGE * stages] rows, zero-padded.
hipError_t launch_i8_restage(const int8_t *x, int64_t ldx, int T, int K, int8_t *dst, hipStream_t st);
hipError_t launch_i8_pack(const moe_linear_config &c, const moe_linear_weights &w, uint8_t *blocks, float *scales,
                          float *bias, hipStream_t st);

} // namespace mxmoe
