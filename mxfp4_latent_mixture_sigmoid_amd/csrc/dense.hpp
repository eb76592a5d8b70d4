// dense.hpp -- launch interfaces of the dense 8-bit path: norm, quantisation and 8-bit products.
#pragma once

#include "common.hpp"
#include "mxmoe.h"

namespace mxmoe {

// moe_norm, or (norm = false) the quantisation of x's rows alone.
hipError_t launch_norm(const moe_norm_args &a, bool norm, hipStream_t st);
hipError_t launch_block_norm(const moe_block_norm_args &a, hipStream_t st);
hipError_t launch_dequantise(const int8_t *codes, int64_t ldc, const float *scales, int32_t T, int32_t K, uint16_t *out,
                             int64_t ldo, hipStream_t st);

// Packed weights of the dense products: N rows (gate and up rows alternating per 16 when gated) padded to 16, K bytes a
// row padded to STAGE_K, in 1 KiB blocks of 16 rows x 64 bytes. Lane l's 16 bytes of a block are its operand of the
// 16x16x64 8-bit or 16x16x32 BF16 matrix-core instruction: row l % 16, bytes 16 (l / 16) .. +15. Blocks are ordered
// by 128-byte K stage, then row block, then 64-byte half: workgroups that go through K together sweep
// one contiguous range (chunks of 4 or 8 stages per row block, or whole rows, were slower by 0 to 15%
// in every few-token product, and equal in the others).
constexpr int BLOCK_BYTES = 1024;
constexpr int STAGE_K = 128;
constexpr int STAGE_BYTES = 2 * BLOCK_BYTES;   // of one row block

__host__ __device__ inline int64_t row_blocks(int64_t n, bool glu) { return (n + 15) / 16 * (glu ? 2 : 1); }
__host__ __device__ inline int64_t stages(int64_t k) { return (k + STAGE_K - 1) / STAGE_K; }

// What every dense product takes.
struct ProductArgs {
    const int8_t *x;       // rows of K bytes
    int64_t ldx;           // bytes between them
    const uint8_t *w;      // packed blocks
    void *out;
    int64_t ldo;           // outputs between rows
    int T, N, K;           // tokens, output columns, bytes
    int nblk;              // row blocks of w
    int glu, out_type;
    int direct;            // direct loads to LDS take x's rows as they are
};
struct I8Args : ProductArgs {
    const float *sx;       // [T]
    const float *sw;       // [16 * row blocks], packed row order
    const float *bias;     // [N] padded to 16, or null
};
// Whether the product of these sizes takes rows that are not `direct`; else they have to be restaged.
bool i8_takes_any_rows(const I8Args &g);
hipError_t launch_i8_product(const I8Args &g, hipStream_t st);
hipError_t launch_i8_pack(const moe_linear_config &c, const moe_linear_weights &w, uint8_t *blocks, float *scales,
                          float *bias, hipStream_t st);

struct Bf16Args : ProductArgs {
    const float *bias;     // [N] padded to 16, or null
    const void *residual;  // [T, N] of res_type, or null; may be `out`
    int64_t ldr;           // values between its rows
    int res_type, act;     // moe_type, moe_linear_act
};
bool bf16_takes_any_rows(const Bf16Args &g);
hipError_t launch_bf16_product(const Bf16Args &g, hipStream_t st);

// T rows of K bytes with any alignment -> rows of STAGE_K * stages(K) bytes, zero-padded.
hipError_t launch_restage(const int8_t *x, int64_t ldx, int T, int K, int8_t *dst, hipStream_t st);
// [n, k bytes] weights (and up weights, or null) -> packed blocks; vectors of the rows in packed order (each may be null).
hipError_t launch_pack_product(const void *w, const void *w_up, int64_t n, int64_t k, uint8_t *blocks, hipStream_t st);
hipError_t launch_pack_vectors(const float *scales, const float *scales_up, const float *bias, int64_t n, int64_t nblk,
                               float *scales_out, float *bias_out, hipStream_t st);

} // namespace mxmoe
