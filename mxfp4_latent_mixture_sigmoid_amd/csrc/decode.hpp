// decode.hpp -- launch interface of the layer for a few tokens in two kernels.
#pragma once

#include "common.hpp"
#include "mxmoe.h"

namespace mxmoe {

constexpr int DECODE_MAX_T = MOE_DECODE_MAX_T;   // the rows of a matrix-core tile

constexpr int DECODE_MAX_E = 1024;
constexpr int DECODE_MAX_WINDOW = 0x7FFF0000;    // bytes of a matrix, of h and of [zc | h_s]

// One to a cache line: two sets of arrival counters, each of DECODE_ARMS and one more for their last arrivals; three flags,
// each in 64 places.
enum { DECODE_GATE, DECODE_DOWN };
enum { DECODE_READY, DECODE_GATE_DONE, DECODE_DOWN_DONE };
constexpr int DECODE_ARMS = 16, DECODE_COUNTERS = 2 * (DECODE_ARMS + 1);
constexpr int DECODE_PATIENCE = 1000;   // times that a flag is asked for, about a microsecond each
constexpr int DECODE_COUNTER_WORDS = 32;
constexpr int DECODE_COUNTER_LINES = DECODE_COUNTERS + 3 * 64;
constexpr int DECODE_PARTS = 4;   // workgroups that share 16 columns of the down product, for more than one token
constexpr int DECODE_STAGE_WORDS = 1856;         // LDS of a wave for its activations

struct DecodeArgs {
    const uint16_t *x;               // [T, Hin]
    const float *bias;               // [E], or null
    int T, Hin, H, Lt, E, K, I;
    int shared;                      // channels of all shared experts, 0 without
    int has_latent;
    // packed weights
    const uint8_t *w_router, *w_latent, *w_shared, *w_out, *gateup, *down;
    int64_t n_router_rows, n_latent_rows, n_shared_rows, shared_at;   // rows of their matrices; the shared ones' first row
    int64_t gateup_stride, down_stride;
    // workspace
    uint32_t *counters;              // DECODE_COUNTER_LINES lines
    uint32_t *column_counters;       // [Lt / 16] arrivals of a column block's parts
    uint32_t *claims;                // [items] of the second kernel
    int patience;
    float *partial;                  // [Lt / 16][T K][16] their y
    float *logits;                   // [T, E]
    float *weights;                  // [T, K]
    int32_t *list;                   // [most] distinct experts, ascending
    int16_t *pairs;                  // [most, 16] the pair of (expert, token), or -1
    int most;                        // min(T K, E)
    uint16_t *z;                     // [T, Lt]; x itself without latent projections
    uint16_t *z_rest;                // [T, Lt] what z's rounding left; unused without latent projections
    uint16_t *acat;                  // [T, ldcat]: zc, then h_s
    int ldcat;
    uint16_t *h;                     // [T K, I]
    // outputs
    int32_t *ids_out;                // [T, K], or null
    float *weights_out;              // [T, K], or null
    uint16_t *out;                   // [T, H] ([T, Lt] without latent projections)
};

// Work items of the second kernel, numbered kind after kind. One token's experts are few enough for one
// workgroup to a column block; more are shared by DECODE_PARTS.
struct DecodeItems {
    int top, gate, down, out, parts;
};
// One token's gate and up product by 16 channels, where a wave's part of z and of its remainders fits its LDS; else by 64.
__host__ __device__ inline bool decode_gate_one(const DecodeArgs &a)
{
    return a.T == 1 && 2 * ((a.Lt / 128 + 3) / 4 * 64 + 4) <= DECODE_STAGE_WORDS;
}
__host__ __device__ inline DecodeItems decode_items(const DecodeArgs &a)
{
    const int parts = a.T == 1 ? 1 : DECODE_PARTS;
    return {1, a.most * (a.I / (decode_gate_one(a) ? 16 : 64)), a.Lt / 16 * parts, a.has_latent ? a.H / 16 : 0, parts};
}
__host__ __device__ inline int decode_item_count(const DecodeItems &n) { return n.top + n.gate + n.down + n.out; }

hipError_t launch_decode(const DecodeArgs &a, hipStream_t st);

} // namespace mxmoe
