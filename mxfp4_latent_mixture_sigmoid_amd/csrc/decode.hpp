// decode.hpp -- launch interface of the layer for a few tokens in two kernels.
#pragma once

#include "common.hpp"
#include "mxmoe.h"

namespace mxmoe {

constexpr int DECODE_MAX_T = MOE_DECODE_MAX_T;   // the rows of a matrix-core tile

// Counters, on cache lines of their own.
enum { DECODE_TICKET, DECODE_TOP, DECODE_READY, DECODE_GATE, DECODE_DOWN, DECODE_COUNTERS };
constexpr int DECODE_COUNTER_WORDS = 32;

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
    uint32_t *counters;
    float *logits;                   // [T, E]
    int32_t *ids;                    // [T, K]
    float *weights;                  // [T, K]
    int32_t *list;                   // [most] distinct experts, ascending
    int32_t *pairs;                  // [most, 16] the pair of (expert, token), or -1
    float *shares;                   // [most, 16] its weight
    int most;                        // min(T K, E)
    uint16_t *z;                     // [T, Lt]; x itself without latent projections
    uint16_t *acat;                  // [T, ldcat]: zc, then h_s
    int ldcat;
    uint16_t *h;                     // [T K, I]
    // outputs
    int32_t *ids_out;                // [T, K], or null
    float *weights_out;              // [T, K], or null
    uint16_t *out;                   // [T, H] ([T, Lt] without latent projections)
};

// Work items of the second kernel, in the order in which they are taken.
struct DecodeItems {
    int top, gate, down, out;
};
__host__ __device__ inline DecodeItems decode_items(const DecodeArgs &a)
{
    return {(a.T + 3) / 4, a.most * (a.I / 16), a.Lt / 16, a.has_latent ? a.H / 16 : 0};
}

hipError_t launch_decode(const DecodeArgs &a, hipStream_t st);

} // namespace mxmoe
