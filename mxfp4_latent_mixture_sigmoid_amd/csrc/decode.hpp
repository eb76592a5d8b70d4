// decode.hpp -- launch interface of the layer for a few tokens.
#pragma once

#include "common.hpp"
#include "mxmoe.h"

namespace mxmoe {

constexpr int DECODE_MAX_T = MOE_DECODE_MAX_T;   // the rows of a matrix-core tile

constexpr int DECODE_MAX_E = 1024;
constexpr int DECODE_MAX_WINDOW = 0x7FFF0000;    // bytes of a matrix, of h, y and [z | h_s]

// One to a cache line: counters (z has DECODE_ARMS and one more for their last arrivals); three flags, each in 64 places; then
// a counter for every expert of the list and one for every 256 columns.
constexpr int DECODE_ARMS = 16;
enum { DECODE_ROUTER, DECODE_TOP, DECODE_CAT, DECODE_Z, DECODE_FLAGS = DECODE_Z + DECODE_ARMS + 1 };
enum { DECODE_READY, DECODE_Z_DONE, DECODE_CAT_DONE };
constexpr int DECODE_COUNTER_WORDS = 32, DECODE_SHARED_LINES = DECODE_FLAGS + 3 * 64;
constexpr int DECODE_PATIENCE = 1000;        // times that a flag is asked for, about a microsecond each
constexpr int DECODE_DOWN_COLUMNS = 256;     // of a workgroup in the down product
constexpr int DECODE_ROUTER_PARTS = 4;       // workgroups that share 16 of the router's rows
constexpr int DECODE_STAGE_WORDS = 1856;     // LDS of a wave for its activations
constexpr int DECODE_OUT_STAGE_WORDS = 3200; // ... in the output product, whose activations come with their remainders

// Work items, numbered kind after kind; a kind waits for earlier ones only.
struct DecodeItems {
    int router, latent, top, gate, shared, down, sums, out;
};
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
    uint32_t *counters;              // decode_counter_lines of them
    uint32_t *claims;                // [items]
    int patience;
    float *partial;                  // [T K, Lt] y
    float *logits;                   // [DECODE_ROUTER_PARTS, T, E]
    float *weights;                  // [T, K]
    int32_t *chosen;                 // [T, K] experts
    int32_t *list;                   // [most] distinct experts, ascending
    int16_t *pairs;                  // [most, 16] the pair of (expert, token), or -1
    int most;                        // min(T K, E)
    uint16_t *z;                     // [T, ldz]: z, and zc in its place when every expert is done with it, then h_s; x itself without latent projections
    uint16_t *z_rest;                // [T, ldz]: what their rounding left; unused without latent projections
    int ldz;                         // Lt + shared
    uint16_t *h;                     // [2, T K, I]: and what its rounding left
    DecodeItems items;               // decode_items of the above
    // outputs
    float *logits_out;               // [T, E], or null
    int32_t *ids_out;                // [T, K], or null
    float *weights_out;              // [T, K], or null
    uint16_t *out;                   // [T, H] ([T, Lt] without latent projections)
};

// One token's gate and up product by 16 channels, where a wave's part of z and of its remainders fits its LDS; else by 64.
// (One token: 54 us, 57 by 64; two, with twice the experts: 65 us by 16, 64 by 64.)
__host__ __device__ inline bool decode_gate_one(const DecodeArgs &a)
{
    return a.T == 1 && 2 * ((a.Lt / 128 + 3) / 4 * 64 + 4) <= DECODE_STAGE_WORDS;
}
__host__ __device__ inline int decode_gate_items(const DecodeArgs &a) { return a.I / (decode_gate_one(a) ? 16 : 64); }   // of an expert
__host__ __device__ inline int decode_groups(const DecodeArgs &a) { return (a.Lt + DECODE_DOWN_COLUMNS - 1) / DECODE_DOWN_COLUMNS; }

// Groups of 256 columns of a down item, whose look-ups and h are then shared: two, where there are more items than places (3
// on each of 256 CUs). 8 tokens: 114 us with one, 112 with two; 4 tokens 81 with two, 87 with four; a layer of 512 latent
// columns, 3 tokens of 6 experts, 24 us with one, 27 with two.
__host__ __device__ inline int decode_down_span(const DecodeArgs &a) { return a.most * decode_groups(a) <= 768 ? 1 : 2; }
__host__ __device__ inline int decode_down_items(const DecodeArgs &a)   // of an expert
{
    return (decode_groups(a) + decode_down_span(a) - 1) / decode_down_span(a);
}

inline DecodeItems decode_items(const DecodeArgs &a)
{
    const int quads = (a.T + 3) / 4, groups = decode_groups(a);
    return {(int)(a.n_router_rows / 16) * DECODE_ROUTER_PARTS, a.has_latent ? a.Lt / 16 : 0, quads, a.most * decode_gate_items(a), a.shared / 16,
            a.most * decode_down_items(a), quads * groups, a.has_latent ? a.H / 16 : 0};
}
inline int decode_item_count(const DecodeItems &n)
{
    return n.router + n.latent + n.top + n.gate + n.shared + n.down + n.sums + n.out;
}

// Arrivals of the list's expert r at its h; of the down items at the columns of group g.
inline int decode_counter_lines(const DecodeArgs &a) { return DECODE_SHARED_LINES + a.most + decode_groups(a); }
__host__ __device__ inline uint32_t *decode_gates(const DecodeArgs &a, int r)
{
    return a.counters + (DECODE_SHARED_LINES + r) * DECODE_COUNTER_WORDS;
}
__host__ __device__ inline uint32_t *decode_columns(const DecodeArgs &a, int g) { return decode_gates(a, a.most + g); }

hipError_t launch_decode(const DecodeArgs &a, hipStream_t st);

} // namespace mxmoe
