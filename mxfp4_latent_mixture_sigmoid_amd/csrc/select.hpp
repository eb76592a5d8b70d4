// select.hpp -- deterministic top-K of one token's logits by one wave, with sigmoid gate weights.
#pragma once

#include "wave.hpp"

namespace mxmoe {

// Order-preserving key of a float: unsigned comparison of keys equals the float comparison, with
// -0 mapped to the key of +0 so the two compare equal. Every non-NaN value has a key > 0.
__device__ inline uint32_t order_key(float f)
{
    uint32_t u = __float_as_uint(f);
    if (u == 0x80000000u)
        u = 0u;
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ inline float key_value(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k); }

// Top-K of one token by one wave from the order keys (0 = no expert), ties to the lower expert, and
// the gate weights: sigmoid of the selected logits over their sum. Lane k < K gets the rank-k expert and its weight.
// Every candidate becomes one 64-bit value, key above the complemented expert index, so the order
// (key descending, expert ascending) is plain unsigned order and all values differ.
//  1. bound: the K-th largest of the 64 lane maxima (keys only), built bit by bit from the top with
//     one ballot per bit. At least K lanes hold a key >= bound, so every selected key is >= bound.
//  2. The candidates (keys >= bound; K or a few more in practice) are gathered into `scratch` (64
//     entries of this wave); each ranks itself against all of them by lane broadcasts, and the K
//     best are placed at their ranks, so lane k then holds the rank-k expert.
//  3. With more than 64 candidates (heavy ties), K rounds of wave-wide maxima select directly.
template <int SLOTS>
__device__ inline void select_best(int K, const uint32_t *key, uint64_t *scratch, int *id, float *weight)
{
    const int lane = threadIdx.x & (WAVE - 1);
    uint64_t c[SLOTS];
    uint32_t mk = 0u;
#pragma unroll
    for (int j = 0; j < SLOTS; j++) {
        c[j] = key[j] ? ((uint64_t)key[j] << 32) | (uint32_t)~(uint32_t)(lane + WAVE * j) : 0;
        mk = key[j] > mk ? key[j] : mk;
    }
    uint32_t bound = 0u;
    for (int b = 31; b >= 0; b--) {
        const uint32_t cand = bound | (1u << b);
        if ((int)__popcll(__ballot(mk >= cand)) >= K)
            bound = cand;
    }
    int n = 0;
#pragma unroll
    for (int j = 0; j < SLOTS; j++)
        n += (key[j] != 0u && key[j] >= bound) ? 1 : 0;
    const int incl = wave_incl_scan(n);
    const int total = __shfl(incl, WAVE - 1, WAVE);
    uint32_t my_key = 0u;
    int my_id = 0;
    if (total <= WAVE) {
        int pos = incl - n;
#pragma unroll
        for (int j = 0; j < SLOTS; j++)
            if (key[j] != 0u && key[j] >= bound)
                scratch[pos++] = c[j];
        meet_lanes();
        const uint64_t mine = lane < total ? scratch[lane] : 0;
        const uint32_t mh = (uint32_t)(mine >> 32), ml = (uint32_t)mine;
        int rank = 0;
        for (int m = 0; m < total; m++) {   // candidate m broadcast from its lane
            const uint32_t oh = __builtin_amdgcn_readlane(mh, m), ol = __builtin_amdgcn_readlane(ml, m);
            rank += (oh > mh || (oh == mh && ol > ml)) ? 1 : 0;
        }
        meet_lanes();
        if (lane < total && rank < K)
            scratch[rank] = mine;
        meet_lanes();
        const uint64_t r = lane < K ? scratch[lane] : 0;
        meet_lanes();   // the caller's next token
        my_key = (uint32_t)(r >> 32);
        my_id = (int)~(uint32_t)r;
    } else {
        uint64_t left[SLOTS];
#pragma unroll
        for (int j = 0; j < SLOTS; j++)
            left[j] = c[j];
        for (int k = 0; k < K; k++) {
            uint64_t bm = left[0];
#pragma unroll
            for (int j = 1; j < SLOTS; j++)
                bm = left[j] > bm ? left[j] : bm;
            const uint32_t wk = wave_max_u32((uint32_t)(bm >> 32));
            const uint32_t wl = wave_max_u32((uint32_t)(bm >> 32) == wk ? (uint32_t)bm : 0u);
            if (lane == k) {
                my_key = wk;
                my_id = (int)~wl;
            }
            const uint64_t win = ((uint64_t)wk << 32) | wl;
#pragma unroll
            for (int j = 0; j < SLOTS; j++)
                if (left[j] == win)
                    left[j] = 0;
        }
    }
    const float s = lane < K ? 1.0f / (1.0f + expf(-key_value(my_key))) : 0.0f;
    const float sum = wave_sum_f32(s);
    *id = my_id;
    *weight = s / sum;
}

} // namespace mxmoe
