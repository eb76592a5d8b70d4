// decode.hip -- the whole layer for up to 16 tokens in two kernels.
//
// The tokens are one row tile of the matrix-core instruction, so every weight is read once, from memory, and
// multiplied with all tokens at once: the time is the weights' (184 MB for one token of a TP8 share: the router, latent
// and shared matrices in BF16, 16 experts in MXFP4).
//
//  front_kernel  what only needs x: the router's logits, z = bf16(x W_down^T), h_s = bf16(silu(x Wg_s^T) (x Wu_s^T)).
//  rest_kernel   everything after it, one work item per workgroup, taken in the order of a ticket counter:
//    top    top-K of four tokens each; the last to finish lists the distinct experts and each one's tokens
//    gate   (expert, 16 inner channels): h = bf16(silu(z Wg^T) (z Wu^T)) of the expert's tokens
//    down   16 latent columns of every chosen expert: zc = bf16(sum w (h Wd^T)), the sum in FP32
//    out    16 output columns: out = bf16([zc | h_s] [W_up | W_ds]^T)
//
// Kinds wait for each other on counters. An item waits only for items of earlier kinds, all of which have lower tickets, and
// a ticket is drawn by a workgroup that already runs: so whatever an item waits for is done or running, and the waits end
// however many workgroups the card holds at once and whatever else runs on it. What one workgroup hands to another
// goes through agent-coherent stores and loads (sync.hpp). The front kernel clears the counters for the rest kernel.
#include "decode.hpp"
#include "select.hpp"
#include "sync.hpp"

namespace mxmoe {

namespace {

constexpr int ROWS = DECODE_MAX_T;
constexpr int FRONT_WAVES = 8, REST_WAVES = 4;

__device__ inline uint32_t *counter(const DecodeArgs &a, int i) { return a.counters + i * DECODE_COUNTER_WORDS; }

// Lane l's 16 bytes of an activation operand: row l % 16, values 8 (l / 16) .. +7 from column k on; rows past the tokens are 0.
__device__ inline u32x4_t load_operand(const uint16_t *x, int64_t ld, int T, int k)
{
    const int lane = threadIdx.x & (WAVE - 1), r = lane & 15;
    return r < T ? load16(x + r * ld + k + 8 * (lane >> 4)) : u32x4_t{0u, 0u, 0u, 0u};
}

// Lane l's four sums of a fragment are those of rows 4 (l / 16) .. +3 in column l % 16.
__device__ inline void store_sums(float *red, f32x4_t v)
{
    const int lane = threadIdx.x & (WAVE - 1);
#pragma unroll
    for (int i = 0; i < 4; i++)
        red[(4 * (lane >> 4) + i) * 16 + (lane & 15)] = v[i];
}

// Sum of one element over the waves' fragments, in wave order.
template <int WAVES>
__device__ inline float total(const float *red, int stride, int at)
{
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; w++)
        v += red[w * stride + at];
    return v;
}

// NB row blocks of a BF16 matrix [N, K] times the activations: this wave's part of K, added to acc. Loads run a batch ahead.
template <int NB, int WAVES, class Operand>
__device__ inline void bf16_blocks(const uint8_t *w, int64_t N, int64_t K, const int (&nb)[NB], f32x4_t (&acc)[NB],
                                   Operand operand)
{
    constexpr int BATCH = 4 / NB;
    const int lane = threadIdx.x & (WAVE - 1), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int steps = (int)(K / BF16_STEP), s0 = steps * wv / WAVES, s1 = steps * (wv + 1) / WAVES;
    struct Batch {
        u32x4_t b[BATCH][NB], x[BATCH];
    } now, next;
    auto load = [&](int s, Batch &q) {
#pragma unroll
        for (int i = 0; i < BATCH; i++)
            if (s + i < s1)
#pragma unroll
                for (int j = 0; j < NB; j++)
                    q.b[i][j] = load16_nt(w + bf16_block_index(nb[j], s + i, N, K) * BF16_BLOCK_BYTES + lane * 16);
#pragma unroll
        for (int i = 0; i < BATCH; i++)
            if (s + i < s1)
                q.x[i] = operand((s + i) * BF16_STEP);
    };
    load(s0, now);
    for (int s = s0; s < s1; s += BATCH) {
        load(s + BATCH, next);
#pragma unroll
        for (int i = 0; i < BATCH; i++)
            if (s + i < s1)
#pragma unroll
                for (int j = 0; j < NB; j++)
                    acc[j] = mfma16(as_bf16x8(now.x[i]), as_bf16x8(now.b[i][j]), acc[j]);
        now = next;
    }
}

// Items: pairs of shared gate and up blocks first, which take twice as long, then the latent's blocks, then the router's.
__global__ __launch_bounds__(WAVE *FRONT_WAVES, 4) void front_kernel(const DecodeArgs a)
{
    __shared__ float red[FRONT_WAVES * 2 * 256];
    const int t = threadIdx.x, wv = t / WAVE;
    if (blockIdx.x == 0 && t < DECODE_COUNTERS)
        *counter(a, t) = 0u;
    auto operand = [&](int k) { return load_operand(a.x, a.Hin, a.T, k); };
    const int pairs = a.shared / 16, latent = a.has_latent ? a.Lt / 16 : 0;
    int item = blockIdx.x;
    const int row = t / 16, col = t % 16;
    if (item < pairs) {
        f32x4_t acc[2] = {};
        const int first = (int)(a.shared_at / 16) + 2 * item, nb[2] = {first, first + 1};
        bf16_blocks<2, FRONT_WAVES>(a.w_shared, a.n_shared_rows, a.Hin, nb, acc, operand);
        store_sums(red + wv * 512, acc[0]);
        store_sums(red + wv * 512 + 256, acc[1]);
        __syncthreads();
        if (t < 256 && row < a.T) {
            const float g = total<FRONT_WAVES>(red, 512, t), u = total<FRONT_WAVES>(red, 512, 256 + t);
            a.acat[(int64_t)row * a.ldcat + a.Lt + item * 16 + col] = (uint16_t)f32_to_bf16_bits(silu_f32(g) * u);
        }
        return;
    }
    item -= pairs;
    const bool z = item < latent;
    if (!z)
        item -= latent;
    f32x4_t acc[1] = {};
    const int nb[1] = {item};
    bf16_blocks<1, FRONT_WAVES>(z ? a.w_latent : a.w_router, z ? a.n_latent_rows : a.n_router_rows, a.Hin, nb, acc, operand);
    store_sums(red + wv * 256, acc[0]);
    __syncthreads();
    if (t >= 256 || row >= a.T)
        return;
    const float v = total<FRONT_WAVES>(red, 256, t);
    const int n = item * 16 + col;
    if (z)
        a.z[(int64_t)row * a.Lt + n] = (uint16_t)f32_to_bf16_bits(v);
    else if (n < a.E)
        a.logits[(int64_t)row * a.E + n] = a.bias ? v + a.bias[n] : v;
}

// Until counter i has reached `target`. One thread asks; what follows in any thread is after the answer.
__device__ inline uint32_t wait_for(const DecodeArgs &a, int i, uint32_t target, uint32_t *sh)
{
    if (threadIdx.x == 0) {
        uint32_t v;
        while ((v = __hip_atomic_load(counter(a, i), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) < target)
            __builtin_amdgcn_s_sleep(1);
        *sh = v;
    }
    __syncthreads();
    const uint32_t v = *sh;
    __syncthreads();
    asm volatile("" ::: "memory");
    return v;
}

// This workgroup's stores have completed; then its arrival. Returns the arrivals before it (to thread 0).
__device__ inline uint32_t arrive(const DecodeArgs &a, int i)
{
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    asm volatile("" ::: "memory");
    __syncthreads();
    return threadIdx.x == 0 ? __hip_atomic_fetch_add(counter(a, i), 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0u;
}

template <int SLOTS>
__device__ inline void top_item(const DecodeArgs &a, int item, uint32_t *words)
{
    __shared__ uint64_t scratch[REST_WAVES][WAVE];
    const int lane = threadIdx.x & (WAVE - 1), wv = threadIdx.x / WAVE, t = item * REST_WAVES + wv;
    const int T = a.T, K = a.K, E = a.E, P = T * K;
    const auto ids = flat_rsrc(a.ids, (int64_t)P * 4), weights = flat_rsrc(a.weights, (int64_t)P * 4);
    if (t < T) {
        uint32_t key[SLOTS];
#pragma unroll
        for (int j = 0; j < SLOTS; j++) {
            const int e = lane + WAVE * j;
            // no key is 0, which stands for no expert (only a NaN with every bit set has it): ids are always in range
            key[j] = e < E ? max(order_key(a.logits[(int64_t)t * E + e]), 1u) : 0u;
        }
        int id;
        float w;
        select_best<SLOTS>(K, key, scratch[wv], &id, &w);
        if (lane < K) {
            store4_sc1(ids, (t * K + lane) * 4, (uint32_t)id);
            store4_sc1(weights, (t * K + lane) * 4, __float_as_uint(w));
            if (a.ids_out)
                a.ids_out[t * K + lane] = id;
            if (a.weights_out)
                a.weights_out[t * K + lane] = w;
        }
    }
    const uint32_t before = arrive(a, DECODE_TOP);
    if (threadIdx.x == 0)
        words[0] = before;
    __syncthreads();
    if (words[0] != (uint32_t)((T + REST_WAVES - 1) / REST_WAVES - 1))
        return;
    __syncthreads();
    // The last workgroup lists the experts that any token chose, in ascending order, and for each the pair and weight of
    // every token (pair -1: not chosen).
    uint32_t *masks = words;              // of an expert's tokens
    int *chosen = reinterpret_cast<int *>(words + E), *sh = chosen + P;
    constexpr int NTHR = WAVE * REST_WAVES;
    for (int e = threadIdx.x; e < E; e += NTHR)
        masks[e] = 0u;
    __syncthreads();
    for (int p = threadIdx.x; p < P; p += NTHR) {
        const int e = (int)load4_sc1(ids, p * 4);
        chosen[p] = e;
        atomicOr(&masks[e], 1u << p / K);
    }
    __syncthreads();
    const int per = (E + NTHR - 1) / NTHR, e0 = (int)threadIdx.x * per, e1 = min(E, e0 + per);
    int n = 0, count;
    for (int e = e0; e < e1; e++)
        n += masks[e] != 0u;
    int rank = block_excl_scan(n, sh, &count);
    const auto list = flat_rsrc(a.list, (int64_t)a.most * 4);
    const auto pairs = flat_rsrc(a.pairs, (int64_t)a.most * ROWS * 4), shares = flat_rsrc(a.shares, (int64_t)a.most * ROWS * 4);
    for (int e = e0; e < e1; e++) {
        if (masks[e] == 0u)
            continue;
        store4_sc1(list, rank * 4, (uint32_t)e);
        for (int r = 0; r < ROWS; r++) {
            int p = -1;
            if (masks[e] >> r & 1u)
                for (int j = 0; j < K; j++)
                    if (chosen[r * K + j] == e)
                        p = r * K + j;
            store4_sc1(pairs, (rank * ROWS + r) * 4, (uint32_t)p);
            store4_sc1(shares, (rank * ROWS + r) * 4, p < 0 ? 0u : load4_sc1(weights, p * 4));
        }
        rank++;
    }
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    asm volatile("" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0)
        __hip_atomic_store(counter(a, DECODE_READY), (uint32_t)count, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// One MX block times a step's activations.
__device__ inline f32x4_t mx_step(u32x4_t codes, uint32_t scales, const u32x4_t (&x)[4], f32x4_t acc)
{
#pragma unroll
    for (int j = 0; j < 4; j++)
        acc = mfma16(as_bf16x8(x[j]), mx_dequant8(codes[j], e8m0_to_f32((scales >> (8 * j)) & 0xFFu)), acc);
    return acc;
}

__device__ inline void gate_item(const DecodeArgs &a, int item, float *red, uint32_t *sh)
{
    const int lane = threadIdx.x & (WAVE - 1), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int cols = a.I / 16, r = item / cols, cp = item % cols;
    const int experts = (int)wait_for(a, DECODE_READY, 1, sh);
    if (r >= experts)
        return;
    const auto pairs = flat_rsrc(a.pairs, (int64_t)a.most * ROWS * 4);
    const int e = __builtin_amdgcn_readfirstlane((int)load4_sc1(flat_rsrc(a.list, (int64_t)a.most * 4), r * 4));
    const int pair = (int)load4_sc1(pairs, (r * ROWS + (int)threadIdx.x / 8 % ROWS) * 4);   // of the row stored below
    const int steps = a.Lt / MX_STEP, s0 = steps * wv / REST_WAVES, s1 = steps * (wv + 1) / REST_WAVES;
    const uint8_t *w = a.gateup + e * a.gateup_stride + (int64_t)2 * cp * steps * MX_BLOCK_BYTES;
    constexpr int BATCH = 4;   // steps in flight
    f32x4_t acc[2] = {};
    for (int s = s0; s < s1; s += BATCH) {
        u32x4_t codes[BATCH][2];
        uint32_t scales[BATCH][2];
#pragma unroll
        for (int i = 0; i < BATCH; i++)
            if (s + i < s1)
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    const uint8_t *blk = w + ((int64_t)j * steps + s + i) * MX_BLOCK_BYTES;
                    codes[i][j] = load16_nt(blk + lane * 16);
                    scales[i][j] = load4_nt(blk + MX_CODE_BYTES + 4 * (lane & 15));
                }
#pragma unroll
        for (int i = 0; i < BATCH; i++)
            if (s + i < s1) {
                u32x4_t x[4];
#pragma unroll
                for (int j = 0; j < 4; j++)
                    x[j] = load_operand(a.z, a.Lt, a.T, (s + i) * MX_STEP + 32 * j);
#pragma unroll
                for (int j = 0; j < 2; j++)
                    acc[j] = mx_step(codes[i][j], scales[i][j], x, acc[j]);
            }
    }
    store_sums(red + wv * 512, acc[0]);
    store_sums(red + wv * 512 + 256, acc[1]);
    __syncthreads();
    // two channels of a row per thread
    const int t = threadIdx.x, row = t / 8, c = t % 8 * 2;
    if (row < a.T && row < ROWS && pair >= 0) {
        float h[2];
#pragma unroll
        for (int i = 0; i < 2; i++)
            h[i] = silu_f32(total<REST_WAVES>(red, 512, row * 16 + c + i)) *
                   total<REST_WAVES>(red, 512, 256 + row * 16 + c + i);
        store4_sc1(flat_rsrc(a.h, (int64_t)a.T * a.K * a.I * 2), (pair * a.I + cp * 16 + c) * 2, pack_bf16x2(h[0], h[1]));
    }
    arrive(a, DECODE_GATE);
}

// Expert e is wave e % 4's, and a wave adds its experts in ascending order: so a token's sum is added in an order that its own
// experts alone decide, and its outputs are the same bits whatever tokens come with it.
__device__ inline void down_item(const DecodeArgs &a, int item, float *red, uint32_t *sh)
{
    __shared__ uint32_t mine[REST_WAVES][ROWS * 32];   // this wave's experts: rank, and number above
    const int lane = threadIdx.x & (WAVE - 1), wv = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int experts = (int)wait_for(a, DECODE_READY, 1, sh);
    const auto list = flat_rsrc(a.list, (int64_t)a.most * 4);
    int count = 0;
    for (int r0 = 0; r0 < experts; r0 += WAVE) {
        const int r = r0 + lane, e = r < experts ? (int)load4_sc1(list, r * 4) : -1;
        const bool own = e >= 0 && e % REST_WAVES == wv;
        const uint64_t owned = __ballot(own);
        if (own)
            mine[wv][count + __popcll(owned & ((1ull << lane) - 1))] = (uint32_t)(r | e << 16);
        count += (int)__popcll(owned);
    }
    wait_for(a, DECODE_GATE, (uint32_t)(experts * (a.I / 16)), sh);   // its barriers order the list above, too
    const auto h = flat_rsrc(a.h, (int64_t)a.T * a.K * a.I * 2);
    const auto pairs = flat_rsrc(a.pairs, (int64_t)a.most * ROWS * 4), shares = flat_rsrc(a.shares, (int64_t)a.most * ROWS * 4);
    const int steps = a.I / MX_STEP;
    f32x4_t sum = {};
    for (int i = 0; i < count; i++) {
        const uint32_t next = (uint32_t)__builtin_amdgcn_readfirstlane((int)mine[wv][i]);
        const int r = next & 0xFFFF, e = next >> 16;
        const int pair = (int)load4_sc1(pairs, (r * ROWS + (lane & 15)) * 4);   // of the operand's row
        const u32x4_t theirs = __builtin_bit_cast(u32x4_t, load16_sc1(pairs, (r * ROWS + 4 * (lane >> 4)) * 4));   // the sums' rows
        const f32x4_t share = load16_sc1(shares, (r * ROWS + 4 * (lane >> 4)) * 4);
        const uint8_t *w = a.down + e * a.down_stride + (int64_t)item * steps * MX_BLOCK_BYTES;
        f32x4_t y = {};
        for (int s = 0; s < steps; s++) {
            const uint8_t *blk = w + (int64_t)s * MX_BLOCK_BYTES;
            const u32x4_t codes = load16_nt(blk + lane * 16);
            const uint32_t scales = load4_nt(blk + MX_CODE_BYTES + 4 * (lane & 15));
            u32x4_t x[4];
#pragma unroll
            for (int j = 0; j < 4; j++)
                x[j] = pair >= 0 ? __builtin_bit_cast(u32x4_t, load16_sc1(h, (pair * a.I + s * MX_STEP + 32 * j + 8 * (lane >> 4)) * 2))
                                 : u32x4_t{0u, 0u, 0u, 0u};
            y = mx_step(codes, scales, x, y);
        }
#pragma unroll
        for (int i = 0; i < 4; i++)   // an expert's values that are not finite reach its own tokens only
            sum[i] = (int)theirs[i] >= 0 ? fmaf(share[i], y[i], sum[i]) : sum[i];
    }
    store_sums(red + wv * 256, sum);
    __syncthreads();
    const int t = threadIdx.x, row = t / 8, c = t % 8 * 2;
    if (row < a.T && row < ROWS) {
        const uint32_t v = pack_bf16x2(total<REST_WAVES>(red, 256, row * 16 + c), total<REST_WAVES>(red, 256, row * 16 + c + 1));
        if (a.has_latent)
            store4_sc1(flat_rsrc(a.acat, (int64_t)a.T * a.ldcat * 2), (row * a.ldcat + item * 16 + c) * 2, v);
        else
            *reinterpret_cast<uint32_t *>(a.out + (int64_t)row * a.Lt + item * 16 + c) = v;
    }
    if (a.has_latent)
        arrive(a, DECODE_DOWN);
}

__device__ inline void out_item(const DecodeArgs &a, int item, float *red, uint32_t *sh)
{
    const int wv = threadIdx.x / WAVE;
    wait_for(a, DECODE_DOWN, (uint32_t)(a.Lt / 16), sh);
    const auto acat = flat_rsrc(a.acat, (int64_t)a.T * a.ldcat * 2);
    f32x4_t acc[1] = {};
    const int nb[1] = {item}, lane = threadIdx.x & (WAVE - 1), r = lane & 15;
    bf16_blocks<1, REST_WAVES>(a.w_out, a.H, a.ldcat, nb, acc, [&](int k) {
        return r < a.T ? __builtin_bit_cast(u32x4_t, load16_sc1(acat, (r * a.ldcat + k + 8 * (lane >> 4)) * 2))
                       : u32x4_t{0u, 0u, 0u, 0u};
    });
    store_sums(red + wv * 256, acc[0]);
    __syncthreads();
    const int t = threadIdx.x, row = t / 8, c = t % 8 * 2;
    if (row < a.T && row < ROWS)
        *reinterpret_cast<uint32_t *>(a.out + (int64_t)row * a.H + item * 16 + c) =
            pack_bf16x2(total<REST_WAVES>(red, 256, row * 16 + c), total<REST_WAVES>(red, 256, row * 16 + c + 1));
}

template <int SLOTS>
__global__ __launch_bounds__(WAVE *REST_WAVES, 4) void rest_kernel(const DecodeArgs a)
{
    // the items' sums over the waves; the list's masks, chosen experts and scan
    constexpr int SUMS = REST_WAVES * 512, WORDS = SLOTS * WAVE + ROWS * 32 + 16;
    __shared__ uint32_t lds[SUMS > WORDS ? SUMS : WORDS];
    __shared__ uint32_t sh;
    float *red = reinterpret_cast<float *>(lds);
    if (threadIdx.x == 0)
        sh = __hip_atomic_fetch_add(counter(a, DECODE_TICKET), 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    int item = __builtin_amdgcn_readfirstlane((int)sh);
    __syncthreads();
    const DecodeItems n = decode_items(a);
    if (item < n.top)
        return top_item<SLOTS>(a, item, lds);
    item -= n.top;
    if (item < n.gate)
        return gate_item(a, item, red, &sh);
    item -= n.gate;
    if (item < n.down)
        return down_item(a, item, red, &sh);
    out_item(a, item - n.down, red, &sh);
}

} // namespace

hipError_t launch_decode(const DecodeArgs &a, hipStream_t st)
{
    const unsigned front = (unsigned)(a.shared / 16 + (a.has_latent ? a.Lt / 16 : 0) + a.n_router_rows / 16);
    hipLaunchKernelGGL(front_kernel, dim3(front), dim3(WAVE * FRONT_WAVES), 0, st, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    const DecodeItems n = decode_items(a);
    const dim3 grid((unsigned)(n.top + n.gate + n.down + n.out)), threads(WAVE * REST_WAVES);
    if (a.E <= 4 * WAVE)
        hipLaunchKernelGGL(rest_kernel<4>, grid, threads, 0, st, a);
    else
        hipLaunchKernelGGL(rest_kernel<16>, grid, threads, 0, st, a);
    return hipGetLastError();
}

} // namespace mxmoe
