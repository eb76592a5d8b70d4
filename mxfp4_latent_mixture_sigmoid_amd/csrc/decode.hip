// decode.hip -- the whole layer for up to 16 tokens in two kernels.
//
// The tokens are one row tile of the matrix-core instruction, so every weight is read once, from memory, and
// multiplied with all tokens at once: the time is the weights' (184 MB for one token of a TP8 share: the router, latent
// and shared matrices in BF16, 16 experts in MXFP4).
//
//  front_kernel  what only needs x: the router's logits, z = x W_down^T, h_s = bf16(silu(x Wg_s^T) (x Wu_s^T)).
//  rest_kernel   everything after it, one work item per workgroup, taken in the order of a ticket counter:
//    top    the top-K of every token; the list of distinct experts and each one's tokens
//    gate   (expert, 16 or 32 inner channels): h = bf16(silu(z Wg^T) (z Wu^T)) of the expert's tokens
//    down   16 latent columns of every chosen expert, or of a quarter of them: zc = bf16(sum w (h Wd^T)), summed in FP32
//    out    16 output columns: out = bf16([zc | h_s] [W_up | W_ds]^T)
//
// z is kept in two BF16 parts, the rounded value and what the rounding left, because its rounding alone reaches every
// expert's gate, up and product (0.4% of a small layer's output in the mean square, against 0.3% without); the
// remainders are rows 8 to 15 of the tile for up to 8 tokens, at no cost, and a second operand for more.
//
// Kinds wait for each other. An item waits only for items of earlier kinds, all of which have lower tickets, and a ticket
// is drawn by a workgroup that already runs: so whatever an item waits for is done or
// being worked on, and the waits end however many workgroups the card holds at once and whatever else runs on it. What one
// workgroup hands to another goes through agent-coherent stores and loads (sync.hpp). A counter that hundreds of
// workgroups ask for is a queue at one memory channel (1057 of them: 100 us): the last to arrive therefore writes a flag in
// 64 places, and each workgroup asks for one of them. The front kernel clears counters and flags for the rest kernel.
#include "decode.hpp"
#include "select.hpp"
#include "sync.hpp"

namespace mxmoe {

namespace {

constexpr int ROWS = DECODE_MAX_T, HALF = ROWS / 2;
constexpr int FRONT_WAVES = 8, REST_WAVES = 4;
constexpr int FLAGS = WAVE;                 // places of a flag
constexpr int STAGE_WORDS = 2048;           // LDS of a wave for its activations, where they fit

__device__ inline uint32_t *counter(const DecodeArgs &a, int i) { return a.counters + i * DECODE_COUNTER_WORDS; }
__device__ inline uint32_t *flag(const DecodeArgs &a, int i, int place)
{
    return a.counters + (DECODE_COUNTERS + i * FLAGS + place) * DECODE_COUNTER_WORDS;
}

__device__ inline int lane_id() { return threadIdx.x & (WAVE - 1); }
__device__ inline int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE); }
constexpr u32x4_t ZERO = {0u, 0u, 0u, 0u};

// Lane l's four sums of a fragment are those of rows 4 (l / 16) .. +3 in column l % 16.
__device__ inline void store_sums(float *red, f32x4_t v)
{
    const int lane = lane_id();
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

// A wave's part of a BF16 product: 32-wide steps s0 .. s1 - 1 of NB row blocks, all T tokens at once. The weights are loaded
// DEPTH steps ahead, the first before anything is known of the activations. Those go through LDS where the wave's part of
// them fits (few tokens: a step's operand would be a load with 4 T lanes of use), else straight to registers, AHEAD
// steps ahead.
template <int NB, int DEPTH, int AHEAD>
struct Bf16Part {
    static_assert(DEPTH % AHEAD == 0, "slots");
    u32x4_t b[DEPTH][NB];
    const uint8_t *w, *at;   // the matrix, and the next step's first block
    int64_t N, K;
    int nb0, s0, s1, next, pitch;   // next step, blocks from a row block to the next one in its K chunk

    __device__ void seek()
    {
        at = w + bf16_block_index(nb0, next, N, K) * BF16_BLOCK_BYTES;
        pitch = min(BF16_CHUNK_STEPS, (int)(K / BF16_STEP) - next / BF16_CHUNK_STEPS * BF16_CHUNK_STEPS);
    }
    // Steps are loaded one after another, each into slot (step - s0) % DEPTH.
    __device__ void load(int slot)
    {
        if (next >= s1)
            return;
#pragma unroll
        for (int j = 0; j < NB; j++)
            b[slot][j] = load16_nt(at + j * pitch * BF16_BLOCK_BYTES + lane_id() * 16);
        at += BF16_BLOCK_BYTES;
        if (++next % BF16_CHUNK_STEPS == 0)
            seek();
    }
    __device__ void start(const uint8_t *weights, int64_t rows, int64_t width, int block, int wave, int waves)
    {
        w = weights;
        N = rows;
        K = width;
        nb0 = block;
        const int steps = (int)(K / BF16_STEP);
        next = s0 = steps * wave / waves;
        s1 = steps * (wave + 1) / waves;
        seek();
#pragma unroll
        for (int i = 0; i < DEPTH; i++)
            load(i);
        asm volatile("" ::: "memory");   // issued here
    }
    // get(row, k): 16 bytes of a token's activations from column k on.
    template <class Get>
    __device__ void finish(int T, uint32_t *stage, f32x4_t (&acc)[NB], Get get)
    {
        const int lane = lane_id(), n = s1 - s0, pitch = n * 16 + 4;   // words of a token's part in LDS
        const int r = lane & 15, c = lane >> 4;
        if (T * pitch <= STAGE_WORDS) {
            for (int i0 = 0; i0 < T * n * 4; i0 += 4 * WAVE) {
                u32x4_t v[4];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int at = i0 + i * WAVE + lane;
                    if (at < T * n * 4)
                        v[i] = get(at / (n * 4), s0 * BF16_STEP + at % (n * 4) * 8);
                }
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int at = i0 + i * WAVE + lane;
                    if (at < T * n * 4)
                        *reinterpret_cast<u32x4_t *>(stage + at / (n * 4) * pitch + at % (n * 4) * 4) = v[i];
                }
            }
            // rows past the tokens repeat the last one: their sums are not used
            const uint32_t *mine = stage + min(r, T - 1) * pitch + c * 4;
            for (int s = s0; s < s1; s += DEPTH)
#pragma unroll
                for (int i = 0; i < DEPTH; i++)
                    if (s + i < s1) {
                        const u32x4_t x = *reinterpret_cast<const u32x4_t *>(mine + (s + i - s0) * 16);
#pragma unroll
                        for (int j = 0; j < NB; j++)
                            acc[j] = mfma16(as_bf16x8(x), as_bf16x8(b[i][j]), acc[j]);
                        load(i);
                    }
            return;
        }
        u32x4_t x[AHEAD];
        auto operand = [&](int s, int slot) {
            if (s < s1)
                x[slot] = r < T ? get(r, s * BF16_STEP + c * 8) : ZERO;
        };
#pragma unroll
        for (int i = 0; i < AHEAD; i++)
            operand(s0 + i, i);
        for (int s = s0; s < s1; s += DEPTH)
#pragma unroll
            for (int i = 0; i < DEPTH; i++)
                if (s + i < s1) {
#pragma unroll
                    for (int j = 0; j < NB; j++)
                        acc[j] = mfma16(as_bf16x8(x[i % AHEAD]), as_bf16x8(b[i][j]), acc[j]);
                    load(i);
                    operand(s + i + AHEAD, i % AHEAD);
                }
    }
};

// Items: pairs of shared gate and up blocks first, which take twice as long, then the latent's blocks, then the router's.
template <int NB>
__device__ inline void front_product(const DecodeArgs &a, const uint8_t *w, int64_t rows, int block, uint32_t *lds)
{
    const int wv = wave_id();
    f32x4_t acc[NB] = {};
    Bf16Part<NB, NB == 1 ? 8 : 4, 4> part;
    part.start(w, rows, a.Hin, block, wv, FRONT_WAVES);
    part.finish(a.T, lds + wv * STAGE_WORDS, acc, [&](int r, int k) { return load16(a.x + (int64_t)r * a.Hin + k); });
    __syncthreads();
    float *red = reinterpret_cast<float *>(lds);
#pragma unroll
    for (int j = 0; j < NB; j++)
        store_sums(red + (wv * NB + j) * 256, acc[j]);
    __syncthreads();
}

__global__ __launch_bounds__(WAVE *FRONT_WAVES, 4) void front_kernel(const DecodeArgs a)
{
    __shared__ uint32_t lds[FRONT_WAVES * STAGE_WORDS];
    const float *red = reinterpret_cast<const float *>(lds);
    const int t = threadIdx.x;
    if (blockIdx.x == 0 && t < DECODE_COUNTERS + DECODE_FLAGS * FLAGS)
        a.counters[t * DECODE_COUNTER_WORDS] = 0u;
    if (blockIdx.x == 0 && a.T > 1)
        for (int i = t; i < a.Lt / 16; i += WAVE * FRONT_WAVES)
            a.column_counters[i] = 0u;
    const int pairs = a.shared / 16, latent = a.has_latent ? a.Lt / 16 : 0;
    int item = blockIdx.x;
    const int row = t / 16, col = t % 16;
    if (item < pairs) {
        front_product<2>(a, a.w_shared, a.n_shared_rows, (int)(a.shared_at / 16) + 2 * item, lds);
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
    front_product<1>(a, z ? a.w_latent : a.w_router, z ? a.n_latent_rows : a.n_router_rows, item, lds);
    if (t >= 256 || row >= a.T)
        return;
    const float v = total<FRONT_WAVES>(red, 256, t);
    const int n = item * 16 + col;
    if (z) {
        const uint32_t high = f32_to_bf16_bits(v);
        const int64_t at = (int64_t)row * a.Lt + n;
        a.z[at] = (uint16_t)high;
        a.z_rest[at] = (uint16_t)f32_to_bf16_bits(v - bf16_bits_to_f32(high));
    } else if (n < a.E) {
        a.logits[(int64_t)row * a.E + n] = a.bias ? v + a.bias[n] : v;
    }
}

// Until flag i is set. One thread asks; what follows in any thread is after the answer. Returns the flag less one.
__device__ inline int wait_for(const DecodeArgs &a, int i, uint32_t *sh)
{
    if (threadIdx.x == 0) {
        const uint32_t *at = flag(a, i, blockIdx.x % FLAGS);
        uint32_t v;
        while ((v = __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) == 0u)
            __builtin_amdgcn_s_sleep(2);
        *sh = v - 1;
    }
    __syncthreads();
    const int v = __builtin_amdgcn_readfirstlane((int)*sh);
    __syncthreads();
    asm volatile("" ::: "memory");
    return v;
}

__device__ inline void set_flag(const DecodeArgs &a, int i, uint32_t v)   // by a wave
{
    __hip_atomic_store(flag(a, i, lane_id()), v + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Every wave's stores have completed.
__device__ inline void stores_done()
{
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    asm volatile("" ::: "memory");
    __syncthreads();
}

// This workgroup's arrival at a counter after its stores; true in the first wave of the last of `all` to arrive.
__device__ inline bool arrive(uint32_t *at, uint32_t all)
{
    stores_done();
    if (wave_id() != 0)
        return false;
    uint32_t before = 0u;
    if (lane_id() == 0)
        before = __hip_atomic_fetch_add(at, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)before) == all - 1;
}

template <int SLOTS>
__device__ inline void top_item(const DecodeArgs &a, uint32_t *words)
{
    __shared__ uint64_t scratch[REST_WAVES][WAVE];
    const int lane = lane_id(), wv = wave_id();
    const int T = a.T, K = a.K, E = a.E, P = T * K;
    uint32_t *masks = words;              // of an expert's tokens
    int *chosen = reinterpret_cast<int *>(words + E), *sh = chosen + P;
    constexpr int NTHR = WAVE * REST_WAVES;
    for (int e = threadIdx.x; e < E; e += NTHR)
        masks[e] = 0u;
    __syncthreads();
    const auto weights = flat_rsrc(a.weights, (int64_t)P * 4);
    for (int t = wv; t < T; t += REST_WAVES) {
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
            const int p = t * K + lane;
            chosen[p] = id;
            atomicOr(&masks[id], 1u << t);
            store4_sc1(weights, p * 4, __float_as_uint(w));
            if (a.ids_out)
                a.ids_out[p] = id;
            if (a.weights_out)
                a.weights_out[p] = w;
        }
    }
    __syncthreads();
    // the experts that any token chose, and for each the pairs of its tokens, two to a word
    const int per = (E + NTHR - 1) / NTHR, e0 = (int)threadIdx.x * per, e1 = min(E, e0 + per);
    int n = 0, count;
    for (int e = e0; e < e1; e++)
        n += masks[e] != 0u;
    int rank = block_excl_scan(n, sh, &count);
    const auto list = flat_rsrc(a.list, (int64_t)a.most * 4), pairs = flat_rsrc(a.pairs, (int64_t)a.most * ROWS * 2);
    for (int e = e0; e < e1; e++) {
        const uint32_t mask = masks[e];
        if (mask == 0u)
            continue;
        store4_sc1(list, rank * 4, (uint32_t)e);
        for (int r = 0; r < ROWS; r += 2) {
            uint32_t two = 0u;
            for (int i = 0; i < 2; i++) {
                int p = -1;
                if (mask >> (r + i) & 1u)
                    for (int j = 0; j < K; j++)
                        if (chosen[(r + i) * K + j] == e)
                            p = (r + i) * K + j;
                two |= (uint32_t)(p & 0xFFFF) << (16 * i);
            }
            store4_sc1(pairs, (rank * ROWS + r) * 2, two);
        }
        rank++;
    }
    stores_done();
    if (wv == 0)
        set_flag(a, DECODE_READY, (uint32_t)count);
}

// One MX block times a step's activations.
__device__ inline f32x4_t mx_step(u32x4_t codes, uint32_t scales, const u32x4_t (&x)[4], f32x4_t acc)
{
#pragma unroll
    for (int j = 0; j < 4; j++)
        acc = mfma16(as_bf16x8(x[j]), mx_dequant8(codes[j], e8m0_to_f32((scales >> (8 * j)) & 0xFFu)), acc);
    return acc;
}

// NP pairs of 16 gate and 16 up channels of one expert; the waves share the K axis. Up to 8 tokens: one operand, whose
// rows 8 .. 15 are the remainders of rows 0 .. 7; more: two operands (PARTS).
template <int NP, int PARTS>
__device__ inline void gate_item(const DecodeArgs &a, int item, float *red, uint32_t *sh)
{
    __shared__ uint32_t tokens[ROWS / 2];   // the expert's pairs, two to a word
    const int lane = lane_id(), wv = wave_id();
    const int groups = (a.I / 16 + NP - 1) / NP, r = item / groups, cp = item % groups * NP, np = min(NP, a.I / 16 - cp);
    const int experts = wait_for(a, DECODE_READY, sh);
    if (r >= experts)
        return;
    const int e = __builtin_amdgcn_readfirstlane((int)load4_sc1(flat_rsrc(a.list, (int64_t)a.most * 4), r * 4));
    if (threadIdx.x < ROWS / 2)
        tokens[threadIdx.x] = load4_sc1(flat_rsrc(a.pairs, (int64_t)a.most * ROWS * 2), (r * ROWS + 2 * (int)threadIdx.x) * 2);
    const int steps = a.Lt / MX_STEP, s0 = steps * wv / REST_WAVES, s1 = steps * (wv + 1) / REST_WAVES;
    const uint8_t *w = a.gateup + e * a.gateup_stride + (int64_t)2 * cp * steps * MX_BLOCK_BYTES;
    constexpr int BATCH = PARTS == 1 ? 7 : 4, NB = 2 * NP;   // steps in flight
    const int row = PARTS == 1 ? lane & 7 : lane & 15;
    const bool rest = PARTS == 1 && (lane & 8);
    const uint16_t *x0 = (rest ? a.z_rest : a.z) + (int64_t)row * a.Lt + 8 * (lane >> 4);
    const uint16_t *x1 = a.z_rest + (int64_t)row * a.Lt + 8 * (lane >> 4);
    const bool live0 = row < a.T && (!rest || a.has_latent), live1 = row < a.T && a.has_latent;
    f32x4_t acc[PARTS][NB] = {};
    for (int s = s0; s < s1; s += BATCH) {
        u32x4_t codes[BATCH][NB];
        uint32_t scales[BATCH][NB];
#pragma unroll
        for (int i = 0; i < BATCH; i++)
            if (s + i < s1)
#pragma unroll
                for (int j = 0; j < NB; j++)
                    if (j < 2 * np) {
                        const uint8_t *blk = w + ((int64_t)j * steps + s + i) * MX_BLOCK_BYTES;
                        codes[i][j] = load16_nt(blk + lane * 16);
                        scales[i][j] = load4_nt(blk + MX_CODE_BYTES + 4 * (lane & 15));
                    }
        asm volatile("" ::: "memory");
#pragma unroll
        for (int i = 0; i < BATCH; i++)
            if (s + i < s1) {
                u32x4_t x[PARTS][4];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    x[0][j] = live0 ? load16(x0 + (s + i) * MX_STEP + 32 * j) : ZERO;
                    if constexpr (PARTS == 2)
                        x[1][j] = live1 ? load16(x1 + (s + i) * MX_STEP + 32 * j) : ZERO;
                }
#pragma unroll
                for (int j = 0; j < NB; j++)
                    if (j < 2 * np)
#pragma unroll
                        for (int p = 0; p < PARTS; p++)
                            acc[p][j] = mx_step(codes[i][j], scales[i][j], x[p], acc[p][j]);
            }
    }
#pragma unroll
    for (int j = 0; j < NB; j++) {
        f32x4_t v = acc[0][j];
        if constexpr (PARTS == 2)
            v += acc[1][j];
        store_sums(red + (wv * NB + j) * 256, v);
    }
    __syncthreads();
    // two channels of a row per thread
    auto sum = [&](int b, int at) {
        if constexpr (PARTS == 2)
            return total<REST_WAVES>(red + b * 256, NB * 256, at);
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < REST_WAVES; k++)
            v += red[(k * NB + b) * 256 + at] + red[(k * NB + b) * 256 + HALF * 16 + at];
        return v;
    };
    const auto h = flat_rsrc(a.h, (int64_t)a.T * a.K * a.I * 2);
    for (int i = threadIdx.x; i < np * a.T * 8; i += WAVE * REST_WAVES) {
        const int c = i % 8 * 2, token = i / 8 % a.T, b = i / 8 / a.T, pair = (int16_t)(tokens[token / 2] >> (16 * (token % 2)));
        if (pair < 0)
            continue;
        float v[2];
#pragma unroll
        for (int k = 0; k < 2; k++)
            v[k] = silu_f32(sum(2 * b, token * 16 + c + k)) * sum(2 * b + 1, token * 16 + c + k);
        store4_sc1(h, (pair * a.I + (cp + b) * 16 + c) * 2, pack_bf16x2(v[0], v[1]));
    }
    if (arrive(counter(a, DECODE_GATE), (uint32_t)(experts * groups)))
        set_flag(a, DECODE_GATE_DONE, 0u);
}

// 16 latent columns of every chosen expert (parts = 1) or of part `part` of 4. Experts fall into 16 classes by their number
// e: part e / 4 % 4, wave e % 4. A class is added in ascending order, the classes of a part in wave order, the parts in
// order: so a token's sum is added in an order that its own experts alone decide, and its outputs are the same bits
// whatever tokens come with it. With four parts the last workgroup to arrive at the columns adds them.
constexpr int PARTS_MAX = DECODE_PARTS;
__device__ inline void down_item(const DecodeArgs &a, int item, int parts, uint32_t *lds, uint32_t *sh)
{
    constexpr int NTHR = WAVE * REST_WAVES, MOST = ROWS * 32;   // distinct experts
    // the waves' sums; then the routing: the pairs of (expert, token), or -1, their weights, the experts, and the ranks of
    // each wave's own experts
    float *red = reinterpret_cast<float *>(lds);
    int16_t *pairs = reinterpret_cast<int16_t *>(lds + (parts == 1 ? PARTS_MAX : 1) * REST_WAVES * 256);
    float *weights = reinterpret_cast<float *>(pairs + a.most * ROWS);
    uint16_t *list = reinterpret_cast<uint16_t *>(weights + MOST), *own = list + MOST + wave_id() * MOST;
    const int lane = lane_id(), wv = wave_id(), part = parts == 1 ? 0 : item % parts, col = parts == 1 ? item : item / parts;
    const int experts = wait_for(a, DECODE_READY, sh);
    {
        const auto gl = flat_rsrc(a.list, (int64_t)a.most * 4), gp = flat_rsrc(a.pairs, (int64_t)a.most * ROWS * 2);
        const auto gw = flat_rsrc(a.weights, (int64_t)a.T * a.K * 4);
        for (int i = threadIdx.x; i < experts; i += NTHR)
            list[i] = (uint16_t)load4_sc1(gl, i * 4);
        for (int i = threadIdx.x; i < experts * (ROWS / 2); i += NTHR)
            reinterpret_cast<uint32_t *>(pairs)[i] = load4_sc1(gp, i * 4);
        for (int i = threadIdx.x; i < a.T * a.K; i += NTHR)
            weights[i] = __uint_as_float(load4_sc1(gw, i * 4));
    }
    __syncthreads();
    int count = 0, ends[PARTS_MAX];   // of the experts of part 0, 0 .. 1, ...
#pragma unroll
    for (int k = 0; k < PARTS_MAX; k++) {
        if (parts == 1 || k == part)
            for (int r0 = 0; r0 < experts; r0 += WAVE) {
                const int r = r0 + lane, e = r < experts ? list[r] : -1;
                const bool mine = e >= 0 && e % REST_WAVES == wv && e / REST_WAVES % PARTS_MAX == k;
                const uint64_t all = __ballot(mine);
                if (mine)
                    own[count + __popcll(all & ((1ull << lane) - 1))] = (uint16_t)r;
                count += (int)__popcll(all);
            }
        ends[k] = count;
    }
    __syncthreads();
    // The blocks of this wave, expert by expert: DEPTH blocks ahead, the first weights before h is known. `at` and `of`
    // walk over (expert, step) for the weights and for the activations.
    constexpr int DEPTH = 3;
    const int steps = a.I / MX_STEP;
    const auto h = flat_rsrc(a.h, (int64_t)a.T * a.K * a.I * 2);
    struct Walk {
        int i, s;   // own expert, step
    };
    Walk at{0, 0}, of{0, 0};
    const uint8_t *blk = nullptr;
    int pair = -1;
    u32x4_t codes[DEPTH], x[DEPTH][4];
    uint32_t scales[DEPTH];
    auto load = [&](int slot) {
        if (at.i >= count)
            return;
        if (at.s == 0)
            blk = a.down + __builtin_amdgcn_readfirstlane((int)list[own[at.i]]) * a.down_stride + (int64_t)col * steps * MX_BLOCK_BYTES;
        codes[slot] = load16_nt(blk + lane * 16);
        scales[slot] = load4_nt(blk + MX_CODE_BYTES + 4 * (lane & 15));
        blk += MX_BLOCK_BYTES;
        if (++at.s == steps)
            at = Walk{at.i + 1, 0};
    };
    auto operand = [&](int slot) {
        if (of.i >= count)
            return;
        if (of.s == 0)
            pair = pairs[own[of.i] * ROWS + (lane & 15)];
#pragma unroll
        for (int j = 0; j < 4; j++)
            x[slot][j] = pair >= 0 ? __builtin_bit_cast(u32x4_t, load16_sc1(h, (pair * a.I + of.s * MX_STEP + 32 * j + 8 * (lane >> 4)) * 2))
                                   : ZERO;
        if (++of.s == steps)
            of = Walk{of.i + 1, 0};
    };
#pragma unroll
    for (int d = 0; d < DEPTH; d++)
        load(d);
    asm volatile("" ::: "memory");
    wait_for(a, DECODE_GATE_DONE, sh);
#pragma unroll
    for (int d = 0; d < DEPTH; d++)
        operand(d);
    f32x4_t sum = {}, y = {};
    int k = 0;   // the class being added
    auto end_classes = [&](int i) {   // those that own expert i is past
        while (k < PARTS_MAX && i >= ends[k]) {
            if (parts == 1 || k == part)
                store_sums(red + ((parts == 1 ? k : 0) * REST_WAVES + wv) * 256, sum);
            sum = f32x4_t{0.f, 0.f, 0.f, 0.f};
            k++;
        }
    };
    Walk now{0, 0};
    end_classes(0);
    while (now.i < count)
#pragma unroll
        for (int d = 0; d < DEPTH; d++) {
            if (now.i >= count)
                break;
            y = mx_step(codes[d], scales[d], x[d], y);
            load(d);
            operand(d);
            if (++now.s == steps) {   // the expert's values times the weights of its tokens
                const int16_t *of_rows = pairs + own[now.i] * ROWS + 4 * (lane >> 4);
#pragma unroll
                for (int j = 0; j < 4; j++) {   // values that are not finite reach the expert's own tokens only
                    const int p = of_rows[j];
                    sum[j] = p >= 0 ? fmaf(weights[max(p, 0)], y[j], sum[j]) : sum[j];
                }
                y = f32x4_t{0.f, 0.f, 0.f, 0.f};
                now = Walk{now.i + 1, 0};
                end_classes(now.i);
            }
        }
    __syncthreads();
    const int t = threadIdx.x, row = t / 16, c = t % 16;
    float v = 0.f;
    if (parts == 1) {
#pragma unroll
        for (int p = 0; p < PARTS_MAX; p++)
            v += total<REST_WAVES>(red + p * REST_WAVES * 256, 256, t);
    } else {
        const auto partial = flat_rsrc(a.partial + (int64_t)col * PARTS_MAX * 256, PARTS_MAX * 256 * 4);
        if (row < a.T)
            store4_sc1(partial, (part * 256 + t) * 4, __float_as_uint(total<REST_WAVES>(red, 256, t)));
        const bool last = arrive(a.column_counters + col, PARTS_MAX);
        if (t == 0)
            *sh = last;
        __syncthreads();
        const bool mine = *sh != 0u;
        __syncthreads();
        if (!mine)
            return;
        if (row < a.T)
#pragma unroll
            for (int p = 0; p < PARTS_MAX; p++)
                v += __uint_as_float(load4_sc1(partial, (p * 256 + t) * 4));
    }
    // two columns to a word
    const uint32_t two = pack_bf16x2(v, __shfl_down(v, 1));
    if (row < a.T && c % 2 == 0) {
        if (a.has_latent)
            store4_sc1(flat_rsrc(a.acat, (int64_t)a.T * a.ldcat * 2), (row * a.ldcat + col * 16 + c) * 2, two);
        else
            *reinterpret_cast<uint32_t *>(a.out + (int64_t)row * a.Lt + col * 16 + c) = two;
    }
    if (a.has_latent && arrive(counter(a, DECODE_DOWN), (uint32_t)(a.Lt / 16)))
        set_flag(a, DECODE_DOWN_DONE, 0u);
}

__device__ inline void out_item(const DecodeArgs &a, int item, uint32_t *lds, uint32_t *sh)
{
    const int wv = wave_id();
    Bf16Part<1, 12, 4> part;
    part.start(a.w_out, a.H, a.ldcat, item, wv, REST_WAVES);
    wait_for(a, DECODE_DOWN_DONE, sh);
    const auto acat = flat_rsrc(a.acat, (int64_t)a.T * a.ldcat * 2);
    f32x4_t acc[1] = {};
    part.finish(a.T, lds + wv * STAGE_WORDS, acc,
                [&](int r, int k) { return __builtin_bit_cast(u32x4_t, load16_sc1(acat, (r * a.ldcat + k) * 2)); });
    __syncthreads();
    float *red = reinterpret_cast<float *>(lds);
    store_sums(red + wv * 256, acc[0]);
    __syncthreads();
    const int t = threadIdx.x, row = t / 8, c = t % 8 * 2;
    if (row < a.T && row < ROWS)
        *reinterpret_cast<uint32_t *>(a.out + (int64_t)row * a.H + item * 16 + c) =
            pack_bf16x2(total<REST_WAVES>(red, 256, row * 16 + c), total<REST_WAVES>(red, 256, row * 16 + c + 1));
}

template <int SLOTS, bool FEW>
__global__ __launch_bounds__(WAVE *REST_WAVES, 4) void rest_kernel(const DecodeArgs a)
{
    // the items' activations, sums over the waves, and the routing as they need it
    constexpr int TOP = SLOTS * WAVE + ROWS * 32 + 16, ITEM = REST_WAVES * STAGE_WORDS;
    constexpr int DOWN = REST_WAVES * 256 + ROWS * 32 * (ROWS / 2 + 1) + (1 + REST_WAVES) * ROWS * 16;
    static_assert(TOP <= ITEM && DOWN <= ITEM && REST_WAVES * 1024 <= ITEM, "room");
    static_assert(PARTS_MAX * REST_WAVES * 256 + 32 * (ROWS / 2) + ROWS * 32 + (1 + REST_WAVES) * ROWS * 16 <= ITEM, "room");
    __shared__ uint32_t lds[ITEM];
    __shared__ uint32_t sh;
    float *red = reinterpret_cast<float *>(lds);
    if (threadIdx.x == 0)
        sh = __hip_atomic_fetch_add(counter(a, DECODE_TICKET), 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    int item = __builtin_amdgcn_readfirstlane((int)sh);
    __syncthreads();
    const DecodeItems n = decode_items(a);
    if (item < n.top)
        return top_item<SLOTS>(a, lds);
    item -= n.top;
    if (item < n.gate)
        return gate_item<1, FEW ? 1 : 2>(a, item, red, &sh);
    item -= n.gate;
    if (item < n.down)
        return down_item(a, item, n.parts, lds, &sh);
    out_item(a, item - n.down, lds, &sh);
}

template <int SLOTS>
void launch_rest(const DecodeArgs &a, hipStream_t st)
{
    const DecodeItems n = decode_items(a);
    const dim3 grid((unsigned)(n.top + n.gate + n.down + n.out)), threads(WAVE * REST_WAVES);
    if (a.T <= HALF)
        hipLaunchKernelGGL((rest_kernel<SLOTS, true>), grid, threads, 0, st, a);
    else
        hipLaunchKernelGGL((rest_kernel<SLOTS, false>), grid, threads, 0, st, a);
}

} // namespace

hipError_t launch_decode(const DecodeArgs &a, hipStream_t st)
{
    const unsigned front = (unsigned)(a.shared / 16 + (a.has_latent ? a.Lt / 16 : 0) + a.n_router_rows / 16);
    hipLaunchKernelGGL(front_kernel, dim3(front), dim3(WAVE * FRONT_WAVES), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    if (a.E <= 4 * WAVE)
        launch_rest<4>(a, st);
    else
        launch_rest<16>(a, st);
    return hipGetLastError();
}

} // namespace mxmoe
