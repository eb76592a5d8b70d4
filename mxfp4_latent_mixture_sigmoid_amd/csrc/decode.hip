// decode.hip -- the whole layer for up to 16 tokens in two kernels.
//
// The tokens are one row tile of the matrix-core instruction, so every weight is read once, from memory, and
// multiplied with all tokens at once: the time is the weights' (184 MB for one token of a TP8 share: the router, latent
// and shared matrices in BF16, 16 experts in MXFP4).
//
//  front_kernel  what only needs x: the router's logits, z = x W_down^T, h_s = bf16(silu(x Wg_s^T) (x Wu_s^T)).
//  rest_kernel   everything after it, in work items, one for each workgroup:
//    top    the top-K of every token; the list of distinct experts and each one's tokens
//    gate   (expert, 16 or 64 inner channels): h = bf16(silu(z Wg^T) (z Wu^T)) of the expert's tokens
//    down   16 latent columns of every chosen expert, or of a quarter of them: zc = bf16(sum w (h Wd^T)), in slot order
//    out    16 output columns: out = bf16([zc | h_s] [W_up | W_ds]^T)
//
// z is kept in two BF16 parts, the rounded value and what the rounding left, because its rounding alone reaches every
// expert's gate, up and product (0.4% of a small layer's output in the mean square, against 0.3% without); the
// remainders are rows 8 to 15 of the tile for up to 8 tokens, at no cost, and a second operand for more.
//
// Kinds wait for each other on flags. A workgroup takes the item of its number by claiming it; it waits for a flag PATIENCE
// times, far longer than a call takes, and if the flag has not come by then (its workgroups may not even have started:
// another call's, which wait for theirs, may hold their places) it claims and does whatever item of an earlier kind is
// still free, in order, and waits again. Then every item that it waits for is done or being worked on by a workgroup that
// runs, so that all waits end, however many workgroups the card holds at once and whatever else runs on it. (Drawing
// items from one ticket counter gives that too, but additions to one address take 12 ns each: 1057 workgroups kept the
// top-K's loads waiting for 9 us behind theirs.) For the same reason arrivals are counted at 16 counters first, and the
// last one writes its flag in 64 places, each asked for by a part of the workgroups. What one workgroup hands to another
// goes through agent-coherent stores and loads (sync.hpp). The front kernel clears counters, flags and claims.
//
// Two things set the pace of code that runs once. Instructions come from memory at about 1 KiB a microsecond the first
// time: so the top-K is written to be short, and while an item waits it goes once through what it will do, with empty
// windows for its loads and stores (`go` = 0). And a load under a condition is a wait for the loads before it: so no
// load has one; loads past the end lie outside their window, which costs nothing.
#include "decode.hpp"
#include "select.hpp"
#include "sync.hpp"

namespace mxmoe {

namespace {

constexpr int ROWS = DECODE_MAX_T, HALF = ROWS / 2;
constexpr int FRONT_WAVES = 8, REST_WAVES = 4;
constexpr int OUT_DEPTH = 24;
constexpr int FLAGS = WAVE;                 // places of a flag
constexpr int ARMS = DECODE_ARMS;
constexpr int STAGE_WORDS = 1856;           // LDS of a wave for its activations, where they fit
constexpr int LDS_WORDS = REST_WAVES * STAGE_WORDS + REST_WAVES * 512;   // of an item; four workgroups share a CU

__device__ inline uint32_t *counter(const DecodeArgs &a, int i) { return a.counters + i * DECODE_COUNTER_WORDS; }
__device__ inline uint32_t *flag(const DecodeArgs &a, int i, int place)
{
    return a.counters + (DECODE_COUNTERS + i * FLAGS + place) * DECODE_COUNTER_WORDS;
}

__device__ inline int lane_id() { return threadIdx.x & (WAVE - 1); }
__device__ inline int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE); }

// Windows for loads and stores: those outside read zeros and write nothing, without touching memory. `go` = 0: an empty one.
constexpr int OUTSIDE = DECODE_MAX_WINDOW;   // an offset past every window
__device__ inline __amdgpu_buffer_rsrc_t window(const void *base, int64_t bytes, int go) { return flat_rsrc(base, go ? bytes : 0); }
template <int CPOL>
__device__ inline u32x4_t fetch16(__amdgpu_buffer_rsrc_t w, int offset)
{
    return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(w, offset, 0, CPOL));
}
template <int CPOL>
__device__ inline uint32_t fetch4(__amdgpu_buffer_rsrc_t w, int offset)
{
    return (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(w, offset, 0, CPOL);
}

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
template <int NB, int DEPTH, int AHEAD, bool STAGED>
struct Bf16Part {
    static_assert(DEPTH % AHEAD == 0, "slots");
    // Whether K values of T tokens, divided among the waves, fit their parts of LDS.
    static __device__ bool fits(int T, int K, int waves) { return T * ((K / BF16_STEP + waves - 1) / waves * 16 + 4) <= STAGE_WORDS; }
    u32x4_t b[DEPTH][NB];
    __amdgpu_buffer_rsrc_t w;
    int s0, s1, next, at, jump, last, tail;   // steps; the next step's first block

    // Steps are loaded one after another, each into slot (step - s0) % DEPTH.
    __device__ void load(int slot)
    {
        const int pitch = next >= last ? tail : BF16_CHUNK_STEPS;   // blocks from a row block to the next in this K chunk
        const int off = next < s1 ? at * BF16_BLOCK_BYTES : OUTSIDE;
#pragma unroll
        for (int j = 0; j < NB; j++)
            b[slot][j] = fetch16<CPOL_NT>(w, off + (next < s1 ? j * pitch * BF16_BLOCK_BYTES : 0) + lane_id() * 16);
        next++;
        at += next % BF16_CHUNK_STEPS == 0 ? next == last ? jump + 1 - (BF16_CHUNK_STEPS - tail) * block : jump + 1 : 1;
    }
    int block;
    __device__ void start(const uint8_t *weights, int64_t N, int64_t K, int nb, int wave, int waves, int go = 1)
    {
        const int steps = (int)(K / BF16_STEP);
        w = window(weights, N * K * 2, go);
        next = s0 = steps * wave / waves;
        s1 = steps * (wave + 1) / waves;
        block = nb;
        last = steps / BF16_CHUNK_STEPS * BF16_CHUNK_STEPS;   // the first step of a last chunk of `tail` steps
        tail = steps % BF16_CHUNK_STEPS;
        jump = BF16_CHUNK_STEPS * (int)(N / 16) - BF16_CHUNK_STEPS;   // from the end of a chunk's part to the next one's
        at = (int)bf16_block_index(nb, next, N, K);
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
        if constexpr (STAGED) {
#pragma unroll 1
            for (int i0 = 0; i0 < T * n * 4; i0 += 4 * WAVE) {
                u32x4_t v[4];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int at = min(i0 + i * WAVE + lane, T * n * 4 - 1);
                    v[i] = get(at / (n * 4), s0 * BF16_STEP + at % (n * 4) * 8);
                }
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int at = min(i0 + i * WAVE + lane, T * n * 4 - 1);
                    *reinterpret_cast<u32x4_t *>(stage + at / (n * 4) * pitch + at % (n * 4) * 4) = v[i];
                }
            }
            // rows past the tokens repeat the last one: their sums are not used. Steps past the end multiply zeros.
            const uint32_t *mine = stage + min(r, T - 1) * pitch + c * 4;
#pragma unroll 1
            for (int s = 0; s < n; s += DEPTH)
#pragma unroll
                for (int i = 0; i < DEPTH; i++) {
                    const u32x4_t x = *reinterpret_cast<const u32x4_t *>(mine + min(s + i, n - 1) * 16);
#pragma unroll
                    for (int j = 0; j < NB; j++)
                        acc[j] = step(x, b[i][j], acc[j], s + i < n);
                    load(i);
                    if (i % 4 == 3)
                        __builtin_amdgcn_sched_barrier(0);   // not all operands at once
                }
            return;
        }
        u32x4_t x[AHEAD];
        auto operand = [&](int s, int slot) { x[slot] = get(min(r, T - 1), (s0 + min(s, n - 1)) * BF16_STEP + c * 8); };
#pragma unroll
        for (int i = 0; i < AHEAD; i++)
            operand(i, i);
#pragma unroll 1
        for (int s = 0; s < n; s += DEPTH)
#pragma unroll
            for (int i = 0; i < DEPTH; i++) {
#pragma unroll
                for (int j = 0; j < NB; j++)
                    acc[j] = step(x[i % AHEAD], b[i][j], acc[j], s + i < n);
                load(i);
                operand(s + i + AHEAD, i % AHEAD);
            }
    }
    // A step past the end adds nothing, whatever the activations are.
    static __device__ f32x4_t step(u32x4_t x, u32x4_t w, f32x4_t acc, bool in)
    {
        const f32x4_t v = mfma16(as_bf16x8(x), as_bf16x8(w), acc);
        return in ? v : acc;
    }
};

// Items: pairs of shared gate and up blocks first, which take twice as long, then the latent's blocks, then the router's.
template <int NB>
__device__ inline void front_product(const DecodeArgs &a, const uint8_t *w, int64_t rows, int block, uint32_t *lds)
{
    const int wv = wave_id();
    f32x4_t acc[NB] = {};
    auto run = [&](auto part) {
        part.start(w, rows, a.Hin, block, wv, FRONT_WAVES);
        part.finish(a.T, lds + wv * STAGE_WORDS, acc, [&](int r, int k) { return load16(a.x + (int64_t)r * a.Hin + k); });
    };
    using Staged = Bf16Part<NB, NB == 1 ? 16 : 8, 4, true>;
    if (Staged::fits(a.T, a.Hin, FRONT_WAVES))
        run(Staged());
    else
        run(Bf16Part<NB, NB == 1 ? 8 : 4, 4, false>());
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
    static_assert(DECODE_COUNTER_LINES <= WAVE * FRONT_WAVES, "a thread each");
    if (blockIdx.x == 0 && t < DECODE_COUNTER_LINES)
        a.counters[t * DECODE_COUNTER_WORDS] = 0u;
    const int threads = gridDim.x * WAVE * FRONT_WAVES, number = blockIdx.x * WAVE * FRONT_WAVES + t;
    for (int i = number; i < decode_item_count(decode_items(a)); i += threads)
        a.claims[i] = 0u;
    if (a.T > 1)
        for (int i = number; i < a.Lt / 16; i += threads)
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

// Until flag i is set: its value less one, or -1 when patience runs out (HELP: never). One thread asks; what follows in any
// thread is after the answer.
template <bool HELP>
__device__ inline int wait_for(const DecodeArgs &a, int i, uint32_t *sh)
{
    if (threadIdx.x == 0) {
        const uint32_t *at = flag(a, i, blockIdx.x % FLAGS);
        uint32_t v;
        int left = a.patience;
        while ((v = __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) == 0u && (HELP || left-- > 0))
            __builtin_amdgcn_s_sleep(2);
        *sh = v - 1;
    }
    __syncthreads();
    const int v = __builtin_amdgcn_readfirstlane((int)*sh);
    __syncthreads();
    asm volatile("" ::: "memory");
    return v;
}

// Whether item `i` is this workgroup's now.
template <bool HELP>
__device__ inline bool claim(const DecodeArgs &a, int i, uint32_t *sh)
{
    if (threadIdx.x == 0) {
        uint32_t *at = a.claims + i;
        *sh = !(HELP && __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != 0u) &&
              __hip_atomic_fetch_add(at, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == 0u;
    }
    __syncthreads();
    const bool mine = __builtin_amdgcn_readfirstlane((int)*sh) != 0;
    __syncthreads();
    return mine;
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

__device__ inline bool last_at(uint32_t *at, int all)   // by a wave
{
    uint32_t before = 0u;
    if (lane_id() == 0)
        before = __hip_atomic_fetch_add(at, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return __builtin_amdgcn_readfirstlane((int)before) == all - 1;
}

// Arrival number i of `all` at counter set `at` after this workgroup's stores; true in the first wave of the last to
// arrive. Additions to one address take 12 ns each, so the arrivals are counted at ARMS counters first.
__device__ inline bool arrive(const DecodeArgs &a, int set, int i, int all)
{
    stores_done();
    if (wave_id() != 0)
        return false;
    const int arm = i % ARMS, at = set * (ARMS + 1);
    return last_at(counter(a, at + arm), (all - arm + ARMS - 1) / ARMS) && last_at(counter(a, at + ARMS), min(all, ARMS));
}

// select_best of select.hpp in little code, from a token's logits in memory; the keys are kept in LDS (`words`, E rounded up to
// 256), four of a lane side by side. No key of an expert is 0, which stands for none (only a NaN with every bit set
// would have it), so that ids are always in range.
__device__ inline void select_short(const float *logits, int E, int K, uint32_t *words, uint64_t *scratch, int *id, float *weight)
{
    constexpr int QUADS = DECODE_MAX_E / (4 * WAVE);
    const int lane = lane_id(), quads = (E + 4 * WAVE - 1) / (4 * WAVE);
    const auto row = flat_rsrc(logits, (int64_t)E * 4);
    u32x4_t raw[QUADS];
#pragma unroll
    for (int q = 0; q < QUADS; q++)
        raw[q] = fetch16<0>(row, (q * WAVE + lane) * 16);
#pragma unroll
    for (int q = 0; q < QUADS; q++)
        *reinterpret_cast<u32x4_t *>(words + (q * WAVE + lane) * 4) = raw[q];
    uint32_t top = 0u;
#pragma unroll 1
    for (int q = 0; q < quads; q++) {
        u32x4_t v = *reinterpret_cast<const u32x4_t *>(words + (q * WAVE + lane) * 4);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            v[j] = (q * WAVE + lane) * 4 + j < E ? max(order_key(__uint_as_float(v[j])), 1u) : 0u;
            top = max(top, v[j]);
        }
        *reinterpret_cast<u32x4_t *>(words + (q * WAVE + lane) * 4) = v;
    }
    uint32_t bound = 0u;
#pragma unroll 1
    for (uint32_t bit = 1u << 31; bit; bit >>= 1)
        if ((int)__popcll(__ballot(top >= (bound | bit))) >= K)
            bound |= bit;
    int total = 0;
#pragma unroll 1
    for (int q = 0; q < quads; q++) {
        const u32x4_t v = *reinterpret_cast<const u32x4_t *>(words + (q * WAVE + lane) * 4);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const bool in = v[j] != 0u && v[j] >= bound;
            const uint64_t all = __ballot(in);
            const int at = total + (int)__popcll(all & ((1ull << lane) - 1));
            if (in && at < WAVE)
                scratch[at] = ((uint64_t)v[j] << 32) | (uint32_t)~(uint32_t)((q * WAVE + lane) * 4 + j);
            total += (int)__popcll(all);
        }
    }
    uint64_t mine = 0;
    if (total <= WAVE) {
        mine = lane < total ? scratch[lane] : 0;
        int rank = 0;
#pragma unroll 2
        for (int m = 0; m < total; m++) {
            const uint64_t other = ((uint64_t)__builtin_amdgcn_readlane((int)(mine >> 32), m) << 32) |
                                   (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)mine, m);
            rank += other > mine;
        }
        if (lane < total && rank < K)
            scratch[rank] = mine;
        mine = lane < K ? scratch[lane] : 0;
    } else {   // heavy ties: one maximum after another
#pragma unroll 1
        for (int k = 0; k < K; k++) {
            uint64_t best = 0;
#pragma unroll 1
            for (int e = lane; e < E; e += WAVE)
                if (words[e]) {
                    const uint64_t v = ((uint64_t)words[e] << 32) | (uint32_t)~(uint32_t)e;
                    best = v > best ? v : best;
                }
            const uint32_t high = wave_max_u32((uint32_t)(best >> 32));
            const uint32_t low = wave_max_u32((uint32_t)(best >> 32) == high ? (uint32_t)best : 0u);
            if (lane == k)
                mine = ((uint64_t)high << 32) | low;
            if (((uint64_t)high << 32 | low) == best)
                words[~low] = 0u;
        }
    }
    const float s = lane < K ? 1.0f / (1.0f + expf(-key_value((uint32_t)(mine >> 32)))) : 0.0f;
    *id = (int)~(uint32_t)mine;
    *weight = s / wave_sum_f32(s);
}

__device__ inline void top_item(const DecodeArgs &a, uint32_t *words)
{
    __shared__ uint64_t scratch[REST_WAVES][WAVE];
    const int lane = lane_id(), wv = wave_id();
    const int T = a.T, K = a.K, E = a.E, P = T * K;
    constexpr int NTHR = WAVE * REST_WAVES;
    // whether any token chose an expert, then its place in the list; the experts of the pairs; then the waves' keys, and
    // after them the list's pairs, two to a word
    int *ranks = reinterpret_cast<int *>(words), *chosen = ranks + DECODE_MAX_E, *sh = chosen + ROWS * 32;
    uint32_t *table = words + DECODE_MAX_E + ROWS * 32 + 16, *mine = table + wv * DECODE_MAX_E;
    for (int i = threadIdx.x; i < E; i += NTHR)
        ranks[i] = 0;
    __syncthreads();
    const auto weights = flat_rsrc(a.weights, (int64_t)P * 4);
#pragma unroll 1
    for (int t = wv; t < T; t += REST_WAVES) {
        int id;
        float w;
        select_short(a.logits + (int64_t)t * E, E, K, mine, scratch[wv], &id, &w);
        if (lane < K) {
            const int p = t * K + lane;
            chosen[p] = id;
            ranks[id] = 1;
            store4_sc1(weights, p * 4, __float_as_uint(w));
            if (a.ids_out)
                a.ids_out[p] = id;
            if (a.weights_out)
                a.weights_out[p] = w;
        }
    }
    __syncthreads();
    // the distinct experts in ascending order, and for each the pairs of its tokens
    const auto list = flat_rsrc(a.list, (int64_t)a.most * 4), pairs = flat_rsrc(a.pairs, (int64_t)a.most * ROWS * 2);
    for (int i = threadIdx.x; i < a.most * (ROWS / 2); i += NTHR)
        table[i] = ~0u;
    const int per = (E + NTHR - 1) / NTHR, e0 = (int)threadIdx.x * per, e1 = min(E, e0 + per);
    int n = 0, count;
    for (int e = e0; e < e1; e++)
        n += ranks[e];
    int rank = block_excl_scan(n, sh, &count);
    for (int e = e0; e < e1; e++)
        if (ranks[e]) {
            store4_sc1(list, rank * 4, (uint32_t)e);
            ranks[e] = rank++;
        }
    __syncthreads();
    for (int p = threadIdx.x; p < P; p += NTHR)
        reinterpret_cast<int16_t *>(table)[ranks[chosen[p]] * ROWS + p / K] = (int16_t)p;
    __syncthreads();
    for (int i = threadIdx.x; i < count * (ROWS / 2); i += NTHR)
        store4_sc1(pairs, i * 4, table[i]);
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

// The experts' gate and up product with one token: a pair of 16 gate and 16 up channels per workgroup, whose waves share the
// K axis; each wave's part of z (and of its remainders, row 8 of the operand) is in LDS before the expert is known.
template <bool HELP>
__device__ inline bool gate_one(const DecodeArgs &a, int item, uint32_t *lds, uint32_t *sh)
{
    const int lane = lane_id(), wv = wave_id(), t = threadIdx.x;
    const int pairs16 = a.I / 16, r = item / pairs16, cp = item % pairs16;
    const int steps = a.Lt / MX_STEP, s0 = steps * wv / REST_WAVES, n = steps * (wv + 1) / REST_WAVES - s0;
    constexpr int BATCH = 7;   // steps in flight
    uint32_t *stage = lds + wv * STAGE_WORDS;
    float *red = reinterpret_cast<float *>(lds + REST_WAVES * STAGE_WORDS);
    const int pitch = n * MX_STEP / 2 + 4, chunks = n * 16;   // words of a staged row; 16-byte pieces
#pragma unroll 1
    for (int i = lane; i < 2 * chunks; i += WAVE) {
        const int k = i >= chunks, j = i - k * chunks;
        *reinterpret_cast<u32x4_t *>(stage + k * pitch + j * 4) = load16((k && a.has_latent ? a.z_rest : a.z) + s0 * MX_STEP + j * 8);
    }
    const uint32_t *staged = stage + (lane & 8 ? pitch : 0) + (lane >> 4) * 4;   // rows 1 .. 7, 9 .. 15 are not used
    const auto h = flat_rsrc(a.h, (int64_t)a.K * a.I * 2);
    int experts = 0;
#pragma unroll 1
    for (int go = HELP ? 1 : 0; go < 2; go++) {
        int e = 0, pair = 0;
        if (go) {
            experts = wait_for<HELP>(a, DECODE_READY, sh);
            if (r >= experts)
                return experts >= 0;
            e = __builtin_amdgcn_readfirstlane((int)load4_sc1(flat_rsrc(a.list, (int64_t)a.most * 4), r * 4));
            pair = (int)(load4_sc1(flat_rsrc(a.pairs, (int64_t)a.most * ROWS * 2), r * ROWS * 2) & 0xFFFFu);
        }
        const auto w = window(a.gateup + e * a.gateup_stride + (int64_t)2 * cp * steps * MX_BLOCK_BYTES,
                              2 * (int64_t)steps * MX_BLOCK_BYTES, go);
        f32x4_t acc[2] = {};
#pragma unroll 1
        for (int s = 0; s < n; s += BATCH) {
            u32x4_t codes[BATCH][2];
            uint32_t scales[BATCH][2];
#pragma unroll
            for (int i = 0; i < BATCH; i++)
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    const int off = s + i < n ? (j * steps + s0 + s + i) * MX_BLOCK_BYTES : OUTSIDE;
                    codes[i][j] = fetch16<CPOL_NT>(w, off + lane * 16);
                    scales[i][j] = fetch4<CPOL_NT>(w, off + MX_CODE_BYTES + 4 * (lane & 15));
                }
            asm volatile("" ::: "memory");
#pragma unroll
            for (int i = 0; i < BATCH; i++) {
                u32x4_t x[4];
#pragma unroll
                for (int j = 0; j < 4; j++)
                    x[j] = *reinterpret_cast<const u32x4_t *>(staged + min(s + i, n - 1) * (MX_STEP / 2) + j * 16);
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    const f32x4_t v = mx_step(codes[i][j], scales[i][j], x, acc[j]);
                    acc[j] = s + i < n ? v : acc[j];
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        store_sums(red + (wv * 2) * 256, acc[0]);
        store_sums(red + (wv * 2 + 1) * 256, acc[1]);
        __syncthreads();
        if (t < 8) {   // two channels per thread
            float v[2][2];
#pragma unroll
            for (int j = 0; j < 2; j++)
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    v[j][i] = 0.f;
#pragma unroll
                    for (int k = 0; k < REST_WAVES; k++) {
                        const float *p = red + (k * 2 + j) * 256 + 2 * t + i;
                        v[j][i] += a.has_latent ? p[0] + p[HALF * 16] : p[0];
                    }
                }
            store4_sc1(h, go ? (pair * a.I + cp * 16 + 2 * t) * 2 : OUTSIDE,
                       pack_bf16x2(silu_f32(v[0][0]) * v[1][0], silu_f32(v[0][1]) * v[1][1]));
        }
    }
    if (arrive(a, DECODE_GATE, item, experts * pairs16))
        set_flag(a, DECODE_GATE_DONE, 0u);
    return true;
}

// ... with several: four such pairs per workgroup, one to a wave, each over all of K, so that z goes through LDS once for
// them all, STEPS steps at a time; weights come a chunk of as many steps ahead. Up to 8 tokens: one operand, whose rows
// 8 .. 15 are the remainders of rows 0 .. 7; more: two operands (PARTS). K is summed in four quarters, as above, so that a
// token's h is the same bits whatever tokens come with it.
template <int PARTS, bool HELP>
__device__ inline bool gate_many(const DecodeArgs &a, int item, uint32_t *lds, uint32_t *sh)
{
    constexpr int STEPS = 4, PITCH = STEPS * MX_STEP / 2 + 4, NTHR = WAVE * REST_WAVES;   // words of a row in LDS
    constexpr int PIECES = STEPS * 16 * 16 * PARTS / NTHR;   // 16-byte pieces of a chunk per thread
    static_assert(16 * PARTS * PITCH <= LDS_WORDS, "room for a chunk");
    const int lane = lane_id(), wv = wave_id(), t = threadIdx.x;
    const int groups = a.I / 16 / REST_WAVES, r = item / groups, cp = item % groups * REST_WAVES + wv;
    const int steps = a.Lt / MX_STEP;
    // piece i of this thread: 8 values of row i (t / 16 ..): a token's z, or HALF or ROWS rows further its remainders.
    // Rows past the tokens repeat the last one: their sums are not used.
    const auto z0 = flat_rsrc(a.z, (int64_t)a.T * a.Lt * 2), z1 = flat_rsrc(a.has_latent ? a.z_rest : a.z, (int64_t)a.T * a.Lt * 2);
    u32x4_t zs[PIECES];
    auto fetch = [&](int s) {
#pragma unroll
        for (int i = 0; i < PIECES; i++) {
            const int p = i * NTHR + t, row = p / (STEPS * 16), c = p % (STEPS * 16);
            const int token = min(row % (PARTS == 1 ? HALF : ROWS), a.T - 1), k = s * MX_STEP + c * 8;
            zs[i] = fetch16<0>(row >= (PARTS == 1 ? HALF : ROWS) ? z1 : z0, k < a.Lt ? (token * a.Lt + k) * 2 : OUTSIDE);
        }
    };
    fetch(0);
    const int experts = wait_for<HELP>(a, DECODE_READY, sh);
    if (r >= experts)
        return experts >= 0;
    const int e = __builtin_amdgcn_readfirstlane((int)load4_sc1(flat_rsrc(a.list, (int64_t)a.most * 4), r * 4));
    // the pairs of this lane's rows 4 (l / 16) .. +3
    const auto pairs = flat_rsrc(a.pairs, (int64_t)a.most * ROWS * 2);
    const uint32_t pair01 = load4_sc1(pairs, (r * ROWS + 4 * (lane >> 4)) * 2), pair23 = load4_sc1(pairs, (r * ROWS + 4 * (lane >> 4)) * 2 + 4);
    const auto w = window(a.gateup + e * a.gateup_stride + (int64_t)2 * cp * steps * MX_BLOCK_BYTES,
                          2 * (int64_t)steps * MX_BLOCK_BYTES, 1);
    struct Chunk {
        u32x4_t codes[STEPS][2];
        uint32_t scales[STEPS][2];
    } now, next;
    auto load = [&](int s, Chunk &q) {
#pragma unroll
        for (int i = 0; i < STEPS; i++)
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int off = s + i < steps ? (j * steps + s + i) * MX_BLOCK_BYTES : OUTSIDE;
                q.codes[i][j] = fetch16<CPOL_NT>(w, off + lane * 16);
                q.scales[i][j] = fetch4<CPOL_NT>(w, off + MX_CODE_BYTES + 4 * (lane & 15));
            }
    };
    load(0, now);
    f32x4_t acc[PARTS][2] = {}, sum[2] = {};
    int quarter = 1;   // ends at this many fourths of the steps; with fewer than four, some are empty
    while (steps * quarter / REST_WAVES == 0)
        quarter++;
    const uint32_t *mine = lds + (lane & 15) * PITCH + (lane >> 4) * 4;
#pragma unroll 1
    for (int s = 0; s < steps; s += STEPS) {
        __syncthreads();   // every wave is past the chunk before this one
#pragma unroll
        for (int i = 0; i < PIECES; i++) {
            const int p = i * NTHR + t;
            *reinterpret_cast<u32x4_t *>(lds + p / (STEPS * 16) * PITCH + p % (STEPS * 16) * 4) = zs[i];
        }
        fetch(s + STEPS);
        load(s + STEPS, next);
        asm volatile("" ::: "memory");
        __syncthreads();
#pragma unroll
        for (int i = 0; i < STEPS; i++) {   // steps past the end multiply zeros
#pragma unroll
            for (int p = 0; p < PARTS; p++) {
                u32x4_t x[4];
#pragma unroll
                for (int j = 0; j < 4; j++)
                    x[j] = *reinterpret_cast<const u32x4_t *>(mine + p * ROWS * PITCH + i * (MX_STEP / 2) + j * 16);
#pragma unroll
                for (int j = 0; j < 2; j++)
                    acc[p][j] = mx_step(now.codes[i][j], now.scales[i][j], x, acc[p][j]);
            }
            if (s + i + 1 == steps * quarter / REST_WAVES) {
#pragma unroll
                for (int j = 0; j < 2; j++) {
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const float rest = PARTS == 1 ? __shfl_xor(acc[0][j][k], 32) : acc[PARTS - 1][j][k];
                        sum[j][k] += a.has_latent ? acc[0][j][k] + rest : acc[0][j][k];
                    }
#pragma unroll
                    for (int p = 0; p < PARTS; p++)
                        acc[p][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
                }
                while (steps * quarter / REST_WAVES == s + i + 1)
                    quarter++;
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        now = next;
    }
    // two channels to a word; rows of the upper half of the lanes are remainders where PARTS = 1
    const auto h = flat_rsrc(a.h, (int64_t)a.T * a.K * a.I * 2);
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const float v = silu_f32(sum[0][k]) * sum[1][k], after = __shfl_down(v, 1);
        const int pair = (int16_t)((k < 2 ? pair01 : pair23) >> (16 * (k % 2))), token = 4 * (lane >> 4) + k;
        const bool keep = pair >= 0 && token < a.T && lane % 2 == 0;
        store4_sc1(h, keep ? (pair * a.I + cp * 16 + (lane & 15)) * 2 : OUTSIDE, pack_bf16x2(v, after));
    }
    if (arrive(a, DECODE_GATE, item, experts * groups))
        set_flag(a, DECODE_GATE_DONE, 0u);
    return true;
}

// 16 latent columns of every chosen expert, by `parts` workgroups: expert number r of the list is workgroup r % parts's, and
// of its own the i-th is wave i % 4's. Every expert's y goes to memory (or, of one workgroup, to LDS) by pairs of token and
// slot; the last workgroup to arrive at the columns adds each token's in slot order: so a token's outputs are the same
// bits whatever tokens come with it.
//
// Experts come in units of up to STEPS blocks: weights RING units ahead, the first before h is known, with everything that
// is looked up of a unit. IN_LDS: all of h fits there; else an operand is loaded when it is needed. False when patience
// runs out.
struct DownPart {
    int16_t *pairs;      // LDS: [experts][16] the pair of (expert, token), or -1
    uint16_t *list;      // LDS: [experts]
    float *y;            // LDS: [pairs][16], for one workgroup
    uint32_t *staged;    // LDS: h
    int col, part, parts;
};
template <bool IN_LDS, bool HELP>
__device__ inline bool down_part(const DecodeArgs &a, const DownPart &q, uint32_t *sh)
{
    constexpr int STEPS = 3, RING = IN_LDS ? 4 : 2, NTHR = WAVE * REST_WAVES;
    const int lane = lane_id(), wv = wave_id();
    const int steps = a.I / MX_STEP, groups = (steps + STEPS - 1) / STEPS, P = a.T * a.K;
    const int h_pitch = IN_LDS ? a.I / 2 + 4 : a.I / 2;   // words of a row
    struct Unit {
        u32x4_t codes[STEPS];
        uint32_t scales[STEPS];
        int row;           // words to the operand's row: any where the token did not choose the expert
        uint2 pairs;       // of the sums' rows
    } ring[RING];
    const auto y_out = flat_rsrc(a.partial + (int64_t)q.col * P * 16, (int64_t)P * 64);
#pragma unroll 1
    for (int go = !HELP && a.T <= 2 ? 0 : 1; go < 2; go++) {
        int count = 0;   // own experts
        if (go) {
            const int experts = wait_for<HELP>(a, DECODE_READY, sh);
            if (experts < 0)
                return false;
            const auto gl = flat_rsrc(a.list, (int64_t)a.most * 4), gp = flat_rsrc(a.pairs, (int64_t)a.most * ROWS * 2);
#pragma unroll 1
            for (int i = threadIdx.x; i < experts * (ROWS / 2); i += NTHR)
                reinterpret_cast<uint32_t *>(q.pairs)[i] = load4_sc1(gp, i * 4);
#pragma unroll 1
            for (int i = threadIdx.x; i < experts; i += NTHR)
                q.list[i] = (uint16_t)load4_sc1(gl, i * 4);
            __syncthreads();
            const int first = q.part + q.parts * wv;
            count = first < experts ? (experts - first - 1) / (q.parts * REST_WAVES) + 1 : 0;
        }
        const int units = go ? count * groups : RING;
        const auto h = window(a.h, (int64_t)P * a.I * 2, go);
        int at = 0, at_group = 0;   // the next unit: own expert and group
        auto load = [&](Unit &u) {
            const bool in = at < count;
            const int r = in ? q.part + q.parts * (wv + REST_WAVES * at) : 0;
            const int e = in ? __builtin_amdgcn_readfirstlane((int)q.list[r]) : 0;
            const auto w = window(a.down + e * a.down_stride + ((int64_t)q.col * steps + at_group * STEPS) * MX_BLOCK_BYTES,
                                  (int64_t)min(steps - at_group * STEPS, STEPS) * MX_BLOCK_BYTES, in);
#pragma unroll
            for (int s = 0; s < STEPS; s++) {
                u.codes[s] = fetch16<CPOL_NT>(w, s * MX_BLOCK_BYTES + lane * 16);
                u.scales[s] = fetch4<CPOL_NT>(w, s * MX_BLOCK_BYTES + MX_CODE_BYTES + 4 * (lane & 15));
            }
            u.row = min(max((int)q.pairs[r * ROWS + (lane & 15)], 0), P - 1) * h_pitch + at_group * STEPS * (MX_STEP / 2) + 4 * (lane >> 4);
            u.pairs = *reinterpret_cast<const uint2 *>(q.pairs + r * ROWS + 4 * (lane >> 4));
            const bool end = at_group + 1 == groups;
            at += end;
            at_group = end ? 0 : at_group + 1;
        };
#pragma unroll
        for (int d = 0; d < RING; d++)
            load(ring[d]);
        asm volatile("" ::: "memory");
        if (go && wait_for<HELP>(a, DECODE_GATE_DONE, sh) < 0)
            return false;
        if constexpr (IN_LDS) {
            const int chunks = a.I / 8;
#pragma unroll 1
            for (int i0 = threadIdx.x; i0 < P * chunks; i0 += 4 * NTHR) {
                u32x4_t v[4];
#pragma unroll
                for (int k = 0; k < 4; k++)
                    v[k] = fetch16<CPOL_SC1>(h, min(i0 + k * NTHR, P * chunks - 1) * 16);
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const int i = min(i0 + k * NTHR, P * chunks - 1);
                    *reinterpret_cast<u32x4_t *>(q.staged + i / chunks * h_pitch + i % chunks * 4) = v[k];
                }
            }
            __syncthreads();
        }
        f32x4_t y[STEPS] = {};   // three chains of sums, each over every third block
        int group = 0;
#pragma unroll 1
        for (int u0 = 0; u0 < units; u0 += RING)
#pragma unroll
            for (int d = 0; d < RING; d++) {
                Unit &u = ring[d];
                u32x4_t x[STEPS][4];
#pragma unroll
                for (int s = 0; s < STEPS; s++) {   // past the row's end, where the weights are zeros: anything
                    const int word = u.row + (group * STEPS + s < steps ? s * (MX_STEP / 2) : 0);
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        if constexpr (IN_LDS)
                            x[s][j] = *reinterpret_cast<const u32x4_t *>(q.staged + word + j * 16);
                        else
                            x[s][j] = fetch16<CPOL_SC1>(h, (word + j * 16) * 4);
                }
#pragma unroll
                for (int s = 0; s < STEPS; s++) {
                    const f32x4_t v = mx_step(u.codes[s], u.scales[s], x[s], y[s]);
                    y[s] = group * STEPS + s < steps ? v : y[s];
                }
                const bool end = group + 1 == groups;
                if (end) {
                    const f32x4_t v = y[0] + y[1] + y[2];
                    const bool live = go && u0 + d < units;
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const int pair = (int16_t)((j < 2 ? u.pairs.x : u.pairs.y) >> (16 * (j % 2)));
                        const bool keep = live && pair >= 0;
                        if (q.parts > 1)
                            store4_sc1(y_out, keep ? (pair * 16 + (lane & 15)) * 4 : OUTSIDE, __float_as_uint(v[j]));
                        else if (keep)
                            q.y[pair * 16 + (lane & 15)] = v[j];
                    }
#pragma unroll
                    for (int s = 0; s < STEPS; s++)
                        y[s] = f32x4_t{0.f, 0.f, 0.f, 0.f};
                }
                __builtin_amdgcn_sched_barrier(0);   // no more at a time than there are registers for
                group = end ? 0 : group + 1;
                load(u);
            }
    }
    return true;
}

template <bool HELP>
__device__ inline bool down_item(const DecodeArgs &a, int item, int parts, uint32_t *lds, uint32_t *sh)
{
    const int wv = wave_id(), t = threadIdx.x, row = t / 16, c = t % 16, K = a.K, P = a.T * K;
    DownPart q;
    q.pairs = reinterpret_cast<int16_t *>(lds);
    q.list = reinterpret_cast<uint16_t *>(lds + a.most * (ROWS / 2));
    uint32_t *after = lds + a.most * (ROWS / 2) + (a.most + 7) / 8 * 4;
    q.y = reinterpret_cast<float *>(after);
    q.staged = after + (parts == 1 ? P * 16 : 0);
    q.col = item / parts;
    q.part = item % parts;
    q.parts = parts;
    const bool in_lds = (int)(q.staged - lds) + P * (a.I / 2 + 4) <= LDS_WORDS;
    if (!(in_lds ? down_part<true, HELP>(a, q, sh) : down_part<false, HELP>(a, q, sh)))
        return false;
    if (parts > 1) {
        stores_done();
        if (wv == 0) {
            const bool last = last_at(a.column_counters + q.col, parts);
            if (t == 0)
                *sh = last;
        }
    }
    __syncthreads();
    const bool mine = parts == 1 || *sh != 0u;
    __syncthreads();
    if (!mine)
        return true;
    const auto weights = flat_rsrc(a.weights, (int64_t)P * 4), y = flat_rsrc(a.partial + (int64_t)q.col * P * 16, (int64_t)P * 64);
    float v = 0.f;
#pragma unroll 1
    for (int j0 = 0; j0 < K; j0 += 8) {   // slots past the last are a weight of zero times zero
        float w[8], ys[8];
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int pair = row * K + j0 + j;
            const bool in = row < a.T && j0 + j < K;
            w[j] = __uint_as_float(fetch4<CPOL_SC1>(weights, in ? pair * 4 : OUTSIDE));
            ys[j] = parts == 1 ? q.y[(in ? pair : 0) * 16 + c] : __uint_as_float(fetch4<CPOL_SC1>(y, in ? (pair * 16 + c) * 4 : OUTSIDE));
        }
#pragma unroll
        for (int j = 0; j < 8; j++)
            v = j0 + j < K ? fmaf(w[j], ys[j], v) : v;
    }
    // two columns to a word
    const uint32_t two = pack_bf16x2(v, __shfl_down(v, 1));
    if (row < a.T && c % 2 == 0) {
        if (a.has_latent)
            store4_sc1(flat_rsrc(a.acat, (int64_t)a.T * a.ldcat * 2), (row * a.ldcat + q.col * 16 + c) * 2, two);
        else
            *reinterpret_cast<uint32_t *>(a.out + (int64_t)row * a.Lt + q.col * 16 + c) = two;
    }
    if (a.has_latent && arrive(a, DECODE_DOWN, q.col, a.Lt / 16))
        set_flag(a, DECODE_DOWN_DONE, 0u);
    return true;
}

template <bool HELP>
__device__ inline bool out_item(const DecodeArgs &a, int item, uint32_t *lds, uint32_t *sh)
{
    const int wv = wave_id(), t = threadIdx.x, row = t / 8, c = t % 8 * 2;
    float *red = reinterpret_cast<float *>(lds + REST_WAVES * STAGE_WORDS);
    const auto out = flat_rsrc(a.out, (int64_t)a.T * a.H * 2);
    auto run = [&](auto part) {
#pragma unroll 1
        for (int go = !HELP && a.T <= 2 ? 0 : 1; go < 2; go++) {
            part.start(a.w_out, a.H, a.ldcat, item, wv, REST_WAVES, go);
            if (go && wait_for<HELP>(a, DECODE_DOWN_DONE, sh) < 0)
                return false;
            const auto acat = window(a.acat, (int64_t)a.T * a.ldcat * 2, go);
            f32x4_t acc[1] = {};
            part.finish(a.T, lds + wv * STAGE_WORDS, acc,
                        [&](int r, int k) { return fetch16<CPOL_SC1>(acat, (r * a.ldcat + k) * 2); });
            store_sums(red + wv * 256, acc[0]);
            __syncthreads();
            if (row < a.T && row < ROWS)
                __builtin_amdgcn_raw_buffer_store_b32((int)pack_bf16x2(total<REST_WAVES>(red, 256, row * 16 + c),
                                                                       total<REST_WAVES>(red, 256, row * 16 + c + 1)),
                                                      out, go ? (row * a.H + item * 16 + c) * 2 : OUTSIDE, 0, 0);
            __syncthreads();
        }
        return true;
    };
    using Staged = Bf16Part<1, OUT_DEPTH, 4, true>;   // all of a wave's weights at the widths of a TP8 share, and some more
    if (Staged::fits(a.T, a.ldcat, REST_WAVES))
        return run(Staged());
    return run(Bf16Part<1, 12, 4, false>());
}

// Item i, as numbered by decode_items. False when patience ran out before anything was handed on (HELP: never).
template <bool FEW, bool HELP>
__device__ inline bool do_item(const DecodeArgs &a, const DecodeItems &n, int i, uint32_t *lds, uint32_t *sh)
{
    if (i < n.top) {
        top_item(a, lds);
        return true;
    }
    i -= n.top;
    if (i < n.gate) {
        if constexpr (FEW)
            if (decode_gate_one(a))
                return gate_one<HELP>(a, i, lds, sh);
        return gate_many<FEW ? 1 : 2, HELP>(a, i, lds, sh);
    }
    i -= n.gate;
    if (i < n.down)
        return down_item<HELP>(a, i, n.parts, lds, sh);
    return out_item<HELP>(a, i - n.down, lds, sh);
}

template <bool FEW>
__global__ __launch_bounds__(WAVE *REST_WAVES, 3) void rest_kernel(const DecodeArgs a)
{
    constexpr int TOP = DECODE_MAX_E + ROWS * 32 + 16, MOST = ROWS * 32;   // MOST: pairs, and distinct experts
    static_assert(TOP + REST_WAVES * DECODE_MAX_E <= LDS_WORDS && TOP + MOST * (ROWS / 2) <= LDS_WORDS, "room for the list");
    static_assert(MOST * (ROWS / 2) + MOST / 2 <= LDS_WORDS && 32 * (ROWS / 2) + 16 + 32 * 16 <= LDS_WORDS, "... and the routing");
    static_assert(STAGE_WORDS == DECODE_STAGE_WORDS && REST_WAVES == 4, "what decode.hpp says");
    __shared__ alignas(16) uint32_t lds[LDS_WORDS];
    __shared__ uint32_t sh;
    const DecodeItems n = decode_items(a);
    const int item = blockIdx.x;
    if (!claim<false>(a, item, &sh) || do_item<FEW, false>(a, n, item, lds, &sh))
        return;
    const int kind = item < n.top + n.gate ? n.top : item < n.top + n.gate + n.down ? n.top + n.gate : n.top + n.gate + n.down;
#pragma unroll 1
    for (int i = 0; i <= kind; i++)   // the earlier kinds' items that are still free, and then this one
        if (i == kind || claim<true>(a, i, &sh))
            do_item<FEW, true>(a, n, i == kind ? item : i, lds, &sh);
}

} // namespace

hipError_t launch_decode(const DecodeArgs &a, hipStream_t st)
{
    const unsigned front = (unsigned)(a.shared / 16 + (a.has_latent ? a.Lt / 16 : 0) + a.n_router_rows / 16);
    hipLaunchKernelGGL(front_kernel, dim3(front), dim3(WAVE * FRONT_WAVES), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    const DecodeItems n = decode_items(a);
    const dim3 grid((unsigned)decode_item_count(n)), threads(WAVE * REST_WAVES);
    if (a.T <= HALF)
        hipLaunchKernelGGL((rest_kernel<true>), grid, threads, 0, st, a);
    else
        hipLaunchKernelGGL((rest_kernel<false>), grid, threads, 0, st, a);
    return hipGetLastError();
}

} // namespace mxmoe
