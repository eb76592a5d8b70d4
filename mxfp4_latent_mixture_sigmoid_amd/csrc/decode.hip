// decode.hip -- the whole layer for up to 16 tokens in one kernel, after a small one that clears its counters.
//
// The tokens are one row tile of the matrix-core instruction, so every weight is read once, from memory, and
// multiplied with all tokens at once: the time is the weights' (184 MB for one token of a TP8 share: the router, latent
// and shared matrices in BF16, 16 experts in MXFP4; 640 MB and 220 experts for 16). The kernel is a list of work items,
// one for each workgroup, numbered kind after kind:
//    router  (16 experts, a quarter of x): their part of x W_r^T
//    latent  16 columns of z = x W_down^T
//    top     the top-K of 4 tokens; the list of distinct experts and each one's tokens
//    gate    (expert, 16 or 64 inner channels): h = silu(z Wg^T) (z Wu^T) of the expert's tokens
//    shared  16 channels of h_s = silu(x Wg_s^T) (x Wu_s^T)
//    down    (expert, 256 or 512 latent columns): y = h Wd^T of the expert's tokens, in FP32
//    sums    (4 tokens, 256 latent columns): zc = sum w y, in slot order
//    out     16 output columns: out = bf16([zc | h_s] [W_up | W_ds]^T)
// so that the memory's rate is not lost at the borders of launches: an item's first weights are asked for before what it
// waits for is there. One token takes 54 us (3.4 TB/s), and 68 as separate launches (moe_route_forward); 4 tokens 75 and
// 82, 8 99 and 103, 9 122 and 107, 16 166 and 136: with many experts an item's start, 5 us of claiming and looking up while its place
// waits, costs more than the launches. One token's way: z after 16 us, the experts 19, h 31, y 37, zc 41, out 52.
//
// z, h, h_s and zc are kept in two BF16 parts, the rounded value and what the rounding left, 16 bits of each value: rounded to
// one, z and h cost 0.4% of the layer's output in the mean square, h_s and zc 0.17%; with both parts the output's own
// rounding is what is left, 0.17%. The remainders are rows 8 to 15 of the tile for up to 8 tokens, and a second operand
// for more (16 tokens: 190 us, 178 with h rounded, when it was added). The output product reads twice the activations for
// them: 4 tokens 75.4 us (74.8 without), 8 98.6 (97.0), 16 166 (166), where zc and h_s lie as z does; 80, 105 and 181 with
// zc among y.
//
// Kinds wait for each other on flags. A workgroup takes the item of its number by claiming it; it waits for a flag PATIENCE
// times, far longer than a call takes, and if the flag has not come by then (its workgroups may not even have started:
// another call's, which wait for theirs, may hold their places) it claims and does whatever item of an earlier kind is
// still free, in order, and waits again. Then every item that it waits for is done or being worked on by a workgroup that
// runs, so that all waits end, however many workgroups the card holds at once and whatever else runs on it. (Drawing
// items from one ticket counter gives that too, but additions to one address take 12 ns each: 1057 workgroups kept the
// top-K's loads waiting for 9 us behind theirs.) For the same reason a flag that every workgroup asks for is written in 64
// places; the gate items of an expert, and the down items of 256 columns, have a counter of their own, on which the few
// items wait that need them. What one workgroup hands to another goes through agent-coherent stores and loads (sync.hpp).
//
// Two things set the pace of code that runs once. Instructions come from memory at about 1 KiB a microsecond the first
// time: so while an item waits it goes once through what it will do, with empty windows for its loads and stores
// (`go` = 0). And a load under a condition is a wait for the loads before it: so no load of weights has one; loads past the
// end lie outside their window, which costs nothing. Workgroups that start when the experts are known leave the first pass out
// (with it in every down item, and none before the gate items of several tokens, 8 tokens took 104 us, 97 so).
//
// Three workgroups share a CU (168 registers a thread). The items fit those, but for the down item of more than 8 tokens, which
// keeps 18 in memory; what else the compiler reports as spilled is in the items' second form, for helpers, in the same kernel,
// which hardly ever runs. With four workgroups of 128 more of them start early, but one token took 61 us.
//
// Batches of loads divide a wave's part of the widths 7168 and 3584, for which these figures are: 7 of the gate product's 28 / 4 steps, 14 of
// the front products' 224 / 4 and 224 / 16. Other widths end in a batch that is partly empty windows: right, and at most a batch's
// latency longer.
#include "decode.hpp"
#include "select.hpp"
#include "sync.hpp"

// Each item is compiled several times (for the helpers, for up to 8 tokens and more), and has to give the same bits in each: a
// product and a sum are one operation only where the code says so. Left to choose, the compiler took the remainder of
// silu(g) u from the unrounded product in the helpers' copy of one token's gate item, and from the rounded one in the other.
#pragma clang fp contract(off)

namespace mxmoe {

namespace {

constexpr int ROWS = DECODE_MAX_T, HALF = ROWS / 2;
constexpr int REST_WAVES = 4, ROUTER_PARTS = DECODE_ROUTER_PARTS;
constexpr int FLAGS = WAVE;                 // places of a flag
constexpr int STAGE_WORDS = DECODE_STAGE_WORDS;
constexpr int OUT_STAGE_WORDS = DECODE_OUT_STAGE_WORDS;
constexpr int LDS_WORDS = REST_WAVES * (STAGE_WORDS + 512 > OUT_STAGE_WORDS ? STAGE_WORDS + 512 : OUT_STAGE_WORDS);   // of an item
static_assert((LDS_WORDS * 4 + 16 + 1279) / 1280 * 1280 * 3 <= 160 * 1024, "three workgroups share a CU");

__device__ __forceinline__ uint32_t *counter(const DecodeArgs &a, int i) { return a.counters + i * DECODE_COUNTER_WORDS; }
__device__ __forceinline__ uint32_t *flag(const DecodeArgs &a, int i, int place) { return counter(a, DECODE_FLAGS + i * FLAGS + place); }
__device__ __forceinline__ uint32_t ask(const uint32_t *at) { return __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

__device__ __forceinline__ int lane_id() { return threadIdx.x & (WAVE - 1); }
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE); }

// Windows for loads and stores: those outside read zeros and write nothing, without touching memory. `go` = 0: an empty one.
constexpr int OUTSIDE = DECODE_MAX_WINDOW;   // an offset past every window
__device__ __forceinline__ __amdgpu_buffer_rsrc_t window(const void *base, int64_t bytes, int go) { return flat_rsrc(base, go ? bytes : 0); }
template <int CPOL>
__device__ __forceinline__ u32x4_t fetch16(__amdgpu_buffer_rsrc_t w, int offset)
{
    return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(w, offset, 0, CPOL));
}
template <int CPOL>
__device__ __forceinline__ uint32_t fetch4(__amdgpu_buffer_rsrc_t w, int offset)
{
    return (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(w, offset, 0, CPOL);
}

// Lane l's four sums of a fragment are those of rows 4 (l / 16) .. +3 in column l % 16.
__device__ __forceinline__ void store_sums(float *red, f32x4_t v)
{
    const int lane = lane_id();
#pragma unroll
    for (int i = 0; i < 4; i++)
        red[(4 * (lane >> 4) + i) * 16 + (lane & 15)] = v[i];
}

// Two values as BF16 and what that rounding left, in BF16 as well: 16 bits of each value in all.
__device__ __forceinline__ void split(float v0, float v1, uint32_t &high, uint32_t &rest)
{
    high = pack_bf16x2(v0, v1);
    const float h0 = __uint_as_float(high << 16), h1 = __uint_as_float(high & 0xFFFF0000u);
    rest = pack_bf16x2(fabsf(h0) < INFINITY ? v0 - h0 : 0.f, fabsf(h1) < INFINITY ? v1 - h1 : 0.f);
}

// Sum of one element over the waves' fragments, in wave order.
template <int WAVES>
__device__ __forceinline__ float total(const float *red, int stride, int at)
{
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; w++)
        v += red[w * stride + at];
    return v;
}

// A wave's part of a BF16 product: 32-wide steps s0 .. s1 - 1 of NB row blocks, all T tokens at once. The weights are loaded
// DEPTH steps ahead, the first before anything is known of the activations. Those go through the wave's part of LDS: all of
// them where they fit (CHUNK = 0: few tokens), else CHUNK steps at a time, each chunk loaded while the one before it is
// multiplied. (Straight to registers a step's operand is 64 bytes of every row: 8 tokens 111 us in place of 104.)
//
// REST: activations come with what their rounding to BF16 left, which is multiplied as well: 1, in rows 8 to 15 of the operand, of up
// to 8 tokens; 2, as a second operand, of more.
template <int NB, int DEPTH, int CHUNK, int REST = 0>
struct Bf16Part {
    static_assert(CHUNK == 0 || DEPTH % CHUNK == 0, "slots");
    static constexpr int WORDS = REST ? OUT_STAGE_WORDS : STAGE_WORDS, OPERANDS = REST == 2 ? 2 : 1;
    // Whether K values of T tokens, divided among the waves, fit their parts of LDS.
    static __device__ bool fits(int T, int K, int waves) { return T * (REST ? 2 : 1) * ((K / BF16_STEP + waves - 1) / waves * 16 + 4) <= WORDS; }
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
    // get(row, k, in, i): 16 bytes of a token's activations from column k on, or zeros; i = 1: of their remainders.
    struct Loaded {
        u32x4_t v[REST ? 2 : 1];
    };
    template <class Get>
    static __device__ __forceinline__ Loaded loaded(Get &get, int row, int k, bool in)
    {
        Loaded l;
#pragma unroll
        for (int i = 0; i < (REST ? 2 : 1); i++)
            l.v[i] = get(row, k, in, i);
        return l;
    }
    // The values to `at`, the remainders `rest` words further.
    static __device__ __forceinline__ void put(const Loaded &l, uint32_t *at, int rest)
    {
#pragma unroll
        for (int i = 0; i < (REST ? 2 : 1); i++)
            *reinterpret_cast<u32x4_t *>(at + i * rest) = l.v[i];
    }
    // One step: `at` is this lane's place in the first operand, the second is `second` words further.
    __device__ __forceinline__ void multiply(const uint32_t *at, int second, int slot, bool in, f32x4_t (&acc)[OPERANDS][NB])
    {
#pragma unroll
        for (int p = 0; p < OPERANDS; p++) {
            const u32x4_t x = *reinterpret_cast<const u32x4_t *>(at + p * second);
#pragma unroll
            for (int j = 0; j < NB; j++)
                acc[p][j] = step(x, b[slot][j], acc[p][j], in);
        }
    }
    template <class Get>
    __device__ __forceinline__ void finish(int T, uint32_t *stage, f32x4_t (&acc)[OPERANDS][NB], Get get)
    {
        const int lane = lane_id(), n = s1 - s0;
        // rows past the tokens repeat the last one: their sums are not used. Steps past the end multiply zeros.
        const int row = lane & 15, r = min(REST == 1 ? row % HALF : row, T - 1), c = lane >> 4;
        if constexpr (CHUNK == 0) {
            static_assert(REST < 2, "one operand");
            const int pitch = n * 16 + 4;   // words of a token's part in LDS
#pragma unroll 1
            for (int i0 = 0; i0 < T * n * 4; i0 += 4 * WAVE) {
                Loaded v[4];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int at = min(i0 + i * WAVE + lane, T * n * 4 - 1);
                    v[i] = loaded(get, at / (n * 4), s0 * BF16_STEP + at % (n * 4) * 8, true);
                }
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int at = min(i0 + i * WAVE + lane, T * n * 4 - 1);
                    put(v[i], stage + at / (n * 4) * pitch + at % (n * 4) * 4, T * pitch);
                }
            }
            meet_lanes();
            const uint32_t *mine = stage + ((REST == 1 && row >= HALF ? T : 0) + r) * pitch + c * 4;
#pragma unroll 1
            for (int s = 0; s < n; s += DEPTH)
#pragma unroll
                for (int i = 0; i < DEPTH; i++) {
                    multiply(mine + min(s + i, n - 1) * 16, 0, i, s + i < n, acc);
                    load(i);
                    if (i % 4 == 3)
                        __builtin_amdgcn_sched_barrier(0);   // not all operands at once
                }
        } else {
            constexpr int PITCH = CHUNK * 16 + 4, PER_ROW = CHUNK * 4, TOKENS = REST == 0 ? WORDS / PITCH : REST == 1 ? HALF : ROWS;
            constexpr int PIECES = TOKENS * PER_ROW / WAVE, SECOND = TOKENS * PITCH;
            static_assert(TOKENS * PER_ROW % WAVE == 0 && TOKENS * (REST ? 2 : 1) * PITCH <= WORDS, "pieces; room");
            Loaded v[PIECES];
            auto fetch = [&](int s) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < PIECES; i++) {
                    const int at = i * WAVE + lane, token = at / PER_ROW, col = at % PER_ROW;
                    v[i] = loaded(get, token, (s0 + s) * BF16_STEP + col * 8, token < T && s + col / 4 < n);
                }
            };
            const uint32_t *mine = stage + (REST == 1 && row >= HALF ? SECOND : 0) + r * PITCH + c * 4;
            fetch(0);
#pragma unroll 1
            for (int s = 0; s < n; s += DEPTH)
#pragma unroll
                for (int h = 0; h < DEPTH; h += CHUNK) {
#pragma unroll
                    for (int i = 0; i < PIECES; i++)
                        put(v[i], stage + (i * WAVE + lane) / PER_ROW * PITCH + (i * WAVE + lane) % PER_ROW * 4, SECOND);
                    meet_lanes();
                    fetch(s + h + CHUNK);
#pragma unroll
                    for (int i = 0; i < CHUNK; i++) {
                        multiply(mine + i * 16, SECOND, h + i, s + h + i < n, acc);
                        load(h + i);
                        if (i % 4 == 3)
                            __builtin_amdgcn_sched_barrier(0);
                    }
                    meet_lanes();   // the chunk is read before it is overwritten
                }
        }
    }
    // A step past the end adds nothing, whatever the activations are.
    static __device__ f32x4_t step(u32x4_t x, u32x4_t w, f32x4_t acc, bool in)
    {
        const f32x4_t v = mfma16(as_bf16x8(x), as_bf16x8(w), acc);
        return in ? v : acc;
    }
};

// Until the flag or counter at `at` is at least `least`: its value, or -1 when patience runs out (HELP: never). `v` is what it
// was before. One thread asks; what follows in any thread is after the answer.
template <bool HELP>
__device__ __forceinline__ int wait_for(const DecodeArgs &a, const uint32_t *at, uint32_t least, uint32_t *sh, uint32_t v = 0u)
{
    if (threadIdx.x == 0) {
        int left = a.patience;
        while (v < least && (HELP || left-- > 0)) {
            v = ask(at);
            if (v < least)
                __builtin_amdgcn_s_sleep(2);
        }
        *sh = v < least ? ~0u : v;
    }
    __syncthreads();
    const int got = __builtin_amdgcn_readfirstlane((int)*sh);
    __syncthreads();
    asm volatile("" ::: "memory");
    return got;
}
struct Seen {
    uint32_t ready, z;   // two flags as they were a while ago
    int first_pass;      // 0: none through the code before the experts are known (they are, or this is a helper)
};
// Until the experts are known: how many, or -1.
template <bool HELP>
__device__ __forceinline__ int wait_ready(const DecodeArgs &a, const Seen &seen, uint32_t *sh)
{
    const int v = wait_for<HELP>(a, flag(a, DECODE_READY, blockIdx.x % FLAGS), 1u, sh, seen.ready);
    return v < 0 ? v : v - 1;
}
// Until z is there.
template <bool HELP>
__device__ __forceinline__ bool wait_z(const DecodeArgs &a, const Seen &seen, uint32_t *sh)
{
    return !a.has_latent || wait_for<HELP>(a, flag(a, DECODE_Z_DONE, blockIdx.x % FLAGS), 1u, sh, seen.z) >= 0;
}

// Whether item `i` is this workgroup's now. `also` goes into *sh beside the answer.
template <bool HELP>
__device__ __forceinline__ bool claim(const DecodeArgs &a, int i, uint32_t *sh, uint32_t also = 0u)
{
    if (threadIdx.x == 0) {
        uint32_t *at = a.claims + i;
        const bool free = !(HELP && ask(at) != 0u) && __hip_atomic_fetch_add(at, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == 0u;
        *sh = (free ? 1u : 0u) | also;
    }
    __syncthreads();
    const bool mine = (__builtin_amdgcn_readfirstlane((int)*sh) & 1) != 0;
    __syncthreads();
    return mine;
}

__device__ __forceinline__ void set_flag(const DecodeArgs &a, int i, uint32_t v)   // by a wave
{
    __hip_atomic_store(flag(a, i, lane_id()), v + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Every wave's stores have completed.
__device__ __forceinline__ void stores_done()
{
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    asm volatile("" ::: "memory");
    __syncthreads();
}

__device__ __forceinline__ bool last_at(uint32_t *at, int all)   // by a wave
{
    uint32_t before = 0u;
    if (lane_id() == 0)
        before = __hip_atomic_fetch_add(at, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return __builtin_amdgcn_readfirstlane((int)before) == all - 1;
}

// Counts this workgroup after its stores.
__device__ __forceinline__ void arrive(uint32_t *at)
{
    stores_done();
    if (threadIdx.x == 0)
        __hip_atomic_fetch_add(at, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ... after its part of [zc | h_s].
__device__ __forceinline__ void arrive_out(const DecodeArgs &a)
{
    stores_done();
    if (wave_id() == 0 && last_at(counter(a, DECODE_CAT), a.items.shared + a.items.sums))
        set_flag(a, DECODE_CAT_DONE, 0u);
}

// 16 columns (NB = 2: two such blocks) of a BF16 product over x; the waves share the K axis and leave their sums in LDS. The
// weights are asked for before the item is claimed. False when another workgroup has it.
template <int NB, bool HELP>
__device__ __forceinline__ bool front_product(const DecodeArgs &a, const uint8_t *w, int64_t rows, int block, uint32_t *lds, uint32_t *sh, int part_of_k = 0, int parts = 1)
{
    const int wv = wave_id();
    const auto x = flat_rsrc(a.x, (int64_t)a.T * a.Hin * 2);
    f32x4_t acc[1][NB] = {};
    auto run = [&](auto part) __attribute__((always_inline)) {
        part.start(w, rows, a.Hin, block, part_of_k * REST_WAVES + wv, parts * REST_WAVES);
        if (!HELP && !claim<false>(a, blockIdx.x, sh))
            return false;
        part.finish(a.T, lds + wv * STAGE_WORDS, acc, [&](int r, int k, bool in, int) __attribute__((always_inline)) { return fetch16<0>(x, in ? (r * a.Hin + k) * 2 : OUTSIDE); });
        return true;
    };
    using Staged = Bf16Part<NB, 16 / NB, 0>;
    if (!(Staged::fits(a.T, a.Hin, parts * REST_WAVES) ? run(Staged()) : run(Bf16Part<NB, 14 / NB, 7>())))
        return false;
    __syncthreads();
    float *red = reinterpret_cast<float *>(lds);
#pragma unroll
    for (int j = 0; j < NB; j++)
        store_sums(red + (wv * NB + j) * 256, acc[0][j]);
    __syncthreads();
    return true;
}

// 16 experts' logits over one of ROUTER_PARTS parts of x. (All front items run at once and share the memory's rate: so the
// router's are short, and the top-K is done before z.)
template <bool HELP>
__device__ __forceinline__ void router_item(const DecodeArgs &a, int item, uint32_t *lds, uint32_t *sh)
{
    const int part = item % ROUTER_PARTS, block = item / ROUTER_PARTS;
    if (!front_product<1, HELP>(a, a.w_router, a.n_router_rows, block, lds, sh, part, ROUTER_PARTS))
        return;
    const int t = threadIdx.x, row = t / 16, n = block * 16 + t % 16;
    const float v = total<REST_WAVES>(reinterpret_cast<const float *>(lds), 256, t);
    if (row < a.T && n < a.E)
        store4_sc1(flat_rsrc(a.logits, (int64_t)ROUTER_PARTS * a.T * a.E * 4), ((part * a.T + row) * a.E + n) * 4, __float_as_uint(v));
    arrive(counter(a, DECODE_ROUTER));
}

// 16 latent columns.
template <bool HELP>
__device__ __forceinline__ void latent_item(const DecodeArgs &a, int item, int items, uint32_t *lds, uint32_t *sh)
{
    if (!front_product<1, HELP>(a, a.w_latent, a.n_latent_rows, item, lds, sh))
        return;
    const int t = threadIdx.x, row = t / 8, c = t % 8 * 2;
    if (row < a.T) {   // a wave each of 8 rows: at most 16 rows, two waves
        const float *red = reinterpret_cast<const float *>(lds);
        const float v0 = total<REST_WAVES>(red, 256, row * 16 + c), v1 = total<REST_WAVES>(red, 256, row * 16 + c + 1);
        uint32_t high, rest;
        split(v0, v1, high, rest);
        const int at = (row * a.ldz + item * 16 + c) * 2;
        store4_sc1(flat_rsrc(a.z, (int64_t)a.T * a.ldz * 2), at, high);
        store4_sc1(flat_rsrc(a.z_rest, (int64_t)a.T * a.ldz * 2), at, rest);
    }
    stores_done();
    if (wave_id() != 0)
        return;
    const int arm = item % DECODE_ARMS;   // additions to one address take 12 ns each
    if (last_at(counter(a, DECODE_Z + arm), (items - arm + DECODE_ARMS - 1) / DECODE_ARMS) &&
        last_at(counter(a, DECODE_Z + DECODE_ARMS), min(items, DECODE_ARMS)))
        set_flag(a, DECODE_Z_DONE, 0u);
}

// 16 channels of the shared experts.
template <bool HELP>
__device__ __forceinline__ void shared_item(const DecodeArgs &a, int item, uint32_t *lds, uint32_t *sh)
{
    if (!front_product<2, HELP>(a, a.w_shared, a.n_shared_rows, (int)(a.shared_at / 16) + 2 * item, lds, sh))
        return;
    const int t = threadIdx.x, row = t / 8, c = t % 8 * 2;
    if (row < a.T) {
        const float *red = reinterpret_cast<const float *>(lds) + row * 16 + c;
        float v[2];
#pragma unroll
        for (int i = 0; i < 2; i++)
            v[i] = silu_f32(total<REST_WAVES>(red, 512, i)) * total<REST_WAVES>(red, 512, 256 + i);
        uint32_t high, rest;
        split(v[0], v[1], high, rest);
        const int at = (row * a.ldz + a.Lt + item * 16 + c) * 2;
        store4_sc1(flat_rsrc(a.z, (int64_t)a.T * a.ldz * 2), at, high);
        store4_sc1(flat_rsrc(a.z_rest, (int64_t)a.T * a.ldz * 2), at, rest);
    }
    arrive_out(a);
}

// select_best of select.hpp in little code, for token t, from its logits' parts in memory. No key of an expert is 0, which stands for none (only a NaN with every bit set
// would have it), so that ids are always in range. `go` = 0: keys that are all different in place of the logits.
__device__ __forceinline__ void select_short(const DecodeArgs &a, int t, int go, uint32_t *words, uint64_t *scratch, int *id, float *weight)
{
    constexpr int QUADS = DECODE_MAX_E / (4 * WAVE);
    const int lane = lane_id(), E = a.E, K = a.K;
    const auto bias = window(a.bias, (int64_t)E * 4, a.bias != nullptr), logits = window(a.logits_out + (int64_t)t * E, (int64_t)E * 4, go && a.logits_out);
    u32x4_t raw[QUADS][ROUTER_PARTS + 1];
#pragma unroll
    for (int p = 0; p < ROUTER_PARTS; p++) {
        const auto row = window(a.logits + ((int64_t)p * a.T + t) * E, (int64_t)E * 4, go);
#pragma unroll
        for (int q = 0; q < QUADS; q++)
            raw[q][p] = fetch16<CPOL_SC1>(row, (q * WAVE + lane) * 16);
    }
#pragma unroll
    for (int q = 0; q < QUADS; q++)
        raw[q][ROUTER_PARTS] = fetch16<0>(bias, (q * WAVE + lane) * 16);
    uint32_t keys[QUADS * 4], top = 0u;
#pragma unroll
    for (int q = 0; q < QUADS; q++) {
        u32x4_t sum;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            float v = __uint_as_float(raw[q][0][j]);
#pragma unroll
            for (int p = 1; p < ROUTER_PARTS; p++)
                v += __uint_as_float(raw[q][p][j]);
            v = a.bias ? v + __uint_as_float(raw[q][ROUTER_PARTS][j]) : v;
            sum[j] = __float_as_uint(v);
            const int e = (q * WAVE + lane) * 4 + j;
            const uint32_t key = e < E ? go ? max(order_key(v), 1u) : 1u + e : 0u;
            keys[q * 4 + j] = key;
            top = max(top, key);
        }
#pragma unroll
        for (int j = 0; j < 4; j++)
            __builtin_amdgcn_raw_buffer_store_b32((int)sum[j], logits, (q * WAVE + lane) * 16 + j * 4, 0, 0);
    }
    // K lanes hold a key of at least `bound`, so the best K keys are among those
    uint32_t bound = 0u;
    int held = WAVE;
#pragma unroll 1
    for (uint32_t bit = 1u << 31; bit && held != K; bit >>= 1) {
        const int n = (int)__popcll(__ballot(top >= (bound | bit)));
        if (n >= K) {
            bound |= bit;
            held = n;
        }
    }
    int total = 0;
#pragma unroll
    for (int i = 0; i < QUADS * 4; i++) {
        const bool in = keys[i] != 0u && keys[i] >= bound;
        const uint64_t all = __ballot(in);
        const int at = total + (int)__popcll(all & ((1ull << lane) - 1));
        if (in && at < WAVE)
            scratch[at] = ((uint64_t)keys[i] << 32) | (uint32_t)~(uint32_t)((i / 4 * WAVE + lane) * 4 + i % 4);
        total += (int)__popcll(all);
    }
    uint64_t mine = 0;
    meet_lanes();
    if (total <= WAVE) {
        mine = lane < total ? scratch[lane] : 0;
        int rank = 0;
#pragma unroll 2
        for (int m = 0; m < total; m++) {
            const uint64_t other = ((uint64_t)__builtin_amdgcn_readlane((int)(mine >> 32), m) << 32) |
                                   (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)mine, m);
            rank += other > mine;
        }
        meet_lanes();
        if (lane < total && rank < K)
            scratch[rank] = mine;
        meet_lanes();
        mine = lane < K ? scratch[lane] : 0;
    } else {   // heavy ties: one maximum after another
#pragma unroll
        for (int i = 0; i < QUADS * 4; i++)
            words[(i / 4 * WAVE + lane) * 4 + i % 4] = keys[i];
        meet_lanes();
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

// The top-K of four tokens, one to a wave; the last of these items to arrive makes the list: the distinct experts in ascending
// order, and for each the pairs of its tokens.
template <bool HELP>
__device__ __forceinline__ bool top_item(const DecodeArgs &a, int item, int items, uint32_t *words, uint32_t *sh)
{
    const int lane = lane_id(), wv = wave_id();
    const int T = a.T, K = a.K, E = a.E, P = T * K;
    constexpr int NTHR = WAVE * REST_WAVES;
    // whether any token chose an expert, then its place in the list; the experts of the pairs; then the waves' keys, and
    // after them the list's pairs, two to a word
    int *ranks = reinterpret_cast<int *>(words), *chosen = ranks + DECODE_MAX_E, *scan = chosen + ROWS * 32;
    uint32_t *table = words + DECODE_MAX_E + ROWS * 32 + 16, *mine = table + wv * DECODE_MAX_E;
    uint64_t *scratch = reinterpret_cast<uint64_t *>(table + REST_WAVES * DECODE_MAX_E) + wv * WAVE;
    const int t = item * REST_WAVES + wv;
#pragma unroll 1
    for (int go = HELP ? 1 : 0; go < 2; go++) {
        if (go && wait_for<HELP>(a, counter(a, DECODE_ROUTER), (uint32_t)(a.n_router_rows / 16 * ROUTER_PARTS), sh) < 0)
            return false;
        const auto weights = window(a.weights, (int64_t)P * 4, go), all = window(a.chosen, (int64_t)P * 4, go);
        for (int p = threadIdx.x; p < P; p += NTHR)
            chosen[p] = 0;
        for (int i = threadIdx.x; i < E; i += NTHR)
            ranks[i] = 0;
        __syncthreads();
        if (t < T) {
            int id;
            float w;
            select_short(a, t, go, mine, scratch, &id, &w);
            if (lane < K) {
                const int p = t * K + lane;
                chosen[p] = id;
                store4_sc1(weights, p * 4, __float_as_uint(w));
                store4_sc1(all, items > 1 ? p * 4 : OUTSIDE, (uint32_t)id);
                if (go && a.ids_out)
                    a.ids_out[p] = id;
                if (go && a.weights_out)
                    a.weights_out[p] = w;
            }
        }
        if (go && items > 1) {
            stores_done();
            if (wv == 0) {
                const bool last = last_at(counter(a, DECODE_TOP), items);
                if (lane == 0)
                    *sh = last;
            }
            __syncthreads();
            const bool last = *sh != 0u;
            __syncthreads();
            if (!last)
                return true;
            for (int p = threadIdx.x; p < P; p += NTHR)
                chosen[p] = min((int)load4_sc1(all, p * 4), E - 1);
        }
        __syncthreads();
        for (int p = threadIdx.x; p < P; p += NTHR)
            ranks[chosen[p]] = 1;
        const auto list = window(a.list, (int64_t)a.most * 4, go), pairs = window(a.pairs, (int64_t)a.most * ROWS * 2, go);
        for (int i = threadIdx.x; i < a.most * (ROWS / 2); i += NTHR)
            table[i] = ~0u;
        __syncthreads();
        const int per = (E + NTHR - 1) / NTHR, e0 = (int)threadIdx.x * per, e1 = min(E, e0 + per);
        int n = 0, count;
        for (int e = e0; e < e1; e++)
            n += ranks[e];
        int rank = block_excl_scan(n, scan, &count);
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
        if (go && wv == 0)
            set_flag(a, DECODE_READY, (uint32_t)count);
    }
    return true;
}

// One MX block times a step's activations.
__device__ __forceinline__ f32x4_t mx_step(u32x4_t codes, uint32_t scales, const u32x4_t (&x)[4], f32x4_t acc)
{
#pragma unroll
    for (int j = 0; j < 4; j++)
        acc = mfma16(as_bf16x8(x[j]), mx_dequant8(codes[j], e8m0_to_f32((scales >> (8 * j)) & 0xFFu)), acc);
    return acc;
}
// N of them times one operand or two, a sum each.
template <int PARTS, int N>
__device__ __forceinline__ void mx_steps(const u32x4_t (&codes)[N], const uint32_t (&scales)[N], const uint32_t *rows, int second,
                                         f32x4_t (&acc)[PARTS][N])
{
    u32x4_t x[PARTS][4];
#pragma unroll
    for (int p = 0; p < PARTS; p++)
#pragma unroll
        for (int i = 0; i < 4; i++)
            x[p][i] = *reinterpret_cast<const u32x4_t *>(rows + p * second + i * 16);
#pragma unroll
    for (int j = 0; j < N; j++) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const auto w = mx_dequant8(codes[j][i], e8m0_to_f32((scales[j] >> (8 * i)) & 0xFFu));
#pragma unroll
            for (int p = 0; p < PARTS; p++)
                acc[p][j] = mfma16(as_bf16x8(x[p][i]), w, acc[p][j]);
        }
        if (PARTS == 2 && N > 2)
            __builtin_amdgcn_sched_barrier(0);   // no more weights at a time than there are registers for
    }
}

// The experts' gate and up product with one token: a pair of 16 gate and 16 up channels per workgroup, whose waves share the
// K axis; each wave's part of z (and of its remainders, row 8 of the operand) goes through LDS. The first weights are asked
// for before z is there.
template <bool HELP>
__device__ __forceinline__ bool gate_one(const DecodeArgs &a, int item, const Seen &seen, uint32_t *lds, uint32_t *sh)
{
    const int lane = lane_id(), wv = wave_id(), t = threadIdx.x;
    const int pairs16 = a.I / 16, r = item / pairs16, cp = item % pairs16;
    const int steps = a.Lt / MX_STEP, s0 = steps * wv / REST_WAVES, n = steps * (wv + 1) / REST_WAVES - s0;
    constexpr int BATCH = 7;   // steps in flight
    uint32_t *stage = lds + wv * STAGE_WORDS;
    float *red = reinterpret_cast<float *>(lds + REST_WAVES * STAGE_WORDS);
    const int pitch = n * MX_STEP / 2 + 4, chunks = n * 16;   // words of a staged row; 16-byte pieces
    const uint32_t *staged = stage + (lane & 8 ? pitch : 0) + (lane >> 4) * 4;   // sums of rows 1 .. 7, 9 .. 15 are not used
    const auto h = flat_rsrc(a.h, (int64_t)a.K * a.I * 4);
#pragma unroll 1
    for (int go = 1 - seen.first_pass; go < 2; go++) {
        int e = 0, pair = 0;
        if (go) {
            const int experts = wait_ready<HELP>(a, seen, sh);
            if (r >= experts)
                return experts >= 0;
            e = __builtin_amdgcn_readfirstlane((int)load4_sc1(flat_rsrc(a.list, (int64_t)a.most * 4), r * 4));
            pair = (int)(load4_sc1(flat_rsrc(a.pairs, (int64_t)a.most * ROWS * 2), r * ROWS * 2) & 0xFFFFu);
        }
        const auto w = window(a.gateup + e * a.gateup_stride + (int64_t)2 * cp * steps * MX_BLOCK_BYTES,
                              2 * (int64_t)steps * MX_BLOCK_BYTES, go);
        u32x4_t codes[BATCH][2];
        uint32_t scales[BATCH][2];
        auto load = [&](int slot, int s) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int off = s < n ? (j * steps + s0 + s) * MX_BLOCK_BYTES : OUTSIDE;
                codes[slot][j] = fetch16<CPOL_NT>(w, off + lane * 16);
                scales[slot][j] = fetch4<CPOL_NT>(w, off + MX_CODE_BYTES + 4 * (lane & 15));
            }
        };
#pragma unroll
        for (int i = 0; i < BATCH; i++)
            load(i, i);
        asm volatile("" ::: "memory");
        if (go && !wait_z<HELP>(a, seen, sh))
            return false;
        const auto z0 = window(a.z, (int64_t)a.Lt * 2, go), z1 = window(a.has_latent ? a.z_rest : a.z, (int64_t)a.Lt * 2, go);
#pragma unroll 1
        for (int j = lane; j < chunks; j += 2 * WAVE) {
            const int off = (s0 * MX_STEP + j * 8) * 2, off2 = j + WAVE < chunks ? off + WAVE * 16 : OUTSIDE;
            uint32_t *to = stage + j * 4;
            const u32x4_t v0 = fetch16<CPOL_SC1>(z0, off), v1 = fetch16<CPOL_SC1>(z0, off2);
            const u32x4_t v2 = fetch16<CPOL_SC1>(z1, off), v3 = fetch16<CPOL_SC1>(z1, off2);
            *reinterpret_cast<u32x4_t *>(to) = v0;
            *reinterpret_cast<u32x4_t *>(to + pitch) = v2;
            if (j + WAVE < chunks) {
                *reinterpret_cast<u32x4_t *>(to + WAVE * 4) = v1;
                *reinterpret_cast<u32x4_t *>(to + WAVE * 4 + pitch) = v3;
            }
        }
        meet_lanes();
        f32x4_t acc[2] = {};
#pragma unroll 1
        for (int s = 0; s < n; s += BATCH)
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
                load(i, s + i + BATCH);
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
            uint32_t high, rest;
            split(silu_f32(v[0][0]) * v[1][0], silu_f32(v[0][1]) * v[1][1], high, rest);
            store4_sc1(h, go ? (pair * a.I + cp * 16 + 2 * t) * 2 : OUTSIDE, high);
            store4_sc1(h, go ? ((a.K + pair) * a.I + cp * 16 + 2 * t) * 2 : OUTSIDE, rest);
        }
    }
    arrive(decode_gates(a, r));
    return true;
}

// ... with several: four such pairs per workgroup, one to a wave, each over all of K, so that z goes through LDS once for
// them all, a chunk of STEPS steps at a time, each loaded a chunk ahead; weights come AHEAD steps ahead. Up to 8 tokens: one operand, whose rows
// 8 .. 15 are the remainders of rows 0 .. 7; more: two operands (PARTS). K is summed in four quarters, as above, so that a
// token's h is the same bits whatever tokens come with it.
template <int PARTS, bool HELP>
__device__ __forceinline__ bool gate_many(const DecodeArgs &a, int item, const Seen &seen, uint32_t *lds, uint32_t *sh)
{
    constexpr int AHEAD = 4, STEPS = AHEAD / PARTS, PITCH = STEPS * MX_STEP / 2 + 4, NTHR = WAVE * REST_WAVES;   // words of a row in LDS
    constexpr int PIECES = STEPS * 16 * 16 * PARTS / NTHR;   // 16-byte pieces of a chunk per thread
    static_assert(2 * ROWS * PARTS * PITCH <= LDS_WORDS, "room for two chunks");
    const int lane = lane_id(), wv = wave_id(), t = threadIdx.x;
    const int groups = a.I / 16 / REST_WAVES, r = item / groups, cp = item % groups * REST_WAVES + wv;
    const int steps = a.Lt / MX_STEP;
    // piece i of this thread: 8 values of row i (t / 16 ..): a token's z, or HALF or ROWS rows further its remainders.
    // Rows past the tokens are zeros, and everything in the first pass.
    int z_there = 0;
    const auto z0 = flat_rsrc(a.z, (int64_t)a.T * a.ldz * 2), z1 = flat_rsrc(a.has_latent ? a.z_rest : a.z, (int64_t)a.T * a.ldz * 2);
    u32x4_t zs[PIECES];
    auto fetch = [&](int s) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < PIECES; i++) {
            const int p = i * NTHR + t, row = p / (STEPS * 16), c = p % (STEPS * 16);
            const int token = row % (PARTS == 1 ? HALF : ROWS), k = s * MX_STEP + c * 8;
            zs[i] = fetch16<CPOL_SC1>(row >= (PARTS == 1 ? HALF : ROWS) ? z1 : z0, z_there && k < a.Lt && token < a.T ? (token * a.ldz + k) * 2 : OUTSIDE);
        }
    };
#pragma unroll 1
    for (int go = 1 - seen.first_pass; go < 2; go++) {
        int e = 0;
        uint32_t pair01 = ~0u, pair23 = ~0u;   // the pairs of this lane's rows 4 (l / 16) .. +3
        if (go) {
            const int experts = wait_ready<HELP>(a, seen, sh);
            if (r >= experts)
                return experts >= 0;
            e = __builtin_amdgcn_readfirstlane((int)load4_sc1(flat_rsrc(a.list, (int64_t)a.most * 4), r * 4));
            const auto pairs = flat_rsrc(a.pairs, (int64_t)a.most * ROWS * 2);
            pair01 = load4_sc1(pairs, (r * ROWS + 4 * (lane >> 4)) * 2);
            pair23 = load4_sc1(pairs, (r * ROWS + 4 * (lane >> 4)) * 2 + 4);
        }
        const auto w = window(a.gateup + e * a.gateup_stride + (int64_t)2 * cp * steps * MX_BLOCK_BYTES,
                              2 * (int64_t)steps * MX_BLOCK_BYTES, go);
        u32x4_t codes[AHEAD][2];
        uint32_t scales[AHEAD][2];
        auto load = [&](int slot, int s) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int off = s < steps ? (j * steps + s) * MX_BLOCK_BYTES : OUTSIDE;
                codes[slot][j] = fetch16<CPOL_NT>(w, off + lane * 16);
                scales[slot][j] = fetch4<CPOL_NT>(w, off + MX_CODE_BYTES + 4 * (lane & 15));
            }
        };
#pragma unroll
        for (int i = 0; i < AHEAD; i++)
            load(i, i);
        asm volatile("" ::: "memory");
        if (go && !wait_z<HELP>(a, seen, sh))
            return false;
        z_there = go;
        fetch(0);
        f32x4_t acc[PARTS][2] = {}, sum[2] = {};
        int quarter = 1;   // ends at this many fourths of the steps; with fewer than four, some are empty
        while (steps * quarter / REST_WAVES == 0)
            quarter++;
        int half = 0;   // which half of LDS: a wave that writes it has seen every wave past the chunk before the last
#pragma unroll 1
        for (int s = 0; s < (go ? steps : 1); s += AHEAD)
#pragma unroll
            for (int c = 0; c < PARTS; c++, half ^= 1) {
                uint32_t *chunk = lds + half * ROWS * PARTS * PITCH;
                const uint32_t *mine = chunk + (lane & 15) * PITCH + (lane >> 4) * 4;
#pragma unroll
                for (int i = 0; i < PIECES; i++) {
                    const int p = i * NTHR + t;
                    *reinterpret_cast<u32x4_t *>(chunk + p / (STEPS * 16) * PITCH + p % (STEPS * 16) * 4) = zs[i];
                }
                fetch(s + (c + 1) * STEPS);
                __syncthreads();
#pragma unroll
                for (int i = 0; i < STEPS; i++) {   // steps past the end multiply zeros
                    const int slot = c * STEPS + i;
                    mx_steps<PARTS>(codes[slot], scales[slot], mine + i * (MX_STEP / 2), ROWS * PITCH, acc);
                    if (s + slot + 1 == steps * quarter / REST_WAVES) {
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
                        while (steps * quarter / REST_WAVES == s + slot + 1)
                            quarter++;
                    }
                    __builtin_amdgcn_sched_barrier(0);
                    load(slot, s + slot + AHEAD);
                }
            }
        // two channels to a word; rows of the upper half of the lanes are remainders where PARTS = 1
        const int P = a.T * a.K;
        const auto h = flat_rsrc(a.h, (int64_t)P * a.I * 4);
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const float v = silu_f32(sum[0][k]) * sum[1][k], after = __shfl_down(v, 1);
            const int pair = (int16_t)((k < 2 ? pair01 : pair23) >> (16 * (k % 2))), token = 4 * (lane >> 4) + k;
            const bool keep = go && pair >= 0 && token < a.T && lane % 2 == 0;
            uint32_t high, rest;
            split(v, after, high, rest);
            store4_sc1(h, keep ? (pair * a.I + cp * 16 + (lane & 15)) * 2 : OUTSIDE, high);
            store4_sc1(h, keep ? ((P + pair) * a.I + cp * 16 + (lane & 15)) * 2 : OUTSIDE, rest);
        }
        __syncthreads();   // LDS is free for the next pass
    }
    arrive(decode_gates(a, r));
    return true;
}

// decode_down_span times 256 latent columns of one expert's down product, 64 of 256 to a wave: y of its tokens' pairs, to
// memory. The weights come in units of STEPS steps, a unit ahead, the first before h is known, which takes that expert's
// gate items only. h and its remainders go through LDS, STEPS steps at a time (once for all columns, if those are all): one
// operand for up to 8 tokens, two for more (PARTS). Each column of a pair is two chains of sums over K, h's and the
// remainders', the same whatever tokens come with it.
template <int PARTS, bool HELP>
__device__ __forceinline__ bool down_item(const DecodeArgs &a, int item, const Seen &seen, uint32_t *lds, uint32_t *sh)
{
    constexpr int STEPS = 3, NB = DECODE_DOWN_COLUMNS / (16 * REST_WAVES), NTHR = WAVE * REST_WAVES;
    constexpr int PITCH = STEPS * MX_STEP / 2 + 4, PER_ROW = STEPS * MX_STEP / 8, TOKENS = PARTS == 1 ? HALF : ROWS;
    constexpr int PIECES = 2 * TOKENS * PER_ROW / NTHR;
    static_assert(2 * ROWS * PITCH + ROWS / 2 <= LDS_WORDS && PIECES * NTHR == 2 * TOKENS * PER_ROW, "room; pieces");
    const int lane = lane_id(), t = threadIdx.x, span = decode_down_span(a), per = decode_down_items(a), r = item / per, g0 = item % per * span;
    const int groups = min(span, decode_groups(a) - g0), steps = a.I / MX_STEP, P = a.T * a.K, blocks = a.Lt / 16;
#pragma unroll 1
    for (int go = 1 - seen.first_pass; go < 2; go++) {
        int e = 0, from[PIECES];   // this thread's pieces of h and the remainders: the row and the column, in bytes
#pragma unroll
        for (int i = 0; i < PIECES; i++)
            from[i] = OUTSIDE;
        uint32_t arrived = 0u;
        if (go) {
            const int experts = wait_ready<HELP>(a, seen, sh);
            if (r >= experts)
                return experts >= 0;
            const auto pairs = flat_rsrc(a.pairs, (int64_t)a.most * ROWS * 2);
#pragma unroll
            for (int i = 0; i < PIECES; i++)
                from[i] = (int)load4_sc1(pairs, (r * ROWS + (i * NTHR + t) / PER_ROW % TOKENS / 2 * 2) * 2);
            const uint32_t two = load4_sc1(pairs, (r * ROWS + t % (ROWS / 2) * 2) * 2);
            e = __builtin_amdgcn_readfirstlane((int)load4_sc1(flat_rsrc(a.list, (int64_t)a.most * 4), r * 4));
            arrived = ask(decode_gates(a, r));
            if (t < ROWS / 2)
                lds[2 * ROWS * PITCH + t] = two;
#pragma unroll
            for (int i = 0; i < PIECES; i++) {
                const int pair = (int16_t)((i * NTHR + t) / PER_ROW % 2 ? from[i] >> 16 : from[i]);
                from[i] = pair >= 0 ? ((pair + (i * NTHR + t) / PER_ROW / TOKENS * P) * a.I + (i * NTHR + t) % PER_ROW * 8) * 2 : OUTSIDE;
            }
        }
        const int n = go ? steps : 1, units = go ? groups * ((steps + STEPS - 1) / STEPS) : 1;
        const auto w = window(a.down + e * a.down_stride, (int64_t)blocks * steps * MX_BLOCK_BYTES, go);
        const auto h = window(a.h, (int64_t)P * a.I * 4, go), y = window(a.partial, (int64_t)P * a.Lt * 4, go);
        u32x4_t codes[STEPS][NB], hs[PIECES];
        uint32_t scales[STEPS][NB];
        auto load = [&](int slot, int col, int s) __attribute__((always_inline)) {
#pragma unroll
            for (int j = 0; j < NB; j++) {
                const int off = s < n && col + j < blocks ? ((col + j) * steps + s) * MX_BLOCK_BYTES : OUTSIDE;
                codes[slot][j] = fetch16<CPOL_NT>(w, off + lane * 16);
                scales[slot][j] = fetch4<CPOL_NT>(w, off + MX_CODE_BYTES + 4 * (lane & 15));
            }
        };
        auto fetch = [&](int s) __attribute__((always_inline)) {   // zeros past the row's end
#pragma unroll
            for (int i = 0; i < PIECES; i++)
                hs[i] = fetch16<CPOL_SC1>(h, from[i] != OUTSIDE && s * MX_STEP + (i * NTHR + t) % PER_ROW * 8 < n * MX_STEP
                                                 ? from[i] + s * MX_STEP * 2 : OUTSIDE);
        };
        int col = (g0 * REST_WAVES + wave_id()) * NB, s = 0;   // the unit's first column block and step
#pragma unroll
        for (int i = 0; i < STEPS; i++)
            load(i, col, i);
        asm volatile("" ::: "memory");
        if (go && wait_for<HELP>(a, decode_gates(a, r), (uint32_t)decode_gate_items(a), sh, arrived) < 0)
            return false;
        f32x4_t acc[PARTS][NB] = {};
        const uint32_t *mine = lds + (lane & 15) * PITCH + (lane >> 4) * 4;
#pragma unroll 1
        for (int u = 0; u < units; u++) {
            if (u == 0 || n > STEPS) {   // another part of h
                fetch(s);
                __syncthreads();
#pragma unroll
                for (int i = 0; i < PIECES; i++)
                    *reinterpret_cast<u32x4_t *>(lds + (i * NTHR + t) / PER_ROW * PITCH + (i * NTHR + t) % PER_ROW * 4) = hs[i];
                __syncthreads();
            }
            const bool end = s + STEPS >= n;   // of these columns
            const int next = u + 1 == units ? blocks : end ? col + NB * REST_WAVES : col, next_s = end ? 0 : s + STEPS;
#pragma unroll
            for (int i = 0; i < STEPS; i++) {   // steps past the end multiply zeros
                mx_steps<PARTS>(codes[i], scales[i], mine + i * (MX_STEP / 2), ROWS * PITCH, acc);
                __builtin_amdgcn_sched_barrier(0);
                load(i, next, next_s + i);
            }
            if (end) {
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const int pair = reinterpret_cast<const int16_t *>(lds + 2 * ROWS * PITCH)[4 * (lane >> 4) + k];
#pragma unroll
                    for (int j = 0; j < NB; j++) {
                        const float rest = PARTS == 1 ? __shfl_xor(acc[0][j][k], 32) : acc[PARTS - 1][j][k];
                        store4_sc1(y, go && pair >= 0 && pair < P && col + j < blocks ? (pair * a.Lt + (col + j) * 16 + (lane & 15)) * 4 : OUTSIDE,
                                   __float_as_uint(acc[0][j][k] + rest));
                    }
                }
#pragma unroll
                for (int p = 0; p < PARTS; p++)
#pragma unroll
                    for (int j = 0; j < NB; j++)
                        acc[p][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            }
            col = next;
            s = next_s;
        }
        __syncthreads();   // LDS is free for the next pass
    }
    stores_done();
    if (t < groups)
        __hip_atomic_fetch_add(decode_columns(a, g0 + t), 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return true;
}

// The weighted sum of the experts' y, in slot order: 256 latent columns of four tokens.
template <bool HELP>
__device__ __forceinline__ bool sum_item(const DecodeArgs &a, int item, const Seen &seen, uint32_t *sh)
{
    constexpr int SLOTS = 8;   // loaded at a time
    const int groups = decode_groups(a), g = item % groups, K = a.K, P = a.T * K;
    const int token = item / groups * 4 + wave_id(), col = g * DECODE_DOWN_COLUMNS + lane_id() * 4;
    const bool live = token < a.T && col < a.Lt;
#pragma unroll 1
    for (int go = HELP ? 1 : 0; go < 2; go++) {
        if (go) {
            const int experts = wait_ready<HELP>(a, seen, sh);
            if (experts < 0 || wait_for<HELP>(a, decode_columns(a, g), (uint32_t)experts, sh) < 0)
                return false;
        }
        const auto weights = window(a.weights, (int64_t)P * 4, go), y = window(a.partial, (int64_t)P * a.Lt * 4, go);
        f32x4_t v = {};
#pragma unroll 1
        for (int j0 = 0; j0 < K; j0 += SLOTS) {   // slots past the last are skipped, not added: y may hold anything
            u32x4_t ys[SLOTS];
            float w[SLOTS];
#pragma unroll
            for (int j = 0; j < SLOTS; j++) {
                const int pair = token * K + j0 + j;
                const bool in = live && j0 + j < K;
                w[j] = __uint_as_float(fetch4<CPOL_SC1>(weights, in ? pair * 4 : OUTSIDE));
                ys[j] = fetch16<CPOL_SC1>(y, in ? (pair * a.Lt + col) * 4 : OUTSIDE);
            }
#pragma unroll
            for (int j = 0; j < SLOTS; j++)
#pragma unroll
                for (int i = 0; i < 4; i++)
                    v[i] = j0 + j < K ? fmaf(w[j], __uint_as_float(ys[j][i]), v[i]) : v[i];
        }
        // zc in the place of z, which every listed expert has been multiplied with: all their down items are done
        const auto to = window(a.has_latent ? a.z : a.out, (int64_t)a.T * a.ldz * 2, go);
        const auto left = window(a.z_rest, (int64_t)a.T * a.ldz * 2, go && a.has_latent);
        const int at = live ? (token * a.ldz + col) * 2 : OUTSIDE;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            uint32_t high, rest;
            split(v[2 * i], v[2 * i + 1], high, rest);
            store4_sc1(to, at + 4 * i, high);
            store4_sc1(left, at + 4 * i, rest);
        }
    }
    if (a.has_latent)
        arrive_out(a);
    return true;
}

template <bool FEW, bool HELP>
__device__ __forceinline__ bool out_item(const DecodeArgs &a, int item, uint32_t *lds, uint32_t *sh)
{
    const int wv = wave_id(), t = threadIdx.x, row = t / 8, c = t % 8 * 2, cat = a.ldz;
    float *red = reinterpret_cast<float *>(lds);
    const auto out = flat_rsrc(a.out, (int64_t)a.T * a.H * 2);
    auto run = [&](auto part) __attribute__((always_inline)) {
        using Part = decltype(part);
#pragma unroll 1
        for (int go = !HELP && a.T <= 2 ? 0 : 1; go < 2; go++) {   // of more tokens it delays the weights (4: 84 us, 81 without)
            part.start(a.w_out, a.H, cat, item, wv, REST_WAVES, go);
            if (go && wait_for<HELP>(a, flag(a, DECODE_CAT_DONE, blockIdx.x % FLAGS), 1u, sh) < 0)
                return false;
            const auto high = window(a.z, (int64_t)a.T * cat * 2, go), rest = window(a.z_rest, (int64_t)a.T * cat * 2, go);
            f32x4_t acc[Part::OPERANDS][1] = {};
            part.finish(a.T, lds + wv * OUT_STAGE_WORDS, acc, [&](int r, int k, bool in, int i) __attribute__((always_inline)) {
                return fetch16<CPOL_SC1>(i ? rest : high, in ? (r * cat + k) * 2 : OUTSIDE);
            });
            __syncthreads();   // the sums take the place of the activations
            store_sums(red + wv * 256, FEW ? acc[0][0] : acc[0][0] + acc[Part::OPERANDS - 1][0]);
            __syncthreads();
            if (row < a.T && row < ROWS) {
                float v[2] = {0.f, 0.f};
#pragma unroll
                for (int w = 0; w < REST_WAVES; w++)
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const float *p = red + w * 256 + row * 16 + c + i;
                        v[i] += FEW ? p[0] + p[HALF * 16] : p[0];
                    }
                __builtin_amdgcn_raw_buffer_store_b32((int)pack_bf16x2(v[0], v[1]), out, go ? (row * a.H + item * 16 + c) * 2 : OUTSIDE, 0, 0);
            }
            __syncthreads();
        }
        return true;
    };
    if constexpr (FEW) {
        if (using Staged = Bf16Part<1, 16, 0, 1>; Staged::fits(a.T, cat, REST_WAVES))
            return run(Staged());
        return run(Bf16Part<1, 12, 6, 1>());
    } else {
        return run(Bf16Part<1, 12, 6, 2>());
    }
}

// The kernel's arguments, read from memory again: they do not fit the scalar registers all at once.
__device__ __forceinline__ const DecodeArgs &arguments()
{
    auto *at = (const __attribute__((address_space(4))) DecodeArgs *)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(at));
    return *(const DecodeArgs *)at;
}

// Item i, as numbered by decode_items. False when patience ran out before anything was handed on (HELP: never).
template <bool FEW, bool HELP>
__device__ __forceinline__ bool do_item(const DecodeItems &n, int i, const Seen &seen, uint32_t *lds, uint32_t *sh)
{
    if (i < n.router) {
        router_item<HELP>(arguments(), i, lds, sh);
        return true;
    }
    i -= n.router;
    if (i < n.latent) {
        latent_item<HELP>(arguments(), i, n.latent, lds, sh);
        return true;
    }
    i -= n.latent;
    if (i < n.top)
        return top_item<HELP>(arguments(), i, n.top, lds, sh);
    i -= n.top;
    if (i < n.gate) {
        if constexpr (FEW)
            if (decode_gate_one(arguments()))
                return gate_one<HELP>(arguments(), i, seen, lds, sh);
        return gate_many<FEW ? 1 : 2, HELP>(arguments(), i, seen, lds, sh);
    }
    i -= n.gate;
    if (i < n.shared) {
        shared_item<HELP>(arguments(), i, lds, sh);
        return true;
    }
    i -= n.shared;
    if (i < n.down)
        return down_item<FEW ? 1 : 2, HELP>(arguments(), i, seen, lds, sh);
    i -= n.down;
    if (i < n.sums)
        return sum_item<HELP>(arguments(), i, seen, sh);
    return out_item<FEW, HELP>(arguments(), i - n.sums, lds, sh);
}

template <bool FEW>
__global__ __launch_bounds__(WAVE *REST_WAVES, 3) void decode_kernel(const DecodeArgs a)
{
    constexpr int TOP = DECODE_MAX_E + ROWS * 32 + 16, MOST = ROWS * 32;   // MOST: pairs, and distinct experts
    static_assert(TOP % 2 == 0 && TOP + REST_WAVES * (DECODE_MAX_E + 2 * WAVE) <= LDS_WORDS && TOP + MOST * (ROWS / 2) <= LDS_WORDS, "room for the list");
    static_assert(REST_WAVES == 4 && STAGE_WORDS >= HALF * (14 * 16 + 4) && STAGE_WORDS >= ROWS * (7 * 16 + 4), "what the items assume");
    __shared__ alignas(16) uint32_t lds[LDS_WORDS];
    __shared__ uint32_t sh;
    const DecodeItems n = a.items;
    const int item = blockIdx.x;
    const bool late = item < n.router + n.latent ||   // claimed in front_product
                      (item >= n.router + n.latent + n.top + n.gate && item < n.router + n.latent + n.top + n.gate + n.shared);
    Seen seen{ask(flag(a, DECODE_READY, item % FLAGS)), ask(flag(a, DECODE_Z_DONE, item % FLAGS)), 0};   // come with the claim
    if (!late) {
        if (!claim<false>(a, item, &sh, seen.ready == 0u ? 2u : 0u))
            return;
        seen.first_pass = __builtin_amdgcn_readfirstlane((int)sh) >> 1;   // one wave's answer for all
        __syncthreads();
    }
    if (do_item<FEW, false>(n, item, seen, lds, &sh))
        return;
    int kind = 0;   // the first item of this one's kind
    for (const int size : {n.router, n.latent, n.top, n.gate, n.shared, n.down, n.sums})
        if (item >= kind + size)
            kind += size;
        else
            break;
#pragma unroll 1
    for (int i = 0; i <= kind; i++)   // the earlier kinds' items that are still free, and then this one
        if (i == kind || claim<true>(a, i, &sh))
            do_item<FEW, true>(n, i == kind ? item : i, Seen{0u, 0u, 0}, lds, &sh);
}

// Counters, flags and claims at zero.
__global__ __launch_bounds__(256) void clear_kernel(uint32_t *counters, int lines, uint32_t *claims, int items)
{
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i < lines)
        counters[i * DECODE_COUNTER_WORDS] = 0u;
    else if (i - lines < items)
        claims[i - lines] = 0u;
}

} // namespace

hipError_t launch_decode(const DecodeArgs &args, hipStream_t st)
{
    DecodeArgs a = args;
    a.items = decode_items(a);
    const int items = decode_item_count(a.items), lines = decode_counter_lines(a);
    hipLaunchKernelGGL(clear_kernel, dim3((unsigned)((items + lines + 255) / 256)), dim3(256), 0, st, a.counters, lines, a.claims, items);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    const dim3 grid((unsigned)items), threads(WAVE * REST_WAVES);
    if (a.T <= HALF)
        hipLaunchKernelGGL((decode_kernel<true>), grid, threads, 0, st, a);
    else
        hipLaunchKernelGGL((decode_kernel<false>), grid, threads, 0, st, a);
    return hipGetLastError();
}

} // namespace mxmoe
