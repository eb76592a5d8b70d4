// int8.hip -- dense products of 8-bit codes, out[t, n] = sx[t] sw[n] sum_k x[t, k] w[n, k] (+ bias), and
// their gated form silu(gate) * up, on the 16x16x64 8-bit matrix-core instruction.
//
// The sums are exact in 32-bit integers, so any split of K and any order of adding give the same
// bits; scales, bias and the gate are applied in FP32 in the epilogue. Weights are packed once
// (dense.hpp); activations are read as they are.
#include "dense.hpp"

#include <type_traits>
#include <utility>

namespace mxmoe {

namespace {

typedef int32_t acc_t __attribute__((ext_vector_type(4)));
constexpr int CUS = 256;
constexpr int XCDS = 8;      // workgroups are dealt to the XCDs round-robin by linear id
constexpr int GROUP_M = 4;   // row tiles per group, walked row-fastest

__device__ inline acc_t mfma(u32x4_t a, u32x4_t b, acc_t c)
{
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(acc_t, a), __builtin_bit_cast(acc_t, b), c, 0, 0,
                                                 0);
}

typedef __attribute__((address_space(3))) void *lds_ptr;

// Direct global -> LDS load of 16 bytes per lane: lane l's from byte `off` of the window [base, base +
// bytes) -- zeros when it lies outside -- to byte 16 l of `dst` (both wave-uniform but `off`).
template <int CPOL = 0>
__device__ inline void load_lds(const void *base, int bytes, int off, u32x4_t *dst)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, bytes, 0x00020000), (lds_ptr)dst, 16, off, 0,
        0, CPOL);
}

// v without its first n bytes (n >= 0), zeros at the end.
__device__ inline u32x4_t drop_bytes(u32x4_t v, int n)
{
    const unsigned __int128 x = __builtin_bit_cast(unsigned __int128, v);
    return __builtin_bit_cast(u32x4_t, n < 16 ? x >> (8 * n) : (unsigned __int128)0);
}

// Chunk c (16 codes) of row r of a staged activation tile (rows of I8_STAGE bytes) lies at chunk c ^ swizzle(r) of
// that row. The operand read (lane l: row l % 16, chunk c0 + l / 16, c0 even) then falls on distinct chunk
// places modulo 8, 16 and 32 in every group of 8, 16 and 32 consecutive lanes.
__host__ __device__ constexpr int swizzle(int r) { return (((r >> 2) ^ (r << 1 & 2)) & 3) << 1 | (r >> 1 & 1); }
constexpr bool swizzle_spreads(int lanes)
{
    for (int first = 0; first < 64; first += lanes)
        for (int a = first; a < first + lanes; a++)
            for (int b = a + 1; b < first + lanes; b++) {
                const int pa = a % 16 * 8 + (a / 16 ^ swizzle(a % 16)), pb = b % 16 * 8 + (b / 16 ^ swizzle(b % 16));
                if (pa % lanes == pb % lanes)
                    return false;
            }
    return true;
}
static_assert(swizzle_spreads(8) && swizzle_spreads(16) && swizzle_spreads(32), "bank conflicts");

// Linear workgroup id -> (column tile, row tile): each XCD takes a contiguous run of the items, which go
// in groups of GROUP_M row tiles, so that the workgroups sharing one L2 share operands. False past the end.
__device__ inline bool tile_item(int gx, int gy, int &bx, int &by)
{
    const int total = gx * gy, per = (total + XCDS - 1) / XCDS;
    const int slot = blockIdx.x / XCDS, item = (blockIdx.x % XCDS) * per + slot;
    if (slot >= per || item >= total)
        return false;
    const int first = item / (GROUP_M * gx) * GROUP_M;
    const int rows = min(gy - first, GROUP_M);
    const int in = item - first * gx;
    by = first + in % rows;
    bx = in / rows;
    return true;
}

// Four consecutive outputs of token row r from column n on.
__device__ inline void store4(const I8Args &g, int r, int n, const float *v)
{
    if (g.out_type == MOE_TYPE_F32) {
        float *o = static_cast<float *>(g.out) + r * g.ldo + n;
        if (n + 4 <= g.N)
            __builtin_memcpy(o, v, 16);
        else
#pragma unroll
            for (int i = 0; i < 4; i++)
                if (n + i < g.N)
                    o[i] = v[i];
    } else {
        uint16_t *o = static_cast<uint16_t *>(g.out) + r * g.ldo + n;
        const uint2 h{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        if (n + 4 <= g.N)
            __builtin_memcpy(o, &h, 8);
        else
#pragma unroll
            for (int i = 0; i < 4; i++)
                if (n + i < g.N)
                    o[i] = (uint16_t)((i < 2 ? h.x : h.y) >> (16 * (i % 2)));
    }
}

// Sixteen bytes of outputs of token row r from column n on.
__device__ inline void store16(const I8Args &g, int r, int n, u32x4_t v)
{
    if (g.out_type == MOE_TYPE_F32) {
        float *o = static_cast<float *>(g.out) + r * g.ldo + n;
        if (n + 4 <= g.N)
            __builtin_memcpy(o, &v, 16);
        else
#pragma unroll
            for (int i = 0; i < 4; i++)
                if (n + i < g.N)
                    o[i] = __uint_as_float(v[i]);
    } else {
        uint16_t *o = static_cast<uint16_t *>(g.out) + r * g.ldo + n;
        if (n + 8 <= g.N)
            __builtin_memcpy(o, &v, 16);
        else
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (n + i < g.N)
                    o[i] = (uint16_t)(v[i / 2] >> (16 * (i % 2)));
    }
}

// An output from its exact sum, and from those of gate and up. Every kernel computes them by these steps,
// each rounded to FP32 (no contraction), so that a token's outputs are the same bits in any batch.
__device__ inline float scaled(int32_t sum, float sx, float sw, float bias)
{
#pragma clang fp contract(off)
    return (float)sum * sx * sw + bias;
}
// g / (1 + exp(-g)) is taken on the hardware's exponential and reciprocal, each within a unit in the last
// place. The exponent's rounding costs |g| 2^-24 relative, beside the 2 |g| 2^-24 that g's own two roundings do: far
// below the output's BF16; in FP32 outputs up to 84 x 2^-24 for gates of -40 to -20, where FP32 with a library's exponential
// has 64, and 11.5 against 9 for gates of -5 to 5. exp overflows to infinity, whose reciprocal is 0.
__device__ inline float gated(int32_t gate, int32_t up, float sx, float sg, float su)
{
#pragma clang fp contract(off)
    const float g = (float)gate * sx * sg, u = (float)up * sx * su;
    return g * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * g)) * u;
}

// What one fragment's outputs take besides its sums: the token's scale, and for the lane's four columns their scales
// and the up columns' scales or the bias.
struct Factors {
    float sx;
    f32x4_t sw, other;
};

// The weights are the first matrix operand, so lane l of a fragment holds token row l % 16 and the packed
// columns 4 (l / 16) .. +3 of row block nb. Rows and blocks past the end take the last ones' factors.
__device__ inline Factors load_factors(const I8Args &g, int r, int nb)
{
    const int q = (threadIdx.x & (WAVE - 1)) >> 4, at = min(nb, g.nblk - (g.glu ? 2 : 1)) * 16 + 4 * q;
    const float *other = g.glu ? g.sw + 16 : g.bias ? g.bias : g.sw;
    Factors v{g.sx[min(r, g.T - 1)], *reinterpret_cast<const f32x4_t *>(g.sw + at),
              *reinterpret_cast<const f32x4_t *>(other + at)};
    if (!g.glu && !g.bias)
        v.other = f32x4_t{0.f, 0.f, 0.f, 0.f};
    return v;
}

// Outputs of one fragment of row block nb (a gate block with its up block's sums in `up` when glu).
__device__ inline void emit(const I8Args &g, int r, int nb, const Factors &c, acc_t sum, acc_t up)
{
    const int q = (threadIdx.x & (WAVE - 1)) >> 4, n = (g.glu ? nb / 2 : nb) * 16 + 4 * q;
    if (r >= g.T || n >= g.N)
        return;
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; i++)
        v[i] = g.glu ? gated(sum[i], up[i], c.sx, c.sw[i], c.other[i]) : scaled(sum[i], c.sx, c.sw[i], c.other[i]);
    store4(g, r, n, v);
}

// Sixteen bytes from byte `off` of the window [base, base + bytes), zeros when they lie outside.
template <int CPOL>
__device__ inline u32x4_t load_window(const void *base, int bytes, int off)
{
    return __builtin_amdgcn_raw_buffer_load_b128(
        __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, bytes, 0x00020000), off, 0, CPOL);
}

// f(0), f(1), ... with constants.
template <int... I, class F>
__device__ inline void each(std::integer_sequence<int, I...>, F f)
{
    (f(std::integral_constant<int, I>{}), ...);
}

// Tiles of 16 MF tokens x 16 NF NW packed columns by KG groups of NW waves; group k takes every KG-th stage of
// 128 codes, and the groups' sums are added through LDS at the end. A wave has all rows of the tile and columns
// of its own, so its weights go straight to registers, in the order they are packed in, and only the activations
// pass through LDS, loaded directly to it, 8 rows x 128 bytes (whole lines) with an instruction; rows past T lie
// outside the loads' window and read as zeros without touching memory. Loads run D - 1 stages ahead. With NW = 1 a
// wave reads only what it loaded itself, and no barrier is met before the one for the sums.
//
// Bounds: the weights' bytes from memory (1 x 28672 x 7168: 36.0 us, 5.7 TB/s), and for several row or column tiles
// the loads of a CU: 64 x 64 tiles take 64 + 64 bytes a code and CU, 65 GB/s of them (256 x 3584 x 7168: 19 us).
// Weights through LDS as well cost 128 more bytes of its traffic a code in those tiles: 777 x 1001 x 3584
// 11.1 us against 9.6, 1 x 3584 x 7168 7.3 against 6.9.
//
// ONCE: there is one row tile, so weights are read once, and are not to displace the activations in the caches.
// ANY: activations whose rows the direct loads cannot take (any address, any K >= 16) pass through
// registers on their way to LDS; rows past T, whose sums are never stored, repeat the last one -- or, in
// 16-token tiles, where they can be most, are not loaded (4 x 1792 x 12288: 8.8 us against 12.4) -- and the chunk that
// crosses K is loaded from 16 codes before K and shifted into place.
template <int MF, int NF, int NW, int KG, int D, bool ONCE, bool ANY>
__global__ __launch_bounds__(WAVE *NW *KG) __attribute__((amdgpu_waves_per_eu(NW * KG / 4)))
void tile_kernel(const I8Args g, int gx, int gy)
{
    constexpr int AL = 2 * MF / NW, LOADS = AL + 2 * NF;      // loads per wave and stage
    constexpr int STAGE = MF * 128;   // 16-byte slots of a stage's activations
    constexpr int SUMS = KG > 1 ? KG * NW * MF * NF * WAVE : 0;
    static_assert(AL * NW == 2 * MF && D >= 2 && (D - 1) * LOADS < 64, "tile");
    __shared__ u32x4_t lds[D * KG * STAGE > SUMS ? D * KG * STAGE : SUMS];
    const int lane = threadIdx.x & (WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int wv = wave % NW, kg = wave / NW;
    int bx, by;
    if (!tile_item(gx, gy, bx, by))
        return;
    const int m0 = by * 16 * MF, nb0 = bx * NF * NW + wv * NF;
    const int nst = (int)i8_stages(g.K);
    const int8_t *xt = g.x + (int64_t)m0 * g.ldx;
    const int xbytes = ANY ? 0 : (min(g.T - m0, 16 * MF) - 1) * (int)g.ldx + g.K;
    const uint8_t *wt = g.w + (int64_t)min(nb0, g.nblk - 1) * I8_STAGE_BYTES;
    const int wbytes = max(min(g.nblk - nb0, NF), 0) * I8_STAGE_BYTES;
    const int64_t wstep = (int64_t)g.nblk * I8_STAGE_BYTES;
    int64_t arow[AL];   // byte offsets of this lane's rows, and codes of its chunks in a stage
    int ak[AL];
#pragma unroll
    for (int i = 0; i < AL; i++) {
        const int row = (wv * AL + i) * 8 + (lane >> 3);
        arow[i] = !ANY || row < g.T - m0 ? row * g.ldx : MF == 1 ? -1 : (g.T - 1 - m0) * g.ldx;
        ak[i] = ((lane & 7) ^ swizzle(row)) * 16;
    }
    // Group k finishes every KG-th fragment (or pair of a gate and an up fragment); `row` and `col` are its i-th's place
    // in the tile. Their factors are loaded first of all, so that the end does not wait for them.
    constexpr int ENDS = (MF * NF + KG - 1) / KG;
    constexpr int PAIRS = NF / 2 + NF % 2;
    auto row = [&](int i) { return KG == 1 ? i / NF : g.glu ? (i * KG + kg) / PAIRS : (i * KG + kg) / NF; };
    auto col = [&](int i) { return KG == 1 ? i % NF : g.glu ? (i * KG + kg) % PAIRS * 2 : (i * KG + kg) % NF; };
    Factors factors[ENDS];
#pragma unroll
    for (int i = 0; i < ENDS; i++)
        factors[i] = load_factors(g, m0 + row(i) * 16 + (lane & 15), nb0 + col(i));
    struct Stage {
        u32x4_t b[2][NF], x[ANY ? AL : 1];
    } stage[D];
    u32x4_t *group = &lds[kg * STAGE];   // this group's part of a buffer
    auto load = [&](int it, int slot) {
        const int s = __builtin_amdgcn_readfirstlane(it * KG + kg), last = min(s, nst - 1);
        const int in = -(int)(s < nst);   // past K (another group's last): empty windows
        Stage &q = stage[slot];
        const uint8_t *ws = wt + last * wstep;
#pragma unroll
        for (int j = 0; j < NF; j++)
#pragma unroll
            for (int h = 0; h < 2; h++)
                q.b[h][j] = load_window<ONCE ? CPOL_NT : 0>(ws, wbytes & in, (j * 2 + h) * I8_BLOCK_BYTES + lane * 16);
#pragma unroll
        for (int i = 0; i < AL; i++) {
            if constexpr (ANY) {
                // past K: the last stage again, which is not used
                if (MF > 1 || arow[i] >= 0)
                    __builtin_memcpy(&q.x[i], xt + arow[i] + min(last * I8_STAGE + ak[i], g.K - 16), 16);
            } else {
                load_lds(xt + last * I8_STAGE, (xbytes - last * I8_STAGE) & in, (int)arow[i] + ak[i],
                         &group[slot * KG * STAGE + (wv * AL + i) * WAVE]);
            }
        }
        // The counts below are of loads in this order.
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    auto store_x = [&](int it, int slot) {
        const int s = it * KG + kg;
#pragma unroll
        for (int i = 0; i < AL; i++) {
            u32x4_t v = stage[slot].x[i];
            if ((s + 1) * I8_STAGE > g.K)   // the stage that crosses K
                v = drop_bytes(v, max(s * I8_STAGE + ak[i] - (g.K - 16), 0));
            group[slot * KG * STAGE + (wv * AL + i) * WAVE + lane] = v;
        }
    };
    acc_t acc[MF][NF];
#pragma unroll
    for (int f = 0; f < MF; f++)
#pragma unroll
        for (int j = 0; j < NF; j++)
            acc[f][j] = acc_t{0, 0, 0, 0};
    auto multiply = [&](int slot) {
        const u32x4_t *at = &group[slot * KG * STAGE];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            u32x4_t a[MF];
            const int r = lane & 15, c = (h * 4 + (lane >> 4)) ^ swizzle(r);
#pragma unroll
            for (int f = 0; f < MF; f++)
                a[f] = at[(f * 16 + r) * 8 + c];
#pragma unroll
            for (int j = 0; j < NF; j++)
#pragma unroll
                for (int f = 0; f < MF; f++)
                    acc[f][j] = mfma(stage[slot].b[h][j], a[f], acc[f][j]);
        }
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    // The activations of iteration `it` are in LDS: all but LATER stages' loads of this wave have landed. Its reads
    // of the iteration before are done; with NW > 1, past the barrier, so are every wave's.
    auto meet = [&](int it, int slot, auto later) {
        if constexpr (ANY)
            store_x(it, slot);
        __builtin_amdgcn_s_waitcnt(vmcnt_lgkm_imm(ANY ? 63 : later * LOADS));
        asm volatile("" ::: "memory");
        if constexpr (NW > 1) {
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    const int nit = NW > 1 ? (nst + KG - 1) / KG : (nst - kg + KG - 1) / KG;   // the same for waves that meet
    auto step = [&](int it, auto d) {
        if constexpr (NW == 1)
            load(it + D - 1, (d + D - 1) % D);
        meet(it, d, std::integral_constant<int, NW == 1 ? D - 1 : D - 2>{});
        if constexpr (NW > 1)
            load(it + D - 1, (d + D - 1) % D);
    };
    // No load is issued for stages that do not follow: an empty window costs a load's time in the address unit.
    if (nit >= D - 1) {
        int it = 0;
#pragma unroll
        for (int d = 0; d < D - 1; d++)
            load(d, d);
        for (; it + 2 * D - 2 < nit; it += D)
            each(std::make_integer_sequence<int, D>{}, [&](auto d) {
                step(it + d, d);
                multiply(d);
            });
        each(std::make_integer_sequence<int, 2 * D - 2>{}, [&](auto d) {
            if (it + d < nit) {
                if (it + d + D - 1 < nit)
                    step(it + d, std::integral_constant<int, d % D>{});
                else
                    meet(it + d, d % D, std::integral_constant<int, 0>{});
                multiply(d % D);
            }
        });
    } else {
#pragma unroll
        for (int d = 0; d < D - 2; d++)
            if (d < nit)
                load(d, d);
#pragma unroll
        for (int d = 0; d < D - 2; d++)
            if (d < nit) {
                meet(d, d, std::integral_constant<int, 0>{});
                multiply(d);
            }
    }
    __builtin_amdgcn_s_waitcnt(vmcnt_lgkm_imm(0));   // nothing may land in LDS any more
    if constexpr (KG > 1) {
        __syncthreads();   // every wave is past its last stage: LDS holds the groups' sums from here
        u32x4_t *mine = &lds[wave * MF * NF * WAVE + lane];
#pragma unroll
        for (int f = 0; f < MF; f++)
#pragma unroll
            for (int j = 0; j < NF; j++)
                mine[(f * NF + j) * WAVE] = __builtin_bit_cast(u32x4_t, acc[f][j]);
        __syncthreads();
    }
    auto total = [&](int f, int j) {
        if constexpr (KG == 1) {
            return acc[f][j];
        } else {
            acc_t sum{0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < KG; k++)
                sum += __builtin_bit_cast(acc_t, lds[((k * NW + wv) * MF * NF + f * NF + j) * WAVE + lane]);
            return sum;
        }
    };
#pragma unroll
    for (int i = 0; i < ENDS; i++) {
        const int f = row(i), j = col(i), nb = nb0 + j;
        if (f >= MF || nb >= g.nblk || (g.glu && j % 2))
            continue;
        acc_t up{0, 0, 0, 0};
        if constexpr (NF % 2 == 0)   // launched with glu
            if (g.glu)
                up = total(f, j | 1);
        emit(g, m0 + f * 16 + (lane & 15), nb, factors[i], total(f, j), up);
    }
}

// Many tokens, where the time is the matrix cores': the largest tile, 256 tokens x 256 packed columns, by four waves
// of 128 x 128, one per SIMD. Per 64 codes a wave multiplies for 1024 clocks (64 instructions) and reads 16 KiB of
// operands, so the LDS is busy 512 clocks with all reads and 256 with the loads' writes; eight waves of 128
// x 64 would read 1.5 times as much and leave the LDS no slack. A wave reads the operands of the next half
// stage, and issues the loads, between the instructions that multiply the current one. The 160 KiB of LDS hold
// three 128-code stages of activations (whole lines) and four 64-code halves of weights, loaded three to four
// halves ahead of their reads.
//
// 8192 x (2 x 14336) x 7168 gated takes 1.20 to 1.26 ms, 2.7 to 2.8 POP/s (a library product of 8-bit codes of these
// sizes without scales or gate: 1.58 ms), 8192 x 7168 x 14336 0.61 to 0.67 ms. The gated one is 2.4 M clocks whatever the
// codes, 67% of them multiplication (1331 us at 1.79 GHz in one profiled run); a tile's loop takes 20.3 clocks a code
// for 16 of multiplication, its start and end 27000 clocks that nothing overlaps. Codes that are all zero run at 2.3 to
// 2.4 GHz (1.05 ms), codes as they come at 1.6 to 1.9: energy sets the clock. The 16x16x64 instruction moves a
// fifth less through the register files than 32x32x32 (1.45 ms so), four waves 128 x 128 a third less
// through the LDS than eight of 128 x 64 (1.42 ms).

// acc += a . b with the sums kept in accumulation registers (left to itself the compiler moves some of the 64
// sums of a wave between register files around every instruction: 1.65 ms). The compiler does not know
// what is in the statement, so its waits are the caller's: operands come from LDS reads, waited for in
// meet(), never from vector instructions right before; sums are set, and read, with settle() between.
__device__ inline void mfma_acc(u32x4_t a, u32x4_t b, acc_t &acc)
{
    asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}
template <int MF, int NF>
__device__ inline void settle(acc_t (&acc)[MF][NF])
{
    // more clocks than a result takes to leave the matrix cores, or a written register to be read by them
    asm volatile("s_nop 15\n\ts_nop 15");
#pragma unroll
    for (int f = 0; f < MF; f++)
#pragma unroll
        for (int j = 0; j < NF; j++)
            asm volatile("" : "+a"(acc[f][j]));   // no copy of a sum moves across
}

// Between what lanes of a wave write to LDS and what its other lanes read of it, or write over it next: the memory
// model orders the two only past a fence and a barrier, though a wave's accesses to LDS are done in order anyway, so
// that neither costs an instruction here.
__device__ inline void meet_lanes()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// MF and NF: row and column fragments per wave; tiles of 32 MF x 32 NF. 128-token tiles take 80 KiB of LDS or
// less and half the registers, so that two workgroups share a CU. With 7 column fragments a tile loads, but
// does not use, the two row blocks after its own.
template <int MF, int NF, bool GLU, bool F32>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(MF == 8 ? 1 : 2)))
void wide_kernel(const I8Args g, int gx, int gy)
{
    constexpr int BM = 32 * MF, BN = (NF + 1) / 2 * 64;             // MF x NF fragments of 16 x 16 per wave
    constexpr int ASLOT = BM * 8, BSLOT = BN * 4, NA = 3, NB = 4;   // 16-byte slots per stage / half; how many
    constexpr int AL = BM / 8 / 4, BL = BN / 16 / 4;                // loads per wave per stage / half
    __shared__ u32x4_t lds[NA * ASLOT + NB * BSLOT];
    const int lane = threadIdx.x & (WAVE - 1);
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    int bx, by;
    if (!tile_item(gx, gy, bx, by))
        return;
    const int m0 = by * BM, nb0 = bx * (2 * NF);
    const int nst = (int)i8_stages(g.K);
    const int8_t *xt = g.x + (int64_t)m0 * g.ldx;
    const int xbytes = (min(g.T - m0, BM) - 1) * (int)g.ldx + g.K;
    const uint8_t *wt = g.w + (int64_t)nb0 * I8_STAGE_BYTES;
    const int wbytes = min(g.nblk - nb0, BN / 16) * I8_STAGE_BYTES;
    const int64_t wstep = (int64_t)g.nblk * I8_STAGE_BYTES;
    int aoff[AL];
#pragma unroll
    for (int i = 0; i < AL; i++) {
        const int row = (wv * AL + i) * 8 + (lane >> 3);
        aoff[i] = row * (int)g.ldx + ((lane & 7) ^ swizzle(row)) * 16;
    }
    // Load i of this wave's part of stage s (activations) or half hs % 2 of stage hs / 2 (weights).
    auto load_a = [&](int s, int i) {
        const int k = min(s, nst - 1) * I8_STAGE, bytes = (xbytes - k) & -(int)(s < nst);
        load_lds(xt + k, bytes, aoff[i], &lds[s % NA * ASLOT + (wv * AL + i) * WAVE]);
    };
    auto load_b = [&](int hs, int i) {
        const int64_t at = min(hs / 2, nst - 1) * wstep + hs % 2 * I8_BLOCK_BYTES;
        const int bytes = (wbytes - hs % 2 * I8_BLOCK_BYTES) & -(int)(hs < 2 * nst);
        load_lds(wt + at, bytes, (wv * BL + i) * I8_STAGE_BYTES + lane * 16,
                 &lds[NA * ASLOT + hs % NB * BSLOT + (wv * BL + i) * WAVE]);
    };
    // The loads issued while half hs multiplies: the weights of half hs + 4 and one half of those of a stage
    // of activations, whose slots every wave has left. As many in every half, so that the wait for the next
    // half's data is always for all but the last two halves' loads.
    constexpr int PER = AL / 2 + BL;
    auto load = [&](int hs, int i) {
        if (i < BL)
            load_b(hs + 4, i);
        else
            load_a((hs + 5) / 2, i - BL + (hs % 2 ? 0 : AL / 2));
    };
    const int fa = wv / 2 * MF, fb = wv % 2 * NF;   // this wave's first fragments
    const int r16 = lane & 15, ar = (fa * 16 + r16) * 8, ac = (lane >> 4) ^ swizzle(r16);
    struct Operands {   // of half a stage
        u32x4_t a[MF], b[NF];
    };
    // Read i of half hs, in the order of use: the first weights, the activations, the other weights.
    auto read = [&](int hs, int i, Operands &o) {
        if (i >= 1 && i <= MF)
            o.a[i - 1] = lds[hs / 2 % NA * ASLOT + ar + (i - 1) * 16 * 8 + (ac ^ hs % 2 * 4)];
        else
            o.b[i ? i - MF : 0] = lds[NA * ASLOT + hs % NB * BSLOT + (fb + (i ? i - MF : 0)) * WAVE + lane];
    };
    acc_t acc[MF][NF];
#pragma unroll
    for (int f = 0; f < MF; f++)
#pragma unroll
        for (int j = 0; j < NF; j++)
            acc[f][j] = acc_t{0, 0, 0, 0};
    // One half stage: its MF * NF instructions, and among them the reads of the next half into the other
    // operands and the loads. The order is fixed: left to itself the compiler gathers the reads at
    // the end, right before the wait for them. Rows of fragments are walked back and forth, so that
    // consecutive instructions share an operand.
    auto half = [&](const Operands &now, int hs, Operands &next) {
        constexpr int ALL = MF * NF, READS = MF + NF;
#pragma unroll
        for (int x = 0; x < ALL; x++) {
            const int j = x / MF, f = j % 2 ? MF - 1 - x % MF : x % MF;
            mfma_acc(now.b[j], now.a[f], acc[f][j]);
#pragma unroll
            for (int i = 0; i < READS; i++)
                if (x == i * ALL / READS + 1)
                    read(hs + 1, i, next);
#pragma unroll
            for (int i = 0; i < PER; i++)
                if (x == i * ALL / PER + 1)
                    load(hs, i);
            if (x % 4 == 3)
                __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto meet = [&](auto ahead) {   // all but the last loads have landed and this wave's reads are done; then every wave's
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(vmcnt_lgkm_imm(decltype(ahead)::value));
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    // Stages 0 and 1 and the loads that halves -1, -2 and -3 would have issued.
#pragma unroll
    for (int i = 0; i < AL; i++)
        load_a(0, i);
#pragma unroll
    for (int i = 0; i < BL; i++)
        load_b(0, i);
#pragma unroll
    for (int i = 0; i < AL / 2; i++)
        load_a(1, i);
#pragma unroll
    for (int i = 0; i < BL; i++)
        load_b(1, i);
#pragma unroll
    for (int i = 0; i < PER; i++)
        load(-2, i);
#pragma unroll
    for (int i = 0; i < PER; i++)
        load(-1, i);
    meet(std::integral_constant<int, 3 * PER>());
    Operands even, odd;
#pragma unroll
    for (int i = 0; i < MF + NF; i++)
        read(0, i, even);
    settle(acc);
    for (int s = 0; s < nst; s++) {
        meet(std::integral_constant<int, 2 * PER>());   // half 2s + 1 has landed; half 2s is in every wave's registers
        half(even, 2 * s, odd);
        meet(std::integral_constant<int, 2 * PER>());
        half(odd, 2 * s + 1, even);
    }
    __builtin_amdgcn_s_waitcnt(vmcnt_lgkm_imm(0));   // nothing may land in LDS any more
    __syncthreads();                                 // and every wave is past its reads

    settle(acc);

    // Epilogue, 16 tokens at a time through this wave's part of LDS, to store whole 16-byte pieces of rows.
    // Lane (q = l / 16, c = l % 16) of fragment (f, j) holds token 16 f + c and packed columns 16 j + 4 q ..
    // +3; when GLU, fragment j + 1 (odd) holds the up sums of fragment j.
    constexpr int JO = GLU ? NF / 2 : NF, SIZE = F32 ? 4 : 2;        // output fragments, bytes per output
    constexpr int PIECES = JO * 16 * SIZE / 16, PITCH = PIECES * 16 + 16;
    static_assert(4 * 16 * PITCH <= (NA * ASLOT + NB * BSLOT) * 16, "room for the outputs");
    uint8_t *stage = reinterpret_cast<uint8_t *>(lds) + wv * (16 * PITCH);
    const int n1 = (nb0 + fb) / (GLU ? 2 : 1) * 16, q4 = 4 * (lane >> 4);   // first output column of this wave
    f32x4_t sw[JO], other[JO];                                       // other: the up scales, or the bias
#pragma unroll
    for (int j = 0; j < JO; j++) {
        const int col = min(nb0 + fb + j * (GLU ? 2 : 1), g.nblk - (GLU ? 2 : 1)) * 16 + q4;
        sw[j] = *reinterpret_cast<const f32x4_t *>(g.sw + col);
        if (GLU)
            other[j] = *reinterpret_cast<const f32x4_t *>(g.sw + col + 16);
        else
            other[j] = g.bias ? *reinterpret_cast<const f32x4_t *>(g.bias + col) : f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    float sx[MF];
#pragma unroll
    for (int f = 0; f < MF; f++)
        sx[f] = g.sx[min(m0 + (fa + f) * 16 + r16, g.T - 1)];
#pragma unroll
    for (int f = 0; f < MF; f++) {
        uint8_t *at = stage + r16 * PITCH + q4 * SIZE;
#pragma unroll
        for (int j = 0; j < JO; j++) {
            f32x4_t v;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                if constexpr (GLU)
                    v[e] = gated(acc[f][2 * j][e], acc[f][2 * j + 1][e], sx[f], sw[j][e], other[j][e]);
                else
                    v[e] = scaled(acc[f][j][e], sx[f], sw[j][e], other[j][e]);
            }
            if constexpr (F32)
                *reinterpret_cast<f32x4_t *>(at + j * 64) = v;
            else
                *reinterpret_cast<uint2 *>(at + j * 32) = uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        }
        meet_lanes();
#pragma unroll
        for (int i = 0; i < (16 * PIECES + WAVE - 1) / WAVE; i++) {
            const int p = i * WAVE + lane, r = p / PIECES, c = p % PIECES;
            const int row = m0 + (fa + f) * 16 + r;
            if (r < 16 && row < g.T)
                store16(g, row, n1 + c * (16 / SIZE), *reinterpret_cast<const u32x4_t *>(stage + r * PITCH + c * 16));
        }
        meet_lanes();
    }
}

// Rows of K codes at any alignment -> rows of 16 `chunks` codes, zero past K. The chunk that crosses K is loaded from 16
// codes before K and shifted into place; one by one its codes took every wave 16 loads (4745 x 4657 codes: 10.3 us, so 12.1).
__global__ __launch_bounds__(256) void restage_kernel(const int8_t *x, int64_t ldx, int K, uint32_t chunks,
                                                      uint32_t total, int8_t *dst)
{
    const uint32_t i = blockIdx.x * 256 + threadIdx.x;   // below 2^32: the host checks
    if (i >= total)
        return;
    const uint32_t r = i / chunks;
    const int c = (int)(i - r * chunks) * 16;
    const int8_t *s = x + r * ldx;
    u32x4_t v{0, 0, 0, 0};
    if (K >= 16) {
        __builtin_memcpy(&v, s + min(c, K - 16), 16);
        v = drop_bytes(v, max(c - (K - 16), 0));
    } else {
        int8_t few[16];
        for (int j = 0; j < 16; j++)
            few[j] = c + j < K ? s[c + j] : (int8_t)0;
        __builtin_memcpy(&v, few, 16);
    }
    *reinterpret_cast<u32x4_t *>(dst + (int64_t)i * 16) = v;
}

// One thread per lane of a block.
__global__ __launch_bounds__(256) void pack_kernel(const int8_t *w, const int8_t *up, int64_t N, int64_t K, int64_t nblk,
                                                   int64_t total, uint8_t *dst)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= total)
        return;
    const int lane = (int)(i % WAVE);
    const int64_t block = i / WAVE, half = block % 2, nb = block / 2 % nblk, stage = block / 2 / nblk;
    const int8_t *src = up && nb % 2 ? up : w;
    const int64_t n = (up ? nb / 2 : nb) * 16 + lane % 16, k = stage * I8_STAGE + half * 64 + lane / 16 * 16;
    int8_t v[16];
    if (n < N && k + 16 <= K)
        __builtin_memcpy(v, src + n * K + k, 16);
    else
        for (int j = 0; j < 16; j++)
            v[j] = n < N && k + j < K ? src[n * K + k + j] : (int8_t)0;
    __builtin_memcpy(dst + i * 16, v, 16);
}

__global__ __launch_bounds__(256) void pack_vectors_kernel(const float *s, const float *up, const float *bias, int64_t N,
                                                           int64_t nblk, float *scales, float *bias_out)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= nblk * 16)
        return;
    const int64_t nb = i / 16, n = (up ? nb / 2 : nb) * 16 + i % 16;
    scales[i] = n < N ? (up && nb % 2 ? up : s)[n] : 0.f;
    if (bias)
        bias_out[i] = n < N ? bias[n] : 0.f;
}

// ONE: launched for one row tile at most, so that only its form for one is built.
template <int MF, int NF, int NW, int KG, int D, bool ONE = false>
hipError_t launch_tile(const I8Args &g, hipStream_t st)
{
    const int gx = (g.nblk + NF * NW - 1) / (NF * NW), gy = (g.T + 16 * MF - 1) / (16 * MF);
    const dim3 grid((unsigned)((gx * gy + XCDS - 1) / XCDS * XCDS)), threads(WAVE * NW * KG);
    if (gy == 1 && g.direct)
        hipLaunchKernelGGL((tile_kernel<MF, NF, NW, KG, D, true, false>), grid, threads, 0, st, g, gx, gy);
    else if (gy == 1)
        hipLaunchKernelGGL((tile_kernel<MF, NF, NW, KG, D, true, true>), grid, threads, 0, st, g, gx, gy);
    else if constexpr (ONE)
        return hipErrorInvalidValue;
    else if (g.direct)
        hipLaunchKernelGGL((tile_kernel<MF, NF, NW, KG, D, false, false>), grid, threads, 0, st, g, gx, gy);
    else
        hipLaunchKernelGGL((tile_kernel<MF, NF, NW, KG, D, false, true>), grid, threads, 0, st, g, gx, gy);
    return hipGetLastError();
}

template <int MF, int NF>
hipError_t launch_wide(const I8Args &g, hipStream_t st)
{
    const int gx = (g.nblk + 2 * NF - 1) / (2 * NF), gy = (g.T + 32 * MF - 1) / (32 * MF);
    const dim3 grid((unsigned)((gx * gy + XCDS - 1) / XCDS * XCDS)), threads(256);
    const bool f32 = g.out_type == MOE_TYPE_F32;
    if constexpr (NF % 2 == 0) {
        if (g.glu && f32)
            hipLaunchKernelGGL((wide_kernel<MF, NF, true, true>), grid, threads, 0, st, g, gx, gy);
        else if (g.glu)
            hipLaunchKernelGGL((wide_kernel<MF, NF, true, false>), grid, threads, 0, st, g, gx, gy);
    }
    if (!g.glu && f32)
        hipLaunchKernelGGL((wide_kernel<MF, NF, false, true>), grid, threads, 0, st, g, gx, gy);
    else if (!g.glu)
        hipLaunchKernelGGL((wide_kernel<MF, NF, false, false>), grid, threads, 0, st, g, gx, gy);
    return hipGetLastError();
}

int64_t tile_count(const I8Args &g, int bm, int bn)
{
    return (int64_t)((g.T + bm - 1) / bm) * ((g.nblk * 16 + bn - 1) / bn);
}
bool one_round(const I8Args &g, int bm, int bn) { return tile_count(g, bm, bn) <= CUS; }

// Many tokens: more than one round of 64 x 64 tiles.
bool many(const I8Args &g) { return g.T > 64 && !one_round(g, 64, 64); }

// Tiles for many tokens: 128 x 64 if they are one round of workgroups, one for each CU; else the shape with the
// least estimated time. A round of tiles over the CUs costs its K loop and a start and end worth some codes more;
// measured, a round of 256 x 256 takes 10.3 ns x (K + 1000), of 256 x 224 9.4 ns x (K + 1400), of 256 x 128 6.1 ns x
// (K + 800). Two 128 x 128 workgroups share a CU and overlap: 7.6 ns x (K + 550) for 2 per CU, 4.7 for one, and
// a last round that is not full less. Microseconds, 7168 x 7168 weights, 256 x 256 / 256 x 128 / 128 x 128 / 128 x
// 64: 256 tokens - / - / 36 / 29; 512 - / 50 / 36 / 45; 1024 78 / 53 / 60 / 80; 1280 74 / 94 / 81 / 96; 2048 82 / 101
// / 113 / -. 2000 x 7000 outputs: 512 codes 18.9 / 20.3 / 17.3 / 20.3, 2048 codes 33.5 / 40.6 / 40.2 / 48; 928 x
// 2416 x 4064 - / 30.9 / 20.0 / 25.7. 8192 x 7168 outputs are 4 rounds of 224 columns and 3.5, so 4, of 256: 605
// against 619 with 14336 codes.
hipError_t launch_many(const I8Args &g, hipStream_t st)
{
    if (one_round(g, 128, 64))
        return launch_wide<4, 2>(g, st);
    auto cost = [&](int bn, int64_t rate, int64_t extra) {
        return (tile_count(g, 256, bn) + CUS - 1) / CUS * rate * (g.K + extra);
    };
    const int64_t c256 = cost(256, 103, 1000), c128 = cost(128, 61, 800);
    const int64_t c224 = g.glu ? INT64_MAX : cost(224, 94, 1400);   // 7 would part a gate from its up block
    const int64_t small = tile_count(g, 128, 128), rest = small % (2 * CUS);
    const int64_t last = rest == 0 ? 0 : rest <= CUS ? 47 : (rest > 448 ? rest : 448) * 76 / (2 * CUS);
    const int64_t cpair = (small / (2 * CUS) * 76 + last) * (g.K + 550);
    if (cpair <= c128 && cpair <= c256 && cpair <= c224)
        return launch_wide<4, 4>(g, st);
    if (c128 <= c256 && c128 <= c224)
        return launch_wide<8, 4>(g, st);
    return c224 < c256 ? launch_wide<8, 7>(g, st) : launch_wide<8, 8>(g, st);
}

} // namespace

// Passing rows through registers saves the restaging launch and its pass over x, and costs some of the product's
// time. Registers against restaging, rows of odd stride, weights from memory: 1 x 1000 x 1000 3.3 us against 5.0, 300 x 3000
// x 999 6.9 / 8.6, 777 x 1001 x 3583 15.8 / 14.9, 32 x 28672 x 7167 36.6 / 38.0, 64 x 14336 x 4095 19.0 / 18.8; from 2^32
// operations on mostly longer: 64 x 14336 x 7167 29.6 / 28.2, 256 x 4096 x 7167 25.0 / 22.3, 64 x 7168 x 14335 41.0 / 32.5,
// 64 x 28672 x 7167 43.9 / 40.3, 500 x 2040 x 14335 45.1 / 35.6. Strides of whole 16 bytes stay ahead: 64 x 28672 x 7167
// 36.9 / 39.5, 256 x 4096 x 28671 64 / 68. The limit, of 2^33, is between the two. Many tokens are restaged: 600 x
// 4096 x 2047 15.5 against 18.4 with 128 x 128 tiles fed from registers, 2504 x 1920 x 356 11.8 against 18.2, though
// 3000 x 1000 x 999 13.2 against 12.1.
bool i8_takes_any_rows(const I8Args &g)
{
    return g.K >= 16 && !many(g) && (int64_t)g.T * g.nblk * 16 * g.K <= (int64_t)1 << 33;
}

// Below that, the smallest tile that is one round of workgroups, one for each CU: less work for each of them than
// with larger tiles, and less to load than with several rounds of smaller ones. 16 columns, or 32 when a gate and an
// up block have to be together, up to the most that a few tokens take; the smaller the tile, the more groups of waves
// share the K axis. Measured, microseconds (tokens x columns x codes; the largest weights not in any cache), with the
// neighbours: 1 x 4352 x 4096: 32 columns 6.7, 16 7.0, 64 8.7; 1 x 3584 x 7168: 16 6.6, 32 8.1; 1 x 10240 x 4096: 64
// 10.3, 32 11.1; 16 x 28672 x 7168: 128 36.2, 64 37.3; 32 x 3584 x 7168: 32 x 16 9.2, 16 x 32 10.6, 16 x 16 12.1, 32
// x 32 11.3; 32 x 10240 x 4096: 32 x 64 12.6, 32 x 32 15.0, 32 x 128 16.2; 32 x 18432 x 4096: 32 x 128 19.6, 32 x 64
// 20.8; 64 x 4352 x 4096: 64 x 32 8.8, 32 x 32 10.9, 64 x 64 13.2; 64 x 10240 x 4096: 64 x 64 14.9, 64 x 32 16.7; 64
// x 18432 x 4096: 64 x 128 22.7, 64 x 64 27.0; 727 x 232 x 7424: 32 x 32 8.5, 16 x 32 9.9, 64 x 32 10.5; 437 x 695 x
// 752: 64 x 32 4.6, 64 x 64 5.6, 32 x 32 6.4; 355 x 1811 x 6256: 64 x 64 14.4, 64 x 32 19.5, 128 x 64 20.7; 438 x
// 2943 x 1024: 128 x 64 7.8, 128 x 128 9.4, 64 x 64 11.3.
hipError_t launch_i8_product(const I8Args &g, hipStream_t st)
{
    auto round = [&](int bm, int bn) { return one_round(g, bm, bn); };
    if (many(g))
        return launch_many(g, st);
    if (!g.glu && round(16, 16))
        return launch_tile<1, 1, 1, 8, 4>(g, st);
    if (g.T <= 16) {
        if (round(16, 32))
            return launch_tile<1, 2, 1, 8, 5>(g, st);
        return round(16, 64) ? launch_tile<1, 2, 2, 4, 4, true>(g, st) : launch_tile<1, 4, 2, 2, 3, true>(g, st);
    }
    if (g.glu && round(16, 32))
        return launch_tile<1, 2, 1, 8, 5>(g, st);
    if (!g.glu && round(32, 16))
        return launch_tile<2, 1, 1, 8, 4>(g, st);
    if (round(32, 32))
        return launch_tile<2, 2, 1, 8, 3>(g, st);
    if (g.T <= 32)
        return round(32, 64) ? launch_tile<2, 2, 2, 4, 3, true>(g, st) : launch_tile<2, 2, 4, 1, 4, true>(g, st);
    if (round(64, 32))
        return launch_tile<4, 2, 1, 4, 3>(g, st);
    return g.T > 64 || round(64, 64) ? launch_tile<4, 2, 2, 4, 3>(g, st) : launch_tile<4, 2, 4, 1, 4, true>(g, st);
}

hipError_t launch_i8_restage(const int8_t *x, int64_t ldx, int T, int K, int8_t *dst, hipStream_t st)
{
    const uint32_t chunks = (uint32_t)i8_stages(K) * (I8_STAGE / 16), total = (uint32_t)T * chunks;
    hipLaunchKernelGGL(restage_kernel, dim3((total + 255) / 256), dim3(256), 0, st, x, ldx, K, chunks, total,
                       dst);
    return hipGetLastError();
}

hipError_t launch_i8_pack(const moe_linear_config &c, const moe_linear_weights &w, uint8_t *blocks, float *scales,
                          float *bias, hipStream_t st)
{
    const int64_t nblk = i8_row_blocks(c.n, c.glu), total = i8_stages(c.k) * nblk * 2 * WAVE;
    hipLaunchKernelGGL(pack_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, st, w.w, w.w_up, (int64_t)c.n,
                       (int64_t)c.k, nblk, total, blocks);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(pack_vectors_kernel, dim3((unsigned)((nblk * 16 + 255) / 256)), dim3(256), 0, st, w.scales,
                       w.scales_up, w.bias, (int64_t)c.n, nblk, scales, bias);
    return hipGetLastError();
}

} // namespace mxmoe
