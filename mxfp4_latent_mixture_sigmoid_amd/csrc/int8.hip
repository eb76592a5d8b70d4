// int8.hip -- dense products of 8-bit codes, out[t, n] = sx[t] sw[n] sum_k x[t, k] w[n, k] (+ bias), and
// their gated form silu(gate) * up, on the 16x16x64 8-bit matrix-core instruction.
//
// The sums are exact in 32-bit integers, so any split of K and any order of adding give the same
// bits; scales, bias and the gate are applied in FP32 in the epilogue. Weights are packed once
// (dense.hpp); activations are read as they are.
#include "dense.hpp"

namespace mxmoe {

namespace {

typedef int32_t acc_t __attribute__((ext_vector_type(4)));
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

// Where chunk c (16 codes) of row r of a staged activation tile (rows of I8_STAGE bytes) lies: the
// operand reads -- 8 or 16 consecutive rows, one chunk -- then fall in distinct banks.
__device__ inline int swizzle(int r) { return (r & 7) ^ ((r >> 3) & 1); }

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

// Outputs of one fragment of row block nb (a gate block with its up block's sums in `up` when glu), token
// row r. The weights are the first matrix operand, so lane l holds row l % 16 and the packed
// columns 4 (l / 16) .. +3.
__device__ inline void emit(const I8Args &g, int r, float sx, int nb, acc_t sum, acc_t up)
{
    const int q = (threadIdx.x & (WAVE - 1)) >> 4;
    const int n = (g.glu ? nb / 2 : nb) * 16 + 4 * q;
    if (n >= g.N)
        return;
    const f32x4_t sw = *reinterpret_cast<const f32x4_t *>(g.sw + nb * 16 + 4 * q);
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; i++)
        v[i] = (float)sum[i] * sx * sw[i];
    if (g.glu) {
        const f32x4_t su = *reinterpret_cast<const f32x4_t *>(g.sw + nb * 16 + 16 + 4 * q);
#pragma unroll
        for (int i = 0; i < 4; i++)
            v[i] = silu_f32(v[i]) * ((float)up[i] * sx * su[i]);
    } else if (g.bias) {
        const f32x4_t b = *reinterpret_cast<const f32x4_t *>(g.bias + n);
#pragma unroll
        for (int i = 0; i < 4; i++)
            v[i] += b[i];
    }
    store4(g, r, n, v);
}

// Tiles of BM tokens x BN packed columns by KG groups of NWM x NWN waves; group k takes every KG-th stage of
// 128 codes, and the groups' sums are added through LDS at the end. Both operands pass through LDS in
// NBUF buffers of KG stages, filled by direct global -> LDS loads: one instruction fills 1 KiB, of the
// activations 8 rows x 128 bytes (whole lines), of the weights one packed block. Rows past T and stages
// past K lie outside the loads' windows and read as zeros without touching memory. ONCE: there is
// one row tile, so weights are read once, and are not to displace the activations in the caches.
template <int BM, int BN, int NWM, int NWN, int KG, int NBUF, bool ONCE>
__global__ __launch_bounds__(WAVE *NWM *NWN *KG) void tile_kernel(const I8Args g, int gx, int gy)
{
    constexpr int NW = NWM * NWN, WMF = BM / NWM / 16, WNF = BN / NWN / 16;
    constexpr int AL = BM / 8 / NW, BL = BN / 8 / NW;   // loads per wave and stage
    constexpr int STAGE = (BM + BN) * 8;                // 16-byte slots
    static_assert(AL * NW * 8 == BM && BL * NW * 8 == BN, "tile");
    static_assert(KG == 1 || NBUF * STAGE >= NW * WMF * WNF * WAVE, "room for the groups' sums");
    __shared__ u32x4_t lds[NBUF * KG * STAGE];
    const int lane = threadIdx.x & (WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int wv = wave % NW, kg = wave / NW;
    int bx, by;
    if (!tile_item(gx, gy, bx, by))
        return;
    const int m0 = by * BM, nb0 = bx * (BN / 16);
    const int nst = (int)i8_stages(g.K);
    const int8_t *xt = g.x + (int64_t)m0 * g.ldx;
    const int xbytes = (min(g.T - m0, BM) - 1) * (int)g.ldx + g.K;
    const uint8_t *wt = g.w + (int64_t)nb0 * I8_STAGE_BYTES;
    const int wbytes = min(g.nblk - nb0, BN / 16) * I8_STAGE_BYTES;
    int aoff[AL];
#pragma unroll
    for (int i = 0; i < AL; i++) {
        const int row = (wv * AL + i) * 8 + (lane >> 3);
        aoff[i] = row * (int)g.ldx + ((lane & 7) ^ swizzle(row)) * 16;
    }
    auto issue = [&](int it) {
        u32x4_t *buf = &lds[(it % NBUF * KG + kg) * STAGE];
        const int s = it * KG + kg, k = s * I8_STAGE;
        const bool in = s < nst;
        const int8_t *xs = xt + (in ? k : 0);
        const uint8_t *ws = wt + (in ? (int64_t)s * g.nblk * I8_STAGE_BYTES : 0);
#pragma unroll
        for (int i = 0; i < BL; i++)
            load_lds<ONCE ? CPOL_NT : 0>(ws, in ? wbytes : 0, (wv * BL + i) * I8_BLOCK_BYTES + lane * 16,
                                         &buf[BM * 8 + (wv * BL + i) * WAVE]);
#pragma unroll
        for (int i = 0; i < AL; i++)
            load_lds(xs, in ? xbytes - k : 0, aoff[i], &buf[(wv * AL + i) * WAVE]);
    };
    acc_t acc[WMF][WNF];
#pragma unroll
    for (int f = 0; f < WMF; f++)
#pragma unroll
        for (int j = 0; j < WNF; j++)
            acc[f][j] = acc_t{0, 0, 0, 0};
    const int fa = (wv / NWN) * WMF, fb = (wv % NWN) * WNF;
    const int nit = (nst + KG - 1) / KG;
#pragma unroll
    for (int it = 0; it < NBUF - 1; it++)
        issue(it);
    for (int it = 0; it < nit; it++) {
        // This wave's part of these stages has landed and its reads of the last ones are done; past the
        // barrier, every wave's, so that the last ones' buffer can be filled again.
        __builtin_amdgcn_s_waitcnt(vmcnt_lgkm_imm((NBUF - 2) * (AL + BL)));
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        issue(it + NBUF - 1);
        const u32x4_t *buf = &lds[(it % NBUF * KG + kg) * STAGE];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            u32x4_t a[WMF], b[WNF];
            const int r = lane & 15, c = (h * 4 + (lane >> 4)) ^ swizzle(r);
#pragma unroll
            for (int f = 0; f < WMF; f++)
                a[f] = buf[((fa + f) * 16 + r) * 8 + c];
#pragma unroll
            for (int j = 0; j < WNF; j++)
                b[j] = buf[BM * 8 + ((fb + j) * 2 + h) * WAVE + lane];
#pragma unroll
            for (int j = 0; j < WNF; j++)
#pragma unroll
                for (int f = 0; f < WMF; f++)
                    acc[f][j] = mfma(b[j], a[f], acc[f][j]);
        }
        asm volatile("" ::: "memory");
    }
    __builtin_amdgcn_s_waitcnt(vmcnt_lgkm_imm(0));   // nothing may land in LDS any more
    if constexpr (KG > 1) {
        __syncthreads();   // every wave is past its last stage: LDS holds the groups' sums from here
        u32x4_t *mine = &lds[((kg * NW + wv) * WMF * WNF) * WAVE + lane];
#pragma unroll
        for (int f = 0; f < WMF; f++)
#pragma unroll
            for (int j = 0; j < WNF; j++)
                mine[(f * WNF + j) * WAVE] = __builtin_bit_cast(u32x4_t, acc[f][j]);
        __syncthreads();
    }
    // Group k finishes every KG-th fragment (or pair of a gate and an up fragment).
    auto total = [&](int f, int j) {
        if constexpr (KG == 1) {
            return acc[f][j];
        } else {
            acc_t sum{0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < KG; k++)
                sum += __builtin_bit_cast(acc_t, lds[((k * NW + wv) * WMF * WNF + f * WNF + j) * WAVE + lane]);
            return sum;
        }
    };
#pragma unroll
    for (int f = 0; f < WMF; f++) {
        const int r = m0 + (fa + f) * 16 + (lane & 15);
#pragma unroll
        for (int j = 0; j < WNF; j++) {
            const int nb = nb0 + fb + j, unit = g.glu ? (f * WNF + j) / 2 : f * WNF + j;
            if (nb >= g.nblk || (g.glu && j % 2) || (KG > 1 && unit % KG != kg) || r >= g.T)
                continue;
            acc_t up{0, 0, 0, 0};
            if constexpr (WNF % 2 == 0)   // launched with glu
                if (g.glu)
                    up = total(f, j | 1);
            emit(g, r, g.sx[r], nb, total(f, j), up);
        }
    }
}

// Rows of K codes at any alignment -> rows of `width` codes (a multiple of 16), zero past K.
__global__ __launch_bounds__(256) void restage_kernel(const int8_t *x, int64_t ldx, int K, int chunks, int64_t total,
                                                      int8_t *dst)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= total)
        return;
    const int64_t r = i / chunks;
    const int c = (int)(i % chunks) * 16;
    const int8_t *s = x + r * ldx + c;
    int8_t v[16];
    if (c + 16 <= K)
        __builtin_memcpy(v, s, 16);
    else
        for (int j = 0; j < 16; j++)
            v[j] = c + j < K ? s[j] : (int8_t)0;
    __builtin_memcpy(dst + i * 16, v, 16);
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

template <int BM, int BN, int NWM, int NWN, int KG, int NBUF>
hipError_t launch_tile(const I8Args &g, hipStream_t st)
{
    const int gx = (g.nblk * 16 + BN - 1) / BN, gy = (g.T + BM - 1) / BM;
    const dim3 grid((unsigned)((gx * gy + XCDS - 1) / XCDS * XCDS)), threads(WAVE * NWM * NWN * KG);
    if (gy == 1)
        hipLaunchKernelGGL((tile_kernel<BM, BN, NWM, NWN, KG, NBUF, true>), grid, threads, 0, st, g, gx, gy);
    else
        hipLaunchKernelGGL((tile_kernel<BM, BN, NWM, NWN, KG, NBUF, false>), grid, threads, 0, st, g, gx, gy);
    return hipGetLastError();
}

} // namespace

// Tiles by the number of workgroups: the widest that still makes FILL of them, three quarters of the
// card's 256 CUs, else the narrowest (16 columns; 32 when a gate and an up block have to be together),
// with the K axis over more groups of waves the narrower the tile. Measured, microseconds (weights not in
// any cache), chosen against the next wider or narrower tile: 1 x 3584 x 7168: 16 columns 7.4, 32 8.1;
// 16 x 7168 x 4352: 32 8.4, 16 11.7, 64 9.8; 16 x 14336 x 3584: 64 10.7, 32 12.8, 128 14.3; 64 x 7168 x
// 4352: 32 11.2, 64 13.1, 16 16.6; 64 x (2 x 14336) x 7168: 128 38.3, 64 42.6, 256 47.
hipError_t launch_i8_product(const I8Args &g, hipStream_t st)
{
    constexpr int64_t FILL = 192;
    auto fills = [&](int bm, int bn) {
        return (int64_t)((g.T + bm - 1) / bm) * ((g.nblk * 16 + bn - 1) / bn) >= FILL;
    };
    if (g.T <= 16) {
        if (fills(16, 64))
            return launch_tile<16, 64, 1, 2, 2, 4>(g, st);
        if (fills(16, 32) || g.glu)
            return launch_tile<16, 32, 1, 1, 4, 4>(g, st);
        return launch_tile<16, 16, 1, 1, 8, 3>(g, st);
    }
    if (g.T <= 32) {
        if (fills(32, 128))
            return launch_tile<32, 128, 1, 4, 1, 4>(g, st);
        if (fills(32, 64))
            return launch_tile<32, 64, 1, 2, 2, 4>(g, st);
        if (fills(32, 32) || g.glu)
            return launch_tile<32, 32, 1, 1, 4, 3>(g, st);
        return launch_tile<32, 16, 1, 1, 8, 3>(g, st);
    }
    const int64_t area = (int64_t)g.T * g.nblk * 16;
    if (area >= (int64_t)256 * 256 * 256)
        return launch_tile<256, 256, 2, 4, 1, 2>(g, st);
    if (area >= (int64_t)128 * 128 * 256)
        return launch_tile<128, 128, 2, 2, 1, 2>(g, st);
    if (fills(64, 128))
        return launch_tile<64, 128, 2, 4, 1, 3>(g, st);
    if (fills(64, 64))
        return launch_tile<64, 64, 2, 2, 2, 3>(g, st);
    if (fills(64, 32) || g.glu)
        return launch_tile<64, 32, 2, 1, 2, 3>(g, st);
    return launch_tile<64, 16, 2, 1, 4, 3>(g, st);
}

hipError_t launch_i8_restage(const int8_t *x, int64_t ldx, int T, int K, int8_t *dst, hipStream_t st)
{
    const int chunks = (int)i8_stages(K) * (I8_STAGE / 16);
    const int64_t total = (int64_t)T * chunks;
    hipLaunchKernelGGL(restage_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, st, x, ldx, K, chunks, total,
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
