// int8.hip -- dense products of 8-bit codes, out[t, n] = sx[t] sw[n] sum_k x[t, k] w[n, k] (+ bias), and
// their gated form silu(gate) * up, on the 16x16x64 8-bit matrix-core instruction; kernels in products.hpp.
//
// The sums are exact in 32-bit integers, so any split of K and any order of adding give the same
// bits; scales, bias and the gate are applied in FP32 in the epilogue. Weights are packed once
// (dense.hpp); activations are read as they are.
#include "products.hpp"

namespace mxmoe {

namespace {

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

struct Int8 {
    using Args = I8Args;
    using Acc = sums_t;
    static constexpr bool APART = true;
    static __device__ __forceinline__ Acc mfma(u32x4_t a, u32x4_t b, Acc c)
    {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(Acc, a), __builtin_bit_cast(Acc, b), c, 0, 0, 0);
    }
    static __device__ __forceinline__ void mfma_acc(u32x4_t a, u32x4_t b, Acc &acc)
    {
        asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
    }

    // What one fragment's outputs take besides its sums: the token's scale, and for the lane's four columns their scales
    // and the up columns' scales or the bias.
    struct Factors {
        float sx;
        f32x4_t sw, other;
    };

    // The weights are the first matrix operand, so lane l of a fragment holds token row l % 16 and the packed
    // columns 4 (l / 16) .. +3 of row block nb. Rows and blocks past the end take the last ones' factors.
    static __device__ __forceinline__ Factors load_factors(const I8Args &g, int r, int nb)
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
    static __device__ __forceinline__ void emit(const I8Args &g, int r, int nb, const Factors &c, Acc sum, Acc up)
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

    // Epilogue, 16 tokens at a time through this wave's part of LDS, to store whole 16-byte pieces of rows.
    // Lane (q = l / 16, c = l % 16) of fragment (f, j) holds token 16 f + c and packed columns 16 j + 4 q ..
    // +3; when GLU, fragment j + 1 (odd) holds the up sums of fragment j.
    template <int MF, int NF, bool GLU, bool F32>
    static constexpr int finish_bytes() { return 4 * 16 * ((GLU ? NF / 2 : NF) * 16 * (F32 ? 4 : 2) + 16); }
    template <int MF, int NF, bool GLU, bool F32>
    static __device__ __forceinline__ void finish(const I8Args &g, Acc (&acc)[MF][NF], u32x4_t *lds, int m0, int nb0, int wv)
    {
        const int lane = threadIdx.x & (WAVE - 1), r16 = lane & 15, fa = wv / 2 * MF, fb = wv % 2 * NF;
        constexpr int JO = GLU ? NF / 2 : NF, SIZE = F32 ? 4 : 2;        // output fragments, bytes per output
        constexpr int PIECES = JO * 16 * SIZE / 16, PITCH = PIECES * 16 + 16;
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
};

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
    const int64_t n = (up ? nb / 2 : nb) * 16 + lane % 16, k = stage * STAGE_K + half * 64 + lane / 16 * 16;
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
    if (s)
        scales[i] = n < N ? (up && nb % 2 ? up : s)[n] : 0.f;
    if (bias)
        bias_out[i] = n < N ? bias[n] : 0.f;
}

} // namespace

bool i8_takes_any_rows(const I8Args &g) { return any_rows(g); }

hipError_t launch_i8_product(const I8Args &g, hipStream_t st) { return launch_product<Int8>(g, st); }

hipError_t launch_restage(const int8_t *x, int64_t ldx, int T, int K, int8_t *dst, hipStream_t st)
{
    const uint32_t chunks = (uint32_t)stages(K) * (STAGE_K / 16), total = (uint32_t)T * chunks;
    hipLaunchKernelGGL(restage_kernel, dim3((total + 255) / 256), dim3(256), 0, st, x, ldx, K, chunks, total,
                       dst);
    return hipGetLastError();
}

hipError_t launch_pack_product(const void *w, const void *w_up, int64_t n, int64_t k, uint8_t *blocks, hipStream_t st)
{
    const int64_t nblk = row_blocks(n, w_up), total = stages(k) * nblk * 2 * WAVE;
    hipLaunchKernelGGL(pack_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, st, static_cast<const int8_t *>(w),
                       static_cast<const int8_t *>(w_up), n, k, nblk, total, blocks);
    return hipGetLastError();
}

hipError_t launch_pack_vectors(const float *scales, const float *scales_up, const float *bias, int64_t n, int64_t nblk,
                               float *scales_out, float *bias_out, hipStream_t st)
{
    hipLaunchKernelGGL(pack_vectors_kernel, dim3((unsigned)((nblk * 16 + 255) / 256)), dim3(256), 0, st, scales, scales_up,
                       bias, n, nblk, scales_out, bias_out);
    return hipGetLastError();
}

hipError_t launch_i8_pack(const moe_linear_config &c, const moe_linear_weights &w, uint8_t *blocks, float *scales,
                          float *bias, hipStream_t st)
{
    const hipError_t e = launch_pack_product(w.w, w.w_up, c.n, c.k, blocks, st);
    return e != hipSuccess ? e : launch_pack_vectors(w.scales, w.scales_up, w.bias, c.n, row_blocks(c.n, c.glu), scales, bias,
                                                     st);
}

} // namespace mxmoe
