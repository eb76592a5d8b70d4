// bf16.hip -- dense products of BF16 values with bias, activation and residual in their epilogue,
//   out[t, n] = a(sum_k x[t, k] w[n, k] + bias[n]) + residual[t, n],
// and their gated form a(gate) * up + residual, on the 16x16x32 BF16 matrix-core instruction; kernels in products.hpp.
//
// Sums are FP32, in an order that depends on the sizes (the tile and how many groups of waves share K), never on
// timing; bias, activation, gate and residual are FP32, and the result is rounded once to its type.
//
// Bounds: few tokens, the weights from memory (7168 x 7168: 1 token 18.2 us, 5.6 TB/s; 32 21.2; 64 gated 40, 5.2 TB/s); 128 to
// 512, the load path of a CU (256 tokens 51.5 us); more, the matrix cores (1024 97 us, 8192 620 to 660, 1.27 to 1.36 PFLOP/s; the
// library's 23.2, 25.0, 67.2, 99.8, 569).
#include "products.hpp"

namespace mxmoe {

namespace {

// v / (1 + exp(-gate)) on the hardware's exponential and reciprocal, each within a unit in the last place; the rounding of the
// exponent adds |gate| 2^-23 relative. Past 2^126 the exponential's reciprocal is 0, and so is the result from gate = -87.3 down.
__device__ inline float silu_of(float gate, float v)
{
    return v * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * gate));
}

// v Phi(v). Phi(-a) exp(a^2 / 2) falls from 1/2 to 0.4 / a: t (c0 + c1 t .. + c8 t^8) with t = 1 / (1 + p a), coefficients fitted over
// 0 <= a <= 15 by Lawson's weighted least squares to the smallest relative error, 0.6 x 2^-24. The exponential's argument is
// taken in two parts, so that its rounding (a^2 2^-24 of the result) is not felt. In all 7 x 2^-24 of the result as computed,
// 24 by the roundings' bounds, for both signs and however small the result is (below 2^-126 it is 0). Abramowitz and Stegun
// 7.1.26, whose absolute error is small, is off by 5 x 10^-4 of the result at -4 and by 1% at -8, and was not faster. The library's erff, with its
// branches, 256 times in a large tile's epilogue is more than the compiler unrolls.
__device__ inline float gelu(float v)
{
    constexpr float P = 0x1.0f5c28p-2f, C[9] = {0x1.b11bb6p-4f, 0x1.af3fdcp-4f, 0x1.a38134p-4f, 0x1.f75a5ep-5f, 0x1.14f2fep-3f,
                                                -0x1.cc0788p-4f, 0x1.b6a0d6p-3f, -0x1.23aaeep-3f, 0x1.f2af1ep-6f};
    constexpr float HIGH = -0x1.715476p-1f, LOW = -0x1.4ae0cp-27f, LN2 = 0x1.62e43p-1f;   // HIGH + LOW = -log2(e) / 2
    const float a = fminf(fabsf(v), 15.f), t = __builtin_amdgcn_rcpf(fmaf(P, a, 1.f));   // a NaN is one in the last product
    float poly = C[8];
#pragma unroll
    for (int i = 7; i >= 0; i--)
        poly = fmaf(t, poly, C[i]);
    const float sq = a * a, arg = sq * HIGH;
    const float rest = fmaf(sq, LOW, fmaf(fmaf(a, a, -sq), HIGH, fmaf(sq, HIGH, -arg)));
    const float e = __builtin_amdgcn_exp2f(arg), tail = t * poly * fmaf(e, rest * LN2, e);   // Phi(-a)
    return v * (v < 0.f ? tail : 1.f - tail);
}

template <int ACT>
__device__ inline float activated(float v)
{
    if constexpr (ACT == MOE_LINEAR_SILU)
        return silu_of(v, v);
    if constexpr (ACT == MOE_LINEAR_GELU)
        return gelu(v);
    if constexpr (ACT == MOE_LINEAR_GELU_TANH)   // v / 2 (1 + tanh(c)) = v / (1 + exp(-2 c))
        return silu_of(1.59576912f * fmaf(0.044715f * v * v, v, v), v);
    if constexpr (ACT == MOE_LINEAR_RELU)
        return v < 0.f ? 0.f : v;   // NaN stays
    return v;
}

// f with the activation as a constant.
template <class F>
__device__ inline void with_activation(int act, F f)
{
    switch (act) {
    case MOE_LINEAR_SILU:
        return f(std::integral_constant<int, MOE_LINEAR_SILU>{});
    case MOE_LINEAR_GELU:
        return f(std::integral_constant<int, MOE_LINEAR_GELU>{});
    case MOE_LINEAR_GELU_TANH:
        return f(std::integral_constant<int, MOE_LINEAR_GELU_TANH>{});
    case MOE_LINEAR_RELU:
        return f(std::integral_constant<int, MOE_LINEAR_RELU>{});
    default:
        return f(std::integral_constant<int, MOE_LINEAR_NONE>{});
    }
}

// Four consecutive values of row r of the residual from column n on, zeros past the end.
__device__ inline void load_residual(const Bf16Args &g, int r, int n, float *v)
{
    constexpr int N = 4;
#pragma unroll
    for (int i = 0; i < N; i++)
        v[i] = 0.f;
    if (!g.residual || r >= g.T || n >= g.N)
        return;
    if (g.res_type == MOE_TYPE_F32) {
        const float *p = static_cast<const float *>(g.residual) + r * g.ldr + n;
        if (n + N <= g.N)
            __builtin_memcpy(v, p, 4 * N);
        else
#pragma unroll
            for (int i = 0; i < N; i++)
                if (n + i < g.N)
                    v[i] = p[i];
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(g.residual) + r * g.ldr + n;
        uint16_t raw[N] = {};
        if (n + N <= g.N)
            __builtin_memcpy(raw, p, 2 * N);
        else
#pragma unroll
            for (int i = 0; i < N; i++)
                if (n + i < g.N)
                    raw[i] = p[i];
#pragma unroll
        for (int i = 0; i < N; i++)
            v[i] = bf16_bits_to_f32(raw[i]);
    }
}

// Eight consecutive values of the residual, as they come from memory.
struct Piece {
    u32x4_t lo, hi;
    // of row r from column n on; nothing past the end
    __device__ void load(const Bf16Args &g, int r, int n)
    {
        if (!g.residual || r >= g.T || n >= g.N)
            return;
        const int size = g.res_type == MOE_TYPE_F32 ? 4 : 2;
        const uint8_t *p = static_cast<const uint8_t *>(g.residual) + (r * g.ldr + n) * size;
        if (n + 8 <= g.N) {
            __builtin_memcpy(&lo, p, 16);
            if (size == 4)
                __builtin_memcpy(&hi, p + 16, 16);
            return;
        }
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (n + i < g.N)
                w[i] = size == 4 ? reinterpret_cast<const uint32_t *>(p)[i] : reinterpret_cast<const uint16_t *>(p)[i];
            else
                w[i] = 0;
        lo = size == 4 ? u32x4_t{w[0], w[1], w[2], w[3]}
                       : u32x4_t{w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16};
        hi = u32x4_t{w[4], w[5], w[6], w[7]};
    }
    __device__ void add(const Bf16Args &g, float *v) const
    {
#pragma unroll
        for (int i = 0; i < 8; i++)
            if (g.res_type == MOE_TYPE_F32)
                v[i] += __uint_as_float(i < 4 ? lo[i] : hi[i - 4]);
            else
                v[i] += __uint_as_float(i % 2 ? lo[i / 2] & 0xFFFF0000u : lo[i / 2] << 16);
    }
};

__device__ inline void store8(const Bf16Args &g, int r, int n, const float *v)
{
    if (g.out_type == MOE_TYPE_F32) {
        u32x4_t lo, hi;
        __builtin_memcpy(&lo, v, 16);
        __builtin_memcpy(&hi, v + 4, 16);
        store16(g, r, n, lo);
        store16(g, r, n + 4, hi);
    } else {
        store16(g, r, n, u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                 pack_bf16x2(v[6], v[7])});
    }
}

struct Bf16 {
    using Args = Bf16Args;
    using Acc = f32x4_t;
    static constexpr bool APART = false;
    static __device__ __forceinline__ Acc mfma(u32x4_t a, u32x4_t b, Acc c) { return mfma16(as_bf16x8(a), as_bf16x8(b), c); }
    static __device__ __forceinline__ void mfma_acc(u32x4_t a, u32x4_t b, Acc &acc)
    {
        asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
    }

    // What one fragment's outputs take besides its sums, for lane l's token row l % 16 and the columns 4 (l / 16) .. +3
    // of row block nb. The residual may be the output itself: the lane that reads an element here is the one that writes it.
    struct Factors {
        f32x4_t bias, residual;
    };
    static __device__ __forceinline__ Factors load_factors(const Bf16Args &g, int r, int nb)
    {
        const int q = (threadIdx.x & (WAVE - 1)) >> 4, n = (g.glu ? nb / 2 : nb) * 16 + 4 * q;
        Factors v{{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        if (nb >= g.nblk)
            return v;
        if (g.bias)
            v.bias = *reinterpret_cast<const f32x4_t *>(g.bias + n);
        float res[4];
        load_residual(g, r, n, res);
        v.residual = f32x4_t{res[0], res[1], res[2], res[3]};
        return v;
    }

    // Outputs of one fragment of row block nb (a gate block with its up block's sums in `up` when glu).
    static __device__ __forceinline__ void emit(const Bf16Args &g, int r, int nb, const Factors &c, Acc sum, Acc up)
    {
        const int q = (threadIdx.x & (WAVE - 1)) >> 4, n = (g.glu ? nb / 2 : nb) * 16 + 4 * q;
        if (r >= g.T || n >= g.N)
            return;
        float v[4];
        with_activation(g.act, [&](auto act) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float a = activated<act>(sum[i] + c.bias[i]);
                v[i] = (g.glu ? a * up[i] : a) + c.residual[i];
            }
        });
        store4(g, r, n, v);
    }

    // Epilogue of the large tiles: half of this wave's sums at a time through its part of LDS, in FP32, so that the residual
    // is added before the one rounding, and is read, and the outputs stored, in whole 16-byte pieces of rows. Lane (q = l /
    // 16, c = l % 16) of fragment (f, j) holds token 16 f + c and packed columns 16 j + 4 q .. +3; when GLU, fragment j + 1
    // (odd) holds the up sums of fragment j. What follows the way through LDS is a loop, one piece of 8 outputs per
    // lane and round, G rounds a step, whose residuals are loaded a step ahead: unrolled over all sums the code was too
    // long for the compiler, which then kept the sums in memory (11 ms for 8192 x 7168 x 7168).
    template <int MF, int NF>
    static constexpr int pitch() { return NF * 64 + 16; }   // bytes of a token's sums
    template <int MF, int NF, bool GLU, bool>
    static constexpr int finish_bytes() { return 4 * MF * 8 * pitch<MF, NF>(); }
    template <int MF, int NF, bool GLU, bool>
    static __device__ __forceinline__ void finish(const Bf16Args &g, Acc (&acc)[MF][NF], u32x4_t *lds, int m0, int nb0, int wv)
    {
        const int lane = threadIdx.x & (WAVE - 1), fa = wv / 2 * MF, fb = wv % 2 * NF;
        constexpr int PITCH = pitch<MF, NF>(), PIECES = (GLU ? NF / 2 : NF) * 2;   // pieces of a row
        constexpr int ROUNDS = MF * 8 * PIECES / WAVE, G = ROUNDS % 4 == 0 ? 4 : ROUNDS % 2 == 0 ? 2 : 1;
        static_assert(ROUNDS * WAVE == MF * 8 * PIECES && ROUNDS % G == 0, "whole rounds");
        uint8_t *stage = reinterpret_cast<uint8_t *>(lds) + wv * (MF * 8 * PITCH);
        const int n1 = (nb0 + fb) / (GLU ? 2 : 1) * 16;   // first output column of this wave
#pragma unroll
        for (int half = 0; half < 2; half++) {
            const int r1 = m0 + fa * 16 + half * MF * 8;
            Piece next[G];
            auto load = [&](int round) {
#pragma unroll
                for (int i = 0; i < G; i++) {
                    const int p = (round + i) * WAVE + lane;
                    next[i].load(g, r1 + p / PIECES, n1 + p % PIECES * 8);
                }
            };
            load(0);
#pragma unroll
            for (int f = 0; f < MF / 2; f++)
#pragma unroll
                for (int j = 0; j < NF; j++)
                    *reinterpret_cast<f32x4_t *>(stage + (f * 16 + (lane & 15)) * PITCH + j * 64 + (lane >> 4) * 16) =
                        acc[half * MF / 2 + f][j];
            meet_lanes();
#pragma unroll 1
            for (int round = 0; round < ROUNDS; round += G) {
                Piece now[G];
#pragma unroll
                for (int i = 0; i < G; i++)
                    now[i] = next[i];
                if (round + G < ROUNDS)
                    load(round + G);
#pragma unroll
                for (int i = 0; i < G; i++) {
                    const int p = (round + i) * WAVE + lane, r = p / PIECES, c = p % PIECES, n = n1 + c * 8;
                    const uint8_t *at = stage + r * PITCH + (GLU ? c / 2 * 128 + c % 2 * 32 : c * 32);
                    if (r1 + r >= g.T || n >= g.N)
                        continue;
                    float v[8], up[8];
                    __builtin_memcpy(v, __builtin_assume_aligned(at, 16), 32);
                    if constexpr (GLU)
                        __builtin_memcpy(up, __builtin_assume_aligned(at + 64, 16), 32);
                    else if (g.bias) {   // padded to 16 columns
                        float b[8];
                        __builtin_memcpy(b, __builtin_assume_aligned(g.bias + n, 16), 32);
#pragma unroll
                        for (int e = 0; e < 8; e++)
                            v[e] += b[e];
                    }
                    with_activation(g.act, [&](auto act) {
#pragma unroll
                        for (int e = 0; e < 8; e++)
                            v[e] = activated<act>(v[e]);
                    });
                    if constexpr (GLU)
#pragma unroll
                        for (int e = 0; e < 8; e++)
                            v[e] *= up[e];
                    if (g.residual)
                        now[i].add(g, v);
                    store8(g, r1 + r, n, v);
                }
            }
            meet_lanes();
        }
    }
};

} // namespace

bool bf16_takes_any_rows(const Bf16Args &g) { return any_rows(g); }

hipError_t launch_bf16_product(const Bf16Args &g, hipStream_t st) { return launch_product<Bf16>(g, st); }

} // namespace mxmoe
