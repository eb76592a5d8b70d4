// bf16.hip -- dense products of BF16 values with bias, activation and residual in their epilogue,
//   out[t, n] = a(sum_k x[t, k] w[n, k] + bias[n]) + residual[t, n],
// and their gated form a(gate) * up + residual, on the 16x16x32 BF16 matrix-core instruction; kernels in products.hpp.
//
// Sums are FP32, in an order that depends on the sizes (the tile and how many groups of waves share K), never on
// timing; bias, activation, gate and residual are FP32, and the result is rounded once to its type.
#include "products.hpp"

namespace mxmoe {

namespace {

// v / (1 + exp(-v)) on the hardware's exponential and reciprocal, each within a unit in the last place; the rounding of the
// exponent adds |v| 2^-23 relative. exp overflows to infinity, whose reciprocal is 0.
__device__ inline float silu_of(float gate, float v)
{
    return v * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * gate));
}

__device__ inline float activated(float v, int act)
{
    switch (act) {
    case MOE_LINEAR_SILU:
        return silu_of(v, v);
    case MOE_LINEAR_GELU:
        return 0.5f * v * (1.f + erff(0.70710678f * v));
    case MOE_LINEAR_GELU_TANH:   // v / 2 (1 + tanh(c)) = v / (1 + exp(-2 c))
        return silu_of(1.59576912f * fmaf(0.044715f * v * v, v, v), v);
    case MOE_LINEAR_RELU:
        return v < 0.f ? 0.f : v;   // NaN stays
    default:
        return v;
    }
}

// N consecutive values of row r of the residual from column n on, zeros past the end.
template <int N>
__device__ inline void load_residual(const Bf16Args &g, int r, int n, float *v)
{
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

struct Bf16 {
    using Args = Bf16Args;
    using Acc = f32x4_t;
    static constexpr bool APART = false;
    static __device__ Acc mfma(u32x4_t a, u32x4_t b, Acc c) { return mfma16(as_bf16x8(a), as_bf16x8(b), c); }
    static __device__ void mfma_acc(u32x4_t a, u32x4_t b, Acc &acc)
    {
        asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
    }

    // What one fragment's outputs take besides its sums, for lane l's token row l % 16 and the columns 4 (l / 16) .. +3
    // of row block nb. The residual may be the output itself: the lane that reads an element here is the one that writes it.
    struct Factors {
        f32x4_t bias, residual;
    };
    static __device__ Factors load_factors(const Bf16Args &g, int r, int nb)
    {
        const int q = (threadIdx.x & (WAVE - 1)) >> 4, n = (g.glu ? nb / 2 : nb) * 16 + 4 * q;
        Factors v{{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        if (nb >= g.nblk)
            return v;
        if (g.bias)
            v.bias = *reinterpret_cast<const f32x4_t *>(g.bias + n);
        float res[4];
        load_residual<4>(g, r, n, res);
        v.residual = f32x4_t{res[0], res[1], res[2], res[3]};
        return v;
    }

    // Outputs of one fragment of row block nb (a gate block with its up block's sums in `up` when glu).
    static __device__ void emit(const Bf16Args &g, int r, int nb, const Factors &c, Acc sum, Acc up)
    {
        const int q = (threadIdx.x & (WAVE - 1)) >> 4, n = (g.glu ? nb / 2 : nb) * 16 + 4 * q;
        if (r >= g.T || n >= g.N)
            return;
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float a = activated(sum[i] + c.bias[i], g.act);
            v[i] = (g.glu ? a * up[i] : a) + c.residual[i];
        }
        store4(g, r, n, v);
    }

    // Epilogue of the large tiles, 16 tokens at a time through this wave's part of LDS (in FP32, so that the residual is
    // added before the one rounding), to read the residual and store whole 16-byte pieces of rows. Lane (q = l / 16, c =
    // l % 16) of fragment (f, j) holds token 16 f + c and packed columns 16 j + 4 q .. +3; when GLU, fragment j + 1 (odd)
    // holds the up sums of fragment j. The residual of the next 16 tokens is on its way while these are worked on.
    template <int MF, int NF, bool GLU, bool>
    static constexpr int finish_bytes() { return 4 * 16 * ((GLU ? NF / 2 : NF) * 64 + 16); }
    template <int MF, int NF, bool GLU, bool>
    static __device__ void finish(const Bf16Args &g, Acc (&acc)[MF][NF], u32x4_t *lds, int m0, int nb0, int wv)
    {
        const int lane = threadIdx.x & (WAVE - 1), r16 = lane & 15, fa = wv / 2 * MF, fb = wv % 2 * NF;
        constexpr int JO = GLU ? NF / 2 : NF, PITCH = JO * 64 + 16;      // output fragments, bytes of a row in LDS
        constexpr int PIECES = JO * 2, ROUNDS = (16 * PIECES + WAVE - 1) / WAVE;   // of 8 outputs, per row and lane
        uint8_t *stage = reinterpret_cast<uint8_t *>(lds) + wv * (16 * PITCH);
        const int n1 = (nb0 + fb) / (GLU ? 2 : 1) * 16, q4 = 4 * (lane >> 4);   // first output column of this wave
        f32x4_t bias[JO];
#pragma unroll
        for (int j = 0; j < JO; j++)
            bias[j] = !GLU && g.bias ? *reinterpret_cast<const f32x4_t *>(g.bias + min(nb0 + fb + j, g.nblk - 1) * 16 + q4)
                                     : f32x4_t{0.f, 0.f, 0.f, 0.f};
        float res[2][ROUNDS][8];
        auto load = [&](int f) {
#pragma unroll
            for (int i = 0; i < ROUNDS; i++) {
                const int p = i * WAVE + lane, r = p / PIECES;
                load_residual<8>(g, r < 16 ? m0 + (fa + f) * 16 + r : g.T, n1 + p % PIECES * 8, res[f % 2][i]);
            }
        };
        load(0);
#pragma unroll
        for (int f = 0; f < MF; f++) {
            if (f + 1 < MF)
                load(f + 1);
            uint8_t *at = stage + r16 * PITCH + q4 * 4;
#pragma unroll
            for (int j = 0; j < JO; j++) {
                f32x4_t v;
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    if constexpr (GLU)
                        v[e] = activated(acc[f][2 * j][e], g.act) * acc[f][2 * j + 1][e];
                    else
                        v[e] = activated(acc[f][j][e] + bias[j][e], g.act);
                }
                *reinterpret_cast<f32x4_t *>(at + j * 64) = v;
            }
            meet_lanes();
#pragma unroll
            for (int i = 0; i < ROUNDS; i++) {
                const int p = i * WAVE + lane, r = p / PIECES, c = p % PIECES;
                const int row = m0 + (fa + f) * 16 + r, n = n1 + c * 8;
                if (r >= 16 || row >= g.T)
                    continue;
                f32x4_t lo = *reinterpret_cast<const f32x4_t *>(stage + r * PITCH + c * 32);
                f32x4_t hi = *reinterpret_cast<const f32x4_t *>(stage + r * PITCH + c * 32 + 16);
                const float *s = res[f % 2][i];
                lo += f32x4_t{s[0], s[1], s[2], s[3]};
                hi += f32x4_t{s[4], s[5], s[6], s[7]};
                if (g.out_type == MOE_TYPE_F32) {
                    store16(g, row, n, __builtin_bit_cast(u32x4_t, lo));
                    store16(g, row, n + 4, __builtin_bit_cast(u32x4_t, hi));
                } else {
                    store16(g, row, n, u32x4_t{pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]),
                                               pack_bf16x2(hi[0], hi[1]), pack_bf16x2(hi[2], hi[3])});
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
