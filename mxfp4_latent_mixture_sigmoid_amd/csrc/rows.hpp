// rows.hpp -- what the kernels share that keep rows in registers (8 consecutive values per thread and load): loads and
// stores of any alignment, codes of a row, reductions over a row's threads, and norms of rows whose squares
// leave FP32's range.
#pragma once

#include "dense.hpp"
#include "wave.hpp"

namespace mxmoe {

constexpr int CHUNK = 8;   // consecutive values per thread and load
constexpr int MANY_ROWS = 1024;   // from here on the rows alone keep the card busy

// Rows need not be aligned beyond their element size: the copies below compile to one wide global
// access, which gfx950 serves at any byte address.
template <typename T>
__device__ inline T load_any(const void *p)
{
    T v;
    __builtin_memcpy(&v, p, sizeof(T));
    return v;
}
template <typename T>
__device__ inline void store_any(void *p, const T &v) { __builtin_memcpy(p, &v, sizeof(T)); }
// The residual stream and the normalised BF16 rows leave past the caches: 8192 x 2048 rows with every output
// 31 -> 24 us, 1024 x 14336 30 -> 22, 8192 x 7168 97 -> 91. The codes stay cached for the product that
// reads them next (norm and reading back of 8192 x 7168: 109 us with both cached, 112 with neither, 105 so).
template <typename T>
__device__ inline void store_streamed(void *p, const T &v)
{
    typedef T Any __attribute__((aligned(1)));
    __builtin_nontemporal_store(v, static_cast<Any *>(p));
}

// CHUNK BF16 values from column c on of a row of n values (zeros past n).
__device__ inline u32x4_t load_bf16(const uint16_t *row, int c, int n)
{
    if (c + CHUNK <= n)
        return load_any<u32x4_t>(row + c);
    u32x4_t r;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t lo = c + 2 * i < n ? row[c + 2 * i] : 0, hi = c + 2 * i + 1 < n ? row[c + 2 * i + 1] : 0;
        r[i] = lo | hi << 16;
    }
    return r;
}
__device__ inline void unpack(u32x4_t r, float *v)
{
#pragma unroll
    for (int i = 0; i < 4; i++) {
        v[2 * i] = __uint_as_float(r[i] << 16);
        v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
    }
}

// The same as FP32, of either type.
__device__ inline void load_row(const uint16_t *row, int c, int n, float *v) { unpack(load_bf16(row, c, n), v); }
__device__ inline void load_row(const float *row, int c, int n, float *v)
{
    if (c + CHUNK <= n) {
        const f32x4_t a = load_any<f32x4_t>(row + c), b = load_any<f32x4_t>(row + c + 4);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[i] = a[i];
            v[4 + i] = b[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < CHUNK; i++)
            v[i] = c + i < n ? row[c + i] : 0.f;
    }
}

__device__ inline void store_row(uint16_t *row, int c, int n, const float *v)
{
    u32x4_t r;
#pragma unroll
    for (int i = 0; i < 4; i++)
        r[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    if (c + CHUNK <= n) {
        store_streamed(row + c, r);
    } else {
#pragma unroll
        for (int i = 0; i < CHUNK; i++)
            if (c + i < n)
                row[c + i] = (uint16_t)(r[i / 2] >> (16 * (i % 2)));
    }
}
__device__ inline void store_row(float *row, int c, int n, const float *v)
{
    if (c + CHUNK <= n) {
        store_streamed(row + c, f32x4_t{v[0], v[1], v[2], v[3]});
        store_streamed(row + c + 4, f32x4_t{v[4], v[5], v[6], v[7]});
    } else {
#pragma unroll
        for (int i = 0; i < CHUNK; i++)
            if (c + i < n)
                row[c + i] = v[i];
    }
}
// What takes a row's values to their codes: code = v / scale to nearest even.
struct Coder {
    float up;               // what v and scale are multiplied by first; 0 for a row without codes
    float scale, inverse;   // of the multiplied values; the inverse to a unit or so
};

// Codes: the FP32 quotient v / scale, rounded to nearest even. v * inverse is off by up to 1.5 units, which puts some
// quotients next to a half on its other side (310 of 117 M codes of normal values); one step with the exact remainder
// gives the quotient's own rounding. (|v| is at most 127 scales up to rounding, which the last step takes back.)
// Adding 1.5 x 2^23 leaves the whole number in the low bits. With a rounding and a conversion in its place 8192 x 14336
// BF16 rows took 9% longer.
__device__ inline uint32_t code_bits(float v, const Coder &k)
{
    const float near = v * k.inverse;
    return __float_as_uint(fmaf(fmaf(-near, k.scale, v), k.inverse, near) + 0x1.8p23f);
}
__device__ inline uint32_t four_codes(const float *v, const Coder &k)
{
    constexpr uint32_t PAIR = 0x0C0C0400u, HALVES = 0x05040100u;   // low bytes, then low halves, of second:first
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(code_bits(v[3], k), code_bits(v[2], k), PAIR),
                                 __builtin_amdgcn_perm(code_bits(v[1], k), code_bits(v[0], k), PAIR), HALVES);
}
__device__ inline void store_codes(int8_t *row, int c, int n, float *v, const Coder &k)
{
    if (k.up != 1.f)   // the same in the whole row, and rare
#pragma unroll
        for (int i = 0; i < CHUNK; i++)
            v[i] = k.up != 0.f ? v[i] * k.up : 0.f;
    const uint2 r{four_codes(v, k), four_codes(v + 4, k)};
    if (c + CHUNK <= n) {
        store_any(row + c, r);
    } else {
#pragma unroll
        for (int i = 0; i < CHUNK; i++)
            if (c + i < n)
                row[c + i] = (int8_t)((i < 4 ? r.x : r.y) >> (8 * (i % 4)));
    }
}

// Reductions over the NT threads of a row, in a fixed order; every thread gets the result. `sh` holds
// one word per wave (and chunk) and is not reused by the other reduction.
//
// The sum is over part[i] of chunk t + i * NT of each thread t: each 64 consecutive chunks by their wave, then
// those sums as lanes of one wave, in their place in the row. So it is the same bits whatever NT and NV, and a row's
// norm does not depend on how many rows come with it, which the choice of the two looks at. (Adding a thread's chunks
// up first saves a wave sum and no time: 8192 x 7168 sum and codes 74 us both. Adding the waves' sums one by one took
// 16 registers more with 32 of them, and with those half of the waves: 8192 x 12288 223 us against 154.)
template <int NT, int NV>
__device__ inline float row_sum(const float *part, float *sh)
{
    constexpr int SUMS = NV * (NT / WAVE);
    static_assert(SUMS <= WAVE, "one for each lane");
    const int lane = threadIdx.x & (WAVE - 1);
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const float sum = wave_sum_f32(part[i]);
        if (NT == WAVE)
            v += sum;
        else if (lane == 0)
            sh[i * (NT / WAVE) + threadIdx.x / WAVE] = sum;
    }
    if constexpr (NT > WAVE) {
        __syncthreads();
        v = wave_sum_f32(lane < SUMS ? sh[lane] : 0.f);
    }
    return v;
}
template <int NT>
__device__ inline uint32_t row_max(uint32_t v, uint32_t *sh)
{
    v = wave_max_u32(v);
    if constexpr (NT > WAVE) {
        if ((threadIdx.x & (WAVE - 1)) == 0)
            sh[threadIdx.x / WAVE] = v;
        __syncthreads();
        v = 0u;
#pragma unroll
        for (int w = 0; w < NT / WAVE; w++)
            v = max(v, sh[w]);
    }
    return v;
}

// Scale of a row from the bits of its largest magnitude (as unsigned integers magnitudes order like
// their values, with infinities and then NaNs above), and what takes a value to its code: tiny rows are lifted
// first, so that their scale has all its bits and its inverse is finite.
__device__ inline float row_scale(uint32_t top, Coder &k)
{
    k = Coder{0.f, 0.f, 0.f};
    if (top == 0u)
        return 0.f;
    if (top >= 0x7F800000u)
        return __uint_as_float(0x7FC00000u);
    float m = __uint_as_float(top);
    k.up = m < 0x1p-60f ? 0x1p80f : 1.f;
    const float stored = m / 127.f;
    m *= k.up;
    k.scale = m / 127.f;
    k.inverse = 127.f / m;   // not of the scale, which would have to be waited for
    return stored;
}

// 1 / sqrt(mean(s^2) + eps) for rows whose squares leave FP32's range: sums past it (values of 2e17 and more in a row
// of 7168) would take the whole row to zero, and squares below it are lost where mean + eps is under 2^-120 (with an
// eps that small). Such a row's squares are taken of its values times 2^-80 or 2^100, where no sum of the widest row
// leaves the range again. The power is given back last for the large, y = s * rstd * 2^-80, and first for the
// small, y = s * 2^100 * rstd, so that no product underflows that y does not. Rows with a NaN or an infinity come
// here too, and have the same outputs as without it.
struct Far {
    float squares;         // what values are multiplied by before they are squared
    float before, after;   // and before and after they are multiplied by rstd
};
__device__ inline bool in_range(float mean_eps) { return mean_eps >= 0x1p-120f && mean_eps < __builtin_inff(); }
__device__ inline Far far_factors(float mean_eps)
{
    return mean_eps < 0x1p-120f ? Far{0x1p100f, 0x1p100f, 1.f} : Far{0x1p-80f, 1.f, 0x1p-80f};
}
__device__ inline float far_rstd(float sum, float H, float eps, const Far &f)
{
    return 1.f / sqrtf(sum / H + eps * f.squares * f.squares);
}

// A launch has fewer than 2^32 threads: more rows go in several launches.
constexpr int MAX_ROWS = 1 << 21;

// p, `bytes` further; null stays null.
template <typename P>
inline P *advanced(P *p, int64_t bytes)
{
    return p ? reinterpret_cast<P *>(reinterpret_cast<uintptr_t>(p) + bytes) : p;
}

} // namespace mxmoe
