// norm.hip -- residual addition with RMS norm, quantisation per token, and its reading back.
//
// One pass: a row's values stay in registers, as FP32, from their load to the last output, so each
// input is read once and each output written once; the row's sum of squares and its largest
// magnitude are two reductions over the threads that share the row. Bound by HBM: per value about
// eight FP32 operations for 5 to 13 bytes.
#include "dense.hpp"
#include "wave.hpp"

namespace mxmoe {

namespace {

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

// NT threads per row (64: four rows per workgroup, one per wave; else one workgroup per row), NV
// chunks of 8 values per thread; H <= NT * NV * 8.
template <typename X, int NT, int NV, bool NORM>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void norm_kernel(const moe_norm_args a)
{
    __shared__ float sh_sum[NV * (NT / WAVE)];
    __shared__ uint32_t sh_max[NT / WAVE];
    constexpr int ROWS = NT < 256 ? 256 / NT : 1;
    const int t = threadIdx.x % NT;
    const int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / NT;
    if (ROWS > 1 && r >= a.T)
        return;   // whole waves, and rows of one wave meet no barrier
    const X *x = static_cast<const X *>(a.x) + r * a.ldx;
    float v[NV][CHUNK];
#pragma unroll
    for (int i = 0; i < NV; i++)
        load_row(x, (t + i * NT) * CHUNK, a.H, v[i]);
    if constexpr (NORM) {
        u32x4_t weight[NV];   // loaded before anything waits or is stored
        if (a.weight)
#pragma unroll
            for (int i = 0; i < NV; i++)
                weight[i] = load_bf16(static_cast<const uint16_t *>(a.weight), (t + i * NT) * CHUNK, a.H);
        if (a.delta) {
            const uint16_t *d = static_cast<const uint16_t *>(a.delta) + r * a.ldd;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                float w[CHUNK];
                load_row(d, (t + i * NT) * CHUNK, a.H, w);
#pragma unroll
                for (int j = 0; j < CHUNK; j++)
                    v[i][j] += w[j];
            }
        }
        if (a.sum) {
            X *s = static_cast<X *>(a.sum) + r * a.lds;
#pragma unroll
            for (int i = 0; i < NV; i++)
                store_row(s, (t + i * NT) * CHUNK, a.H, v[i]);
        }
        float ss[NV];
#pragma unroll
        for (int i = 0; i < NV; i++) {
            ss[i] = 0.f;
#pragma unroll
            for (int j = 0; j < CHUNK; j++)
                ss[i] = fmaf(v[i][j], v[i][j], ss[i]);
        }
        const float mean = row_sum<NT, NV>(ss, sh_sum) / (float)a.H + a.eps;
        float rstd = 1.f / sqrtf(mean);
        if (!in_range(mean)) {   // the same in the whole row
            const Far far = far_factors(mean);
#pragma unroll
            for (int i = 0; i < NV; i++) {
                ss[i] = 0.f;
#pragma unroll
                for (int j = 0; j < CHUNK; j++) {
                    const float s = v[i][j] * far.squares;
                    ss[i] = fmaf(s, s, ss[i]);
                }
            }
            if constexpr (NT > WAVE)
                __syncthreads();   // every thread has read the first sums
            rstd = far_rstd(row_sum<NT, NV>(ss, sh_sum), (float)a.H, a.eps, far);
#pragma unroll
            for (int i = 0; i < NV; i++)
#pragma unroll
                for (int j = 0; j < CHUNK; j++)
                    v[i][j] = v[i][j] * far.before * rstd * far.after;
            rstd = 1.f;
        }
#pragma unroll
        for (int i = 0; i < NV; i++) {
            float w[CHUNK];
            if (a.weight)
                unpack(weight[i], w);
#pragma unroll
            for (int j = 0; j < CHUNK; j++)
                v[i][j] = a.weight ? v[i][j] * rstd * w[j] : v[i][j] * rstd;
        }
        if (a.out) {
            uint16_t *o = static_cast<uint16_t *>(a.out) + r * a.ldo;
#pragma unroll
            for (int i = 0; i < NV; i++)
                store_row(o, (t + i * NT) * CHUNK, a.H, v[i]);
        }
        if (!a.codes)
            return;
    }
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int j = 0; j < CHUNK; j++)   // columns past H hold 0, or 0 * rstd = NaN where rstd is not finite
            top = max(top, (t + i * NT) * CHUNK + j < a.H ? __float_as_uint(v[i][j]) & 0x7FFFFFFFu : 0u);
    Coder coder;
    const float scale = row_scale(row_max<NT>(top, sh_max), coder);
    if (t == 0)
        a.scales[r] = scale;
    int8_t *q = a.codes + r * a.ldc;
#pragma unroll
    for (int i = 0; i < NV; i++)
        store_codes(q, (t + i * NT) * CHUNK, a.H, v[i], coder);
}

// Rows longer than the registers of one workgroup hold: three passes over the row, the second and
// third out of cache. `sum` may be x, so it is written in the last pass only.
template <typename X, bool NORM>
__global__ __launch_bounds__(1024) void norm_long_kernel(const moe_norm_args a)
{
    constexpr int NT = 1024;
    static_assert(MOE_MAX_WIDTH <= INT32_MAX - (NT * CHUNK - 1), "the column past the last fits its type");
    __shared__ float sh_sum[NT / WAVE];
    __shared__ uint32_t sh_max[NT / WAVE];
    const int t = threadIdx.x;
    const int64_t r = blockIdx.x;
    const X *x = static_cast<const X *>(a.x) + r * a.ldx;
    const uint16_t *d = static_cast<const uint16_t *>(a.delta) + r * a.ldd;
    auto summed = [&](int c, float *v) {
        load_row(x, c, a.H, v);
        if (NORM && a.delta) {
            float w[CHUNK];
            load_row(d, c, a.H, w);
#pragma unroll
            for (int j = 0; j < CHUNK; j++)
                v[j] += w[j];
        }
    };
    float rstd = 1.f;
    Far far{1.f, 1.f, 1.f};
    if constexpr (NORM) {
        auto squares = [&] {
            // A thread's chunks are added up in 64 bits: in 32, one square after another, the sum of 2^24 equal values was
            // off by 1800 x 2^-24 of itself and that of 2^26 by 0.06%.
            double total = 0.;
            for (int c = t * CHUNK; c < a.H; c += NT * CHUNK) {
                float v[CHUNK], ss = 0.f;
                summed(c, v);
#pragma unroll
                for (int j = 0; j < CHUNK; j++) {
                    const float s = v[j] * far.squares;
                    ss = fmaf(s, s, ss);
                }
                total += ss;
            }
            const float ss = (float)total;
            return row_sum<NT, 1>(&ss, sh_sum);
        };
        const float mean = squares() / (float)a.H + a.eps;
        rstd = 1.f / sqrtf(mean);
        if (!in_range(mean)) {   // the same in the whole row
            far = far_factors(mean);
            __syncthreads();   // every thread has read the first sums
            rstd = far_rstd(squares(), (float)a.H, a.eps, far);
        }
    }
    auto scaled = [&](int c, float *v) {
        if constexpr (NORM) {
            float w[CHUNK];
            if (a.weight)
                load_row(static_cast<const uint16_t *>(a.weight), c, a.H, w);
#pragma unroll
            for (int j = 0; j < CHUNK; j++) {
                const float y = v[j] * far.before * rstd * far.after;
                v[j] = a.weight ? y * w[j] : y;
            }
        }
    };
    Coder coder{0.f, 0.f, 0.f};
    if (a.codes) {
        uint32_t top = 0u;
        for (int c = t * CHUNK; c < a.H; c += NT * CHUNK) {
            float v[CHUNK];
            summed(c, v);
            scaled(c, v);
#pragma unroll
            for (int j = 0; j < CHUNK; j++)
                top = max(top, c + j < a.H ? __float_as_uint(v[j]) & 0x7FFFFFFFu : 0u);
        }
        const float scale = row_scale(row_max<NT>(top, sh_max), coder);
        if (t == 0)
            a.scales[r] = scale;
    }
    for (int c = t * CHUNK; c < a.H; c += NT * CHUNK) {
        float v[CHUNK];
        summed(c, v);
        if (NORM && a.sum)
            store_row(static_cast<X *>(a.sum) + r * a.lds, c, a.H, v);
        scaled(c, v);
        if (NORM && a.out)
            store_row(static_cast<uint16_t *>(a.out) + r * a.ldo, c, a.H, v);
        if (a.codes)
            store_codes(a.codes + r * a.ldc, c, a.H, v, coder);
    }
}

// One chunk of a row per thread.
__global__ __launch_bounds__(256) void dequantise_kernel(const int8_t *codes, int64_t ldc, const float *scales, int K,
                                                         uint32_t chunks, uint32_t total, uint16_t *out, int64_t ldo)
{
    const uint32_t i = blockIdx.x * 256 + threadIdx.x;
    if (i >= total)
        return;
    const int64_t r = i / chunks;
    const int c = (int)(i % chunks) * CHUNK;
    const int8_t *q = codes + r * ldc + c;
    const float s = scales[r];
    uint2 w{0u, 0u};
    if (c + CHUNK <= K) {
        w = load_any<uint2>(q);
    } else {
#pragma unroll
        for (int j = 0; j < CHUNK; j++) {
            const uint32_t b = c + j < K ? (uint8_t)q[j] : 0u;
            (j < 4 ? w.x : w.y) |= b << (8 * (j % 4));
        }
    }
    u32x4_t v;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const uint32_t pair = (j < 2 ? w.x : w.y) >> (16 * (j % 2));
        v[j] = pack_bf16x2((float)(int8_t)pair * s, (float)(int8_t)(pair >> 8) * s);
    }
    uint16_t *o = out + r * ldo + c;
    if (c + CHUNK <= K) {
        store_any(o, v);
    } else {
#pragma unroll
        for (int j = 0; j < CHUNK; j++)
            if (c + j < K)
                o[j] = (uint16_t)(v[j / 2] >> (16 * (j % 2)));
    }
}

// One chunk of 8 values per thread up to 8192 columns, so that a row's loads are all in flight at once and its
// reductions short: 1 x 7168, every output: 1024 threads 4.1 us, 512 with two chunks 4.8, 256 with four
// 6.0; 8192 x 7168 FP32: 134, 139, 152. With many BF16 rows, two chunks keep more bytes in flight: 8192 x 7168 to
// codes 78 us against 85, 8192 x 3000 sum and codes 34 against 41, 8192 x 5120 (320 threads) 51 against 58 with
// 512; and up to 1024 columns a wave with two for any rows: 8192 x 1024 sum and codes 11.9 us against 17.3
// with 256 threads (FP32 19.8 against 18.5), 4 x 1024 the same. 2560 columns by 320 threads: 8192 rows 29 us, by
// 512 35. "Many" is from 1024 rows on; sum and codes with one chunk against two at 256 / 512 / 1000 / 1536 / 4096 rows: 2568
// columns 4.7 : 5.3 / 6.0 : 6.4 / 8.1 : 8.0 / 10.7 : 10.0 / 25.3 : 21.6 us, 4096 4.6 : 4.7 / 5.9 : 6.0 / 8.6 : 8.1 / 11.9 :
// 11.3 / 26.9 : 24.9, 7168 5.7 : 5.8 / 8.3 : 8.2 / 14.3 : 14.4 / 21.5 : 20.9 / 45.7 : 41.4. Where one chunk leaves many
// threads idle (5120 columns) or none (8192), two are ahead from 128 rows on: 7.5 : 6.7 and 8.7 : 8.1 at 512.
template <typename X, bool NORM>
hipError_t launch_rows(const moe_norm_args &a, hipStream_t st)
{
    const dim3 rows((unsigned)a.T), quarter((unsigned)((a.T + 3) / 4));
    const int H = a.H;
    if (H <= 64 * CHUNK) {
        hipLaunchKernelGGL((norm_kernel<X, 64, 1, NORM>), quarter, dim3(256), 0, st, a);
        return hipGetLastError();
    }
    if constexpr (sizeof(X) == 2) {
        const bool many = a.T >= MANY_ROWS;
        if (H <= 64 * CHUNK * 2) {
            hipLaunchKernelGGL((norm_kernel<X, 64, 2, NORM>), quarter, dim3(256), 0, st, a);
            return hipGetLastError();
        }
        if (H > 320 * CHUNK && H <= 256 * CHUNK * 2 && many) {
            hipLaunchKernelGGL((norm_kernel<X, 256, 2, NORM>), rows, dim3(256), 0, st, a);
            return hipGetLastError();
        }
        if (H > 512 * CHUNK && H <= 320 * CHUNK * 2 && many) {
            hipLaunchKernelGGL((norm_kernel<X, 320, 2, NORM>), rows, dim3(320), 0, st, a);
            return hipGetLastError();
        }
        if (H > 512 * CHUNK && H <= 512 * CHUNK * 2 && many) {
            hipLaunchKernelGGL((norm_kernel<X, 512, 2, NORM>), rows, dim3(512), 0, st, a);
            return hipGetLastError();
        }
    }
    if (H <= 256 * CHUNK)
        hipLaunchKernelGGL((norm_kernel<X, 256, 1, NORM>), rows, dim3(256), 0, st, a);
    else if (H <= 320 * CHUNK)
        hipLaunchKernelGGL((norm_kernel<X, 320, 1, NORM>), rows, dim3(320), 0, st, a);
    else if (H <= 512 * CHUNK)
        hipLaunchKernelGGL((norm_kernel<X, 512, 1, NORM>), rows, dim3(512), 0, st, a);
    else if (H <= 1024 * CHUNK)
        hipLaunchKernelGGL((norm_kernel<X, 1024, 1, NORM>), rows, dim3(1024), 0, st, a);
    else if (H <= 1024 * CHUNK * 2)
        hipLaunchKernelGGL((norm_kernel<X, 1024, 2, NORM>), rows, dim3(1024), 0, st, a);
    else
        hipLaunchKernelGGL((norm_long_kernel<X, NORM>), rows, dim3(1024), 0, st, a);
    return hipGetLastError();
}

} // namespace

// A launch has fewer than 2^32 threads: more rows go in several launches.
constexpr int MAX_ROWS = 1 << 21;
constexpr int64_t MAX_THREADS = (int64_t)1 << 31;

hipError_t launch_norm(const moe_norm_args &all, bool norm, hipStream_t st)
{
    const int size = all.x_type == MOE_TYPE_F32 ? 4 : 2;
    auto from = [](auto p, int64_t bytes) {   // null stays null
        return p ? reinterpret_cast<decltype(p)>(reinterpret_cast<uintptr_t>(p) + bytes) : p;
    };
    for (int64_t r = 0; r < all.T; r += MAX_ROWS) {
        moe_norm_args a = all;
        a.T = (int32_t)(all.T - r < MAX_ROWS ? all.T - r : MAX_ROWS);
        a.x = from(all.x, r * all.ldx * size);
        a.delta = from(all.delta, r * all.ldd * 2);
        a.sum = from(all.sum, r * all.lds * size);
        a.out = from(all.out, r * all.ldo * 2);
        a.codes = from(all.codes, r * all.ldc);
        a.scales = from(all.scales, r * 4);
        hipError_t e;
        if (a.x_type == MOE_TYPE_F32)
            e = norm ? launch_rows<float, true>(a, st) : launch_rows<float, false>(a, st);
        else
            e = norm ? launch_rows<uint16_t, true>(a, st) : launch_rows<uint16_t, false>(a, st);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

hipError_t launch_dequantise(const int8_t *codes, int64_t ldc, const float *scales, int32_t T, int32_t K, uint16_t *out,
                             int64_t ldo, hipStream_t st)
{
    const int64_t chunks = ((int64_t)K + CHUNK - 1) / CHUNK, rows = MAX_THREADS / chunks;
    for (int64_t r = 0; r < T; r += rows) {
        const int64_t total = (T - r < rows ? T - r : rows) * chunks;
        hipLaunchKernelGGL(dequantise_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, st, codes + r * ldc, ldc,
                           scales + r, K, (uint32_t)chunks, (uint32_t)total, out + r * ldo, ldo);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

} // namespace mxmoe
