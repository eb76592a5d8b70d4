// block_norm.hip -- between two blocks of a decoder: the norm after the one, its gate, the scaled residual addition,
// and the norm before the next:
//   n = y / sqrt(mean(y^2) + eps) * post_weight;   s = residual_scale x + scale a(gate) n;
//   out = s / sqrt(mean(s^2) + eps) * weight, in BF16 and / or in 8 bits
//
// One pass, as in norm.hip: a row's x, y and gate are read once into registers, three reductions over the row's
// threads (the two sums of squares, the largest magnitude), every output is written once from FP32 values.
//
// Memory bounds many rows: 8192 x 7168 of FP32 with a gate row and every output, 763 MB, 155 us (4.9 TB/s, nearly a copy's rate); 4096
// rows of BF16 41 us (5.7 TB/s). Few rows take three times a load and a reduction: one row 4.9 us.
#include "rows.hpp"

namespace mxmoe {

namespace {

// exp(v) for a BF16 value of at most 174: v times the upper 15 bits of log2(e) is exact, so the hardware's exponential
// (within a unit in the last place) has an exact argument, and the lower bits are a factor next to one: 2 u and a
// little, where a rounded argument would cost up to 2 |v| u.
__device__ inline float exp_bf16(float v)
{
    constexpr float HIGH = 0x1.7154p0f, LOW = 0x1.d94ae1p-18f /* log2(e) - HIGH */, LN2 = 0x1.62e43p-1f;
    const float e = __builtin_amdgcn_exp2f(v * HIGH);
    return fmaf(e, v * (LOW * LN2), e);
}

// The gate's activation, of a BF16 value. Past 87 both ends of the sigmoid are constant (off by under 2^-125).
__device__ inline float gate_value(float v, int act)
{
    if (act == MOE_GATE_SIGMOID) {
        const float w = v < -87.f ? -87.f : v > 87.f ? 87.f : v;   // NaN stays
        const float g = __builtin_amdgcn_rcpf(1.f + exp_bf16(-w));
        return v < -87.f ? 0.f : g;
    }
    if (act == MOE_GATE_TANH) {
        // Taylor's series below 0.35, where its next term is under 2^-26 of the value; 1 - 2 / (exp(2 |v|) + 1) above,
        // where the difference has lost less than two bits
        const float a = fabsf(v), q = v * v;
        if (a < 0.35f)
            return fmaf(v * q, fmaf(q, fmaf(q, fmaf(q, fmaf(q, -1382.f / 155925, 62.f / 2835), -17.f / 315), 2.f / 15),
                                    -1.f / 3), v);
        const float t = a > 20.f ? 20.f : a;
        return copysignf(fmaf(-2.f, __builtin_amdgcn_rcpf(exp_bf16(2.f * t) + 1.f), 1.f), v);
    }
    return v;
}

// s of one value. Every kernel takes these steps, so that a row's outputs are the same bits in any batch.
__device__ inline float mixed(const moe_block_norm_args &a, float x, float n, float g)
{
#pragma clang fp contract(off)
    return fmaf(a.residual_scale, x, a.scale * g * n);
}

// 1 / sqrt(mean(v^2) + eps) over a row, which each thread holds NV chunks of; rows whose squares leave
// FP32's range are scaled here instead.
template <int NT, int NV>
__device__ inline float row_rstd(float (&v)[NV][CHUNK], float H, float eps, float *sh)
{
    auto squares = [&](float f) {
        float ss[NV];
#pragma unroll
        for (int i = 0; i < NV; i++) {
            ss[i] = 0.f;
#pragma unroll
            for (int j = 0; j < CHUNK; j++) {
                const float s = v[i][j] * f;
                ss[i] = fmaf(s, s, ss[i]);
            }
        }
        return row_sum<NT, NV>(ss, sh);
    };
    const float mean = squares(1.f) / H + eps;
    if (in_range(mean))
        return 1.f / sqrtf(mean);
    const Far far = far_factors(mean);   // the same in the whole row
    if constexpr (NT > WAVE)
        __syncthreads();   // every thread has read the first sums
    const float rstd = far_rstd(squares(far.squares), H, eps, far);
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int j = 0; j < CHUNK; j++)
            v[i][j] = v[i][j] * far.before * rstd * far.after;
    return 1.f;
}

// NT threads per row (64: four rows per workgroup, one per wave; else one workgroup per row), NV chunks of 8
// values per thread; H <= NT * NV * 8.
template <typename X, int NT, int NV>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void block_norm_kernel(const moe_block_norm_args a)
{
    __shared__ float sh_post[NV * (NT / WAVE)], sh_sum[NV * (NT / WAVE)];
    __shared__ uint32_t sh_max[NT / WAVE];
    constexpr int ROWS = NT < 256 ? 256 / NT : 1;
    const int t = threadIdx.x % NT;
    const int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / NT;
    if (ROWS > 1 && r >= a.T)
        return;   // whole waves, and rows of one wave meet no barrier
    const X *x = static_cast<const X *>(a.x) + r * a.ldx;
    const uint16_t *y = static_cast<const uint16_t *>(a.y) + r * a.ldy;
    const uint16_t *gate = static_cast<const uint16_t *>(a.gate) + r * a.ldg;
    const bool wide = a.gate && a.gate_width > 1;
    // everything is loaded before anything waits
    u32x4_t raw[NV], open[NV], post[NV], weight[NV];
    float v[NV][CHUNK], n[NV][CHUNK];
#pragma unroll
    for (int i = 0; i < NV; i++)
        raw[i] = load_bf16(y, (t + i * NT) * CHUNK, a.H);
#pragma unroll
    for (int i = 0; i < NV; i++)
        load_row(x, (t + i * NT) * CHUNK, a.H, v[i]);
    if (wide)
#pragma unroll
        for (int i = 0; i < NV; i++)
            open[i] = load_bf16(gate, (t + i * NT) * CHUNK, a.H);
    if (a.post_weight)
#pragma unroll
        for (int i = 0; i < NV; i++)
            post[i] = load_bf16(static_cast<const uint16_t *>(a.post_weight), (t + i * NT) * CHUNK, a.H);
    if (a.weight)
#pragma unroll
        for (int i = 0; i < NV; i++)
            weight[i] = load_bf16(static_cast<const uint16_t *>(a.weight), (t + i * NT) * CHUNK, a.H);
    const float one = a.gate && !wide ? gate_value(bf16_bits_to_f32(*gate), a.gate_act) : 1.f;
#pragma unroll
    for (int i = 0; i < NV; i++)
        unpack(raw[i], n[i]);
    const float rpost = row_rstd<NT, NV>(n, (float)a.H, a.eps, sh_post);
#pragma unroll
    for (int i = 0; i < NV; i++) {
        float w[CHUNK], g[CHUNK];
        if (a.post_weight)
            unpack(post[i], w);
        if (wide)
            unpack(open[i], g);
#pragma unroll
        for (int j = 0; j < CHUNK; j++) {
            const float z = a.post_weight ? n[i][j] * rpost * w[j] : n[i][j] * rpost;
            v[i][j] = mixed(a, v[i][j], z, wide ? gate_value(g[j], a.gate_act) : one);
        }
    }
    if (a.sum) {
        X *s = static_cast<X *>(a.sum) + r * a.lds;
#pragma unroll
        for (int i = 0; i < NV; i++)
            store_row(s, (t + i * NT) * CHUNK, a.H, v[i]);
    }
    if (!a.out && !a.codes)
        return;
    const float rstd = row_rstd<NT, NV>(v, (float)a.H, a.eps, sh_sum);
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
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int j = 0; j < CHUNK; j++)   // columns past H hold 0, or NaN where a root is not finite
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

// Rows longer than the registers of one workgroup hold: four passes over the row, all but the first out of cache (4096 x 20480 of BF16
// 182 us, 3.7 TB/s, with codes 237; 16384 columns, in one pass, 109 and 139). `sum` may
// be x, so it is written in the last pass only.
template <typename X>
__global__ __launch_bounds__(1024) void block_norm_long_kernel(const moe_block_norm_args a)
{
    constexpr int NT = 1024;
    static_assert(MOE_MAX_WIDTH <= INT32_MAX - (NT * CHUNK - 1), "the column past the last fits its type");
    __shared__ float sh_sum[2][NT / WAVE];
    __shared__ uint32_t sh_max[NT / WAVE];
    const int t = threadIdx.x;
    const int64_t r = blockIdx.x;
    const X *x = static_cast<const X *>(a.x) + r * a.ldx;
    const uint16_t *y = static_cast<const uint16_t *>(a.y) + r * a.ldy;
    const uint16_t *gate = static_cast<const uint16_t *>(a.gate) + r * a.ldg;
    const bool wide = a.gate && a.gate_width > 1;
    const float one = a.gate && !wide ? gate_value(bf16_bits_to_f32(*gate), a.gate_act) : 1.f;
    struct Root {
        float rstd;
        Far far;
    };
    // the row's values are get(c, v); a thread's chunks are added up in 64 bits, see norm.hip
    auto root = [&](auto get, float *sh) {
        auto squares = [&](float f) {
            double total = 0.;
            for (int c = t * CHUNK; c < a.H; c += NT * CHUNK) {
                float v[CHUNK], ss = 0.f;
                get(c, v);
#pragma unroll
                for (int j = 0; j < CHUNK; j++) {
                    const float s = v[j] * f;
                    ss = fmaf(s, s, ss);
                }
                total += ss;
            }
            const float ss = (float)total;
            return row_sum<NT, 1>(&ss, sh);
        };
        Root k{1.f, Far{1.f, 1.f, 1.f}};
        const float mean = squares(1.f) / (float)a.H + a.eps;
        k.rstd = 1.f / sqrtf(mean);
        if (!in_range(mean)) {   // the same in the whole row
            k.far = far_factors(mean);
            __syncthreads();   // every thread has read the first sums
            k.rstd = far_rstd(squares(k.far.squares), (float)a.H, a.eps, k.far);
        }
        return k;
    };
    auto normed = [&](const Root &k, const void *weight, int c, float *v) {
        float w[CHUNK];
        if (weight)
            load_row(static_cast<const uint16_t *>(weight), c, a.H, w);
#pragma unroll
        for (int j = 0; j < CHUNK; j++) {
            const float z = v[j] * k.far.before * k.rstd * k.far.after;
            v[j] = weight ? z * w[j] : z;
        }
    };
    const Root post = root([&](int c, float *v) { load_row(y, c, a.H, v); }, sh_sum[0]);
    auto summed = [&](int c, float *v) {
        float s[CHUNK], g[CHUNK];
        load_row(y, c, a.H, v);
        normed(post, a.post_weight, c, v);
        load_row(x, c, a.H, s);
        if (wide)
            load_row(gate, c, a.H, g);
#pragma unroll
        for (int j = 0; j < CHUNK; j++)
            v[j] = mixed(a, s[j], v[j], wide ? gate_value(g[j], a.gate_act) : one);
    };
    const bool next = a.out || a.codes;
    Root k{1.f, Far{1.f, 1.f, 1.f}};
    if (next)
        k = root(summed, sh_sum[1]);
    Coder coder{0.f, 0.f, 0.f};
    if (a.codes) {
        uint32_t top = 0u;
        for (int c = t * CHUNK; c < a.H; c += NT * CHUNK) {
            float v[CHUNK];
            summed(c, v);
            normed(k, a.weight, c, v);
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
        if (a.sum)
            store_row(static_cast<X *>(a.sum) + r * a.lds, c, a.H, v);
        if (!next)
            continue;
        normed(k, a.weight, c, v);
        if (a.out)
            store_row(static_cast<uint16_t *>(a.out) + r * a.ldo, c, a.H, v);
        if (a.codes)
            store_codes(a.codes + r * a.ldc, c, a.H, v, coder);
    }
}

template <typename X>
hipError_t launch_rows(const moe_block_norm_args &a, hipStream_t st)
{
    // The fewest threads with one chunk each, in whole powers of two; under a row of 1024 one wave takes two, since
    // workgroups that hold four rows need no barrier. 8192 BF16 rows, us: of 512 values 64 x 1 8.0, 256 x 1 19.5; of 1024 64 x 2
    // 12.0, 256 x 1 20.1; of 2048 256 x 1 23.3, 512 x 1 35.4; of 3584 512 x 1 40.1, 256 x 2 43.0. 4096 rows of 7168: 1024 x 1 41.0,
    // 512 x 2 45.7, 256 x 4 48.1.
    const dim3 rows((unsigned)a.T), quarter((unsigned)((a.T + 3) / 4));
    const int H = a.H;
    if (H <= 64 * CHUNK)
        hipLaunchKernelGGL((block_norm_kernel<X, 64, 1>), quarter, dim3(256), 0, st, a);
    else if (H <= 64 * CHUNK * 2)
        hipLaunchKernelGGL((block_norm_kernel<X, 64, 2>), quarter, dim3(256), 0, st, a);
    else if (H <= 256 * CHUNK)
        hipLaunchKernelGGL((block_norm_kernel<X, 256, 1>), rows, dim3(256), 0, st, a);
    else if (H <= 512 * CHUNK)
        hipLaunchKernelGGL((block_norm_kernel<X, 512, 1>), rows, dim3(512), 0, st, a);
    else if (H <= 1024 * CHUNK)
        hipLaunchKernelGGL((block_norm_kernel<X, 1024, 1>), rows, dim3(1024), 0, st, a);
    else if (H <= 1024 * CHUNK * 2)
        hipLaunchKernelGGL((block_norm_kernel<X, 1024, 2>), rows, dim3(1024), 0, st, a);
    else
        hipLaunchKernelGGL((block_norm_long_kernel<X>), rows, dim3(1024), 0, st, a);
    return hipGetLastError();
}

} // namespace

hipError_t launch_block_norm(const moe_block_norm_args &all, hipStream_t st)
{
    const int size = all.x_type == MOE_TYPE_F32 ? 4 : 2;
    for (int64_t r = 0; r < all.T; r += MAX_ROWS) {
        moe_block_norm_args a = all;
        a.T = (int32_t)(all.T - r < MAX_ROWS ? all.T - r : MAX_ROWS);
        a.x = advanced(all.x, r * all.ldx * size);
        a.y = advanced(all.y, r * all.ldy * 2);
        a.gate = advanced(all.gate, r * all.ldg * 2);
        a.sum = advanced(all.sum, r * all.lds * size);
        a.out = advanced(all.out, r * all.ldo * 2);
        a.codes = advanced(all.codes, r * all.ldc);
        a.scales = advanced(all.scales, r * 4);
        const hipError_t e = a.x_type == MOE_TYPE_F32 ? launch_rows<float>(a, st) : launch_rows<uint16_t>(a, st);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

} // namespace mxmoe
