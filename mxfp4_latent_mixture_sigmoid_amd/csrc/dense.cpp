// dense.cpp -- the C ABI of the dense 8-bit path declared in include/mxmoe.h: validation, packed-buffer
// and workspace layouts, launches on the caller's stream.
#include "dense.hpp"

#include <climits>
#include <new>

using namespace mxmoe;

struct moe_linear {
    moe_linear_config cfg;
    uint8_t *blocks;
    const float *scales, *bias;
};

namespace {

bool aligned(const void *p, uintptr_t a) { return (uintptr_t)p % a == 0; }
int64_t align_up(int64_t v) { return (v + 255) / 256 * 256; }
moe_status hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

bool valid_type(int32_t t) { return t == MOE_TYPE_BF16 || t == MOE_TYPE_F32; }
uintptr_t type_size(int32_t t) { return t == MOE_TYPE_F32 ? 4 : 2; }

// One thread per 16 values, fewer than 2^32 in a launch.
bool chunks_fit(int64_t rows, int64_t width) { return rows * ((width + 15) / 16) <= (int64_t)UINT32_MAX - 256; }

// A given matrix: rows at least `width` apart, element-aligned.
bool valid_rows(const void *p, int64_t ld, int64_t width, uintptr_t size) { return p && ld >= width && aligned(p, size); }

struct LinearLayout {
    int64_t scales, bias, total;
};

LinearLayout linear_layout(const moe_linear_config *c)
{
    const int64_t nblk = i8_row_blocks(c->n, c->glu);
    LinearLayout L;
    L.scales = align_up(nblk * i8_stages(c->k) * I8_STAGE_BYTES);
    L.bias = align_up(L.scales + nblk * 16 * 4);
    L.total = align_up(L.bias + nblk * 16 * 4);
    return L;
}

bool valid_linear(const moe_linear_config *c)
{
    return c && c->n >= 1 && c->k >= 1 && (c->glu == 0 || c->glu == 1) && valid_type(c->out_type);
}

// The sum fits 32 bits, and the packing kernel's launch (a thread per 16 codes) and the packed rows their indexes.
bool supported_linear(const moe_linear_config *c)
{
    const int64_t nblk = i8_row_blocks(c->n, c->glu);
    return c->k <= MOE_LINEAR_MAX_K && nblk * 16 <= INT32_MAX / 2 && chunks_fit(nblk * 16, i8_stages(c->k) * I8_STAGE);
}

// Whether the products' direct loads to LDS can take the activations as they are: rows at 16-byte steps from a
// 16-byte aligned address, K whole 16-byte chunks, a tile's rows within one load window. Others go
// through registers or, in large products, are first laid out in the workspace.
constexpr int64_t LD_MAX = 1 << 22;
bool direct(const int8_t *x, int64_t ldx, int64_t K) { return aligned(x, 16) && ldx % 16 == 0 && K % 16 == 0 && ldx <= LD_MAX; }

int64_t workspace_bytes_for(const moe_linear_config *c, int64_t T) { return align_up(T * i8_stages(c->k) * I8_STAGE); }

// More than a round of workgroups comes in tiles of 128 columns at least and of 128 rows or all there are, of 512
// threads at most; restaging takes a thread per 16 codes.
constexpr int64_t XCD_PAD = 8;   // the grid is rounded up to the XCDs
bool linear_fits(const moe_linear_config *c, int64_t T)
{
    const int64_t tiles = ((T + 127) / 128) * ((i8_row_blocks(c->n, c->glu) + 7) / 8);
    return tiles < (UINT32_MAX / 512) - XCD_PAD && chunks_fit(T, i8_stages(c->k) * I8_STAGE);
}

} // namespace

extern "C" {

moe_status moe_norm(const moe_norm_args *a, void *stream)
{
    if (!a || a->T < 0 || a->H < 1 || !valid_type(a->x_type) || !(a->eps >= 0.f))
        return MOE_ERR_INVALID_ARG;
    if (a->H > MOE_MAX_WIDTH)
        return MOE_ERR_UNSUPPORTED;
    if (a->T == 0)
        return MOE_OK;
    if ((!a->sum && !a->out && !a->codes) || !a->codes != !a->scales)
        return MOE_ERR_INVALID_ARG;
    const uintptr_t sz = type_size(a->x_type);
    if (!valid_rows(a->x, a->ldx, a->H, sz) || (a->delta && !valid_rows(a->delta, a->ldd, a->H, 2)) ||
        (a->weight && !aligned(a->weight, 2)) || (a->sum && !valid_rows(a->sum, a->lds, a->H, sz)) ||
        (a->out && !valid_rows(a->out, a->ldo, a->H, 2)) ||
        (a->codes && (a->ldc < a->H || !aligned(a->scales, 4))) || (a->sum == a->x && a->lds != a->ldx))
        return MOE_ERR_INVALID_ARG;
    return hip_status(launch_norm(*a, true, static_cast<hipStream_t>(stream)));
}

moe_status moe_quantise(const void *x, int32_t x_type, int64_t ldx, int32_t T, int32_t K, int8_t *codes, int64_t ldc,
                        float *scales, void *stream)
{
    if (T < 0 || K < 1 || !valid_type(x_type))
        return MOE_ERR_INVALID_ARG;
    if (K > MOE_MAX_WIDTH)
        return MOE_ERR_UNSUPPORTED;
    if (T == 0)
        return MOE_OK;
    if (!valid_rows(x, ldx, K, type_size(x_type)) || !valid_rows(codes, ldc, K, 1) || !scales || !aligned(scales, 4))
        return MOE_ERR_INVALID_ARG;
    moe_norm_args a{};
    a.x = x;
    a.ldx = ldx;
    a.x_type = x_type;
    a.T = T;
    a.H = K;
    a.codes = codes;
    a.ldc = ldc;
    a.scales = scales;
    return hip_status(launch_norm(a, false, static_cast<hipStream_t>(stream)));
}

moe_status moe_dequantise(const int8_t *codes, int64_t ldc, const float *scales, int32_t T, int32_t K, void *out,
                          int64_t ldo, void *stream)
{
    if (T < 0 || K < 1)
        return MOE_ERR_INVALID_ARG;
    if (K > MOE_MAX_WIDTH)
        return MOE_ERR_UNSUPPORTED;
    if (T == 0)
        return MOE_OK;
    if (!valid_rows(codes, ldc, K, 1) || !scales || !aligned(scales, 4) || !valid_rows(out, ldo, K, 2))
        return MOE_ERR_INVALID_ARG;
    return hip_status(launch_dequantise(codes, ldc, scales, T, K, static_cast<uint16_t *>(out), ldo,
                                        static_cast<hipStream_t>(stream)));
}

moe_status moe_linear_query(const moe_linear_config *cfg, int32_t T_max, size_t *packed_bytes, size_t *workspace_bytes)
{
    if (!valid_linear(cfg) || T_max < 0)
        return MOE_ERR_INVALID_ARG;
    if (!supported_linear(cfg))
        return MOE_ERR_UNSUPPORTED;
    if (!linear_fits(cfg, T_max))
        return MOE_ERR_INVALID_ARG;
    if (packed_bytes)
        *packed_bytes = (size_t)linear_layout(cfg).total;
    if (workspace_bytes)
        *workspace_bytes = (size_t)workspace_bytes_for(cfg, T_max);
    return MOE_OK;
}

moe_status moe_linear_create(const moe_linear_config *cfg, const moe_linear_weights *w, void *packed, size_t packed_bytes,
                             void *stream, moe_linear **out)
{
    if (out)
        *out = nullptr;
    if (!out || !valid_linear(cfg) || !w || !packed || !aligned(packed, 256))
        return MOE_ERR_INVALID_ARG;
    if (!supported_linear(cfg))
        return MOE_ERR_UNSUPPORTED;
    if (!w->w || !w->scales || !w->w_up != !cfg->glu || !w->scales_up != !cfg->glu || (cfg->glu && w->bias))
        return MOE_ERR_INVALID_ARG;
    if (!aligned(w->scales, 4) || !aligned(w->scales_up, 4) || !aligned(w->bias, 4))
        return MOE_ERR_INVALID_ARG;
    const LinearLayout L = linear_layout(cfg);
    if (packed_bytes < (size_t)L.total)
        return MOE_ERR_BUFFER_TOO_SMALL;
    moe_linear *l = new (std::nothrow) moe_linear;
    if (!l)
        return MOE_ERR_HIP;
    uint8_t *p = static_cast<uint8_t *>(packed);
    float *scales = reinterpret_cast<float *>(p + L.scales), *bias = reinterpret_cast<float *>(p + L.bias);
    l->cfg = *cfg;
    l->blocks = p;
    l->scales = scales;
    l->bias = w->bias ? bias : nullptr;
    const moe_status st = hip_status(launch_i8_pack(*cfg, *w, p, scales, bias, static_cast<hipStream_t>(stream)));
    if (st != MOE_OK) {
        delete l;
        return st;
    }
    *out = l;
    return MOE_OK;
}

moe_status moe_linear_forward(moe_linear *l, const int8_t *x, int64_t ldx, const float *scales, int32_t T, void *out,
                              int64_t ldo, void *workspace, size_t workspace_bytes, void *stream)
{
    if (!l || T < 0 || !linear_fits(&l->cfg, T))
        return MOE_ERR_INVALID_ARG;
    if (T == 0)
        return MOE_OK;
    const moe_linear_config *c = &l->cfg;
    if (!valid_rows(x, ldx, c->k, 1) || !scales || !aligned(scales, 4) ||
        !valid_rows(out, ldo, c->n, type_size(c->out_type)) || !aligned(workspace, 256) ||
        (!workspace && workspace_bytes))
        return MOE_ERR_INVALID_ARG;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    I8Args g{};
    g.x = x;
    g.ldx = ldx;
    g.sx = scales;
    g.w = l->blocks;
    g.sw = l->scales;
    g.bias = l->bias;
    g.out = out;
    g.ldo = ldo;
    g.T = T;
    g.N = c->n;
    g.K = c->k;
    g.nblk = (int)i8_row_blocks(c->n, c->glu);
    g.glu = c->glu;
    g.out_type = c->out_type;
    g.direct = direct(x, ldx, c->k);
    if (!g.direct && !i8_takes_any_rows(g)) {
        if (workspace_bytes < (size_t)workspace_bytes_for(c, T))
            return MOE_ERR_BUFFER_TOO_SMALL;
        int8_t *staged = static_cast<int8_t *>(workspace);
        const hipError_t e = launch_i8_restage(x, ldx, T, c->k, staged, st);
        if (e != hipSuccess)
            return MOE_ERR_HIP;
        g.x = staged;
        g.ldx = g.K = (int)(i8_stages(c->k) * I8_STAGE);
        g.direct = 1;
    }
    return hip_status(launch_i8_product(g, st));
}

void moe_linear_destroy(moe_linear *l) { delete l; }

} // extern "C"
