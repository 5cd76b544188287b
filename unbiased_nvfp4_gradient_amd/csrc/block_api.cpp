// block_api.cpp -- C ABI of the feed-forward block's operators and of AdamW (include/nvfp4_block.h):
// argument checks and dispatch to the kernels in block_linear.hip, block_act.hip and block_adamw.hip.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <new>
#include <vector>

#include "nvfp4_block.h"

extern "C" hipError_t nvfp4t_mx_linear(const uint8_t *a_codes, const uint8_t *a_scales,
                                       const uint8_t *b_codes, const uint8_t *b_scales, int64_t M,
                                       int64_t n, int64_t K, int tiled, int rotated_pair, int gated,
                                       int act, int type, int bias_type, const void *bias,
                                       const void *residual, int64_t residual_stride, void *y,
                                       void *z, hipStream_t st);
extern "C" size_t nvfp4t_act_workspace(int type, int gated, int64_t rows, int64_t n);
extern "C" hipError_t nvfp4t_act_bwd(int type, int bias_type, int act, int gated, const void *dy,
                                     int64_t dy_stride, const void *z, int64_t z_stride,
                                     int64_t rows, int64_t n, void *dz, void *dbias, float *partial,
                                     hipStream_t st);
extern "C" hipError_t nvfp4t_adamw(const adamw_tensor *tensors, int64_t count,
                                   const adamw_options *options, hipStream_t st);
extern "C" hipError_t nvfp4t_moment_values(const uint8_t *codes, const uint8_t *scales,
                                           int64_t blocks, int second, float *out, hipStream_t st);

namespace {

constexpr int64_t MAX_DIM = (int64_t)1 << 31;
constexpr int64_t MAX_ELEMS = (int64_t)1 << 40;
constexpr int64_t BLOCK8 = 128;

bool fits(int64_t a, int64_t b)
{
    return a < MAX_DIM && b < MAX_DIM && (a == 0 || b <= (MAX_ELEMS - 1) / a);
}

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

uintptr_t bytes_of(int type) { return type == NVFP4_F32 ? 4 : 2; }

int check_device()
{
    int n = 0;
    if (hipGetDeviceCount(&n) != hipSuccess || n <= 0) {
        (void)hipGetLastError();
        return NVFP4_ERR_HIP;
    }
    return NVFP4_OK;
}

int done(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP; }

bool is_finite(double x) { return x - x == 0.0; }

int check_adamw_tensor(const adamw_tensor &t)
{
    if (t.type < NVFP4_F32 || t.type > NVFP4_F16) return NVFP4_ERR_ARG;
    if (t.bits != 32 && t.bits != 8) return NVFP4_ERR_ARG;
    if (t.size < 0) return NVFP4_ERR_SHAPE;
    if (t.size >= MAX_ELEMS) return NVFP4_ERR_ARG;
    if (t.master && t.type == NVFP4_F32) return NVFP4_ERR_ARG;
    if (t.size == 0) return NVFP4_OK;
    if (!t.param || !t.grad || !t.m || !t.v) return NVFP4_ERR_NULL;
    if (t.bits == 8 && (!t.m_scale || !t.v_scale)) return NVFP4_ERR_NULL;
    const uintptr_t moment = t.bits == 8 ? 8 : 4;
    if (!aligned(t.param, bytes_of(t.type)) || !aligned(t.grad, bytes_of(t.type)) ||
        !aligned(t.m, moment) || !aligned(t.v, moment) || !aligned(t.master, 4))
        return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

// Ranges of memory in order, or put in order, and whether two of them overlap.
struct Span { uintptr_t begin, end; };

bool meets(std::vector<Span> &s)
{
    const auto before = [](const Span &a, const Span &b) { return a.begin < b.begin; };
    if (!std::is_sorted(s.begin(), s.end(), before)) std::sort(s.begin(), s.end(), before);
    for (size_t i = 1; i < s.size(); ++i)
        if (s[i].begin < s[i - 1].end) return true;
    return false;
}

void add(std::vector<Span> &s, const void *p, int64_t bytes)
{
    if (p && bytes) s.push_back({(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes});
}

// Whether a tensor that is written shares memory with another one.  Gradients are read only, and
// may share memory with each other, so each is held against the others' sorted spans.  The
// lists of a training step mostly come in the order of their addresses, kind by kind: such
// lists are checked one by one, and together only where the ranges that they cover meet.
int check_overlap(const adamw_tensor *t, int64_t count)
try {
    constexpr int KINDS = 6;
    std::vector<Span> kind[KINDS], grads;
    for (auto &s : kind) s.reserve((size_t)count);
    grads.reserve((size_t)count);
    for (int64_t i = 0; i < count; ++i) {
        const int64_t n = t[i].size, e = n * (int64_t)bytes_of(t[i].type);
        if (n == 0) continue;
        const int64_t blocks = (n + BLOCK8 - 1) / BLOCK8;
        const int64_t moment = t[i].bits == 8 ? blocks * BLOCK8 : n * 4;
        add(kind[0], t[i].param, e);
        add(kind[1], t[i].m, moment);
        add(kind[2], t[i].v, moment);
        if (t[i].bits == 8) {
            add(kind[3], t[i].m_scale, blocks);
            add(kind[4], t[i].v_scale, blocks);
        }
        add(kind[5], t[i].master, n * 4);
        add(grads, t[i].grad, e);
    }
    std::vector<Span> covers, all;
    for (auto &s : kind) {
        if (meets(s)) return NVFP4_ERR_ARG;
        if (!s.empty()) covers.push_back({s.front().begin, s.back().end});
    }
    Span g{UINTPTR_MAX, 0};
    for (const Span &s : grads) g = {std::min(g.begin, s.begin), std::max(g.end, s.end)};
    if (!grads.empty()) covers.push_back(g);
    if (!meets(covers)) return NVFP4_OK;
    for (const auto &s : kind) all.insert(all.end(), s.begin(), s.end());
    if (meets(all)) return NVFP4_ERR_ARG;
    for (const Span &s : grads) {
        // the first written range that ends after the gradient begins
        const auto w = std::partition_point(all.begin(), all.end(),
                                            [&](const Span &x) { return x.end <= s.begin; });
        if (w != all.end() && w->begin < s.end) return NVFP4_ERR_ARG;
    }
    return NVFP4_OK;
} catch (const std::bad_alloc &) {
    return NVFP4_ERR_WORKSPACE;
}

}  // namespace

extern "C" {

int mxfp4_linear_forward(const mxfp4_tensor *a, const mxfp4_tensor *b, int64_t M, int64_t n,
                         int64_t K, int rotated_pair, int gated, int activation, int type,
                         int bias_type, const void *bias, const void *residual,
                         int64_t residual_stride, void *y, void *z, void *stream)
{
    if (!a || !b) return NVFP4_ERR_NULL;
    if ((rotated_pair != 0 && rotated_pair != 1) || (gated != 0 && gated != 1)) return NVFP4_ERR_ARG;
    if ((a->k_tiled != 0 && a->k_tiled != 1) || a->k_tiled != b->k_tiled) return NVFP4_ERR_ARG;
    if (activation < NVFP4_ACT_NONE || activation > NVFP4_ACT_SILU) return NVFP4_ERR_ARG;
    if (type < NVFP4_F32 || type > NVFP4_F16) return NVFP4_ERR_ARG;
    if (bias && bias_type != type && bias_type != NVFP4_F32) return NVFP4_ERR_ARG;
    if (gated && residual) return NVFP4_ERR_ARG;
    if (M < 0 || n < 0 || K < 0) return NVFP4_ERR_SHAPE;
    if (n >= MAX_DIM) return NVFP4_ERR_ARG;
    const int64_t rows = gated ? 2 * n : n;
    if (!fits(M, rows) || !fits(M, K) || !fits(rows, K)) return NVFP4_ERR_ARG;
    if (K % 128 || (residual && M > 1 && residual_stride < n)) return NVFP4_ERR_SHAPE;
    if (residual && M > 1 && !fits(M, residual_stride)) return NVFP4_ERR_ARG;
    const bool empty = M == 0 || n == 0;
    if (!empty && (!y || (K > 0 && (!a->codes || !a->scales || !b->codes || !b->scales))))
        return NVFP4_ERR_NULL;
    if (!aligned(a->codes, 16) || !aligned(b->codes, 16) || !aligned(a->scales, 4) ||
        !aligned(b->scales, 4) || !aligned(y, bytes_of(type)) || !aligned(z, bytes_of(type)) ||
        !aligned(residual, bytes_of(type)) || (bias && !aligned(bias, bytes_of(bias_type))))
        return NVFP4_ERR_ALIGN;
    const int rc = check_device();
    if (rc) return rc;
    if (empty) return NVFP4_OK;
    return done(nvfp4t_mx_linear(a->codes, a->scales, b->codes, b->scales, M, n, K, a->k_tiled,
                                 rotated_pair, gated, activation, type, bias_type, bias, residual,
                                 residual_stride, y, z, static_cast<hipStream_t>(stream)));
}

size_t activation_backward_workspace_bytes(int type, int gated, int64_t rows, int64_t n)
{
    if (rows < 0 || n < 1 || !fits(rows, gated ? 2 * n : n)) return 0;
    return nvfp4t_act_workspace(type, gated, rows, n);
}

int activation_backward(int type, int bias_type, int activation, int gated, const void *dy,
                        int64_t dy_stride, const void *z, int64_t z_stride, int64_t rows,
                        int64_t n, void *dz, void *dbias, void *workspace,
                        size_t workspace_bytes, void *stream)
{
    if (type < NVFP4_F32 || type > NVFP4_F16) return NVFP4_ERR_ARG;
    if (bias_type != type && bias_type != NVFP4_F32) return NVFP4_ERR_ARG;
    if (activation < NVFP4_ACT_NONE || activation > NVFP4_ACT_SILU) return NVFP4_ERR_ARG;
    if (gated != 0 && gated != 1) return NVFP4_ERR_ARG;
    if (rows < 0 || n < 1) return NVFP4_ERR_SHAPE;
    if (n >= MAX_DIM) return NVFP4_ERR_ARG;
    const int64_t width = gated ? 2 * n : n;
    const bool reads_z = gated || activation != NVFP4_ACT_NONE;
    if (rows > 1 && (dy_stride < n || (reads_z && z_stride < width))) return NVFP4_ERR_SHAPE;
    if (!fits(rows, width)) return NVFP4_ERR_ARG;
    if (rows > 1 && (!fits(rows, dy_stride) || (reads_z && !fits(rows, z_stride))))
        return NVFP4_ERR_ARG;
    if (rows > 0 && (!dy || !dz || (reads_z && !z))) return NVFP4_ERR_NULL;
    if (!aligned(dy, bytes_of(type)) || !aligned(z, bytes_of(type)) ||
        !aligned(dz, bytes_of(type)) || !aligned(dbias, bytes_of(bias_type)))
        return NVFP4_ERR_ALIGN;
    if (dbias) {
        const size_t need = nvfp4t_act_workspace(type, gated, rows, n);
        if (need && (!workspace || workspace_bytes < need)) return NVFP4_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
    }
    const int rc = check_device();
    if (rc) return rc;
    return done(nvfp4t_act_bwd(type, bias_type, activation, gated, dy, dy_stride, z, z_stride, rows,
                               n, dz, dbias, static_cast<float *>(workspace),
                               static_cast<hipStream_t>(stream)));
}

int adamw_step(const adamw_tensor *tensors, int64_t count, const adamw_options *options,
               void *stream)
{
    if (!options || (count > 0 && !tensors)) return NVFP4_ERR_NULL;
    if (count < 0) return NVFP4_ERR_SHAPE;
    if (count >= (int64_t)1 << 31) return NVFP4_ERR_ARG;
    const adamw_options &o = *options;
    if (!(o.beta1 >= 0.0 && o.beta1 < 1.0) || !(o.beta2 >= 0.0 && o.beta2 < 1.0))
        return NVFP4_ERR_ARG;
    if (!(o.eps >= 0.0) || !is_finite(o.eps) || !(o.weight_decay >= 0.0) || !is_finite(o.weight_decay))
        return NVFP4_ERR_ARG;
    if (!o.lr_device && (!(o.lr >= 0.0) || !is_finite(o.lr))) return NVFP4_ERR_ARG;
    if (!o.step_device && o.step < 1) return NVFP4_ERR_ARG;
    if (o.norm && !(o.max_norm >= 0.0f)) return NVFP4_ERR_ARG;
    if (o.bounded != 0 && o.bounded != 1) return NVFP4_ERR_ARG;
    if (!aligned(o.lr_device, 4) || !aligned(o.step_device, 8) || !aligned(o.norm, 4))
        return NVFP4_ERR_ALIGN;
    for (int64_t i = 0; i < count; ++i) {
        const int rc = check_adamw_tensor(tensors[i]);
        if (rc) return rc;
    }
    int rc = check_overlap(tensors, count);
    if (rc) return rc;
    rc = check_device();
    if (rc) return rc;
    return done(nvfp4t_adamw(tensors, count, options, static_cast<hipStream_t>(stream)));
}

int adamw_moment_values(const uint8_t *codes, const uint8_t *scales, int64_t blocks, int second,
                        float *out, void *stream)
{
    if (second != 0 && second != 1) return NVFP4_ERR_ARG;
    if (blocks < 0) return NVFP4_ERR_SHAPE;
    if (blocks >= MAX_ELEMS / BLOCK8) return NVFP4_ERR_ARG;
    if (blocks > 0 && (!codes || !scales || !out)) return NVFP4_ERR_NULL;
    if (!aligned(codes, 8) || !aligned(out, 4)) return NVFP4_ERR_ALIGN;
    const int rc = check_device();
    if (rc) return rc;
    return done(nvfp4t_moment_values(codes, scales, blocks, second, out,
                                     static_cast<hipStream_t>(stream)));
}

}  // extern "C"
