// train_api.cpp -- C ABI of the training-step operators of libnvfp4.so (include/nvfp4_train.h):
// argument checks and dispatch to the kernels in train_norm.hip, train_ce.hip and
// train_clip.hip.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdlib.h>

#include <algorithm>

#include "nvfp4_train.h"

extern "C" size_t nvfp4t_ln_workspace(int type, int64_t rows, int64_t n);
extern "C" hipError_t nvfp4t_ln_fwd(int type, int p_type, const void *x, const void *weight,
                                    const void *bias, int64_t rows, int64_t n, int64_t x_stride,
                                    float eps, void *y, float *mean, float *rstd, hipStream_t st);
extern "C" hipError_t nvfp4t_ln_bwd(int type, int p_type, const void *dy, const void *x,
                                    const float *mean, const float *rstd, const void *weight,
                                    int64_t rows, int64_t n, int64_t dy_stride, int64_t x_stride,
                                    void *dx, void *dw, void *db, float *partial, hipStream_t st);
extern "C" size_t nvfp4t_ce_workspace(int backward, int64_t t, int64_t d, int64_t v);
extern "C" hipError_t nvfp4t_ce_fwd(int type, const void *h, int64_t h_stride, const void *w,
                                    int64_t w_stride, const int64_t *target, int64_t t, int64_t d,
                                    int64_t v, int64_t ignore, int reduction, float *loss,
                                    float *lse, void *workspace, hipStream_t st);
extern "C" hipError_t nvfp4t_ce_bwd(int type, const float *dloss, const void *h, int64_t h_stride,
                                    const void *w, int64_t w_stride, const int64_t *target,
                                    const float *lse, int64_t t, int64_t d, int64_t v,
                                    int64_t ignore, int reduction, void *dh, void *dw,
                                    void *workspace, hipStream_t st);
extern "C" size_t nvfp4t_norm_workspace(const int64_t *sizes, int64_t count);
extern "C" hipError_t nvfp4t_norm(const void *const *in, const int64_t *sizes,
                                  const int32_t *types, int64_t count, int inf, float *norm,
                                  void *workspace, hipStream_t st);
extern "C" hipError_t nvfp4t_clip(const void *const *in, void *const *out, const int64_t *sizes,
                                  const int32_t *types, int64_t count, float max_norm,
                                  const float *norm, hipStream_t st);

namespace {

constexpr int64_t MAX_DIM = (int64_t)1 << 31;
constexpr int64_t MAX_ROWS = (int64_t)1 << 28;
constexpr int64_t MAX_ELEMS = (int64_t)1 << 40;

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

// A workspace of at least `need` bytes (none where need is 0).
int check_workspace(const void *ws, size_t bytes, size_t need, uintptr_t align)
{
    if (need && (!ws || bytes < need)) return NVFP4_ERR_WORKSPACE;
    return aligned(ws, align) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

int check_norm(int type, int p_type, int64_t rows, int64_t n, int64_t stride)
{
    if (type < NVFP4_F32 || type > NVFP4_F16) return NVFP4_ERR_ARG;
    if (p_type != type && p_type != NVFP4_F32) return NVFP4_ERR_ARG;
    if (rows < 0 || n < 1 || (rows > 1 && stride < n)) return NVFP4_ERR_SHAPE;
    if (!fits(rows, n) || (rows > 1 && !fits(rows, stride))) return NVFP4_ERR_ARG;
    return NVFP4_OK;
}

// Tokens and words take up to 8 threads each of a launch, which holds fewer than 2^32; where they
// take more, the kernels walk what is left.
bool loss_fits(int64_t t, int64_t d, int64_t v)
{
    return t < MAX_ROWS && v < MAX_ROWS && fits(t, d) && fits(v, d) && fits(t, v);
}

// Shared by the loss's two passes.
int check_loss(int type, const void *h, int64_t h_stride, const void *w, int64_t w_stride,
               const int64_t *target, int64_t t, int64_t d, int64_t v, int reduction)
{
    if (type != NVFP4_BF16 && type != NVFP4_F16) return NVFP4_ERR_ARG;
    if (reduction < NVFP4_SUM || reduction > NVFP4_NONE) return NVFP4_ERR_ARG;
    if (t < 0 || d < 1 || v < 1) return NVFP4_ERR_SHAPE;
    if ((t > 1 && h_stride < d) || (v > 1 && w_stride < d)) return NVFP4_ERR_SHAPE;
    if (!loss_fits(t, d, v)) return NVFP4_ERR_ARG;
    if ((t > 1 && !fits(t, h_stride)) || (v > 1 && !fits(v, w_stride))) return NVFP4_ERR_ARG;
    if (!w || (t > 0 && (!h || !target))) return NVFP4_ERR_NULL;
    if (!aligned(h, 2) || !aligned(w, 2) || !aligned(target, 8)) return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

int check_tensors(const void *const *tensors, void *const *outs, bool clip, const int64_t *sizes,
                  const int32_t *types, int64_t count, int inf, const float *norm)
{
    if (!norm) return NVFP4_ERR_NULL;
    if (inf != 0 && inf != 1) return NVFP4_ERR_ARG;
    if (count < 0) return NVFP4_ERR_SHAPE;
    if (count > 0 && (!tensors || !sizes || !types || (clip && !outs))) return NVFP4_ERR_NULL;
    if (!aligned(norm, 4)) return NVFP4_ERR_ALIGN;
    for (int64_t i = 0; i < count; ++i) {
        if (types[i] < NVFP4_F32 || types[i] > NVFP4_F16) return NVFP4_ERR_ARG;
        if (sizes[i] < 0) return NVFP4_ERR_SHAPE;
        if (sizes[i] >= MAX_ELEMS) return NVFP4_ERR_ARG;
        if (sizes[i] == 0) continue;
        if (!tensors[i] || (clip && !outs[i])) return NVFP4_ERR_NULL;
        if (!aligned(tensors[i], bytes_of(types[i])) ||
            (clip && !aligned(outs[i], bytes_of(types[i]))))
            return NVFP4_ERR_ALIGN;
    }
    return NVFP4_OK;
}

struct Span { uintptr_t begin, end; };

bool before(const Span &a, const Span &b) { return a.begin < b.begin; }

void in_order(Span *s, int64_t n)
{
    if (!std::is_sorted(s, s + n, before)) std::sort(s, s + n, before);
}

// Whether a tensor that is written shares memory with another one, written or read (one that is
// clipped in place is written only).  The lists of a training step mostly come in the order of
// their addresses: then this is one pass.
int check_overlap(const void *const *tensors, void *const *outs, const int64_t *sizes,
                  const int32_t *types, int64_t count)
{
    if (count == 0) return NVFP4_OK;
    Span *writes = static_cast<Span *>(malloc(2 * (size_t)count * sizeof(Span)));
    if (!writes) return NVFP4_ERR_WORKSPACE;
    Span *reads = writes + count;
    int64_t w = 0, r = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (sizes[i] == 0) continue;
        const uintptr_t bytes = (uintptr_t)sizes[i] * bytes_of(types[i]);
        const uintptr_t o = (uintptr_t)outs[i], t = (uintptr_t)tensors[i];
        writes[w++] = {o, o + bytes};
        if (o != t) reads[r++] = {t, t + bytes};
    }
    in_order(writes, w);
    in_order(reads, r);
    bool found = false;
    for (int64_t i = 1; i < w; ++i) found |= writes[i].begin < writes[i - 1].end;
    // both in order, the writes apart: a read meets the first write that ends after it begins
    for (int64_t i = 0, k = 0; i < r && !found; ++i) {
        while (k < w && writes[k].end <= reads[i].begin) ++k;
        found = k < w && writes[k].begin < reads[i].end;
    }
    free(writes);
    return found ? NVFP4_ERR_ARG : NVFP4_OK;
}

}  // namespace

extern "C" {

int layer_norm_forward(int type, int p_type, const void *x, const void *weight, const void *bias,
                       int64_t rows, int64_t n, int64_t x_stride, float eps, void *y,
                       float *mean, float *rstd, void *stream)
{
    int rc = check_norm(type, p_type, rows, n, x_stride);
    if (rc) return rc;
    if (!(eps >= 0.0f && eps <= 3.40282347e+38f)) return NVFP4_ERR_ARG;
    if (rows > 0 && (!x || !y || !mean || !rstd)) return NVFP4_ERR_NULL;
    if (!aligned(x, bytes_of(type)) || !aligned(y, bytes_of(type)) ||
        !aligned(weight, bytes_of(p_type)) || !aligned(bias, bytes_of(p_type)) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
        return NVFP4_ERR_ALIGN;
    rc = check_device();
    if (rc) return rc;
    return done(nvfp4t_ln_fwd(type, p_type, x, weight, bias, rows, n, x_stride, eps, y, mean, rstd,
                              static_cast<hipStream_t>(stream)));
}

size_t layer_norm_workspace_bytes(int type, int64_t rows, int64_t n)
{
    if (rows < 0 || n < 1 || !fits(rows, n)) return 0;
    return nvfp4t_ln_workspace(type, rows, n);
}

int layer_norm_backward(int type, int p_type, const void *dy, const void *x, const float *mean,
                        const float *rstd, const void *weight, int64_t rows, int64_t n,
                        int64_t dy_stride, int64_t x_stride, void *dx, void *dweight,
                        void *dbias, void *workspace, size_t workspace_bytes, void *stream)
{
    int rc = check_norm(type, p_type, rows, n, x_stride);
    if (rc) return rc;
    rc = check_norm(type, p_type, rows, n, dy_stride);
    if (rc) return rc;
    if (rows > 0 && (!dy || !x || !mean || !rstd || !dx)) return NVFP4_ERR_NULL;
    if (!aligned(x, bytes_of(type)) || !aligned(dy, bytes_of(type)) ||
        !aligned(dx, bytes_of(type)) || !aligned(weight, bytes_of(p_type)) ||
        !aligned(dweight, bytes_of(p_type)) || !aligned(dbias, bytes_of(p_type)) ||
        !aligned(mean, 4) || !aligned(rstd, 4))
        return NVFP4_ERR_ALIGN;
    rc = check_workspace(workspace, workspace_bytes,
                         dweight || dbias ? nvfp4t_ln_workspace(type, rows, n) : 0, 16);
    if (rc) return rc;
    rc = check_device();
    if (rc) return rc;
    return done(nvfp4t_ln_bwd(type, p_type, dy, x, mean, rstd, weight, rows, n, dy_stride,
                              x_stride, dx, dweight, dbias, static_cast<float *>(workspace),
                              static_cast<hipStream_t>(stream)));
}

size_t linear_cross_entropy_workspace_bytes(int backward, int64_t t, int64_t d, int64_t v)
{
    if (t < 0 || d < 1 || v < 1 || !loss_fits(t, d, v)) return 0;
    return nvfp4t_ce_workspace(backward, t, d, v);
}

int linear_cross_entropy_forward(int type, const void *h, int64_t h_stride, const void *w,
                                 int64_t w_stride, const int64_t *target, int64_t t, int64_t d,
                                 int64_t v, int64_t ignore_index, int reduction, float *loss,
                                 float *lse, void *workspace, size_t workspace_bytes,
                                 void *stream)
{
    int rc = check_loss(type, h, h_stride, w, w_stride, target, t, d, v, reduction);
    if (rc) return rc;
    if ((t > 0 && !lse) || ((t > 0 || reduction != NVFP4_NONE) && !loss)) return NVFP4_ERR_NULL;
    if (!aligned(loss, 4) || !aligned(lse, 4)) return NVFP4_ERR_ALIGN;
    rc = check_workspace(workspace, workspace_bytes, nvfp4t_ce_workspace(0, t, d, v), 256);
    if (rc) return rc;
    rc = check_device();
    if (rc) return rc;
    return done(nvfp4t_ce_fwd(type, h, h_stride, w, w_stride, target, t, d, v, ignore_index,
                              reduction, loss, lse, workspace, static_cast<hipStream_t>(stream)));
}

int linear_cross_entropy_backward(int type, const float *dloss, const void *h, int64_t h_stride,
                                  const void *w, int64_t w_stride, const int64_t *target,
                                  const float *lse, int64_t t, int64_t d, int64_t v,
                                  int64_t ignore_index, int reduction, void *dh, void *dw,
                                  void *workspace, size_t workspace_bytes, void *stream)
{
    int rc = check_loss(type, h, h_stride, w, w_stride, target, t, d, v, reduction);
    if (rc) return rc;
    if ((t > 0 && !lse) || ((t > 0 || reduction != NVFP4_NONE) && !dloss)) return NVFP4_ERR_NULL;
    if (!aligned(dloss, 4) || !aligned(lse, 4) || !aligned(dh, 2) || !aligned(dw, 2))
        return NVFP4_ERR_ALIGN;
    rc = check_workspace(workspace, workspace_bytes, nvfp4t_ce_workspace(1, t, d, v), 256);
    if (rc) return rc;
    rc = check_device();
    if (rc) return rc;
    return done(nvfp4t_ce_bwd(type, dloss, h, h_stride, w, w_stride, target, lse, t, d, v,
                              ignore_index, reduction, dh, dw, workspace,
                              static_cast<hipStream_t>(stream)));
}

size_t grad_norm_workspace_bytes(const int64_t *sizes, int64_t count)
{
    if (!sizes) return 0;
    for (int64_t i = 0; i < count; ++i)
        if (sizes[i] < 0 || sizes[i] >= MAX_ELEMS) return 0;
    return nvfp4t_norm_workspace(sizes, count);
}

int grad_norm(const void *const *tensors, const int64_t *sizes, const int32_t *types,
              int64_t count, int inf, float *norm, void *workspace, size_t workspace_bytes,
              void *stream)
{
    int rc = check_tensors(tensors, nullptr, false, sizes, types, count, inf, norm);
    if (rc) return rc;
    rc = check_workspace(workspace, workspace_bytes, nvfp4t_norm_workspace(sizes, count), 8);
    if (rc) return rc;
    rc = check_device();
    if (rc) return rc;
    return done(nvfp4t_norm(tensors, sizes, types, count, inf, norm, workspace,
                            static_cast<hipStream_t>(stream)));
}

int clip_grads(const void *const *tensors, void *const *outs, const int64_t *sizes,
               const int32_t *types, int64_t count, float max_norm, int inf, float *norm,
               void *workspace, size_t workspace_bytes, void *stream)
{
    int rc = check_tensors(tensors, outs, true, sizes, types, count, inf, norm);
    if (rc) return rc;
    if (!(max_norm >= 0.0f)) return NVFP4_ERR_ARG;
    rc = check_overlap(tensors, outs, sizes, types, count);
    if (rc) return rc;
    rc = check_workspace(workspace, workspace_bytes, nvfp4t_norm_workspace(sizes, count), 8);
    if (rc) return rc;
    rc = check_device();
    if (rc) return rc;
    const hipError_t e = nvfp4t_norm(tensors, sizes, types, count, inf, norm, workspace,
                                     static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return done(e);
    return done(nvfp4t_clip(tensors, outs, sizes, types, count, max_norm, norm,
                            static_cast<hipStream_t>(stream)));
}

}  // extern "C"
