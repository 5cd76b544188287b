// train_ce.h -- what the kernels of the linear head's cross entropy share (train_ce.hip: products
// in tiles of 256 x 256; train_ce_few.hip: a few tokens): matrix instructions, the gathered
// tokens, and the launches for a few tokens.
#pragma once
#include "train_device.h"

namespace nvfp4t {

typedef float f32x16 __attribute__((ext_vector_type(16)));
// a vector type, not the struct uint4: for reads of a struct the compiler would wait for every
// load into LDS in flight first
typedef int int4v __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr float LOG2E = 1.44269504088896340736f, LN2 = 0.693147180559945309417f;

// What the products need to know about the tokens, written by k_ce_tokens.
struct Info {
    int32_t kept;          // tokens that count
    float scale;           // factor of dh and dw (see k_ce_tokens)
};

__device__ __forceinline__ f32x16 mfma(bf16, int4v a, int4v b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ f32x16 mfma(f16, int4v a, int4v b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// q is held this power of two times its value: for float16 2^15, which keeps probabilities down to
// 2^-29 out of its subnormal range.
template <typename T> constexpr int Q_EXP = 0;
template <> inline constexpr int Q_EXP<f16> = 15;
template <typename T> constexpr float Q_ONE = (float)(1 << Q_EXP<T>);

// Per gathered token, padded to a multiple of 256: where it came from, its target (-1: none in
// range), its lse and, with a dloss for each token, the factor of its row of q in dw (see
// k_ce_tokens).
struct Tokens {
    Info *info;
    int32_t *index, *target;
    float *lse, *share;
};

// What a part's exponentials are taken against: an infinite maximum is not subtracted, the sum is
// then 0 or infinite, as it should.
__device__ __forceinline__ float base_of(float top) { return __builtin_isinf(top) ? 0.0f : top; }

// e^x / e^base.  The difference comes first: the largest logit then counts exactly 1, and the
// others lose nothing to the size that all of them share.
__device__ __forceinline__ float exp_from(float x, float base)
{
    return __builtin_amdgcn_exp2f((x - base) * LOG2E);
}

// Largest logit and sum of exponentials against it, of two parts together.  An empty or
// minus-infinite part adds nothing, whatever its maximum.
__device__ __forceinline__ float2 join_stats(float2 x, float2 y)
{
    const float m = fmaxf(x.x, y.x), base = base_of(m);
    const float a = x.y == 0.0f ? 0.0f : x.y * exp_from(base_of(x.x), base);
    const float b = y.y == 0.0f ? 0.0f : y.y * exp_from(base_of(y.x), base);
    return make_float2(m, a + b);
}

__device__ __forceinline__ float lse_of(float2 s)
{
    return base_of(s.x) + __builtin_amdgcn_logf(s.y) * LN2;
}

// lse - own without lse's rounding: where the target's logit is the largest, what is left is the
// logarithm alone (logits of 1024 and losses below 1e-4: off by up to 8e-5 from a rounded lse).
__device__ __forceinline__ float loss_of(float2 s, float own)
{
    return (base_of(s.x) - own) + __builtin_amdgcn_logf(s.y) * LN2;
}

__device__ __forceinline__ uint32_t pack2(bf16, float a, float b)
{
    return (uint32_t)from_f32<bf16>(a).bits | (uint32_t)from_f32<bf16>(b).bits << 16;
}

__device__ __forceinline__ uint32_t pack2(f16, float a, float b)
{
    return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)a) |
           (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)b) << 16;
}

// Eight elements in a row from u[0..3], of which a lane holds elements 0..3 and 8..11 (lower half
// of the wave) or 4..7 and 12..15 of 16: the halves trade, the lower keeps 0..7.
__device__ __forceinline__ uint4 join16(const uint32_t *u)
{
    const auto a = __builtin_amdgcn_permlane32_swap(u[0], u[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(u[1], u[3], false, false);
    return make_uint4(a[0], b[0], a[1], b[1]);
}

// The factor of a gathered token's row of dh.
template <typename T>
__device__ __forceinline__ float dh_scale(const Tokens &tok, const float *dloss, int64_t slot)
{
    return dloss ? dloss[tok.index[slot]] / Q_ONE<T> : tok.info->scale;
}

// Tokens up to which the kernels of train_ce_few.hip are taken.
constexpr int64_t FEW = 128;

inline int64_t up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// Sizes of a few tokens' workspace.
struct FewSizes {
    int blocks;               // of 32 tokens: 1, 2 or 4
    int words;                // to a workgroup: 32 or 64
    int64_t groups;           // workgroups over the vocabulary
    int64_t slices, runs;     // of dh: of the head's columns and of its words
    int64_t slice_elems;      // columns of a slice
    int64_t partial_bytes, q_bytes, sums_bytes;
};
FewSizes few_sizes(int64_t t, int64_t d, int64_t v);

struct Head {
    const void *h;
    int64_t h_stride;
    const void *w;
    int64_t w_stride, t, d, v;
};

template <typename T>
void few_forward(const Head &a, const int64_t *target, int64_t ignore, const Tokens &tok,
                 const uint8_t *hk, int64_t hk_rows, float2 *partial, float *at_target,
                 float *loss_each, float *lse, float *loss_kept, hipStream_t st);
// q, and dw where not null.  weighted: tok.share counts.
template <typename T>
void few_grad(const Head &a, const Tokens &tok, bool weighted, const uint8_t *hk, int64_t hk_rows,
              const uint8_t *ht, int64_t dp, uint8_t *q, void *dw, hipStream_t st);
// dloss: of each token, or null.
template <typename T>
void few_dh(const Head &a, const Tokens &tok, const float *dloss, const uint8_t *q, float *sums,
            void *dh, hipStream_t st);

}  // namespace nvfp4t
