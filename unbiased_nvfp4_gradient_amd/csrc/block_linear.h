// block_linear.h -- what the MXFP4 products with an epilogue share (block_linear.hip: tiles;
// block_linear_few.hip: a few tokens): operands, the epilogue, and reads and writes of eight
// elements of a type known at run time.
#pragma once
#include "block_math.h"

namespace nvfp4t {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));

// Row-major: codes [rows][K/2], scales [rows][K/32]; K-tiled: codes [K/128][rows][64], scales
// [K/128][rows][4].
struct MxRows {
    const uint8_t *codes;
    const uint8_t *scales;
    int64_t rows;
};

// z = f product + bias; y = act(z) + residual, or of z = (gate, up) y = act(gate) up.  y [M][n], z
// [M][n] or [M][2n] (null: not kept), in one type.
struct Epilogue {
    float f;
    int act, type, bias_type;
    const void *bias;            // null: none
    const void *residual;        // null: none
    int64_t residual_stride;
    void *y, *z;
    int64_t m, n;
};

template <typename T>
__device__ __forceinline__ void load8_of(const void *p, int64_t at, int64_t left, float (&v)[8])
{
    const Pack<T, 8> x = load_row<T, 8>(static_cast<const T *>(p) + at, 0, left);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(x.v[i]);
}

// Elements [at, at + 8) of p, of which `left` exist (zeros beyond).
__device__ __forceinline__ void load8(const void *p, int type, int64_t at, int64_t left,
                                      float (&v)[8])
{
    if (type == F32) load8_of<float>(p, at, left, v);
    else if (type == BF16) load8_of<bf16>(p, at, left, v);
    else load8_of<f16>(p, at, left, v);
}

template <typename T>
__device__ __forceinline__ void store8_of(void *p, int64_t at, int64_t left, const float (&v)[8])
{
    Pack<T, 8> x;
#pragma unroll
    for (int i = 0; i < 8; ++i) x.v[i] = from_f32<T>(v[i]);
    store_row<T, 8>(static_cast<T *>(p) + at, 0, left, x);
}

__device__ __forceinline__ void store8(void *p, int type, int64_t at, int64_t left,
                                       const float (&v)[8])
{
    if (type == F32) store8_of<float>(p, at, left, v);
    else if (type == BF16) store8_of<bf16>(p, at, left, v);
    else store8_of<f16>(p, at, left, v);
}

template <int ACT> __device__ __forceinline__ void activate8_of(float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = activate<ACT>(v[i]);
}

__device__ __forceinline__ void activate8(int act, float (&v)[8])
{
    switch (act) {
    case RELU: activate8_of<RELU>(v); break;
    case GELU: activate8_of<GELU>(v); break;
    case GELU_TANH: activate8_of<GELU_TANH>(v); break;
    case SILU: activate8_of<SILU>(v); break;
    default: break;
    }
}

// What the epilogue reads once for a lane's eight columns.
template <bool GATED> struct Bias8 {
    float b[GATED ? 2 : 1][8];
    __device__ __forceinline__ void load(const Epilogue &e, int64_t col)
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) b[0][i] = 0.0f;
        if constexpr (GATED)
#pragma unroll
            for (int i = 0; i < 8; ++i) b[1][i] = 0.0f;
        if (!e.bias || col >= e.n) return;
        load8(e.bias, e.bias_type, col, e.n - col, b[0]);
        if constexpr (GATED) load8(e.bias, e.bias_type, e.n + col, e.n - col, b[1]);
    }
};

// Eight columns of a row, col < n and row < m: `z` holds the products' sums (gated: gate and up).
template <bool GATED>
__device__ __forceinline__ void finish8(const Epilogue &e, int64_t row, int64_t col,
                                        const Bias8<GATED> &bias, float (&z)[GATED ? 2 : 1][8])
{
    const int64_t left = e.n - col;
    constexpr int Z = GATED ? 2 : 1;
#pragma unroll
    for (int k = 0; k < Z; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) z[k][i] = __builtin_fmaf(z[k][i], e.f, bias.b[k][i]);
    if (e.z) {
#pragma unroll
        for (int k = 0; k < Z; ++k) store8(e.z, e.type, row * (Z * e.n) + k * e.n + col, left, z[k]);
    }
    activate8(e.act, z[0]);
    if constexpr (GATED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) z[0][i] *= z[1][i];
    } else if (e.residual) {
        float r[8];
        load8(e.residual, e.type, row * e.residual_stride + col, left, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[0][i] += r[i];
    }
    store8(e.y, e.type, row * e.n + col, left, z[0]);
}

}  // namespace nvfp4t
