// block_linear.h -- what the MXFP4 products with an epilogue share (block_linear.hip: tiles;
// block_linear_few.hip: a few rows): operands, the epilogue's arguments, and the matrix
// instruction.
#pragma once
#include <type_traits>

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

// z = f product + bias; y = act(z) + residual, or of z = (gate, up) y = act(gate) up.  y [m][n], z
// [m][n] or [m][2n] (null: not kept), in one type.
struct Epilogue {
    float f;
    int act, bias_type;
    const void *bias;            // null: none
    const void *residual;        // null: none
    int64_t residual_stride;
    void *y, *z;
    int64_t m, n;
    bool passing;                // y and z, of 16 bits, are too large for the caches to keep
};

// Products with a few rows (block_linear_few.hip).
hipError_t linear_few(int type, const MxRows &A, const MxRows &B, int64_t K, bool tiled, bool gated,
                      const Epilogue &e, hipStream_t st);

// acc[r] += the products of 64 elements: 32 rows of x by 32 rows of w, FP4 codes under one power of
// two per 32 (byte 2 Q of each scale word).  Lane l supplies row l % 32 of both and elements
// 32 (l / 32) .. +31; its accumulator r is w's row 8 (r / 4) + 4 (l / 32) + r % 4, x's row l % 32.
template <int Q>
__device__ __forceinline__ f32x16 mx_multiply(v8i w, uint32_t w_scale, v8i x, uint32_t x_scale,
                                              f32x16 acc)
{
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x, acc, 4, 4, 2 * Q, (int)w_scale,
                                                           2 * Q, (int)x_scale);
}

__device__ __forceinline__ v8i mx_fragment(const uint8_t *p)
{
    const v4i v = *reinterpret_cast<const v4i *>(p);
    return v8i{v.x, v.y, v.z, v.w, 0, 0, 0, 0};
}

template <int ACT, int N> __device__ __forceinline__ void activate_of(float (&v)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = activate<ACT>(v[i]);
}

template <int N> __device__ __forceinline__ void activate_all(int act, float (&v)[N])
{
    switch (act) {
    case RELU: activate_of<RELU>(v); break;
    case GELU: activate_of<GELU>(v); break;
    case GELU_TANH: activate_of<GELU_TANH>(v); break;
    case SILU: activate_of<SILU>(v); break;
    default: break;
    }
}

// Two values as the 16-bit type's bits, the first one lower.
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b)
{
    struct Two { T a, b; };
    return __builtin_bit_cast(uint32_t, Two{from_f32<T>(a), from_f32<T>(b)});
}

template <typename T> __device__ __forceinline__ void unpack2(uint32_t x, float &a, float &b)
{
    struct Two { T a, b; };
    const Two t = __builtin_bit_cast(Two, x);
    a = to_f32(t.a);
    b = to_f32(t.b);
}

// Exchange a's lanes 32..63 with b's 0..31.
__device__ __forceinline__ void swap32(uint32_t &a, uint32_t &b)
{
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

// Exchange a's lanes 16..31 and 48..63 with b's 0..15 and 32..47.
__device__ __forceinline__ void swap16(uint32_t &a, uint32_t &b)
{
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

// 16 bytes, aligned like the smallest element.
typedef uint32_t Words4 __attribute__((ext_vector_type(4), aligned(2)));

// A 32 x 32 block of a matrix of type T, between a lane's accumulators (v[r]: column 8 (r / 4) + 4
// (lane / 32) + r % 4, row lane % 32) and memory: the lanes exchange words until each has 16 bytes of
// one row and four neighbours have 64 (32-bit types: two and two), so that an access is 16 rows of
// whole 64-byte pieces.  Piece p of a lane lies at row 16 (p % 2) + lane % 16.  16 bits: pieces 0, 1,
// column 8 [0, 2, 1, 3][lane / 16]; 32 bits: pieces 0 .. 3, column 16 (p / 2) + [0, 8, 4, 12][lane / 16].
template <typename T> struct Block {
    static constexpr int PIECES = sizeof(T) == 2 ? 2 : 4, V = 16 / (int)sizeof(T);
    uint32_t w[PIECES][4];

    static __device__ __forceinline__ int row(int p, int lane) { return 16 * (p & 1) + (lane & 15); }
    static __device__ __forceinline__ int column(int p, int lane)
    {
        const int q = lane >> 4, at = 2 * (q & 1) + (q >> 1);       // 0, 2, 1, 3
        return sizeof(T) == 2 ? 8 * at : 16 * (p >> 1) + 4 * at;
    }
    __device__ __forceinline__ void exchange16()
    {
#pragma unroll
        for (int p = 0; p < PIECES; p += 2)
#pragma unroll
            for (int k = 0; k < 4; ++k) swap16(w[p][k], w[p + 1][k]);
    }
    // words k and k + 2 of a piece: the lower and the upper half's
    __device__ __forceinline__ void exchange32()
    {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int k = 0; k < 2; ++k) swap32(w[p][k], w[p][k + 2]);
        }
    }
    __device__ __forceinline__ void put(const float (&v)[16])
    {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[p][k] = pack2<T>(v[8 * p + 4 * (k >> 1) + 2 * (k & 1)],
                                       v[8 * p + 4 * (k >> 1) + 2 * (k & 1) + 1]);
        } else {
#pragma unroll
            for (int r = 0; r < 16; ++r) w[r >> 2][r & 3] = __float_as_uint(v[r]);
        }
        exchange32();
        exchange16();
    }
    __device__ __forceinline__ void add_to(float (&v)[16])
    {
        exchange16();
        exchange32();
#pragma unroll
        for (int p = 0; p < PIECES; ++p)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (sizeof(T) == 2) {
                    float a, b;
                    unpack2<T>(w[p][k], a, b);
                    v[8 * p + 4 * (k >> 1) + 2 * (k & 1)] += a;
                    v[8 * p + 4 * (k >> 1) + 2 * (k & 1) + 1] += b;
                } else {
                    v[4 * p + k] += __uint_as_float(w[p][k]);
                }
            }
    }
    // Rows [row0, m) and columns [col0, n) of the matrix exist.  WHOLE: all of the block's columns do.
    // PASSING (with WHOLE): the caches are asked not to keep it.
    template <bool WHOLE, bool PASSING>
    __device__ __forceinline__ void store(T *to, int64_t stride, int64_t row0, int64_t m,
                                          int64_t col0, int64_t n, int lane) const
    {
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
            const int64_t r = row0 + row(p, lane), c = col0 + column(p, lane);
            if (r >= m) continue;
            T *at = to + r * stride + c;
            if constexpr (WHOLE) {
                const Words4 x{w[p][0], w[p][1], w[p][2], w[p][3]};
                if constexpr (PASSING) __builtin_nontemporal_store(x, reinterpret_cast<Words4 *>(at));
                else *reinterpret_cast<Words4 *>(at) = x;
            } else {
                const Pack<T, V> x = __builtin_bit_cast(Pack<T, V>, w[p]);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (c + i < n) at[i] = x.v[i];
            }
        }
    }
    template <bool WHOLE>
    __device__ __forceinline__ void load(const T *from, int64_t stride, int64_t row0, int64_t m,
                                         int64_t col0, int64_t n, int lane)
    {
#pragma unroll
        for (int p = 0; p < PIECES; ++p) {
            const int64_t r = row0 + row(p, lane), c = col0 + column(p, lane);
            const T *at = from + r * stride + c;
#pragma unroll
            for (int k = 0; k < 4; ++k) w[p][k] = 0;
            if (r >= m) continue;
            if constexpr (WHOLE) {
                const Words4 x = *reinterpret_cast<const Words4 *>(at);
#pragma unroll
                for (int k = 0; k < 4; ++k) w[p][k] = x[k];
            } else {
                Pack<T, V> x{};
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (c + i < n) x.v[i] = at[i];
                __builtin_memcpy(w[p], &x, 16);
            }
        }
    }
};

template <typename P, bool WHOLE>
__device__ __forceinline__ void bias_from(const void *bias, int64_t at, int64_t left, float (&b)[16])
{
    const P *p = static_cast<const P *>(bias) + at;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        if constexpr (WHOLE) {
            const Pack<P, 4> x = *reinterpret_cast<const Pack<P, 4> *>(p + 8 * g);
#pragma unroll
            for (int q = 0; q < 4; ++q) b[4 * g + q] = to_f32(x.v[q]);
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                b[4 * g + q] = 8 * g + q < left ? to_f32(p[8 * g + q]) : 0.0f;
        }
    }
}

// v = f v + the biases of the block's columns, from element `first` of the bias on.
template <bool WHOLE>
__device__ __forceinline__ void scale_and_bias(const Epilogue &e, int64_t first, int64_t col0,
                                               int lane, float (&v)[16])
{
    if (!e.bias) {
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] *= e.f;
        return;
    }
    const int64_t c = col0 + 4 * (lane >> 5), at = first + c, left = e.n - c;
    float b[16];
    if (e.bias_type == F32) bias_from<float, WHOLE>(e.bias, at, left, b);
    else if (e.bias_type == BF16) bias_from<bf16, WHOLE>(e.bias, at, left, b);
    else bias_from<f16, WHOLE>(e.bias, at, left, b);
#pragma unroll
    for (int r = 0; r < 16; ++r) v[r] = __builtin_fmaf(v[r], e.f, b[r]);
}

// The epilogue of a 32 x 32 block at (row0, col0): v holds the products' sums (gated: gate and up).
template <typename T, bool GATED, bool WHOLE, bool PASSING>
__device__ __forceinline__ void finish_block(const Epilogue &e, int64_t row0, int64_t col0, int lane,
                                             float (&v)[GATED ? 2 : 1][16])
{
    constexpr int Z = GATED ? 2 : 1;
    Block<T> block;
#pragma unroll
    for (int k = 0; k < Z; ++k) {
        scale_and_bias<WHOLE>(e, k * e.n, col0, lane, v[k]);
        if (e.z) {
            block.put(v[k]);
            block.template store<WHOLE, PASSING>(static_cast<T *>(e.z) + k * e.n, Z * e.n, row0, e.m,
                                                 col0, e.n, lane);
        }
    }
    activate_all(e.act, v[0]);
    if constexpr (GATED) {
#pragma unroll
        for (int r = 0; r < 16; ++r) v[0][r] *= v[1][r];
    } else if (e.residual) {
        block.template load<WHOLE>(static_cast<const T *>(e.residual), e.residual_stride, row0, e.m,
                                   col0, e.n, lane);
        block.add_to(v[0]);
    }
    block.put(v[0]);
    block.template store<WHOLE, PASSING>(static_cast<T *>(e.y), e.n, row0, e.m, col0, e.n,
                                         lane);
}

}  // namespace nvfp4t
