// train_device.h -- device helpers of the training-step kernels (layer norm, the linear head's
// cross entropy, gradient clipping): element types, loads and stores of eight or four
// elements at any element alignment, and reductions over a wave or a workgroup.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4t {

enum { F32 = 0, BF16 = 1, F16 = 2 };   // NVFP4_F32, NVFP4_BF16, NVFP4_F16

struct bf16 { uint16_t bits; };
struct f16 { _Float16 v; };

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(bf16 x) { return __uint_as_float((uint32_t)x.bits << 16); }
__device__ __forceinline__ float to_f32(f16 x) { return (float)x.v; }

// Rounding to the element type: to nearest even, once (bf16: gfx950's conversion instruction).
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ bf16 from_f32<bf16>(float x)
{
    return bf16{__builtin_bit_cast(uint16_t, (__bf16)x)};
}
template <> __device__ __forceinline__ f16 from_f32<f16>(float x) { return f16{(_Float16)x}; }

// Workgroups of a launch at most, where a workgroup stands for a row or a few columns or tokens: a
// launch holds fewer than 2^32 threads in a dimension, so the kernels walk what is left.
constexpr int64_t MAX_GROUPS = (int64_t)1 << 21;

// Workgroups of a launch at most in its second dimension.
constexpr int64_t MAX_GROUPS_Y = 65535;

// Elements of one 16-byte access.
template <typename T> constexpr int VEC = 16 / (int)sizeof(T);

// V elements in a row, aligned like one element: rows of odd lengths and views of wider
// tensors take the same wide accesses as aligned ones (gfx950 global accesses need no more
// than their element's alignment).
template <typename T, int V> struct __attribute__((packed, aligned(sizeof(T)))) Pack { T v[V]; };

// Elements [at, at + V) of a row of n, zeros past its end.
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_row(const T *__restrict__ row, int64_t at, int64_t n)
{
    if (at + V <= n) return *reinterpret_cast<const Pack<T, V> *>(row + at);
    Pack<T, V> p;
#pragma unroll
    for (int i = 0; i < V; ++i) p.v[i] = at + i < n ? row[at + i] : T{};
    return p;
}

template <typename T, int V>
__device__ __forceinline__ void store_row(T *__restrict__ row, int64_t at, int64_t n,
                                          const Pack<T, V> &p)
{
    if (at + V <= n) {
        *reinterpret_cast<Pack<T, V> *>(row + at) = p;
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (at + i < n) row[at + i] = p.v[i];
}

// The same where n is a multiple of V: all of the pack lies inside or none.
template <bool EVEN, typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T *__restrict__ row, int64_t at, int64_t n)
{
    if constexpr (EVEN) {
        Pack<T, V> p{};
        if (at < n) p = *reinterpret_cast<const Pack<T, V> *>(row + at);
        return p;
    } else {
        return load_row<T, V>(row, at, n);
    }
}

template <bool EVEN, typename T, int V>
__device__ __forceinline__ void store_pack(T *__restrict__ row, int64_t at, int64_t n,
                                           const Pack<T, V> &p)
{
    if constexpr (EVEN) {
        if (at < n) *reinterpret_cast<Pack<T, V> *>(row + at) = p;
    } else {
        if (at < n) store_row<T, V>(row, at, n, p);
    }
}

// The sum over LANES neighbouring lanes, in each of them.
template <int LANES = 64, typename S> __device__ __forceinline__ S wave_sum(S x)
{
#pragma unroll
    for (int d = LANES / 2; d; d >>= 1) x += __shfl_xor(x, d);
    return x;
}

__device__ __forceinline__ float wave_max(float x)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) x = fmaxf(x, __shfl_xor(x, d));
    return x;
}

// Sums of a and b over a group of THREADS threads (a wave or a part of one, or the whole
// workgroup through `lds`, two floats per wave): the same bits in every thread, in a fixed
// order.
template <int THREADS>
__device__ __forceinline__ void group_sum2(float &a, float &b, float2 *lds)
{
    a = wave_sum<THREADS < 64 ? THREADS : 64>(a);
    b = wave_sum<THREADS < 64 ? THREADS : 64>(b);
    if constexpr (THREADS > 64) {
        __syncthreads();                       // earlier readers of lds are done
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = make_float2(a, b);
        __syncthreads();
        a = b = 0.0f;
#pragma unroll
        for (int w = 0; w < THREADS / 64; ++w) {
            a += lds[w].x;
            b += lds[w].y;
        }
    }
}

}  // namespace nvfp4t
