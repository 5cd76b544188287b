// block_linear_few.hip -- MXFP4 products with an epilogue for a few rows, for gfx950.
//
// With few rows of A, B [n][K] is what has to move, 17 / 32 of a byte an element; with few of both, what
// counts is how long the sum over K takes.  A workgroup takes 32 rows of B (gated: 32 features, a row
// of gate and of up each) and up to 128 of A, its eight waves take K in turns of U steps of 128
// elements, and every operand goes from memory straight into the fragments of
// v_mfma_scale_f32_32x32x64_f8f6f4, so that nothing waits for anything but its own loads; the waves'
// sums join in their order through LDS, where the epilogue takes them.  Within a graph, 8192x2048
// (9 MB, 1.7 us at a copy's rate): 1 row 5.0 us, 32 rows 5.5, 128 rows 10.2; 32768x4096 (71 MB, 13.5
// us): 1 row 17.5, 32 rows 22.4.
#include "block_linear.h"

#pragma clang fp contract(fast)

namespace nvfp4t {

constexpr int FEW_WAVES = 8;

// One step's fragments of 32 rows: both sub-steps' codes and the scale word, shifted so that byte 2 q
// is the lane's block's in sub-step q.
struct Step {
    v8i codes[2];
    uint32_t scale;
};

// A lane's place in 32 rows of an operand.
template <bool TILED> struct Lane {
    const uint8_t *codes, *scales;
    int64_t step, sstep;
    __device__ __forceinline__ void aim(const MxRows &m, int64_t row, int64_t K, int lane)
    {
        const int half = lane >> 5;
        codes = m.codes + row * (TILED ? 64 : (K >> 1)) + 16 * half;
        scales = m.scales + row * (TILED ? 4 : (K >> 5));
        step = TILED ? m.rows * 64 : 64;
        sstep = TILED ? m.rows * 4 : 4;
    }
    __device__ __forceinline__ Step load(int64_t kt, int lane) const
    {
        Step s;
        s.codes[0] = mx_fragment(codes + kt * step);
        s.codes[1] = mx_fragment(codes + kt * step + 32);
        s.scale = *reinterpret_cast<const uint32_t *>(scales + kt * sstep) >> (8 * (lane >> 5));
        return s;
    }
};

template <typename P> __device__ __forceinline__ float one_of(const void *p, int64_t at)
{
    return to_f32(static_cast<const P *>(p)[at]);
}

__device__ __forceinline__ float bias_at(const Epilogue &e, int64_t at)
{
    if (!e.bias) return 0.0f;
    if (e.bias_type == F32) return one_of<float>(e.bias, at);
    return e.bias_type == BF16 ? one_of<bf16>(e.bias, at) : one_of<f16>(e.bias, at);
}

// 32 NB rows of A from 32 NB blockIdx.y on; workgroup blockIdx.x takes 32 columns of y at a time.
template <typename T, int NB, bool TILED, bool GATED>
__global__ void __launch_bounds__(64 * FEW_WAVES)
    k_mx_few(MxRows A, MxRows B, int64_t K, Epilogue e)
{
    constexpr int Z = GATED ? 2 : 1, U = NB == 1 ? 4 : NB == 2 ? 2 : 1;
    constexpr int STRIDE = 68;                   // floats of a row of sums: 4 apart in banks
    __shared__ float sums[Z][FEW_WAVES][16 * STRIDE];
    const int lane = threadIdx.x & 63, r = lane & 31;
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t nk = K / 128, row0 = (int64_t)blockIdx.y * 32 * NB;
    Lane<TILED> a[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int64_t row = row0 + 32 * i + r;
        a[i].aim(A, row < A.rows ? row : A.rows - 1, K, lane);
    }
    for (int64_t col0 = (int64_t)blockIdx.x * 32; col0 < e.n; col0 += (int64_t)gridDim.x * 32) {
        const int64_t col = col0 + r < e.n ? col0 + r : e.n - 1;
        Lane<TILED> b[Z];
#pragma unroll
        for (int k = 0; k < Z; ++k) b[k].aim(B, k * e.n + col, K, lane);
        f32x16 acc[NB][Z];
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int k = 0; k < Z; ++k) acc[i][k] = f32x16{};
        int64_t kt = (int64_t)w * U;
        for (; kt + U <= nk; kt += FEW_WAVES * U) {
            Step x[U][NB], y[U][Z];
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int k = 0; k < Z; ++k) y[u][k] = b[k].load(kt + u, lane);
#pragma unroll
                for (int i = 0; i < NB; ++i) x[u][i] = a[i].load(kt + u, lane);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int k = 0; k < Z; ++k) {
                        acc[i][k] = mx_multiply<0>(y[u][k].codes[0], y[u][k].scale, x[u][i].codes[0],
                                                   x[u][i].scale, acc[i][k]);
                        acc[i][k] = mx_multiply<1>(y[u][k].codes[1], y[u][k].scale, x[u][i].codes[1],
                                                   x[u][i].scale, acc[i][k]);
                    }
        }
        for (int64_t last = kt + U; kt < nk && kt < last; ++kt)
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const Step x = a[i].load(kt, lane);
#pragma unroll
                for (int k = 0; k < Z; ++k) {
                    const Step y = b[k].load(kt, lane);
                    acc[i][k] = mx_multiply<0>(y.codes[0], y.scale, x.codes[0], x.scale, acc[i][k]);
                    acc[i][k] = mx_multiply<1>(y.codes[1], y.scale, x.codes[1], x.scale, acc[i][k]);
                }
            }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            __syncthreads();                     // the sums before have been read
#pragma unroll
            for (int k = 0; k < Z; ++k)
#pragma unroll
                for (int q = 0; q < 16; ++q) sums[k][w][q * STRIDE + lane] = acc[i][k][q];
            __syncthreads();
            // thread t: column t % 32 of rows t / 32, t / 32 + 16
            const int c = threadIdx.x & 31;
            const int at = (4 * (c >> 3) + (c & 3)) * STRIDE + 32 * ((c >> 2) & 1);
            const int64_t y_col = col0 + c;
            for (int m = threadIdx.x >> 5; m < 32; m += 2 * FEW_WAVES) {
                const int64_t row = row0 + 32 * i + m;
                if (row >= e.m || y_col >= e.n) break;
                float z[Z];
#pragma unroll
                for (int k = 0; k < Z; ++k) {
                    float s = 0.0f;
#pragma unroll
                    for (int q = 0; q < FEW_WAVES; ++q) s += sums[k][q][at + m];
                    z[k] = __builtin_fmaf(s, e.f, bias_at(e, k * e.n + y_col));
                    if (e.z) static_cast<T *>(e.z)[row * Z * e.n + k * e.n + y_col] = from_f32<T>(z[k]);
                }
                float v[1] = {z[0]};
                activate_all(e.act, v);
                if constexpr (GATED) v[0] *= z[1];
                else if (e.residual) v[0] += one_of<T>(e.residual, row * e.residual_stride + y_col);
                static_cast<T *>(e.y)[row * e.n + y_col] = from_f32<T>(v[0]);
            }
        }
    }
}

template <typename T, int NB, bool GATED>
void few_rows(const MxRows &A, const MxRows &B, int64_t K, bool tiled, const Epilogue &e,
              hipStream_t st)
{
    const int64_t groups = (e.n + 31) / 32;
    const dim3 grid((unsigned)(groups < MAX_GROUPS ? groups : MAX_GROUPS),
                    (unsigned)((A.rows + 32 * NB - 1) / (32 * NB)));
    if (tiled) k_mx_few<T, NB, true, GATED><<<grid, 64 * FEW_WAVES, 0, st>>>(A, B, K, e);
    else k_mx_few<T, NB, false, GATED><<<grid, 64 * FEW_WAVES, 0, st>>>(A, B, K, e);
}

template <typename T, bool GATED>
hipError_t few_of(const MxRows &A, const MxRows &B, int64_t K, bool tiled, const Epilogue &e,
                  hipStream_t st)
{
    if (A.rows <= 32) few_rows<T, 1, GATED>(A, B, K, tiled, e, st);
    else if (A.rows <= 64) few_rows<T, 2, GATED>(A, B, K, tiled, e, st);
    else few_rows<T, 4, GATED>(A, B, K, tiled, e, st);
    return hipGetLastError();
}

hipError_t linear_few(int type, const MxRows &A, const MxRows &B, int64_t K, bool tiled, bool gated,
                      const Epilogue &e, hipStream_t st)
{
    switch (type) {
    case F32: return gated ? few_of<float, true>(A, B, K, tiled, e, st)
                           : few_of<float, false>(A, B, K, tiled, e, st);
    case BF16: return gated ? few_of<bf16, true>(A, B, K, tiled, e, st)
                            : few_of<bf16, false>(A, B, K, tiled, e, st);
    default: return gated ? few_of<f16, true>(A, B, K, tiled, e, st)
                          : few_of<f16, false>(A, B, K, tiled, e, st);
    }
}

}  // namespace nvfp4t
