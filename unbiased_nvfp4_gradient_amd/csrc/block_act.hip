// block_act.hip -- the backward pass of a linear layer's epilogue (activation or gating, and the
// bias), for gfx950.
//
//   dz = dy act'(z),  or of z = (gate, up):  dgate = dy up act'(gate),  dup = dy act(gate);
//   dbias = the sums of dz over the rows
// Bound by memory: dy and z are read once and dz is written once.  A lane keeps the same columns,
// 16 bytes of them, over its rows, so dbias is summed in registers from the unrounded FP32 values;
// the sums of a workgroup's row lanes join in LDS.  Of up to ACT_SHORT rows they are dbias then: a
// workgroup takes all rows of narrow columns, from a line of memory on.  Of more rows they leave as one row
// of `partial`, which a second launch adds up in a fixed order.
#include "block_math.h"

#pragma clang fp contract(fast)

namespace nvfp4t {

struct ActShape {
    int64_t rows, n, dy_stride, z_stride;
    int lanes;                  // lanes side by side over a row's columns, a power of two up to 64
};

// Rows up to which one workgroup takes all of them where their sums are wanted (within a graph 128x2048
// bf16 4.9 us, 8.9 with two launches; 257x1000 f32 6.0 and 7.3; 512x1000 8.5 and 8.0, 512x8192 bf16 12.1 and
// 11.2: there it only saves a call its second launch and its workspace).
constexpr int ACT_SHORT = 512;

// Where the sums over the rows go: to dbias, or to partial [gridDim.y][columns of dz] (both null: none).
struct ActSums {
    float *partial;
    void *dbias;
    int type;                   // of dbias
};

// Rows of a lane whose loads are in flight together (gated 32768x8192 bf16 584 us, with 4 rows and half
// as many waves a SIMD 610).
constexpr int ACT_ROWS = 2;

template <bool WHOLE, typename T, int V = VEC<T>>
__device__ __forceinline__ Pack<T, V> load_lane(const T *row, int64_t at, int64_t end)
{
    if constexpr (WHOLE) return *reinterpret_cast<const Pack<T, V> *>(row + at);
    else return load_row<T, V>(row, at, end);
}

template <bool WHOLE, typename T, int V>
__device__ __forceinline__ void store_lane(T *row, int64_t at, int64_t end, const Pack<T, V> &p)
{
    if constexpr (WHOLE) *reinterpret_cast<Pack<T, V> *>(row + at) = p;
    else store_row<T, V>(row, at, end, p);
}

// A lane's rows: row0, row0 + step, .. of its V columns from `col` on.  WHOLE: all of them exist.
// Lanes whose columns end inside go through the loop by themselves, so that the others' accesses are
// each one instruction (gated 32768x8192 bf16 735 us with ends looked for in every access, 610
// without).
template <typename T, int ACT, bool GATED, bool WHOLE>
__device__ __forceinline__ void act_rows(const T *__restrict__ dy, const T *__restrict__ z,
                                         const ActShape &s, T *__restrict__ dz, int64_t row0,
                                         int64_t step, int64_t col,
                                         float (&sum)[GATED ? 2 : 1][VEC<T>])
{
    constexpr int V = VEC<T>, Z = GATED ? 2 : 1;
    constexpr bool READS_Z = GATED || ACT != NONE;
    const int64_t end = WHOLE ? col + V : s.n;
    for (; row0 < s.rows; row0 += ACT_ROWS * step) {
        Pack<T, V> g[ACT_ROWS], x[ACT_ROWS][Z];
#pragma unroll
        for (int u = 0; u < ACT_ROWS; ++u) {
            const int64_t row = row0 + u * step;
            if (row >= s.rows) break;
            g[u] = load_lane<WHOLE>(dy + row * s.dy_stride, col, end);
            if constexpr (READS_Z) {
                const T *zr = z + row * s.z_stride;
                x[u][0] = load_lane<WHOLE>(zr, col, end);
                if constexpr (GATED) x[u][1] = load_lane<WHOLE>(zr + s.n, col, end);
            }
        }
#pragma unroll
        for (int u = 0; u < ACT_ROWS; ++u) {
            const int64_t row = row0 + u * step;
            if (row >= s.rows) break;
            Pack<T, V> out[Z];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = to_f32(g[u].v[i]);
                float value, slope = 1.0f;
                if constexpr (READS_Z) activate2<ACT>(to_f32(x[u][0].v[i]), value, slope);
                float o[Z];
                o[0] = d;
                if constexpr (GATED) {
                    o[0] = d * to_f32(x[u][1].v[i]);
                    o[1] = d * value;
                }
                if constexpr (ACT == RELU) o[0] = slope == 0.0f ? 0.0f : o[0];   // whatever d is
                else o[0] *= slope;
#pragma unroll
                for (int k = 0; k < Z; ++k) {
                    out[k].v[i] = from_f32<T>(o[k]);
                    sum[k][i] += o[k];
                }
            }
            T *to = dz + row * Z * s.n;
#pragma unroll
            for (int k = 0; k < Z; ++k) store_lane<WHOLE>(to + k * s.n, col, end, out[k]);
        }
    }
}

// Columns 16 bytes a lane, `lanes` of them in a workgroup at blockIdx.x; its 256 / lanes row lanes
// take every gridDim.y-th group of rows.
template <typename T, int ACT, bool GATED>
__global__ void __launch_bounds__(256)
    k_act_bwd(const T *__restrict__ dy, const T *__restrict__ z, ActShape s, T *__restrict__ dz,
              ActSums sums)
{
    constexpr int V = VEC<T>, Z = GATED ? 2 : 1;
    const int lane = threadIdx.x & (s.lanes - 1), row_lane = threadIdx.x / s.lanes;
    const int row_lanes = 256 / s.lanes;
    const int64_t col = ((int64_t)blockIdx.x * s.lanes + lane) * V;
    const int64_t width = Z * s.n;
    const int64_t step = (int64_t)gridDim.y * row_lanes;
    const int64_t row0 = (int64_t)blockIdx.y * row_lanes + row_lane;
    float sum[Z][V] = {};
    if (col + V <= s.n)
        act_rows<T, ACT, GATED, true>(dy, z, s, dz, row0, step, col, sum);
    else if (col < s.n)
        act_rows<T, ACT, GATED, false>(dy, z, s, dz, row0, step, col, sum);
    if (!sums.partial && !sums.dbias) return;
    __shared__ float lds[256 * V];
#pragma unroll
    for (int k = 0; k < Z; ++k) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) lds[i * 256 + threadIdx.x] = sum[k][i];
        __syncthreads();
        // thread t joins columns t, t + 256, .. of the workgroup's lanes * V
        for (int c = threadIdx.x; c < s.lanes * V; c += 256) {
            const int64_t at = (int64_t)blockIdx.x * s.lanes * V + c;
            if (at >= s.n) break;
            float total = 0.0f;
            for (int r = 0; r < row_lanes; ++r)
                total += lds[(c % V) * 256 + r * s.lanes + c / V];
            const int64_t to = k * s.n + at;
            if (sums.partial) sums.partial[(int64_t)blockIdx.y * width + to] = total;
            else if (sums.type == F32) static_cast<float *>(sums.dbias)[to] = total;
            else static_cast<T *>(sums.dbias)[to] = from_f32<T>(total);
        }
    }
}

// dbias: the sums of `count` partial rows in order, 64 columns a workgroup, four parts of the rows
// side by side.
template <typename P>
__global__ void __launch_bounds__(256)
    k_act_columns(const float *__restrict__ partial, int count, int64_t width, P *__restrict__ dbias)
{
    __shared__ float lds[256];
    const int lane = threadIdx.x & 63, part = threadIdx.x >> 6;
    for (int64_t base = (int64_t)blockIdx.x * 64; base < width; base += (int64_t)gridDim.x * 64) {
        const int64_t col = base + lane;
        float s = 0.0f;
        if (col < width)
#pragma unroll 8
            for (int k = part; k < count; k += 4) s += partial[(int64_t)k * width + col];
        __syncthreads();
        lds[threadIdx.x] = s;
        __syncthreads();
        if (part == 0 && col < width)
            dbias[col] = from_f32<P>((lds[lane] + lds[64 + lane]) +
                                     (lds[128 + lane] + lds[192 + lane]));
    }
}

// Lanes over a row of n elements: a wave's.  With few rows (see ACT_SHORT) a line's, but more of them
// where there are fewer rows than row lanes and workgroups for every compute unit all the same
// (1x16777216 f32 within a graph 36 us, 248 with 8 lanes; 512x65536 bf16 45 with 64 lanes, 35 with 8), or
// where there would be more workgroups than a launch holds.
int act_lanes(int64_t rows, int64_t n, int v)
{
    int lanes = rows <= ACT_SHORT ? 8 : 64;
    while (lanes < 64) {
        const int64_t groups = (n - 1) / (lanes * v) + 1;
        if (groups <= MAX_GROUPS && (256 / lanes <= rows || groups < 512)) break;
        lanes *= 2;
    }
    while (lanes > 1 && (int64_t)(lanes / 2) * v >= n) lanes /= 2;
    return lanes;
}

// Workgroups over the rows, about 2048 in all, so that a compute unit has 8, with eight rows a lane at
// least.  Few rows: one with sums (see ACT_SHORT); without, whose workgroups have nothing to join, two rows
// a lane (within a graph 512x64 bf16 3.1 us, 10.0 with one workgroup; 512x1000 f32 3.2 and 7.8).
int act_groups(int64_t rows, int64_t n, int v, bool sums)
{
    if (rows <= ACT_SHORT && sums) return 1;
    const int lanes = act_lanes(rows, n, v), each = rows <= ACT_SHORT ? ACT_ROWS : 8;
    const int64_t wide = (n + lanes * v - 1) / (lanes * v);
    const int64_t most = (rows + each * (256 / lanes) - 1) / (each * (256 / lanes));
    const int64_t want = 2048 / wide < 1 ? 1 : 2048 / wide;
    const int64_t groups = want < most ? want : most;
    return (int)(groups < 1 ? 1 : groups);
}

dim3 act_grid(int64_t rows, int64_t n, int v, bool sums)
{
    const int64_t strip = (int64_t)act_lanes(rows, n, v) * v;
    return dim3((unsigned)((n + strip - 1) / strip), (unsigned)act_groups(rows, n, v, sums));
}

template <typename T, int ACT, bool GATED>
void act_launch(const void *dy, const void *z, const ActShape &s, void *dz, const ActSums &sums,
                hipStream_t st)
{
    const dim3 grid = act_grid(s.rows, s.n, VEC<T>, sums.partial || sums.dbias);
    k_act_bwd<T, ACT, GATED><<<grid, 256, 0, st>>>((const T *)dy, (const T *)z, s, (T *)dz, sums);
}

template <typename T, bool GATED>
void act_kind(int act, const void *dy, const void *z, const ActShape &s, void *dz, const ActSums &sums,
              hipStream_t st)
{
    switch (act) {
    case RELU: act_launch<T, RELU, GATED>(dy, z, s, dz, sums, st); break;
    case GELU: act_launch<T, GELU, GATED>(dy, z, s, dz, sums, st); break;
    case GELU_TANH: act_launch<T, GELU_TANH, GATED>(dy, z, s, dz, sums, st); break;
    case SILU: act_launch<T, SILU, GATED>(dy, z, s, dz, sums, st); break;
    default: act_launch<T, NONE, GATED>(dy, z, s, dz, sums, st);
    }
}

template <typename T>
hipError_t act_bwd(int act, bool gated, const void *dy, const void *z, ActShape s, void *dz,
                   const ActSums &sums, hipStream_t st)
{
    s.lanes = act_lanes(s.rows, s.n, VEC<T>);
    if (gated) act_kind<T, true>(act, dy, z, s, dz, sums, st);
    else act_kind<T, false>(act, dy, z, s, dz, sums, st);
    return hipGetLastError();
}

template <typename P>
void act_columns(const float *partial, int count, int64_t width, void *dbias, hipStream_t st)
{
    const int64_t groups = (width + 63) / 64;
    k_act_columns<P><<<(unsigned)(groups < MAX_GROUPS ? groups : MAX_GROUPS), 256, 0, st>>>(
        partial, count, width, (P *)dbias);
}

}  // namespace nvfp4t

// Threads of k_act_bwd's launch in each dimension, which a launch holds fewer than 2^32 of.
extern "C" void nvfp4t_act_threads(int type, int64_t rows, int64_t n, int sums, int64_t *x, int64_t *y)
{
    const dim3 grid = nvfp4t::act_grid(rows, n, type == nvfp4t::F32 ? 4 : 8, sums);
    *x = (int64_t)grid.x * 256;
    *y = grid.y;
}

extern "C" size_t nvfp4t_act_workspace(int type, int gated, int64_t rows, int64_t n)
{
    const int groups = nvfp4t::act_groups(rows, n, type == nvfp4t::F32 ? 4 : 8, true);
    return groups == 1 ? 0 : (size_t)groups * (gated ? 2 : 1) * (size_t)n * sizeof(float);
}

extern "C" hipError_t nvfp4t_act_bwd(int type, int bias_type, int act, int gated, const void *dy,
                                     int64_t dy_stride, const void *z, int64_t z_stride,
                                     int64_t rows, int64_t n, void *dz, void *dbias, float *partial,
                                     hipStream_t st)
{
    using namespace nvfp4t;
    if (rows == 0 && !dbias) return hipSuccess;
    const ActShape s{rows, n, dy_stride, z_stride, 0};
    const int count = act_groups(rows, n, type == F32 ? 4 : 8, true);
    ActSums sums{nullptr, nullptr, bias_type};
    if (dbias && count == 1) sums.dbias = dbias;
    else if (dbias) sums.partial = partial;
    const hipError_t e = type == F32    ? act_bwd<float>(act, gated, dy, z, s, dz, sums, st)
                         : type == BF16 ? act_bwd<bf16>(act, gated, dy, z, s, dz, sums, st)
                                        : act_bwd<f16>(act, gated, dy, z, s, dz, sums, st);
    if (e != hipSuccess || !sums.partial) return e;
    const int64_t width = (gated ? 2 : 1) * n;
    if (bias_type == F32) act_columns<float>(partial, count, width, dbias, st);
    else if (bias_type == BF16) act_columns<bf16>(partial, count, width, dbias, st);
    else act_columns<f16>(partial, count, width, dbias, st);
    return hipGetLastError();
}
