// train_norm.hip -- layer norm, forward and backward, for gfx950.
//
// For each row x of n elements (products and sums in FP32, outputs rounded once):
//   forward   mean = sum x / n,  var = sum (x - mean)^2 / n,  rstd = 1 / sqrt(var + eps)
//             z = (x - mean) rstd,  y = z weight + bias
//   backward  g = dy weight,  dx = rstd (g - mean(g) - z mean(g z))
//             dweight = sum over rows of dy z,  dbias = sum over rows of dy
// Both are bound by memory: the forward reads x and writes y, the backward reads x and dy and
// writes dx.  A row stays in registers between its reductions and its output (so the variance
// is the two-pass one and x is read once), and rows whose length is a multiple of a 16-byte
// access have kernels without any code for ends inside one: 32768x2048 bf16 forward 48 us (5.6
// TB/s; a copy of these bytes reaches 5.3), backward 82 us (4.9) and 5 for the column sums.  On the
// same tensors again and again, in part from the cache, 44 and 86 us; 56 and 94 with that code.
#include "train_device.h"

#pragma clang fp contract(fast)

namespace nvfp4t {

// A row is spread over TPR threads of C chunks of VEC elements each; chunk c of thread t
// holds elements VEC (c TPR + t) onwards.  EVEN: the row's length is a multiple of VEC, so that no
// chunk ends inside a thread's elements.
template <typename T, int TPR, int C, bool EVEN> struct Row {
    static constexpr int V = VEC<T>;
    Pack<T, V> p[C];
    __device__ __forceinline__ void load(const T *__restrict__ row, int t, int64_t n)
    {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t at = (int64_t)V * (c * TPR + t);
            // the same answer in every lane: only a row's last chunk looks at its end
            if ((int64_t)V * TPR * (c + 1) <= n)
                p[c] = *reinterpret_cast<const Pack<T, V> *>(row + at);
            else
                p[c] = load_pack<EVEN, T, V>(row, at, n);
        }
    }
};

struct NormIn {
    int64_t rows, n, x_stride, dy_stride;   // strides in elements; outputs are contiguous
};

// Threads of a workgroup, and rows it holds at a time.
template <int TPR> constexpr int BLOCK = TPR <= 64 ? 256 : TPR;
template <int TPR> constexpr int ROWS = BLOCK<TPR> / TPR;

// Rows blockIdx.x * ROWS + r, then every gridDim.x * ROWS further: weight and bias stay in
// registers, and the next row loads while the present one is reduced.
template <typename T, typename P, int TPR, int C, bool EVEN>
__global__ void __launch_bounds__(BLOCK<TPR>)
    k_ln_fwd(const T *__restrict__ x, const P *__restrict__ weight, const P *__restrict__ bias,
             NormIn in, float eps, T *__restrict__ y, float *__restrict__ mean_out,
             float *__restrict__ rstd_out)
{
    constexpr int V = VEC<T>;
    constexpr bool AHEAD = TPR * C * V < 32768;      // the longest rows leave no registers for it
    __shared__ float2 lds[(TPR + 63) / 64];
    const int t = threadIdx.x % TPR;
    const int64_t n = in.n, step = (int64_t)gridDim.x * ROWS<TPR>;
    int64_t row = (int64_t)blockIdx.x * ROWS<TPR> + threadIdx.x / TPR;
    if (row >= in.rows) return;              // all TPR threads of a row, a wave at the most
    Row<T, TPR, C, EVEN> r, next;
    r.load(x + row * in.x_stride, t, n);
    Pack<P, V> w[C], b[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int64_t at = (int64_t)V * (c * TPR + t);
        if (weight) w[c] = load_pack<EVEN, P, V>(weight, at, n);
        if (bias) b[c] = load_pack<EVEN, P, V>(bias, at, n);
    }
    for (; row < in.rows; row += step) {
        if (AHEAD && row + step < in.rows) next.load(x + (row + step) * in.x_stride, t, n);
        float s = 0.0f, q = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < V; ++i) s += to_f32(r.p[c].v[i]);   // zeros past the end
        group_sum2<TPR>(s, q, lds);
        const float mean = s / (float)n;
        q = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t at = (int64_t)V * (c * TPR + t);
            const bool whole = (int64_t)V * TPR * (c + 1) <= n;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = to_f32(r.p[c].v[i]) - mean;
                q += whole || at + (EVEN ? 0 : i) < n ? d * d : 0.0f;
            }
        }
        s = 0.0f;
        group_sum2<TPR>(q, s, lds);
        const float rstd = 1.0f / sqrtf(q / (float)n + eps);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t at = (int64_t)V * (c * TPR + t);
            Pack<T, V> o;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float z = (to_f32(r.p[c].v[i]) - mean) * rstd;
                if (weight) z *= to_f32(w[c].v[i]);
                if (bias) z += to_f32(b[c].v[i]);
                o.v[i] = from_f32<T>(z);
            }
            store_pack<EVEN, T, V>(y + row * n, at, n, o);
        }
        if (t == 0) {
            mean_out[row] = mean;
            rstd_out[row] = rstd;
        }
        if constexpr (AHEAD) r = next;
        else if (row + step < in.rows) r.load(x + (row + step) * in.x_stride, t, n);
    }
}

// The backward pass of rows blockIdx.x * ROWS + r, then every gridDim.x * ROWS further.  A
// thread's columns are the same in every row, so the workgroup's sums for dweight and dbias
// stay in registers and leave once, as one row of `partial` [gridDim.x][2][n] (null: not
// wanted); k_ln_columns adds those.  The next row is loaded while the present one is reduced
// (not at 1024 threads, whose 128 registers have no room for it).
template <typename T, typename P, int TPR, int C, bool EVEN>
__global__ void __launch_bounds__(BLOCK<TPR>, TPR == 64 && VEC<T> == 8 ? 2 : 1)
    k_ln_bwd(const T *__restrict__ dy, const T *__restrict__ x, const float *__restrict__ mean_in,
             const float *__restrict__ rstd_in, const P *__restrict__ weight, NormIn in,
             T *__restrict__ dx, float *__restrict__ partial)
{
    constexpr int V = VEC<T>;
    constexpr bool AHEAD = TPR < 1024;
    __shared__ float2 lds[(TPR + 63) / 64];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const int64_t n = in.n, step = (int64_t)gridDim.x * ROWS<TPR>;
    int64_t row = (int64_t)blockIdx.x * ROWS<TPR> + sub;
    float dw[C][V], db[C][V];
    Pack<P, V> w[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (weight) w[c] = load_pack<EVEN, P, V>(weight, (int64_t)V * (c * TPR + t), n);
#pragma unroll
        for (int i = 0; i < V; ++i) dw[c][i] = db[c][i] = 0.0f;
    }
    Row<T, TPR, C, EVEN> rx, rd, nx, nd;
    if (AHEAD && row < in.rows) {
        rx.load(x + row * in.x_stride, t, n);
        rd.load(dy + row * in.dy_stride, t, n);
    }
    for (; row < in.rows; row += step) {
        if constexpr (AHEAD) {
            const int64_t next = row + step < in.rows ? row + step : row;
            nx.load(x + next * in.x_stride, t, n);
            nd.load(dy + next * in.dy_stride, t, n);
        } else {
            rx.load(x + row * in.x_stride, t, n);
            rd.load(dy + row * in.dy_stride, t, n);
        }
        const float mean = mean_in[row], rstd = rstd_in[row];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                // dy is 0 past the end, so nothing there counts
                const float d = to_f32(rd.p[c].v[i]);
                const float z = (to_f32(rx.p[c].v[i]) - mean) * rstd;
                const float g = weight ? d * to_f32(w[c].v[i]) : d;
                dw[c][i] += d * z;
                db[c][i] += d;
                s1 += g;
                s2 += g * z;
            }
        group_sum2<TPR>(s1, s2, lds);
        s1 /= (float)n;
        s2 /= (float)n;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t at = (int64_t)V * (c * TPR + t);
            Pack<T, V> o;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = to_f32(rd.p[c].v[i]);
                const float z = (to_f32(rx.p[c].v[i]) - mean) * rstd;
                const float g = weight ? d * to_f32(w[c].v[i]) : d;
                o.v[i] = from_f32<T>(rstd * (g - s1 - z * s2));
            }
            store_pack<EVEN, T, V>(dx + row * n, at, n, o);
        }
        if constexpr (AHEAD) {
            rx = nx;
            rd = nd;
        }
    }
    if (!partial) return;
    float *out = partial + (int64_t)blockIdx.x * 2 * n;
    if constexpr (ROWS<TPR> > 1) {
        // the sums of a wave's rows, then the waves' in their order
        __shared__ float sum[2 * TPR * V * C];
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int d = TPR; d < 64; d <<= 1) {
                    dw[c][i] += __shfl_xor(dw[c][i], d);
                    db[c][i] += __shfl_xor(db[c][i], d);
                }
        for (int k = 0; k < BLOCK<TPR> / 64; ++k) {
            if (wave == k && lane < TPR) {
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        float *a = sum + (c * V + i) * TPR + t, *b = a + TPR * V * C;
                        *a = k ? *a + dw[c][i] : dw[c][i];
                        *b = k ? *b + db[c][i] : db[c][i];
                    }
            }
            __syncthreads();
        }
        for (int e = threadIdx.x; e < TPR * V * C; e += BLOCK<TPR>) {
            const int lane_of = e % TPR, slot = e / TPR;    // slot = c V + i
            const int64_t at = (int64_t)V * ((slot / V) * TPR + lane_of) + slot % V;
            if (at < n) {
                out[at] = sum[e];
                out[n + at] = sum[e + TPR * V * C];
            }
        }
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t at = (int64_t)V * (c * TPR + t);
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (at + i < n) {
                    out[at + i] = dw[c][i];
                    out[n + at + i] = db[c][i];
                }
        }
    }
}

// dweight (blockIdx.y = 0) and dbias (1): the sums of `count` partial rows, 32 columns at a time,
// 32 threads to a column that take every 32nd row each, joined in a fixed order.
template <typename P>
__global__ void __launch_bounds__(1024)
    k_ln_columns(const float *__restrict__ partial, int count, int64_t n, P *__restrict__ dweight,
                 P *__restrict__ dbias)
{
    __shared__ float lds[32][33];
    P *out = blockIdx.y ? dbias : dweight;
    if (!out) return;
    const int in = threadIdx.x & 31, g = threadIdx.x >> 5;
    for (int64_t first = (int64_t)blockIdx.x * 32; first < n; first += (int64_t)gridDim.x * 32) {
        const int64_t col = first + in;
        float s = 0.0f;
        if (col < n) {
#pragma unroll 8
            for (int k = g; k < count; k += 32)
                s += partial[((int64_t)k * 2 + blockIdx.y) * n + col];
        }
        lds[g][in] = s;
        __syncthreads();
        s = lds[in][g];                       // 32 lanes to a column
        __syncthreads();                      // lds is free for the next columns
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor(s, d);
        const int64_t c = first + g;
        if (in == 0 && c < n) out[c] = from_f32<P>(s);
    }
}

// Rows that do not fit a workgroup's registers: 1024 threads walk the row once per reduction
// and once for the output.
template <typename T, typename P>
__global__ void __launch_bounds__(1024)
    k_ln_fwd_long(const T *__restrict__ x, const P *__restrict__ weight,
                  const P *__restrict__ bias, NormIn in, float eps, T *__restrict__ y,
                  float *__restrict__ mean_out, float *__restrict__ rstd_out)
{
    constexpr int V = VEC<T>;
    __shared__ float2 lds[16];
    const int64_t n = in.n;
    for (int64_t row = blockIdx.x; row < in.rows; row += gridDim.x) {
        const T *xr = x + row * in.x_stride;
        float s = 0.0f, q = 0.0f;
        for (int64_t at = V * threadIdx.x; at < n; at += V * 1024) {
            const Pack<T, V> p = load_row<T, V>(xr, at, n);
#pragma unroll
            for (int i = 0; i < V; ++i) s += to_f32(p.v[i]);
        }
        group_sum2<1024>(s, q, lds);
        const float mean = s / (float)n;
        q = 0.0f;
        for (int64_t at = V * threadIdx.x; at < n; at += V * 1024) {
            const Pack<T, V> p = load_row<T, V>(xr, at, n);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = to_f32(p.v[i]) - mean;
                q += at + i < n ? d * d : 0.0f;
            }
        }
        s = 0.0f;
        group_sum2<1024>(q, s, lds);
        const float rstd = 1.0f / sqrtf(q / (float)n + eps);
        for (int64_t at = V * threadIdx.x; at < n; at += V * 1024) {
            const Pack<T, V> p = load_row<T, V>(xr, at, n);
            Pack<P, V> w, b;
            if (weight) w = load_row<P, V>(weight, at, n);
            if (bias) b = load_row<P, V>(bias, at, n);
            Pack<T, V> o;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float z = (to_f32(p.v[i]) - mean) * rstd;
                if (weight) z *= to_f32(w.v[i]);
                if (bias) z += to_f32(b.v[i]);
                o.v[i] = from_f32<T>(z);
            }
            store_row<T, V>(y + row * n, at, n, o);
        }
        if (threadIdx.x == 0) {
            mean_out[row] = mean;
            rstd_out[row] = rstd;
        }
    }
}

template <typename T, typename P>
__global__ void __launch_bounds__(1024)
    k_ln_bwd_long(const T *__restrict__ dy, const T *__restrict__ x,
                  const float *__restrict__ mean_in, const float *__restrict__ rstd_in,
                  const P *__restrict__ weight, NormIn in, T *__restrict__ dx)
{
    constexpr int V = VEC<T>;
    __shared__ float2 lds[16];
    const int64_t n = in.n;
    for (int64_t row = blockIdx.x; row < in.rows; row += gridDim.x) {
        const T *xr = x + row * in.x_stride, *dr = dy + row * in.dy_stride;
        const float mean = mean_in[row], rstd = rstd_in[row];
        float s1 = 0.0f, s2 = 0.0f;
        for (int pass = 0; pass < 2; ++pass) {
            for (int64_t at = V * threadIdx.x; at < n; at += V * 1024) {
                const Pack<T, V> px = load_row<T, V>(xr, at, n), pd = load_row<T, V>(dr, at, n);
                Pack<P, V> w;
                if (weight) w = load_row<P, V>(weight, at, n);
                Pack<T, V> o;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float z = (to_f32(px.v[i]) - mean) * rstd;
                    float g = to_f32(pd.v[i]);
                    if (weight) g *= to_f32(w.v[i]);
                    if (pass) {
                        o.v[i] = from_f32<T>(rstd * (g - s1 - z * s2));
                    } else {
                        s1 += g;
                        s2 += g * z;
                    }
                }
                if (pass) store_row<T, V>(dx + row * n, at, n, o);
            }
            if (pass == 0) {
                group_sum2<1024>(s1, s2, lds);
                s1 /= (float)n;
                s2 /= (float)n;
            }
        }
    }
}

// Column sums of long rows: 256 columns a workgroup, every gridDim.y-th row, into `partial`
// [gridDim.y][2][n].
template <typename T>
__global__ void __launch_bounds__(256)
    k_ln_partial_long(const T *__restrict__ dy, const T *__restrict__ x,
                      const float *__restrict__ mean_in, const float *__restrict__ rstd_in,
                      NormIn in, float *__restrict__ partial)
{
    const int64_t col = (int64_t)blockIdx.x * 256 + threadIdx.x, n = in.n;
    if (col >= n) return;
    float dw = 0.0f, db = 0.0f;
    for (int64_t row = blockIdx.y; row < in.rows; row += gridDim.y) {
        const float d = to_f32(dy[row * in.dy_stride + col]);
        dw += d * ((to_f32(x[row * in.x_stride + col]) - mean_in[row]) * rstd_in[row]);
        db += d;
    }
    partial[(int64_t)blockIdx.y * 2 * n + col] = dw;
    partial[((int64_t)blockIdx.y * 2 + 1) * n + col] = db;
}

// Threads of a row and its chunks a thread.  Short rows take part of a wave, several rows to a
// wave (262144x64 bf16: forward 14 us, 86 with a wave to a row; backward 24, 213), rows up to
// 2048 elements a wave, so that no barrier stands between reductions (backward 32768x2048 bf16:
// 86 us, 105 with 256 threads to a row; in float32, whose two rows would fill the registers, up
// to 1024), longer ones a workgroup.  The forward pass holds up to 32 elements a thread (float32
// 16384x8192: 204 us, 209 with 1024 threads of 8), the backward pass, with two rows, the next two
// and two sums for each element, 16 where a row takes a workgroup (16384x3000 f16: 79 us, 96 with
// 32; 16384x4096 bf16 87 and 99; from 4097 to 8192 elements, though, 16384x8192 bf16 194 and 179,
// 8192x8192 f16 116 and 105).
struct Shape { int tpr, chunks; };

Shape fwd_shape(int64_t n, int v)
{
    for (const int tpr : {8, 16, 32, 64})
        if (n <= tpr * v) return {tpr, 1};
    for (const int tpr : {64, 256, 1024})
        for (const int c : {2, 4, 8})
            if ((c < 8 || (tpr == 256 && v == 4)) && n <= (int64_t)tpr * v * c) return {tpr, c};
    return {0, 0};
}

Shape bwd_shape(int64_t n, int v)
{
    for (const int tpr : {8, 16, 32, 64})
        if (n <= tpr * 8) return {tpr, 8 / v};
    for (const int e : {16, 32})
        if ((e == 16 || v == 8) && n <= 64 * e) return {64, e / v};
    if (n <= 2048) return {256, 8 / v};
    for (const int tpr : {256, 512, 1024})
        if (n <= tpr * 16) return {tpr, 16 / v};
    return {0, 0};
}

// Workgroups of the forward pass: as many as the compute units hold at a time.
unsigned fwd_groups(int64_t rows, int per, int block)
{
    const int64_t want = (rows + per - 1) / per, most = 256 * (2048 / block);
    return (unsigned)(want < most ? want : most);
}

// Workgroups of the backward pass whose partial sums are kept: two to a compute unit, four
// where rows are short and the sums are little beside the rows.
int max_partials(int64_t n) { return n <= 512 ? 1024 : 512; }

unsigned groups(int64_t want) { return (unsigned)(want < MAX_GROUPS ? want : MAX_GROUPS); }

int partials(int64_t rows, int64_t n, int v)
{
    const Shape s = bwd_shape(n, v);
    const int64_t per = s.tpr <= 64 ? 256 / (s.tpr ? s.tpr : 256) : 1;
    const int64_t want = s.tpr ? (rows + per - 1) / per : rows;
    const int64_t cap = s.tpr ? max_partials(n) : 64;
    return (int)(want < cap ? want : cap);
}

template <typename T, typename P>
void fwd(const void *x, const void *weight, const void *bias, const NormIn &in, float eps,
         void *y, float *mean, float *rstd, hipStream_t st)
{
    const T *xp = (const T *)x;
    const P *wp = (const P *)weight, *bp = (const P *)bias;
    const Shape s = fwd_shape(in.n, VEC<T>);
    const bool even = in.n % VEC<T> == 0;
#define NVFP4T_FWD(TPR, C)                                                                     \
    if (s.tpr == TPR && s.chunks == C)                                                         \
        return (even ? k_ln_fwd<T, P, TPR, C, true> : k_ln_fwd<T, P, TPR, C, false>)           \
            <<<fwd_groups(in.rows, ROWS<TPR>, BLOCK<TPR>), BLOCK<TPR>, 0, st>>>(               \
                xp, wp, bp, in, eps, (T *)y, mean, rstd);
    NVFP4T_FWD(8, 1) NVFP4T_FWD(16, 1) NVFP4T_FWD(32, 1)
    NVFP4T_FWD(64, 1) NVFP4T_FWD(64, 2) NVFP4T_FWD(64, 4)
    NVFP4T_FWD(256, 2) NVFP4T_FWD(256, 4) NVFP4T_FWD(1024, 4)
    if constexpr (VEC<T> == 4) { NVFP4T_FWD(256, 8) }
    else { NVFP4T_FWD(1024, 2) }
#undef NVFP4T_FWD
    k_ln_fwd_long<T, P><<<groups(in.rows), 1024, 0, st>>>(xp, wp, bp, in, eps, (T *)y, mean,
                                                          rstd);
}

template <typename T, typename P>
void bwd(const void *dy, const void *x, const float *mean, const float *rstd, const void *weight,
         const NormIn &in, void *dx, void *dweight, void *dbias, float *partial, hipStream_t st)
{
    const T *dp = (const T *)dy, *xp = (const T *)x;
    const P *wp = (const P *)weight;
    const Shape s = bwd_shape(in.n, VEC<T>);
    const bool even = in.n % VEC<T> == 0;
    const int count = partials(in.rows, in.n, VEC<T>);
    const bool sums = dweight || dbias;
    float *part = sums ? partial : nullptr;
    if (in.rows) {
#define NVFP4T_BWD(TPR, C)                                                                     \
    if (s.tpr == TPR && s.chunks == C)                                                         \
        (even ? k_ln_bwd<T, P, TPR, C, true> : k_ln_bwd<T, P, TPR, C, false>)                  \
            <<<(unsigned)count, BLOCK<TPR>, 0, st>>>(dp, xp, mean, rstd, wp, in, (T *)dx, part);
        constexpr int C8 = 8 / VEC<T>, C16 = 16 / VEC<T>, C32 = 32 / VEC<T>;
        NVFP4T_BWD(8, C8) NVFP4T_BWD(16, C8) NVFP4T_BWD(32, C8)
        NVFP4T_BWD(64, C8) NVFP4T_BWD(64, C16)
        if constexpr (VEC<T> == 8) { NVFP4T_BWD(64, C32) }
        else { NVFP4T_BWD(256, C8) }
        NVFP4T_BWD(256, C16) NVFP4T_BWD(512, C16) NVFP4T_BWD(1024, C16)
#undef NVFP4T_BWD
        if (!s.tpr) {
            k_ln_bwd_long<T, P><<<groups(in.rows), 1024, 0, st>>>(dp, xp, mean, rstd, wp, in,
                                                                  (T *)dx);
            if (sums)
                k_ln_partial_long<T><<<dim3((unsigned)((in.n + 255) / 256), (unsigned)count), 256,
                                       0, st>>>(dp, xp, mean, rstd, in, part);
        }
    }
    if (sums)
        k_ln_columns<P><<<dim3(groups((in.n + 31) / 32), 2), 1024, 0, st>>>(
            part, count, in.n, (P *)dweight, (P *)dbias);
}

}  // namespace nvfp4t

extern "C" size_t nvfp4t_ln_workspace(int type, int64_t rows, int64_t n)
{
    return (size_t)nvfp4t::partials(rows, n, type == nvfp4t::F32 ? 4 : 8) * 2 * sizeof(float) *
           (size_t)n;
}

// Element type `type` of x, dy, y and dx; `p_type` (the same or F32) of weight, bias and their
// gradients.
extern "C" hipError_t nvfp4t_ln_fwd(int type, int p_type, const void *x, const void *weight,
                                    const void *bias, int64_t rows, int64_t n, int64_t x_stride,
                                    float eps, void *y, float *mean, float *rstd, hipStream_t st)
{
    using namespace nvfp4t;
    const NormIn in{rows, n, x_stride, 0};
    if (rows == 0) return hipSuccess;
    if (type == F32) fwd<float, float>(x, weight, bias, in, eps, y, mean, rstd, st);
    else if (type == BF16 && p_type == F32)
        fwd<bf16, float>(x, weight, bias, in, eps, y, mean, rstd, st);
    else if (type == BF16) fwd<bf16, bf16>(x, weight, bias, in, eps, y, mean, rstd, st);
    else if (p_type == F32) fwd<f16, float>(x, weight, bias, in, eps, y, mean, rstd, st);
    else fwd<f16, f16>(x, weight, bias, in, eps, y, mean, rstd, st);
    return hipGetLastError();
}

extern "C" hipError_t nvfp4t_ln_bwd(int type, int p_type, const void *dy, const void *x,
                                    const float *mean, const float *rstd, const void *weight,
                                    int64_t rows, int64_t n, int64_t dy_stride, int64_t x_stride,
                                    void *dx, void *dw, void *db, float *partial, hipStream_t st)
{
    using namespace nvfp4t;
    const NormIn in{rows, n, x_stride, dy_stride};
    if (type == F32) bwd<float, float>(dy, x, mean, rstd, weight, in, dx, dw, db, partial, st);
    else if (type == BF16 && p_type == F32)
        bwd<bf16, float>(dy, x, mean, rstd, weight, in, dx, dw, db, partial, st);
    else if (type == BF16) bwd<bf16, bf16>(dy, x, mean, rstd, weight, in, dx, dw, db, partial, st);
    else if (p_type == F32) bwd<f16, float>(dy, x, mean, rstd, weight, in, dx, dw, db, partial, st);
    else bwd<f16, f16>(dy, x, mean, rstd, weight, in, dx, dw, db, partial, st);
    return hipGetLastError();
}
