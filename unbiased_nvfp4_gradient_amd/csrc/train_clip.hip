// train_clip.hip -- the norm of many gradient tensors together, and clipping by it, for gfx950.
//
//   norm = sqrt(sum of x^2)  or  max |x|  over every element of every tensor
//   out  = x * min(1, max_norm / (norm + 1e-6))
// Both passes are bound by memory.  Squares are taken and summed in 64 bits, so neither the
// smallest nor the largest float32 gradients are lost.  The tensors are cut into chunks, one
// workgroup each; the chunks' sums are joined in a fixed order, so a result does not depend on
// the order in which workgroups run.
//
// The tensors' addresses and sizes travel in the kernel arguments (4 KiB at most), a table of
// up to NORM_TABLE or CLIP_TABLE tensors a launch: nothing is copied from host memory, so a
// launch captured into a graph keeps what it was given.
#include "train_device.h"

#pragma clang fp contract(fast)

namespace nvfp4t {

constexpr int NORM_TABLE = 192, CLIP_TABLE = 140;

// Chunks of FEW_CHUNK elements up to which one workgroup takes the whole norm: two rounds of its
// waves (9x4099 float32: 9.7 us a call, 12.1 with a launch for the chunks and one to join them).
constexpr int FEW_CHUNK = 4096, FEW_CHUNKS = 32;

// Tensor i holds `size` elements and chunks first[i] .. first[i + 1] - 1 of the launch.  The
// element type lies in the upper byte of `size_type`.
template <int N> struct Table {
    const void *in[N];
    uint64_t size_type[N];
    uint32_t first[N + 1];
    int32_t count;
};

struct ClipTable {
    Table<CLIP_TABLE> t;
    void *out[CLIP_TABLE];
};

static_assert(sizeof(Table<NORM_TABLE>) + 64 <= 4096 && sizeof(ClipTable) + 64 <= 4096,
              "the table has to fit the kernel arguments");

template <int N>
__device__ __forceinline__ int find(const Table<N> &t, uint32_t chunk)
{
    int lo = 0, hi = t.count - 1;          // the last tensor whose first chunk is not past it
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= chunk) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Running result of one thread: a sum of squares in 64 bits, or the bit pattern of the largest
// |x| (ordered as integers, where a NaN is above infinity and so is never lost).
template <bool INF> struct Acc;
template <> struct Acc<false> {
    double s = 0.0;
    __device__ __forceinline__ void add(float x)
    {
        const double d = x;
        s = __builtin_fma(d, d, s);
    }
    __device__ __forceinline__ void join(double o) { s += o; }
    __device__ __forceinline__ double value() const { return s; }
};
template <> struct Acc<true> {
    uint32_t m = 0;
    __device__ __forceinline__ void add(float x)
    {
        const uint32_t b = __float_as_uint(x) & 0x7FFFFFFFu;
        m = b > m ? b : m;
    }
    __device__ __forceinline__ void join(double o) { add((float)o); }
    __device__ __forceinline__ double value() const { return __uint_as_float(m); }
};

// The workgroup's result, in thread 0.
template <bool INF> __device__ __forceinline__ double join_block(Acc<INF> a, double *lds)
{
    double v = a.value();
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        Acc<INF> b;
        b.join(v);
        b.join(__shfl_xor(v, d));
        v = b.value();
    }
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    Acc<INF> r;
    if (threadIdx.x == 0)
        for (int w = 0; w < (int)blockDim.x / 64; ++w) r.join(lds[w]);
    return r.value();
}

// n elements over THREADS threads, four loads of 16 bytes in flight in each.
template <typename T, int THREADS, bool INF>
__device__ __forceinline__ void norm_chunk(const T *__restrict__ p, int64_t n, Acc<INF> &a)
{
    constexpr int V = VEC<T>, U = 4;
    int64_t at = (int64_t)V * (threadIdx.x % THREADS);
    Acc<INF> part[U];
    for (; at + (U - 1) * THREADS * V + V <= n; at += U * THREADS * V) {
        Pack<T, V> x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = load_row<T, V>(p, at + u * THREADS * V, n);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < V; ++i) part[u].add(to_f32(x[u].v[i]));
    }
    for (; at < n; at += THREADS * V) {
        const Pack<T, V> x = load_row<T, V>(p, at, n);       // zeros past the end
#pragma unroll
        for (int i = 0; i < V; ++i) part[0].add(to_f32(x.v[i]));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) a.join(part[u].value());
}

// Elements [at, at + n) of tensor i.
template <int THREADS, bool INF>
__device__ __forceinline__ void norm_part(const Table<NORM_TABLE> &t, int i, int64_t at, int64_t n,
                                          Acc<INF> &a)
{
    switch (t.size_type[i] >> 56) {
    case F32: norm_chunk<float, THREADS, INF>((const float *)t.in[i] + at, n, a); break;
    case BF16: norm_chunk<bf16, THREADS, INF>((const bf16 *)t.in[i] + at, n, a); break;
    default: norm_chunk<f16, THREADS, INF>((const f16 *)t.in[i] + at, n, a); break;
    }
}

template <bool INF>
__global__ void __launch_bounds__(256)
    k_norm_chunks(Table<NORM_TABLE> t, int64_t chunk_size, double *__restrict__ partial)
{
    __shared__ double lds[4];
    const uint32_t chunk = blockIdx.x;
    const int i = find(t, chunk);
    const int64_t size = t.size_type[i] & ((1ull << 56) - 1);
    const int64_t at = (int64_t)(chunk - t.first[i]) * chunk_size;
    const int64_t n = size - at < chunk_size ? size - at : chunk_size;
    Acc<INF> a;
    norm_part<256, INF>(t, i, at, n, a);
    const double v = join_block<INF>(a, lds);
    if (threadIdx.x == 0) partial[chunk] = v;
}

// All of a few small tensors in one launch: the 16 waves of one workgroup take a chunk each in
// turns.
template <bool INF>
__global__ void __launch_bounds__(1024)
    k_norm_few(Table<NORM_TABLE> t, float *__restrict__ norm)
{
    __shared__ double lds[16];
    Acc<INF> a;
    for (uint32_t chunk = threadIdx.x >> 6; chunk < t.first[t.count]; chunk += 16) {
        const int i = find(t, chunk);
        const int64_t size = t.size_type[i] & ((1ull << 56) - 1);
        const int64_t at = (int64_t)(chunk - t.first[i]) * FEW_CHUNK;
        norm_part<64, INF>(t, i, at, size - at < FEW_CHUNK ? size - at : FEW_CHUNK, a);
    }
    const double v = join_block<INF>(a, lds);
    if (threadIdx.x == 0) norm[0] = (float)(INF ? v : sqrt(v));
}

template <bool INF>
__global__ void __launch_bounds__(1024)
    k_norm_join(const double *__restrict__ partial, int64_t count, float *__restrict__ norm)
{
    __shared__ double lds[16];
    Acc<INF> a;
    for (int64_t k = threadIdx.x; k < count; k += 1024) a.join(partial[k]);
    const double v = join_block<INF>(a, lds);
    if (threadIdx.x == 0) norm[0] = (float)(INF ? v : sqrt(v));
}

template <typename T>
__device__ __forceinline__ void clip_chunk(const T *in, T *out, int64_t n, float c)
{
    constexpr int V = VEC<T>, U = 4;
    int64_t at = (int64_t)V * threadIdx.x;
    for (; at + (U - 1) * 256 * V + V <= n; at += U * 256 * V) {
        Pack<T, V> x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = load_row<T, V>(in, at + u * 256 * V, n);
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int i = 0; i < V; ++i) x[u].v[i] = from_f32<T>(to_f32(x[u].v[i]) * c);
            store_row<T, V>(out, at + u * 256 * V, n, x[u]);
        }
    }
    for (; at < n; at += 256 * V) {
        Pack<T, V> x = load_row<T, V>(in, at, n);
#pragma unroll
        for (int i = 0; i < V; ++i) x.v[i] = from_f32<T>(to_f32(x.v[i]) * c);
        store_row<T, V>(out, at, n, x);
    }
}

// A factor of 1 leaves tensors that are clipped in place as they are.
__global__ void __launch_bounds__(256)
    k_clip_chunks(ClipTable ct, int64_t chunk_size, const float *__restrict__ norm, float max_norm)
{
    const float r = max_norm / (norm[0] + 1e-6f);
    const float c = r > 1.0f ? 1.0f : r;             // NaN stays
    const Table<CLIP_TABLE> &t = ct.t;
    const uint32_t chunk = gridDim.x - 1 - blockIdx.x;
    const int i = find(t, chunk);
    if (c == 1.0f && ct.out[i] == t.in[i]) return;
    const int64_t size = t.size_type[i] & ((1ull << 56) - 1);
    const int64_t at = (int64_t)(chunk - t.first[i]) * chunk_size;
    const int64_t n = size - at < chunk_size ? size - at : chunk_size;
    switch (t.size_type[i] >> 56) {
    case F32: clip_chunk((const float *)t.in[i] + at, (float *)ct.out[i] + at, n, c); break;
    case BF16: clip_chunk((const bf16 *)t.in[i] + at, (bf16 *)ct.out[i] + at, n, c); break;
    default: clip_chunk((const f16 *)t.in[i] + at, (f16 *)ct.out[i] + at, n, c); break;
    }
}

// Elements of a chunk: about 4096 chunks in all, 4096 elements at least (so that a workgroup's
// start is paid for: 300x40001 float32 clipped within a graph in 24.6 us, 24.2 with 2048, 26.4 with
// 8192; a call for 20 x 1M bf16 normed 10.8, 14.7 and 10.8), in steps of 4096.
int64_t chunk_size(const int64_t *sizes, int64_t count)
{
    int64_t total = 0;
    for (int64_t i = 0; i < count; ++i) total += sizes[i];
    const int64_t want = (total / 4096 + 4095) / 4096 * 4096;
    return want < 4096 ? 4096 : want;
}

int64_t chunks_of(int64_t size, int64_t chunk) { return (size + chunk - 1) / chunk; }

// Fills the launch's table with up to N tensors that are not empty at a time and runs it on
// their chunks.
template <int N, typename Launch>
hipError_t each_table(const void *const *in, const int64_t *sizes, const int32_t *types,
                      int64_t count, Table<N> &t, Launch &launch)
{
    int64_t i = 0;
    while (i < count) {
        t.count = 0;
        uint32_t chunks = 0;
        for (; i < count && t.count < N; ++i) {
            if (sizes[i] == 0) continue;
            t.in[t.count] = in[i];
            t.size_type[t.count] = (uint64_t)sizes[i] | (uint64_t)types[i] << 56;
            t.first[t.count] = chunks;
            launch.entry(t.count, i);
            ++t.count;
            chunks += (uint32_t)chunks_of(sizes[i], launch.chunk);
        }
        t.first[t.count] = chunks;
        if (chunks) {
            launch.run(chunks);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    return hipSuccess;
}

// Whether the tensors fit one table and FEW_CHUNKS chunks.
bool few(const int64_t *sizes, int64_t count)
{
    int64_t chunks = 0, tensors = 0;
    for (int64_t i = 0; i < count && chunks <= FEW_CHUNKS; ++i) {
        chunks += chunks_of(sizes[i], FEW_CHUNK);
        tensors += sizes[i] != 0;
    }
    return chunks <= FEW_CHUNKS && tensors > 0;
}

struct NormLaunch {
    Table<NORM_TABLE> t;
    bool inf;
    int64_t chunk;
    double *partial;
    hipStream_t st;
    float *norm;              // of the whole, where one workgroup takes it
    void entry(int, int64_t) {}
    void run(uint32_t chunks)
    {
        if (norm) {
            if (inf) k_norm_few<true><<<1, 1024, 0, st>>>(t, norm);
            else k_norm_few<false><<<1, 1024, 0, st>>>(t, norm);
            return;
        }
        if (inf) k_norm_chunks<true><<<chunks, 256, 0, st>>>(t, chunk, partial);
        else k_norm_chunks<false><<<chunks, 256, 0, st>>>(t, chunk, partial);
        partial += chunks;
    }
};

struct ClipLaunch {
    ClipTable ct;
    void *const *outs;
    int64_t chunk;
    const float *norm;
    float max_norm;
    hipStream_t st;
    void entry(int slot, int64_t i) { ct.out[slot] = outs[i]; }
    void run(uint32_t chunks)
    {
        k_clip_chunks<<<chunks, 256, 0, st>>>(ct, chunk, norm, max_norm);
    }
};

}  // namespace nvfp4t

// 8 bytes for every chunk.
extern "C" size_t nvfp4t_norm_workspace(const int64_t *sizes, int64_t count)
{
    const int64_t chunk = nvfp4t::chunk_size(sizes, count);
    int64_t chunks = 0;
    for (int64_t i = 0; i < count; ++i) chunks += nvfp4t::chunks_of(sizes[i], chunk);
    return (size_t)chunks * sizeof(double);
}

extern "C" hipError_t nvfp4t_norm(const void *const *in, const int64_t *sizes,
                                  const int32_t *types, int64_t count, int inf, float *norm,
                                  void *workspace, hipStream_t st)
{
    using namespace nvfp4t;
    const bool one = few(sizes, count);
    NormLaunch l{{}, inf != 0, one ? FEW_CHUNK : chunk_size(sizes, count), (double *)workspace, st,
                 one ? norm : nullptr};
    const hipError_t e = each_table(in, sizes, types, count, l.t, l);
    if (e != hipSuccess || one) return e;
    const int64_t partials = l.partial - (double *)workspace;
    if (inf) k_norm_join<true><<<1, 1024, 0, st>>>((const double *)workspace, partials, norm);
    else k_norm_join<false><<<1, 1024, 0, st>>>((const double *)workspace, partials, norm);
    return hipGetLastError();
}

extern "C" hipError_t nvfp4t_clip(const void *const *in, void *const *out, const int64_t *sizes,
                                  const int32_t *types, int64_t count, float max_norm,
                                  const float *norm, hipStream_t st)
{
    using namespace nvfp4t;
    ClipLaunch l{{}, out, chunk_size(sizes, count), norm, max_norm, st};
    return each_table(in, sizes, types, count, l.ct.t, l);
}
