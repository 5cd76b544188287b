// block_adamw.hip -- one AdamW step over many tensors, for gfx950.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
//   p = p (1 - lr decay) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// Bound by memory: every element's parameter, gradient and moments are read once and the first and
// the last two written once, 28 bytes for float32 and for bfloat16 with a master copy, 10 for
// bfloat16 with moments in 8 bits.  The tensors are cut into chunks, one workgroup each, and
// their addresses travel in the kernel arguments, as in train_clip.hip.  Every operation is rounded
// by itself (no fused multiply-add): a code of an 8-bit moment hangs on its last bit, and so
// does whether two programs agree on it.
//
// Moments in 8 bits: a code is the upper bits of the float32 pattern of x 2^(15 - 127 - E), E
// the block's exponent: that moves exponents of 1 .. 15 over the float32's own smallest ones, below
// which a float32 has subnormals exactly where the code has them.  Rounding is an integer addition
// of noise below the cut, and decoding a shift of bits and one of the exponent.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "nvfp4_block.h"
#include "nvfp4_device.h"
#include "train_device.h"

namespace nvfp4t {

constexpr int TABLE32 = 72, TABLE8 = 52;
constexpr int BLOCK8 = 128;              // elements of a block, 8 in each of 16 lanes
constexpr int UNIT = 2048;               // elements that a workgroup takes at a time

// What one step multiplies by, from the step's number and the options.
struct Factors {
    float coef;                          // of the gradients
    float b1, c1, b2, c2;                // beta1, 1 - beta1, beta2, 1 - beta2
    float decay, rate, root, eps;        // 1 - lr decay, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
    uint32_t step;
};

struct Options {
    double lr, b1, b2, decay;
    int64_t step;
    const float *lr_device;
    const int64_t *step_device;
    const float *norm;
    float max_norm;
    uint32_t lowest;                     // code of an 8-bit r > 0: 1 or 0
    uint64_t seed;
    Factors f;                           // of the host's lr and step
};

// b^t by squaring: the same operations on the host and on the device, so the same bits.
__host__ __device__ inline double power(double b, int64_t t)
{
    double r = 1.0;
    for (; t > 0; t >>= 1, b *= b)
        if (t & 1) r *= b;
    return r;
}

__host__ __device__ inline void set_factors(Factors &f, double lr, double b1, double b2,
                                            double decay, int64_t step)
{
    if (step < 1) step = 1;
    f.decay = (float)(1.0 - lr * decay);
    f.rate = (float)(lr / (1.0 - power(b1, step)));
    f.root = (float)(1.0 / sqrt(1.0 - power(b2, step)));
    f.step = (uint32_t)step;
}

__device__ __forceinline__ Factors factors(const Options &o)
{
    Factors f = o.f;
    if (o.lr_device || o.step_device)
        set_factors(f, o.lr_device ? (double)*o.lr_device : o.lr, o.b1, o.b2, o.decay,
                    o.step_device ? *o.step_device : o.step);
    if (o.norm) {
        const float r = o.max_norm / (*o.norm + 1e-6f);
        f.coef = r > 1.0f ? 1.0f : r;                  // NaN stays
    }
    return f;
}

// Tensor i holds `size` elements and chunks first[i] .. first[i + 1] - 1 of the launch.  The
// element type lies in the upper byte of `size_type`.
template <int N> struct Tensors {
    void *p[N];
    const void *g[N];
    void *m[N];
    void *v[N];
    float *master[N];
    uint64_t size_type[N];
    uint32_t first[N + 1];
    int32_t count;
};

struct Tensors8 {
    Tensors<TABLE8> t;
    uint8_t *m_scale[TABLE8];
    uint8_t *v_scale[TABLE8];
    uint32_t index[TABLE8];
};

static_assert(sizeof(Tensors<TABLE32>) + sizeof(Options) + 16 <= 4096 &&
                  sizeof(Tensors8) + sizeof(Options) + 16 <= 4096,
              "the tables have to fit the kernel arguments");

// The tensor that a chunk belongs to: the last one whose first chunk is not past it, found by a wave in
// one read of the table (a search by halves is six reads, each waiting for the one before).
template <int N>
__device__ __forceinline__ int tensor_of(const Tensors<N> &t, uint32_t chunk)
{
    const int lane = threadIdx.x & 63;
    int before = 0;
#pragma unroll
    for (int k = 0; k < N; k += 64) {
        const bool reached = k + lane < t.count && t.first[k + lane < N ? k + lane : N] <= chunk;
        before += __popcll(__ballot(reached));
    }
    return __builtin_amdgcn_readfirstlane(before) - 1;
}

template <typename T, int N>
__device__ __forceinline__ T *at_of(void *const (&a)[N], int i, int64_t at)
{
    return static_cast<T *>(a[i]) + at;
}

// V elements at a thread's place; WHOLE: all of them exist (else zeros past n, and none written).  Units
// without an end have a loop of their own, in which every access is one instruction.
template <bool WHOLE, typename T, int V>
__device__ __forceinline__ Pack<T, V> load_at(const T *p, int64_t at, int64_t n)
{
    if constexpr (WHOLE) return *reinterpret_cast<const Pack<T, V> *>(p + at);
    else return load_row<T, V>(p, at, n);
}

template <bool WHOLE, typename T, int V>
__device__ __forceinline__ void store_at(T *p, int64_t at, int64_t n, const Pack<T, V> &x)
{
    if constexpr (WHOLE) *reinterpret_cast<Pack<T, V> *>(p + at) = x;
    else store_row<T, V>(p, at, n, x);
}

// One parameter's elements with moments in 32 bits.
__device__ __forceinline__ void update(float &p, float &m, float &v, float g, const Factors &f)
{
    g = g * f.coef;
    m = f.b1 * m + f.c1 * g;
    v = f.b2 * v + f.c2 * (g * g);
    p = p * f.decay - f.rate * (m / (sqrtf(v) * f.root + f.eps));
}

// Elements [base, base + UNIT) of a workgroup, four a thread at a time.  WHOLE: all of them exist.
template <typename T, bool MASTER, bool WHOLE>
__device__ __forceinline__ void unit32(T *__restrict__ p, const T *__restrict__ g,
                                       float *__restrict__ m, float *__restrict__ v,
                                       float *__restrict__ master, int64_t base, int64_t n,
                                       const Factors &f)
{
    constexpr int V = 4, U = UNIT / 256 / V;
    Pack<T, V> pp[U], gg[U];
    Pack<float, V> mm[U], vv[U], ww[U];
    base += V * threadIdx.x;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t at = base + u * 256 * V;
        gg[u] = load_at<WHOLE, T, V>(g, at, n);
        if constexpr (MASTER) ww[u] = load_at<WHOLE, float, V>(master, at, n);
        else pp[u] = load_at<WHOLE, T, V>(p, at, n);
        mm[u] = load_at<WHOLE, float, V>(m, at, n);
        vv[u] = load_at<WHOLE, float, V>(v, at, n);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t at = base + u * 256 * V;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float x = MASTER ? ww[u].v[i] : to_f32(pp[u].v[i]);
            update(x, mm[u].v[i], vv[u].v[i], to_f32(gg[u].v[i]), f);
            pp[u].v[i] = from_f32<T>(x);
            ww[u].v[i] = x;
        }
        store_at<WHOLE, T, V>(p, at, n, pp[u]);
        if constexpr (MASTER) store_at<WHOLE, float, V>(master, at, n, ww[u]);
        store_at<WHOLE, float, V>(m, at, n, mm[u]);
        store_at<WHOLE, float, V>(v, at, n, vv[u]);
    }
}

template <typename T, bool MASTER>
__device__ __forceinline__ void step32(T *__restrict__ p, const T *__restrict__ g,
                                       float *__restrict__ m, float *__restrict__ v,
                                       float *__restrict__ master, int64_t n, const Factors &f)
{
    int64_t base = 0;
    for (; base + UNIT <= n; base += UNIT) unit32<T, MASTER, true>(p, g, m, v, master, base, n, f);
    if (base < n) unit32<T, MASTER, false>(p, g, m, v, master, base, n, f);
}

template <typename T, int N>
__device__ __forceinline__ void chunk32(const Tensors<N> &t, int i, int64_t at, int64_t n,
                                        const Factors &f)
{
    T *p = at_of<T>(t.p, i, at);
    const T *g = static_cast<const T *>(t.g[i]) + at;
    float *m = at_of<float>(t.m, i, at), *v = at_of<float>(t.v, i, at);
    if constexpr (!std::is_same<T, float>::value) {
        if (t.master[i]) {
            step32<T, true>(p, g, m, v, t.master[i] + at, n, f);
            return;
        }
    }
    step32<T, false>(p, g, m, v, nullptr, n, f);
}

__global__ void __launch_bounds__(256) k_adamw32(Tensors<TABLE32> t, int64_t chunk_size, Options o)
{
    const Factors f = factors(o);
    const int i = tensor_of(t, blockIdx.x);
    const int64_t size = t.size_type[i] & ((1ull << 56) - 1);
    const int64_t at = (int64_t)(blockIdx.x - t.first[i]) * chunk_size;
    const int64_t n = size - at < chunk_size ? size - at : chunk_size;
    switch (t.size_type[i] >> 56) {
    case F32: chunk32<float>(t, i, at, n, f); break;
    case BF16: chunk32<bf16>(t, i, at, n, f); break;
    default: chunk32<f16>(t, i, at, n, f); break;
    }
}

// The largest over a block's 16 lanes (a row of the data-parallel primitives), in each of them.
template <int ROTATE> __device__ __forceinline__ uint32_t row_max(uint32_t x)
{
    const uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x120 + ROTATE, 0xf, 0xf,
                                                             false);
    return x > y ? x : y;
}

__device__ __forceinline__ uint32_t block_max(uint32_t x)
{
    return row_max<1>(row_max<2>(row_max<4>(row_max<8>(x))));
}

// The scale byte of a block whose largest magnitude has the bits `top`: the exponent of the smallest
// number of FRACTION bits that is not below it.
template <int FRACTION> __device__ __forceinline__ uint32_t scale_byte(uint32_t top)
{
    const uint32_t e = (top + (1u << (23 - FRACTION)) - 1) >> 23;
    return e < 1 ? 1 : e > 253 ? 255 : e;
}

// |x| as a code, by 16 bits of noise; shift = 15 - scale byte.  The block's scale covers every |x|, so
// noise cannot carry past the largest code (a block that is not finite has any codes).
template <int FRACTION>
__device__ __forceinline__ uint32_t encode(float x, int shift, uint32_t noise)
{
    constexpr int CUT = 23 - FRACTION;
    return (__float_as_uint(ldexpf(fabsf(x), shift)) + (noise << (CUT - 16))) >> CUT;
}

// r's value of byte `at` of four codes; shift = scale byte - 15.
__device__ __forceinline__ float decode_r(uint32_t codes, int at, int shift)
{
    return ldexpf(__uint_as_float((codes >> (8 * at) & 255u) << 19), shift);
}

// m's: the byte's sign and magnitude, from the top, to the places of a float32's.
__device__ __forceinline__ float decode_m(uint32_t codes, int at, int shift)
{
    const uint32_t x = (uint32_t)((int32_t)(codes << (24 - 8 * at)) >> 4) & 0x87F00000u;
    return ldexpf(__uint_as_float(x), shift);
}

// sqrt rounded to nearest for x = 0 or x >= 2^-96 (below, where the instruction's own 2 U do not
// hold, through sqrtf): of the instruction's result and its two neighbours the one whose
// boundaries hold x.
__device__ __forceinline__ float root_of(float x)
{
    const float s = __builtin_amdgcn_sqrtf(x);
    const float down = __uint_as_float(__float_as_uint(s) - 1), up = __uint_as_float(
                                                                    __float_as_uint(s) + 1);
    float r = s;
    if (__builtin_fmaf(-down, s, x) <= 0.0f) r = down;
    if (__builtin_fmaf(-up, s, x) > 0.0f) r = up;
    return x == 0.0f || x == __builtin_huge_valf() ? x : r;
}

// v[0] last, the others one place on: a loop over a few registers without its body eight times.
template <int N> __device__ __forceinline__ void rotate(float (&v)[N])
{
    const float first = v[0];
#pragma unroll
    for (int i = 0; i + 1 < N; ++i) v[i] = v[i + 1];
    v[N - 1] = first;
}

// A unit with moments in 8 bits: 8 elements a lane, a block in 16 lanes.  `first` is the chunk's
// first element in the tensor, n its elements; the last block's lanes past the end hold zeros.
// Vector instructions bound it, 85 an element (Philox is a third of their time): 100 million elements
// bf16 in 225 us, 4.5 TB/s (280 with two multiplications for each shift of an exponent, sqrtf and
// quotients rounded once).
template <typename T, bool MASTER, bool WHOLE>
__device__ __forceinline__ void unit8(T *__restrict__ p, const T *__restrict__ g,
                                      uint8_t *__restrict__ m, uint8_t *__restrict__ r,
                                      uint8_t *__restrict__ m_scale, uint8_t *__restrict__ r_scale,
                                      float *__restrict__ master, int64_t first, int64_t base,
                                      int64_t n, uint32_t tensor, uint64_t seed, uint32_t lowest,
                                      const Factors &f)
{
    constexpr int V = 8;
    const int64_t at = base + V * threadIdx.x;
    if (at / BLOCK8 * BLOCK8 >= n) return;             // the whole block: 16 lanes together
    const int64_t block = at / BLOCK8;
    const Pack<T, V> gg = load_at<WHOLE, T, V>(g, at, n);
    Pack<T, V> pp{};
    Pack<float, V> ww{};
    if constexpr (MASTER) ww = load_at<WHOLE, float, V>(master, at, n);
    else pp = load_at<WHOLE, T, V>(p, at, n);
    const uint2 mc = *reinterpret_cast<const uint2 *>(m + at);
    const uint2 rc = *reinterpret_cast<const uint2 *>(r + at);
    const uint32_t ms = m_scale[block], rs = r_scale[block];
    // of a block that is not finite nothing is kept but that
    const float nan = __uint_as_float(0x7FC00000u);
    const float b1 = ms == 255u ? nan : f.b1, b2 = rs == 255u ? nan : f.b2;
    const int m_shift = (int)ms - 15, r_shift = (int)rs - 15;
    float mm[V], rr[V], least = __builtin_huge_valf();
    uint32_t m_top = 0, r_top = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float grad = to_f32(gg.v[i]) * f.coef;
        const float old = decode_r(i < 4 ? rc.x : rc.y, i & 3, r_shift);
        mm[i] = b1 * decode_m(i < 4 ? mc.x : mc.y, i & 3, m_shift) + f.c1 * grad;
        rr[i] = b2 * (old * old) + f.c2 * (grad * grad);
        if (rr[i] != 0.0f) least = fminf(least, rr[i]);
    }
    if (__any(least < 0x1p-96f)) {
#pragma unroll 1
        for (int i = 0; i < V; ++i) rr[0] = sqrtf(rr[0]), rotate(rr);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) rr[i] = root_of(rr[i]);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t a = __float_as_uint(mm[i]) & 0x7FFFFFFFu, b = __float_as_uint(rr[i]);
        m_top = a > m_top ? a : m_top;
        r_top = b > r_top ? b : r_top;
        float x = MASTER ? ww.v[i] : to_f32(pp.v[i]);
        // (a quotient rounded once would take 14 us more for 100 million elements bf16)
        x = x * f.decay - f.rate * (mm[i] * __builtin_amdgcn_rcpf(rr[i] * f.root + f.eps));
        pp.v[i] = from_f32<T>(x);
        ww.v[i] = x;
    }
    store_at<WHOLE, T, V>(p, at, n, pp);
    if constexpr (MASTER) store_at<WHOLE, float, V>(master, at, n, ww);
    // (r's sign bit is only ever a NaN's, whose bits scale_byte would carry past the word's end)
    const uint32_t sm = scale_byte<3>(block_max(m_top));
    const uint32_t sr = scale_byte<4>(block_max(r_top & 0x7FFFFFFFu));
    const int m_out = 15 - (int)sm, r_out = 15 - (int)sr;
    uint32_t cm[2] = {0, 0}, cr[2] = {0, 0};
    const uint64_t group = (uint64_t)(first + at) >> 2;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const nvfp4k::Word4 w = nvfp4k::philox(seed, (uint32_t)(group + q),
                                               (uint32_t)((group + q) >> 32),
                                               0x80000000u + tensor, f.step);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t c = encode<3>(mm[4 * q + i], m_out, w.w[i] >> 16);
            const uint32_t sign = c ? __float_as_uint(mm[4 * q + i]) >> 24 & 128u : 0u;
            cm[q] |= (c | sign) << (8 * i);
            const uint32_t d = encode<4>(rr[4 * q + i], r_out, w.w[i] & 0xFFFFu);
            // code 1 at least, where asked for and r is not 0
            const uint32_t r_bits = __float_as_uint(rr[4 * q + i]);
            const uint32_t floor = r_bits < lowest ? r_bits : lowest;
            cr[q] |= (d > floor ? d : floor) << (8 * i);
        }
    }
    *reinterpret_cast<uint2 *>(m + at) = make_uint2(cm[0], cm[1]);
    *reinterpret_cast<uint2 *>(r + at) = make_uint2(cr[0], cr[1]);
    if (threadIdx.x % 16 == 0) {
        m_scale[block] = (uint8_t)sm;
        r_scale[block] = (uint8_t)sr;
    }
}

template <typename T, bool MASTER>
__device__ __forceinline__ void step8(T *__restrict__ p, const T *__restrict__ g,
                                      uint8_t *__restrict__ m, uint8_t *__restrict__ r,
                                      uint8_t *__restrict__ m_scale, uint8_t *__restrict__ r_scale,
                                      float *__restrict__ master, int64_t first, int64_t n,
                                      uint32_t tensor, uint64_t seed, uint32_t lowest,
                                      const Factors &f)
{
    int64_t base = 0;
    for (; base + UNIT <= n; base += UNIT)
        unit8<T, MASTER, true>(p, g, m, r, m_scale, r_scale, master, first, base, n, tensor, seed, lowest,
                               f);
    if (base < n)
        unit8<T, MASTER, false>(p, g, m, r, m_scale, r_scale, master, first, base, n, tensor, seed,
                                lowest, f);
}

template <typename T>
__device__ __forceinline__ void chunk8(const Tensors8 &t8, int i, int64_t at, int64_t n,
                                       uint64_t seed, uint32_t lowest, const Factors &f)
{
    const Tensors<TABLE8> &t = t8.t;
    T *p = at_of<T>(t.p, i, at);
    const T *g = static_cast<const T *>(t.g[i]) + at;
    uint8_t *m = at_of<uint8_t>(t.m, i, at), *r = at_of<uint8_t>(t.v, i, at);
    uint8_t *ms = t8.m_scale[i] + at / BLOCK8, *rs = t8.v_scale[i] + at / BLOCK8;
    if constexpr (!std::is_same<T, float>::value) {
        if (t.master[i]) {
            step8<T, true>(p, g, m, r, ms, rs, t.master[i] + at, at, n, t8.index[i], seed, lowest,
                           f);
            return;
        }
    }
    step8<T, false>(p, g, m, r, ms, rs, nullptr, at, n, t8.index[i], seed, lowest, f);
}

__global__ void __launch_bounds__(256) k_adamw8(Tensors8 t8, int64_t chunk_size, Options o)
{
    const Factors f = factors(o);
    const Tensors<TABLE8> &t = t8.t;
    const int i = tensor_of(t, blockIdx.x);
    const int64_t size = t.size_type[i] & ((1ull << 56) - 1);
    const int64_t at = (int64_t)(blockIdx.x - t.first[i]) * chunk_size;
    const int64_t n = size - at < chunk_size ? size - at : chunk_size;
    switch (t.size_type[i] >> 56) {
    case F32: chunk8<float>(t8, i, at, n, o.seed, o.lowest, f); break;
    case BF16: chunk8<bf16>(t8, i, at, n, o.seed, o.lowest, f); break;
    default: chunk8<f16>(t8, i, at, n, o.seed, o.lowest, f); break;
    }
}

// 8 codes a thread; a workgroup's 2048 codes are 16 blocks.
template <bool SECOND>
__global__ void __launch_bounds__(256)
    k_moment_values(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                    int64_t count, float *__restrict__ out)
{
    const int64_t stride = (int64_t)gridDim.x * UNIT;
    for (int64_t at = (int64_t)blockIdx.x * UNIT + 8 * threadIdx.x; at < count; at += stride) {
        const uint2 c = *reinterpret_cast<const uint2 *>(codes + at);
        const uint32_t s = scales[at / BLOCK8];
        const int shift = (int)s - 15;
        Pack<float, 4> x[2];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t four = i < 4 ? c.x : c.y;
            const float v = SECOND ? decode_r(four, i & 3, shift) : decode_m(four, i & 3, shift);
            x[i >> 2].v[i & 3] = s == 255u ? __uint_as_float(0x7FC00000u) : v;
        }
        *reinterpret_cast<Pack<float, 4> *>(out + at) = x[0];
        *reinterpret_cast<Pack<float, 4> *>(out + at + 4) = x[1];
    }
}

// Elements of a chunk: about 4096 chunks in all, whole units (the same elements share a block of
// an 8-bit moment, whatever the chunks).
int64_t adamw_chunk(const adamw_tensor *t, int64_t count)
{
    int64_t total = 0;
    for (int64_t i = 0; i < count; ++i) total += t[i].size;
    const int64_t want = (total / 4096 + UNIT - 1) / UNIT * UNIT;
    return want < UNIT ? UNIT : want;
}

template <int N> void put(Tensors<N> &t, const adamw_tensor &x, int64_t chunk, uint32_t &chunks)
{
    const int k = t.count++;
    t.p[k] = x.param;
    t.g[k] = x.grad;
    t.m[k] = x.m;
    t.v[k] = x.v;
    t.master[k] = x.master;
    t.size_type[k] = (uint64_t)x.size | (uint64_t)x.type << 56;
    t.first[k] = chunks;
    chunks += (uint32_t)((x.size + chunk - 1) / chunk);
    t.first[k + 1] = chunks;
}

}  // namespace nvfp4t

extern "C" hipError_t nvfp4t_adamw(const adamw_tensor *tensors, int64_t count,
                                   const adamw_options *options, hipStream_t st)
{
    using namespace nvfp4t;
    Options o{};
    o.lr = options->lr;
    o.b1 = options->beta1;
    o.b2 = options->beta2;
    o.decay = options->weight_decay;
    o.step = options->step;
    o.lr_device = options->lr_device;
    o.step_device = options->step_device;
    o.norm = options->norm;
    o.max_norm = options->max_norm;
    o.lowest = (uint32_t)options->bounded;
    o.seed = options->seed;
    o.f.coef = 1.0f;
    o.f.b1 = (float)o.b1;
    o.f.c1 = (float)(1.0 - o.b1);
    o.f.b2 = (float)o.b2;
    o.f.c2 = (float)(1.0 - o.b2);
    o.f.eps = (float)options->eps;
    set_factors(o.f, o.lr, o.b1, o.b2, o.decay, o.step);
    const int64_t chunk = adamw_chunk(tensors, count);
    Tensors<TABLE32> t32;
    Tensors8 t8;
    t32.count = t8.t.count = 0;
    uint32_t chunks32 = 0, chunks8 = 0;
    auto run32 = [&] {
        if (chunks32) k_adamw32<<<chunks32, 256, 0, st>>>(t32, chunk, o);
        t32.count = chunks32 = 0;
        return hipGetLastError();
    };
    auto run8 = [&] {
        if (chunks8) k_adamw8<<<chunks8, 256, 0, st>>>(t8, chunk, o);
        t8.t.count = chunks8 = 0;
        return hipGetLastError();
    };
    for (int64_t i = 0; i < count; ++i) {
        const adamw_tensor &x = tensors[i];
        if (x.size == 0) continue;
        hipError_t e = hipSuccess;
        if (x.bits == 32) {
            put(t32, x, chunk, chunks32);
            if (t32.count == TABLE32) e = run32();
        } else {
            const int k = t8.t.count;
            t8.m_scale[k] = x.m_scale;
            t8.v_scale[k] = x.v_scale;
            t8.index[k] = (uint32_t)i;
            put(t8.t, x, chunk, chunks8);
            if (t8.t.count == TABLE8) e = run8();
        }
        if (e != hipSuccess) return e;
    }
    const hipError_t e = run32();
    return e != hipSuccess ? e : run8();
}

extern "C" hipError_t nvfp4t_moment_values(const uint8_t *codes, const uint8_t *scales,
                                           int64_t blocks, int second, float *out, hipStream_t st)
{
    using namespace nvfp4t;
    if (blocks == 0) return hipSuccess;
    const int64_t groups = (blocks * BLOCK8 + UNIT - 1) / UNIT;
    const unsigned grid = (unsigned)(groups < MAX_GROUPS ? groups : MAX_GROUPS);
    const int64_t n = blocks * BLOCK8;
    if (second) k_moment_values<true><<<grid, 256, 0, st>>>(codes, scales, n, out);
    else k_moment_values<false><<<grid, 256, 0, st>>>(codes, scales, n, out);
    return hipGetLastError();
}
