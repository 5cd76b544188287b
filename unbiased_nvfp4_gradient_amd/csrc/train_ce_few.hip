// train_ce_few.hip -- the linear head's cross entropy for up to 128 tokens, for gfx950.
//
// With few tokens the head w [v][d] is what has to move: the products read it as it lies, rows
// straight into matrix-instruction fragments, once in the forward pass and twice in the
// backward pass (logits and dw; dh), with nothing laid out first and no tiles of 256 tokens.
//   k_ce_few     32 or 64 words a workgroup: logits, then either their largest and sum of
//                exponentials, or q and the words' rows of dw
//   k_ce_few_dh  256 (or 128) columns and a run of words a workgroup: FP32 sums of q w
// Measured, 2048x131072 bf16 (537 MB of head): 7 tokens forward 110 us (4.9 TB/s, a large copy's
// rate), backward 384 (4.2 TB/s of the three passes over the head); 128 tokens 220 and 666, where
// the tokens' rows from L2 weigh as much as the head.
// Every product is v_mfma_f32_32x32x16, whose K elements may be taken in any order as long as
// both operands agree; that order is chosen so that a wave's loads are whole lines.
#include "train_ce.h"

#pragma clang fp contract(fast)

namespace nvfp4t {

// Eight elements from `at` of a row of n (zeros past its end), as a fragment.
template <typename T> __device__ __forceinline__ int4v fragment(const T *row, int64_t at)
{
    return __builtin_bit_cast(int4v, *reinterpret_cast<const Pack<T, 8> *>(row + at));
}

template <typename T>
__device__ __forceinline__ int4v fragment(const T *row, int64_t at, int64_t n)
{
    return __builtin_bit_cast(int4v, load_row<T, 8>(row, at, n));
}

// q as two numbers of 16 bits, itself rounded (HALF 0) and what that leaves rounded (1), whose
// products with the other operand add up in FP32.  A gradient of a few tokens can be a single
// product, in which one rounding of q would weigh as much as the output's own (13 tokens f16: dw off
// by up to 0.00038 of its norm, 0.00021 with both halves).  The head's bytes bound these kernels up
// to some 64 tokens, not the products (2048x131072 bf16 backward, with one half and with both: 7
// tokens 378 and 384 us, 64 tokens 427 and 461, 128 tokens 583 and 666).
template <typename T, int HALF> __device__ __forceinline__ T half_of(float x)
{
    const T hi = from_f32<T>(x);
    if constexpr (HALF == 0) return hi;
    return from_f32<T>(__builtin_isinf(x) ? 0.0f : x - to_f32(hi));
}

// Row and column of accumulator r of lane l in a 32 x 32 block: [row_of(r, l)][l % 32].
__device__ __forceinline__ int row_of(int r, int lane)
{
    return 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
}

template <int N> struct Number { static constexpr int value = N; };

// A forward pass gathers the tokens that count itself (their order kept; every workgroup does,
// the first one leaves it for the kernel that joins the parts).
struct Gather {
    const int64_t *target;
    int64_t ignore;
    float *loss_each, *lse;    // outputs, 0 where a token does not count; loss_each may be null
};

// 32 WB words and all 32 NB tokens a workgroup.  Its four waves share the head's columns, 16 J
// at a time in turns, and join their sums in their order through LDS; a thread then holds
// words 8 i + 4 (lane / 32) + wave of every 32 for one token of every 32.
// h comes as it lies, or from hk [column / 32][hk_rows tokens][32 columns] where that is given.
// GRAD false: partial[token][group] = (largest logit, sum of exponentials against it) of the
// group's words, and the target's logit.
// GRAD true: q [half][word / 32][32 NB tokens][32 words], and dw = scale q^T h from it (where
// weighted, with the tokens' weights in it) while it lies in LDS, h coming from ht
// [token / 32][dp][32 tokens].
template <typename T, int NB, int WB, bool GRAD>
__global__ void __launch_bounds__(256)
    k_ce_few(Head a, Gather gather, Tokens tok, const T *__restrict__ hk, int64_t hk_rows,
             float2 *__restrict__ partial, float *__restrict__ at_target, bool weighted,
             const uint8_t *__restrict__ ht, int64_t dp, uint8_t *__restrict__ q_out,
             T *__restrict__ dw)
{
    constexpr int N = 32 * NB, J = NB == 4 ? 2 : 4, KS = 16 * J;
    constexpr int PARTS = NB * WB > 1 ? 2 : 1;
    constexpr int QS = N + 8, QT = 40;           // row lengths of q in LDS, by word and by token
    constexpr int PART_BYTES = PARTS * 4 * 16 * 64 * 4;
    constexpr int Q_BYTES = GRAD ? 2 * 32 * WB * QS + 2 * WB * N * QT : 0;
    constexpr int OUT_ROW = 144, OUT_BYTES = GRAD ? 4 * 32 * OUT_ROW : 0;    // dw on its way
    constexpr int MOST = PART_BYTES > Q_BYTES ? PART_BYTES : Q_BYTES;
    __shared__ __attribute__((aligned(16))) uint8_t lds[MOST > OUT_BYTES ? MOST : OUT_BYTES];
    __shared__ int32_t index[N], target[N];
    __shared__ float2 stats[4][N];
    __shared__ int32_t counts[2];
    const int lane = threadIdx.x & 63, half = lane >> 5, r = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    int32_t kept;
    if constexpr (GRAD) {
        kept = tok.info->kept;
        if (threadIdx.x < N) {
            index[threadIdx.x] = tok.index[threadIdx.x];
            target[threadIdx.x] = tok.target[threadIdx.x];
        }
    } else {
        const int64_t y = threadIdx.x < a.t ? gather.target[threadIdx.x] : gather.ignore;
        const bool keep = y != gather.ignore;
        const uint64_t mask = __ballot(keep);
        if (lane == 0 && wave < 2) counts[wave] = __popcll(mask);
        __syncthreads();
        kept = counts[0] + counts[1];            // t is 128 at most: two waves' tokens
        if (keep) {
            const int slot = (wave ? counts[0] : 0) + __popcll(mask & ((1ull << lane) - 1));
            index[slot] = (int32_t)threadIdx.x;
            target[slot] = y >= 0 && y < a.v ? (int32_t)y : -1;
            if (blockIdx.x == 0) {
                tok.index[slot] = index[slot];
                tok.target[slot] = target[slot];
            }
        } else if (blockIdx.x == 0 && threadIdx.x < a.t) {
            gather.lse[threadIdx.x] = 0.0f;
            if (gather.loss_each) gather.loss_each[threadIdx.x] = 0.0f;
        }
        if (blockIdx.x == 0 && threadIdx.x == 0) tok.info->kept = kept;
        if (kept == 0) return;
    }
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * 32 * WB;

    // logits: rows are words, columns tokens.  Words past the vocabulary read its last row, and
    // tokens past the last one that counts read that: neither's results are used.
    f32x16 acc[WB][NB];
#pragma unroll
    for (int i = 0; i < WB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = f32x16{};
    if (kept > 0) {
        const T *wr[WB], *hr[NB];
#pragma unroll
        for (int i = 0; i < WB; ++i) {
            const int64_t word = first + 32 * i + r;
            wr[i] = (const T *)a.w + (word < a.v ? word : a.v - 1) * a.w_stride;
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int slot = 32 * j + r;
            hr[j] = hk ? hk + 32 * slot
                       : (const T *)a.h + index[slot < kept ? slot : kept - 1] * a.h_stride;
        }
        const int64_t h32 = hk ? 32 * hk_rows : 32;       // from 32 columns to the next
        const int64_t whole = a.d / KS;          // steps that end inside the rows
        // the next step's w loads while the present one is multiplied; h comes from L2
        int4v wn[WB][J];
        int64_t k = wave;
        auto load_w = [&](int64_t step) {
#pragma unroll
            for (int i = 0; i < WB; ++i)
#pragma unroll
                for (int x = 0; x < J; ++x)
                    wn[i][x] = fragment<T>(wr[i], step * KS + 16 * x + 8 * half);
        };
        auto multiply = [&](const int4v (&wf)[WB][J], const int4v (&hf)[NB][J]) {
#pragma unroll
            for (int x = 0; x < J; ++x)
#pragma unroll
                for (int i = 0; i < WB; ++i)
#pragma unroll
                    for (int j = 0; j < NB; ++j)
                        acc[i][j] = mfma(T{}, wf[i][x], hf[j][x], acc[i][j]);
        };
        if (k < whole) load_w(k);
        for (; k < whole; k += 4) {
            int4v wf[WB][J], hf[NB][J];
#pragma unroll
            for (int i = 0; i < WB; ++i)
#pragma unroll
                for (int x = 0; x < J; ++x) wf[i][x] = wn[i][x];
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int x = 0; x < J; ++x)
                    hf[j][x] = fragment<T>(hr[j], (k * (J / 2) + (x >> 1)) * h32 + 16 * (x & 1) +
                                                      8 * half);
            if (k + 4 < whole) load_w(k + 4);
            multiply(wf, hf);
        }
        if (k == whole && a.d % KS) {            // the rows' last elements, zeros past them
            int4v wf[WB][J], hf[NB][J];
#pragma unroll
            for (int x = 0; x < J; ++x) {
                const int64_t at = k * KS + 16 * x + 8 * half;
#pragma unroll
                for (int i = 0; i < WB; ++i) wf[i][x] = fragment<T>(wr[i], at, a.d);
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    hf[j][x] = int4v{};
                    if (!hk)
                        hf[j][x] = fragment<T>(hr[j], at, a.d);
                    else if (at < a.d)           // zeros from a.d to the end of the 32
                        hf[j][x] = fragment<T>(hr[j], (at >> 5) * h32 + (at & 31));
                }
            }
            multiply(wf, hf);
        }
    }

    // the waves' sums together: wave g takes accumulators g, 4 + g, 8 + g and 12 + g of every
    // lane
    float l[WB][NB][4];
    float *part = reinterpret_cast<float *>(lds);
#pragma unroll
    for (int i = 0; i < WB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            float *p = part + (PARTS == 2 ? (i * NB + j) & 1 : 0) * 4 * 1024;
#pragma unroll
            for (int x = 0; x < 16; ++x) p[wave * 1024 + x * 64 + lane] = acc[i][j][x];
            __syncthreads();
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float *s = p + (4 * x + wave) * 64 + lane;
                l[i][j][x] = ((s[0] + s[1024]) + s[2048]) + s[3072];
            }
        }
    // l[i][j][x]: word first + 32 i + 8 x + mine, token 32 j + r
    const int mine = 4 * half + wave;
    const int left = (int)(a.v - first < 32 * WB ? a.v - first : 32 * WB) - mine;

    if constexpr (!GRAD) {
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int y = (int)(target[32 * j + r < kept ? 32 * j + r : 0] - first) - mine;
            float top = -__builtin_inff(), sum = 0.0f;
#pragma unroll
            for (int i = 0; i < WB; ++i)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    if (32 * i + 8 * x == y && 32 * j + r < kept)
                        at_target[32 * j + r] = l[i][j][x];
                    l[i][j][x] = 32 * i + 8 * x < left ? l[i][j][x] : -__builtin_inff();
                    top = fmaxf(top, l[i][j][x]);
                }
            const float base = base_of(top);
#pragma unroll
            for (int i = 0; i < WB; ++i)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    sum += exp_from(l[i][j][x], base);
            const float2 own = make_float2(top, sum);
            const float2 all = join_stats(
                own, make_float2(__shfl_xor(own.x, 32), __shfl_xor(own.y, 32)));
            if (half == 0) stats[wave][32 * j + r] = all;
        }
        __syncthreads();
        if ((int)threadIdx.x < kept) {
            float2 s = stats[0][threadIdx.x];
            for (int g = 1; g < 4; ++g) s = join_stats(s, stats[g][threadIdx.x]);
            partial[(int64_t)threadIdx.x * gridDim.x + blockIdx.x] = s;
        }
    } else {
        using U = uint16_t;
        U *qw = reinterpret_cast<U *>(lds), *qt = qw + 32 * WB * QS;
        __syncthreads();                         // the last of `part` has been read
        float share[NB];
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int t = 32 * j + r;
            const float lse = tok.lse[t];
            const int y = (int)(target[t] - first) - mine;
            share[j] = weighted ? tok.share[t] : 1.0f;
#pragma unroll
            for (int i = 0; i < WB; ++i)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int word = 32 * i + 8 * x;
                    float v = exp_from(l[i][j][x], lse);
                    v = (v - (y == word ? 1.0f : 0.0f)) * Q_ONE<T>;
                    l[i][j][x] = word < left && t < kept ? v : 0.0f;
                }
        }
        // one half after the other through the same LDS
        int4v qf[2][WB][2 * NB];
        auto halve = [&](auto second) {
            constexpr int HALF = decltype(second)::value;
#pragma unroll
            for (int j = 0; j < NB; ++j)
#pragma unroll
                for (int i = 0; i < WB; ++i)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int word = 32 * i + 8 * x + mine, t = 32 * j + r;
                        const float v = l[i][j][x];
                        qt[(i * N + t) * QT + 8 * x + mine] =
                            __builtin_bit_cast(U, half_of<T, HALF>(v));
                        qw[word * QS + t] = __builtin_bit_cast(U, half_of<T, HALF>(v * share[j]));
                    }
            __syncthreads();
            // a tile of 32 words by 32 NB tokens: 64 bytes a token
            uint8_t *out = q_out + (HALF * (int64_t)gridDim.x + blockIdx.x) * WB * N * 64;
            for (int e = threadIdx.x; e < WB * N * 4; e += 256)
                *reinterpret_cast<uint4 *>(out + 16 * e) =
                    *reinterpret_cast<const uint4 *>(qt + (e >> 2) * QT + 8 * (e & 3));
#pragma unroll
            for (int i = 0; i < WB; ++i)
#pragma unroll
                for (int x = 0; x < 2 * NB; ++x)
                    qf[HALF][i][x] = *reinterpret_cast<const int4v *>(
                        qw + (32 * i + r) * QS + 16 * x + 8 * half);
            __syncthreads();                     // q has been read, its place is taken
        };
        halve(Number<0>{});
        halve(Number<1>{});
        if (!dw) return;
        // dw: rows are the head's columns, columns words; K runs over the tokens that count
        const float scale = tok.info->scale;
        uint8_t *mine_out = lds + wave * 32 * OUT_ROW;
        // two blocks of 32 columns at a time: 128 bytes of each word's row, which 8 lanes then
        // store in one piece (one token, 4096x131072: backward 769 us, 905 with 32 bytes from each
        // of two lanes)
        for (int64_t c0 = 64 * wave; c0 < a.d; c0 += 256) {
            f32x16 o[2][WB];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < WB; ++i) o[b][i] = f32x16{};
#pragma unroll
            for (int x = 0; x < 2 * NB; ++x) {
                if (16 * x >= kept) break;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int4v hf = *reinterpret_cast<const int4v *>(
                        ht + (((x >> 1) * dp + c0 + 32 * b + r) << 6) + 32 * (x & 1) + 16 * half);
#pragma unroll
                    for (int i = 0; i < WB; ++i) {
                        o[b][i] = mfma(T{}, hf, qf[0][i][x], o[b][i]);
                        o[b][i] = mfma(T{}, hf, qf[1][i][x], o[b][i]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < WB; ++i) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    uint32_t u[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        u[k] = pack2(T{}, o[b][i][2 * k] * scale, o[b][i][2 * k + 1] * scale);
#pragma unroll
                    for (int k = 0; k < 8; k += 4)
                        *reinterpret_cast<uint4 *>(mine_out + r * OUT_ROW + 64 * b + 8 * k +
                                                   16 * half) = join16(u + k);
                }
                __builtin_amdgcn_wave_barrier();         // a wave's LDS accesses keep their order
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int row = 8 * k + (lane >> 3), at = 8 * (lane & 7);
                    const uint4 p =
                        *reinterpret_cast<const uint4 *>(mine_out + row * OUT_ROW + 2 * at);
                    const int64_t word = first + 32 * i + row;
                    if (word < a.v)
                        store_row<T, 8>(dw + word * a.d, c0 + at, a.d,
                                        __builtin_bit_cast(Pack<T, 8>, p));
                }
                __builtin_amdgcn_wave_barrier();
            }
        }
    }
}

// lse and loss of a token a workgroup, from the groups' parts.
__global__ void __launch_bounds__(256)
    k_ce_few_join(const float2 *__restrict__ partial, int64_t groups, Tokens tok,
                  const float *__restrict__ at_target, float *__restrict__ loss_each,
                  float *__restrict__ lse_out, float *__restrict__ loss_kept)
{
    __shared__ float2 lds[4];
    const int slot = blockIdx.x;
    if (slot >= tok.info->kept) return;
    float2 s = make_float2(-__builtin_inff(), 0.0f);
    for (int64_t g = threadIdx.x; g < groups; g += 256)
        s = join_stats(s, partial[slot * groups + g]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        s = join_stats(s, make_float2(__shfl_xor(s.x, d), __shfl_xor(s.y, d)));
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x) return;
    for (int w = 1; w < 4; ++w) s = join_stats(s, lds[w]);
    const float lse = lse_of(s);
    const float loss = tok.target[slot] < 0 ? __builtin_nanf("") : loss_of(s, at_target[slot]);
    const int32_t i = tok.index[slot];
    lse_out[i] = lse;
    if (loss_each) loss_each[i] = loss;
    else loss_kept[slot] = loss;
}

// Columns of w that a lane loads at a time.
template <int NB> constexpr int COLS = NB == 4 ? 4 : 8;

// sums = q w over run blockIdx.y of the words, for slice blockIdx.x of 32 COLS columns, both halves
// of q into one accumulator.  A lane
// loads COLS columns of 8 words; transposed in its registers these are one row (a column of w)
// of COLS fragments, so fragment f holds columns f, COLS + f, ...  A step is 16 words; the waves
// take steps in turns and join their sums in their order through LDS.  The sums leave as the
// accumulators lie: [run][slice][f][token block][accumulator][lane].
template <typename T, int NB>
__global__ void __launch_bounds__(256)
    k_ce_few_dh(Head a, const Info *__restrict__ info, const uint8_t *__restrict__ q,
                int64_t steps, int64_t per, float *__restrict__ sums)
{
    constexpr int N = 32 * NB, C = COLS<NB>, D = C / 2;      // D: dwords of a row
    __shared__ float part[2][4][16][64];
    if (info->kept == 0) return;
    const int lane = threadIdx.x & 63, half = lane >> 5, r = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t col = (int64_t)blockIdx.x * 32 * C + C * r;
    const int64_t begin = (int64_t)blockIdx.y * per;
    const int64_t end = begin + per < steps ? begin + per : steps;
    const bool inside = ((int64_t)blockIdx.x + 1) * 32 * C <= a.d;       // of the whole slice
    typedef Pack<T, C> Row;
    const T *w0 = (const T *)a.w + 8 * half * a.w_stride;
    f32x16 acc[C][NB];
#pragma unroll
    for (int f = 0; f < C; ++f)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[f][j] = f32x16{};
    Row next[8];
    int4v qn[2][NB];
    const int64_t second = steps * 32 * N;       // of q's halves, 16 words a step
    auto load = [&](int64_t s) {
        const T *p = w0 + 16 * s * a.w_stride;
        if (inside && 16 * s + 16 <= a.v) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                next[i] = *reinterpret_cast<const Row *>(p + i * a.w_stride + col);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                next[i] = Row{};
                if (16 * s + 8 * half + i < a.v && col < a.d)
                    next[i] = load_row<T, C>(p + i * a.w_stride, col, a.d);
            }
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const uint8_t *p = q + (((s >> 1) * N + 32 * j + r) << 6) + 32 * (s & 1) + 16 * half;
            qn[0][j] = *reinterpret_cast<const int4v *>(p);
            qn[1][j] = *reinterpret_cast<const int4v *>(p + second);
        }
    };
    int64_t s = begin + wave;
    if (s < end) load(s);
    for (; s < end; s += 4) {
        uint32_t x[8][D];
        int4v qf[2][NB];
#pragma unroll
        for (int i = 0; i < 8; ++i) __builtin_memcpy(x[i], &next[i], sizeof(Row));
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            qf[0][j] = qn[0][j];
            qf[1][j] = qn[1][j];
        }
        if (s + 4 < end) load(s + 4);
#pragma unroll
        for (int f = 0; f < C; ++f) {
            // words 2 k and 2 k + 1 of column f
            const uint32_t pick = f & 1 ? 0x07060302u : 0x05040100u;
            int4v wf;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                wf[k] = (int)__builtin_amdgcn_perm(x[2 * k + 1][f >> 1], x[2 * k][f >> 1], pick);
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                acc[f][j] = mfma(T{}, wf, qf[0][j], acc[f][j]);
                acc[f][j] = mfma(T{}, wf, qf[1][j], acc[f][j]);
            }
        }
    }
    float *out = sums + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * C * NB * 1024;
#pragma unroll
    for (int f = 0; f < C; ++f)
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            auto &p = part[(f * NB + j) & 1];
#pragma unroll
            for (int k = 0; k < 16; ++k) p[wave][k][lane] = acc[f][j][k];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = 4 * wave + i;
                out[(f * NB + j) * 1024 + k * 64 + lane] =
                    ((p[0][k][lane] + p[1][k][lane]) + p[2][k][lane]) + p[3][k][lane];
            }
        }
}

// dh: accumulator blockIdx.y % 16 of token block blockIdx.y / 16 of slice blockIdx.x, the token's
// factor times the sum over the runs: each of the 4 waves every 4th, then joined in their order; zeros in the
// rows of the tokens that do not count.
template <typename T, int NB>
__global__ void __launch_bounds__(256)
    k_ce_few_dh_out(const float *__restrict__ sums, int64_t runs, Tokens tok,
                    const float *__restrict__ dloss, int64_t t, int64_t d, T *__restrict__ dh)
{
    constexpr int C = COLS<NB>;
    __shared__ float part[4][C][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int k = blockIdx.y & 15, j = blockIdx.y >> 4;
    const int slot = 32 * j + (lane & 31);
    const int32_t kept = tok.info->kept;
    if (32 * j >= t) return;
    float s[C];
#pragma unroll
    for (int f = 0; f < C; ++f) s[f] = 0.0f;
    // all lanes read, those past the tokens that count as well: padding, not used
    for (int64_t run = wave; run < runs && 32 * j < kept; run += 4) {
        const float *p = sums + (run * gridDim.x + blockIdx.x) * C * NB * 1024 + j * 1024 + k * 64;
#pragma unroll
        for (int f = 0; f < C; ++f) s[f] += p[f * NB * 1024 + lane];
    }
#pragma unroll
    for (int f = 0; f < C; ++f) part[wave][f][lane] = s[f];
    __syncthreads();
    if (wave || slot >= t) return;
    const float scale = slot < kept ? dh_scale<T>(tok, dloss, slot) : 0.0f;
    Pack<T, C> o;
#pragma unroll
    for (int f = 0; f < C; ++f) {
        const float sum = ((part[0][f][lane] + part[1][f][lane]) + part[2][f][lane]) +
                          part[3][f][lane];
        o.v[f] = slot < kept ? from_f32<T>(sum * scale) : T{};
    }
    const int64_t col = (int64_t)blockIdx.x * 32 * C + C * row_of(k, lane);
    if (col < d) store_row<T, C>(dh + (int64_t)tok.index[slot] * d, col, d, o);
}

FewSizes few_sizes(int64_t t, int64_t d, int64_t v)
{
    FewSizes f{};
    f.blocks = t <= 32 ? 1 : t <= 64 ? 2 : 4;
    // more words share the tokens' rows from L2 where there are more of those
    f.words = f.blocks == 1 ? 32 : 64;
    f.groups = (v + f.words - 1) / f.words;
    const int64_t n = 32 * f.blocks, cols = f.blocks == 4 ? COLS<4> : COLS<1>;
    f.slice_elems = 32 * cols;
    f.slices = (d + f.slice_elems - 1) / f.slice_elems;
    // a workgroup to a compute unit (their accumulators leave room for one), of at least 16 steps
    // of 16 words, four to a wave: shorter runs write and read more sums than they spare
    // (32 tokens, 1024x8192 bf16: backward 37 us, 40 with 4 steps; 512 workgroups 54;
    // 2048x32768: 95 and 105 with 512)
    const int64_t steps = f.groups * f.words / 16;
    int64_t runs = (256 + f.slices - 1) / f.slices;
    runs = runs < (steps + 15) / 16 ? runs : (steps + 15) / 16;
    const int64_t per = (steps + runs - 1) / runs;
    f.runs = (steps + per - 1) / per;
    f.partial_bytes = 8 * n * f.groups;
    f.q_bytes = 2 * 2 * n * f.groups * f.words;
    f.sums_bytes = 4 * n * f.runs * f.slices * f.slice_elems;
    return f;
}

template <typename T>
void few_forward(const Head &a, const int64_t *target, int64_t ignore, const Tokens &tok,
                 const uint8_t *hk, int64_t hk_rows, float2 *partial, float *at_target,
                 float *loss_each, float *lse, float *loss_kept, hipStream_t st)
{
    const FewSizes f = few_sizes(a.t, a.d, a.v);
    const Gather g{target, ignore, loss_each, lse};
    const unsigned n = (unsigned)f.groups;
#define NVFP4T_FEW(NB, WB)                                                                       \
    if (f.blocks == NB)                                                                          \
        k_ce_few<T, NB, WB, false><<<n, 256, 0, st>>>(a, g, tok, (const T *)hk, hk_rows,         \
                                                      partial, at_target, false, nullptr, 0,     \
                                                      nullptr, nullptr);
    NVFP4T_FEW(1, 1) NVFP4T_FEW(2, 2) NVFP4T_FEW(4, 2)
#undef NVFP4T_FEW
    k_ce_few_join<<<(unsigned)a.t, 256, 0, st>>>(partial, f.groups, tok, at_target, loss_each, lse,
                                                 loss_kept);
}

template <typename T>
void few_grad(const Head &a, const Tokens &tok, bool weighted, const uint8_t *hk, int64_t hk_rows,
              const uint8_t *ht, int64_t dp, uint8_t *q, void *dw, hipStream_t st)
{
    const FewSizes f = few_sizes(a.t, a.d, a.v);
    const unsigned n = (unsigned)f.groups;
#define NVFP4T_FEW(NB, WB)                                                                       \
    if (f.blocks == NB)                                                                          \
        k_ce_few<T, NB, WB, true><<<n, 256, 0, st>>>(a, Gather{}, tok, (const T *)hk, hk_rows,   \
                                                     nullptr, nullptr, weighted, ht, dp, q,      \
                                                     (T *)dw);
    NVFP4T_FEW(1, 1) NVFP4T_FEW(2, 2) NVFP4T_FEW(4, 2)
#undef NVFP4T_FEW
}

template <typename T>
void few_dh(const Head &a, const Tokens &tok, const float *dloss, const uint8_t *q, float *sums,
            void *dh, hipStream_t st)
{
    const FewSizes f = few_sizes(a.t, a.d, a.v);
    const int64_t steps = f.groups * f.words / 16, per = (steps + f.runs - 1) / f.runs;
    const dim3 grid((unsigned)f.slices, (unsigned)f.runs);
    const dim3 out((unsigned)f.slices, (unsigned)(16 * f.blocks));
#define NVFP4T_FEW(NB)                                                                          \
    if (f.blocks == NB) {                                                                       \
        k_ce_few_dh<T, NB><<<grid, 256, 0, st>>>(a, tok.info, q, steps, per, sums);             \
        k_ce_few_dh_out<T, NB><<<out, 256, 0, st>>>(sums, f.runs, tok, dloss, a.t, a.d,         \
                                                    (T *)dh);                                   \
    }
    NVFP4T_FEW(1) NVFP4T_FEW(2) NVFP4T_FEW(4)
#undef NVFP4T_FEW
}

#define NVFP4T_FEW(T)                                                                            \
    template void few_forward<T>(const Head &, const int64_t *, int64_t, const Tokens &,         \
                                 const uint8_t *, int64_t, float2 *, float *, float *, float *,  \
                                 float *, hipStream_t);                                          \
    template void few_grad<T>(const Head &, const Tokens &, bool, const uint8_t *, int64_t,      \
                              const uint8_t *, int64_t, uint8_t *, void *, hipStream_t);         \
    template void few_dh<T>(const Head &, const Tokens &, const float *, const uint8_t *,        \
                            float *, void *, hipStream_t);
NVFP4T_FEW(bf16)
NVFP4T_FEW(f16)
#undef NVFP4T_FEW

}  // namespace nvfp4t
