// train_ce.hip -- softmax cross entropy of a linear head over a large vocabulary, with its
// gradient, for gfx950, without ever holding the logits.
//
//   l = h w^T (h [t][d], w [v][d]),  lse = log sum_v exp(l),  loss = lse - l[target]
//   q = share (exp(l - lse) - onehot(target)),  dh = q w,  dw = q^T h
// Only tokens whose target is not the ignored one count.  They are gathered to the front first,
// so the products run over the tokens that count, and whatever stands in the others (NaN
// included) reaches nothing.  The vocabulary is taken in pieces: the forward pass keeps, for
// every token and 128 words, the largest logit and the sum of exponentials against it; the
// backward pass computes each piece's logits again from lse and holds its q in 16 bits.
//
// Up to 128 tokens, whose products are bound by reading the head, take the kernels of
// train_ce_few.hip instead (2048x131072 bf16, with those kernels and with the tiles below: 7 tokens
// forward 109 and 159 us, backward 384 and 869; 64 tokens 149 and 161, 461 and 887; 128 tokens 220
// and 162, 666 and 912: the forward pass alone gains no more above some 64 tokens).
//
// All three products run on one kernel frame (products): C = A B^T with both operands K-tiled,
// [K / 32][rows][32] elements, so that a step of 32 along K of 256 rows is 16 KiB in one piece
// (the logits' head lies in plain rows where those allow it).  A tile of 256 x 256 per workgroup
// of 4 waves, each 128 x 128 (4 x 4 blocks of v_mfma_f32_32x32x16, 256 FP32 accumulators a lane);
// steps of 32 go straight from memory into one of four LDS stages, up to four steps ahead of the
// one the matrix cores work on.  Products with few tiles take 128 x 128 to a workgroup, with
// eight stages.
#include "train_ce.h"

#pragma clang fp contract(fast)

namespace nvfp4t {

constexpr int TILE = 256, STEP = 32;                 // TILE: what the operands' rows are padded to
constexpr int ROW_BYTES = STEP * 2;                  // one row of one step

// A tile of a product whose waves hold B x B blocks of 32 x 32: B is 4, or 2 where tiles of 256
// would leave most compute units without one.
template <int B> struct Tile {
    static constexpr int SIZE = 64 * B, WAVE = 32 * B;
    static constexpr int STAGE_BYTES = 2 * SIZE * ROW_BYTES;     // A and B
    static constexpr int STAGES = B == 4 ? 4 : 8;
    static constexpr int LOADS = 2 * B;              // 16-byte loads of a lane per stage
};

#define NVFP4T_LDS(p) ((__attribute__((address_space(3))) void *)(p))
// Chunk c (16 bytes) of row i of a stage's operand sits in slot 4 i + (c ^ ((i >> 2) & 3)): the
// 16 rows that one LDS cycle of a 16-byte read serves then cover all 64 banks.
__device__ __forceinline__ int slot(int i, int c) { return 4 * i + (c ^ ((i >> 2) & 3)); }

// Waits until at most LEFT loads of this wave are in flight and all its LDS reads are done,
// then for every wave.
template <int LEFT> __device__ __forceinline__ void stage_barrier()
{
    // s_waitcnt fields (gfx9): vmcnt bits 3:0 and 15:14, expcnt 6:4 (7: no wait), lgkmcnt 11:8
    __builtin_amdgcn_sched_barrier(0);
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070 | (LEFT & 15) | (LEFT >> 4) << 14);
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

template <bool V> struct Flag { static constexpr bool value = V; };

template <int B> struct Frags { int4v a[B], b[B]; };

// One tile's work: its first rows in A and B and its steps along K.
struct Item {
    int64_t m0, n0, k0;
    int32_t steps;            // at least 1
    int32_t run;
};

// The items of a product, by index.  Workgroup b takes items b, b + gridDim.x, ...: gridDim.x is
// a multiple of 8, so they stay on the XCD of that workgroup, and the workgroups of one XCD
// take a run of tiles in which 8 tiles of m alternate fastest, so that its 32 compute units
// share 8 tiles of A and 4 of B.  K is cut into runs of `per` steps.
template <int B> struct Items {
    uint32_t mt, nt, count;   // tiles of m and n; mt * nt * runs
    int32_t steps, per;

    __device__ __forceinline__ Item operator[](uint32_t id) const
    {
        const uint32_t tiles = mt * nt, run = id / tiles, in_run = id - run * tiles;
        const uint32_t share = tiles / 8, left = tiles % 8, x = in_run % 8;
        const uint32_t at = x * share + (x < left ? x : left) + in_run / 8;
        const uint32_t group = at / (8 * nt), in = at - group * 8 * nt;
        const uint32_t high = mt - group * 8 < 8 ? mt - group * 8 : 8;
        const int32_t k0 = (int32_t)run * per;
        constexpr int64_t size = Tile<B>::SIZE;
        return {(int64_t)(group * 8 + in % high) * size, (int64_t)(in / high) * size, k0,
                steps - k0 < per ? steps - k0 : per, (int32_t)run};
    }
};

template <int B>
__device__ __forceinline__ Items<B> items_of(int64_t m, int64_t n, int64_t steps, int64_t per,
                                             int64_t runs)
{
    constexpr int64_t size = Tile<B>::SIZE;
    const uint32_t mt = (uint32_t)((m + size - 1) / size), nt = (uint32_t)((n + size - 1) / size);
    return {mt, nt, (uint32_t)(mt * nt * runs), (int32_t)steps, (int32_t)per};
}

// For each of the workgroup's items: the product of its rows of A and B over its steps, given to
// store(item, acc).  Lane l of a wave supplies row l % 32 of each 32-row block, elements
// 8 (l / 32) .. + 7 of each 16; accumulator r of lane l in acc[i][j] is element
// [32 i + 8 (r / 4) + 4 (l / 32) + r % 4][32 j + l % 32] of the wave's 128 x 128.
//
// The fragment reads run half a step ahead of the matrix instructions: a step reads its second
// half's fragments among its first half's instructions, then, after the barrier that makes the
// next stage visible, the next step's first fragments among its second half's.  That barrier
// also ends the last read of the step's own stage, so the loads that follow it refill that
// stage, four steps ahead.  The order of the instructions is fixed: one read or load after
// each matrix instruction, whose 32 cycles hide its issue.  The steps of all items form one
// sequence: while an item's results are stored, the next item's first stages are loading.
// Past the last item the loads repeat the last step into stages nobody reads.
//
// A is K-tiled as well (a_stride 0), or lies in plain rows, a_stride bytes apart: then its last
// tile repeats the last row.
template <typename T, int B, bool ROWS, typename Store>
__device__ __forceinline__ void products(const uint8_t *a_base, int64_t a_rows, int64_t a_stride,
                                         const uint8_t *b_base, int64_t b_rows,
                                         const Items<B> &items, Store store)
{
    constexpr int STAGES = Tile<B>::STAGES, STAGE_BYTES = Tile<B>::STAGE_BYTES;
    constexpr int LOADS = Tile<B>::LOADS, OPERAND = Tile<B>::SIZE * ROW_BYTES;
    __shared__ __attribute__((aligned(16))) uint8_t lds[STAGES * STAGE_BYTES];
    uint32_t id = blockIdx.x;
    if (id >= items.count) return;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int wm = (w >> 1) * Tile<B>::WAVE, wn = (w & 1) * Tile<B>::WAVE;
    // lane's slot in round q is 256 q + 64 w + lane: row 64 q + i0 at the same chunk.  The rest
    // of a load's address is the same in every lane and so stays in scalar registers.
    const int i0 = (64 * w + lane) >> 2, c0 = (lane & 3) ^ ((i0 >> 2) & 3);
    const uint32_t mine = (uint32_t)(i0 * ROW_BYTES + 16 * c0);
    const int64_t step[2] = {ROWS ? ROW_BYTES : a_rows * ROW_BYTES, b_rows * ROW_BYTES};
    uint32_t rows[B];             // offsets of a lane's rows of A in plain rows
    // the step that is loaded next: item, steps left in it, addresses
    uint32_t load_id = id;
    int32_t load_left;
    const uint8_t *src[2];
    auto aim = [&](const Item &it) {
        load_left = it.steps;
        // a tile may begin past the last of the plain rows: they are padded to 256 in the results
        const int64_t m0 = ROWS && it.m0 >= a_rows ? a_rows - 1 : it.m0, last = a_rows - 1 - m0;
        src[0] = a_base + it.k0 * step[0] + m0 * (ROWS ? a_stride : ROW_BYTES);
        if constexpr (ROWS)
#pragma unroll
            for (int q = 0; q < B; ++q) {
                const int64_t row = 64 * q + i0;
                rows[q] = (uint32_t)((row < last ? row : last) * a_stride) + 16 * c0;
            }
        src[1] = b_base + it.k0 * step[1] + it.n0 * ROW_BYTES;
    };
    auto advance = [&] {
        if (load_left > 1) {
            --load_left;
            src[0] += step[0];
            src[1] += step[1];
        } else if (load_id + gridDim.x < items.count) {
            load_id += gridDim.x;
            aim(items[load_id]);
        }
    };
    auto load = [&](uint8_t *st, int op, int q) {
        __builtin_amdgcn_global_load_lds(
            ROWS && op == 0 ? src[op] + rows[q] : src[op] + q * 64 * ROW_BYTES + mine,
            NVFP4T_LDS(st + op * OPERAND + 16 * (256 * q + 64 * w)), 16, 0, 0);
    };
    const int half = lane >> 5, r = lane & 31;
    uint32_t oa[2], ob[2];        // block 0's offsets for each half step; block i is 2048 i on
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        oa[q] = 16 * slot(wm + r, 2 * q + half);
        ob[q] = OPERAND + 16 * slot(wn + r, 2 * q + half);
    }
    // fragment x of a half step: the blocks of B, then of A
    auto read = [&](Frags<B> &f, const uint8_t *st, int q, int x) {
        if (x < B) f.b[x] = *reinterpret_cast<const int4v *>(st + ob[q] + 32 * ROW_BYTES * x);
        else f.a[x - B] = *reinterpret_cast<const int4v *>(st + oa[q] + 32 * ROW_BYTES * (x - B));
    };
    aim(items[id]);
#pragma unroll
    for (int s = 0; s < STAGES; ++s) {
#pragma unroll
        for (int x = 0; x < LOADS; ++x) load(lds + s * STAGE_BYTES, x & 1, x >> 1);
        advance();
    }
    stage_barrier<0>();
    Frags<B> f0, f1;
#pragma unroll
    for (int x = 0; x < 2 * B; ++x) read(f0, lds, 0, x);
    uint32_t at = 0;              // the stage of the present step
    for (; id < items.count; id += gridDim.x) {
        const Item it = items[id];
        f32x16 acc[B][B];
#pragma unroll
        for (int i = 0; i < B; ++i)
#pragma unroll
            for (int j = 0; j < B; ++j) acc[i][j] = f32x16{};
        auto multiply = [&](const Frags<B> &f, int x) {    // instruction x of a half step
            acc[x / B][x % B] = mfma(T{}, f.a[x / B], f.b[x % B], acc[x / B][x % B]);
        };
        for (int k = 0; k < it.steps; ++k) {
            uint8_t *cur = lds + at * STAGE_BYTES;
            at = (at + 1) & (STAGES - 1);
            const uint8_t *nxt = lds + at * STAGE_BYTES;
#pragma unroll
            for (int x = 0; x < B * B; ++x) {
                multiply(f0, x);
                __builtin_amdgcn_sched_barrier(0);
                if (x < 2 * B) {
                    read(f1, cur, 1, x);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            // the next stage landed; this one has been read to its end
            stage_barrier<(STAGES - 2) * LOADS>();
#pragma unroll
            for (int x = 0; x < B * B; ++x) {
                multiply(f1, x);
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (B == 4) {
                    if (x & 1) load(cur, (x >> 1) & 1, x >> 2);
                    else read(f0, nxt, 0, x >> 1);
                } else {
                    read(f0, nxt, 0, x);
                    load(cur, x & 1, x >> 1);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            advance();
        }
        store(it, wm, wn, lane, acc);
    }
    // the loads still in flight write LDS only; they end before the workgroup's LDS is freed
    stage_barrier<0>();
}

// Partial results of the forward pass for one piece: for a wave's words and every token the
// largest logit and the sum of exponentials against it, and the target's logit.  A lane holds
// half of the words of one token in each of acc's columns, so both reductions end with one
// exchange between the wave's halves.
template <typename T, int B, bool ROWS>
__global__ void __launch_bounds__(256, 1)
    k_ce_stats(const uint8_t *__restrict__ w, int64_t w_stride, int64_t words,
               const uint8_t *__restrict__ h, int64_t wp, int64_t tp, int64_t steps, int64_t v0,
               int64_t v, Tokens tok,
               float2 *__restrict__ partial, float *__restrict__ at_target)
{
    constexpr int WAVE = Tile<B>::WAVE;
    const Items<B> items = items_of<B>(wp, tok.info->kept, steps, steps, 1);
    products<T, B, ROWS>(w, ROWS ? words : wp, w_stride, h, tp, items,
                         [&](const Item &it, int wm, int wn, int lane,
                             const f32x16 (&acc)[B][B]) {
        const int64_t first = v0 + it.m0 + wm;          // the wave's first word
        // accumulator r of block i: word first + mine + 32 i + 8 (r / 4) + r % 4
        const int mine = 4 * (lane >> 5);
        const int n = (int)(v - first < WAVE ? v - first : WAVE), left = n - mine;
        auto column = [&](int j, auto edge) {
            const int64_t t = it.n0 + wn + 32 * j + (lane & 31);
            auto logit = [&](int i, int r) {            // none past the vocabulary's end
                const float x = acc[i][j][r];
                if constexpr (decltype(edge)::value)
                    return 32 * i + 8 * (r >> 2) + (r & 3) < left ? x : -__builtin_inff();
                else
                    return x;
            };
            float top = -__builtin_inff();
#pragma unroll
            for (int i = 0; i < B; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) top = fmaxf(top, logit(i, r));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float base = base_of(top);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < B; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    sum += exp_from(logit(i, r), base);
            sum += __shfl_xor(sum, 32);
            if (lane < 32) partial[first / WAVE * tp + t] = make_float2(top, sum);
            const int y = (int)(tok.target[t] - first) - mine;
            if (__any((unsigned)y < (unsigned)WAVE)) {
                float own = 0.0f;
#pragma unroll
                for (int i = 0; i < B; ++i)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        own = y == 32 * i + 8 * (r >> 2) + (r & 3) ? acc[i][j][r] : own;
                // words y / 8 * 8 + 0..3 of this lane's: every other four are the other half's
                if ((unsigned)y < (unsigned)WAVE && (y & 4) == 0) at_target[t] = own;
            }
        };
        if (n == WAVE) {
#pragma unroll
            for (int j = 0; j < B; ++j) {
                column(j, Flag<false>{});
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
#pragma unroll
            for (int j = 0; j < B; ++j) {
                column(j, Flag<true>{});
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    });
}

__device__ __forceinline__ void store16(uint8_t *p, const uint32_t *u)
{
    *reinterpret_cast<uint4 *>(p) = join16(u);
}

// q of one piece, rounded to the operands' 16 bits (matrix instructions take both operands in
// one type; the rounding, at most half a step of each q, is of the size of the outputs' own, and
// over more than 128 tokens not all of one output's: bf16 gradients off by 0.0019 to 0.0024 of their
// norm, 0.0017 with q in two halves, which would take two products in the place of one),
// in both orders the products need: qv [wp / 32][tp][32 words] for dh, whose rows take their
// token's weight afterwards in FP32, and qt [tp / 32][wp][32 tokens] for dw, which adds over the
// tokens and so takes their weights here, before the rounding (WEIGHTED; 1537x1000x50001 f16: 199
// us, 192 with one rounding, weights and all, for both).
template <typename T, int B, bool ROWS, bool WEIGHTED>
__global__ void __launch_bounds__(256, 1)
    k_ce_grad(const uint8_t *__restrict__ w, int64_t w_stride, int64_t words,
              const uint8_t *__restrict__ h, int64_t wp, int64_t tp, int64_t steps, int64_t v0,
              int64_t v, Tokens tok,
              uint8_t *__restrict__ qv, uint8_t *__restrict__ qt)
{
    constexpr int WAVE = Tile<B>::WAVE;
    const int32_t kept = tok.info->kept;
    const Items<B> items = items_of<B>(wp, kept, steps, steps, 1);
    products<T, B, ROWS>(w, ROWS ? words : wp, w_stride, h, tp, items,
                         [&](const Item &it, int wm, int wn, int lane,
                             const f32x16 (&acc)[B][B]) {
        const int64_t first = v0 + it.m0 + wm;
        // a weight that is infinite or NaN leaves no number in the rows that pad the tokens
        const bool last = it.n0 + Tile<B>::SIZE > kept;
        const int mine = 4 * (lane >> 5), odd = lane & 1;
        const int left = (int)(v - first < WAVE ? v - first : WAVE) - mine;
        // an even lane keeps the low halves of its own pair and its neighbour's, an odd lane the
        // high
        const uint32_t pick = odd ? 0x03020706u : 0x05040100u;
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const int64_t t = it.n0 + wn + 32 * j + (lane & 31);
            const float lse = tok.lse[t], share = WEIGHTED ? tok.share[t] : 1.0f;
            const int y = (int)(tok.target[t] - first) - mine;
            const bool hit = __any((unsigned)y < (unsigned)WAVE);
#pragma unroll
            for (int i = 0; i < B; ++i) {
                float q[16];
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    q[r] = exp_from(acc[i][j][r], lse);
                if (hit)
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        q[r] -= y == 32 * i + 8 * (r >> 2) + (r & 3) ? 1.0f : 0.0f;
#pragma unroll
                for (int r = 0; r < 16; ++r) q[r] *= Q_ONE<T>;
                if (32 * i + 32 - mine > left || last)  // past the vocabulary's or tokens' end
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        q[r] = 32 * i + 8 * (r >> 2) + (r & 3) < left && t < kept ? q[r] : 0.0f;
                uint32_t u[8];           // u[k]: words 8 (k / 2) + 2 (k % 2), + 1 (+ mine)
#pragma unroll
                for (int k = 0; k < 8; ++k) u[k] = pack2(T{}, q[2 * k], q[2 * k + 1]);
                const int64_t m = it.m0 + wm + 32 * i;     // first word of the block
                uint32_t s[8];           // the same with the tokens' weights
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    s[k] = WEIGHTED ? pack2(T{}, q[2 * k] * share, q[2 * k + 1] * share) : u[k];
                // qt: neighbouring lanes (tokens) trade halves; each then holds two tokens of
                // one word
                uint8_t *ct = qt + (((it.n0 + wn + 32 * j) >> 5) * wp + m) * ROW_BYTES;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(
                        0, (int)s[k], 0xB1, 0xF, 0xF, true);       // quad_perm [1, 0, 3, 2]
                    const uint32_t x = __builtin_amdgcn_perm(o, s[k], pick);
                    const int word = 8 * (k >> 1) + 2 * (k & 1) + mine + odd;
                    *reinterpret_cast<uint32_t *>(ct + word * ROW_BYTES + 2 * (lane & 30)) = x;
                }
                // qv: the wave's halves trade, so that each lane holds 8 words of its token in
                // a row
                uint8_t *cv = qv + ((m >> 5) * tp + t) * ROW_BYTES;
#pragma unroll
                for (int k = 0; k < 8; k += 4) store16(cv + 8 * k + 16 * (lane >> 5), u + k);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    });
}

// sums[s][t][dp] (+)= the product of w^T (rows: d) and q (rows: tokens) over the s-th of gridDim.y
// runs of the piece's words.
template <typename T, int B, bool ADD>
__global__ void __launch_bounds__(256, 1)
    k_ce_dh(const uint8_t *__restrict__ wt, const uint8_t *__restrict__ qv, int64_t d, int64_t dp,
            int64_t tp, int64_t steps, int64_t per, int64_t runs, const Info *__restrict__ info,
            float *__restrict__ sums)
{
    const Items<B> items = items_of<B>(d, info->kept, steps, per, runs);
    products<T, B, false>(wt, dp, 0, qv, tp, items, [&](const Item &it, int wm, int wn, int lane,
                                           const f32x16 (&acc)[B][B]) {
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const int64_t t = it.n0 + wn + 32 * j + (lane & 31);
            float *row = sums + (it.run * tp + t) * dp + it.m0 + wm + 4 * (lane >> 5);
#pragma unroll
            for (int i = 0; i < B; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float4 *p = reinterpret_cast<float4 *>(row + 32 * i + 8 * k);
                    float4 x = make_float4(acc[i][j][4 * k], acc[i][j][4 * k + 1],
                                           acc[i][j][4 * k + 2], acc[i][j][4 * k + 3]);
                    if constexpr (ADD) {
                        const float4 o = *p;
                        x = make_float4(x.x + o.x, x.y + o.y, x.z + o.z, x.w + o.w);
                    }
                    *p = x;
                    __builtin_amdgcn_sched_barrier(0);
                }
        }
    });
}

// dw rows of the piece: scale times the product of h^T (rows: d) and q^T (rows: words) over
// the tokens that count.
template <typename T, int B>
__global__ void __launch_bounds__(256, 1)
    k_ce_dw(const uint8_t *__restrict__ ht, const uint8_t *__restrict__ qt, int64_t dp, int64_t wp,
            const Info *__restrict__ info, int64_t words, int64_t d, T *__restrict__ dw)
{
    const float scale = info->scale;
    const int32_t kept = info->kept, steps = (kept + STEP - 1) / STEP;
    if (kept == 0) {
        for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < words * d;
             at += (int64_t)gridDim.x * 256)
            dw[at] = T{};
        return;
    }
    const Items<B> items = items_of<B>(d, wp, steps, steps, 1);
    products<T, B, false>(ht, dp, 0, qt, wp, items, [&](const Item &it, int wm, int wn, int lane,
                                           const f32x16 (&acc)[B][B]) {
#pragma unroll
        for (int j = 0; j < B; ++j) {
            const int64_t word = it.n0 + wn + 32 * j + (lane & 31);
#pragma unroll
            for (int i = 0; i < B; ++i) {
                uint32_t u[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    u[k] = pack2(T{}, acc[i][j][2 * k] * scale, acc[i][j][2 * k + 1] * scale);
#pragma unroll
                for (int k = 0; k < 8; k += 4) {
                    const int64_t at = it.m0 + wm + 32 * i + 4 * k + 8 * (lane >> 5);
                    const uint4 x = join16(u + k);
                    if (word < words)
                        store_row<T, 8>(dw + word * d, at, d, __builtin_bit_cast(Pack<T, 8>, x));
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    });
}

// The products' operands from the rows of a matrix: src rows `index[row]` (or `row`), elements
// [0, d), zeros past `count` rows (or *kept) and past d, 64 rows x 64 of `cols` elements at a time.
// rows_out [dk / 32][rp][32]: steps along d; cols_out [rp / 32][dp][32]: steps along the rows.
// Either may be null.  Four lanes write the 64 bytes of a step's row, so a wave's stores are whole
// lines (2048x32768 into both: 76 us, 5.3 TB/s, a large copy's rate; 105 with a row's 64 bytes
// from four waves).
template <typename T>
__global__ void __launch_bounds__(256)
    k_ce_operands(const T *__restrict__ src, int64_t stride, int64_t d,
                  const int32_t *__restrict__ index, const Info *__restrict__ info, int64_t count,
                  int64_t cols, int64_t rp, int64_t dk, int64_t dp,
                  uint8_t *__restrict__ rows_out, uint8_t *__restrict__ cols_out)
{
    __shared__ __attribute__((aligned(16))) uint16_t tile[64][72];
    const int64_t r0 = (int64_t)blockIdx.x * 64;
    if (info) {
        count = info->kept;
        if (r0 >= (count + TILE - 1) / TILE * TILE) return;     // no product reaches these
    }
    const int t = threadIdx.x;
    for (int64_t c0 = (int64_t)blockIdx.y * 64; c0 < cols; c0 += (int64_t)gridDim.y * 64) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int r = (t >> 3) + 32 * k, c = 8 * (t & 7);
            const int64_t row = r0 + r, col = c0 + c;
            Pack<T, 8> p{};
            if (row < count && col < d)
                p = load_row<T, 8>(src + (index ? index[row] : row) * stride, col, d);
            const uint4 x = __builtin_bit_cast(uint4, p);
            if (cols_out) *reinterpret_cast<uint4 *>(&tile[r][c]) = x;
            if (rows_out && col < dk)
                *reinterpret_cast<uint4 *>(rows_out + ((col >> 5) * rp + row) * ROW_BYTES +
                                           2 * (col & 31)) = x;
        }
        if (!cols_out) continue;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int c = t >> 2, r = 8 * ((t & 3) + 4 * k);  // 8 rows of column c, 64 bytes a quad
            uint16_t e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = tile[r + i][c];
            const uint4 x = make_uint4(e[0] | (uint32_t)e[1] << 16, e[2] | (uint32_t)e[3] << 16,
                                       e[4] | (uint32_t)e[5] << 16, e[6] | (uint32_t)e[7] << 16);
            const int64_t row = r0 + r;
            *reinterpret_cast<uint4 *>(cols_out + ((row >> 5) * dp + c0 + c) * ROW_BYTES +
                                       2 * (row & 31)) = x;
        }
        if (c0 + (int64_t)gridDim.y * 64 < cols) __syncthreads();    // the tile is free again
    }
}

// How the losses of the tokens are joined.
enum { SUM = 0, MEAN = 1, NONE = 2 };

// Gathers the tokens that count, in their order (one workgroup).  A target outside the
// vocabulary has no logit: its loss is NaN, and so are the gradients.
//
// Backward: q holds the bare probabilities (-1 and 0 among them are exact) times a power of two
// (Q_EXP), and dloss is left to the products' FP32 results.  Only where dw adds tokens of different
// dloss does it go into q first, relative to the power of two above the largest (share).
__global__ void __launch_bounds__(1024)
    k_ce_tokens(const int64_t *__restrict__ target, int64_t t, int64_t tp, int64_t v,
                int64_t ignore, bool backward, const float *__restrict__ dloss, int reduction,
                int q_exp, const float *__restrict__ lse_in, Tokens tok,
                float *__restrict__ loss_out, float *__restrict__ lse_out)
{
    __shared__ int32_t counts[16];
    __shared__ float tops[16];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int top_exp = 0;
    if (backward && reduction == NONE) {
        float top = 0.0f;
        for (int64_t i = threadIdx.x; i < t; i += 1024) {
            const float x = fabsf(dloss[i]);
            if (target[i] != ignore && x < __builtin_inff()) top = fmaxf(top, x);
        }
        top = wave_max(top);
        if (lane == 0) tops[w] = top;
        __syncthreads();
        for (int k = 0; k < 16; ++k) top = fmaxf(top, tops[k]);
        top_exp = top > 0.0f ? __builtin_amdgcn_frexp_expf(top) : 0;     // top < 2^top_exp
        // a factor of 2^128 is none: shares then reach 2, which bfloat16's q has room for
        if (top_exp > 127 + q_exp) top_exp = 127 + q_exp;
    }
    int32_t kept = 0;
    for (int64_t at = 0; at < t; at += 1024) {
        const int64_t i = at + threadIdx.x;
        const int64_t y = i < t ? target[i] : ignore;
        const bool keep = i < t && y != ignore;
        const uint64_t mask = __ballot(keep);
        if (lane == 0) counts[w] = __popcll(mask);
        __syncthreads();
        int32_t before = kept;
        for (int k = 0; k < 16; ++k) {
            if (k < w) before += counts[k];
            kept += counts[k];
        }
        __syncthreads();
        if (keep) {
            const int32_t slot = before + __popcll(mask & ((1ull << lane) - 1));
            const bool inside = y >= 0 && y < v;
            tok.index[slot] = (int32_t)i;
            tok.target[slot] = inside ? (int32_t)y : -1;
            if (backward) {
                if (reduction == NONE) tok.share[slot] = ldexpf(dloss[i], -top_exp);
                tok.lse[slot] = inside ? lse_in[i] : __builtin_nanf("");
            }
        } else if (i < t) {
            // from slot t - 1 down, for the kernel that writes dh
            const int64_t dropped = i - before - __popcll(mask & ((1ull << lane) - 1));
            if (backward) tok.index[t - 1 - dropped] = (int32_t)i;
            if (lse_out) lse_out[i] = 0.0f;
            if (loss_out) loss_out[i] = 0.0f;
        }
    }
    for (int64_t slot = kept + threadIdx.x; slot < tp; slot += 1024) {
        if (slot >= t) tok.index[slot] = 0;
        tok.target[slot] = -1;
        if (backward) {
            tok.share[slot] = 0.0f;                       // exp(l - inf) is 0, and q too
            tok.lse[slot] = __builtin_inff();
        }
    }
    if (threadIdx.x == 0) {
        float scale = 1.0f;
        if (backward && reduction != NONE)
            scale = reduction == MEAN ? dloss[0] / (float)(kept ? kept : 1) : dloss[0];
        tok.info->kept = kept;
        // where no token counts the gradients are 0, whatever dloss is
        tok.info->scale = kept ? ldexpf(scale, top_exp - q_exp) : 0.0f;
    }
}

// lse and loss of 16 tokens at a time from the `slices` partial results, 64 threads to a token
// that take every 64th slice each, joined in their order (8192 tokens, 1024 slices: 16 us,
// 40 with 64 tokens to a workgroup).
__global__ void __launch_bounds__(1024)
    k_ce_join(const float2 *__restrict__ partial, int64_t slices, int64_t tp, Tokens tok,
              const float *__restrict__ at_target, float *__restrict__ loss_out,
              float *__restrict__ lse_out, float *__restrict__ loss_kept)
{
    __shared__ float2 lds[64][17];
    const int in = threadIdx.x & 15, part = threadIdx.x >> 4;
    const int32_t kept = tok.info->kept;
    for (int64_t first = (int64_t)blockIdx.x * 16; first < kept; first += (int64_t)gridDim.x * 16) {
        float2 all = make_float2(-__builtin_inff(), 0.0f);
#pragma unroll 4
        for (int64_t s = part; s < slices; s += 64)
            all = join_stats(all, partial[s * tp + first + in]);
        lds[part][in] = all;
        __syncthreads();
        // a wave to a token
        const int64_t slot = first + (threadIdx.x >> 6);
        all = lds[threadIdx.x & 63][threadIdx.x >> 6];
        __syncthreads();                                 // lds is free for the next tokens
#pragma unroll
        for (int d = 1; d < 64; d <<= 1)
            all = join_stats(all, make_float2(__shfl_xor(all.x, d), __shfl_xor(all.y, d)));
        if ((threadIdx.x & 63) || slot >= kept) continue;
        const float lse = lse_of(all);
        const float loss =
            tok.target[slot] < 0 ? __builtin_nanf("") : loss_of(all, at_target[slot]);
        const int32_t i = tok.index[slot];
        lse_out[i] = lse;
        if (loss_out) loss_out[i] = loss;
        else loss_kept[slot] = loss;
    }
}

// The sum or the mean of the losses, added in 64 bits.
__global__ void __launch_bounds__(1024)
    k_ce_reduce(const float *__restrict__ loss_kept, const Info *__restrict__ info, int mean,
                float *__restrict__ loss)
{
    __shared__ double lds[16];
    const int32_t kept = info->kept;
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < kept; i += 1024) s += loss_kept[i];
    s = wave_sum(s);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x) return;
    s = 0.0;
    for (int w = 0; w < 16; ++w) s += lds[w];
    loss[0] = (float)(mean ? s / (kept ? kept : 1) : s);
}

// dh of 4 elements a thread at a time: the token's factor (dloss, where not null, is of each token) times the
// sum of the runs' sums, in their order, in the rows the tokens came from; zeros in the rows of
// those that do not count.
template <typename T>
__global__ void __launch_bounds__(256)
    k_ce_dh_out(const float *__restrict__ sums, int runs, int64_t tp, int64_t dp, int64_t d,
                Tokens tok, const float *__restrict__ dloss, int64_t t, T *__restrict__ dh)
{
    const int32_t kept = tok.info->kept;
    for (int64_t at = ((int64_t)blockIdx.y * 256 + threadIdx.x) * 4; at < d;
         at += (int64_t)gridDim.y * 1024)
        for (int64_t slot = blockIdx.x; slot < t; slot += gridDim.x) {
            T *row = dh + (int64_t)tok.index[slot] * d;
            if (slot >= kept) {
                store_row<T, 4>(row, at, d, Pack<T, 4>{});
                continue;
            }
            const float scale = dh_scale<T>(tok, dloss, slot);
            float4 s = *reinterpret_cast<const float4 *>(sums + slot * dp + at);
            for (int k = 1; k < runs; ++k) {
                const float4 x =
                    *reinterpret_cast<const float4 *>(sums + ((int64_t)k * tp + slot) * dp + at);
                s = make_float4(s.x + x.x, s.y + x.y, s.z + x.z, s.w + x.w);
            }
            const Pack<T, 4> o{{from_f32<T>(s.x * scale), from_f32<T>(s.y * scale),
                                from_f32<T>(s.z * scale), from_f32<T>(s.w * scale)}};
            store_row<T, 4>(row, at, d, o);
        }
}

// Words of a piece: what keeps its q (backward) or its operand of w (forward) at 512 MiB, and at
// least one tile.
constexpr int64_t PIECE_BYTES = (int64_t)512 << 20;

int64_t piece(int64_t v, int64_t row_elems)
{
    const int64_t n = PIECE_BYTES / (2 * row_elems) / TILE * TILE;
    const int64_t all = up(v, TILE);
    return n < TILE ? TILE : (n < all ? n : all);
}

// Workgroups of a product: one to a compute unit.
constexpr int64_t UNITS = 256;

// Tiles of 256 up to which a product takes tiles of 128, and steps of 32 words to a run up to
// which dh does.
constexpr int64_t SMALL = 192, DH_STEPS = 64;

// Tiles of a product of m x n.
int64_t tiles(int64_t m, int64_t n, bool small_tiles)
{
    const int64_t size = small_tiles ? Tile<2>::SIZE : Tile<4>::SIZE;
    return ((m + size - 1) / size) * ((n + size - 1) / size);
}

unsigned units(int64_t items) { return (unsigned)(items < UNITS ? up(items, 8) : UNITS); }

// Whether a product of m x n takes tiles of 128: where those of 256 would leave compute units
// without one (1262x2048x844 bf16: forward 66 -> 38 us, backward 141 -> 77; 96 to 192 tiles
// 1024x1024x8192: 43 -> 39 and 123 -> 102).
bool small(int64_t m, int64_t n)
{
    return ((m + TILE - 1) / TILE) * ((n + TILE - 1) / TILE) <= SMALL;
}

// Tiles of dh (blocks to a side of a wave) and the runs that the `steps` of a piece's words are
// cut into, so that every compute unit has a tile.  Large tiles write four times the sums, which
// long runs make up for (2048x2048x32768, runs of 256 steps: backward 747 us, 838 with tiles of
// 128).
struct Cut { int blocks, runs; };

Cut dh_cut(int64_t t, int64_t d, int64_t steps)
{
    for (const int b : {4, 2}) {
        const int64_t size = 64 * b, tiles = ((t + size - 1) / size) * ((d + size - 1) / size);
        const int64_t most = (UNITS + tiles - 1) / tiles;
        const int64_t runs = most < steps ? most : steps;
        if (b == 2 || !small(t, d) || steps / runs > DH_STEPS) return {b, (int)runs};
    }
    return {4, 1};
}

// Hands out 256-byte aligned pieces of the workspace.
struct Carve {
    uint8_t *at;
    size_t used = 0;
    template <typename X> X *take(int64_t bytes)
    {
        X *p = reinterpret_cast<X *>(at + used);
        used += (size_t)up(bytes, 256);
        return p;
    }
};

struct Work {
    Tokens tok;
    int64_t tp, dk, dp, wp;
    int64_t slices;           // parts of the vocabulary in `partial`
    Cut cut;
    uint8_t *hk, *ht, *wk, *wt, *qv, *qt;
    float2 *partial;
    float *at_target, *loss_kept, *sums;
    size_t bytes;
};

Work carve(void *base, bool backward, int64_t t, int64_t d, int64_t v)
{
    Work k{};
    Carve c{(uint8_t *)base};
    if (t > 0 && t <= FEW) {
        const FewSizes f = few_sizes(t, d, v);
        k.tp = up(t, 64);
        k.dk = up(d, STEP);
        k.dp = up(d, TILE);
        k.tok.info = c.take<Info>(sizeof(Info));
        k.tok.index = c.take<int32_t>(4 * k.tp);
        k.tok.target = c.take<int32_t>(4 * k.tp);
        k.hk = c.take<uint8_t>(2 * k.tp * k.dk);
        if (backward) {
            k.tok.lse = c.take<float>(4 * k.tp);
            k.tok.share = c.take<float>(4 * k.tp);
            k.ht = c.take<uint8_t>(2 * k.tp * k.dp);
            k.qv = c.take<uint8_t>(f.q_bytes);
            k.sums = c.take<float>(f.sums_bytes);
        } else {
            k.partial = c.take<float2>(f.partial_bytes);
            k.at_target = c.take<float>(4 * k.tp);
            k.loss_kept = c.take<float>(4 * k.tp);
        }
        k.bytes = c.used;
        return k;
    }
    k.tp = up(t < 1 ? 1 : t, TILE);
    k.dk = up(d, STEP);
    k.dp = up(d, TILE);
    k.wp = piece(v, backward ? k.tp : k.dk);
    k.tok.info = c.take<Info>(sizeof(Info));
    k.tok.index = c.take<int32_t>(4 * k.tp);
    k.tok.target = c.take<int32_t>(4 * k.tp);
    if (backward) {
        k.tok.lse = c.take<float>(4 * k.tp);
        k.tok.share = c.take<float>(4 * k.tp);
    }
    k.hk = c.take<uint8_t>(2 * k.tp * k.dk);
    k.wk = c.take<uint8_t>(2 * k.wp * k.dk);
    if (backward) {
        k.ht = c.take<uint8_t>(2 * k.tp * k.dp);
        k.wt = c.take<uint8_t>(2 * k.wp * k.dp);
        k.qv = c.take<uint8_t>(2 * k.tp * k.wp);
        k.qt = c.take<uint8_t>(2 * k.tp * k.wp);
        k.cut = dh_cut(k.tp, d, k.wp / STEP);
        k.sums = c.take<float>(4 * k.tp * k.dp * k.cut.runs);
    } else {
        k.slices = up(v, TILE) / (small(v, k.tp) ? Tile<2>::WAVE : Tile<4>::WAVE);
        k.partial = c.take<float2>(8 * k.tp * k.slices);
        k.at_target = c.take<float>(4 * k.tp);
        k.loss_kept = c.take<float>(4 * k.tp);
    }
    k.bytes = c.used;
    return k;
}

unsigned groups_y(int64_t want) { return (unsigned)(want < MAX_GROUPS_Y ? want : MAX_GROUPS_Y); }

// The operands of words [v0, v0 + n) of w, n up to the piece's length.
template <typename T>
void word_operands(const T *w, int64_t stride, int64_t d, int64_t n, bool plain, const Work &k,
                   hipStream_t st)
{
    const int64_t rows = up(n, TILE), cols = k.wt ? k.dp : up(k.dk, 64);
    k_ce_operands<T><<<dim3((unsigned)(rows / 64), groups_y(cols / 64)), 256, 0, st>>>(
        w, stride, d, nullptr, nullptr, n, cols, rows, k.dk, k.dp, plain ? nullptr : k.wk, k.wt);
}

template <typename T>
void token_operands(const T *h, int64_t stride, int64_t d, const Work &k, hipStream_t st)
{
    const int64_t cols = k.ht ? k.dp : up(k.dk, 64);
    k_ce_operands<T><<<dim3((unsigned)(k.tp / 64), groups_y(cols / 64)), 256, 0, st>>>(
        h, stride, d, k.tok.index, k.tok.info, 0, cols, k.tp, k.dk, k.dp, k.hk, k.ht);
}

// Whether the logits' products read the head as it lies: rows of whole steps at 16-byte
// boundaries.  Its rows arrive in pieces of 64 bytes, which costs the product little and spares the
// copy (200x4096x65536 bf16 forward: 380 -> 168 us, 8192x2048x131072: 3680 -> 3573).
bool reads_rows(const void *w, int64_t w_stride, int64_t d)
{
    return (uintptr_t)w % 16 == 0 && w_stride % 8 == 0 && d % STEP == 0 &&
           w_stride < (int64_t)1 << 22;          // 256 rows stay within 32-bit offsets
}

// The backward pass copies the head for dh in any case and leaves its second copy out up to this
// many tokens (512x2048x32768: 362 -> 339 us, 2048: 754 -> 750, 4096: 1323 -> 1341;
// 8192x2048x131072: 9.68 -> 9.97 ms, the slower product outweighs it).
constexpr int64_t ROWS_TOKENS = 2048;

// Whether the forward pass of a few tokens lays them out first, which is two launches more: where
// the head is large enough and the tokens' rows, read by every workgroup, are many (128 tokens,
// 2048x131072: 220 us, 267 without; 64 tokens: 149 either way) or not aligned (64 tokens,
// 999x50001: 57 us, 77 without).
template <typename T>
bool few_lays_tokens(const void *h, int64_t h_stride, int64_t t, int64_t d, int64_t v)
{
    const bool odd = (uintptr_t)h % 16 || h_stride % 8;
    return t > (odd ? 32 : 64) && d * v > (int64_t)1 << 24;
}

template <typename T>
void forward(const void *h, int64_t h_stride, const void *w, int64_t w_stride,
             const int64_t *target, int64_t t, int64_t d, int64_t v, int64_t ignore,
             int reduction, float *loss, float *lse, void *workspace, hipStream_t st)
{
    const Work k = carve(workspace, false, t, d, v);
    float *each = reduction == NONE ? loss : nullptr;
    if (t > 0 && t <= FEW) {
        const bool laid = few_lays_tokens<T>(h, h_stride, t, d, v);
        if (laid) {
            k_ce_tokens<<<1, 1024, 0, st>>>(target, t, k.tp, v, ignore, false, nullptr, reduction,
                                            0, nullptr, k.tok, each, lse);
            token_operands((const T *)h, h_stride, d, k, st);
        }
        few_forward<T>({h, h_stride, w, w_stride, t, d, v}, target, ignore, k.tok,
                       laid ? k.hk : nullptr, k.tp, k.partial, k.at_target, each, lse, k.loss_kept,
                       st);
        if (reduction != NONE)
            k_ce_reduce<<<1, 1024, 0, st>>>(k.loss_kept, k.tok.info, reduction == MEAN, loss);
        return;
    }
    k_ce_tokens<<<1, 1024, 0, st>>>(target, t, k.tp, v, ignore, false, nullptr, reduction, 0,
                                    nullptr, k.tok, each, lse);
    if (t > 0) {
        const bool plain = reads_rows(w, w_stride, d);
        token_operands((const T *)h, h_stride, d, k, st);
        for (int64_t v0 = 0; v0 < v; v0 += k.wp) {
            const int64_t n = v - v0 < k.wp ? v - v0 : k.wp, rows = up(n, TILE);
            const bool s = small(v, k.tp);
            if (!plain) word_operands((const T *)w + v0 * w_stride, w_stride, d, n, false, k, st);
            const uint8_t *wp = plain ? (const uint8_t *)w + 2 * v0 * w_stride : k.wk;
            (s ? plain ? k_ce_stats<T, 2, true> : k_ce_stats<T, 2, false>
               : plain ? k_ce_stats<T, 4, true> : k_ce_stats<T, 4, false>)<<<
                units(tiles(rows, k.tp, s)), 256, 0, st>>>(wp, 2 * w_stride, n, k.hk, rows, k.tp,
                                                           k.dk / STEP, v0, v, k.tok, k.partial,
                                                           k.at_target);
        }
        const int64_t joins = k.tp / 16;
        k_ce_join<<<(unsigned)(joins < MAX_GROUPS ? joins : MAX_GROUPS), 1024, 0, st>>>(
            k.partial, k.slices, k.tp, k.tok, k.at_target, each, lse, k.loss_kept);
    }
    if (reduction != NONE)
        k_ce_reduce<<<1, 1024, 0, st>>>(k.loss_kept, k.tok.info, reduction == MEAN, loss);
}

template <typename T, bool WEIGHTED> auto grad_kernel(bool small_tiles, bool plain)
{
    return small_tiles ? plain ? k_ce_grad<T, 2, true, WEIGHTED> : k_ce_grad<T, 2, false, WEIGHTED>
                       : plain ? k_ce_grad<T, 4, true, WEIGHTED> : k_ce_grad<T, 4, false, WEIGHTED>;
}

template <typename T>
void backward(const float *dloss, const void *h, int64_t h_stride, const void *w,
              int64_t w_stride, const int64_t *target, const float *lse, int64_t t, int64_t d,
              int64_t v, int64_t ignore, int reduction, void *dh, void *dw, void *workspace,
              hipStream_t st)
{
    const Work k = carve(workspace, true, t, d, v);
    k_ce_tokens<<<1, 1024, 0, st>>>(target, t, k.tp, v, ignore, true, dloss, reduction, Q_EXP<T>,
                                    lse, k.tok, nullptr, nullptr);
    token_operands((const T *)h, h_stride, d, k, st);
    const bool weighted = reduction == NONE;
    const float *each = weighted ? dloss : nullptr;
    if (t > 0 && t <= FEW) {
        const Head a{h, h_stride, w, w_stride, t, d, v};
        few_grad<T>(a, k.tok, weighted, k.hk, k.tp, k.ht, k.dp, k.qv, dw, st);
        if (dh) few_dh<T>(a, k.tok, each, k.qv, k.sums, dh, st);
        return;
    }
    // runs that have sums: those that the first piece fills (never more than asked for), and so no
    // later piece fills more
    int64_t runs = k.cut.runs;
    const bool few = k.cut.blocks == 2, plain = reads_rows(w, w_stride, d) && t <= ROWS_TOKENS;
    for (int64_t v0 = 0; v0 < v; v0 += k.wp) {
        const int64_t n = v - v0 < k.wp ? v - v0 : k.wp, rows = up(n, TILE);
        word_operands((const T *)w + v0 * w_stride, w_stride, d, n, plain, k, st);
        const bool s = small(rows, k.tp), sw = small(d, rows);
        const uint8_t *wp = plain ? (const uint8_t *)w + 2 * v0 * w_stride : k.wk;
        (weighted ? grad_kernel<T, true>(s, plain) : grad_kernel<T, false>(s, plain))<<<
            units(tiles(rows, k.tp, s)), 256, 0, st>>>(
            wp, 2 * w_stride, n, k.hk, rows, k.tp, k.dk / STEP, v0, v, k.tok, k.qv, k.qt);
        const int64_t steps = rows / STEP, per = (steps + runs - 1) / runs;
        const int64_t used = (steps + per - 1) / per;         // a short last piece fills fewer
        if (dh)
            (few ? v0 ? k_ce_dh<T, 2, true> : k_ce_dh<T, 2, false>
                 : v0 ? k_ce_dh<T, 4, true> : k_ce_dh<T, 4, false>)<<<
                units(tiles(d, k.tp, few) * used), 256, 0, st>>>(
                k.wt, k.qv, d, k.dp, k.tp, steps, per, used, k.tok.info, k.sums);
        if (v0 == 0) runs = used;
        if (dw)
            (sw ? k_ce_dw<T, 2> : k_ce_dw<T, 4>)<<<units(tiles(d, rows, sw)), 256, 0, st>>>(
                k.ht, k.qt, k.dp, rows, k.tok.info, n, d, (T *)dw + v0 * d);
    }
    if (dh && t > 0) {
        const unsigned groups = (unsigned)(t < MAX_GROUPS ? t : MAX_GROUPS);
        k_ce_dh_out<T><<<dim3(groups, groups_y((d + 1023) / 1024)), 256, 0, st>>>(
            k.sums, (int)runs, k.tp, k.dp, d, k.tok, each, t, (T *)dh);
    }
}

}  // namespace nvfp4t

extern "C" size_t nvfp4t_ce_workspace(int backward, int64_t t, int64_t d, int64_t v)
{
    return nvfp4t::carve(nullptr, backward != 0, t, d, v).bytes;
}

extern "C" hipError_t nvfp4t_ce_fwd(int type, const void *h, int64_t h_stride, const void *w,
                                    int64_t w_stride, const int64_t *target, int64_t t, int64_t d,
                                    int64_t v, int64_t ignore, int reduction, float *loss,
                                    float *lse, void *workspace, hipStream_t st)
{
    using namespace nvfp4t;
    if (type == BF16)
        forward<bf16>(h, h_stride, w, w_stride, target, t, d, v, ignore, reduction, loss, lse,
                      workspace, st);
    else
        forward<f16>(h, h_stride, w, w_stride, target, t, d, v, ignore, reduction, loss, lse,
                      workspace, st);
    return hipGetLastError();
}

extern "C" hipError_t nvfp4t_ce_bwd(int type, const float *dloss, const void *h, int64_t h_stride,
                                    const void *w, int64_t w_stride, const int64_t *target,
                                    const float *lse, int64_t t, int64_t d, int64_t v,
                                    int64_t ignore, int reduction, void *dh, void *dw,
                                    void *workspace, hipStream_t st)
{
    using namespace nvfp4t;
    if (type == BF16)
        backward<bf16>(dloss, h, h_stride, w, w_stride, target, lse, t, d, v, ignore, reduction,
                       dh, dw, workspace, st);
    else
        backward<f16>(dloss, h, h_stride, w, w_stride, target, lse, t, d, v, ignore, reduction,
                       dh, dw, workspace, st);
    return hipGetLastError();
}
