// block_linear.hip -- products of two MXFP4 operands on gfx950's FP4 matrix cores with a linear
// layer's bias, activation, residual or gating in the same kernel.
//
//   z = f A B^T + bias,  y = act(z) + residual;  gated (B holds gate rows, then up rows):
//   z = (gate, up),      y = act(gate) up
// The K loop is the K-tiled product's of nvfp4_gemm.hip: steps of 128 elements straight from memory
// into one of four LDS stages, three steps ahead, on v_mfma_scale_f32_32x32x64_f8f6f4.  A workgroup
// stays on its compute unit and takes one tile after another, and its loads run ahead over the tiles'
// ends: a tile begins with its first three steps in LDS.  They are waited for before the epilogue of
// the tile before, during which nothing is loaded.  The epilogue works on the
// accumulators where they are (B's rows first in the instruction, so that a lane's accumulators are
// columns of one row of A) and needs no LDS; see Block in block_linear.h.  A gated wave's columns are
// half gate, half up of the same features, so both meet in a lane.
//
// Of many calls in a row (the first 20 from an idle card take up to 1.35 times as long): 16384x8192x8192
// bf16 with bias, gelu and z 620-640 us (3.4-3.5 PFLOP/s); its steps alone 480, the rest tile ends and 0.54 GB
// written.  Gated 32768x8192x2048 with silu and z 740-760 us: the steps again 480, 1.6 GB written.  Counters: 1.9
// GHz, matrix cores 41 and 35 % busy, waves waiting 30 %.  With an epilogue through LDS after each tile, in
// workgroups of one tile, these took 694 and 999 us.  2048x2048x8192, a tile of 128 to a compute unit, 28 us
// (2.4 PFLOP/s): loads bound it, 17 us without them and 24 without the products; eight stages or eight
// waves change nothing.
#include "block_linear.h"

#pragma clang fp contract(fast)

namespace nvfp4t {

constexpr int KSTEP = 128, ROW = KSTEP / 2;

#define LDS_PTR(p) ((__attribute__((address_space(3))) void *)(p))

// Chunk c (16 bytes) of row i of a stage: 16 rows at one chunk fall into 16 distinct bank groups.
__device__ __forceinline__ int slot(int i, int c) { return 4 * i + (c ^ ((i >> 2) & 3)); }

// A tile of 32 WI MW x 32 WJ NW of C: MW x NW waves of WI x WJ matrix instructions, NSTAGE stages.
template <int WI_, int WJ_, int MW_, int NW_, int NSTAGE_> struct Tile {
    static constexpr int WI = WI_, WJ = WJ_, MW = MW_, NW = NW_, NSTAGE = NSTAGE_;
    static constexpr int M = 32 * WI * MW, N = 32 * WJ * NW, THREADS = 64 * MW * NW;
    static constexpr int CODES = (M + N) * ROW, STAGE = CODES + 4 * (M + N);
    static constexpr int RA = 4 * M / THREADS, RB = 4 * N / THREADS;   // code loads of a thread
    static constexpr int RS = (M + N + THREADS - 1) / THREADS;         // scale loads
    static constexpr int LOADS = RA + RB + RS;
    static_assert(4 * M % THREADS == 0 && 4 * N % THREADS == 0, "even loads");
    static_assert(M % 64 == 0 && N % 64 == 0, "a wave's scales are one operand's");
};

// Row of B that the tile's B row i stands for.  Gated: in each wave's columns first its gate rows,
// then its up rows.
template <typename TILE, bool GATED>
__device__ __forceinline__ int64_t b_row(int64_t block, int i, int64_t rows)
{
    if constexpr (GATED) {
        constexpr int W = 32 * TILE::WJ, H = W / 2;
        const int64_t n = rows / 2, at = block * (TILE::N / 2) + (i / W) * H + i % H;
        return (at < n ? at : n - 1) + (i % W < H ? 0 : n);
    } else {
        const int64_t at = block * TILE::N + i;
        return at < rows ? at : rows - 1;
    }
}

// Where a thread's loads of a stage come from: the steps of one tile after another.
template <typename TILE, bool TILED, bool GATED> struct Cursor {
    static constexpr int T = TILE::THREADS, CODES = TILE::RA + TILE::RB;
    const uint8_t *src[CODES], *ssrc[TILE::RS];
    uint32_t dst[CODES], sdst[TILE::RS];       // offsets in a stage, the same for a wave's lanes
    int64_t step[2], sstep[2];                 // bytes to the next step, of A and of B

    __device__ __forceinline__ void init(const MxRows &A, const MxRows &B, int w)
    {
#pragma unroll
        for (int k = 0; k < CODES; ++k)
            dst[k] = (uint32_t)(k < TILE::RA ? 16 * (T * k + 64 * w)
                                             : TILE::M * ROW + 16 * (T * (k - TILE::RA) + 64 * w));
#pragma unroll
        for (int k = 0; k < TILE::RS; ++k)
            sdst[k] = (uint32_t)(TILE::CODES + 4 * scale_row(k, w));
        step[0] = TILED ? A.rows * ROW : ROW;
        step[1] = TILED ? B.rows * ROW : ROW;
        sstep[0] = TILED ? A.rows * 4 : 4;
        sstep[1] = TILED ? B.rows * 4 : 4;
    }
    // First of the 64 rows whose scales wave w loads in round k; waves past the last rows repeat
    // others' loads, so that every wave has as many in flight.
    static __device__ __forceinline__ int scale_row(int k, int w)
    {
        return (T * k + 64 * w) % (TILE::M + TILE::N);
    }
    __device__ __forceinline__ void aim(const MxRows &A, const MxRows &B, int64_t K, int64_t bm,
                                        int64_t bn, int w, int lane)
    {
        const auto a_row = [&](int i) {
            const int64_t at = bm * TILE::M + i;
            return at < A.rows ? at : A.rows - 1;
        };
#pragma unroll
        for (int k = 0; k < CODES; ++k) {
            const bool on_b = k >= TILE::RA;
            const int s = T * (on_b ? k - TILE::RA : k) + 64 * w + lane;
            const int i = s >> 2, c = (s & 3) ^ ((i >> 2) & 3);
            const int64_t row = on_b ? b_row<TILE, GATED>(bn, i, B.rows) : a_row(i);
            src[k] = (on_b ? B.codes : A.codes) + row * (TILED ? ROW : (K >> 1)) + 16 * c;
        }
#pragma unroll
        for (int k = 0; k < TILE::RS; ++k) {
            const int t = scale_row(k, w) + lane;
            const bool on_b = scale_row(k, w) >= TILE::M;
            const int64_t row = on_b ? b_row<TILE, GATED>(bn, t - TILE::M, B.rows) : a_row(t);
            ssrc[k] = (on_b ? B.scales : A.scales) + row * (TILED ? 4 : (K >> 5));
        }
    }
    __device__ __forceinline__ void advance(int w)
    {
#pragma unroll
        for (int k = 0; k < CODES; ++k) src[k] += step[k >= TILE::RA];
#pragma unroll
        for (int k = 0; k < TILE::RS; ++k) ssrc[k] += sstep[scale_row(k, w) >= TILE::M];
    }
};

// Wait for all of this wave's loads and stores but the NEWEST (63: for none) and its LDS reads, then for
// every wave.
template <int NEWEST> __device__ __forceinline__ void stage_barrier()
{
    // s_waitcnt fields: vmcnt bits 3:0 and 15:14, expcnt 6:4 (7: no wait), lgkmcnt 11:8
    static_assert(NEWEST < 64, "vmcnt's bits");
    __builtin_amdgcn_sched_barrier(0);
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070 | (NEWEST & 15) | (NEWEST >> 4) << 14);
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

template <typename TILE> struct Frags {
    v8i a[TILE::WI], b[TILE::WJ];
};

template <typename TILE> struct Scales {
    uint32_t a[TILE::WI], b[TILE::WJ];
};

// A lane's offsets in a stage.  Rows 32 apart share the swizzle: 32 rows are 2048 bytes.
struct Offsets {
    uint32_t a[2], b[2], sa, sb;
};

template <typename TILE> __device__ __forceinline__ Offsets offsets(int wm, int wn, int lane)
{
    const int half = lane >> 5, r = lane & 31;
    Offsets o;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        o.a[q] = 16 * slot(wm + r, 2 * q + half);
        o.b[q] = TILE::M * ROW + 16 * slot(wn + r, 2 * q + half);
    }
    o.sa = TILE::CODES + 4 * (wm + r);
    o.sb = TILE::CODES + 4 * (TILE::M + wn + r);
    return o;
}

template <typename TILE>
__device__ __forceinline__ Frags<TILE> read(const uint8_t *stage, const Offsets &o, int q)
{
    Frags<TILE> f;
#pragma unroll
    for (int i = 0; i < TILE::WI; ++i) f.a[i] = mx_fragment(stage + o.a[q] + 32 * ROW * i);
#pragma unroll
    for (int j = 0; j < TILE::WJ; ++j) f.b[j] = mx_fragment(stage + o.b[q] + 32 * ROW * j);
    return f;
}

template <typename TILE>
__device__ __forceinline__ Scales<TILE> read_scales(const uint8_t *stage, const Offsets &o)
{
    Scales<TILE> s;
#pragma unroll
    for (int i = 0; i < TILE::WI; ++i)
        s.a[i] = *reinterpret_cast<const uint32_t *>(stage + o.sa + 128 * i);
#pragma unroll
    for (int j = 0; j < TILE::WJ; ++j)
        s.b[j] = *reinterpret_cast<const uint32_t *>(stage + o.sb + 128 * j);
    return s;
}

// Byte 2 q of a shifted scale word is the lane's 32-block's in sub-step q.
template <typename TILE>
__device__ __forceinline__ Scales<TILE> shifted(const Scales<TILE> &s, int by)
{
    Scales<TILE> r;
#pragma unroll
    for (int i = 0; i < TILE::WI; ++i) r.a[i] = s.a[i] >> by;
#pragma unroll
    for (int j = 0; j < TILE::WJ; ++j) r.b[j] = s.b[j] >> by;
    return r;
}

template <typename TILE, int Q>
__device__ __forceinline__ void multiply(f32x16 (&acc)[TILE::WI][TILE::WJ], const Frags<TILE> &f,
                                         const Scales<TILE> &s)
{
#pragma unroll
    for (int i = 0; i < TILE::WI; ++i)
#pragma unroll
        for (int j = 0; j < TILE::WJ; ++j)
            acc[i][j] = mx_multiply<Q>(f.b[j], s.b[j], f.a[i], s.a[i], acc[i][j]);
    // The products stay here: the compiler would move them to the end of the step, behind the
    // barrier and the loads that they are to cover, as nothing before it needs them.  The statement is
    // empty: no instruction of it reads a result early.
#pragma unroll
    for (int i = 0; i < TILE::WI; ++i)
#pragma unroll
        for (int j = 0; j < TILE::WJ; ++j) __asm__ volatile("" : "+v"(acc[i][j]));
}

// The epilogue of a wave's blocks; (row0, col0) is its first one's corner in y.
template <typename TILE, typename T, bool GATED, bool WHOLE, bool PASSING>
__device__ __forceinline__ void finish_wave(const Epilogue &e, int64_t row0, int64_t col0, int lane,
                                            const f32x16 (&acc)[TILE::WI][TILE::WJ])
{
    constexpr int Z = GATED ? 2 : 1, COLS = TILE::WJ / Z;
#pragma unroll
    for (int i = 0; i < TILE::WI; ++i)
#pragma unroll
        for (int j = 0; j < COLS; ++j) {
            float v[Z][16];
#pragma unroll
            for (int k = 0; k < Z; ++k)
#pragma unroll
                for (int r = 0; r < 16; ++r) v[k][r] = acc[i][j + k * COLS][r];
            finish_block<T, GATED, WHOLE, PASSING>(e, row0 + 32 * i, col0 + 32 * j, lane, v);
            __builtin_amdgcn_sched_barrier(0);
        }
}

// Tiles blockIdx.x, blockIdx.x + gridDim.x, .. of `across` to a row of tiles.  lds: the stages.
//
// Stages hold the steps of all the workgroup's tiles in turn.  A tile begins with its first
// S - 1 steps in LDS: every wave waits for all of its loads before its epilogue, whose stores the next
// tile's first steps then need not wait for (the counter of loads in flight counts stores too, in
// order); from step S - 2 on a step waits for the loads of the one after it.
template <typename TILE, typename T, bool TILED, bool GATED>
__device__ __forceinline__ void linear_tiles(const MxRows &A, const MxRows &B, int64_t K,
                                             const Epilogue &e, int64_t across, int64_t tiles,
                                             uint8_t *lds)
{
    constexpr int S = TILE::NSTAGE, OUT = GATED ? TILE::N / 2 : TILE::N;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int wm = (w / TILE::NW) * 32 * TILE::WI, wn = (w % TILE::NW) * 32 * TILE::WJ;
    const int by = 8 * (lane >> 5);
    const int64_t nk = K / KSTEP;
    const Offsets of = offsets<TILE>(wm, wn, lane);
    Cursor<TILE, TILED, GATED> cur;
    const int64_t stride = gridDim.x;
    int64_t load_tile = blockIdx.x, left = nk;       // the step to load: its tile, steps left in it
    cur.init(A, B, w);
    auto load = [&](int at) {
        uint8_t *to = lds + at * TILE::STAGE;
#pragma unroll
        for (int k = 0; k < cur.CODES; ++k)
            __builtin_amdgcn_global_load_lds(cur.src[k], LDS_PTR(to + cur.dst[k]), 16, 0, 0);
#pragma unroll
        for (int k = 0; k < TILE::RS; ++k)
            __builtin_amdgcn_global_load_lds(cur.ssrc[k], LDS_PTR(to + cur.sdst[k]), 4, 0, 0);
    };
    // on to the next step; past the last tile's end the last step stays, which nobody reads again
    auto advance = [&] {
        if (--left > 0) {
            cur.advance(w);
        } else if (load_tile + stride < tiles) {
            load_tile += stride;
            left = nk;
            cur.aim(A, B, K, load_tile / across, load_tile % across, w, lane);
        } else {
            left = 1;
        }
    };
    if (nk > 0) {
        cur.aim(A, B, K, load_tile / across, load_tile % across, w, lane);
        for (int k = 0; k < S - 1; ++k) {
            load(k);
            advance();
        }
    }
    stage_barrier<0>();
    int at = 0;                                        // the stage of the step that comes next
    for (int64_t t = blockIdx.x; t < tiles; t += stride) {
        f32x16 acc[TILE::WI][TILE::WJ];
#pragma unroll
        for (int i = 0; i < TILE::WI; ++i)
#pragma unroll
            for (int j = 0; j < TILE::WJ; ++j) acc[i][j] = f32x16{};
        const auto next_stage = [&] { at = at == S - 1 ? 0 : at + 1; };
        using None = std::integral_constant<int, 63>;
        using Newest = std::integral_constant<int, (S - 3) * TILE::LOADS>;
        int64_t kt = 0;
        if (nk > 0) {
            Frags<TILE> f0 = read<TILE>(lds + at * TILE::STAGE, of, 0);
            Scales<TILE> sc = shifted<TILE>(read_scales<TILE>(lds + at * TILE::STAGE, of), by);
            auto step = [&](auto newest) {
                const Frags<TILE> f1 = read<TILE>(lds + at * TILE::STAGE, of, 1);
                __builtin_amdgcn_sched_barrier(0);
                multiply<TILE, 0>(acc, f0, sc);
                // the next step has landed; the stage of the step before was last read before this
                stage_barrier<decltype(newest)::value>();
                load(at == 0 ? S - 1 : at - 1);
                next_stage();
                f0 = read<TILE>(lds + at * TILE::STAGE, of, 0);
                const Scales<TILE> raw = read_scales<TILE>(lds + at * TILE::STAGE, of);
                __builtin_amdgcn_sched_barrier(0);
                multiply<TILE, 1>(acc, f1, sc);
                __builtin_amdgcn_sched_barrier(0);
                sc = shifted<TILE>(raw, by);
            };
#pragma clang loop unroll(disable)
            for (; kt < nk && kt < S - 2; ++kt) {
                step(None{});
                advance();
            }
            // most steps: loads of the same tile, whose end no step has to look for (2048x2048x8192
            // 28 us with that in every step, 24 without, as a kernel)
#pragma clang loop unroll(disable)
            for (; kt < nk && left > 1; ++kt) {
                step(Newest{});
                cur.advance(w);
                --left;
            }
#pragma clang loop unroll(disable)
            for (; kt < nk; ++kt) {
                step(Newest{});
                advance();
            }
        }
        stage_barrier<0>();
        const int64_t row0 = (t / across) * TILE::M + wm;
        const int64_t col0 = (t % across) * OUT + wn / (GATED ? 2 : 1);
        constexpr int COLS = 32 * TILE::WJ / (GATED ? 2 : 1);
        if (col0 + COLS > e.n) {
            if (col0 < e.n) finish_wave<TILE, T, GATED, false, false>(e, row0, col0, lane, acc);
            continue;
        }
        if constexpr (sizeof(T) == 2) {
            if (e.passing) {
                finish_wave<TILE, T, GATED, true, true>(e, row0, col0, lane, acc);
                continue;
            }
        }
        finish_wave<TILE, T, GATED, true, false>(e, row0, col0, lane, acc);
    }
}

template <typename TILE, typename T, bool TILED, bool GATED, int PER_CU>
__global__ void __launch_bounds__(TILE::THREADS, PER_CU)
    k_mx_linear(MxRows A, MxRows B, int64_t K, Epilogue e, int64_t across, int64_t tiles)
{
    __shared__ __attribute__((aligned(16))) uint8_t lds[TILE::NSTAGE * TILE::STAGE];
    linear_tiles<TILE, T, TILED, GATED>(A, B, K, e, across, tiles, lds);
}

using Large = Tile<2, 4, 4, 2, 4>;   // 256 x 256, 8 waves, one workgroup a compute unit
using Small = Tile<2, 2, 2, 2, 4>;   // 128 x 128, 4 waves, two workgroups

template <typename TILE, int PER_CU, typename T, bool GATED>
hipError_t launch_tiles(const MxRows &A, const MxRows &B, int64_t K, bool tiled, const Epilogue &e,
                        hipStream_t st)
{
    constexpr int COLS = GATED ? TILE::N / 2 : TILE::N;
    const int64_t across = (e.n + COLS - 1) / COLS, tiles = across * ((e.m + TILE::M - 1) / TILE::M);
    const unsigned grid = (unsigned)(tiles < 256 * PER_CU ? tiles : 256 * PER_CU);
    if (tiled)
        k_mx_linear<TILE, T, true, GATED, PER_CU><<<grid, TILE::THREADS, 0, st>>>(A, B, K, e, across,
                                                                                 tiles);
    else
        k_mx_linear<TILE, T, false, GATED, PER_CU><<<grid, TILE::THREADS, 0, st>>>(A, B, K, e, across,
                                                                                  tiles);
    return hipGetLastError();
}

template <typename T>
hipError_t linear(const MxRows &A, const MxRows &B, int64_t K, bool tiled, bool gated,
                  const Epilogue &e, hipStream_t st)
{
    // Tiles of 256 where they are enough for every compute unit, and from 200 of them where K is long:
    // tiles of 128 then fill their 512 places not quite twice.  K-tiled, 128 and 256: 3840x3840x4096
    // (225 tiles of 256) 50.7 us and 44.3, 3000x5000x8192 (240) 89 and 78; K = 512 20.7 and 24.8, K =
    // 2048 32.7 and 36.4; 4096x3000x8192 (192) 71 and 74.  Row-major: 3840x3840x4096 74.9 us and 53.3,
    // 3000x5000x2176 40.5 and 39.0.
    const int64_t large = ((A.rows + 255) / 256) * ((B.rows + 255) / 256);
    if (large < 256 && (large < 200 || K < (tiled ? 4096 : 2048)))
        return gated ? launch_tiles<Small, 2, T, true>(A, B, K, tiled, e, st)
                     : launch_tiles<Small, 2, T, false>(A, B, K, tiled, e, st);
    return gated ? launch_tiles<Large, 1, T, true>(A, B, K, tiled, e, st)
                 : launch_tiles<Large, 1, T, false>(A, B, K, tiled, e, st);
}

// Whether the kernel for a few rows takes the product: up to 32 rows, or where its workgroups (of 32
// rows of B and up to 128 of A) find a compute unit each, as tiles of 128 then leave most units without
// one.  K-tiled, 8192x2048: 128 rows 10.2 us, tiles 11.8; 256 rows 17.4 and 12.0; 2048x8192: 512 rows
// 17.5 and 25.5, 1024 rows 33 and 26; 1024x1024: 1024 rows 7.9 and 9.0, 2048 rows 13.9 and 9.2.
// Row-major operands, whose rows it reads in pieces, up to 64 rows (2048x8192: 64 rows 19.7 us and
// 26.7, 128 rows 34.5 and 28.3).
bool few(const MxRows &A, const MxRows &B, bool tiled)
{
    if (A.rows <= 32) return true;
    return (tiled || A.rows <= 64) && ((A.rows + 127) / 128) * ((B.rows + 31) / 32) <= 256;
}

// Elements of y and z of 16 bits from which on their stores pass by the caches: as much as the last one, of
// 256 MB, holds.  bf16 back to back (and each after a write of 1 GB): gated 32768x8192x2048 with z 769 us
// (769), kept 843 (808); 32768x8192x2048 347 (337), kept 377 (354); 16384x8192x512 79 (92), kept 89 (98).
// float32 keeps them: 16384x8192x512 171 (168), kept 155 (132); 32768x8192x2048 442 (504), kept 437 (423);
// gated 32768x4096x2048 with z, the one that loses, 531 (643), kept 586 (566); and below 2^27 elements
// 8192x8192x512 88 (86), kept 61 (68).
constexpr int64_t PASSING = (int64_t)1 << 27;

}  // namespace nvfp4t

extern "C" hipError_t nvfp4t_mx_linear(const uint8_t *a_codes, const uint8_t *a_scales,
                                       const uint8_t *b_codes, const uint8_t *b_scales, int64_t M,
                                       int64_t n, int64_t K, int tiled, int rotated_pair, int gated,
                                       int act, int type, int bias_type, const void *bias,
                                       const void *residual, int64_t residual_stride, void *y,
                                       void *z, hipStream_t st)
{
    using namespace nvfp4t;
    const MxRows A{a_codes, a_scales, M}, B{b_codes, b_scales, gated ? 2 * n : n};
    const Epilogue e{rotated_pair ? 0.0078125f : 1.0f, act, bias_type, bias, residual,
                     residual_stride, y, z, M, n,
                     type != F32 && M * (n + (z ? B.rows : 0)) >= PASSING};
    if (few(A, B, tiled)) return linear_few(type, A, B, K, tiled, gated, e, st);
    if (type == F32) return linear<float>(A, B, K, tiled, gated, e, st);
    if (type == BF16) return linear<bf16>(A, B, K, tiled, gated, e, st);
    return linear<f16>(A, B, K, tiled, gated, e, st);
}
