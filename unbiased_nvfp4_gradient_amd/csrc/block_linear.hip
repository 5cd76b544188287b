// block_linear.hip -- products of two MXFP4 operands on gfx950's FP4 matrix cores with a linear
// layer's bias, activation, residual or gating in the same kernel.
//
//   z = f A B^T + bias,  y = act(z) + residual;  gated (B holds gate rows, then up rows):
//   z = (gate, up),      y = act(gate) up
// The K loop is the K-tiled product's of nvfp4_gemm.hip: steps of 128 elements straight from memory
// into one of four LDS stages, three steps ahead; matrix instruction v_mfma_scale_f32_32x32x64_f8f6f4,
// lane l supplying row l % 32 (A) or column l % 32 (B), elements 32 (l / 32) .. +31 of 64 and their
// block's scale; accumulator r of lane l is [8 (r / 4) + 4 (l / 32) + r % 4][l % 32].  A gated
// wave's columns are half gate, half up of the same features, so both meet in a lane.  After the loop
// the stages are free: each wave passes its accumulators through them, 32 rows at a time, to lanes of
// eight columns of one row, so that bias, residual, z and y move in 16-byte accesses of whole lines.
#include "block_linear.h"

#pragma clang fp contract(fast)

namespace nvfp4t {

constexpr int KSTEP = 128, ROW = KSTEP / 2, NSTAGE = 4;

#define LDS_PTR(p) ((__attribute__((address_space(3))) void *)(p))

// Chunk c (16 bytes) of row i of a stage: 16 rows at one chunk fall into 16 distinct bank groups.
__device__ __forceinline__ int slot(int i, int c) { return 4 * i + (c ^ ((i >> 2) & 3)); }

// A tile of 32 WI MW x 32 WJ NW of C: MW x NW waves of WI x WJ matrix instructions.
template <int WI_, int WJ_, int MW_, int NW_> struct Tile {
    static constexpr int WI = WI_, WJ = WJ_, MW = MW_, NW = NW_;
    static constexpr int M = 32 * WI * MW, N = 32 * WJ * NW, THREADS = 64 * MW * NW;
    static constexpr int CODES = (M + N) * ROW, STAGE = CODES + 4 * (M + N);
    static constexpr int RA = 4 * M / THREADS, RB = 4 * N / THREADS;   // code loads of a thread
    static constexpr int LOADS = RA + RB + 1;
    static constexpr int OUT_ROW = 32 * WJ + 8;       // floats; rows 4 apart are half the banks apart
    static_assert(4 * M % THREADS == 0 && 4 * N % THREADS == 0 && M + N == THREADS, "even loads");
    static_assert(MW * NW * 32 * OUT_ROW * 4 <= NSTAGE * STAGE, "the epilogue's rows fit the stages");
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

// A thread's loads of a stage (sources of step 0 and what a step adds; offsets in a stage).
template <typename TILE> struct Loads {
    const uint8_t *src[TILE::RA + TILE::RB], *ssrc;
    int64_t step[2], sstep;
    uint32_t dst[TILE::RA + TILE::RB], sdst;
};

template <typename TILE, bool TILED, bool GATED>
__device__ __forceinline__ Loads<TILE> loads(const MxRows &A, const MxRows &B, int64_t K, int64_t bm,
                                             int64_t bn)
{
    constexpr int T = TILE::THREADS;
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    Loads<TILE> l;
    const auto a_row = [&](int i) {
        const int64_t at = bm * TILE::M + i;
        return at < A.rows ? at : A.rows - 1;
    };
#pragma unroll
    for (int k = 0; k < TILE::RA + TILE::RB; ++k) {
        const bool on_b = k >= TILE::RA;
        const int first = T * (on_b ? k - TILE::RA : k) + 64 * w, s = first + lane;
        const int i = s >> 2, c = (s & 3) ^ ((i >> 2) & 3);
        const int64_t row = on_b ? b_row<TILE, GATED>(bn, i, B.rows) : a_row(i);
        l.src[k] = (on_b ? B.codes : A.codes) + row * (TILED ? ROW : (K >> 1)) + 16 * c;
        l.dst[k] = (uint32_t)((on_b ? TILE::M * ROW : 0) + 16 * first);
    }
    l.step[0] = TILED ? A.rows * ROW : ROW;
    l.step[1] = TILED ? B.rows * ROW : ROW;
    // threads of whole waves on one operand's scales
    const int t = 64 * w + lane;
    const bool on_b = 64 * w >= TILE::M;
    const int64_t row = on_b ? b_row<TILE, GATED>(bn, t - TILE::M, B.rows) : a_row(t);
    l.ssrc = (on_b ? B.scales : A.scales) + row * (TILED ? 4 : (K >> 5));
    l.sstep = TILED ? (on_b ? B.rows : A.rows) * 4 : 4;
    l.sdst = (uint32_t)(TILE::CODES + 4 * 64 * w);
    return l;
}

// Wait for this wave's loads of every stage but the newest (`all`: of every stage) and its LDS
// reads, then for every wave.
template <int NEWEST> __device__ __forceinline__ void stage_barrier(bool all)
{
    // s_waitcnt fields: vmcnt bits 3:0, expcnt 6:4 (7: no wait), lgkmcnt 11:8
    static_assert(NEWEST < 16, "vmcnt's low bits");
    __builtin_amdgcn_sched_barrier(0);
    __asm__ volatile("" ::: "memory");
    if (all) __builtin_amdgcn_s_waitcnt(0x0070);
    else __builtin_amdgcn_s_waitcnt(0x0070 | NEWEST);
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

__device__ __forceinline__ v8i fragment(const uint8_t *p)
{
    const v4i v = *reinterpret_cast<const v4i *>(p);
    return v8i{v.x, v.y, v.z, v.w, 0, 0, 0, 0};
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
    for (int i = 0; i < TILE::WI; ++i) f.a[i] = fragment(stage + o.a[q] + 32 * ROW * i);
#pragma unroll
    for (int j = 0; j < TILE::WJ; ++j) f.b[j] = fragment(stage + o.b[q] + 32 * ROW * j);
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
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                f.a[i], f.b[j], acc[i][j], 4, 4, 2 * Q, (int)s.a[i], 2 * Q, (int)s.b[j]);
}

// Tile (bm, bn); lds: the stages.
template <typename TILE, bool TILED, bool GATED>
__device__ __forceinline__ void linear_tile(const MxRows &A, const MxRows &B, int64_t K,
                                            const Epilogue &e, int64_t bm, int64_t bn, uint8_t *lds)
{
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int wm = (w / TILE::NW) * 32 * TILE::WI, wn = (w % TILE::NW) * 32 * TILE::WJ;
    f32x16 acc[TILE::WI][TILE::WJ];
#pragma unroll
    for (int i = 0; i < TILE::WI; ++i)
#pragma unroll
        for (int j = 0; j < TILE::WJ; ++j) acc[i][j] = f32x16{};
    const int64_t nk = K / KSTEP;
    if (nk > 0) {
        const Loads<TILE> ld = loads<TILE, TILED, GATED>(A, B, K, bm, bn);
        const Offsets of = offsets<TILE>(wm, wn, lane);
        const int by = 8 * (lane >> 5);
        // past the last step the loads repeat the last step's data into stages nobody reads
        auto stage = [&](int64_t s) {
            const int64_t kt = s < nk ? s : nk - 1;
            uint8_t *to = lds + (int)(s & (NSTAGE - 1)) * TILE::STAGE;
#pragma unroll
            for (int k = 0; k < TILE::RA + TILE::RB; ++k)
                __builtin_amdgcn_global_load_lds(ld.src[k] + kt * ld.step[k >= TILE::RA],
                                                 LDS_PTR(to + ld.dst[k]), 16, 0, 0);
            __builtin_amdgcn_global_load_lds(ld.ssrc + kt * ld.sstep, LDS_PTR(to + ld.sdst), 4, 0, 0);
        };
        stage(0);
        stage(1);
        stage(2);
        stage_barrier<0>(true);
        Frags<TILE> f0 = read<TILE>(lds, of, 0);
        Scales<TILE> sc = shifted<TILE>(read_scales<TILE>(lds, of), by);
        for (int64_t kt = 0; kt < nk; ++kt) {
            const uint8_t *cur = lds + (int)(kt & (NSTAGE - 1)) * TILE::STAGE;
            const Frags<TILE> f1 = read<TILE>(cur, of, 1);
            __builtin_amdgcn_sched_barrier(0);
            multiply<TILE, 0>(acc, f0, sc);
            // step kt + 1 has landed; the stage of step kt - 1 was last read before this barrier
            stage_barrier<TILE::LOADS>(false);
            stage(kt + NSTAGE - 1);
            const uint8_t *nxt = lds + (int)((kt + 1) & (NSTAGE - 1)) * TILE::STAGE;
            f0 = read<TILE>(nxt, of, 0);
            const Scales<TILE> raw = read_scales<TILE>(nxt, of);
            __builtin_amdgcn_sched_barrier(0);
            multiply<TILE, 1>(acc, f1, sc);
            __builtin_amdgcn_sched_barrier(0);
            sc = shifted<TILE>(raw, by);
        }
        stage_barrier<0>(true);          // the stages are free, loads past the last step included
    }
    // The epilogue: 32 rows of the wave at a time through rows of its own.
    constexpr int COLS = 32 * TILE::WJ / (GATED ? 2 : 1), LANES = COLS / 8, ROWS = 64 / LANES;
    float *rows = reinterpret_cast<float *>(lds) + w * 32 * TILE::OUT_ROW;
    const int64_t col = bn * (GATED ? TILE::N / 2 : TILE::N) + wn / (GATED ? 2 : 1) +
                        8 * (lane % LANES);
    Bias8<GATED> bias;
    bias.load(e, col);
#pragma unroll
    for (int i = 0; i < TILE::WI; ++i) {
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < TILE::WJ; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r)
                rows[(8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)) * TILE::OUT_ROW + 32 * j +
                     (lane & 31)] = acc[i][j][r];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        for (int p = 0; p < 32; p += ROWS) {
            const int r = p + lane / LANES;
            const int64_t row = bm * TILE::M + wm + 32 * i + r;
            if (row >= e.m || col >= e.n) continue;
            const float *from = rows + r * TILE::OUT_ROW + 8 * (lane % LANES);
            float z[GATED ? 2 : 1][8];
#pragma unroll
            for (int k = 0; k < (GATED ? 2 : 1); ++k)
#pragma unroll
                for (int q = 0; q < 8; ++q) z[k][q] = from[k * COLS + q];
            finish8<GATED>(e, row, col, bias, z);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

template <typename TILE, bool TILED, bool GATED, int PER_CU>
__global__ void __launch_bounds__(TILE::THREADS, PER_CU)
    k_mx_linear(MxRows A, MxRows B, int64_t K, Epilogue e)
{
    __shared__ __attribute__((aligned(16))) uint8_t lds[NSTAGE * TILE::STAGE];
    constexpr int COLS = GATED ? TILE::N / 2 : TILE::N;
    const int64_t across = (e.n + COLS - 1) / COLS, down = (e.m + TILE::M - 1) / TILE::M;
    for (int64_t t = blockIdx.x; t < across * down; t += gridDim.x) {
        if (t != blockIdx.x) __syncthreads();          // the tile before has read its rows
        linear_tile<TILE, TILED, GATED>(A, B, K, e, t / across, t % across, lds);
    }
}

using Large = Tile<2, 4, 4, 2>;      // 256 x 256, 8 waves, one workgroup a compute unit
using Small = Tile<2, 2, 2, 2>;      // 128 x 128, 4 waves, two workgroups

template <typename TILE, int PER_CU, bool GATED>
hipError_t launch_tiles(const MxRows &A, const MxRows &B, int64_t K, bool tiled, const Epilogue &e,
                        hipStream_t st)
{
    const int64_t cols = GATED ? TILE::N / 2 : TILE::N;
    const int64_t tiles = ((e.n + cols - 1) / cols) * ((e.m + TILE::M - 1) / TILE::M);
    const unsigned grid = (unsigned)(tiles < MAX_GROUPS ? tiles : MAX_GROUPS);
    if (tiled) k_mx_linear<TILE, true, GATED, PER_CU><<<grid, TILE::THREADS, 0, st>>>(A, B, K, e);
    else k_mx_linear<TILE, false, GATED, PER_CU><<<grid, TILE::THREADS, 0, st>>>(A, B, K, e);
    return hipGetLastError();
}

}  // namespace nvfp4t

extern "C" size_t nvfp4t_mx_linear_workspace(int gated, int64_t M, int64_t n, int64_t K)
{
    return 0;
}

extern "C" hipError_t nvfp4t_mx_linear(const uint8_t *a_codes, const uint8_t *a_scales,
                                       const uint8_t *b_codes, const uint8_t *b_scales, int64_t M,
                                       int64_t n, int64_t K, int tiled, int rotated_pair, int gated,
                                       int act, int type, int bias_type, const void *bias,
                                       const void *residual, int64_t residual_stride, void *y,
                                       void *z, void *workspace, hipStream_t st)
{
    using namespace nvfp4t;
    const MxRows A{a_codes, a_scales, M}, B{b_codes, b_scales, gated ? 2 * n : n};
    const Epilogue e{rotated_pair ? 0.0078125f : 1.0f, act, type, bias_type, bias, residual,
                     residual_stride, y, z, M, n};
    // tiles of 256 where they are enough for every compute unit
    const int64_t large = ((M + 255) / 256) * ((B.rows + 255) / 256);
    if (large < 256) {
        if (gated) return launch_tiles<Small, 2, true>(A, B, K, tiled, e, st);
        return launch_tiles<Small, 2, false>(A, B, K, tiled, e, st);
    }
    if (gated) return launch_tiles<Large, 1, true>(A, B, K, tiled, e, st);
    return launch_tiles<Large, 1, false>(A, B, K, tiled, e, st);
}
