// The gated feed-forward product and its gradient in FLOAT, on the FMA pipes,
// which keep float32 products exact to one rounding (the tensor cores round
// their operands).
//
// Operations at two a paired FMA bound them.  A block takes 64 rows x 128
// columns: 64 threads with 8 x 16 accumulators each, or 128 with 8 x 8 where
// there are few tiles.  64 paired FMAs (128 cycles) then take six 16-byte reads
// of shared memory and the copies that make pairs of A's elements.  Slices of K,
// 16 deep, come through asynchronous copies two ahead; an operand B stored with
// its K contiguous is transposed through registers.  Measured at [1024, 1024] x
// [1024, 2816]: 221 us, 54 TFLOP/s of the pipes' 79.5; [2048, 2048] x [2048, 5632]:
// 1566 us, 60 TFLOP/s.  Two warps on a scheduler (the accumulators' registers)
// leave the rest to dependent issues, counters say.  What the columns and the K are:
//
//   FWD  64 columns of Wg next to the same 64 of Wu: a thread holds g and u of the
//        same outputs and forms act(g) u from registers
//   DX   one accumulation through dg and Wg, then through du and Wu
//   DW   x' dg and x' du as two outputs of one launch, x (or dg, du) read with its
//        rows along K as it is
//
// Blocks are as many as reside, and each takes the next piece of work when it is
// done with one: first whole tiles, as many as there are full rounds, then the
// other tiles cut along K into pieces, so that no SM idles and blocks that an SM's
// schedulers favoured take more ([1024, 1024] x [1024, 2816]: 608 tiles whole, 96
// in pieces; equal shares given out beforehand: 237 us).  A tile's pieces meet in
// the plan's memory, and the block that brings the last one adds them in the order
// of K: who computed which does not show.
#include "gated_internal.h"
#include "plan_state.h"

namespace olc {
namespace gated {
namespace f32 {

constexpr int TM = 64, TN = 64, KS = 16;          // rows, half of the columns, depth of a slice
constexpr int STAGES = 3;
constexpr int AP = KS + 4;                        // floats between rows of A's tile: four rows in four bank groups
constexpr int A_FLOATS = TM * AP, B_FLOATS = KS * 2 * TN;
constexpr int TILE_VECS = TM * 2 * TN / 4;        // 16-byte vectors of a tile's sums
constexpr int SMEM_BYTES = STAGES * (A_FLOATS + B_FLOATS) * 4;

// blocks that reside (registers)
constexpr int per_sm(int threads) { return threads == 64 ? 4 : 3; }

struct Params {
    const float *a[2], *b[2]; // FWD: a[0] = X, b = Wg, Wu; DX: dg, du and Wg, Wu; DW: the two outputs' operands
    int64_t lda, ldb;
    float* y[3];              // FWD: h, g, u (null: not kept); DX: dX; DW: dWg, dWu
    int64_t M, N, K;          // rows and columns of an output, K of one operand pair
    int64_t tiles_m, tiles_item, tiles;
    int64_t whole;            // tiles taken whole
    int64_t works;            // and the pieces of the others
    int pieces;               // of a tile
    int source_slices;        // slices of one operand pair
    int slices;               // of a tile (DX: both pairs')
    int act;
    float4* sums;             // [pieces of all cut tiles][TILE_VECS]
    unsigned int* taken;      // pieces of work taken beyond the first of each block; zero between launches, like
    unsigned int* left;       // blocks that have left
    unsigned int* arrived;    // [cut tiles] pieces that are there
};

// the first four of n elements at `from`, zeros past the n-th; VEC: whole
// 16-byte vectors
template <bool VEC>
__device__ __forceinline__ float4 four(const float* from, int n) {
    if constexpr (VEC) return n > 0 ? __ldg(reinterpret_cast<const float4*>(from)) : make_float4(0.f, 0.f, 0.f, 0.f);
    float4 v;
    v.x = n > 0 ? __ldg(from) : 0.f;
    v.y = n > 1 ? __ldg(from + 1) : 0.f;
    v.z = n > 2 ? __ldg(from + 2) : 0.f;
    v.w = n > 3 ? __ldg(from + 3) : 0.f;
    return v;
}

template <bool VEC>
__device__ __forceinline__ void put_four(float* row, int64_t i, int64_t n, const float (&v)[4]) {
    if constexpr (VEC) {
        *reinterpret_cast<float4*>(row + i) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (i + q < n) row[i + q] = v[q];
    }
}

// `bytes` (0 to 4 or 16) of a SIZE-byte copy, the rest zeros
template <int SIZE>
__device__ __forceinline__ void copy_async(float* to, const float* from, int bytes) {
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(to));
    if constexpr (SIZE == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(from), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(at), "l"(from), "r"(bytes) : "memory");
}
// the first four of n elements at `from` into four floats of shared memory,
// zeros past the n-th (`any`: an address that can be formed when none is read)
template <bool VEC>
__device__ __forceinline__ void copy_four(float* to, const float* from, const float* any, int n) {
    if constexpr (VEC) {
        copy_async<16>(to, n > 0 ? from : any, n > 0 ? 16 : 0);
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) copy_async<4>(to + q, q < n ? from + q : any, q < n ? 4 : 0);
    }
}

// A_T: A is stored [K, M]; B_T: B is stored [N, K].  THREADS: 64 with 8 x 16
// accumulators each, or 128 with 8 x 8.
template <int MODE, bool VEC, bool A_T, bool B_T, int THREADS>
__global__ void __launch_bounds__(THREADS, per_sm(THREADS)) kernel(const Params p) {
    extern __shared__ __align__(16) float smem[];     // stages of A [64 rows][k] (A_T: [k][64 rows]), B [k][2 x 64]
    __shared__ int last;
    __shared__ unsigned int turn;
    const int t = threadIdx.x;
    // A warp's lanes over its rows and columns.  SPREAD: lanes two apart read the
    // same columns and neighbours the same rows, which lets a 16-byte read of
    // shared memory serve half a warp at once (two wavefronts a read instead of
    // four); otherwise columns along the lanes, which stores faster.  us of
    // [1024, 1024] x [1024, 2816], SPREAD and not: forward 225 and 221, with
    // weights stored [F, D] 266 and 278, gradient 492 and 544.
    constexpr bool SPREAD = MODE != FWD || B_T;
    constexpr int CG = 128 / THREADS;         // groups of 32 columns a thread has of each half
    const int tx = SPREAD ? (t & 1) | ((t >> 1) & 6) | (CG == 1 ? (t >> 2) & 8 : 0) : t % (16 / CG);
    const int ty = SPREAD ? ((t >> 1) & 1) | ((t >> 3) & 2) | (t / (THREADS / 2)) * 4 : t / (16 / CG);
    constexpr int COLS = MODE == FWD ? TN : 2 * TN;
    int m0 = 0, n0 = 0, item = 0;
    const int M = (int)p.M, N = (int)p.N, K = (int)p.K;      // below 2^31
    float* const as = smem;
    float* const bs = smem + STAGES * A_FLOATS;

    // A slice's addresses advance by additions.  An operand with K contiguous:
    // this thread takes rows t / 4 + AR q of A at K elements 4 (t % 4), one row of
    // (each half of) B at all sixteen; one with its rows along K: K elements t / 16
    // + KR q at elements 4 (t % 16).
    constexpr int Q = 256 / THREADS, AR = THREADS / 4, KR = THREADS / 16;
    const float *pa = nullptr, *pb[2] = {nullptr, nullptr};
    int ka = 0, kb = 0;              // their K elements
    unsigned rows_in = 0;
    int left_a = 0, left_b[2] = {0, 0};       // elements from this thread's to the row's end
    const int64_t da = (A_T ? KR : AR) * p.lda, db = KR * p.ldb;
    float* const a_to = A_T ? as + (t >> 4) * TM + (t & 15) * 4 : as + (t >> 2) * AP + (t & 3) * 4;
    float* const b_to = B_T ? bs + t : bs + (t >> 4) * 2 * TN + (t & 15) * 4;
    // from slice s0 of operand pair `source`
    auto begin = [&](int source, int s0) {
        const int k0 = s0 * KS;
        const float* A = MODE == FWD ? p.a[0] : p.a[source];
        if constexpr (A_T) {
            const int row = m0 + (t & 15) * 4;
            left_a = M - row;
            ka = k0 + (t >> 4);
            pa = A + (int64_t)ka * p.lda + row;
        } else {
            const int row = m0 + (t >> 2);
            rows_in = 0;
#pragma unroll
            for (int q = 0; q < Q; ++q) rows_in |= (unsigned)(row + AR * q < M) << q;
            ka = k0 + (t & 3) * 4;
            pa = A + (int64_t)row * p.lda + ka;
        }
        kb = B_T ? k0 : k0 + (t >> 4);
#pragma unroll
        for (int q = 0; q < (B_T ? CG : 2); ++q) {
            const int h = B_T ? (t + q * THREADS) / TN : q;
            const float* B = MODE == FWD ? p.b[h] : p.b[source];
            const int col = n0 + (MODE == FWD ? 0 : h * TN) + (B_T ? t % TN : (t & 15) * 4);
            left_b[q] = N - col;
            pb[q] = B_T ? B + (int64_t)col * p.ldb + kb : B + (int64_t)kb * p.ldb + col;
        }
    };
    auto fetch = [&](int stage) {
        float* a = a_to + stage * A_FLOATS;
        float* b = b_to + stage * B_FLOATS;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            if constexpr (A_T) copy_four<VEC>(a + KR * q * TM, pa + q * da, p.a[0], ka + KR * q < K ? left_a : 0);
            else copy_four<VEC>(a + AR * q * AP, pa + q * da, p.a[0], (rows_in >> q) & 1u ? K - ka : 0);
        }
        pa += A_T ? Q * da : KS;
        ka += KS;
        if constexpr (!B_T) {
#pragma unroll
            for (int q = 0; q < Q; ++q)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    copy_four<VEC>(b + KR * q * 2 * TN + h * TN, pb[h] + q * db, p.b[0],
                                   kb + KR * q < K ? left_b[MODE == FWD ? 0 : h] : 0);
            pb[0] += Q * db;
            pb[1] += Q * db;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if constexpr (B_T) {
#pragma unroll
            for (int h = 0; h < CG; ++h) {
                float4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = four<VEC>(pb[h] + 4 * i, left_b[MODE == FWD ? 0 : h] > 0 ? K - kb - 4 * i : 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float* to = b + 4 * i * 2 * TN + h * TN;
                    to[0] = v[i].x;
                    to[2 * TN] = v[i].y;
                    to[4 * TN] = v[i].z;
                    to[6 * TN] = v[i].w;
                }
            }
            pb[0] += KS;
            if constexpr (CG == 2) pb[1] += KS;
        }
        kb += KS;
    };

    // rows ty + 8 i (A_T: 8 ty + i); columns 32 c + 4 tx + (0..3) of the first half (j < 2 CG), then of the second
    constexpr int J = 4 * CG;
    F2 acc[8][J];

    // acc += the tile's products over slices [s0, s0 + n) of one operand pair
    auto multiply_pair = [&](int source, int s0, int n) {
        __syncthreads();             // all are done with what came before
        begin(source, s0);
        for (int i = 0; i < STAGES - 1; ++i) {
            if (i < n) fetch(i);
            else asm volatile("cp.async.commit_group;" ::: "memory");
        }
        int stage = 0;
        for (int i = 0; i < n; ++i) {
            asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
            __syncthreads();             // this slice is there for all, and all are done with the one before it
            const int next = i + STAGES - 1;
            if (next < n) fetch(stage == 0 ? STAGES - 1 : stage - 1);
            else asm volatile("cp.async.commit_group;" ::: "memory");
            const float* a = as + stage * A_FLOATS + (A_T ? ty * 8 : ty * AP);
            const float* b = bs + stage * B_FLOATS + tx * 4;
            if (++stage == STAGES) stage = 0;
#pragma unroll
            for (int k4 = 0; k4 < KS; k4 += 4) {
                float4 x[8];     // row r at K elements k4 .. k4 + 3 (A_T: rows 4 (i % 2) .. at element k4 + i / 2)
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    x[r] = *reinterpret_cast<const float4*>(A_T ? a + (k4 + (r >> 1)) * TM + (r & 1) * 4 : a + r * 8 * AP + k4);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    F2 w[J];
#pragma unroll
                    for (int h = 0; h < J / 2; ++h) {
                        const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(b + (k4 + k) * 2 * TN + h * (32 * 2 / CG));
                        w[2 * h] = v.x;
                        w[2 * h + 1] = v.y;
                    }
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const float4& v = A_T ? x[2 * k + (r >> 2)] : x[r];
                        const int at = A_T ? r & 3 : k;
                        const float e = at == 0 ? v.x : (at == 1 ? v.y : (at == 2 ? v.z : v.w));
                        const F2 e2 = pack_f2(e, e);
#pragma unroll
                        for (int j = 0; j < J; ++j) fma_f2(acc[r][j], e2, w[j]);
                    }
                }
            }
        }
    };
    // acc = the tile's products over slices [s0, s0 + n)
    auto multiply = [&](int s0, int n) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < J; ++j) acc[i][j] = 0;
        if constexpr (MODE == DX) {
            const int s1 = s0 + n, half = p.source_slices;
#pragma unroll 1
            for (int source = 0; source < 2; ++source) {
                const int from = max(s0, source * half), to = min(s1, (source + 1) * half);
                if (from < to) multiply_pair(source, from - source * half, to - from);
            }
        } else {
            multiply_pair(MODE == DW ? item : 0, s0, n);
        }
    };
    auto finish = [&] {
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const int64_t row = m0 + (A_T ? ty * 8 + r : ty + 8 * r);
            if (row >= M) continue;
#pragma unroll
            for (int c = 0; c < CG; ++c) {
                const int64_t col = n0 + 32 * c + tx * 4;
                float g[4], u[4], h[4];
                unpack_f2(acc[r][2 * c], g[0], g[1]);
                unpack_f2(acc[r][2 * c + 1], g[2], g[3]);
                unpack_f2(acc[r][J / 2 + 2 * c], u[0], u[1]);
                unpack_f2(acc[r][J / 2 + 2 * c + 1], u[2], u[3]);
                if constexpr (MODE == FWD) {
                    if (col >= p.N) continue;
                    by_activation(p.act, [&](auto act) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) h[j] = gate_value<true, act.value>(g[j]) * u[j];
                    });
                    put_four<VEC>(p.y[0] + row * p.N, col, p.N, h);
                    if (p.y[1]) put_four<VEC>(p.y[1] + row * p.N, col, p.N, g);
                    if (p.y[2]) put_four<VEC>(p.y[2] + row * p.N, col, p.N, u);
                } else {
                    float* y = p.y[MODE == DW ? item : 0] + row * p.N;
                    if (col < p.N) put_four<VEC>(y, col, p.N, g);
                    if (col + TN < p.N) put_four<VEC>(y, col + TN, p.N, u);
                }
            }
        }
    };
    auto tile_at = [&](int tile) {
        item = MODE == DW ? tile / (int)p.tiles_item : 0;
        const int in = tile - item * (int)p.tiles_item;
        // rows fastest: the row tiles of a column read its operand B from L2
        m0 = in % (int)p.tiles_m * TM;
        n0 = in / (int)p.tiles_m * COLS;
    };

    const int whole = (int)p.whole, pieces = p.pieces;
    for (int work = blockIdx.x; work < (int)p.works;) {
        if (work < whole) {
            tile_at(work);
            multiply(0, p.slices);
        } else {
            const int cut = (work - whole) / pieces, piece = (work - whole) - cut * pieces;
            const int s0 = (int)((int64_t)piece * p.slices / pieces), s1 = (int)((int64_t)(piece + 1) * p.slices / pieces);
            tile_at(whole + cut);
            multiply(s0, s1 - s0);
        }
        bool complete = work < whole || pieces == 1;
        if (!complete) {
            const int cut = (work - whole) / pieces, piece = (work - whole) - cut * pieces;
            float4* const sums = p.sums + (int64_t)cut * pieces * TILE_VECS + t;
#pragma unroll
            for (int r = 0; r < 8; ++r)
#pragma unroll
                for (int j = 0; j < J; j += 2) {
                    float4 v;
                    unpack_f2(acc[r][j], v.x, v.y);
                    unpack_f2(acc[r][j + 1], v.z, v.w);
                    __stcg(sums + (int64_t)piece * TILE_VECS + (r * (J / 2) + j / 2) * THREADS, v);
                }
            __threadfence();
            __syncthreads();
            if (t == 0) last = atomicAdd(p.arrived + cut, 1u) == (unsigned int)(pieces - 1);
            __syncthreads();
            complete = last;
            if (complete) {
                __threadfence();
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int j = 0; j < J; ++j) acc[i][j] = 0;
                for (int q = 0; q < pieces; ++q) {
#pragma unroll
                    for (int r = 0; r < 8; ++r)
#pragma unroll
                        for (int j = 0; j < J; j += 2) {
                            const float4 v = __ldcg(sums + (int64_t)q * TILE_VECS + (r * (J / 2) + j / 2) * THREADS);
                            acc[r][j] = add2(acc[r][j], pack_f2(v.x, v.y));
                            acc[r][j + 1] = add2(acc[r][j + 1], pack_f2(v.z, v.w));
                        }
                }
                if (t == 0) p.arrived[cut] = 0u;
            }
        }
        if (complete) finish();
        if (t == 0) turn = atomicAdd(p.taken, 1u);
        __syncthreads();
        work = (int)(gridDim.x + turn);
        __syncthreads();             // read by all before it is written again
    }
    // the last block to leave finds every turn taken
    if (t == 0) {
        __threadfence();
        if (atomicAdd(p.left, 1u) == gridDim.x - 1) {
            *p.taken = 0u;
            *p.left = 0u;
        }
    }
}

}  // namespace f32

namespace {

// How a product is cut; rows and columns of one output, K of one operand pair.
struct FloatShape {
    int threads;
    int64_t tiles_m, tiles_item, tiles, grid, whole, works;
    int pieces;
    int source_slices, slices;
};
FloatShape float_shape(int mode, int64_t M, int64_t N, int64_t K, int sm_count) {
    FloatShape f;
    f.tiles_m = ceil_div(M, f32::TM);
    f.tiles_item = f.tiles_m * ceil_div(N, mode == FWD ? f32::TN : 2 * f32::TN);
    f.tiles = f.tiles_item * (mode == DW ? 2 : 1);
    f.source_slices = (int)ceil_div(K, f32::KS);
    f.slices = f.source_slices * (mode == DX ? 2 : 1);
    // less than half a round of the blocks that multiply fastest: twice the warps
    // on a tile, 8 x 8 accumulators a thread ([300, 1000] x [1000, 2730]: 98 us,
    // with 64 threads 118; [16, 1024] x [1024, 2816]: 30 and 35; the gradient of
    // [2048, 2048] x [2048, 5632], 512 tiles: 3630 and 3510)
    f.threads = 2 * f.tiles < (int64_t)f32::per_sm(64) * sm_count ? 128 : 64;
    const int64_t resident = (int64_t)f32::per_sm(f.threads) * sm_count;
    f.whole = f.tiles / resident * resident;
    const int64_t cut = f.tiles - f.whole;
    // Pieces of a tile, each at least four slices, at most 16: as many as cost
    // least, which is rounds x a piece's slices and some three more for its fill
    // and its sums ([1024, 1024] x [1024, 2816], 96 tiles cut: 6 pieces 221 us, 12
    // 226, 16 223; [2048, 2048] x [2048, 5632], 384 tiles: 3 pieces 1566, whole
    // 1643).
    const int64_t most = min64(16, f.slices / 4);
    f.pieces = 1;
    auto cost = [&](int64_t n) { return ceil_div(cut * n, resident) * (ceil_div(f.slices, n) + 3); };
    for (int n = 2; n <= (int)most; ++n)
        if (cost(n) < cost(f.pieces)) f.pieces = n;
    f.works = f.whole + cut * f.pieces;
    f.grid = min64(resident, f.works);
    return f;
}

template <int MODE, bool A_T, bool B_T>
cudaError_t launch_float_as(const f32::Params& p, bool vec, const FloatShape& f, cudaStream_t s) {
    auto* kernel = f.threads == 64
        ? (vec ? f32::kernel<MODE, true, A_T, B_T, 64> : f32::kernel<MODE, false, A_T, B_T, 64>)
        : (vec ? f32::kernel<MODE, true, A_T, B_T, 128> : f32::kernel<MODE, false, A_T, B_T, 128>);
    const cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(kernel), f32::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    return plan_launch(kernel, dim3((unsigned)f.grid), dim3((unsigned)f.threads), (size_t)f32::SMEM_BYTES, s, p);
}

}  // namespace

size_t float_sum_bytes(int mode, int64_t M, int64_t N, int64_t K, int sm_count) {
    const FloatShape f = float_shape(mode, M, N, K, sm_count);
    return f.pieces == 1 ? 0 : (size_t)(f.works - f.whole) * f32::TILE_VECS * sizeof(float4);
}
size_t float_counter_bytes(int sm_count) { return ((size_t)f32::per_sm(64) * sm_count + 2) * sizeof(unsigned int); }

cudaError_t launch_float(const Product& w, void* sums, unsigned int* counters, int sm_count, cudaStream_t s) {
    const FloatShape f = float_shape(w.mode, w.M, w.N, w.K, sm_count);
    f32::Params p;
    // whole vectors: every row of every operand and result starts on a 16-byte
    // boundary and ends with a whole vector (K where it is contiguous, A's rows
    // where they lie along K)
    bool vec = w.N % 4 == 0 && (w.a_mn ? w.M : w.K) % 4 == 0;
    for (int i = 0; i < 2; ++i) {
        p.a[i] = static_cast<const float*>(w.a[i].base);
        p.b[i] = static_cast<const float*>(w.b[i].base);
        vec = vec && plan_aligned16(p.a[i]) && plan_aligned16(p.b[i]) && w.a[i].pitch % 4 == 0 && w.b[i].pitch % 4 == 0;
    }
    for (int i = 0; i < 3; ++i) {
        p.y[i] = static_cast<float*>(w.Y[i]);
        vec = vec && plan_aligned16(p.y[i]);
    }
    p.lda = w.a[0].pitch;
    p.ldb = w.b[0].pitch;
    p.M = w.M;
    p.N = w.N;
    p.K = w.K;
    p.tiles_m = f.tiles_m;
    p.tiles_item = f.tiles_item;
    p.tiles = f.tiles;
    p.whole = f.whole;
    p.works = f.works;
    p.pieces = f.pieces;
    p.source_slices = f.source_slices;
    p.slices = f.slices;
    p.act = w.act;
    p.sums = static_cast<float4*>(sums);
    p.taken = counters;
    p.left = counters + 1;
    p.arrived = counters + 2;
    switch (w.mode) {
        case FWD:
            return w.b_k ? launch_float_as<FWD, false, true>(p, vec, f, s)
                         : launch_float_as<FWD, false, false>(p, vec, f, s);
        case DX:
            return w.b_k ? launch_float_as<DX, false, true>(p, vec, f, s)
                         : launch_float_as<DX, false, false>(p, vec, f, s);
        default: return launch_float_as<DW, true, false>(p, vec, f, s);
    }
}

}  // namespace gated
}  // namespace olc
