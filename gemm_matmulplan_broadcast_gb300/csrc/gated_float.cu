// The gated feed-forward product in FLOAT: act(X Wg) (X Wu) on the FMA pipes,
// which keep float32 products exact to one rounding (the tensor cores round
// their operands).
//
// 4 M D F operations at two a paired FMA bound it.  A block of 64 threads
// takes 64 rows x 64 columns of both products: the shared-memory tile of B
// holds 64 columns of Wg next to the same 64 of Wu, and a thread's
// accumulators are 8 rows x 8 columns of each, so that it forms act(g) u of
// its own outputs from registers.  With 8 x 16 accumulators a thread, 64 paired
// FMAs take six 16-byte reads of shared memory, three quarters of its cycles
// (8 x 8: all of them, which bounds that form).  64-row tiles, because their
// last round over the SMs wastes less than that of 128 rows ([1024, 1024] x
// [1024, 2816]: 704 tiles, 4.6 an SM, against 2.3).  Slices of K, 16 deep, come
// through asynchronous copies two ahead; weights stored [F, D] are transposed
// through registers.
#include "gated_internal.h"
#include "plan_state.h"

namespace olc {
namespace gated {
namespace f32 {

constexpr int TM = 64, TN = 64, KS = 16;          // rows, columns of each product, depth of a slice
constexpr int THREADS = 64;
constexpr int STAGES = 3;
constexpr int AP = KS + 4;                        // floats between rows of X's tile: four rows in four bank groups
constexpr int A_FLOATS = TM * AP, B_FLOATS = KS * 2 * TN;
constexpr int SMEM_BYTES = STAGES * (A_FLOATS + B_FLOATS) * 4;

struct Params {
    const float *X, *Wg, *Wu;
    float *H, *G, *U;         // G, U may be null
    int64_t M, D, F;
    int64_t tiles_m, tiles;
    int64_t rounds;           // whole tiles a block
    int64_t sharers;          // blocks that share the rest, at least four slices each
    int slices;               // of K a tile
    int act;
    float4* shares;           // [2 blocks][32][threads]: partial sums of a block's first and last shared tile
    unsigned int* arrived;    // [shared tiles], zero between launches
};

// the first four of n elements at `from`, zeros past the n-th; VEC: whole
// 16-byte vectors
template <bool VEC>
__device__ __forceinline__ float4 four(const float* from, int64_t n) {
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
__device__ __forceinline__ void copy_four(float* to, const float* from, const float* any, int64_t n) {
    if constexpr (VEC) {
        copy_async<16>(to, n > 0 ? from : any, n > 0 ? 16 : 0);
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) copy_async<4>(to + q, q < n ? from + q : any, q < n ? 4 : 0);
    }
}

// TRANS: the weights are stored [F, D]
template <bool VEC, bool TRANS>
__global__ void __launch_bounds__(THREADS, 4) kernel(const Params p) {
    extern __shared__ __align__(16) float smem[];     // stages of X [64 rows][k], B [k][64 of Wg, 64 of Wu]
    __shared__ int last;
    const int t = threadIdx.x, tx = t & 7, ty = t >> 3;
    const int64_t grid = gridDim.x, block = blockIdx.x;
    // the shared tiles' slices, laid end to end
    const int64_t whole = p.rounds * grid, steps = (p.tiles - whole) * p.slices, sharers = p.sharers;
    const int64_t share0 = block < sharers ? block * steps / sharers : 0;
    const int64_t share1 = block < sharers ? (block + 1) * steps / sharers : 0;
    int64_t m0 = 0, n0 = 0;
    float* const as = smem;
    float* const bs = smem + STAGES * A_FLOATS;

    // A slice's addresses advance by additions: this thread's rows of X are t /
    // 4 + 16 q at K elements 4 (t % 4); its rows of the weights K elements t / 16
    // + 4 q at columns 4 (t % 16), or (TRANS) one column of each at all sixteen.
    const float *pa = nullptr, *pg = nullptr, *pu = nullptr;
    int64_t ka = 0, kb = 0;          // their K elements
    unsigned rows_in = 0;
    bool col_in = false;
    const int64_t da = 16 * p.D, db = 4 * p.F;
    float* const a_to = as + (t >> 2) * AP + (t & 3) * 4;
    float* const b_to = TRANS ? bs + t : bs + (t >> 4) * 2 * TN + (t & 15) * 4;
    auto begin = [&](int64_t s0) {
        const int64_t k0 = s0 * KS;
        const int64_t row = m0 + (t >> 2);
        rows_in = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) rows_in |= (unsigned)(row + 16 * q < p.M) << q;
        ka = k0 + (t & 3) * 4;
        pa = p.X + row * p.D + ka;
        if constexpr (TRANS) {
            const int64_t col = n0 + t;
            col_in = col < p.F;
            kb = k0;
            pg = p.Wg + col * p.D + kb;
            pu = p.Wu + col * p.D + kb;
        } else {
            const int64_t col = n0 + (t & 15) * 4;
            col_in = col < p.F;
            kb = k0 + (t >> 4);
            pg = p.Wg + kb * p.F + col;
            pu = p.Wu + kb * p.F + col;
        }
    };
    auto fetch = [&](int stage) {
        float* a = a_to + stage * A_FLOATS;
        float* b = b_to + stage * B_FLOATS;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            copy_four<VEC>(a + 16 * q * AP, pa + q * da, p.X, (rows_in >> q) & 1u ? p.D - ka : 0);
        pa += KS;
        ka += KS;
        if constexpr (!TRANS) {
            const int64_t left = col_in ? p.F - (n0 + (t & 15) * 4) : 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t n = kb + 4 * q < p.D ? left : 0;
                copy_four<VEC>(b + 4 * q * 2 * TN, pg + q * db, p.Wg, n);
                copy_four<VEC>(b + 4 * q * 2 * TN + TN, pu + q * db, p.Wu, n);
            }
            pg += 4 * db;
            pu += 4 * db;
            kb += KS;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        if constexpr (TRANS) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float* w = q ? pu : pg;
                float4 v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = four<VEC>(w + 4 * i, col_in ? p.D - kb - 4 * i : 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float* to = b + 4 * i * 2 * TN + q * TN;
                    to[0] = v[i].x;
                    to[2 * TN] = v[i].y;
                    to[4 * TN] = v[i].z;
                    to[6 * TN] = v[i].w;
                }
            }
            pg += KS;
            pu += KS;
            kb += KS;
        }
    };

    // rows ty + 8 i; columns 32 c + 4 tx + (0..3) of g (j = 0..3), then of u
    F2 acc[8][8];

    // acc = the tile's products over slices [s0, s0 + n)
    auto multiply = [&](int64_t s0, int n) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i][j] = 0;
        __syncthreads();             // all are done with the tile before
        begin(s0);
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
            const float* a = as + stage * A_FLOATS + ty * AP;
            const float* b = bs + stage * B_FLOATS + tx * 4;
            if (++stage == STAGES) stage = 0;
#pragma unroll
            for (int k4 = 0; k4 < KS; k4 += 4) {
                float4 x[8];
#pragma unroll
                for (int r = 0; r < 8; ++r) x[r] = *reinterpret_cast<const float4*>(a + r * 8 * AP + k4);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    F2 w[8];
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(b + (k4 + k) * 2 * TN + h * 32);
                        w[2 * h] = v.x;
                        w[2 * h + 1] = v.y;
                    }
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        const float e = k == 0 ? x[r].x : (k == 1 ? x[r].y : (k == 2 ? x[r].z : x[r].w));
                        const F2 e2 = pack_f2(e, e);
#pragma unroll
                        for (int j = 0; j < 8; ++j) fma_f2(acc[r][j], e2, w[j]);
                    }
                }
            }
        }
    };
    auto finish = [&] {
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const int64_t row = m0 + ty + 8 * r;
            if (row >= p.M) continue;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int64_t col = n0 + 32 * c + tx * 4;
                if (col >= p.F) continue;
                float g[4], u[4], h[4];
                unpack_f2(acc[r][2 * c], g[0], g[1]);
                unpack_f2(acc[r][2 * c + 1], g[2], g[3]);
                unpack_f2(acc[r][4 + 2 * c], u[0], u[1]);
                unpack_f2(acc[r][4 + 2 * c + 1], u[2], u[3]);
#pragma unroll
                for (int j = 0; j < 4; ++j) h[j] = gate_value<true>(p.act, g[j]) * u[j];
                put_four<VEC>(p.H + row * p.F, col, p.F, h);
                if (p.G) put_four<VEC>(p.G + row * p.F, col, p.F, g);
                if (p.U) put_four<VEC>(p.U + row * p.F, col, p.F, u);
            }
        }
    };
    auto tile_at = [&](int64_t tile) {
        // rows fastest: the row tiles of a column read its weights from L2
        m0 = tile % p.tiles_m * TM;
        n0 = tile / p.tiles_m * TN;
    };

    for (int64_t r = 0; r < p.rounds; ++r) {
        tile_at(block + r * grid);
        multiply(0, p.slices);
        finish();
    }
    for (int64_t s = share0; s < share1;) {
        const int64_t tile = s / p.slices, s0 = s % p.slices;
        const int n = (int)min64(p.slices - s0, share1 - s);
        s += n;
        tile_at(whole + tile);
        multiply(s0, n);
        if (n == p.slices) {
            finish();
            continue;
        }
        // the blocks whose shares hold the tile's first and last slice
        const int64_t u0 = tile * p.slices, u1 = u0 + p.slices - 1;
        const int64_t c0 = ((u0 + 1) * sharers - 1) / steps, c1 = ((u1 + 1) * sharers - 1) / steps;
        auto slot = [&](int64_t c) {          // where block c left this tile: its first shared tile, or its last
            return p.shares + (2 * c + (c * steps / sharers / p.slices == tile ? 0 : 1)) * (32 * THREADS) + t;
        };
        float4* mine = slot(block);
#pragma unroll
        for (int r = 0; r < 8; ++r)
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                float4 v;
                unpack_f2(acc[r][j], v.x, v.y);
                unpack_f2(acc[r][j + 1], v.z, v.w);
                __stcg(mine + (r * 4 + j / 2) * THREADS, v);
            }
        __threadfence();
        __syncthreads();
        if (t == 0) last = atomicAdd(p.arrived + tile, 1u) == (unsigned int)(c1 - c0);
        __syncthreads();
        if (!last) continue;
        __threadfence();
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i][j] = 0;
        for (int64_t c = c0; c <= c1; ++c) {
            const float4* from = slot(c);
#pragma unroll
            for (int r = 0; r < 8; ++r)
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const float4 v = __ldcg(from + (r * 4 + j / 2) * THREADS);
                    acc[r][j] = add2(acc[r][j], pack_f2(v.x, v.y));
                    acc[r][j + 1] = add2(acc[r][j + 1], pack_f2(v.z, v.w));
                }
        }
        finish();
        if (t == 0) p.arrived[tile] = 0u;
    }
}

}  // namespace f32

constexpr int kFloatPerSm = 4;            // blocks that reside (registers)

namespace {
struct FloatShape {
    int64_t tiles_m, tiles, grid, rounds, sharers;
    int slices;
};
FloatShape float_shape(int64_t M, int64_t D, int64_t F, int sm_count) {
    FloatShape f;
    f.tiles_m = ceil_div(M, f32::TM);
    f.tiles = f.tiles_m * ceil_div(F, f32::TN);
    f.slices = (int)ceil_div(D, f32::KS);
    f.grid = max64(1, min64((int64_t)kFloatPerSm * sm_count, f.tiles * max64(1, f.slices / 4)));
    f.rounds = f.tiles / f.grid;
    // no share is empty
    f.sharers = max64(1, min64(f.grid, (f.tiles - f.rounds * f.grid) * f.slices / 4));
    return f;
}
}  // namespace

size_t float_share_bytes(int64_t M, int64_t D, int64_t F, int sm_count) {
    const FloatShape f = float_shape(M, D, F, sm_count);
    return f.tiles == f.rounds * f.grid ? 0 : (size_t)f.grid * 2 * f32::THREADS * 32 * sizeof(float4);
}
size_t float_counter_bytes(int sm_count) { return (size_t)kFloatPerSm * sm_count * sizeof(unsigned int); }

cudaError_t launch_float(const float* X, const float* Wg, const float* Wu, float* H, float* G, float* U, int64_t M,
                         int64_t D, int64_t F, int trans_w, int act, void* shares, unsigned int* counters,
                         int sm_count, cudaStream_t s) {
    const FloatShape f = float_shape(M, D, F, sm_count);
    const f32::Params p{X, Wg, Wu, H, G, U, M, D, F, f.tiles_m, f.tiles, f.rounds, f.sharers, f.slices, act,
                        static_cast<float4*>(shares), counters};
    // whole vectors: along K of X and of transposed weights, along F of the others and of the results
    bool vec = D % 4 == 0 && F % 4 == 0;
    for (const void* q : {(const void*)X, (const void*)Wg, (const void*)Wu, (const void*)H, (const void*)G, (const void*)U})
        vec = vec && plan_aligned16(q);
    auto run = [&](auto kernel) {
        const cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(kernel), f32::SMEM_BYTES);
        if (e != cudaSuccess) return e;
        return plan_launch(kernel, dim3((unsigned)f.grid), dim3(f32::THREADS), (size_t)f32::SMEM_BYTES, s, p);
    };
    if (vec) return trans_w ? run(f32::kernel<true, true>) : run(f32::kernel<true, false>);
    return trans_w ? run(f32::kernel<false, true>) : run(f32::kernel<false, false>);
}

}  // namespace gated
}  // namespace olc
