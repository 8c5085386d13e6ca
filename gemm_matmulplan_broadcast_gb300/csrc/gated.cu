// The gated feed-forward product and its gradient.
//
//   g = X Wg,  u = X Wu,  h = act(g) u                  X [M, D], W [D, F] (or stored [F, D])
//   dg = dh u act'(g),  du = dh act(g)
//   dX = dg Wg' + du Wu',  dWg = X' dg,  dWu = X' du
//
// FLOAT16 / BFLOAT16 run on tcgen05 CTA pairs with 256 x 256 accumulators in
// TMEM (or, FWD of products that leave SMs idle, on single CTAs), the mainloop
// of the general tiles with three choices of operands:
//
//   FWD  each CTA of the pair supplies half of the accumulator's columns: the
//        first 128 columns of Wg, the second the same 128 columns of Wu.  So
//        both CTAs hold g and u of the same outputs side by side and the
//        epilogue forms act(g) u from float32 accumulators: neither product
//        is written unless training asks for it.
//   DX   one accumulator over both terms: the K loop runs through dg and Wg,
//        then through du and Wu; nothing is added in memory.
//   DW   both weights' gradients in one launch.
//
// dg and du are formed by one elementwise pass (five tensors of M x F moved,
// no product) and rounded to 16 bits, because the tensor cores read 16-bit
// operands: their rounding is of the size of the results' own.
// Products bound these kernels (4 M D F operations forward, 8 backward) except
// for few rows, where the weights' bytes do.  Measured in BF16: [16384, 4096] x
// [4096, 14336] forward with g and u kept 2.04 ms after a pause (1882 TFLOP/s,
// the library product's burst rate) and 2.40 ms back to back (1605, under the
// power limit); [8192, 4096] backward 2.26 and 2.50 ms.
#include <cstring>
#include <initializer_list>
#include <new>

#include "gated_internal.h"
#include "plan_state.h"
#include "tc_ptx.cuh"

namespace olc {
namespace gated {

using namespace olc::tc;

// ---- the products on CTA pairs ------------------------------------------------

constexpr int STAGES = 6;
constexpr int A_BYTES = 128 * BK * 2;               // this CTA's 128 rows of A
constexpr int B_BYTES = 128 * BK * 2;               // this CTA's 128 columns of B
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int PAIR_THREADS = 224;                   // A loader, MMA, 4 epilogue warps, B loader
constexpr int STAGE_PITCH = 36;                     // 32-bit words per staged row
constexpr int STAGING_BYTES = 4 * 32 * STAGE_PITCH * 4;
constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + STAGING_BYTES + 1024 + 512;
constexpr int TMEM_COLS = 512;                      // two accumulators
constexpr int RASTER = 8;                           // pair rows a raster group

struct Barriers {
    uint64_t full[STAGES];
    uint64_t empty[STAGES];
    uint64_t acc_full[2];
    uint64_t acc_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
};

struct Params {
    int64_t M, N;             // an output's rows and columns
    int64_t tiles_m, tiles_n;
    int64_t units;            // tiles x outputs x slices
    int64_t k_blocks;         // K blocks of one operand pair
    int64_t k_total;          // K blocks of an accumulator (DX: both pairs')
    int64_t k_slice;          // K blocks a slice takes
    int splits;               // K slices; > 1: float32 partial results
    int items;                // outputs of their own operands (DW: 2)
    int a_mn, b_k, b_blocks;
    int is_bf16, act;
    int aligned;              // every output row on a 16-byte boundary
    int paired;               // every output row on a 4-byte boundary
    void* Y[3];               // FWD: h, g, u (null: not kept); DX: dX; DW: dWg, dWu
    float* partial;           // [split][plane][M][partial_pitch]
    int64_t partial_pitch;
    unsigned int* err;
};

struct Maps {
    CUtensorMap a[2], b[2];
};

// A warp's 32 rows of W packed pairs of 16-bit columns through its staging
// rows, so that a row's run is stored whole.
template <int W>
__device__ __forceinline__ void store_run(const Params& p, void* Y, uint32_t* rows, const uint32_t (&packed)[W],
                                          int lane, int64_t row0, int64_t col0) {
    constexpr int PITCH = W + 4, LANES = W / 4;      // lanes on a row
    uint4* mine = reinterpret_cast<uint4*>(rows + lane * PITCH);
#pragma unroll
    for (int q = 0; q < LANES; ++q)
        mine[q] = make_uint4(packed[4 * q], packed[4 * q + 1], packed[4 * q + 2], packed[4 * q + 3]);
    __syncwarp();
    unsigned short* y = static_cast<unsigned short*>(Y);
    if (p.aligned) {
        const int cq = lane % LANES;
        const int64_t col = col0 + cq * 8;
#pragma unroll
        for (int j = 0; j < LANES; ++j) {
            const int rr = lane / LANES + 32 / LANES * j;
            const uint4 w = *reinterpret_cast<const uint4*>(rows + rr * PITCH + cq * 4);
            if (row0 + rr < p.M && col < p.N) *reinterpret_cast<uint4*>(y + (row0 + rr) * p.N + col) = w;
        }
    } else if (p.paired) {
        const int cw = lane % W;
        const int64_t col = col0 + cw * 2;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const int rr = lane / W + 32 / W * j;
            const uint32_t w = rows[rr * PITCH + cw];
            if (row0 + rr < p.M && col < p.N) *reinterpret_cast<uint32_t*>(y + (row0 + rr) * p.N + col) = w;
        }
    } else {
        const unsigned short* half = reinterpret_cast<const unsigned short*>(rows);
#pragma unroll 8
        for (int rr = 0; rr < 32; ++rr) {
#pragma unroll
            for (int j = 0; j < W / 16; ++j) {
                const int64_t col = col0 + lane + 32 * j;
                if (row0 + rr < p.M && col < p.N)
                    y[(row0 + rr) * p.N + col] = half[rr * PITCH * 2 + lane + 32 * j];
            }
        }
    }
    __syncwarp();                                    // the rows are rewritten by the next run
}

// W float32 columns of the warp's 32 rows into a partial plane
template <int W>
__device__ __forceinline__ void store_partial(const Params& p, float* plane, uint32_t* rows, const uint32_t* r,
                                              int lane, int64_t row0, int64_t col0) {
    constexpr int PITCH = W + 4, LANES = W / 4;
    uint4* mine = reinterpret_cast<uint4*>(rows + lane * PITCH);
#pragma unroll
    for (int q = 0; q < LANES; ++q) mine[q] = make_uint4(r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]);
    __syncwarp();
    const int cq = lane % LANES;
    const int64_t col = col0 + cq * 4;
#pragma unroll
    for (int j = 0; j < LANES; ++j) {
        const int rr = lane / LANES + 32 / LANES * j;
        const uint4 w = *reinterpret_cast<const uint4*>(rows + rr * PITCH + cq * 4);
        if (row0 + rr < p.M && col < p.partial_pitch)
            *reinterpret_cast<uint4*>(plane + (row0 + rr) * p.partial_pitch + col) = w;
    }
    __syncwarp();
}

__device__ __forceinline__ uint32_t pack16(float lo, float hi, int is_bf16) {
    if (is_bf16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// 32 columns of g and u (accumulators) to packed h, g and u
__device__ __forceinline__ void gate_run(const Params& p, const uint32_t (&g)[32], const uint32_t (&x)[32], uint32_t* ph,
                                         uint32_t* pg, uint32_t* pu) {
    by_activation(p.act, [&](auto act) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float h0 = gate_value<false, act.value>(__uint_as_float(g[2 * i])) * __uint_as_float(x[2 * i]);
            const float h1 = gate_value<false, act.value>(__uint_as_float(g[2 * i + 1])) * __uint_as_float(x[2 * i + 1]);
            ph[i] = pack16(h0, h1, p.is_bf16);
        }
    });
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        pg[i] = pack16(__uint_as_float(g[2 * i]), __uint_as_float(g[2 * i + 1]), p.is_bf16);
        pu[i] = pack16(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]), p.is_bf16);
    }
}
template <int W>
__device__ __forceinline__ void store_gated(const Params& p, uint32_t* rows, const uint32_t (&ph)[W],
                                            const uint32_t (&pg)[W], const uint32_t (&pu)[W], int lane, int64_t row0,
                                            int64_t col0) {
    store_run(p, p.Y[0], rows, ph, lane, row0, col0);
    if (p.Y[1]) store_run(p, p.Y[1], rows, pg, lane, row0, col0);
    if (p.Y[2]) store_run(p, p.Y[2], rows, pu, lane, row0, col0);
}

template <int MODE>
__global__ void __launch_bounds__(PAIR_THREADS, 1)
pair_kernel(const __grid_constant__ CUtensorMap map_a0, const __grid_constant__ CUtensorMap map_a1,
            const __grid_constant__ CUtensorMap map_b0, const __grid_constant__ CUtensorMap map_b1, const Params p) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* base =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint32_t* staging = reinterpret_cast<uint32_t*>(base + STAGES * STAGE_BYTES);
    Barriers* s = reinterpret_cast<Barriers*>(base + STAGES * STAGE_BYTES + STAGING_BYTES);
    volatile int* abort_flag = &s->abort_flag;
    const uint32_t rank = pair::cluster_rank();
    const bool leader = rank == 0;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&s->full[i], 2);        // the leader's A and B loaders arm it
            mbar_init(&s->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s->acc_full[i], 1);
            mbar_init(&s->acc_empty[i], 8);   // four epilogue warps in each CTA
        }
        mbar_init(&s->drain, 1);
        s->abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncwarp();
    if (warp == 1) pair::tmem_alloc2(&s->tmem_base, TMEM_COLS);
    tc_fence_before();
    pair::cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = s->tmem_base;

    // unit -> K slice, output, tile (groups of RASTER pair rows, rows fastest)
    const int64_t per_item = p.tiles_m * p.tiles_n;
    auto coords = [&](int64_t u, int& slice, int& item, int64_t& mb, int64_t& nb) {
        slice = (int)(u % p.splits);
        const int64_t t = u / p.splits;
        item = (int)(t / per_item);
        const int64_t r = t % per_item;
        const int64_t span = (int64_t)RASTER * p.tiles_n;
        const int64_t first = r / span * RASTER;
        const int64_t gm = min64(p.tiles_m - first, RASTER);
        const int64_t in = r % span;
        mb = first + in % gm;
        nb = in / gm;
    };

    if (warp == 0 || warp == 6) {
        if (lane == 0) {
            const bool load_a = warp == 0;
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(load_a ? &map_a0 : &map_b0)) : "memory");
            if (MODE != FWD || !load_a)
                asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(load_a ? &map_a1 : &map_b1)) : "memory");
            const uint32_t stage0 = smem_u32(base);
            const uint32_t full0_leader = pair::map_to(&s->full[0], 0);
            uint32_t stage = 0, phase = 0, armed_bits = 0, parity_bits = 0;
            bool ok = true;
            for (int64_t u = pair::cluster_id(); u < p.units && ok; u += pair::cluster_count()) {
                int slice, item;
                int64_t mb, nb;
                coords(u, slice, item, mb, nb);
                const int m0 = (int)(mb * 256 + rank * 128);
                const int n0 = (int)(MODE == FWD ? nb * 128 : nb * 256 + rank * 128);
                const int64_t kb0 = slice * p.k_slice, kb1 = min64(p.k_total, kb0 + p.k_slice);
                const uint32_t tx = load_a ? 2u * A_BYTES : 2u * B_BYTES;
                for (int64_t kb = kb0; kb < kb1; ++kb) {
                    // which operand pair, and where along its K
                    int which = MODE == DW ? item : (MODE == FWD && !load_a ? (int)rank : 0);
                    int k0 = (int)kb * BK;
                    if (MODE == DX && kb >= p.k_blocks) {
                        which = 1;
                        k0 = (int)(kb - p.k_blocks) * BK;
                    }
                    const CUtensorMap* map = load_a ? (which ? &map_a1 : &map_a0) : (which ? &map_b1 : &map_b0);
                    if (!mbar_wait(&s->empty[stage], phase ^ 1, abort_flag, p.err)) { ok = false; break; }
                    const uint32_t sa = stage0 + stage * STAGE_BYTES;
                    const uint32_t sb = sa + A_BYTES;
                    const uint32_t full_leader = full0_leader + stage * (uint32_t)sizeof(uint64_t);
                    if (leader) {
                        mbar_arrive_expect_tx(&s->full[stage], tx);
                        armed_bits |= 1u << stage;
                        parity_bits = (parity_bits & ~(1u << stage)) | (phase << stage);
                    }
                    if (load_a) {
                        if (!p.a_mn) {
                            pair::tma_load_3d_pair(sa, map, full_leader, k0, m0, 0);
                        } else {
                            pair::tma_load_3d_pair(sa, map, full_leader, m0, k0, 0);
                            pair::tma_load_3d_pair(sa + 64 * BK * 2, map, full_leader, m0 + 64, k0, 0);
                        }
                    } else if (p.b_k) {
                        pair::tma_load_3d_pair(sb, map, full_leader, k0, n0, 0);
                    } else if (p.b_blocks) {
                        pair::tma_load_4d_pair(sb, map, full_leader, 0, k0, n0 >> 6, 0);
                    } else {
                        pair::tma_load_3d_pair(sb, map, full_leader, n0, k0, 0);
                        pair::tma_load_3d_pair(sb + 64 * BK * 2, map, full_leader, n0 + 64, k0, 0);
                    }
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
            }
            if (*abort_flag && leader) {
                for (int i = 0; i < STAGES; ++i)
                    if ((armed_bits >> i) & 1u) mbar_wait_drain(&s->full[i], (parity_bits >> i) & 1u);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            const uint32_t idesc = instr_desc(p.is_bf16, 256, 256, p.a_mn, p.b_k ? 0 : 1);
            const uint32_t stage0 = smem_u32(base);
            const uint64_t a_desc0 =
                p.a_mn ? smem_desc(stage0, 64 * BK * 2, 1024, 2u) : smem_desc(stage0, 16, 1024, 2u);
            const uint64_t b_desc0 = p.b_k ? smem_desc(stage0 + A_BYTES, 16, 1024, 2u)
                                           : smem_desc(stage0 + A_BYTES, 64 * BK * 2, 1024, 2u);
            const uint64_t a_step = p.a_mn ? (UMMA_K * 128) >> 4 : (UMMA_K * 2) >> 4;
            const uint64_t b_step = p.b_k ? (UMMA_K * 2) >> 4 : (UMMA_K * 128) >> 4;
            uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
            bool ok = true;
            for (int64_t u = pair::cluster_id(); u < p.units && ok; u += pair::cluster_count()) {
                const int64_t kb0 = (u % p.splits) * p.k_slice, kb1 = min64(p.k_total, kb0 + p.k_slice);
                if (!mbar_wait(&s->acc_empty[acc], acc_phase ^ 1, abort_flag, p.err)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + acc * 256;
                uint32_t first = 0u;
                for (int64_t kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait(&s->full[stage], phase, abort_flag, p.err)) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t so = (uint64_t)((stage * STAGE_BYTES) >> 4);
#pragma unroll
                    for (int kk = 0; kk < BK / UMMA_K; ++kk)
                        pair::mma2_f16(d_tmem, a_desc0 + so + kk * a_step, b_desc0 + so + kk * b_step, idesc,
                                       kk > 0 ? 1u : first);
                    first = 1u;
                    pair::commit2_both(&s->empty[stage]);
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
                if (!ok) break;
                pair::commit2_both(&s->acc_full[acc]);
                if (++acc == 2) { acc = 0; acc_phase ^= 1; }
            }
            pair::commit2_local(&s->drain);
            mbar_wait_drain(&s->drain, 0);
        }
        __syncwarp();
    } else {
        const int lane_group = warp & 3;
        const uint32_t acc_empty_leader[2] = {pair::map_to(&s->acc_empty[0], 0), pair::map_to(&s->acc_empty[1], 0)};
        uint32_t* rows = staging + lane_group * 32 * STAGE_PITCH;
        uint32_t acc = 0, acc_phase = 0;
        for (int64_t u = pair::cluster_id(); u < p.units; u += pair::cluster_count()) {
            int slice, item;
            int64_t mb, nb;
            coords(u, slice, item, mb, nb);
            const bool ok = mbar_wait(&s->acc_full[acc], acc_phase, abort_flag, p.err);
            if (!__all_sync(0xffffffffu, ok)) break;      // the warp stays together for tcgen05.ld
            tc_fence_after();
            const int64_t row0 = mb * 256 + rank * 128 + lane_group * 32;     // the warp's first row
            const uint32_t t_base = tmem_base + ((uint32_t)(lane_group * 32) << 16) + acc * 256;
            if (p.splits > 1) {
                const int planes = MODE == DX ? 1 : 2;
#pragma unroll 1
                for (int c = 0; c < 256; c += 32) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(t_base + c, r);
                    const int plane = MODE == FWD ? c >> 7 : item;
                    const int64_t col0 = MODE == FWD ? nb * 128 + (c & 127) : nb * 256 + c;
                    if (row0 >= p.M || col0 >= p.N) continue;
                    store_partial<32>(p, p.partial + ((int64_t)slice * planes + plane) * p.M * p.partial_pitch, rows, r,
                                  lane, row0, col0);
                }
            } else if constexpr (MODE == FWD) {
#pragma unroll 1
                for (int c = 0; c < 128; c += 64) {
                    uint32_t ph[32], pg[32], pu[32];
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        uint32_t g[32], x[32];
                        tmem_ld_32x32b_x32(t_base + c + hh * 32, g);
                        tmem_ld_32x32b_x32(t_base + 128 + c + hh * 32, x);
                        gate_run(p, g, x, ph + hh * 16, pg + hh * 16, pu + hh * 16);
                    }
                    const int64_t col0 = nb * 128 + c;
                    if (row0 >= p.M || col0 >= p.N) continue;
                    store_gated(p, rows, ph, pg, pu, lane, row0, col0);
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < 256; c += 64) {
                    uint32_t packed[32];
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        uint32_t r[32];
                        tmem_ld_32x32b_x32(t_base + c + hh * 32, r);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            packed[hh * 16 + i] =
                                pack16(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]), p.is_bf16);
                    }
                    const int64_t col0 = nb * 256 + c;
                    if (row0 >= p.M || col0 >= p.N) continue;
                    store_run(p, p.Y[MODE == DW ? item : 0], rows, packed, lane, row0, col0);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) pair::remote_arrive(acc_empty_leader[acc]);
            if (++acc == 2) { acc = 0; acc_phase ^= 1; }
        }
    }

    tc_fence_before();
    __syncwarp();
    __syncthreads();
    pair::cluster_sync();          // no remote arrival may target a CTA that has left
    tc_fence_after();
    if (warp == 1) pair::tmem_dealloc2(tmem_base, TMEM_COLS);
}

// ---- FWD on single CTAs -----------------------------------------------------------

// 128 rows x 64 columns of both products a CTA (one 128 x 128 accumulator): a
// quarter of the pair's tile, for products whose pair tiles would leave SMs
// idle.  Operands pass through shared memory at its full bandwidth here (32
// KiB in and out a K block for 256 cycles of MMAs; both CTAs of a pair share
// B), so large products keep the pairs.  Eight warps form the outputs, since
// nothing hides the only tile's epilogue.
namespace single {

constexpr int COLS = 64;
constexpr int A_BYTES1 = 128 * BK * 2;
constexpr int W_BYTES1 = BK * COLS * 2;
constexpr int STAGE1 = A_BYTES1 + 2 * W_BYTES1;     // 32 KiB
constexpr int EPI_WARPS = 8;                        // 32 rows x 32 columns each
constexpr int THREADS1 = (2 + EPI_WARPS) * 32;      // + loader, MMA
constexpr int ROW_WORDS = 16;                       // words of a staged row
constexpr int STAGING1 = EPI_WARPS * 32 * (ROW_WORDS + 4) * 4;
constexpr int SMEM1 = STAGES * STAGE_BYTES + STAGING1 + 1024 + 512;
constexpr int TMEM1 = 256;                          // two accumulators
static_assert(STAGE1 == STAGE_BYTES, "the pair's ring sizes hold");

}  // namespace single

__global__ void __launch_bounds__(single::THREADS1, 1)
single_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_g,
              const __grid_constant__ CUtensorMap map_u, const Params p) {
    using namespace single;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* base =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint32_t* staging = reinterpret_cast<uint32_t*>(base + STAGES * STAGE1);
    Barriers* s = reinterpret_cast<Barriers*>(base + STAGES * STAGE1 + STAGING1);
    volatile int* abort_flag = &s->abort_flag;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&s->full[i], 1);
            mbar_init(&s->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s->acc_full[i], 1);
            mbar_init(&s->acc_empty[i], EPI_WARPS);
        }
        mbar_init(&s->drain, 1);
        s->abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncwarp();
    if (warp == 1) tmem_alloc(&s->tmem_base, TMEM1);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = s->tmem_base;

    // unit -> K slice, tile (rows fastest: the row tiles of a column share its weights in L2)
    auto coords = [&](int64_t u, int& slice, int64_t& mb, int64_t& nb) {
        slice = (int)(u % p.splits);
        const int64_t t = u / p.splits;
        mb = t % p.tiles_m;
        nb = t / p.tiles_m;
    };

    if (warp == 0) {
        if (lane == 0) {
            uint32_t stage = 0, phase = 0, armed = 0, parity = 0;
            bool ok = true;
            for (int64_t u = blockIdx.x; u < p.units && ok; u += gridDim.x) {
                int slice;
                int64_t mb, nb;
                coords(u, slice, mb, nb);
                const int m0 = (int)(mb * 128), n0 = (int)(nb * COLS);
                const int64_t kb0 = slice * p.k_slice, kb1 = min64(p.k_total, kb0 + p.k_slice);
                for (int64_t kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait(&s->empty[stage], phase ^ 1, abort_flag, p.err)) { ok = false; break; }
                    const uint32_t sa = smem_u32(base) + stage * STAGE1, bar = smem_u32(&s->full[stage]);
                    const int k0 = (int)kb * BK;
                    mbar_arrive_expect_tx(&s->full[stage], STAGE1);
                    armed |= 1u << stage;
                    parity = (parity & ~(1u << stage)) | (phase << stage);
                    tma_load_3d(sa + A_BYTES1, &map_g, bar, p.b_k ? k0 : n0, p.b_k ? n0 : k0, 0);
                    tma_load_3d(sa + A_BYTES1 + W_BYTES1, &map_u, bar, p.b_k ? k0 : n0, p.b_k ? n0 : k0, 0);
                    tma_load_3d(sa, &map_x, bar, k0, m0, 0);
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
            }
            if (*abort_flag)
                for (int i = 0; i < STAGES; ++i)
                    if ((armed >> i) & 1u) mbar_wait_drain(&s->full[i], (parity >> i) & 1u);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = instr_desc(p.is_bf16, 128, 2 * COLS, 0, p.b_k ? 0 : 1);
            const uint32_t stage0 = smem_u32(base);
            const uint64_t a_desc0 = smem_desc(stage0, 16, 1024, 2u);
            const uint64_t b_desc0 = p.b_k ? smem_desc(stage0 + A_BYTES1, 16, 1024, 2u)
                                           : smem_desc(stage0 + A_BYTES1, W_BYTES1, 1024, 2u);
            const uint64_t a_step = (UMMA_K * 2) >> 4;
            const uint64_t b_step = p.b_k ? (UMMA_K * 2) >> 4 : (UMMA_K * 128) >> 4;
            uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
            bool ok = true;
            for (int64_t u = blockIdx.x; u < p.units && ok; u += gridDim.x) {
                const int64_t kb0 = (u % p.splits) * p.k_slice, kb1 = min64(p.k_total, kb0 + p.k_slice);
                if (!mbar_wait(&s->acc_empty[acc], acc_phase ^ 1, abort_flag, p.err)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + acc * 128;
                uint32_t first = 0u;
                for (int64_t kb = kb0; kb < kb1; ++kb) {
                    if (!mbar_wait(&s->full[stage], phase, abort_flag, p.err)) { ok = false; break; }
                    tc_fence_after();
                    const uint64_t so = (uint64_t)((stage * STAGE1) >> 4);
#pragma unroll
                    for (int kk = 0; kk < BK / UMMA_K; ++kk)
                        mma_f16(d_tmem, a_desc0 + so + kk * a_step, b_desc0 + so + kk * b_step, idesc,
                                kk > 0 ? 1u : first);
                    first = 1u;
                    mma_commit(&s->empty[stage]);
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
                if (!ok) break;
                mma_commit(&s->acc_full[acc]);
                if (++acc == 2) { acc = 0; acc_phase ^= 1; }
            }
            mma_commit(&s->drain);
            mbar_wait_drain(&s->drain, 0);
        }
        __syncwarp();
    } else {
        const int lane_group = warp & 3, half = (warp - 2) >> 2;      // rows, columns
        uint32_t* rows = staging + (warp - 2) * 32 * (ROW_WORDS + 4);
        uint32_t acc = 0, acc_phase = 0;
        for (int64_t u = blockIdx.x; u < p.units; u += gridDim.x) {
            int slice;
            int64_t mb, nb;
            coords(u, slice, mb, nb);
            const bool ok = mbar_wait(&s->acc_full[acc], acc_phase, abort_flag, p.err);
            if (!__all_sync(0xffffffffu, ok)) break;      // the warp stays together for tcgen05.ld
            tc_fence_after();
            const int64_t row0 = mb * 128 + lane_group * 32, col0 = nb * COLS + half * 32;
            const uint32_t t_base = tmem_base + ((uint32_t)(lane_group * 32) << 16) + acc * 128 + half * 32;
            if (p.splits > 1) {
#pragma unroll 1
                for (int plane = 0; plane < 2; ++plane) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(t_base + plane * COLS, r);
                    if (row0 >= p.M || col0 >= p.N) continue;
                    float* to = p.partial + ((int64_t)slice * 2 + plane) * p.M * p.partial_pitch;
#pragma unroll
                    for (int c = 0; c < 32; c += ROW_WORDS)
                        store_partial<ROW_WORDS>(p, to, rows, r + c, lane, row0, col0 + c);
                }
            } else {
                uint32_t ph[ROW_WORDS], pg[ROW_WORDS], pu[ROW_WORDS], g[32], x[32];
                tmem_ld_32x32b_x32(t_base, g);
                tmem_ld_32x32b_x32(t_base + COLS, x);
                gate_run(p, g, x, ph, pg, pu);
                if (row0 < p.M) store_gated(p, rows, ph, pg, pu, lane, row0, col0);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s->acc_empty[acc]);
            if (++acc == 2) { acc = 0; acc_phase ^= 1; }
        }
    }
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, TMEM1);
}

// ---- elementwise passes ---------------------------------------------------------

// Slices summed in slice order; FWD: h, g and u from the two planes' sums.
template <typename T>
__global__ void __launch_bounds__(256) join_kernel(const Params p, int mode) {
    const int planes = mode == DX ? 1 : 2;
    const int64_t groups = ceil_div(p.N, 4), plane_elems = p.M * p.partial_pitch;
    const int64_t n = p.M * groups * (mode == DW ? 2 : 1);
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += (int64_t)gridDim.x * 256) {
        const int64_t item = e / (p.M * groups), in = e % (p.M * groups);
        const int64_t row = in / groups, col = in % groups * 4;
        float4 v[2];
        for (int q = 0; q < (mode == FWD ? 2 : 1); ++q) {
            const float* src = p.partial + (mode == FWD ? q : item) * plane_elems + row * p.partial_pitch + col;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int s = 0; s < p.splits; ++s) {
                const float4 x = *reinterpret_cast<const float4*>(src + (int64_t)s * planes * plane_elems);
                a.x += x.x;
                a.y += x.y;
                a.z += x.z;
                a.w += x.w;
            }
            v[q] = a;
        }
        const float a[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
        const int64_t at = row * p.N + col;
        if (mode == FWD) {
            const float b[4] = {v[1].x, v[1].y, v[1].z, v[1].w};
            float h[4];
            by_activation(p.act, [&](auto act) {
#pragma unroll
                for (int i = 0; i < 4; ++i) h[i] = gate_value<false, act.value>(a[i]) * b[i];
            });
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (col + i >= p.N) break;
                static_cast<T*>(p.Y[0])[at + i] = Num<T>::from_acc(h[i]);
                if (p.Y[1]) static_cast<T*>(p.Y[1])[at + i] = Num<T>::from_acc(a[i]);
                if (p.Y[2]) static_cast<T*>(p.Y[2])[at + i] = Num<T>::from_acc(b[i]);
            }
        } else {
            T* y = static_cast<T*>(p.Y[mode == DW ? item : 0]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (col + i < p.N) y[at + i] = Num<T>::from_acc(a[i]);
        }
    }
}

// dg = dh u act'(g), du = dh act(g); outputs with a row pitch.  V = 1: any
// alignment, else 16 bytes an access.  Its bytes bound it ([2048, 14336] BF16:
// 294 MB in 40.8 us).
template <typename T, int V>
__global__ void __launch_bounds__(256) slope_kernel(const T* dH, const T* G, const T* U, T* dG, T* dU, int64_t rows,
                                                    int64_t cols, int64_t pitch, int act) {
    struct alignas(V * sizeof(T)) Pack { T v[V]; };
    constexpr bool EXACT = sizeof(T) == 4;
    const int64_t groups = cols / V;
    for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < rows * groups; e += (int64_t)gridDim.x * 256) {
        const int64_t row = e / groups, col = e % groups * V;
        const Pack h = *reinterpret_cast<const Pack*>(dH + row * cols + col);
        const Pack g = *reinterpret_cast<const Pack*>(G + row * cols + col);
        const Pack u = *reinterpret_cast<const Pack*>(U + row * cols + col);
        Pack a, b;
        by_activation(act, [&](auto which) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float value, slope;
                gate_slope<EXACT, which.value>(Num<T>::to_acc(g.v[i]), value, slope);
                const float d = Num<T>::to_acc(h.v[i]);
                a.v[i] = Num<T>::from_acc(d * Num<T>::to_acc(u.v[i]) * slope);
                b.v[i] = Num<T>::from_acc(d * value);
            }
        });
        *reinterpret_cast<Pack*>(dG + row * pitch + col) = a;
        *reinterpret_cast<Pack*>(dU + row * pitch + col) = b;
    }
}

// Operands that the TMA cannot read in place (rows off 16-byte boundaries) into
// rows of 16-byte groups, up to three in one launch.  A warp takes 32 groups of
// a row at a time, several on their way at once.  Elements come in the widest
// words that the row's address allows; a row two bytes off a word takes five
// words a group and shifts them (the word at either end holds a neighbouring
// element; where the tensor itself ends there, single elements are read).
// Bytes bound it: two tensors [4095, 14335] about 100 us, 4.7 TB/s read and
// written, [4096, 14334] (rows on words) 78 us, 6.0 TB/s.
struct Copies {
    struct One {
        const unsigned short* src;
        uint4* dst;
        int64_t rows, cols, chunks;      // chunks of a row
        int64_t first;                   // its first unit
    } one[3];
    int64_t units;
};
__device__ __forceinline__ uint4 group_of(const unsigned short* at, int64_t left, bool edge) {
    const uint32_t low = (uint32_t)reinterpret_cast<uintptr_t>(at) & 15u;
    if (left >= 8 && !(edge && (low & 3))) {
        if (low == 0) return __ldg(reinterpret_cast<const uint4*>(at));
        if ((low & 7) == 0) {
            const uint2 a = __ldg(reinterpret_cast<const uint2*>(at)), b = __ldg(reinterpret_cast<const uint2*>(at) + 1);
            return make_uint4(a.x, a.y, b.x, b.y);
        }
        uint32_t w[5];
        const bool odd = low & 2;
        const uint32_t* words = reinterpret_cast<const uint32_t*>(reinterpret_cast<uintptr_t>(at) & ~uintptr_t(3));
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __ldg(words + j);
        if (!odd) return make_uint4(w[0], w[1], w[2], w[3]);
        w[4] = __ldg(words + 4);
        return make_uint4(__byte_perm(w[0], w[1], 0x5432), __byte_perm(w[1], w[2], 0x5432),
                          __byte_perm(w[2], w[3], 0x5432), __byte_perm(w[3], w[4], 0x5432));
    }
    uint32_t e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = j < left ? __ldg(at + j) : 0u;
    return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
}
__global__ void __launch_bounds__(256) copy_rows_kernel(const Copies c) {
    constexpr int U = 4;
    const int lane = threadIdx.x & 31;
    // consecutive units a warp: one division, then steps
    const int64_t per = ceil_div(c.units, (int64_t)gridDim.x * 8);
    int64_t u = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * per;
    const int64_t end = min64(c.units, u + per);
#pragma unroll
    for (int n = 0; n < 3; ++n) {
        const Copies::One& o = c.one[n];
        const int64_t last = min64(end, o.first + o.rows * o.chunks);
        if (u >= last) continue;
        int64_t row = (u - o.first) / o.chunks, chunk = (u - o.first) - row * o.chunks;
        while (u < last) {
            uint4 v[U];
            uint4* to[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                to[i] = nullptr;
                if (u >= last) continue;
                const int64_t group = chunk * 32 + lane, left = o.cols - group * 8;
                if (left > 0) {
                    v[i] = group_of(o.src + row * o.cols + group * 8, left,
                                    (row == 0 && group == 0) || (row == o.rows - 1 && left <= 8));
                    to[i] = o.dst + row * ceil_div(o.cols, 8) + group;
                }
                ++u;
                if (++chunk == o.chunks) {
                    chunk = 0;
                    ++row;
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i)
                if (to[i]) *to[i] = v[i];
        }
    }
}

// FLOAT: h = act(g) u; h may be u
__global__ void __launch_bounds__(256) product_kernel(const float* G, const float* U, float* H, int64_t n, int act) {
    by_activation(act, [&](auto which) {
        for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += (int64_t)gridDim.x * 256)
            H[e] = gate_value<true, which.value>(G[e]) * U[e];
    });
}

// ---- host side ---------------------------------------------------------------------

constexpr int64_t pad8(int64_t n) { return (n + 7) / 8 * 8; }
constexpr size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// K slices of a product whose units fill `slots` (CTA pairs, or SMs) at most
// half: enough to fill them, each slice at least four K blocks, if a unit is
// spared more than the pass that joins the slices takes, about 12 K blocks
// (BF16, us: [65, 1024] x [1024, 2816] 8.6 whole, 9.2 in three slices; [128,
// 4096] x [4096, 1024] 22.2 whole, 10.7 in nine).
int slices_of(int64_t tiles, int64_t k_total, int64_t slots) {
    if (tiles <= 0 || 2 * tiles > slots) return 1;
    const int64_t want = min64(slots / tiles, k_total / 4);
    if (want < 2 || k_total - ceil_div(k_total, want) < 12) return 1;
    return (int)ceil_div(k_total, ceil_div(k_total, want));    // no empty slice
}

// How a product is cut: on CTA pairs or (FWD) single CTAs, into how many tiles
// and K slices.
struct Cut {
    bool single;
    int64_t tiles_m, tiles_n;
    int splits;
};
Cut cut_of(int mode, int64_t M, int64_t N, int64_t K, int sm_count) {
    const int64_t kb = ceil_div(K, BK), pairs = sm_count / 2;
    const int64_t k_total = kb * (mode == DX ? 2 : 1);
    Cut c{false, ceil_div(M, 256), ceil_div(N, mode == FWD ? 128 : 256), 1};
    c.splits = slices_of(c.tiles_m * c.tiles_n * (mode == DW ? 2 : 1), k_total, pairs);
    if (mode == FWD) {
        // A K block of a unit takes about 550 cycles on both: the pair's MMAs,
        // or a single CTA's operands on their way into and out of shared
        // memory (twice its MMAs' time).  What surrounds a unit's K blocks
        // takes some 5500 cycles more on a pair.  So single CTAs take what
        // fits them in no more rounds (us: [333, 4000] x [4000, 2736] FP16
        // 22.8 against 25.7; BF16 [512, 1024] x [1024, 4096] 14.4 against
        // 12.8, [2048, 1024] x [1024, 4096] 40.3 against 30.0, [256, 4096] x
        // [4096, 14336] 60.6 against 52.7).
        Cut one{true, ceil_div(M, 128), ceil_div(N, single::COLS), 1};
        one.splits = slices_of(one.tiles_m * one.tiles_n, k_total, sm_count);
        auto cycles = [&](const Cut& x, int64_t slots) {
            return ceil_div(x.tiles_m * x.tiles_n * x.splits, slots) * ceil_div(k_total, x.splits) * 550;
        };
        if (cycles(one, sm_count) < cycles(c, pairs) + 5500) return one;
    }
    return c;
}
size_t product_partial_bytes(int mode, int64_t M, int64_t N, int64_t K, int sm_count) {
    const int s = cut_of(mode, M, N, K, sm_count).splits;
    return s > 1 ? (size_t)s * (mode == DX ? 1 : 2) * (size_t)M * (size_t)pad8(N) * sizeof(float) : 0;
}

template <int MODE>
cudaError_t launch_product(olc_dtype dt, const Product& w, float* partial, int sm_count, cudaStream_t s) {
    const int bf = dt == OLC_BFLOAT16;
    const Cut cut = cut_of(MODE, w.M, w.N, w.K, sm_count);
    // rows of a box of a K-major operand B
    const uint32_t b_rows = cut.single ? single::COLS : 128;
    Maps maps;
    std::memset(&maps, 0, sizeof maps);
    bool blocks = !w.b_k && !cut.single;
    for (int i = 0; i < 2 && blocks; ++i)
        blocks = w.N % 64 == 0 && encode_b_blocks(&maps.b[i], w.b[i].base, bf, w.N, w.K, 1, w.b[i].pitch);
    for (int i = 0; i < 2; ++i) {
        const Stored &a = w.a[i], &b = w.b[i];
        const bool ok_a = w.a_mn ? encode_3d(&maps.a[i], a.base, bf, a.cols, a.rows, 1, 64, BK,
                                             CU_TENSOR_MAP_SWIZZLE_128B, a.pitch)
                                 : encode_3d(&maps.a[i], a.base, bf, a.cols, a.rows, 1, BK, 128,
                                             CU_TENSOR_MAP_SWIZZLE_128B, a.pitch);
        const bool ok_b = blocks || (w.b_k ? encode_3d(&maps.b[i], b.base, bf, b.cols, b.rows, 1, BK, b_rows,
                                                       CU_TENSOR_MAP_SWIZZLE_128B, b.pitch)
                                           : encode_3d(&maps.b[i], b.base, bf, b.cols, b.rows, 1, 64, BK,
                                                       CU_TENSOR_MAP_SWIZZLE_128B, b.pitch));
        if (!ok_a || !ok_b) return cudaErrorInvalidValue;
    }
    Params p;
    std::memset(&p, 0, sizeof p);
    p.M = w.M;
    p.N = w.N;
    p.tiles_m = cut.tiles_m;
    p.tiles_n = cut.tiles_n;
    p.items = MODE == DW ? 2 : 1;
    p.k_blocks = ceil_div(w.K, BK);
    p.k_total = p.k_blocks * (MODE == DX ? 2 : 1);
    p.splits = cut.splits;
    p.k_slice = ceil_div(p.k_total, p.splits);
    p.units = p.tiles_m * p.tiles_n * p.items * p.splits;
    p.a_mn = w.a_mn;
    p.b_k = w.b_k;
    p.b_blocks = blocks;
    p.is_bf16 = bf;
    p.act = w.act;
    p.aligned = w.N % 8 == 0;
    p.paired = w.N % 2 == 0;
    for (int i = 0; i < 3; ++i) {
        p.Y[i] = w.Y[i];
        if (w.Y[i] && !plan_aligned16(w.Y[i])) p.aligned = 0;
        if (w.Y[i] && plan_misaligned(w.Y[i], 4)) p.paired = 0;
    }
    p.partial = partial;
    p.partial_pitch = pad8(w.N);
    p.err = device_error_word();
    cudaError_t e;
    if (cut.single) {
        e = set_smem_limit(reinterpret_cast<const void*>(single_kernel), single::SMEM1);
        if (e == cudaSuccess)
            e = plan_launch(single_kernel, dim3((unsigned)min64(p.units, sm_count)), dim3(single::THREADS1),
                           (size_t)single::SMEM1, s, maps.a[0], maps.b[0], maps.b[1], p);
    } else {
        e = set_smem_limit(reinterpret_cast<const void*>(pair_kernel<MODE>), SMEM_BYTES);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(2 * min64(p.units, sm_count / 2)));
        cfg.blockDim = dim3(PAIR_THREADS);
        cfg.dynamicSmemBytes = SMEM_BYTES;
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, pair_kernel<MODE>, maps.a[0], maps.a[1], maps.b[0], maps.b[1], p);
    }
    if (e != cudaSuccess || p.splits == 1) return e;
    const int64_t work = p.M * ceil_div(p.N, 4) * p.items;
    const dim3 grid((unsigned)min64(ceil_div(work, 256), (int64_t)sm_count * 8));
    return bf ? plan_launch(join_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, p, (int)MODE)
              : plan_launch(join_kernel<__half>, grid, dim3(256), 0, s, p, (int)MODE);
}

template <typename T>
cudaError_t launch_slope(const void* dH, const void* G, const void* U, void* dG, void* dU, int64_t rows, int64_t cols,
                         int64_t pitch, int act, int sm_count, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);
    const bool wide = cols % V == 0 && plan_aligned16(dH) && plan_aligned16(G) && plan_aligned16(U);
    const dim3 grid((unsigned)min64(ceil_div(rows * (wide ? cols / V : cols), 256), (int64_t)sm_count * 16));
    auto run = [&](auto kernel) {
        return plan_launch(kernel, grid, dim3(256), 0, s, static_cast<const T*>(dH), static_cast<const T*>(G),
                           static_cast<const T*>(U), static_cast<T*>(dG), static_cast<T*>(dU), rows, cols, pitch, act);
    };
    return wide ? run(slope_kernel<T, V>) : run(slope_kernel<T, 1>);
}

}  // namespace gated
}  // namespace olc

using namespace olc;

struct olc_gated_plan {
    PlanState state;
    olc_dtype dtype;
    int64_t M, D, F;
    int act, trans_w;
    olc_matmul_plan* forward;    // FLOAT, few rows: X W
    unsigned int* counters;      // FLOAT: arrivals at shared tiles, in the memory's first block
    int reserved;
};

namespace {

// FLOAT, few rows and weights [D, F]: the matrix plan's row kernels stream
// each weight once, where a 64-row tile would multiply mostly nothing (us of
// [rows, 1024] x [1024, 2816], device: 4 rows 15.8 against 30, 8 rows 31.7
// against 30, 16 rows 90 against 30).
constexpr int64_t kFewFloatRows = 4;
bool few_float(const olc_gated_plan* p) { return p->M <= kFewFloatRows && !p->trans_w; }

// The start of a FLOAT plan's memory holds the counters of its first block.
size_t counter_room(const olc_gated_plan* p) {
    return p->dtype == OLC_FLOAT ? gated::round256(gated::float_counter_bytes(p->state.sm_count)) : 0;
}
// of the plan's memory, what follows them
unsigned char* memory_of(const olc_gated_plan* p) {
    return p->state.memory ? static_cast<unsigned char*>(p->state.memory) + counter_room(p) : nullptr;
}
olc_status ensure(olc_gated_plan* p, size_t bytes) {
    return bytes ? p->state.ensure(counter_room(p) + bytes) : OLC_OK;
}

// What every forward call needs, made with the plan (where no device was visible
// then, at the first call): K slices or partial sums, and FLOAT's counters, zero
// before any stream goes on.  They are cleared on a stream of their own: the
// legacy stream would wait for every other one, and break a capture that one of
// them is in.  What depends on the operands' alignment, and what the gradient
// needs, comes with the first call that needs it: a plan may never see one.
olc_status reserve(olc_gated_plan* p) {
    if (p->reserved) return OLC_OK;
    const int sms = p->state.sm_count;
    size_t bytes = 0;
    olc_status st = OLC_OK;
    if (p->dtype != OLC_FLOAT) {
        if (!gated::takes_few(p->M, p->F, sms)) bytes = gated::product_partial_bytes(gated::FWD, p->M, p->F, p->D, sms);
        if (bytes) st = p->state.ensure(bytes);
    } else {
        if (few_float(p)) {
            bytes = (size_t)(p->M * p->F) * sizeof(float);
            const int64_t x[2] = {p->M, p->D}, w[2] = {p->D, p->F};
            if (!p->forward) st = olc_matmul_plan_create(x, 2, w, 2, OLC_FLOAT, &p->forward);
        } else {
            bytes = gated::float_sum_bytes(gated::FWD, p->M, p->F, p->D, sms);
        }
        if (st == OLC_OK) st = p->state.ensure(counter_room(p) + bytes);
        if (st == OLC_OK) {
            cudaStream_t own;
            cudaError_t e = cudaStreamCreateWithFlags(&own, cudaStreamNonBlocking);
            if (e == cudaSuccess) {
                e = cudaMemsetAsync(p->state.memory, 0, counter_room(p), own);
                if (e == cudaSuccess) e = cudaStreamSynchronize(own);
                cudaStreamDestroy(own);
            }
            st = plan_status(e);
        }
        if (st == OLC_OK) p->counters = static_cast<unsigned int*>(p->state.memory);
    }
    if (st == OLC_OK) p->reserved = 1;
    return st;
}

// One call's use of the plan's memory: pieces are taken in order, first to
// size it, then to hand out addresses.
struct Pieces {
    size_t used = 0;
    unsigned char* base = nullptr;
    void* take(size_t bytes) {
        void* at = base ? base + used : nullptr;
        used += gated::round256(bytes);
        return at;
    }
};

// An operand as the TMA reads it: in place, or a copy with rows padded to 16
// bytes in the plan's memory.
struct Operand {
    const void* src;
    int64_t rows, cols;
    bool copy;
    void* dst;
    Operand(const void* p, int64_t r, int64_t c) : src(p), rows(r), cols(c), copy(!plan_aligned16(p) || c % 8 != 0), dst(nullptr) {}
    void place(Pieces& m) {
        if (copy) dst = m.take((size_t)(rows * gated::pad8(cols)) * 2);
    }
    gated::Stored stored() const {
        return copy ? gated::Stored{dst, rows, cols, gated::pad8(cols)} : gated::Stored{src, rows, cols, cols};
    }
};
// the copies of those that need one
cudaError_t fill(std::initializer_list<const Operand*> operands, int sm_count, cudaStream_t s) {
    gated::Copies c;
    std::memset(&c, 0, sizeof c);
    int n = 0;
    for (const Operand* o : operands) {
        if (!o->copy || o->rows == 0 || o->cols == 0) continue;
        c.one[n++] = gated::Copies::One{static_cast<const unsigned short*>(o->src), static_cast<uint4*>(o->dst),
                                        o->rows, o->cols, ceil_div(o->cols, 256), c.units};
        c.units += o->rows * ceil_div(o->cols, 256);
    }
    if (n == 0) return cudaSuccess;
    return plan_launch(gated::copy_rows_kernel, dim3((unsigned)min64(ceil_div(c.units, 8), (int64_t)sm_count * 8)),
                       dim3(256), 0, s, c);
}

olc_status forward16(olc_gated_plan* p, const void* X, const void* Wg, const void* Wu, void* H, void* G, void* U,
                     cudaStream_t s) {
    const int64_t wr = p->trans_w ? p->F : p->D, wc = p->trans_w ? p->D : p->F;
    Operand x(X, p->M, p->D), wg(Wg, wr, wc), wu(Wu, wr, wc);
    const bool few = gated::takes_few(p->M, p->F, p->state.sm_count);
    const size_t partial = few ? 0 : gated::product_partial_bytes(gated::FWD, p->M, p->F, p->D, p->state.sm_count);
    float* part = nullptr;
    for (int pass = 0; pass < 2; ++pass) {
        Pieces m;
        m.base = pass ? static_cast<unsigned char*>(p->state.memory) : nullptr;
        x.place(m);
        wg.place(m);
        wu.place(m);
        part = static_cast<float*>(m.take(partial));
        if (pass == 0) {
            if (m.used == 0) break;
            const olc_status st = p->state.ensure(m.used);
            if (st != OLC_OK) return st;
        }
    }
    const bool uses = x.copy || wg.copy || wu.copy || partial;
    gated::Product w;
    std::memset(&w, 0, sizeof w);
    w.M = p->M;
    w.N = p->F;
    w.K = p->D;
    w.a[0] = w.a[1] = x.stored();
    w.b[0] = wg.stored();
    w.b[1] = wu.stored();
    w.b_k = p->trans_w;
    w.Y[0] = H;
    w.Y[1] = G;
    w.Y[2] = U;
    w.act = p->act;
    auto run = [&] {
        const cudaError_t e = fill({&x, &wg, &wu}, p->state.sm_count, s);
        if (e != cudaSuccess) return e;
        return few ? gated::launch_few(p->dtype, w, p->state.sm_count, s)
                   : gated::launch_product<gated::FWD>(p->dtype, w, part, p->state.sm_count, s);
    };
    return plan_status(uses ? p->state.use(s, run) : run());
}

olc_status backward16(olc_gated_plan* p, const void* dH, const void* X, const void* Wg, const void* Wu, const void* G,
                      const void* U, void* dX, void* dWg, void* dWu, cudaStream_t s) {
    const int64_t wr = p->trans_w ? p->F : p->D, wc = p->trans_w ? p->D : p->F;
    const int64_t pitch = gated::pad8(p->F);
    const int sms = p->state.sm_count;
    Operand x(X, p->M, p->D), wg(Wg, wr, wc), wu(Wu, wr, wc);
    const int64_t wm = p->trans_w ? p->F : p->D, wn = p->trans_w ? p->D : p->F;
    size_t partial = dX ? gated::product_partial_bytes(gated::DX, p->M, p->D, p->F, sms) : 0;
    const size_t pw = dWg ? gated::product_partial_bytes(gated::DW, wm, wn, p->M, sms) : 0;
    if (pw > partial) partial = pw;
    void *dg = nullptr, *du = nullptr;
    float* part = nullptr;
    for (int pass = 0; pass < 2; ++pass) {
        Pieces m;
        m.base = pass ? static_cast<unsigned char*>(p->state.memory) : nullptr;
        dg = m.take((size_t)(p->M * pitch) * 2);
        du = m.take((size_t)(p->M * pitch) * 2);
        if (dWg) x.place(m);
        if (dX) {
            wg.place(m);
            wu.place(m);
        }
        part = static_cast<float*>(m.take(partial));
        if (pass == 0) {
            const olc_status st = p->state.ensure(m.used);
            if (st != OLC_OK) return st;
        }
    }
    return plan_status(p->state.use(s, [&] {
        cudaError_t e = p->dtype == OLC_BFLOAT16
                            ? gated::launch_slope<__nv_bfloat16>(dH, G, U, dg, du, p->M, p->F, pitch, p->act, sms, s)
                            : gated::launch_slope<__half>(dH, G, U, dg, du, p->M, p->F, pitch, p->act, sms, s);
        const gated::Stored sg{dg, p->M, p->F, pitch}, su{du, p->M, p->F, pitch};
        gated::Product w;
        if (dX && e == cudaSuccess) {
            e = fill({&wg, &wu}, sms, s);
            std::memset(&w, 0, sizeof w);
            w.M = p->M;
            w.N = p->D;
            w.K = p->F;
            w.a[0] = sg;
            w.a[1] = su;
            w.b[0] = wg.stored();
            w.b[1] = wu.stored();
            w.b_k = !p->trans_w;
            w.Y[0] = dX;
            if (e == cudaSuccess) e = gated::launch_product<gated::DX>(p->dtype, w, part, sms, s);
        }
        if (dWg && e == cudaSuccess) {
            e = fill({&x}, sms, s);
            std::memset(&w, 0, sizeof w);
            w.M = wm;
            w.N = wn;
            w.K = p->M;
            const gated::Stored sx = x.stored();
            w.a[0] = p->trans_w ? sg : sx;
            w.a[1] = p->trans_w ? su : sx;
            w.b[0] = p->trans_w ? sx : sg;
            w.b[1] = p->trans_w ? sx : su;
            w.a_mn = true;
            w.Y[0] = dWg;
            w.Y[1] = dWu;
            if (e == cudaSuccess) e = gated::launch_product<gated::DW>(p->dtype, w, part, sms, s);
        }
        return e;
    }));
}

olc_status forward32_few(olc_gated_plan* p, const void* X, const void* Wg, const void* Wu, void* H, void* G, void* U,
                         cudaStream_t s) {
    olc_status st = OLC_OK;
    const int64_t n = p->M * p->F;
    // what is not kept: g in the plan's memory, u in H
    void* g = G ? G : memory_of(p);
    void* u = U ? U : H;
    auto run = [&] {
        st = olc_matmul_execute(p->forward, X, Wg, g, s);
        if (st == OLC_OK) st = olc_matmul_execute(p->forward, X, Wu, u, s);
        if (st != OLC_OK) return cudaSuccess;
        return plan_launch(gated::product_kernel,
                           dim3((unsigned)min64(ceil_div(n, 256), (int64_t)p->state.sm_count * 16)), dim3(256), 0, s,
                           static_cast<const float*>(g), static_cast<const float*>(u), static_cast<float*>(H), n, p->act);
    };
    const olc_status ran = plan_status(G ? run() : p->state.use(s, run));
    return st != OLC_OK ? st : ran;
}

olc_status forward32(olc_gated_plan* p, const void* X, const void* Wg, const void* Wu, void* H, void* G, void* U,
                     cudaStream_t s) {
    if (few_float(p)) return forward32_few(p, X, Wg, Wu, H, G, U, s);
    const int sms = p->state.sm_count;
    gated::Product w;
    std::memset(&w, 0, sizeof w);
    w.mode = gated::FWD;
    w.M = p->M;
    w.N = p->F;
    w.K = p->D;
    const int64_t wr = p->trans_w ? p->F : p->D, wc = p->trans_w ? p->D : p->F;
    w.a[0] = w.a[1] = gated::Stored{X, p->M, p->D, p->D};
    w.b[0] = gated::Stored{Wg, wr, wc, wc};
    w.b[1] = gated::Stored{Wu, wr, wc, wc};
    w.b_k = p->trans_w;
    w.Y[0] = H;
    w.Y[1] = G;
    w.Y[2] = U;
    w.act = p->act;
    return plan_status(p->state.use(s, [&] {         // the counters, if nothing else
        return gated::launch_float(w, memory_of(p), p->counters, sms, s);
    }));
}

olc_status backward32(olc_gated_plan* p, const void* dH, const void* X, const void* Wg, const void* Wu, const void* G,
                      const void* U, void* dX, void* dWg, void* dWu, cudaStream_t s) {
    const int sms = p->state.sm_count;
    const int64_t wr = p->trans_w ? p->F : p->D, wc = p->trans_w ? p->D : p->F;
    const int64_t pitch = (p->F + 3) / 4 * 4;      // of dg and du: rows on 16-byte boundaries
    size_t sums = dX ? gated::float_sum_bytes(gated::DX, p->M, p->D, p->F, sms) : 0;
    const size_t more = dWg ? gated::float_sum_bytes(gated::DW, wr, wc, p->M, sms) : 0;
    if (more > sums) sums = more;
    const size_t half = gated::round256((size_t)(p->M * pitch) * sizeof(float));
    const olc_status st = ensure(p, 2 * half + sums);
    if (st != OLC_OK) return st;
    unsigned char* memory = memory_of(p);
    void *dg = memory, *du = memory + half, *part = memory + 2 * half;
    unsigned int* counters = p->counters;
    const gated::Stored sg{dg, p->M, p->F, pitch}, su{du, p->M, p->F, pitch}, sx{X, p->M, p->D, p->D};
    return plan_status(p->state.use(s, [&] {
        cudaError_t e = gated::launch_slope<float>(dH, G, U, dg, du, p->M, p->F, pitch, p->act, sms, s);
        gated::Product w;
        if (dX && e == cudaSuccess) {
            std::memset(&w, 0, sizeof w);
            w.mode = gated::DX;
            w.M = p->M;
            w.N = p->D;
            w.K = p->F;
            w.a[0] = sg;
            w.a[1] = su;
            w.b[0] = gated::Stored{Wg, wr, wc, wc};
            w.b[1] = gated::Stored{Wu, wr, wc, wc};
            w.b_k = !p->trans_w;
            w.Y[0] = dX;
            e = gated::launch_float(w, part, counters, sms, s);
        }
        if (dWg && e == cudaSuccess) {
            std::memset(&w, 0, sizeof w);
            w.mode = gated::DW;
            w.M = wr;
            w.N = wc;
            w.K = p->M;
            w.a[0] = p->trans_w ? sg : sx;
            w.a[1] = p->trans_w ? su : sx;
            w.b[0] = p->trans_w ? sx : sg;
            w.b[1] = p->trans_w ? sx : su;
            w.a_mn = true;
            w.Y[0] = dWg;
            w.Y[1] = dWu;
            e = gated::launch_float(w, part, counters, sms, s);
        }
        return e;
    }));
}

}  // namespace

extern "C" {

olc_status olc_gated_plan_create(int64_t rows, int64_t d_in, int64_t d_hidden, int activation, int trans_w,
                                 olc_dtype dtype, olc_gated_plan** out) {
    if (!out) return OLC_ERR_NULL;
    *out = nullptr;
    if (!plan_dtype_ok(dtype)) return OLC_ERR_DTYPE;
    if (rows < 0 || d_in < 0 || d_hidden < 0) return OLC_ERR_NEGATIVE_DIM;
    const int64_t most = (int64_t(1) << 31) - 65536;       // 32-bit tile coordinates
    if (rows >= most || d_in >= most || d_hidden >= most) return OLC_ERR_INVALID;
    if (activation < OLC_GATE_SILU || activation > OLC_GATE_SIGMOID) return OLC_ERR_INVALID;
    if (!plan_fits(rows, d_in, 4) || !plan_fits(rows, d_hidden, 4) || !plan_fits(d_in, d_hidden, 4))
        return OLC_ERR_INVALID;
    olc_gated_plan* p = new (std::nothrow) olc_gated_plan;
    if (!p) return OLC_ERR_OOM;
    std::memset(static_cast<void*>(p), 0, sizeof *p);
    p->state.init();
    p->dtype = dtype;
    p->M = rows;
    p->D = d_in;
    p->F = d_hidden;
    p->act = activation;
    p->trans_w = trans_w ? 1 : 0;
    if (p->state.device >= 0 && rows > 0 && d_in > 0 && d_hidden > 0) {
        const olc_status st = reserve(p);
        if (st != OLC_OK) {
            olc_gated_plan_destroy(p);
            return st;
        }
    }
    *out = p;
    return OLC_OK;
}

void olc_gated_plan_destroy(olc_gated_plan* plan) {
    if (!plan) return;
    olc_matmul_plan_destroy(plan->forward);
    plan->state.destroy();
    delete plan;
}

olc_status olc_gated_forward(olc_gated_plan* plan, const void* X, const void* Wg, const void* Wu, void* H, void* G,
                             void* U, void* stream) {
    if (!plan) return OLC_ERR_NULL;
    olc_gated_plan* p = plan;
    if (p->M == 0 || p->F == 0) return OLC_OK;
    if (!H || (p->D > 0 && (!X || !Wg || !Wu))) return OLC_ERR_NULL;
    const int64_t eb = plan_elem_bytes(p->dtype);
    for (const void* q : {X, Wg, Wu, (const void*)H, (const void*)G, (const void*)U})
        if (plan_misaligned(q, eb)) return OLC_ERR_INVALID;
    const olc_status st = p->state.bind();
    if (st != OLC_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p->D == 0) {                                       // empty sums: act(0) 0
        cudaError_t e = cudaSuccess;
        for (void* y : {H, G, U})
            if (y && e == cudaSuccess) e = launch_zero_fill(y, p->M * p->F * eb, s);
        return plan_status(e);
    }
    const olc_status ready = reserve(p);
    if (ready != OLC_OK) return ready;
    return p->dtype == OLC_FLOAT ? forward32(p, X, Wg, Wu, H, G, U, s) : forward16(p, X, Wg, Wu, H, G, U, s);
}

olc_status olc_gated_backward(olc_gated_plan* plan, const void* dH, const void* X, const void* Wg, const void* Wu,
                              const void* G, const void* U, void* dX, void* dWg, void* dWu, void* stream) {
    if (!plan) return OLC_ERR_NULL;
    olc_gated_plan* p = plan;
    if ((dWg == nullptr) != (dWu == nullptr)) return OLC_ERR_NULL;
    if (p->M == 0 || p->D == 0) dX = nullptr;              // empty
    if (p->D == 0 || p->F == 0) dWg = dWu = nullptr;
    if (!dX && !dWg) return OLC_OK;
    const int64_t eb = plan_elem_bytes(p->dtype);
    const bool some = p->M > 0 && p->F > 0;                // terms to sum
    if (some && (!dH || !G || !U || (dX && (!Wg || !Wu)) || (dWg && !X))) return OLC_ERR_NULL;
    for (const void* q : {dH, X, Wg, Wu, G, U, (const void*)dX, (const void*)dWg, (const void*)dWu})
        if (plan_misaligned(q, eb)) return OLC_ERR_INVALID;
    const olc_status st = p->state.bind();
    if (st != OLC_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!some) {
        cudaError_t e = dX ? launch_zero_fill(dX, p->M * p->D * eb, s) : cudaSuccess;
        if (dWg && e == cudaSuccess) e = launch_zero_fill(dWg, p->D * p->F * eb, s);
        if (dWg && e == cudaSuccess) e = launch_zero_fill(dWu, p->D * p->F * eb, s);
        return plan_status(e);
    }
    const olc_status ready = reserve(p);
    if (ready != OLC_OK) return ready;
    return p->dtype == OLC_FLOAT ? backward32(p, dH, X, Wg, Wu, G, U, dX, dWg, dWu, s)
                                 : backward16(p, dH, X, Wg, Wu, G, U, dX, dWg, dWu, s);
}

}  // extern "C"
