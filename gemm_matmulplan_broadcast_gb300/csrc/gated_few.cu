// The gated feed-forward product for few rows (up to 64): act(X Wg) (X Wu)
// with both weights streamed once.
//
// 4 D F bytes of weights against 4 M D F operations: the weights' bytes bound
// it, so everything serves one steady stream of them.  A CTA takes 64 columns
// of both weights and a slice of K; the slices of one column tile are the CTAs
// of a cluster.  A loading warp brings 64 x 64 blocks of Wg and Wu and the
// rows' 64 K elements through a TMA ring (about 200 KB on their way per SM);
// four warps read 16 columns each with ldmatrix (transposed where the weights
// are stored [D, F]) as the A operand of mma.sync m16n8k16, the rows being the
// N dimension: the products cost a few percent of the time the bytes take.  The
// slices' float32 sums meet through distributed shared memory in slice order,
// each CTA finishing a share of the tile: activation, product, one rounding.
// Measured: [1, 4096] x [4096, 14336] BF16 39.5 us, 5.9 TB/s (the tile kernels:
// 63), 64 rows 43 (47); [1, 1024] x [1024, 2816] 6.0 (8.2).
#include <cstring>

#include "gated_internal.h"
#include "tc_ptx.cuh"

namespace olc {
namespace gated {

using namespace olc::tc;

namespace few {

constexpr int TILE = 64;                          // hidden columns of a CTA
constexpr int WARPS = 4;
constexpr int THREADS = (WARPS + 1) * 32;         // + the loading warp
constexpr int W_BYTES = BK * TILE * 2;            // one weight's block: 8 KiB
constexpr int MAX_CLUSTER = 8;
constexpr int PER_SM = 3;                         // CTAs whose rings fit an SM

template <int NT>
struct Cfg {
    static constexpr int ROWS = 8 * NT;           // rows of X a CTA holds
    static constexpr int X_BYTES = ROWS * BK * 2;
    static constexpr int STAGE_BYTES = 2 * W_BYTES + X_BYTES;
    static constexpr int STAGES = NT <= 2 ? 4 : 3;
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 1024;
    static_assert(2 * TILE * ROWS * 4 <= STAGES * STAGE_BYTES, "the partial sums fit the ring");
};

struct Bars {
    uint64_t full[4];
    uint64_t empty[4];
    int abort_flag;
};

struct Params {
    int64_t M, F;
    int64_t k_blocks;
    int trans_w, act;
    int quads;                // outputs stored four at a time (8-byte boundaries)
    int cluster;
    void *H, *G, *U;
    unsigned int* err;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr, bool trans) {
    if (trans)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(addr)
                     : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(addr)
                     : "memory");
}
__device__ __forceinline__ void ldsm2(uint32_t (&r)[2], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];"
                 : "=r"(r[0]), "=r"(r[1])
                 : "r"(addr)
                 : "memory");
}
template <bool BF16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float4 ld_remote(const float* local, int rank) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(local)), "r"(rank));
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}

template <typename T>
__device__ __forceinline__ void put4(T* y, const float (&v)[4], int64_t n, bool quads) {
    T o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = Num<T>::from_acc(v[i]);
    if (quads) {
        *reinterpret_cast<uint2*>(y) = *reinterpret_cast<const uint2*>(o);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < n) y[i] = o[i];
}

template <int NT, bool BF16>
__global__ void __launch_bounds__(THREADS, PER_SM)
kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_g,
       const __grid_constant__ CUtensorMap map_u, const Params p) {
    using C = Cfg<NT>;
    using T = std::conditional_t<BF16, __nv_bfloat16, __half>;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ Bars s;
    unsigned char* base =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    volatile int* abort_flag = &s.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cl = p.cluster;
    const int64_t tile = blockIdx.x / cl;
    const int rank = (int)(blockIdx.x % cl);
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], WARPS);
        }
        s.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();
    const int64_t kb0 = p.k_blocks * rank / cl, kb1 = p.k_blocks * (rank + 1) / cl;
    const uint32_t ring = smem_u32(base);
    float acc[2][NT][4];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;

    if (warp == WARPS) {
        if (lane == 0) {
            uint32_t stage = 0, phase = 0, armed = 0, parity = 0;
            const int f0 = (int)tile * TILE;
            for (int64_t kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait(&s.empty[stage], phase ^ 1, abort_flag, p.err)) break;
                mbar_arrive_expect_tx(&s.full[stage], C::STAGE_BYTES);
                armed |= 1u << stage;
                parity = (parity & ~(1u << stage)) | (phase << stage);
                const uint32_t at = ring + stage * C::STAGE_BYTES, bar = smem_u32(&s.full[stage]);
                const int k0 = (int)kb * BK;
                tma_load_3d(at, &map_g, bar, p.trans_w ? k0 : f0, p.trans_w ? f0 : k0, 0);
                tma_load_3d(at + W_BYTES, &map_u, bar, p.trans_w ? k0 : f0, p.trans_w ? f0 : k0, 0);
                tma_load_3d(at + 2 * W_BYTES, &map_x, bar, k0, 0, 0);
                if (++stage == C::STAGES) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            if (*abort_flag)
                for (int i = 0; i < C::STAGES; ++i)
                    if ((armed >> i) & 1u) mbar_wait_drain(&s.full[i], (parity >> i) & 1u);
        }
        __syncwarp();
    } else {
        // this lane's row of the four 8 x 8 matrices ldmatrix takes
        const int q = lane >> 3, r = lane & 7;
        uint32_t stage = 0, phase = 0;
        for (int64_t kb = kb0; kb < kb1; ++kb) {
            const bool ok = mbar_wait(&s.full[stage], phase, abort_flag, p.err);
            if (!__all_sync(0xffffffffu, ok)) break;      // the warp stays together for ldmatrix and mma
            const uint32_t wg = ring + stage * C::STAGE_BYTES, xb = wg + 2 * W_BYTES;
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk) {
                uint32_t off;
                if (p.trans_w) {              // block [f][k]
                    const int f = warp * 16 + (q & 1) * 8 + r;
                    off = f * 128 + (((kk * 2 + (q >> 1)) ^ (f & 7)) << 4);
                } else {                      // block [k][f]: transposed on the way
                    const int k = kk * 16 + (q >> 1) * 8 + r;
                    off = k * 128 + (((warp * 2 + (q & 1)) ^ (k & 7)) << 4);
                }
                uint32_t ag[4], au[4];
                ldsm4(ag, wg + off, !p.trans_w);
                ldsm4(au, wg + W_BYTES + off, !p.trans_w);
                if constexpr (NT == 1) {
                    uint32_t b[2];
                    ldsm2(b, xb + r * 128 + (((kk * 2 + (q & 1)) ^ r) << 4));
                    mma<BF16>(acc[0][0], ag, b[0], b[1]);
                    mma<BF16>(acc[1][0], au, b[0], b[1]);
                } else {
#pragma unroll
                    for (int n = 0; n < NT; n += 2) {
                        uint32_t b[4];
                        const int row = n * 8 + (q >> 1) * 8 + r;
                        ldsm4(b, xb + row * 128 + (((kk * 2 + (q & 1)) ^ r) << 4), false);
                        mma<BF16>(acc[0][n], ag, b[0], b[1]);
                        mma<BF16>(acc[0][n + 1], ag, b[2], b[3]);
                        mma<BF16>(acc[1][n], au, b[0], b[1]);
                        mma<BF16>(acc[1][n + 1], au, b[2], b[3]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.empty[stage]);
            if (++stage == C::STAGES) {
                stage = 0;
                phase ^= 1;
            }
        }
    }
    // this slice's sums: [matrix][row][64 columns] in the ring, which no warp
    // reads any more.  Every barrier from here on is met by whole warps at one
    // place for all roles.
    __syncthreads();
    float* part = reinterpret_cast<float*>(base);
    if (warp < WARPS) {
        const int f = warp * 16 + (lane >> 2), row = (lane & 3) * 2;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float* at = part + (m * C::ROWS + n * 8 + row) * TILE + f;
                at[0] = acc[m][n][0];
                at[TILE] = acc[m][n][1];
                at[8] = acc[m][n][2];
                at[TILE + 8] = acc[m][n][3];
            }
    }
    __syncthreads();
    if (cl > 1) pair::cluster_sync();
    // each CTA finishes its share of the tile's groups of four columns
    constexpr int GROUPS = C::ROWS * TILE / 4;
    const int g0 = GROUPS * rank / cl, g1 = GROUPS * (rank + 1) / cl;
    for (int g = g0 + (int)threadIdx.x; g < g1; g += THREADS) {
        const int row = g / (TILE / 4);
        const int64_t col = tile * TILE + g % (TILE / 4) * 4;
        if (row >= p.M || col >= p.F) continue;
        float v[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const float* at = part + m * C::ROWS * TILE + g * 4;
            float4 x = cl > 1 ? ld_remote(at, 0) : *reinterpret_cast<const float4*>(at);
#pragma unroll
            for (int r = 1; r < MAX_CLUSTER; ++r) {
                if (r >= cl) break;
                const float4 y = ld_remote(at, r);
                x.x += y.x;
                x.y += y.y;
                x.z += y.z;
                x.w += y.w;
            }
            v[m][0] = x.x;
            v[m][1] = x.y;
            v[m][2] = x.z;
            v[m][3] = x.w;
        }
        float h[4];
        by_activation(p.act, [&](auto act) {
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = gate_value<false, act.value>(v[0][i]) * v[1][i];
        });
        const int64_t at = row * p.F + col;
        put4(static_cast<T*>(p.H) + at, h, p.F - col, p.quads);
        if (p.G) put4(static_cast<T*>(p.G) + at, v[0], p.F - col, p.quads);
        if (p.U) put4(static_cast<T*>(p.U) + at, v[1], p.F - col, p.quads);
    }
    __syncthreads();
    if (cl > 1) pair::cluster_sync();          // no CTA leaves while its sums are read
}

// CTAs on one column tile: the most slices (two K blocks each at least) whose
// CTAs all reside at once
int cluster_of(int64_t tiles, int64_t k_blocks, int sm_count) {
    int c = MAX_CLUSTER;
    while (c > 1 && (tiles * c > (int64_t)PER_SM * sm_count || k_blocks < 2 * c)) c /= 2;
    return c;
}

template <int NT, bool BF16>
cudaError_t launch_as(const Product& w, int sm_count, cudaStream_t s) {
    using C = Cfg<NT>;
    CUtensorMap mx, mg, mu;
    std::memset(&mx, 0, sizeof mx);
    std::memset(&mg, 0, sizeof mg);
    std::memset(&mu, 0, sizeof mu);
    auto weight = [&](CUtensorMap* m, const Stored& b) {
        return encode_3d(m, b.base, BF16, b.cols, b.rows, 1, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B, b.pitch);
    };
    if (!encode_3d(&mx, w.a[0].base, BF16, w.a[0].cols, w.a[0].rows, 1, BK, C::ROWS, CU_TENSOR_MAP_SWIZZLE_128B,
                   w.a[0].pitch) ||
        !weight(&mg, w.b[0]) || !weight(&mu, w.b[1]))
        return cudaErrorInvalidValue;
    Params p;
    std::memset(&p, 0, sizeof p);
    p.M = w.M;
    p.F = w.N;
    p.k_blocks = ceil_div(w.K, BK);
    p.trans_w = w.b_k;
    p.act = w.act;
    p.H = w.Y[0];
    p.G = w.Y[1];
    p.U = w.Y[2];
    p.quads = w.N % 4 == 0;
    for (int i = 0; i < 3; ++i)
        if (reinterpret_cast<uintptr_t>(w.Y[i]) & 7) p.quads = 0;
    const int64_t tiles = ceil_div(w.N, TILE);
    p.cluster = cluster_of(tiles, p.k_blocks, sm_count);
    p.err = device_error_word();
    auto* k = kernel<NT, BF16>;
    const cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(k), C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * p.cluster));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k, mx, mg, mu, p);
}

}  // namespace few

cudaError_t launch_few(olc_dtype dt, const Product& w, int sm_count, cudaStream_t s) {
    const bool bf = dt == OLC_BFLOAT16;
    if (w.M <= 8) return bf ? few::launch_as<1, true>(w, sm_count, s) : few::launch_as<1, false>(w, sm_count, s);
    if (w.M <= 16) return bf ? few::launch_as<2, true>(w, sm_count, s) : few::launch_as<2, false>(w, sm_count, s);
    if (w.M <= 32) return bf ? few::launch_as<4, true>(w, sm_count, s) : few::launch_as<4, false>(w, sm_count, s);
    return bf ? few::launch_as<8, true>(w, sm_count, s) : few::launch_as<8, false>(w, sm_count, s);
}

}  // namespace gated
}  // namespace olc
