// Layer norm over the last axis of [rows, cols], forward and backward.
//
//   mean = sum_j x_j / n,  rstd = 1 / sqrt(sum_j (x_j - mean)^2 / n + eps)
//   y_j  = (x_j - mean) rstd gamma_j + beta_j
//
//   with xh = (x - mean) rstd and dxh = dy gamma:
//   dx_j = rstd (dxh_j - mean_j(dxh) - xh_j mean_j(dxh xh))
//   dgamma_j = sum_rows dy xh,  dbeta_j = sum_rows dy
//
// About ten operations an element against two or three elements moved: the
// bytes bound it.  Each row is read once and stays in registers, so that the
// variance is the sum of squared distances from the finished mean (no
// cancellation for rows far from zero); rows too long for the registers are
// read again, mostly from L2.  All sums and statistics are float32; y, dx,
// dgamma and dbeta are rounded to the element type once.
#include <new>

#include "common.cuh"
#include "plan_state.h"

namespace olc {
namespace norm {

struct FwdParams {
    const void* X;
    const void* gamma;      // may be null: 1
    const void* beta;       // may be null: 0
    void* Y;
    float* mean;            // may be null
    float* rstd;            // may be null
    int64_t x_pitch, y_pitch;
    int64_t rows, cols;
    float eps;
    float inv_cols;
};

struct BwdParams {
    const void* dY;
    const void* X;
    const void* gamma;      // may be null: 1
    const float* mean;
    const float* rstd;
    void* dX;               // may be null
    float* partial;         // [blocks][2][cols]: column sums of dy xh, of dy; null: not wanted
    int64_t dy_pitch, x_pitch, dx_pitch;
    int64_t rows, cols;
    float inv_cols;
    int threads_per_row;
};

// V elements of T in one access (V = 1: any alignment; else 16 bytes)
template <typename T, int V>
struct alignas(V * sizeof(T)) Pack {
    T v[V];
};

template <typename T, int V>
__device__ __forceinline__ void load(float (&out)[V], const T* p) {
    const Pack<T, V> k = *reinterpret_cast<const Pack<T, V>*>(p);
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = Num<T>::to_acc(k.v[i]);
}
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const float (&in)[V]) {
    Pack<T, V> k;
#pragma unroll
    for (int i = 0; i < V; ++i) k.v[i] = Num<T>::from_acc(in[i]);
    *reinterpret_cast<Pack<T, V>*>(p) = k;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// sum over the W warps of a block; every thread gets it.  `slot` has W
// floats; consecutive calls take different slots.
template <int W>
__device__ __forceinline__ float block_sum(float v, float* slot) {
    v = warp_sum(v);
    if constexpr (W == 1) return v;
    if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) s += slot[i];
    return s;
}

// W warps on a row, NV packs of V elements a thread, in registers.  W == 1:
// blocks of four independent warps.
template <typename T, int V, int W, int NV>
__global__ void __launch_bounds__(W == 1 ? 128 : W * 32)
forward_kernel(const FwdParams p) {
    __shared__ float slots[2][W];
    const int t = W == 1 ? (threadIdx.x & 31) : threadIdx.x;
    const int64_t row = W == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
    grid_dependency_wait();
    grid_launch_dependents();
    if (row >= p.rows) return;      // whole warps (W == 1); never with W > 1
    const T* x = static_cast<const T*>(p.X) + row * p.x_pitch;
    T* y = static_cast<T*>(p.Y) + row * p.y_pitch;
    const int cols = (int)p.cols;
    Pack<T, V> k[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + i * W * 32) * V;
        if (c < cols) k[i] = *reinterpret_cast<const Pack<T, V>*>(x + c);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if ((t + i * W * 32) * V < cols) {
#pragma unroll
            for (int q = 0; q < V; ++q) s += Num<T>::to_acc(k[i].v[q]);
        }
    const float mean = block_sum<W>(s, slots[0]) * p.inv_cols;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if ((t + i * W * 32) * V < cols) {
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float d = Num<T>::to_acc(k[i].v[q]) - mean;
                s = fmaf(d, d, s);
            }
        }
    const float rstd = 1.0f / sqrtf(fmaf(block_sum<W>(s, slots[1]), p.inv_cols, p.eps));
    if (t == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    const T* gamma = static_cast<const T*>(p.gamma);
    const T* beta = static_cast<const T*>(p.beta);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + i * W * 32) * V;
        if (c >= cols) continue;
        float g[V], b[V], o[V];
        if (gamma) load<T, V>(g, gamma + c);
        if (beta) load<T, V>(b, beta + c);
#pragma unroll
        for (int q = 0; q < V; ++q) {
            o[q] = (Num<T>::to_acc(k[i].v[q]) - mean) * rstd;
            if (gamma) o[q] *= g[q];
            if (beta) o[q] += b[q];
        }
        store<T, V>(y + c, o);
    }
}

// Rows longer than the registers of a block hold: three passes over the row.
template <typename T, int V>
__global__ void __launch_bounds__(1024) forward_long_kernel(const FwdParams p) {
    __shared__ float slots[2][32];
    grid_dependency_wait();
    grid_launch_dependents();
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(p.X) + row * p.x_pitch;
        T* y = static_cast<T*>(p.Y) + row * p.y_pitch;
        float s = 0.f;
        for (int64_t c = (int64_t)threadIdx.x * V; c < p.cols; c += 1024 * V) {
            float v[V];
            load<T, V>(v, x + c);
#pragma unroll
            for (int q = 0; q < V; ++q) s += v[q];
        }
        const float mean = block_sum<32>(s, slots[0]) * p.inv_cols;
        s = 0.f;
        for (int64_t c = (int64_t)threadIdx.x * V; c < p.cols; c += 1024 * V) {
            float v[V];
            load<T, V>(v, x + c);
#pragma unroll
            for (int q = 0; q < V; ++q) s = fmaf(v[q] - mean, v[q] - mean, s);
        }
        const float rstd = 1.0f / sqrtf(fmaf(block_sum<32>(s, slots[1]), p.inv_cols, p.eps));
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
        const T* gamma = static_cast<const T*>(p.gamma);
        const T* beta = static_cast<const T*>(p.beta);
        for (int64_t c = (int64_t)threadIdx.x * V; c < p.cols; c += 1024 * V) {
            float v[V], g[V], b[V];
            load<T, V>(v, x + c);
            if (gamma) load<T, V>(g, gamma + c);
            if (beta) load<T, V>(b, beta + c);
#pragma unroll
            for (int q = 0; q < V; ++q) {
                v[q] = (v[q] - mean) * rstd;
                if (gamma) v[q] *= g[q];
                if (beta) v[q] += b[q];
            }
            store<T, V>(y + c, v);
        }
    }
}

// Backward.  A block is `groups` groups of threads_per_row threads; a thread
// keeps the same NV * V columns of every row its group takes, so that the
// column sums of dgamma and dbeta stay in its registers until the block's
// last row; the groups' sums are then added in group order and written as
// the block's partial sums.  The next row is loaded before this one's
// reduction.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(1024) backward_kernel(const BwdParams p) {
    extern __shared__ float shared[];           // group sums: [groups][cols] x 2, one after the other
    __shared__ float2 slots[2][32];
    const int tpr = p.threads_per_row;
    const int groups = blockDim.x / tpr;
    const int grp = threadIdx.x / tpr, t = threadIdx.x % tpr;
    const int warps = tpr >> 5;
    const int cols = (int)p.cols;
    const bool weights = p.partial != nullptr;
    const bool has_gamma = p.gamma != nullptr;
    grid_dependency_wait();
    grid_launch_dependents();
    Pack<T, V> kx[NV], kd[NV], kg[NV];
    float ag[NV][V], ab[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + i * tpr) * V;
        if (has_gamma && c < cols) kg[i] = *reinterpret_cast<const Pack<T, V>*>(static_cast<const T*>(p.gamma) + c);
#pragma unroll
        for (int q = 0; q < V; ++q) ag[i][q] = ab[i][q] = 0.f;
    }
    const int64_t step = (int64_t)gridDim.x * groups;
    auto fetch = [&](int64_t row) {
        if (row >= p.rows) return;
        const T* x = static_cast<const T*>(p.X) + row * p.x_pitch;
        const T* dy = static_cast<const T*>(p.dY) + row * p.dy_pitch;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * tpr) * V;
            if (c < cols) {
                kx[i] = *reinterpret_cast<const Pack<T, V>*>(x + c);
                kd[i] = *reinterpret_cast<const Pack<T, V>*>(dy + c);
            }
        }
    };
    int64_t row = (int64_t)blockIdx.x * groups + grp;
    fetch(row);
    int buf = 0;
    // every group runs the same number of turns (the block's barriers)
    for (int64_t first = (int64_t)blockIdx.x * groups; first < p.rows; first += step, row += step, buf ^= 1) {
        const bool live = row < p.rows;
        const float mean = live ? p.mean[row] : 0.f, rstd = live ? p.rstd[row] : 0.f;
        float xh[NV][V], dxh[NV][V];
        float c1 = 0.f, c2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool in = live && (t + i * tpr) * V < cols;
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float d = in ? Num<T>::to_acc(kd[i].v[q]) : 0.f;
                xh[i][q] = in ? (Num<T>::to_acc(kx[i].v[q]) - mean) * rstd : 0.f;
                if (weights) {
                    ag[i][q] = fmaf(d, xh[i][q], ag[i][q]);
                    ab[i][q] += d;
                }
                dxh[i][q] = has_gamma && in ? d * Num<T>::to_acc(kg[i].v[q]) : d;
                c1 += dxh[i][q];
                c2 = fmaf(dxh[i][q], xh[i][q], c2);
            }
        }
        fetch(row + step);
        if (!p.dX) continue;                      // uniform over the grid
        c1 = warp_sum(c1);
        c2 = warp_sum(c2);
        if (warps > 1) {
            if ((threadIdx.x & 31) == 0) slots[buf][threadIdx.x >> 5] = make_float2(c1, c2);
            __syncthreads();
            c1 = c2 = 0.f;
            for (int w = 0; w < warps; ++w) {
                const float2 v = slots[buf][grp * warps + w];
                c1 += v.x;
                c2 += v.y;
            }
        }
        c1 *= p.inv_cols;
        c2 *= p.inv_cols;
        if (live) {
            T* dx = static_cast<T*>(p.dX) + row * p.dx_pitch;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = (t + i * tpr) * V;
                if (c >= cols) continue;
                float o[V];
#pragma unroll
                for (int q = 0; q < V; ++q) o[q] = rstd * (dxh[i][q] - c1 - xh[i][q] * c2);
                store<T, V>(dx + c, o);
            }
        }
    }
    if (!weights) return;
    float* out = p.partial + (int64_t)blockIdx.x * 2 * cols;
    if (groups == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * tpr) * V;
            if (c >= cols) continue;
#pragma unroll
            for (int q = 0; q < V; ++q) {
                out[c + q] = ag[i][q];
                out[cols + c + q] = ab[i][q];
            }
        }
        return;
    }
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * tpr) * V;
            if (c >= cols) continue;
#pragma unroll
            for (int q = 0; q < V; ++q) shared[grp * cols + c + q] = which ? ab[i][q] : ag[i][q];
        }
        __syncthreads();
        for (int c = threadIdx.x; c < cols; c += blockDim.x) {
            float s = 0.f;
            for (int g = 0; g < groups; ++g) s += shared[g * cols + c];
            out[which * cols + c] = s;
        }
    }
}

// Rows wider than a block's registers hold: dx alone, two passes over the row.
template <typename T, int V>
__global__ void __launch_bounds__(1024) backward_long_rows_kernel(const BwdParams p) {
    __shared__ float slots[2][32];
    grid_dependency_wait();
    grid_launch_dependents();
    const T* gamma = static_cast<const T*>(p.gamma);
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(p.X) + row * p.x_pitch;
        const T* dy = static_cast<const T*>(p.dY) + row * p.dy_pitch;
        T* dx = static_cast<T*>(p.dX) + row * p.dx_pitch;
        const float mean = p.mean[row], rstd = p.rstd[row];
        float c1 = 0.f, c2 = 0.f;
        for (int64_t c = (int64_t)threadIdx.x * V; c < p.cols; c += 1024 * V) {
            float a[V], d[V], g[V];
            load<T, V>(a, x + c);
            load<T, V>(d, dy + c);
            if (gamma) load<T, V>(g, gamma + c);
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float dxh = gamma ? d[q] * g[q] : d[q];
                c1 += dxh;
                c2 = fmaf(dxh, (a[q] - mean) * rstd, c2);
            }
        }
        c1 = block_sum<32>(c1, slots[0]) * p.inv_cols;
        c2 = block_sum<32>(c2, slots[1]) * p.inv_cols;
        for (int64_t c = (int64_t)threadIdx.x * V; c < p.cols; c += 1024 * V) {
            float a[V], d[V], g[V];
            load<T, V>(a, x + c);
            load<T, V>(d, dy + c);
            if (gamma) load<T, V>(g, gamma + c);
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float dxh = gamma ? d[q] * g[q] : d[q];
                a[q] = rstd * (dxh - c1 - (a[q] - mean) * rstd * c2);
            }
            store<T, V>(dx + c, a);
        }
    }
}

// The column sums of such rows: blockIdx.y takes an equal share of the rows,
// a thread one column.
template <typename T>
__global__ void __launch_bounds__(256) backward_long_cols_kernel(const BwdParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= p.cols) return;
    const int64_t r0 = p.rows * blockIdx.y / gridDim.y, r1 = p.rows * (blockIdx.y + 1) / gridDim.y;
    float g = 0.f, b = 0.f;
    for (int64_t r = r0; r < r1; ++r) {
        const float d = Num<T>::to_acc(static_cast<const T*>(p.dY)[r * p.dy_pitch + c]);
        const float xh = (Num<T>::to_acc(static_cast<const T*>(p.X)[r * p.x_pitch + c]) - p.mean[r]) * p.rstd[r];
        g = fmaf(d, xh, g);
        b += d;
    }
    p.partial[((int64_t)blockIdx.y * 2) * p.cols + c] = g;
    p.partial[((int64_t)blockIdx.y * 2 + 1) * p.cols + c] = b;
}

// Column sums over the blocks' partial sums, in block order within each of
// eight threads' shares and then in share order: the same for every run.
template <typename T>
__global__ void __launch_bounds__(256) column_sum_kernel(const float* __restrict__ partial, int blocks, int64_t cols,
                                                         T* dgamma, T* dbeta) {
    __shared__ float sums[8][33];
    grid_dependency_wait();
    grid_launch_dependents();
    T* out = blockIdx.y ? dbeta : dgamma;
    if (!out) return;
    const int lane = threadIdx.x & 31, share = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < cols)
        for (int b = share; b < blocks; b += 8) s += partial[((int64_t)b * 2 + blockIdx.y) * cols + c];
    sums[share][lane] = s;
    __syncthreads();
    if (share == 0 && c < cols) {
        s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += sums[i][lane];
        out[c] = Num<T>::from_acc(s);
    }
}

// ---- host side -------------------------------------------------------------

template <typename F>
olc_status by_type(olc_dtype dt, F&& f) {
    switch (dt) {
        case OLC_FLOAT: return f(float{});
        case OLC_FLOAT16: return f(__half{});
        case OLC_BFLOAT16: return f(__nv_bfloat16{});
        default: return OLC_ERR_DTYPE;
    }
}

template <typename T, int V>
cudaError_t forward_as(const FwdParams& p, int sm_count, cudaStream_t s) {
    const int64_t packs = ceil_div(p.cols, V);
    // one warp on a row while the row fits 16 packs a lane: no block barrier
    // on the way.  Where such warps would leave SMs idle, and for longer
    // rows, eight or 32 warps share a row.
    const bool few = p.rows < 4 * (int64_t)sm_count;
#define OLC_FWD(W, NV)                                                                                       \
    return launch_pdl(forward_kernel<T, V, W, NV>, dim3((unsigned)(W == 1 ? ceil_div(p.rows, 4) : p.rows)),  \
                      dim3(W == 1 ? 128 : W * 32), 0, s, p)
    if (p.rows <= 0x7fffffff) {
        if (packs <= 32) OLC_FWD(1, 1);
        if (packs <= 64) OLC_FWD(1, 2);
        if (packs <= 128) OLC_FWD(1, 4);
        if (packs <= 256 && !few) OLC_FWD(1, 8);
        if (packs <= 512 && !few) OLC_FWD(1, 16);
        if (packs <= 512) OLC_FWD(8, 2);
        if (packs <= 1024) OLC_FWD(8, 4);
        if (packs <= 2048) OLC_FWD(8, 8);
        if (packs <= 4096) OLC_FWD(32, 4);
        if (packs <= 8192) OLC_FWD(32, 8);
    }
#undef OLC_FWD
    const int64_t grid = min64(p.rows, (int64_t)sm_count * 2);
    return launch_pdl(forward_long_kernel<T, V>, dim3((unsigned)grid), dim3(1024), 0, s, p);
}

constexpr int kColsPerThread = 16;      // float32 column sums of dgamma and dbeta: 32 registers

// the backward launch of one shape: which kernel, how many threads
struct BwdShape {
    int nv = 0;                          // 0: rows wider than a block's registers
    int tpr = 0, groups = 1, threads = 0;
    int64_t blocks = 0;
};

template <int V>
BwdShape backward_shape(int64_t rows, int64_t cols, int sm_count) {
    BwdShape b;
    const int64_t packs = ceil_div(cols, V);
    if (packs > 1024 * (kColsPerThread / V)) {
        b.blocks = min64(max64(rows / 64, 1), max64(1, 8 * (int64_t)sm_count * 256 / cols));
        return b;
    }
    b.nv = 1;
    while (b.nv * V < kColsPerThread && packs > 512 * b.nv) b.nv *= 2;
    b.tpr = (int)(ceil_div(ceil_div(packs, b.nv), 32) * 32);
    b.groups = b.tpr >= 256 ? 1 : 256 / b.tpr;
    b.threads = b.tpr * b.groups;
    const int per_sm = b.threads > 512 ? 1 : 2 * (512 / b.threads);
    b.blocks = max64(1, min64(ceil_div(rows, b.groups), (int64_t)sm_count * per_sm));
    return b;
}

template <typename T, int V, int NV>
cudaError_t backward_rows(const BwdParams& p, const BwdShape& b, cudaStream_t s) {
    const size_t smem = b.groups > 1 ? (size_t)b.groups * p.cols * sizeof(float) : 0;
    return launch_pdl(backward_kernel<T, V, NV>, dim3((unsigned)b.blocks), dim3((unsigned)b.threads), smem, s, p);
}

template <typename T, int V>
cudaError_t backward_as(BwdParams p, int sm_count, T* dgamma, T* dbeta, cudaStream_t s) {
    const BwdShape b = backward_shape<V>(p.rows, p.cols, sm_count);
    cudaError_t e = cudaSuccess;
    p.threads_per_row = b.tpr;
    if (b.nv == 0) {
        // the column sums first: dX may be dY or X
        if (p.partial)
            e = launch_pdl(backward_long_cols_kernel<T>, dim3((unsigned)ceil_div(p.cols, 256), (unsigned)b.blocks),
                           dim3(256), 0, s, p);
        if (e == cudaSuccess && p.dX)
            e = launch_pdl(backward_long_rows_kernel<T, V>, dim3((unsigned)min64(p.rows, (int64_t)sm_count * 2)),
                           dim3(1024), 0, s, p);
    } else if (b.nv == 1) {
        e = backward_rows<T, V, 1>(p, b, s);
    } else if (b.nv == 2) {
        e = backward_rows<T, V, 2>(p, b, s);
    } else if (b.nv == 4) {
        if constexpr (V <= 4) e = backward_rows<T, V, 4>(p, b, s);
    } else if (b.nv == 8) {
        if constexpr (V == 1) e = backward_rows<T, V, 8>(p, b, s);
    } else {
        if constexpr (V == 1) e = backward_rows<T, V, 16>(p, b, s);
    }
    if (e == cudaSuccess && p.partial)
        e = launch_pdl(column_sum_kernel<T>, dim3((unsigned)ceil_div(p.cols, 32), 2), dim3(256), 0, s,
                       (const float*)p.partial, (int)b.blocks, p.cols, dgamma, dbeta);
    return e;
}

}  // namespace norm
}  // namespace olc

using namespace olc;

struct olc_layer_norm_plan {
    PlanState state;
    olc_dtype dtype;
    int64_t rows, cols;
    float eps;
};

extern "C" {

olc_status olc_layer_norm_plan_create(int64_t rows, int64_t cols, double eps, olc_dtype dtype,
                                      olc_layer_norm_plan** out) {
    if (!out) return OLC_ERR_NULL;
    *out = nullptr;
    if (!plan_dtype_ok(dtype)) return OLC_ERR_DTYPE;
    if (rows < 0 || cols < 0) return OLC_ERR_NEGATIVE_DIM;
    // the mean of no elements is undefined; columns are 32-bit in the kernels
    if (cols == 0 || cols >= (int64_t(1) << 31) - 65536 || !(eps >= 0.0) || eps > 3e38) return OLC_ERR_INVALID;
    if (!plan_fits(rows, cols, 4)) return OLC_ERR_INVALID;
    olc_layer_norm_plan* p = new (std::nothrow) olc_layer_norm_plan;
    if (!p) return OLC_ERR_OOM;
    p->state.init();
    p->dtype = dtype;
    p->rows = rows;
    p->cols = cols;
    p->eps = (float)eps;
    *out = p;
    return OLC_OK;
}

void olc_layer_norm_plan_destroy(olc_layer_norm_plan* plan) {
    if (!plan) return;
    plan->state.destroy();
    delete plan;
}

olc_status olc_layer_norm_forward(olc_layer_norm_plan* plan, const void* X, int64_t x_pitch, const void* gamma,
                                  const void* beta, void* Y, int64_t y_pitch, float* mean, float* rstd,
                                  void* stream) {
    if (!plan) return OLC_ERR_NULL;
    if (plan->rows == 0) return OLC_OK;
    if (!X || !Y) return OLC_ERR_NULL;
    const int64_t eb = plan_elem_bytes(plan->dtype);
    if (plan->rows > 1 && (x_pitch < plan->cols || y_pitch < plan->cols)) return OLC_ERR_INVALID;
    if (plan->rows > 1 && (!plan_fits(plan->rows, x_pitch, eb) || !plan_fits(plan->rows, y_pitch, eb)))
        return OLC_ERR_INVALID;
    if (plan_misaligned(X, eb) || plan_misaligned(gamma, eb) || plan_misaligned(beta, eb) || plan_misaligned(Y, eb) ||
        plan_misaligned(mean, 4) || plan_misaligned(rstd, 4))
        return OLC_ERR_INVALID;
    const olc_status st = plan->state.bind();
    if (st != OLC_OK) return st;
    norm::FwdParams p{X, gamma, beta, Y, mean, rstd, x_pitch, y_pitch, plan->rows, plan->cols, plan->eps,
                      (float)(1.0 / (double)plan->cols)};
    // 16-byte packs need every row of every operand on a 16-byte boundary
    const bool wide = plan->cols * eb % 16 == 0 && plan_aligned16(X) && plan_aligned16(Y) && plan_aligned16(gamma) &&
                      plan_aligned16(beta) && (plan->rows == 1 || (x_pitch * eb % 16 == 0 && y_pitch * eb % 16 == 0));
    return norm::by_type(plan->dtype, [&](auto tag) {
        using T = decltype(tag);
        const cudaStream_t s = static_cast<cudaStream_t>(stream);
        return plan_status(wide ? norm::forward_as<T, 16 / sizeof(T)>(p, plan->state.sm_count, s)
                                : norm::forward_as<T, 1>(p, plan->state.sm_count, s));
    });
}

olc_status olc_layer_norm_backward(olc_layer_norm_plan* plan, const void* dY, int64_t dy_pitch, const void* X,
                                   int64_t x_pitch, const void* gamma, const float* mean, const float* rstd, void* dX,
                                   int64_t dx_pitch, void* dgamma, void* dbeta, void* stream) {
    if (!plan) return OLC_ERR_NULL;
    if (!dX && !dgamma && !dbeta) return OLC_OK;
    const int64_t eb = plan_elem_bytes(plan->dtype), rows = plan->rows, cols = plan->cols;
    if (rows > 0 && (!dY || !X || !mean || !rstd)) return OLC_ERR_NULL;
    if (rows > 1 && (dy_pitch < cols || x_pitch < cols || (dX && dx_pitch < cols))) return OLC_ERR_INVALID;
    if (rows > 1 && (!plan_fits(rows, dy_pitch, eb) || !plan_fits(rows, x_pitch, eb) ||
                     (dX && !plan_fits(rows, dx_pitch, eb))))
        return OLC_ERR_INVALID;
    if (plan_misaligned(dY, eb) || plan_misaligned(X, eb) || plan_misaligned(gamma, eb) || plan_misaligned(mean, 4) ||
        plan_misaligned(rstd, 4) || plan_misaligned(dX, eb) || plan_misaligned(dgamma, eb) ||
        plan_misaligned(dbeta, eb))
        return OLC_ERR_INVALID;
    olc_status st = plan->state.bind();
    if (st != OLC_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0) {                        // empty sums
        cudaError_t e = dgamma ? launch_zero_fill(dgamma, cols * eb, s) : cudaSuccess;
        if (e == cudaSuccess && dbeta) e = launch_zero_fill(dbeta, cols * eb, s);
        return plan_status(e);
    }
    const bool wide = cols * eb % 16 == 0 && plan_aligned16(X) && plan_aligned16(dY) && plan_aligned16(gamma) &&
                      plan_aligned16(dX) &&
                      (rows == 1 || (x_pitch * eb % 16 == 0 && dy_pitch * eb % 16 == 0 &&
                                     (!dX || dx_pitch * eb % 16 == 0)));
    norm::BwdParams p{dY, X, gamma, mean, rstd, dX, nullptr, dy_pitch, x_pitch, dx_pitch, rows, cols,
                      (float)(1.0 / (double)cols), 0};
    const bool weights = dgamma || dbeta;
    if (weights) {
        // both layouts' partial sums fit: a call with other alignment does
        // not have to allocate again
        const int sms = plan->state.sm_count;
        const int64_t blocks = max64(plan->dtype == OLC_FLOAT ? norm::backward_shape<4>(rows, cols, sms).blocks
                                                              : norm::backward_shape<8>(rows, cols, sms).blocks,
                                     norm::backward_shape<1>(rows, cols, sms).blocks);
        st = plan->state.ensure((size_t)blocks * 2 * (size_t)cols * sizeof(float));
        if (st != OLC_OK) return st;
        p.partial = static_cast<float*>(plan->state.memory);
        const cudaError_t e = plan->state.before_use(s);
        if (e != cudaSuccess) return plan_status(e);
    }
    return norm::by_type(plan->dtype, [&](auto tag) {
        using T = decltype(tag);
        T *dg = static_cast<T*>(dgamma), *db = static_cast<T*>(dbeta);
        cudaError_t e = wide ? norm::backward_as<T, 16 / sizeof(T)>(p, plan->state.sm_count, dg, db, s)
                             : norm::backward_as<T, 1>(p, plan->state.sm_count, dg, db, s);
        if (e == cudaSuccess && weights) e = plan->state.after_use(s);
        return plan_status(e);
    });
}

}  // extern "C"
