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
// cancellation for rows far from zero, whose mean is corrected by the sum of the
// distances as well); rows too long for the registers are read again, mostly
// from L2.  All sums and statistics are float32; y, dx, dgamma and dbeta are
// rounded to the element type once.  Measured, BF16 [16384, 4096]: forward 44.3 us
// (6.1 TB/s, a plain copy of the tensor 41 to 43.5), backward 66.5 us (6.1 TB/s)
// with the column sums' 4 us.
#include <new>

#include "plan_state.h"
#include "row_packs.cuh"

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
    float count, inv_cols;  // cols, 1 / cols
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
    unsigned int* err;
};

// y = (x - mean) rstd gamma + beta on one pack
template <typename T, int V>
__device__ __forceinline__ void finish(T* y, const Pack<T, V>& k, F2 minus_mean, F2 rstd, const T* gamma,
                                       const T* beta) {
    F2 x[pairs<V>()], w[pairs<V>()];
    widen<T, V>(x, k);
#pragma unroll
    for (int i = 0; i < pairs<V>(); ++i) x[i] = mul2(add2(x[i], minus_mean), rstd);
    if (gamma) {
        widen<T, V>(w, load<T, V>(gamma));
#pragma unroll
        for (int i = 0; i < pairs<V>(); ++i) x[i] = mul2(x[i], w[i]);
    }
    if (beta) {
        widen<T, V>(w, load<T, V>(beta));
#pragma unroll
        for (int i = 0; i < pairs<V>(); ++i) x[i] = add2(x[i], w[i]);
    }
    store<T, V>(y, x);
}
template <typename T, int V>
__device__ __forceinline__ void add_elements(F2& s, const Pack<T, V>& k) {
    F2 x[pairs<V>()];
    widen<T, V>(x, k);
#pragma unroll
    for (int i = 0; i < pairs<V>(); ++i) s = add2(s, x[i]);
}
template <typename T, int V>
__device__ __forceinline__ void add_distances(F2& s, const Pack<T, V>& k, F2 minus_mean) {
    F2 x[pairs<V>()];
    widen<T, V>(x, k);
#pragma unroll
    for (int i = 0; i < pairs<V>(); ++i) s = add2(s, add2(x[i], minus_mean));
}
template <typename T, int V>
__device__ __forceinline__ void add_squares(F2& s, const Pack<T, V>& k, F2 minus_mean) {
    F2 x[pairs<V>()];
    widen<T, V>(x, k);
#pragma unroll
    for (int i = 0; i < pairs<V>(); ++i) {
        const F2 d = add2(x[i], minus_mean);
        s = fma2(d, d, s);
    }
}

// A row's sum over its count, the nearest value of the quotient: the product
// with the rounded 1 / count, corrected by what it leaves (infinities and NaN
// as they are).
__device__ __forceinline__ float mean_of(float sum, const FwdParams& p) {
    const float q = sum * p.inv_cols, rest = fmaf(-q, p.count, sum);
    return rest == rest ? fmaf(rest, p.inv_cols, q) : q;
}
// The mean's error, a few roundings of it, shows where the row's spread is small
// beside it: below 2^-6 of the mean (there it is 2^-16 of the spread).  Such rows
// sum the distances from it too, and take their mean out of the mean and of the
// squares (Chan, Golub and LeVeque's corrected two-pass algorithm), which leaves
// the mean's one rounding, and nothing of a row of equal values.  The test costs
// [16384, 4096] BF16 some 0.5 us; the distances in every row 1.5.
__device__ __forceinline__ bool far_from_zero(float mean, float squares, const FwdParams& p) {
    return __builtin_expect(squares * 4096.f < mean * mean * p.count, 0);   // not for NaN
}
__device__ __forceinline__ void correct(float& mean, float& squares, float distances, const FwdParams& p) {
    const float shift = distances * p.inv_cols;
    mean += shift;
    squares = fmaxf(fmaf(-distances, shift, squares), 0.f);
}
__device__ __forceinline__ float rstd_of(float squares, const FwdParams& p) {
    return 1.0f / sqrtf(fmaf(squares, p.inv_cols, p.eps));
}

// W warps on a row, NV packs (or pairs of elements) a thread, in registers.
// W == 1: blocks of four independent warps (nine of them an SM with four packs
// a thread: [16384, 1024] BF16 14.0 us, eight 14.6).
template <typename T, int V, int W, int NV>
__global__ void __launch_bounds__(W == 1 ? 128 : W * 32, V == 8 && W == 1 && NV == 4 ? 9 : 0)
forward_kernel(const FwdParams p) {
    using C = Columns<T, V>;
    constexpr int P = C::P, TPR = W * 32;
    __shared__ float slots[3][W];
    const int t = W == 1 ? (threadIdx.x & 31) : threadIdx.x;
    const int64_t row = W == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
    if (row >= p.rows) return;      // whole warps (W == 1); never with W > 1
    const T* x = static_cast<const T*>(p.X) + row * p.x_pitch;
    T* y = static_cast<T*>(p.Y) + row * p.y_pitch;
    const int cols = (int)p.cols, whole = V == 1 && W > 1 ? cols / (2 * TPR) : 0;
    typename C::Raw k[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        k[i] = C::read(x, t, i, TPR, cols, true, i < whole);
    }
    F2 s = 0, v[P];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        C::pairs_of(v, k[i]);
#pragma unroll
        for (int q = 0; q < P; ++q) s = add2(s, v[q]);     // zeros past the row's end
    }
    float mean = mean_of(block_sum<W>(sum_of<2>(s), slots[0]), p);
    F2 minus_mean = both(-mean);
    s = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        C::pairs_of(v, k[i]);
        if constexpr (V == 1) {
            v[0] = add2(v[0], minus_mean);
            if (i >= whole) {
                float lo, hi;
                unpack_f2(v[0], lo, hi);
                v[0] = pack_f2(C::in(t, i, 0, TPR, cols) ? lo : 0.f, C::in(t, i, 1, TPR, cols) ? hi : 0.f);
            }
            s = fma2(v[0], v[0], s);
        } else if (C::in(t, i, 0, TPR, cols)) {
#pragma unroll
            for (int q = 0; q < P; ++q) {
                const F2 d = add2(v[q], minus_mean);
                s = fma2(d, d, s);
            }
        }
    }
    float squares = block_sum<W>(sum_of<2>(s), slots[1]);
    if (far_from_zero(mean, squares, p)) {          // the whole row's threads
        float distances = 0.f;
#pragma unroll 1
        for (int c = t; c < cols; c += TPR) distances += Num<T>::to_acc(x[c]) - mean;      // read again: few rows do
        correct(mean, squares, block_sum<W>(distances, slots[2]), p);
        minus_mean = both(-mean);
    }
    const float rstd = rstd_of(squares, p);
    if (t == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
    }
    const F2 scale = both(rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (i >= whole && !C::in(t, i, 0, TPR, cols)) continue;
        F2 w[P];
        C::pairs_of(v, k[i]);
#pragma unroll
        for (int q = 0; q < P; ++q) v[q] = mul2(add2(v[q], minus_mean), scale);
        if (p.gamma) {
            C::pairs_of(w, C::read(static_cast<const T*>(p.gamma), t, i, TPR, cols, true, i < whole));
#pragma unroll
            for (int q = 0; q < P; ++q) v[q] = mul2(v[q], w[q]);
        }
        if (p.beta) {
            C::pairs_of(w, C::read(static_cast<const T*>(p.beta), t, i, TPR, cols, true, i < whole));
#pragma unroll
            for (int q = 0; q < P; ++q) v[q] = add2(v[q], w[q]);
        }
        C::write(y, t, i, TPR, cols, v, i < whole);
    }
}

// Rows of at most L packs (8 or 16): L lanes on a row, R rows a lane one after the
// other, all of them on their way at once.
template <typename T, int L, int R>
__global__ void __launch_bounds__(128) forward_short_kernel(const FwdParams p) {
    constexpr int V = 16 / sizeof(T), P = V / 2, ROWS = 128 / L;
    const int c = (int)(threadIdx.x % L) * V;
    const bool in = c < (int)p.cols;
    const int64_t first = (int64_t)blockIdx.x * (ROWS * R) + threadIdx.x / L;
    const Pack<T, V> zero{};
    Pack<T, V> k[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t row = first + r * ROWS;
        k[r] = in && row < p.rows ? load<T, V>(static_cast<const T*>(p.X) + row * p.x_pitch + c) : zero;
    }
    F2 g[P], b[P];
    if (p.gamma && in) widen<T, V>(g, load<T, V>(static_cast<const T*>(p.gamma) + c));
    if (p.beta && in) widen<T, V>(b, load<T, V>(static_cast<const T*>(p.beta) + c));
    auto sum = [](F2 x) {
        float v = sum_of<2>(x);
#pragma unroll
        for (int d = L / 2; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        return v;
    };
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t row = first + r * ROWS;
        F2 x[P], s = 0;
        widen<T, V>(x, k[r]);
#pragma unroll
        for (int q = 0; q < P; ++q) s = add2(s, x[q]);
        float mean = mean_of(sum(s), p);
        s = 0;
#pragma unroll
        for (int q = 0; q < P; ++q) {
            x[q] = add2(x[q], both(-mean));
            if (in) s = fma2(x[q], x[q], s);
        }
        float squares = sum(s);
        const bool far = far_from_zero(mean, squares, p);
        if (__any_sync(0xffffffffu, far)) {         // any of the warp's rows: the whole warp sums
            s = 0;
#pragma unroll
            for (int q = 0; q < P; ++q)
                if (in) s = add2(s, x[q]);
            const float distances = sum(s);
            if (far) {
                const float before = mean;
                correct(mean, squares, distances, p);
#pragma unroll
                for (int q = 0; q < P; ++q) x[q] = add2(x[q], both(before - mean));
            }
        }
        const float rstd = rstd_of(squares, p);
        if (row >= p.rows) continue;
        if (c == 0) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
#pragma unroll
        for (int q = 0; q < P; ++q) {
            x[q] = mul2(x[q], both(rstd));
            if (p.gamma) x[q] = mul2(x[q], g[q]);
            if (p.beta) x[q] = add2(x[q], b[q]);
        }
        if (in) store<T, V>(static_cast<T*>(p.Y) + row * p.y_pitch + c, x);
    }
}

// Rows longer than the registers of a block hold: three passes over the row.
template <typename T, int V>
__global__ void __launch_bounds__(1024) forward_long_kernel(const FwdParams p) {
    __shared__ float slots[3][32];
    const T* gamma = static_cast<const T*>(p.gamma);
    const T* beta = static_cast<const T*>(p.beta);
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(p.X) + row * p.x_pitch;
        T* y = static_cast<T*>(p.Y) + row * p.y_pitch;
        F2 s = 0;
#pragma unroll 4
        for (int64_t c = (int64_t)threadIdx.x * V; c < p.cols; c += 1024 * V) add_elements<T, V>(s, load<T, V>(x + c));
        float mean = mean_of(block_sum<32>(sum_of<V>(s), slots[0]), p);
        s = 0;
#pragma unroll 4
        for (int64_t c = (int64_t)threadIdx.x * V; c < p.cols; c += 1024 * V)
            add_squares<T, V>(s, load<T, V>(x + c), both(-mean));
        float squares = block_sum<32>(sum_of<V>(s), slots[1]);
        if (far_from_zero(mean, squares, p)) {      // the whole block
            s = 0;
#pragma unroll 1
            for (int64_t c = (int64_t)threadIdx.x * V; c < p.cols; c += 1024 * V)
                add_distances<T, V>(s, load<T, V>(x + c), both(-mean));
            correct(mean, squares, block_sum<32>(sum_of<V>(s), slots[2]), p);
        }
        const float rstd = rstd_of(squares, p);
        if (threadIdx.x == 0) {
            if (p.mean) p.mean[row] = mean;
            if (p.rstd) p.rstd[row] = rstd;
        }
        for (int64_t c = (int64_t)threadIdx.x * V; c < p.cols; c += 1024 * V)
            finish<T, V>(y + c, load<T, V>(x + c), both(-mean), both(rstd), gamma ? gamma + c : nullptr,
                         beta ? beta + c : nullptr);
    }
}

// Backward.  A block is `groups` groups of threads_per_row threads; a thread
// keeps the same NV * V columns of every row its group takes, so that the
// column sums of dgamma and dbeta stay in its registers until the block's
// last row; the groups' sums are then added in group order and written as
// the block's partial sums.  A row is three steps: xh and dxh of the thread's
// columns, the two row sums over the group (one block barrier), dx.
template <typename T, int V, int NV>
struct RowGrads {
    F2 ag[NV][pairs<V>()], ab[NV][pairs<V>()];      // column sums of dy xh and dy
    F2 xh[NV][pairs<V>()], dxh[NV][pairs<V>()];
    F2 g[NV][pairs<V>()];                           // gamma, or ones

    __device__ __forceinline__ void weights(int i, const T* gamma) {
        if (gamma) widen<T, V>(g[i], load<T, V>(gamma));
        else
            for (int q = 0; q < pairs<V>(); ++q) g[i][q] = both(1.f);
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int q = 0; q < pairs<V>(); ++q) ag[i][q] = ab[i][q] = 0;
    }
    // packs past the row's end, and rows past the last one, have dy = 0 and
    // add nothing
    __device__ __forceinline__ void take(int i, const Pack<T, V>& x, const Pack<T, V>& dy, F2 minus_mean, F2 rstd,
                                         F2& c1, F2& c2) {
        F2 d[pairs<V>()];
        widen<T, V>(xh[i], x);
        widen<T, V>(d, dy);
#pragma unroll
        for (int q = 0; q < pairs<V>(); ++q) {
            xh[i][q] = mul2(add2(xh[i][q], minus_mean), rstd);
            ag[i][q] = fma2(d[q], xh[i][q], ag[i][q]);
            ab[i][q] = add2(ab[i][q], d[q]);
            dxh[i][q] = mul2(d[q], g[i][q]);
            c1 = add2(c1, dxh[i][q]);
            c2 = fma2(dxh[i][q], xh[i][q], c2);
        }
    }
    // rstd (dxh - c1 - xh c2)
    __device__ __forceinline__ void put(int i, T* dx, F2 minus_c1, F2 minus_c2, F2 rstd) const {
        F2 o[pairs<V>()];
#pragma unroll
        for (int q = 0; q < pairs<V>(); ++q)
            o[q] = mul2(add2(fma2(xh[i][q], minus_c2, dxh[i][q]), minus_c1), rstd);
        store<T, V>(dx, o);
    }
    // the block's partial sums
    __device__ __forceinline__ void leave(float* out, int cols, int t, int threads) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * threads) * V;
            if (c >= cols) continue;
#pragma unroll
            for (int q = 0; q < pairs<V>(); ++q) {
                *reinterpret_cast<F2*>(out + c + 2 * q) = ag[i][q];
                *reinterpret_cast<F2*>(out + cols + c + 2 * q) = ab[i][q];
            }
        }
    }
};

// the sum of a block's slots (those of absent warps hold 0)
template <int WARPS>
__device__ __forceinline__ float2 sum_slots(const float2* slots) {
    F2 s = 0;
#pragma unroll
    for (int w = 0; w < WARPS; w += 2) {
        const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(slots + w);
        s = add2(add2(s, v.x), v.y);
    }
    float2 c;
    unpack_f2(s, c.x, c.y);
    return c;
}

// Any alignment and few or short rows: the next row is loaded into registers
// before this one's sums.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(512) backward_kernel(const BwdParams p) {
    using C = Columns<T, V>;
    constexpr int P = C::P;
    extern __shared__ float shared[];
    __shared__ alignas(16) float2 slots[2][16];
    const int tpr = p.threads_per_row;
    const int groups = blockDim.x / tpr, warps = tpr >> 5;
    const int grp = threadIdx.x / tpr, t = threadIdx.x - grp * tpr;
    const int cols = (int)p.cols;
    // single elements: a warp's columns lie together, so that their offsets are constants
    const int warp_base = (t >> 5) * (64 * NV);
    const int base = V == 1 ? warp_base + (t & 31) : t, stride = V == 1 ? 32 : tpr;
    const int whole = V == 1 ? (cols - warp_base) / 64 : 0;
    typename C::Raw kx[NV], kd[NV];
    F2 ag[NV][P], ab[NV][P], g[NV][P], xh[NV][P], dxh[NV][P];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (p.gamma) C::pairs_of(g[i], C::read(static_cast<const T*>(p.gamma), base, i, stride, cols, true, i < whole));
#pragma unroll
        for (int q = 0; q < P; ++q) {
            if (!p.gamma) g[i][q] = both(1.f);
            ag[i][q] = ab[i][q] = 0;
        }
    }
    const int64_t step = (int64_t)gridDim.x * groups;
    float mean = 0.f, rstd = 0.f;
    // packs past a row's end, and rows past the last one, have dy = 0 and add nothing
    auto fetch = [&](int64_t row) {
        const bool live = row < p.rows;
        const T* x = static_cast<const T*>(p.X) + row * p.x_pitch;
        const T* dy = static_cast<const T*>(p.dY) + row * p.dy_pitch;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            kx[i] = C::read(x, base, i, stride, cols, live, i < whole);
            kd[i] = C::read(dy, base, i, stride, cols, live, i < whole);
        }
        mean = live ? p.mean[row] : 0.f;
        rstd = live ? p.rstd[row] : 0.f;
    };
    int64_t row = (int64_t)blockIdx.x * groups + grp;
    fetch(row);
    int buf = 0;
    // every group runs the same number of turns: one barrier for the block (one a
    // group: [2049, 1001] FLOAT 14.7 us, so 12.6)
    for (int64_t first = (int64_t)blockIdx.x * groups; first < p.rows; first += step, row += step, buf ^= 1) {
        const F2 scale = both(rstd), minus_mean = both(-mean);
        F2 c1 = 0, c2 = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            F2 d[P];
            C::pairs_of(xh[i], kx[i]);
            C::pairs_of(d, kd[i]);
#pragma unroll
            for (int q = 0; q < P; ++q) {
                xh[i][q] = mul2(add2(xh[i][q], minus_mean), scale);
                ag[i][q] = fma2(d[q], xh[i][q], ag[i][q]);
                ab[i][q] = add2(ab[i][q], d[q]);
                dxh[i][q] = mul2(d[q], g[i][q]);
                c1 = add2(c1, dxh[i][q]);
                c2 = fma2(dxh[i][q], xh[i][q], c2);
            }
        }
        fetch(row + step);
        if (!p.dX) continue;                      // uniform over the grid
        float2 c = make_float2(warp_sum(sum_of<2>(c1)), warp_sum(sum_of<2>(c2)));
        if (warps > 1) {
            if ((threadIdx.x & 31) == 0) slots[buf][threadIdx.x >> 5] = c;
            __syncthreads();
            c = make_float2(0.f, 0.f);
            for (int w = 0; w < warps; ++w) {
                const float2 v = slots[buf][grp * warps + w];
                c.x += v.x;
                c.y += v.y;
            }
        }
        if (row < p.rows) {
            const F2 m1 = both(-c.x * p.inv_cols), m2 = both(-c.y * p.inv_cols);
            T* dx = static_cast<T*>(p.dX) + row * p.dx_pitch;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                F2 o[P];
#pragma unroll
                for (int q = 0; q < P; ++q) o[q] = mul2(add2(fma2(xh[i][q], m2, dxh[i][q]), m1), scale);
                C::write(dx, base, i, stride, cols, o, i < whole);
            }
        }
    }
    if (!p.partial) return;
    float* out = p.partial + (int64_t)blockIdx.x * 2 * cols;
    for (int which = 0; which < 2; ++which) {
        if (groups > 1) __syncthreads();
        float* to = groups > 1 ? shared + grp * cols : out + which * cols;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int q = 0; q < P; ++q) {
                float v[2];
                unpack_f2(which ? ab[i][q] : ag[i][q], v[0], v[1]);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (C::at(base, i, 2 * q + h, stride) < cols) to[C::at(base, i, 2 * q + h, stride)] = v[h];
            }
        if (groups == 1) continue;
        __syncthreads();
        for (int c = threadIdx.x; c < cols; c += blockDim.x) {
            float s = 0.f;
            for (int k = 0; k < groups; ++k) s += shared[k * cols + c];
            out[which * cols + c] = s;
        }
    }
}

// Rows of 16-byte packs: a group of threads takes one row at a time, x and dy
// copied ahead into its own ring of kAhead rows by bulk copies.  The barrier
// of the row's sums also tells that every thread has read the row: its buffer
// takes another.  The groups of a block join their column sums in group order,
// so that an SM leaves one set of partial sums.  WARPS: at least a group's;
// FULL: every thread has NV packs.
constexpr int kAhead = 3;
constexpr int kMaxGroups = 16;        // 512 threads, a warp or more on a row
template <typename T, int NV, int WARPS, bool FULL>
__global__ void __launch_bounds__(512) backward_ring_kernel(const BwdParams p) {
    constexpr int V = 16 / sizeof(T);
    extern __shared__ __align__(128) unsigned char rings[];
    __shared__ alignas(16) float2 all_slots[kMaxGroups][2][WARPS];
    __shared__ uint64_t all_full[kMaxGroups][kAhead];
    __shared__ int abort_flag;
    const int threads = p.threads_per_row, groups = blockDim.x / threads;
    const int grp = threadIdx.x / threads, t = threadIdx.x - grp * threads;
    const int cols = (int)p.cols;
    const uint32_t row_bytes = (uint32_t)cols * sizeof(T);
    unsigned char* const ring = rings + (size_t)grp * kAhead * 2 * row_bytes;
    float2(&slots)[2][WARPS] = all_slots[grp];
    uint64_t(&full)[kAhead] = all_full[grp];
    if (t < WARPS) slots[0][t] = slots[1][t] = make_float2(0.f, 0.f);
    if (threadIdx.x == 0) abort_flag = 0;
    if (t == 0) {
        for (int i = 0; i < kAhead; ++i) tc::mbar_init(&full[i], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();
    auto fetch = [&](int64_t row, int stage) {    // one thread
        if (row >= p.rows) return;
        unsigned char* to = ring + (size_t)stage * 2 * row_bytes;
        tc::mbar_arrive_expect_tx(&full[stage], 2 * row_bytes);
        bulk_copy(to, static_cast<const T*>(p.X) + row * p.x_pitch, row_bytes, &full[stage]);
        bulk_copy(to + row_bytes, static_cast<const T*>(p.dY) + row * p.dy_pitch, row_bytes, &full[stage]);
    };
    const int64_t step = (int64_t)gridDim.x * groups;
    int64_t row = (int64_t)blockIdx.x * groups + grp;
    if (t == 0)
        for (int i = 0; i < kAhead; ++i) fetch(row + i * step, i);
    RowGrads<T, V, NV> r;
    r.clear();
    const Pack<T, V> zero{};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + i * threads) * V;
        r.weights(i, p.gamma && c < cols ? static_cast<const T*>(p.gamma) + c : nullptr);
    }
    int stage = 0, phase = 0, buf = 0;
    float mean = row < p.rows ? p.mean[row] : 0.f, rstd = row < p.rows ? p.rstd[row] : 0.f;
    T* dx = p.dX ? static_cast<T*>(p.dX) + row * p.dx_pitch : nullptr;
    const int64_t dx_step = step * p.dx_pitch;
    for (; row < p.rows; row += step, buf ^= 1, dx += dx_step) {
        // a wait that runs out: the row's sums are of what is there, the error word tells
        tc::mbar_wait(&full[stage], phase, &abort_flag, p.err);
        const T* x = reinterpret_cast<const T*>(ring + (size_t)stage * 2 * row_bytes);
        const T* dy = x + cols;
        const F2 scale = both(rstd), minus_mean = both(-mean);
        F2 c1 = 0, c2 = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int at = (t + i * threads) * V;
            const bool in = FULL || at < cols;
            r.take(i, in ? load<T, V>(x + at) : zero, in ? load<T, V>(dy + at) : zero, minus_mean, scale, c1, c2);
        }
        const int64_t next = row + step;
        if (next < p.rows) {
            mean = p.mean[next];
            rstd = p.rstd[next];
        }
        const float2 own = make_float2(warp_sum(sum_of<V>(c1)), warp_sum(sum_of<V>(c2)));
        if ((t & 31) == 0) slots[buf][t >> 5] = own;
        __syncwarp();
        // the group (named barriers 1 to 15 suffice: 16 groups are warps)
        if (threads > 32) asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "r"(threads) : "memory");
        if (t == 0) fetch(row + kAhead * step, stage);
        if (++stage == kAhead) {
            stage = 0;
            phase ^= 1;
        }
        if (p.dX) {
            const float2 c = sum_slots<WARPS>(slots[buf]);
            const F2 m1 = both(-c.x * p.inv_cols), m2 = both(-c.y * p.inv_cols);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int at = (t + i * threads) * V;
                if (FULL || at < cols) r.put(i, dx + at, m1, m2, scale);
            }
        }
    }
    if (t == 0 && abort_flag) {
        // nothing may land after the block has left: one more wait each for what was asked for
        for (int i = 0; i < kAhead; ++i) {
            tc::mbar_wait_drain(&full[i], 0);
            tc::mbar_wait_drain(&full[i], 1);
        }
    }
    if (!p.partial) return;
    float* const out = p.partial + (int64_t)blockIdx.x * 2 * cols;
    if (groups == 1) {
        r.leave(out, cols, t, threads);
        return;
    }
    __syncthreads();                                 // every row has been read: the rings' memory is free
    r.leave(reinterpret_cast<float*>(rings) + (size_t)grp * 2 * cols, cols, t, threads);
    __syncthreads();
    for (int c = threadIdx.x * 4; c < 2 * cols; c += blockDim.x * 4) {
        float4 a = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(rings) + c);
        for (int g = 1; g < groups; ++g) {
            const float4 b = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(rings) + (size_t)g * 2 * cols + c);
            a.x += b.x;
            a.y += b.y;
            a.z += b.z;
            a.w += b.w;
        }
        *reinterpret_cast<float4*>(out + c) = a;
    }
}

// Rows of 16-byte packs twice as wide: the row stays in the ring until the
// next row's barrier and is read twice, once for the row sums and once for dx
// and the column sums, so that registers hold the column sums alone.
constexpr int kWideThreads = 512, kWideColumns = 32;
template <typename T>
__global__ void __launch_bounds__(kWideThreads) backward_wide_kernel(const BwdParams p, int stages) {
    constexpr int V = 16 / sizeof(T), P = V / 2, NV = kWideColumns / V, WARPS = kWideThreads / 32, MOST = 4;
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ alignas(16) float2 slots[2][WARPS];
    __shared__ uint64_t full[MOST];
    __shared__ int abort_flag;
    const int t = threadIdx.x;
    const int cols = (int)p.cols;
    const uint32_t row_bytes = (uint32_t)cols * sizeof(T);
    if (t == 0) {
        for (int i = 0; i < MOST; ++i) tc::mbar_init(&full[i], 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();
    auto fetch = [&](int64_t row, int stage) {    // one thread
        if (row >= p.rows) return;
        unsigned char* to = ring + (size_t)stage * 2 * row_bytes;
        tc::mbar_arrive_expect_tx(&full[stage], 2 * row_bytes);
        bulk_copy(to, static_cast<const T*>(p.X) + row * p.x_pitch, row_bytes, &full[stage]);
        bulk_copy(to + row_bytes, static_cast<const T*>(p.dY) + row * p.dy_pitch, row_bytes, &full[stage]);
    };
    int64_t row = blockIdx.x;
    if (t == 0)
        for (int i = 0; i < stages; ++i) fetch(row + (int64_t)i * gridDim.x, i);
    F2 ag[NV][P], ab[NV][P];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int q = 0; q < P; ++q) ag[i][q] = ab[i][q] = 0;
    const T* gamma = static_cast<const T*>(p.gamma);
    int stage = 0, phase = 0, buf = 0, last = -1;
    for (; row < p.rows; row += gridDim.x, buf ^= 1) {
        const float mean = p.mean[row], rstd = p.rstd[row];
        tc::mbar_wait(&full[stage], phase, &abort_flag, p.err);
        const T* x = reinterpret_cast<const T*>(ring + (size_t)stage * 2 * row_bytes);
        const T* dy = x + cols;
        const F2 scale = both(rstd), minus_mean = both(-mean);
        auto at_pack = [&](int c, F2 (&xh)[P], F2 (&d)[P], F2 (&dxh)[P]) {
            F2 g[P];
            widen<T, V>(xh, load<T, V>(x + c));
            widen<T, V>(d, load<T, V>(dy + c));
            if (gamma) widen<T, V>(g, load<T, V>(gamma + c));
#pragma unroll
            for (int q = 0; q < P; ++q) {
                xh[q] = mul2(add2(xh[q], minus_mean), scale);
                dxh[q] = gamma ? mul2(d[q], g[q]) : d[q];
            }
        };
        F2 c1 = 0, c2 = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * kWideThreads) * V;
            if (c >= cols) break;
            F2 xh[P], d[P], dxh[P];
            at_pack(c, xh, d, dxh);
#pragma unroll
            for (int q = 0; q < P; ++q) {
                c1 = add2(c1, dxh[q]);
                c2 = fma2(dxh[q], xh[q], c2);
            }
        }
        const float2 own = make_float2(warp_sum(sum_of<2>(c1)), warp_sum(sum_of<2>(c2)));
        if ((t & 31) == 0) slots[buf][t >> 5] = own;
        __syncthreads();
        // every thread is done with the row before this one: its buffer takes another
        if (t == 0 && last >= 0) fetch(row + (int64_t)(stages - 1) * gridDim.x, last);
        last = stage;
        if (++stage == stages) {
            stage = 0;
            phase ^= 1;
        }
        const float2 sums = sum_slots<WARPS>(slots[buf]);
        const F2 m1 = both(-sums.x * p.inv_cols), m2 = both(-sums.y * p.inv_cols);
        T* dx = static_cast<T*>(p.dX) + row * p.dx_pitch;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * kWideThreads) * V;
            if (c >= cols) break;
            F2 xh[P], d[P], dxh[P];
            at_pack(c, xh, d, dxh);
#pragma unroll
            for (int q = 0; q < P; ++q) {
                ag[i][q] = fma2(d[q], xh[q], ag[i][q]);
                ab[i][q] = add2(ab[i][q], d[q]);
                dxh[q] = mul2(add2(fma2(xh[q], m2, dxh[q]), m1), scale);
            }
            if (p.dX) store<T, V>(dx + c, dxh);
        }
    }
    if (t == 0 && abort_flag) {
        // nothing may land after the block has left: one more wait each for what was asked for
        for (int i = 0; i < stages; ++i) {
            tc::mbar_wait_drain(&full[i], 0);
            tc::mbar_wait_drain(&full[i], 1);
        }
    }
    if (!p.partial) return;
    float* out = p.partial + (int64_t)blockIdx.x * 2 * cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (t + i * kWideThreads) * V;
        if (c >= cols) break;
#pragma unroll
        for (int q = 0; q < P; ++q) {
            *reinterpret_cast<F2*>(out + c + 2 * q) = ag[i][q];
            *reinterpret_cast<F2*>(out + cols + c + 2 * q) = ab[i][q];
        }
    }
}

// Rows wider than a block's registers hold: dx alone, two passes over the row.
template <typename T, int V>
__global__ void __launch_bounds__(1024) backward_long_rows_kernel(const BwdParams p) {
    __shared__ float slots[2][32];
    const T* gamma = static_cast<const T*>(p.gamma);
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(p.X) + row * p.x_pitch;
        const T* dy = static_cast<const T*>(p.dY) + row * p.dy_pitch;
        T* dx = static_cast<T*>(p.dX) + row * p.dx_pitch;
        const float mean = p.mean[row], rstd = p.rstd[row];
        const F2 scale = both(rstd), minus_mean = both(-mean);
        RowGrads<T, V, 1> r;
        r.clear();
        F2 s1 = 0, s2 = 0;
        for (int64_t c = (int64_t)threadIdx.x * V; c < p.cols; c += 1024 * V) {
            r.weights(0, gamma ? gamma + c : nullptr);
            r.take(0, load<T, V>(x + c), load<T, V>(dy + c), minus_mean, scale, s1, s2);
        }
        const float c1 = block_sum<32>(sum_of<V>(s1), slots[0]) * p.inv_cols;
        const float c2 = block_sum<32>(sum_of<V>(s2), slots[1]) * p.inv_cols;
        for (int64_t c = (int64_t)threadIdx.x * V; c < p.cols; c += 1024 * V) {
            r.weights(0, gamma ? gamma + c : nullptr);
            r.take(0, load<T, V>(x + c), load<T, V>(dy + c), minus_mean, scale, s1, s2);
            r.put(0, dx + c, both(-c1), both(-c2), scale);
        }
    }
}

// The column sums of such rows: blockIdx.y takes an equal share of the rows,
// a thread one column.
template <typename T>
__global__ void __launch_bounds__(256) backward_long_cols_kernel(const BwdParams p) {
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

// Column sums over the blocks' partial sums, C columns a block: in block order
// within each share of them and then in share order, the same for every run.
template <typename T, int C>
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* __restrict__ partial, int blocks, int64_t cols,
                                                          T* dgamma, T* dbeta) {
    constexpr int SHARES = 1024 / C;
    __shared__ float sums[SHARES][C + 1];
    T* out = blockIdx.y ? dbeta : dgamma;
    if (!out) return;
    const int col = threadIdx.x % C, share = threadIdx.x / C;
    const int64_t c = (int64_t)blockIdx.x * C + col;
    float s = 0.f;
    if (c < cols) {
#pragma unroll 10
        for (int b = share; b < blocks; b += SHARES) s += partial[((int64_t)b * 2 + blockIdx.y) * cols + c];
    }
    sums[share][col] = s;
    __syncthreads();
    // a warp a column
    const int lane = threadIdx.x & 31, mine = threadIdx.x >> 5;
    if (mine >= C) return;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < SHARES / 32; ++i) s += sums[lane + 32 * i][mine];
    s = warp_sum(s);
    const int64_t to = (int64_t)blockIdx.x * C + mine;
    if (lane == 0 && to < cols) out[to] = Num<T>::from_acc(s);
}

// ---- host side -------------------------------------------------------------

// Threads a row: with many rows a thread takes four packs of 16 bytes, so that
// enough of the row is on its way at once and enough blocks reside
// ([16384, 4096] BF16, us: 4 warps x 4 packs 42.4, 8 x 2 46.2, 2 x 8 44.6,
// 16 x 1 69.9, 1 x 16 51.7, persistent warps fed by bulk copies 50.4; a plain
// copy of the tensor 43.5); with few rows more warps share one ([4, 4096] FP16:
// 8 x 2 2.49, 4 x 4 3.17, 2 x 8 4.53).  One warp needs no block barrier.
template <typename T, int V>
cudaError_t forward_as(const FwdParams& p, int sm_count, cudaStream_t s) {
    // single elements go in pairs, twice as many a thread as packs
    const int64_t n = ceil_div(p.cols, V == 1 ? 4 : V);
    constexpr int M = V == 1 ? 2 : 1;
    const bool few = p.rows < 4 * (int64_t)sm_count;
#define OLC_FWD(W, NV)                                                                                          \
    return plan_launch(forward_kernel<T, V, W, NV * M>, dim3((unsigned)(W == 1 ? ceil_div(p.rows, 4) : p.rows)), \
                      dim3(W == 1 ? 128 : W * 32), 0, s, p)
    if (p.rows <= 0x7fffffff) {
        if constexpr (V > 1) {
            // short rows in numbers: a warp takes 8 or more ([100000, 64] BF16: 6.6
            // us, a warp a row 21.3; [100000, 128] 13.8 and 22.6; [100000, 256]
            // would be 24.5 and 23.6)
            if (n <= 16 && p.rows >= 32 * (int64_t)sm_count) {
                auto run = [&](auto kernel, int rows) {
                    return plan_launch(kernel, dim3((unsigned)ceil_div(p.rows, rows)), dim3(128), 0, s, p);
                };
                return n <= 8 ? run(forward_short_kernel<T, 8, 4>, 64) : run(forward_short_kernel<T, 16, 4>, 32);
            }
        }
        if (n <= 32) OLC_FWD(1, 1);
        if (n <= 64) OLC_FWD(1, 2);
        if (n <= 128 && !few) OLC_FWD(1, 4);
        if (n <= 256 && !few) OLC_FWD(2, 4);
        if (n <= 256) OLC_FWD(8, 1);
        if (n <= 512 && !few) OLC_FWD(4, 4);
        if (n <= 512) OLC_FWD(8, 2);
        if (n <= 1024) OLC_FWD(8, 4);
        if (n <= 2048) OLC_FWD(16, 4);
        if (n <= 4096) OLC_FWD(32, 4);
        if (n <= 8192) OLC_FWD(32, 8);
    }
#undef OLC_FWD
    const int64_t grid = min64(p.rows, (int64_t)sm_count * 2);
    return plan_launch(forward_long_kernel<T, V>, dim3((unsigned)grid), dim3(1024), 0, s, p);
}

// Rows of 16-byte packs go through the ring from this width on ([16384, 512]
// BF16: 14.0 us, from registers 21.4; [16384, 256]: 10.8 and 12.6; [16384, 128]:
// 10.8 and 11.4, but [2048, 128] FLOAT 6.3 and 5.1).
constexpr int64_t kRingCols = 256;
// A group takes at least this many rows: more blocks read faster, fewer leave
// fewer partial sums ([608, 4096] BF16: 9.9 us; at least one row 13.1, eight 11.5).
constexpr int64_t kLeastRows = 4;
// Up to this width the column sums are split eight columns a block, above it 32
// ([16384, 1024] BF16 27.0 and 28.0 us, [16384, 4096] 72.4 and 68.9).
constexpr int64_t kNarrowCols = 2048;
constexpr int kRingSmem = kAhead * 2 * 512 * 16 * 4;     // rings of the widest float32 rows
constexpr int64_t kWideSmem = 208 * 1024;   // ring of the wide rows
constexpr int kColsPerThread = 16;      // float32 column sums of dgamma and dbeta: 32 registers

// the backward launch of one shape: which kernel, how many threads
struct BwdShape {
    enum Kind { LONG, WIDE, RING, ANY } kind = LONG;   // LONG: rows wider than a block's registers
    int per_thread = 0;                          // columns
    int tpr = 0, groups = 1, threads = 0;
    int64_t blocks = 0;
};

template <int V>
BwdShape backward_shape(int64_t rows, int64_t cols, int sm_count) {
    BwdShape b;
    constexpr int64_t size = V == 1 ? 0 : 16 / V;
    if (V > 1 && cols > 512 * kColsPerThread && cols <= kWideThreads * kWideColumns &&
        4 * cols * size <= kWideSmem && rows >= kLeastRows * sm_count) {
        // ([4096, 12288] BF16: 83 us, in passes over rows and columns 162; 608 rows
        // 29.5 and 35.4)
        b.kind = BwdShape::WIDE;
        b.blocks = sm_count;
        return b;
    }
    if (cols > 512 * kColsPerThread) {
        b.blocks = min64(max64(rows / 64, 1), max64(1, 8 * (int64_t)sm_count * 256 / cols));
        return b;
    }
    // whole rows of 16-byte packs through the ring, as many groups as rows
    // suffice for ([16384, 4096] BF16: 66.5 us, 403 MB of x, dy and dx at 6.1
    // TB/s; with blocks of one group 68.9; [2048, 1024]: 7.8 and 9.9)
    if (V > 1 && cols >= kRingCols) {
        b.kind = BwdShape::RING;
        b.per_thread = kColsPerThread;
        b.tpr = (int)(ceil_div(ceil_div(cols, kColsPerThread), 32) * 32);
        b.groups = (int)max64(1, min64(512 / b.tpr, ceil_div(rows, kLeastRows * sm_count)));
        b.threads = b.tpr * b.groups;
        // 512 threads an SM, or two blocks of wider rows
        b.blocks = max64(1, min64(ceil_div(rows, kLeastRows * b.groups), (int64_t)sm_count * (b.tpr > 256 ? 2 : 1)));
        return b;
    }
    // packs: fewer than kRingCols columns, so four (FLOAT) or eight a thread
    b.kind = BwdShape::ANY;
    const int least = V == 1 ? 2 : V;            // columns of a pack, or of a pair of single elements
    b.per_thread = least;
    while (b.per_thread < kColsPerThread && cols > 32 * b.per_thread) b.per_thread *= 2;
    b.tpr = (int)(ceil_div(ceil_div(cols, b.per_thread), 32) * 32);
    b.groups = (int)max64(1, min64(512 / b.tpr, ceil_div(2 * rows, sm_count)));
    b.threads = b.tpr * b.groups;
    b.blocks = max64(1, min64(ceil_div(rows, b.groups), (int64_t)sm_count * (b.per_thread > 8 ? 1 : 2)));
    return b;
}

template <typename T, int V, int NV>
cudaError_t backward_rows(const BwdParams& p, const BwdShape& b, cudaStream_t s) {
    const size_t smem = b.groups > 1 ? (size_t)b.groups * p.cols * sizeof(float) : 0;
    return plan_launch(backward_kernel<T, V, NV>, dim3((unsigned)b.blocks), dim3((unsigned)b.threads), smem, s, p);
}

template <typename T, int WARPS, bool FULL>
cudaError_t backward_ring(const BwdParams& p, const BwdShape& b, cudaStream_t s) {
    auto* kernel = backward_ring_kernel<T, kColsPerThread * sizeof(T) / 16, WARPS, FULL>;
    const cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(kernel), kRingSmem);
    if (e != cudaSuccess) return e;
    return plan_launch(kernel, dim3((unsigned)b.blocks), dim3((unsigned)b.threads),
                      b.groups * kAhead * 2 * (size_t)p.cols * sizeof(T), s, p);
}

template <typename T, int V>
cudaError_t backward_as(BwdParams p, int sm_count, T* dgamma, T* dbeta, cudaStream_t s) {
    const BwdShape b = backward_shape<V>(p.rows, p.cols, sm_count);
    cudaError_t e = cudaSuccess;
    p.threads_per_row = b.tpr;
    if (b.kind == BwdShape::LONG) {
        // the column sums first: dX may be dY or X
        if (p.partial)
            e = plan_launch(backward_long_cols_kernel<T>, dim3((unsigned)ceil_div(p.cols, 256), (unsigned)b.blocks),
                           dim3(256), 0, s, p);
        if (e == cudaSuccess && p.dX)
            e = plan_launch(backward_long_rows_kernel<T, V>, dim3((unsigned)min64(p.rows, (int64_t)sm_count * 2)),
                           dim3(1024), 0, s, p);
    } else if (b.kind == BwdShape::WIDE) {
        if constexpr (V > 1) {
            const int64_t row = 2 * p.cols * (int64_t)sizeof(T);
            const int stages = (int)min64(4, kWideSmem / row);
            e = set_smem_limit(reinterpret_cast<const void*>(backward_wide_kernel<T>), (int)kWideSmem);
            if (e == cudaSuccess)
                e = plan_launch(backward_wide_kernel<T>, dim3((unsigned)b.blocks), dim3(kWideThreads),
                               (size_t)(stages * row), s, p, stages);
        }
    } else if (b.kind == BwdShape::RING) {
        if constexpr (V > 1) {
            const bool full = p.cols == (int64_t)b.tpr * kColsPerThread;
            if (b.tpr <= 256)
                e = full ? backward_ring<T, 8, true>(p, b, s) : backward_ring<T, 8, false>(p, b, s);
            else
                e = full ? backward_ring<T, 16, true>(p, b, s) : backward_ring<T, 16, false>(p, b, s);
        }
    } else if (b.per_thread == 8) {
        e = backward_rows<T, V, V == 1 ? 4 : 8 / V>(p, b, s);
    } else if constexpr (V == 1) {
        e = b.per_thread == 16 ? backward_rows<T, 1, 8>(p, b, s)
                               : (b.per_thread == 4 ? backward_rows<T, 1, 2>(p, b, s) : backward_rows<T, 1, 1>(p, b, s));
    } else if constexpr (V == 4) {
        e = backward_rows<T, 4, 1>(p, b, s);
    }
    if (e == cudaSuccess && p.partial) {
        auto run = [&](auto kernel, int c) {
            return plan_launch(kernel, dim3((unsigned)ceil_div(p.cols, c), 2), dim3(1024), 0, s,
                               (const float*)p.partial, (int)b.blocks, p.cols, dgamma, dbeta);
        };
        e = p.cols <= kNarrowCols ? run(column_sum_kernel<T, 8>, 8) : run(column_sum_kernel<T, 32>, 32);
    }
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
                      (float)plan->cols, (float)(1.0 / (double)plan->cols)};
    // 16-byte packs need every row of every operand on a 16-byte boundary
    const bool wide = plan->cols * eb % 16 == 0 && plan_aligned16(X) && plan_aligned16(Y) && plan_aligned16(gamma) &&
                      plan_aligned16(beta) && (plan->rows == 1 || (x_pitch * eb % 16 == 0 && y_pitch * eb % 16 == 0));
    return by_type(plan->dtype, [&](auto tag) {
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
                      (float)(1.0 / (double)cols), 0, device_error_word()};
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
    }
    return by_type(plan->dtype, [&](auto tag) {
        using T = decltype(tag);
        T *dg = static_cast<T*>(dgamma), *db = static_cast<T*>(dbeta);
        auto run = [&] {
            return wide ? norm::backward_as<T, 16 / sizeof(T)>(p, plan->state.sm_count, dg, db, s)
                        : norm::backward_as<T, 1>(p, plan->state.sm_count, dg, db, s);
        };
        return plan_status(weights ? plan->state.use(s, run) : run());
    });
}

}  // extern "C"
