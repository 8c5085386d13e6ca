// The step between two blocks of a model, with its norms:
//
//   n = norm(f) ag + ab  (or n = f),   y = x + scale gate n,   z = norm(y) g + b
//
// forward and backward.  Backward, with hats for the normalised rows, J' of a
// norm being v -> rstd (v - mean(v) - hat mean(v hat)) (without mean(v) for RMS):
//
//   dx = dY + J_y'(dZ g),  dn = scale gate dx,  df = J_f'(dn ag),  dgate = scale n dx
//   dg = sum dZ yhat, db = sum dZ, dag = sum dn fhat, dab = sum dn   (over the rows)
//
// Four tensors move forward, six backward (one or two more with a gate for each
// element), with 20 to 40 operations an element: the bytes bound both.  A row is
// read once and stays in registers from its first sum to its last use; rows wider
// than that are read again.  Statistics and sums are float32; a mean is corrected by
// the sum of the distances from it, in the same pass as the squares (Chan, Golub and
// LeVeque's two-pass algorithm), so that rows far from zero keep their digits.
//
// BF16 [16384, 4096], an RMS norm before and one after: forward 84 us (0.96 of the copy
// rate); backward 138 us with both dgammas (0.88), of which the rows take 128 (issue
// slots 54 %, 128 registers a thread) and the column sums 8.  Few rows: one launch
// forward (3 us), two backward.  Rows without 16-byte packs are bound by their accesses'
// number: FLOAT [2049, 1001] backward 29 us.
#include <new>
#include <type_traits>

#include "plan_state.h"
#include "row_packs.cuh"

namespace olc {
namespace residual {

struct FwdParams {
    const void* X;
    const void* F;
    const void* gate;       // may be null: 1
    const void* ag;         // weights of the norm of f; may be null: 1, 0
    const void* ab;
    const void* g;          // weights of the norm of y; may be null: 1, 0
    const void* b;
    void* Y;
    void* Z;                // may be null
    float* stats;           // may be null
    int64_t x_pitch, f_pitch, gate_pitch, y_pitch, z_pitch;
    int64_t rows, cols;
    float eps, scale, inv_cols;
    int after, rms;
};

enum Sum { DG = 0, DB, DAG, DAB, DGATE, SUMS };

struct BwdParams {
    const void* dY;         // may be null: 0
    const void* dZ;         // may be null: no norm of y
    const void* F;
    const void* Y;
    const float* stats;
    const void* gate;       // may be null: 1
    const void* ag;
    const void* ab;
    const void* g;
    void* dX;               // may be null
    void* dF;               // may be null
    void* dgate;            // of each element; may be null
    float* partial;         // [blocks][SUMS][cols]: what a block adds to each column sum; null: none is wanted
    float* row_sums;        // [4][rows]: the means that J of y and of f subtract (rows wider than a block)
    int64_t dy_pitch, dz_pitch, f_pitch, y_pitch, gate_pitch, dx_pitch, df_pitch, dgate_pitch;
    int64_t rows, cols;
    float scale, inv_cols;
    int after, rms, channel_gate_sum;
    int threads_per_row;
    unsigned int* err;
};

// sums of two values over the W warps of a block; every thread gets them.
// Consecutive calls take different slots.
template <int W>
__device__ __forceinline__ float2 block_sums(float2 v, float2* slot) {
    v.x = warp_sum(v.x);
    v.y = warp_sum(v.y);
    if constexpr (W == 1) return v;
    if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
    __syncthreads();
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < W; ++i) {
        s.x += slot[i].x;
        s.y += slot[i].y;
    }
    return s;
}

struct Stats {
    float mean, rstd;
};
// from the sums of the squared distances and of the distances from `mean`
__device__ __forceinline__ Stats stats_of(float mean, float2 sums, const FwdParams& p) {
    const float shift = p.rms ? 0.f : sums.y * p.inv_cols;
    float squares = p.rms ? sums.x : fmaf(-sums.y, shift, sums.x);
    if (squares < 0.f) squares = 0.f;       // NaN stays
    return Stats{mean + shift, 1.0f / sqrtf(fmaf(squares, p.inv_cols, p.eps))};
}

// A thread's columns as packs that stay the words they were loaded as until they
// are widened (arrays of 16-bit elements cost moves and registers: [16384, 4096] BF16
// 96.7 us, so 79.6).
template <typename T, int V>
struct Words {
    static constexpr int P = V / 2;
    using Raw = uint4;
    static __device__ __forceinline__ bool in(int base, int i, int, int stride, int cols) {
        return (base + i * stride) * V < cols;
    }
    static __device__ __forceinline__ Raw read(const T* row, int base, int i, int stride, int cols, bool, bool) {
        if (in(base, i, 0, stride, cols)) return *reinterpret_cast<const uint4*>(row + (base + i * stride) * V);
        return uint4{0, 0, 0, 0};
    }
    static __device__ __forceinline__ void pairs_of(F2 (&out)[P], const Raw& r) {
        widen<T, V>(out, *reinterpret_cast<const Pack<T, V>*>(&r));
    }
    static __device__ __forceinline__ F2 inside(F2 v, int base, int i, int, int stride, int cols, bool) {
        return in(base, i, 0, stride, cols) ? v : 0;
    }
    static __device__ __forceinline__ void write(T* row, int base, int i, int stride, int cols, const F2 (&o)[P], bool) {
        if (in(base, i, 0, stride, cols)) store<T, V>(row + (base + i * stride) * V, o);
    }
};

// W warps on a row, NV packs (or pairs of elements) a thread, in registers.
// W == 1: blocks of four independent warps.
template <typename T, int V, int W, int NV>
__global__ void __launch_bounds__(W == 1 ? 128 : W * 32, V > 2 && W == 4 && NV == 4 ? 7 : 0) forward_kernel(const FwdParams p) {
    using C = std::conditional_t<(V <= 2), Columns<T, V>, Words<T, V <= 2 ? 4 : V>>;
    constexpr int P = C::P, TPR = W * 32;
    __shared__ float slots1[2][W];
    __shared__ float2 slots2[2][W];
    const int t = W == 1 ? (threadIdx.x & 31) : threadIdx.x;
    const int64_t row = W == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
    if (row >= p.rows) return;      // whole warps (W == 1); never with W > 1
    const T* x = static_cast<const T*>(p.X) + row * p.x_pitch;
    const T* f = static_cast<const T*>(p.F) + row * p.f_pitch;
    const int cols = (int)p.cols, whole = V == 1 && W > 1 ? cols / (2 * TPR) : 0;
    auto read = [&](const void* from, int i) {
        return C::read(static_cast<const T*>(from), t, i, TPR, cols, true, i < whole);
    };
    typename C::Raw kx[NV], kf[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) kf[i] = read(f, i);
#pragma unroll
    for (int i = 0; i < NV; ++i) kx[i] = read(x, i);

    F2 y[NV][P];                     // f, then n, then y, then z
    // the statistics of what y holds; columns past the row's end hold zeros
    auto statistics = [&](int k) {
        float mean = 0.f;
        if (!p.rms) {
            F2 s = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int q = 0; q < P; ++q) s = add2(s, y[i][q]);
            mean = block_sum<W>(sum_of<2>(s), slots1[k]) * p.inv_cols;
        }
        const F2 minus_mean = both(-mean);
        F2 squares = 0, distances = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int q = 0; q < P; ++q) {
                const F2 d = C::inside(add2(y[i][q], minus_mean), t, i, q, TPR, cols, i < whole);
                squares = fma2(d, d, squares);
                distances = add2(distances, d);
            }
        return stats_of(mean, block_sums<W>(make_float2(sum_of<2>(squares), sum_of<2>(distances)), slots2[k]), p);
    };
    auto normalise = [&](Stats s, const void* weight, const void* bias) {
        const F2 minus_mean = both(-s.mean), scale = both(s.rstd);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int q = 0; q < P; ++q) y[i][q] = mul2(add2(y[i][q], minus_mean), scale);
            F2 w[P];
            if (weight) {
                C::pairs_of(w, read(weight, i));
#pragma unroll
                for (int q = 0; q < P; ++q) y[i][q] = mul2(y[i][q], w[q]);
            }
            if (bias) {
                C::pairs_of(w, read(bias, i));
#pragma unroll
                for (int q = 0; q < P; ++q) y[i][q] = add2(y[i][q], w[q]);
            }
        }
    };
    auto keep = [&](Stats s, int k) {
        if (p.stats && t == 0) {
            p.stats[2 * k * p.rows + row] = s.mean;
            p.stats[(2 * k + 1) * p.rows + row] = s.rstd;
        }
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) C::pairs_of(y[i], kf[i]);
    if (p.after) {
        const Stats s = statistics(0);
        keep(s, 1);
        normalise(s, p.ag, p.ab);
    }
    const F2 scale = both(p.scale);
    const T* gate = static_cast<const T*>(p.gate) + (p.gate ? row * p.gate_pitch : 0);
    T* out = static_cast<T*>(p.Y) + row * p.y_pitch;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        F2 v[P], w[P];
        C::pairs_of(v, kx[i]);
        if (p.gate) C::pairs_of(w, read(gate, i));
#pragma unroll
        for (int q = 0; q < P; ++q)
            y[i][q] = C::inside(fma2(p.gate ? mul2(scale, w[q]) : scale, y[i][q], v[q]), t, i, q, TPR, cols, i < whole);
        C::write(out, t, i, TPR, cols, y[i], i < whole);
    }
    if (!p.Z) return;
    const Stats s = statistics(1);
    keep(s, 0);
    normalise(s, p.g, p.b);
    T* z = static_cast<T*>(p.Z) + row * p.z_pitch;
#pragma unroll
    for (int i = 0; i < NV; ++i) C::write(z, t, i, TPR, cols, y[i], i < whole);
}

// Rows longer than the registers of a block hold: each step reads the row again.
template <typename T, int V>
__global__ void __launch_bounds__(1024) forward_long_kernel(const FwdParams p) {
    constexpr int P = pairs<V>();
    __shared__ float slots1[2][32];
    __shared__ float2 slots2[2][32];
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(p.X) + row * p.x_pitch;
        const T* f = static_cast<const T*>(p.F) + row * p.f_pitch;
        const T* gate = static_cast<const T*>(p.gate) + (p.gate ? row * p.gate_pitch : 0);
        auto affine = [&](F2 (&v)[P], Stats s, const void* weight, const void* bias, int64_t c) {
            F2 w[P];
#pragma unroll
            for (int q = 0; q < P; ++q) v[q] = mul2(add2(v[q], both(-s.mean)), both(s.rstd));
            if (weight) {
                widen<T, V>(w, load<T, V>(static_cast<const T*>(weight) + c));
#pragma unroll
                for (int q = 0; q < P; ++q) v[q] = mul2(v[q], w[q]);
            }
            if (bias) {
                widen<T, V>(w, load<T, V>(static_cast<const T*>(bias) + c));
#pragma unroll
                for (int q = 0; q < P; ++q) v[q] = add2(v[q], w[q]);
            }
        };
        auto statistics = [&](int k, auto&& value) {
            float mean = 0.f;
            F2 v[P];
            if (!p.rms) {
                F2 s = 0;
                for (int64_t c = (int64_t)threadIdx.x * V; c < p.cols; c += 1024 * V) {
                    value(v, c);
#pragma unroll
                    for (int q = 0; q < P; ++q) s = add2(s, v[q]);
                }
                mean = block_sum<32>(sum_of<V>(s), slots1[k]) * p.inv_cols;
            }
            F2 squares = 0, distances = 0;
            for (int64_t c = (int64_t)threadIdx.x * V; c < p.cols; c += 1024 * V) {
                value(v, c);
#pragma unroll
                for (int q = 0; q < P; ++q) {
                    const F2 d = add2(v[q], both(-mean));
                    squares = fma2(d, d, squares);
                    distances = add2(distances, d);
                }
            }
            const Stats s = stats_of(mean, block_sums<32>(make_float2(sum_of<V>(squares), sum_of<V>(distances)), slots2[k]), p);
            if (p.stats && threadIdx.x == 0) {
                p.stats[(k ? 0 : 2) * p.rows + row] = s.mean;
                p.stats[(k ? 1 : 3) * p.rows + row] = s.rstd;
            }
            return s;
        };
        auto of_f = [&](F2 (&v)[P], int64_t c) { widen<T, V>(v, load<T, V>(f + c)); };
        Stats sf{0.f, 1.f};
        if (p.after) sf = statistics(0, of_f);
        auto of_y = [&](F2 (&v)[P], int64_t c) {
            F2 w[P];
            of_f(v, c);
            if (p.after) affine(v, sf, p.ag, p.ab, c);
            if (p.gate) {
                widen<T, V>(w, load<T, V>(gate + c));
#pragma unroll
                for (int q = 0; q < P; ++q) w[q] = mul2(both(p.scale), w[q]);
            }
            F2 u[P];
            widen<T, V>(u, load<T, V>(x + c));
#pragma unroll
            for (int q = 0; q < P; ++q) v[q] = fma2(p.gate ? w[q] : both(p.scale), v[q], u[q]);
        };
        Stats sy{0.f, 1.f};
        if (p.Z) sy = statistics(1, of_y);
        for (int64_t c = (int64_t)threadIdx.x * V; c < p.cols; c += 1024 * V) {
            F2 v[P];
            of_y(v, c);
            store<T, V>(static_cast<T*>(p.Y) + row * p.y_pitch + c, v);
            if (p.Z) {
                affine(v, sy, p.g, p.b, c);
                store<T, V>(static_cast<T*>(p.Z) + row * p.z_pitch + c, v);
            }
        }
        __syncthreads();             // the slots serve the next row
    }
}

// ---- backward -----------------------------------------------------------------

// What a thread holds of a row: P pairs of columns.  The steps are the same for
// rows in registers and for rows read again.
template <int P>
struct Grads {
    F2 yh[P], dz[P];        // yhat; dZ g
    F2 fh[P], dn[P];        // fhat (or f); dn, then dn ag
};

template <int P>
__device__ __forceinline__ void add_products(F2& s1, F2& s2, const F2 (&a)[P], const F2 (&b)[P]) {
#pragma unroll
    for (int q = 0; q < P; ++q) {
        s1 = add2(s1, a[q]);
        s2 = fma2(a[q], b[q], s2);
    }
}
// v -> rstd (v - m1 - hat m2), added to `to`
template <int P>
__device__ __forceinline__ void add_through_norm(F2 (&to)[P], const F2 (&v)[P], const F2 (&hat)[P], F2 minus_m1,
                                                 F2 minus_m2, F2 rstd) {
#pragma unroll
    for (int q = 0; q < P; ++q) to[q] = fma2(add2(fma2(hat[q], minus_m2, v[q]), minus_m1), rstd, to[q]);
}

// A block is `groups` groups of threads_per_row threads; a thread keeps the same
// columns (16 bytes of 16-bit types; eight of FLOAT) of every row its group
// takes, so that the column sums stay in its registers until the block's last row; the groups'
// sums are then added in group order.  The next row's loads are on their way while
// this one's two row sums (one after the other: the second needs dx) are formed.
constexpr int kColsPerThread = 8;
constexpr int kThreads = 512;
template <typename T, int V, int NV>
__global__ void __launch_bounds__(kThreads) backward_kernel(const BwdParams p) {
    using C = Columns<T, V>;
    constexpr int P = C::P, Q = NV * P;
    extern __shared__ float shared[];
    __shared__ alignas(16) float2 slots[4][16];
    const int tpr = p.threads_per_row;
    const int groups = blockDim.x / tpr, warps = tpr >> 5;
    const int grp = threadIdx.x / tpr, t = threadIdx.x - grp * tpr;
    const int cols = (int)p.cols;
    // single elements: a warp's columns lie together, so that their offsets are constants
    const int warp_base = (t >> 5) * (64 * NV);
    const int base = V == 1 ? warp_base + (t & 31) : t, stride = V == 1 ? 32 : tpr;
    const int whole = V == 1 ? (cols - warp_base) / 64 : 0;
    struct Raw {
        typename C::Raw r[NV];
    };
    auto read = [&](Raw& k, const void* from, int64_t at, bool live) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            k.r[i] = C::read(static_cast<const T*>(from) + at, base, i, stride, cols, live, i < whole);
    };
    auto widen_all = [&](F2 (&out)[Q], const Raw& k) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            F2 v[P];
            C::pairs_of(v, k.r[i]);
#pragma unroll
            for (int q = 0; q < P; ++q) out[i * P + q] = v[q];
        }
    };
    auto weights = [&](F2 (&out)[Q], const void* from, float none) {
        if (!from) {
#pragma unroll
            for (int q = 0; q < Q; ++q) out[q] = both(none);
            return;
        }
        Raw k;
        read(k, from, 0, true);
        widen_all(out, k);
    };
    auto write = [&](void* to, int64_t at, const F2 (&v)[Q]) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            F2 o[P];
#pragma unroll
            for (int q = 0; q < P; ++q) o[q] = v[i * P + q];
            C::write(static_cast<T*>(to) + at, base, i, stride, cols, o, i < whole);
        }
    };
    F2 sums[SUMS][Q];
#pragma unroll
    for (int k = 0; k < SUMS; ++k)
#pragma unroll
        for (int q = 0; q < Q; ++q) sums[k][q] = 0;
    const bool need_f = p.after || p.dgate || p.channel_gate_sum;
    Raw kdy{}, kdz{}, kf{}, ky{}, kg{};
    Stats sy{0.f, 0.f}, sf{0.f, 0.f};
    // columns past a row's end, and rows past the last one, have gradients of 0 and add nothing
    auto fetch = [&](int64_t row) {
        const bool live = row < p.rows;
        if (p.dZ) {
            read(kdz, p.dZ, row * p.dz_pitch, live);
            read(ky, p.Y, row * p.y_pitch, live);
            sy = live ? Stats{p.stats[row], p.stats[p.rows + row]} : Stats{0.f, 0.f};
        }
        if (p.dY) read(kdy, p.dY, row * p.dy_pitch, live);
        if (need_f) read(kf, p.F, row * p.f_pitch, live);
        if (p.after) sf = live ? Stats{p.stats[2 * p.rows + row], p.stats[3 * p.rows + row]} : Stats{0.f, 0.f};
        if (p.gate && p.gate_pitch) read(kg, p.gate, row * p.gate_pitch, live);
    };
    auto row_means = [&](F2 s1, F2 s2, int slot) {
        float2 c = make_float2(warp_sum(sum_of<2>(s1)), warp_sum(sum_of<2>(s2)));
        if (warps > 1) {
            if ((threadIdx.x & 31) == 0) slots[slot][threadIdx.x >> 5] = c;
            __syncthreads();
            c = make_float2(0.f, 0.f);
            for (int w = 0; w < warps; ++w) {
                const float2 v = slots[slot][grp * warps + w];
                c.x += v.x;
                c.y += v.y;
            }
        }
        if (p.rms) c.x = 0.f;
        return make_float2(-c.x * p.inv_cols, -c.y * p.inv_cols);
    };
    const int64_t step = (int64_t)gridDim.x * groups;
    int64_t row = (int64_t)blockIdx.x * groups + grp;
    fetch(row);
    int buf = 0;
    // every group runs the same number of turns: the barriers are the block's
    for (int64_t first = (int64_t)blockIdx.x * groups; first < p.rows; first += step, row += step, buf ^= 2) {
        const bool live = row < p.rows;
        F2 dx[Q], w[Q];
        widen_all(dx, kdy);                           // zeros without dY
        if (p.dZ) {
            F2 dz[Q], yh[Q];
            widen_all(dz, kdz);
            widen_all(yh, ky);
            const F2 rstd = both(sy.rstd), minus_mean = both(-sy.mean);
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                yh[q] = mul2(add2(yh[q], minus_mean), rstd);
                sums[DG][q] = fma2(dz[q], yh[q], sums[DG][q]);
                sums[DB][q] = add2(sums[DB][q], dz[q]);
            }
            if (p.g) {
                weights(w, p.g, 1.f);
#pragma unroll
                for (int q = 0; q < Q; ++q) dz[q] = mul2(dz[q], w[q]);
            }
            F2 s1 = 0, s2 = 0;
            add_products<Q>(s1, s2, dz, yh);
            const float2 m = row_means(s1, s2, buf);
            add_through_norm<Q>(dx, dz, yh, both(m.x), both(m.y), rstd);
#pragma unroll
            for (int q = 0; q < Q; ++q) dx[q] = C::inside(dx[q], base, q / P, q % P, stride, cols, q / P < whole);
        }
        F2 f[Q], gate[Q];
        widen_all(f, kf);
        if (p.gate && p.gate_pitch) {
            widen_all(gate, kg);
        } else {
            weights(gate, p.gate, 1.f);
        }
        const Stats now = sf;
        fetch(row + step);
        if (live && p.dX) write(p.dX, row * p.dx_pitch, dx);
        const F2 scale = both(p.scale), rstd = both(now.rstd), minus_mean = both(-now.mean);
        if (p.after) {
#pragma unroll
            for (int q = 0; q < Q; ++q) f[q] = mul2(add2(f[q], minus_mean), rstd);
        }
        if (p.dgate || p.channel_gate_sum) {
            F2 n[Q];
#pragma unroll
            for (int q = 0; q < Q; ++q) n[q] = f[q];
            if (p.after) {
                weights(w, p.ag, 1.f);
#pragma unroll
                for (int q = 0; q < Q; ++q) n[q] = mul2(n[q], w[q]);
                weights(w, p.ab, 0.f);
#pragma unroll
                for (int q = 0; q < Q; ++q) n[q] = add2(n[q], w[q]);
            }
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                n[q] = mul2(mul2(n[q], scale), dx[q]);
                sums[DGATE][q] = add2(sums[DGATE][q], n[q]);
            }
            if (live && p.dgate) write(p.dgate, row * p.dgate_pitch, n);
        }
        if (!p.after && !p.dF) continue;              // uniform over the grid
        F2 dn[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) dn[q] = mul2(mul2(scale, gate[q]), dx[q]);
        if (p.after) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                sums[DAG][q] = fma2(dn[q], f[q], sums[DAG][q]);
                sums[DAB][q] = add2(sums[DAB][q], dn[q]);
            }
            if (!p.dF) continue;
            if (p.ag) {
                weights(w, p.ag, 1.f);
#pragma unroll
                for (int q = 0; q < Q; ++q) dn[q] = mul2(dn[q], w[q]);
            }
            F2 s1 = 0, s2 = 0;
            add_products<Q>(s1, s2, dn, f);
            const float2 m = row_means(s1, s2, buf + 1);
            F2 df[Q];
#pragma unroll
            for (int q = 0; q < Q; ++q) df[q] = 0;
            add_through_norm<Q>(df, dn, f, both(m.x), both(m.y), rstd);
            if (live) write(p.dF, row * p.df_pitch, df);
        } else if (live) {
            write(p.dF, row * p.df_pitch, dn);
        }
    }
    if (!p.partial) return;
    float* out = p.partial + (int64_t)blockIdx.x * SUMS * cols;
#pragma unroll
    for (int which = 0; which < SUMS; ++which) {
        if (groups > 1) __syncthreads();
        float* to = groups > 1 ? shared + grp * cols : out + which * cols;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int q = 0; q < P; ++q) {
                float v[2];
                unpack_f2(sums[which][i * P + q], v[0], v[1]);
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

// Rows of 16-byte packs: a group of threads takes one row at a time, its operands
// copied ahead into the group's own ring by bulk copies.  A row has two pairs of row sums,
// one after the other; with 16 columns a thread two rows of 4096 share an SM, and one
// works while the other waits for its sums.  The sums of the biases and of a channel's
// gate do not fit beside that: with them (ALL) a thread has 8 columns.
// The second barrier of a row also tells that every thread has read it: its buffer
// takes another.  The groups' column sums are joined in group order.
constexpr int kMaxGroups = 15;        // named barriers
constexpr int kMaxAhead = 4;
constexpr int kRingSmem = 212 * 1024;
// FULL: every thread has NV packs.  The weights lie in shared memory: what the ring leaves of the L1 cache does not hold them.
template <typename T, int NV, bool ALL, bool GATED, bool FULL>
__global__ void __launch_bounds__(kThreads) backward_ring_kernel(const BwdParams p, int ahead) {
    constexpr int V = 16 / sizeof(T), P = V / 2, Q = NV * P, N = ALL ? SUMS : 2, WARPS = kThreads / 32;
    extern __shared__ __align__(128) unsigned char memory[];
    __shared__ alignas(16) float all_slots[kMaxGroups][2][2][2][WARPS];     // [buffer][norm][sum]; those of absent warps hold 0
    __shared__ uint64_t all_full[kMaxGroups][kMaxAhead];
    __shared__ int abort_flag;
    const int threads = p.threads_per_row, groups = blockDim.x / threads;
    const int grp = threadIdx.x / threads, t = threadIdx.x - grp * threads;
    const int cols = (int)p.cols;
    const bool need_f = p.after || (GATED && (p.dgate || p.channel_gate_sum)), gate_rows = GATED && p.gate && p.gate_pitch;
    const uint32_t row_bytes = (uint32_t)cols * sizeof(T);
    const int at_dy = p.dZ ? 2 : 0, at_f = at_dy + (p.dY ? 1 : 0), at_gate = at_f + need_f, operands = at_gate + gate_rows;
    const uint32_t stage_bytes = operands * row_bytes;
    // the weights first: g, ag, and with a gate ab and one that all rows share
    T* const weights = reinterpret_cast<T*>(memory);
    const void* const given[4] = {p.g, p.after ? p.ag : nullptr, GATED && p.gate && p.after ? p.ab : nullptr,
                                  GATED && !gate_rows ? p.gate : nullptr};
    const T* w_at[4];
    int held = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        w_at[k] = nullptr;
        if (!given[k]) continue;
        for (int c = threadIdx.x * V; c < cols; c += blockDim.x * V)
            *reinterpret_cast<Pack<T, V>*>(weights + held * cols + c) = load<T, V>(static_cast<const T*>(given[k]) + c);
        w_at[k] = weights + held++ * cols;
    }
    unsigned char* const rings = memory + (size_t)held * row_bytes;
    unsigned char* const ring = rings + (size_t)grp * ahead * stage_bytes;
    uint64_t* const full = all_full[grp];
    float(&slots)[2][2][2][WARPS] = all_slots[grp];
    if (threadIdx.x == 0) abort_flag = 0;
    for (int i = threadIdx.x; i < kMaxGroups * 8 * WARPS; i += blockDim.x) (&all_slots[0][0][0][0][0])[i] = 0.f;
    if (t == 0) {
        for (int i = 0; i < ahead; ++i) tc::mbar_init(&full[i], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();
    auto fetch = [&](int64_t row, int stage) {    // one thread
        if (row >= p.rows) return;
        unsigned char* to = ring + (size_t)stage * stage_bytes;
        tc::mbar_arrive_expect_tx(&full[stage], stage_bytes);
        auto copy = [&](int k, const void* from, int64_t pitch) {
            bulk_copy(to + (size_t)k * row_bytes, static_cast<const T*>(from) + row * pitch, row_bytes, &full[stage]);
        };
        if (p.dZ) {
            copy(0, p.dZ, p.dz_pitch);
            copy(1, p.Y, p.y_pitch);
        }
        if (p.dY) copy(at_dy, p.dY, p.dy_pitch);
        if (need_f) copy(at_f, p.F, p.f_pitch);
        if (gate_rows) copy(at_gate, p.gate, p.gate_pitch);
    };
    const int64_t step = (int64_t)gridDim.x * groups;
    int64_t row = (int64_t)blockIdx.x * groups + grp;
    if (t == 0)
        for (int i = 0; i < ahead; ++i) fetch(row + i * step, i);
    F2 sums[N][Q];
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int q = 0; q < Q; ++q) sums[k][q] = 0;
    constexpr int OF_AG = ALL ? (int)DAG : 1;
    // (a thread's packs, zeros past the row's end)
    struct Raw {
        uint4 k[NV];
    };
    auto fetch_raw = [&](const void* from) {
        Raw r{};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * threads) * V;
            if (FULL || c < cols) r.k[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(from) + c);
        }
        return r;
    };
    auto widen_raw = [&](F2 (&out)[Q], const Raw& r) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            F2 v[P];
            widen<T, V>(v, *reinterpret_cast<const Pack<T, V>*>(&r.k[i]));
#pragma unroll
            for (int q = 0; q < P; ++q) out[i * P + q] = v[q];
        }
    };
    auto get = [&](F2 (&out)[Q], const void* from) { widen_raw(out, fetch_raw(from)); };
    auto put = [&](void* to, int64_t at, const F2 (&v)[Q]) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * threads) * V;
            F2 o[P];
#pragma unroll
            for (int q = 0; q < P; ++q) o[q] = v[i * P + q];
            if (FULL || c < cols) store<T, V>(static_cast<T*>(to) + at + c, o);
        }
    };
    auto barrier = [&] {                          // the group
        __syncwarp();
        if (threads > 32) asm volatile("bar.sync %0, %1;" ::"r"(1 + grp), "r"(threads) : "memory");
    };
    // the two sums over the row, over its columns
    auto row_means = [&](F2 s1, F2 s2, float (&slots)[2][WARPS]) {
        // half of the lanes go on with one of the sums each
        const int lane = t & 31;
        const float a = sum_of<2>(s1), b = sum_of<2>(s2);
        float v = (lane & 16 ? b : a) + __shfl_xor_sync(0xffffffffu, lane & 16 ? a : b, 16);
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        if ((lane & 15) == 0) slots[lane >> 4][t >> 5] = v;
        barrier();
        float c[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            F2 s = 0;
#pragma unroll
            for (int w = 0; w < WARPS; w += 4) {
                const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(&slots[k][w]);
                s = add2(add2(s, x.x), x.y);
            }
            c[k] = sum_of<2>(s);
        }
        return make_float2(p.rms ? 0.f : -c[0] * p.inv_cols, -c[1] * p.inv_cols);
    };
    int stage = 0, phase = 0, buf = 0;
    auto stats_at = [&](int64_t r, int k) {
        return r < p.rows ? Stats{p.stats[2 * k * p.rows + r], p.stats[(2 * k + 1) * p.rows + r]} : Stats{0.f, 0.f};
    };
    Stats sy{0.f, 0.f}, sf{0.f, 0.f};
    if (p.dZ) sy = stats_at(row, 0);
    if (p.after) sf = stats_at(row, 1);
    for (; row < p.rows; row += step, buf ^= 1) {
        // a wait that runs out: the row's sums are of what is there, the error word tells
        tc::mbar_wait(&full[stage], phase, &abort_flag, p.err);
        const T* in = reinterpret_cast<const T*>(ring + (size_t)stage * stage_bytes);
        F2 dx[Q];
        Raw raw_f{};
        if (p.dZ) {
            F2 dz[Q], yh[Q];
            get(dz, in);
            get(yh, in + cols);
            const F2 rstd = both(sy.rstd), minus_mean = both(-sy.mean);
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                yh[q] = mul2(add2(yh[q], minus_mean), rstd);
                sums[DG][q] = fma2(dz[q], yh[q], sums[DG][q]);
                if constexpr (ALL) sums[DB][q] = add2(sums[DB][q], dz[q]);
            }
            if (w_at[0]) {
                F2 w[Q];
                get(w, w_at[0]);
#pragma unroll
                for (int q = 0; q < Q; ++q) dz[q] = mul2(dz[q], w[q]);
            }
            F2 s1 = 0, s2 = 0;
            add_products<Q>(s1, s2, dz, yh);
            sy = stats_at(row + step, 0);
            Raw dy{};                              // on their way during the sums
            if (p.dY) dy = fetch_raw(in + at_dy * cols);
            if (need_f) raw_f = fetch_raw(in + at_f * cols);
            const float2 m = row_means(s1, s2, slots[buf][0]);
            widen_raw(dx, dy);
            add_through_norm<Q>(dx, dz, yh, both(m.x), both(m.y), rstd);
#pragma unroll
            for (int q = 0; q < Q; ++q)
                if (!FULL && (t + q / P * threads) * V >= cols) dx[q] = 0;
        } else {
            get(dx, in + at_dy * cols);
            if (need_f) raw_f = fetch_raw(in + at_f * cols);
        }
        if (p.dX) put(p.dX, row * p.dx_pitch, dx);
        F2 f[Q], dn[Q];
        widen_raw(f, raw_f);
        const F2 scale = both(p.scale), rstd = both(sf.rstd);
        if (p.after) {
            const F2 minus_mean = both(-sf.mean);
#pragma unroll
            for (int q = 0; q < Q; ++q) f[q] = mul2(add2(f[q], minus_mean), rstd);
            sf = stats_at(row + step, 1);
        }
        const bool gated = gate_rows || w_at[3];
        if (gated) get(dn, gate_rows ? in + at_gate * cols : w_at[3]);
#pragma unroll
        for (int q = 0; q < Q; ++q) dn[q] = mul2(gated ? mul2(scale, dn[q]) : scale, dx[q]);
        if (GATED && (p.dgate || p.channel_gate_sum)) {
            F2 n[Q], w[Q];
#pragma unroll
            for (int q = 0; q < Q; ++q) n[q] = f[q];
            if (w_at[1]) {
                get(w, w_at[1]);
#pragma unroll
                for (int q = 0; q < Q; ++q) n[q] = mul2(n[q], w[q]);
            }
            if (w_at[2]) {
                get(w, w_at[2]);
#pragma unroll
                for (int q = 0; q < Q; ++q) n[q] = add2(n[q], w[q]);
            }
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                n[q] = mul2(mul2(n[q], scale), dx[q]);
                if constexpr (ALL) sums[DGATE][q] = add2(sums[DGATE][q], n[q]);
            }
            if (p.dgate) put(p.dgate, row * p.dgate_pitch, n);
        }
        float2 m = make_float2(0.f, 0.f);
        if (p.after) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                sums[OF_AG][q] = fma2(dn[q], f[q], sums[OF_AG][q]);
                if constexpr (ALL) sums[DAB][q] = add2(sums[DAB][q], dn[q]);
            }
            if (w_at[1]) {
                F2 w[Q];
                get(w, w_at[1]);
#pragma unroll
                for (int q = 0; q < Q; ++q) dn[q] = mul2(dn[q], w[q]);
            }
            F2 s1 = 0, s2 = 0;
            add_products<Q>(s1, s2, dn, f);
            m = row_means(s1, s2, slots[buf][1]);
        } else {
            barrier();
        }
        if (t == 0) fetch(row + ahead * step, stage);
        if (++stage == ahead) {
            stage = 0;
            phase ^= 1;
        }
        if (p.dF) {
            if (p.after) {
                const F2 m1 = both(m.x), m2 = both(m.y);
#pragma unroll
                for (int q = 0; q < Q; ++q) dn[q] = mul2(add2(fma2(f[q], m2, dn[q]), m1), rstd);
            }
            put(p.dF, row * p.df_pitch, dn);
        }
    }
    if (t == 0 && abort_flag) {
        // nothing may land after the block has left: one more wait each for what was asked for
        for (int i = 0; i < ahead; ++i) {
            tc::mbar_wait_drain(&full[i], 0);
            tc::mbar_wait_drain(&full[i], 1);
        }
    }
    if (!p.partial) return;
    __syncthreads();                                 // every row has been read: the memory is free
    float* const joined = reinterpret_cast<float*>(memory);
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = (t + i * threads) * V;
            if (c >= cols) continue;
            float* const to = joined + ((size_t)grp * N + k) * cols + c;
#pragma unroll
            for (int q = 0; q < P; ++q) *reinterpret_cast<F2*>(to + 2 * q) = sums[k][i * P + q];
        }
    __syncthreads();
    for (int i = threadIdx.x * 4; i < N * cols; i += blockDim.x * 4) {
        float4 a = *reinterpret_cast<const float4*>(joined + i);
        for (int g = 1; g < groups; ++g) {
            const float4 b = *reinterpret_cast<const float4*>(joined + (size_t)g * N * cols + i);
            a.x += b.x;
            a.y += b.y;
            a.z += b.z;
            a.w += b.w;
        }
        const int k = i / cols;
        const int sum = ALL ? k : (k == 0 ? (int)DG : (int)DAG);
        *reinterpret_cast<float4*>(p.partial + ((int64_t)blockIdx.x * SUMS + sum) * cols + (i - k * cols)) = a;
    }
}

// Rows wider than a block keeps: first the row sums (two passes over the row) ...
template <typename T, int V>
struct LongRow {
    static constexpr int P = pairs<V>();
    const BwdParams& p;
    int64_t row;
    Stats sy, sf;
    __device__ __forceinline__ LongRow(const BwdParams& params, int64_t r) : p(params), row(r), sy{0, 0}, sf{0, 0} {
        if (p.dZ) sy = Stats{p.stats[row], p.stats[p.rows + row]};
        if (p.after) sf = Stats{p.stats[2 * p.rows + row], p.stats[3 * p.rows + row]};
    }
    __device__ __forceinline__ void get(F2 (&v)[P], const void* from, int64_t pitch, int64_t c) const {
        widen<T, V>(v, load<T, V>(static_cast<const T*>(from) + row * pitch + c));
    }
    __device__ __forceinline__ void put(void* to, int64_t pitch, int64_t c, const F2 (&v)[P]) const {
        store<T, V>(static_cast<T*>(to) + row * pitch + c, v);
    }
    static __device__ __forceinline__ void weigh(F2 (&v)[P], const void* w, int64_t c) {
        if (!w) return;
        F2 k[P];
        widen<T, V>(k, load<T, V>(static_cast<const T*>(w) + c));
#pragma unroll
        for (int q = 0; q < P; ++q) v[q] = mul2(v[q], k[q]);
    }
    __device__ __forceinline__ void hat(F2 (&v)[P], Stats s) const {
#pragma unroll
        for (int q = 0; q < P; ++q) v[q] = mul2(add2(v[q], both(-s.mean)), both(s.rstd));
    }
    // dZ (to dz) and yhat
    __device__ __forceinline__ void norm_inputs(F2 (&dz)[P], F2 (&yh)[P], int64_t c) const {
        get(dz, p.dZ, p.dz_pitch, c);
        get(yh, p.Y, p.y_pitch, c);
        hat(yh, sy);
    }
    // dx, from dZ g and yhat
    __device__ __forceinline__ void dx_of(F2 (&dx)[P], const F2 (&dz)[P], const F2 (&yh)[P], float2 m, int64_t c) const {
        if (p.dY) get(dx, p.dY, p.dy_pitch, c);
        else
#pragma unroll
            for (int q = 0; q < P; ++q) dx[q] = 0;
        if (p.dZ) add_through_norm<P>(dx, dz, yh, both(m.x), both(m.y), both(sy.rstd));
    }
    // scale gate dx
    __device__ __forceinline__ void dn_of(F2 (&dn)[P], const F2 (&dx)[P], int64_t c) const {
#pragma unroll
        for (int q = 0; q < P; ++q) dn[q] = both(p.scale);
        if (p.gate) weigh(dn, static_cast<const T*>(p.gate) + row * p.gate_pitch, c);
#pragma unroll
        for (int q = 0; q < P; ++q) dn[q] = mul2(dn[q], dx[q]);
    }
};

template <typename T, int V>
__global__ void __launch_bounds__(1024) backward_long_sums_kernel(const BwdParams p) {
    using L = LongRow<T, V>;
    constexpr int P = L::P;
    __shared__ float2 slots[2][32];
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const L r(p, row);
        auto means = [&](F2 s1, F2 s2, int k) {
            float2 c = block_sums<32>(make_float2(sum_of<V>(s1), sum_of<V>(s2)), slots[k]);
            c = make_float2(p.rms ? 0.f : -c.x * p.inv_cols, -c.y * p.inv_cols);
            if (threadIdx.x == 0) {
                p.row_sums[2 * k * p.rows + row] = c.x;
                p.row_sums[(2 * k + 1) * p.rows + row] = c.y;
            }
            return c;
        };
        F2 dz[P], yh[P], s1 = 0, s2 = 0;
        float2 m = make_float2(0.f, 0.f);
        if (p.dZ) {
            for (int64_t c = (int64_t)threadIdx.x * V; c < p.cols; c += 1024 * V) {
                r.norm_inputs(dz, yh, c);
                r.weigh(dz, p.g, c);
                add_products<P>(s1, s2, dz, yh);
            }
            m = means(s1, s2, 0);
        }
        if (p.after) {
            s1 = s2 = 0;
            for (int64_t c = (int64_t)threadIdx.x * V; c < p.cols; c += 1024 * V) {
                F2 dx[P], dn[P], fh[P];
                if (p.dZ) {
                    r.norm_inputs(dz, yh, c);
                    r.weigh(dz, p.g, c);
                }
                r.dx_of(dx, dz, yh, m, c);
                r.dn_of(dn, dx, c);
                r.weigh(dn, p.ag, c);
                r.get(fh, p.F, p.f_pitch, c);
                r.hat(fh, r.sf);
                add_products<P>(s1, s2, dn, fh);
            }
            means(s1, s2, 1);
        }
        __syncthreads();             // the slots serve the next row
    }
}

// ... then everything else, by threads that keep a pack of columns over a share of
// the rows (blockIdx.y).
template <typename T, int V>
__global__ void __launch_bounds__(128) backward_long_kernel(const BwdParams p) {
    using L = LongRow<T, V>;
    constexpr int P = L::P;
    const int64_t c = ((int64_t)blockIdx.x * 128 + threadIdx.x) * V;
    if (c >= p.cols) return;
    const int64_t r0 = p.rows * blockIdx.y / gridDim.y, r1 = p.rows * (blockIdx.y + 1) / gridDim.y;
    F2 sums[SUMS][P];
#pragma unroll
    for (int k = 0; k < SUMS; ++k)
#pragma unroll
        for (int q = 0; q < P; ++q) sums[k][q] = 0;
    for (int64_t row = r0; row < r1; ++row) {
        const L r(p, row);
        F2 dz[P], yh[P], dx[P];
        float2 m = make_float2(0.f, 0.f);
        if (p.dZ) {
            r.norm_inputs(dz, yh, c);
#pragma unroll
            for (int q = 0; q < P; ++q) {
                sums[DG][q] = fma2(dz[q], yh[q], sums[DG][q]);
                sums[DB][q] = add2(sums[DB][q], dz[q]);
            }
            r.weigh(dz, p.g, c);
            m = make_float2(p.row_sums[row], p.row_sums[p.rows + row]);
        }
        r.dx_of(dx, dz, yh, m, c);
        F2 f[P], dn[P];
        if (p.after || p.dgate || p.channel_gate_sum) r.get(f, p.F, p.f_pitch, c);
        r.dn_of(dn, dx, c);                            // reads the gate before dgate may replace it
        if (p.dX) r.put(p.dX, p.dx_pitch, c, dx);
        if (p.after) r.hat(f, r.sf);
        if (p.dgate || p.channel_gate_sum) {
            F2 n[P];
#pragma unroll
            for (int q = 0; q < P; ++q) n[q] = f[q];
            if (p.after) {
                r.weigh(n, p.ag, c);
                if (p.ab) {
                    F2 k[P];
                    widen<T, V>(k, load<T, V>(static_cast<const T*>(p.ab) + c));
#pragma unroll
                    for (int q = 0; q < P; ++q) n[q] = add2(n[q], k[q]);
                }
            }
#pragma unroll
            for (int q = 0; q < P; ++q) {
                n[q] = mul2(mul2(n[q], both(p.scale)), dx[q]);
                sums[DGATE][q] = add2(sums[DGATE][q], n[q]);
            }
            if (p.dgate) r.put(p.dgate, p.dgate_pitch, c, n);
        }
        if (p.after) {
#pragma unroll
            for (int q = 0; q < P; ++q) {
                sums[DAG][q] = fma2(dn[q], f[q], sums[DAG][q]);
                sums[DAB][q] = add2(sums[DAB][q], dn[q]);
            }
            r.weigh(dn, p.ag, c);
            F2 df[P];
#pragma unroll
            for (int q = 0; q < P; ++q) df[q] = 0;
            add_through_norm<P>(df, dn, f, both(p.row_sums[2 * p.rows + row]), both(p.row_sums[3 * p.rows + row]),
                                both(r.sf.rstd));
            if (p.dF) r.put(p.dF, p.df_pitch, c, df);
        } else if (p.dF) {
            r.put(p.dF, p.df_pitch, c, dn);
        }
    }
    if (!p.partial) return;
#pragma unroll
    for (int k = 0; k < SUMS; ++k) {
        float* out = p.partial + ((int64_t)blockIdx.y * SUMS + k) * p.cols + c;
#pragma unroll
        for (int q = 0; q < P; ++q) {
            float lo, hi;
            unpack_f2(sums[k][q], lo, hi);
            out[2 * q] = lo;
            if (V > 1) out[2 * q + 1] = hi;
        }
    }
}

struct Outputs {
    void* to[SUMS];         // null: not wanted
    int wanted[SUMS];       // those that are, in order
};

// Column sums over the blocks' partial sums, 32 columns a block: in block order
// within each share of them and then in share order, the same for every run.  (Eight
// columns a block would be more blocks, each with a quarter of a line to a load: the four
// sums of [8192, 1024] BF16 34.1 us with the gradient, so 30.2; [40, 4096] 27.3 and 14.6.)
constexpr int kSumCols = 32;
template <typename T>
__global__ void __launch_bounds__(1024)
column_sum_kernel(const float* __restrict__ partial, int blocks, int64_t cols, const Outputs outputs) {
    constexpr int C = kSumCols, SHARES = 1024 / C;
    __shared__ float sums[SHARES][C + 1];
    const int which = outputs.wanted[blockIdx.y];
    T* out = static_cast<T*>(outputs.to[which]);
    const int col = threadIdx.x % C, share = threadIdx.x / C;
    const int64_t c = (int64_t)blockIdx.x * C + col;
    float s = 0.f;
    if (c < cols) {
#pragma unroll 10
        for (int b = share; b < blocks; b += SHARES) s += partial[((int64_t)b * SUMS + which) * cols + c];
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

// Threads a row: with many rows a thread takes four packs, so that enough of the row
// is on its way at once and enough blocks reside ([16384, 4096] BF16, us: 4 warps x 4
// packs 79.6, 8 x 2 92.6, 2 x 8 81.0; [32768, 2048]: 2 x 4 78.8, 4 x 2 83.7, 8 x 1 110.9;
// [32768, 1024]: 1 x 4 42.6, 4 x 1 53.2, 2 x 4 66.8); with few rows more warps share a
// short one ([500, 1024] FP16: 4 x 1 2.9, 1 x 4 3.4; [64, 2048]: 8 x 1 2.7, 2 x 4 3.3;
// [4, 4096]: 4 x 4 3.3, 16 x 1 3.2; [300, 4096]: 3.8 and 4.0).  One warp needs no block
// barrier.
template <typename T, int V>
cudaError_t forward_as(const FwdParams& p, int sm_count, cudaStream_t s) {
    // Single elements go in pairs, and pairs (rows of 16-bit elements on 4-byte boundaries)
    // one by one: twice as many a thread as packs.  BF16, layer norm before and after, as
    // single elements and as pairs: [1167, 2058] 19.0 and 16.8 us, [5415, 350] 14.9 and
    // 10.9, [10000, 1350] 67.7 and 54.1, [16384, 4098] 433 and 354.
    const int64_t n = ceil_div(p.cols, V <= 2 ? 4 : V);
    constexpr int M = V <= 2 ? 2 : 1;
    const bool few = p.rows < 4 * (int64_t)sm_count;
#define OLC_FWD(W, NV)                                                                                          \
    return plan_launch(forward_kernel<T, V, W, NV * M>, dim3((unsigned)(W == 1 ? ceil_div(p.rows, 4) : p.rows)), \
                      dim3(W == 1 ? 128 : W * 32), 0, s, p)
    if (p.rows <= 0x7fffffff) {
        if (n <= 32) OLC_FWD(1, 1);
        if (n <= 64) OLC_FWD(1, 2);
        if (n <= 128 && !few) OLC_FWD(1, 4);
        if (n <= 128) OLC_FWD(4, 1);
        if (n <= 256 && !few) OLC_FWD(2, 4);
        if (n <= 256) OLC_FWD(8, 1);
        if (n <= 512) OLC_FWD(4, 4);
        if (n <= 1024) OLC_FWD(8, 4);
        if (n <= 2048) OLC_FWD(16, 4);
        if (n <= 4096) OLC_FWD(32, 4);
    }
#undef OLC_FWD
    const int64_t grid = min64(p.rows, (int64_t)sm_count * 2);
    return plan_launch(forward_long_kernel<T, V>, dim3((unsigned)grid), dim3(1024), 0, s, p);
}

// the backward launch of one shape
struct BwdShape {
    enum Kind { LONG, RING, ANY } kind = LONG;      // LONG: rows wider than a block keeps
    int per_thread = kColsPerThread;                // columns
    int tpr = 0, groups = 1, ahead = 0;
    int64_t blocks = 0;                             // that leave partial sums
    size_t smem = 0;
};
// `operands`: matrices that a row reads; `weights`: vectors; `all`: every column sum
template <int V>
BwdShape backward_shape(int64_t rows, int64_t cols, int sm_count, int operands, int weights, bool gated, bool all) {
    BwdShape b;
    if (V > 2) {
        // (a gate takes registers, too: 16 columns then only where 8 do not reach)
        b.per_thread = all || (gated && cols <= 8 * kThreads) ? 8 : 16;
        const int64_t row = cols * (16 / V) * operands, held = cols * (16 / V) * weights, room = kRingSmem - held;
        b.tpr = (int)min64(ceil_div(ceil_div(cols, b.per_thread), 32) * 32, 2 * kThreads);
        if (b.tpr <= kThreads && 2 * row <= room) {
            b.kind = BwdShape::RING;
            b.groups = (int)max64(1, min64(min64(kThreads / b.tpr, kMaxGroups), ceil_div(rows, sm_count)));
            while (b.groups > 1 && 2 * row * b.groups > room) --b.groups;
            b.ahead = (int)min64(kMaxAhead, room / (row * b.groups));
            b.blocks = max64(1, min64(ceil_div(rows, b.groups), sm_count));
            b.smem = (size_t)max64(held + row * b.groups * b.ahead, (int64_t)b.groups * (all ? SUMS : 2) * cols * 4);
            return b;
        }
    }
    b.per_thread = kColsPerThread;
    if (cols > kThreads * kColsPerThread) {
        const int64_t across = ceil_div(ceil_div(cols, V), 128);
        b.blocks = max64(1, min64(min64(ceil_div(rows, 4), 65535), 8 * (int64_t)sm_count / across));
        return b;
    }
    b.kind = BwdShape::ANY;
    b.tpr = (int)(ceil_div(ceil_div(cols, kColsPerThread), 32) * 32);
    b.groups = (int)max64(1, min64(kThreads / b.tpr, ceil_div(rows, sm_count)));
    b.blocks = max64(1, min64(ceil_div(rows, b.groups), sm_count));
    b.smem = b.groups > 1 ? (size_t)b.groups * cols * sizeof(float) : 0;
    return b;
}

template <typename T, int C, bool ALL, bool GATED>
cudaError_t backward_ring(const BwdParams& p, const BwdShape& b, cudaStream_t s) {
    constexpr int NV = C * sizeof(T) / 16;
    auto* kernel = p.cols == (int64_t)b.tpr * C ? backward_ring_kernel<T, NV, ALL, GATED, true>
                                                : backward_ring_kernel<T, NV, ALL, GATED, false>;
    const cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(kernel), kRingSmem);
    if (e != cudaSuccess) return e;
    return plan_launch(kernel, dim3((unsigned)b.blocks), dim3((unsigned)(b.tpr * b.groups)), b.smem, s, p, b.ahead);
}

template <typename T, int V>
cudaError_t backward_as(BwdParams p, int sm_count, const Outputs& outputs, cudaStream_t s) {
    const bool all = outputs.to[DB] || outputs.to[DAB] || outputs.to[DGATE];
    const int operands = (p.dZ ? 2 : 0) + (p.dY ? 1 : 0) + (p.after || p.dgate || p.channel_gate_sum ? 1 : 0) +
                         (p.gate && p.gate_pitch ? 1 : 0);
    const int weights = (p.g ? 1 : 0) + (p.after && p.ag ? 1 : 0) + (p.gate && p.after && p.ab ? 1 : 0) +
                        (p.gate && !p.gate_pitch ? 1 : 0);
    const BwdShape b = backward_shape<V>(p.rows, p.cols, sm_count, operands, weights, p.gate != nullptr, all);
    cudaError_t e = cudaSuccess;
    p.threads_per_row = b.tpr;
    if (b.kind == BwdShape::RING) {
        if constexpr (V > 2)
            e = all ? backward_ring<T, 8, true, true>(p, b, s)
                : !p.gate ? backward_ring<T, 16, false, false>(p, b, s)
                : b.per_thread == 8 ? backward_ring<T, 8, false, true>(p, b, s)
                                    : backward_ring<T, 16, false, true>(p, b, s);
    } else if (b.kind == BwdShape::LONG) {
        if (p.dZ || p.after)
            e = plan_launch(backward_long_sums_kernel<T, V>, dim3((unsigned)min64(p.rows, (int64_t)sm_count * 2)),
                            dim3(1024), 0, s, p);
        if (e == cudaSuccess)
            e = plan_launch(backward_long_kernel<T, V>,
                            dim3((unsigned)ceil_div(ceil_div(p.cols, V), 128), (unsigned)b.blocks), dim3(128), 0, s, p);
    } else {
        // Rows of packs whose operands overfill the ring come here as single elements do.
        // Pairs (V == 2) go as single elements: [10000, 1350] BF16 takes 127 us so and 139
        // as pairs, whose offsets are not constants ([1167, 2058]: 40 and 38; rows wider
        // than a block keeps gain: [16384, 4098] 1189 as single elements and 819 as pairs).
        constexpr int E = V == 2 ? 1 : V, NV = E == 1 ? kColsPerThread / 2 : kColsPerThread / E;
        e = plan_launch(backward_kernel<T, E, NV>, dim3((unsigned)b.blocks), dim3((unsigned)(b.tpr * b.groups)), b.smem, s, p);
    }
    if (e != cudaSuccess || !p.partial) return e;
    Outputs o = outputs;
    int n = 0;
    for (int k = 0; k < SUMS; ++k)
        if (o.to[k]) o.wanted[n++] = k;
    return plan_launch(column_sum_kernel<T>, dim3((unsigned)ceil_div(p.cols, kSumCols), (unsigned)n), dim3(1024), 0, s,
                       (const float*)p.partial, (int)b.blocks, p.cols, o);
}

}  // namespace residual
}  // namespace olc

using namespace olc;

struct olc_residual_norm_plan {
    PlanState state;
    olc_dtype dtype;
    int64_t rows, cols;
    int64_t most_blocks;    // of a gradient call; 0: none yet
    float eps, scale;
    int rms, after;
};

extern "C" {

olc_status olc_residual_norm_plan_create(int64_t rows, int64_t cols, double eps, double scale, int norm, int after,
                                         olc_dtype dtype, olc_residual_norm_plan** out) {
    if (!out) return OLC_ERR_NULL;
    *out = nullptr;
    if (!plan_dtype_ok(dtype)) return OLC_ERR_DTYPE;
    if (rows < 0 || cols < 0) return OLC_ERR_NEGATIVE_DIM;
    // the mean of no elements is undefined; columns are 32-bit in the kernels
    if (cols == 0 || cols >= (int64_t(1) << 31) - 65536 || !(eps >= 0.0) || eps > 3e38) return OLC_ERR_INVALID;
    if (!(scale >= -3e38 && scale <= 3e38) || (norm != OLC_NORM_LAYER && norm != OLC_NORM_RMS)) return OLC_ERR_INVALID;
    if (!plan_fits(rows, cols, 4) || !plan_fits(rows, 16, 4)) return OLC_ERR_INVALID;
    olc_residual_norm_plan* p = new (std::nothrow) olc_residual_norm_plan;
    if (!p) return OLC_ERR_OOM;
    p->state.init();
    p->dtype = dtype;
    p->rows = rows;
    p->cols = cols;
    p->most_blocks = 0;
    p->eps = (float)eps;
    p->scale = (float)scale;
    p->rms = norm == OLC_NORM_RMS;
    p->after = after != 0;
    *out = p;
    return OLC_OK;
}

void olc_residual_norm_plan_destroy(olc_residual_norm_plan* plan) {
    if (!plan) return;
    plan->state.destroy();
    delete plan;
}

// A [rows, cols] operand that is refused
static bool bad_rows(const olc_residual_norm_plan* plan, const void* m, int64_t pitch) {
    const int64_t eb = plan_elem_bytes(plan->dtype);
    return m && ((plan->rows > 1 && (pitch < plan->cols || !plan_fits(plan->rows, pitch, eb))) || plan_misaligned(m, eb));
}
static bool bad_gate(const olc_residual_norm_plan* plan, const void* m, int64_t pitch) {
    return pitch == 0 ? plan_misaligned(m, plan_elem_bytes(plan->dtype)) : bad_rows(plan, m, pitch);
}
// What the starts of all rows of the given operands divide by: 16, 4 or less
struct Bytes {
    const olc_residual_norm_plan* plan;
    uint64_t all;
    explicit Bytes(const olc_residual_norm_plan* p) : plan(p), all((uint64_t)(p->cols * plan_elem_bytes(p->dtype))) {}
    Bytes& rows(const void* m, int64_t pitch) {
        all |= (uint64_t)reinterpret_cast<uintptr_t>(m);
        if (m && plan->rows > 1) all |= (uint64_t)(pitch * plan_elem_bytes(plan->dtype));
        return *this;
    }
    Bytes& vector(const void* v) {
        all |= (uint64_t)reinterpret_cast<uintptr_t>(v);
        return *this;
    }
    // elements of a pack
    int elements() const {
        const int eb = (int)plan_elem_bytes(plan->dtype);
        return all % 16 == 0 ? 16 / eb : (eb == 2 && all % 4 == 0 ? 2 : 1);
    }
};

olc_status olc_residual_norm_forward(olc_residual_norm_plan* plan, const void* X, int64_t x_pitch, const void* F,
                                     int64_t f_pitch, const void* gate, int64_t gate_pitch, const void* after_gamma,
                                     const void* after_beta, const void* gamma, const void* beta, void* Y,
                                     int64_t y_pitch, void* Z, int64_t z_pitch, float* stats, void* stream) {
    if (!plan) return OLC_ERR_NULL;
    if (plan->rows == 0) return OLC_OK;
    if (!X || !F || !Y) return OLC_ERR_NULL;
    const int64_t eb = plan_elem_bytes(plan->dtype);
    if (bad_rows(plan, X, x_pitch) || bad_rows(plan, F, f_pitch) || bad_gate(plan, gate, gate_pitch) ||
        bad_rows(plan, Y, y_pitch) || bad_rows(plan, Z, z_pitch) || plan_misaligned(after_gamma, eb) ||
        plan_misaligned(after_beta, eb) || plan_misaligned(gamma, eb) || plan_misaligned(beta, eb) ||
        plan_misaligned(stats, 4))
        return OLC_ERR_INVALID;
    const olc_status st = plan->state.bind();
    if (st != OLC_OK) return st;
    const residual::FwdParams p{X, F, gate, after_gamma, after_beta, gamma, beta, Y, Z, stats, x_pitch, f_pitch,
                                gate_pitch, y_pitch, z_pitch, plan->rows, plan->cols, plan->eps, plan->scale,
                                (float)(1.0 / (double)plan->cols), plan->after, plan->rms};
    const int elements = Bytes(plan).rows(X, x_pitch).rows(F, f_pitch).rows(gate, gate_pitch).rows(Y, y_pitch).rows(Z, z_pitch)
                             .vector(after_gamma).vector(after_beta).vector(gamma).vector(beta).elements();
    return by_type(plan->dtype, [&](auto tag) {
        using T = decltype(tag);
        const cudaStream_t s = static_cast<cudaStream_t>(stream);
        const int sms = plan->state.sm_count;
        if (elements == 16 / (int)sizeof(T)) return plan_status(residual::forward_as<T, 16 / sizeof(T)>(p, sms, s));
        if constexpr (sizeof(T) == 2)
            if (elements == 2) return plan_status(residual::forward_as<T, 2>(p, sms, s));
        return plan_status(residual::forward_as<T, 1>(p, sms, s));
    });
}

// Blocks that leave partial sums, at most, whatever a call's alignment, operands and
// outputs: a later call does not have to allocate again.  (Once for a plan: 300 launch
// shapes are 1.6 us of a call.)
static int64_t most_blocks(olc_dtype dtype, int64_t rows, int64_t cols, int sms) {
    int64_t blocks = 0;
    for (int which = 0; which < 5 * 5 * 4; ++which) {
        const int operands = 1 + which % 5, weights = which / 5 % 5;
        const bool gated = which / 25 & 1, all = which / 50;
        auto of = [&](auto shape) { blocks = max64(blocks, shape(rows, cols, sms, operands, weights, gated, all).blocks); };
        of(residual::backward_shape<1>);
        if (dtype == OLC_FLOAT) {
            of(residual::backward_shape<4>);
        } else {
            of(residual::backward_shape<2>);
            of(residual::backward_shape<8>);
        }
    }
    return blocks;
}

olc_status olc_residual_norm_backward(olc_residual_norm_plan* plan, const void* dY, int64_t dy_pitch, const void* dZ,
                                      int64_t dz_pitch, const void* F, int64_t f_pitch, const void* Y, int64_t y_pitch,
                                      const float* stats, const void* gate, int64_t gate_pitch,
                                      const void* after_gamma, const void* after_beta, const void* gamma, void* dX,
                                      int64_t dx_pitch, void* dF, int64_t df_pitch, void* dgate, int64_t dgate_pitch,
                                      void* dgamma, void* dbeta, void* dafter_gamma, void* dafter_beta, void* stream) {
    if (!plan) return OLC_ERR_NULL;
    if (!dX && !dF && !dgate && !dgamma && !dbeta && !dafter_gamma && !dafter_beta) return OLC_OK;
    const int64_t eb = plan_elem_bytes(plan->dtype), rows = plan->rows, cols = plan->cols;
    if (!plan->after && (dafter_gamma || dafter_beta)) return OLC_ERR_INVALID;
    const bool channel_sum = dgate && gate_pitch == 0;
    if (rows > 0) {
        if (!dY && !dZ) return OLC_ERR_NULL;
        if (!dZ && (dgamma || dbeta)) return OLC_ERR_NULL;
        if (dgate && !gate) return OLC_ERR_NULL;
        if (((plan->after || dgate) && !F) || (dZ && !Y) || ((dZ || plan->after) && !stats)) return OLC_ERR_NULL;
    }
    if (bad_rows(plan, dY, dy_pitch) || bad_rows(plan, dZ, dz_pitch) || bad_rows(plan, F, f_pitch) ||
        bad_rows(plan, Y, y_pitch) || bad_gate(plan, gate, gate_pitch) || bad_rows(plan, dX, dx_pitch) ||
        bad_rows(plan, dF, df_pitch) || (channel_sum ? plan_misaligned(dgate, eb) : bad_rows(plan, dgate, dgate_pitch)) ||
        plan_misaligned(stats, 4) || plan_misaligned(after_gamma, eb) || plan_misaligned(after_beta, eb) ||
        plan_misaligned(gamma, eb) || plan_misaligned(dgamma, eb) || plan_misaligned(dbeta, eb) ||
        plan_misaligned(dafter_gamma, eb) || plan_misaligned(dafter_beta, eb))
        return OLC_ERR_INVALID;
    olc_status st = plan->state.bind();
    if (st != OLC_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const residual::Outputs outputs{{dgamma, dbeta, dafter_gamma, dafter_beta, channel_sum ? dgate : nullptr}, {}};
    bool sums = false;
    for (void* o : outputs.to) sums = sums || o;
    if (rows == 0) {                        // empty sums
        cudaError_t e = cudaSuccess;
        for (void* o : outputs.to)
            if (e == cudaSuccess && o) e = launch_zero_fill(o, cols * eb, s);
        return plan_status(e);
    }
    const int elements = Bytes(plan).rows(dY, dy_pitch).rows(dZ, dz_pitch).rows(F, f_pitch).rows(Y, y_pitch)
                             .rows(gate, gate_pitch).rows(dX, dx_pitch).rows(dF, df_pitch)
                             .rows(channel_sum ? nullptr : dgate, dgate_pitch).vector(after_gamma).vector(after_beta)
                             .vector(gamma).elements();
    residual::BwdParams p{dY, dZ, F, Y, stats, gate, after_gamma, after_beta, gamma, dX, dF, channel_sum ? nullptr : dgate,
                          nullptr, nullptr, dy_pitch, dz_pitch, f_pitch, y_pitch, gate_pitch, dx_pitch, df_pitch,
                          dgate_pitch, rows, cols, plan->scale, (float)(1.0 / (double)cols), plan->after, plan->rms,
                          channel_sum, 0, device_error_word()};
    const int sms = plan->state.sm_count;
    if (plan->most_blocks == 0) plan->most_blocks = most_blocks(plan->dtype, rows, cols, sms);
    const int64_t blocks = plan->most_blocks;
    const size_t row_floats = cols > residual::kThreads * residual::kColsPerThread ? ((size_t)rows * 4 + 3) / 4 * 4 : 0;
    const size_t floats = row_floats + (size_t)blocks * residual::SUMS * (size_t)cols;
    st = plan->state.ensure(floats * sizeof(float));
    if (st != OLC_OK) return st;
    p.row_sums = static_cast<float*>(plan->state.memory);
    if (sums) p.partial = p.row_sums + row_floats;
    return by_type(plan->dtype, [&](auto tag) {
        using T = decltype(tag);
        return plan_status(plan->state.use(s, [&] {
            if (elements == 16 / (int)sizeof(T)) return residual::backward_as<T, 16 / sizeof(T)>(p, sms, outputs, s);
            if constexpr (sizeof(T) == 2)
                if (elements == 2) return residual::backward_as<T, 2>(p, sms, outputs, s);
            return residual::backward_as<T, 1>(p, sms, outputs, s);
        }));
    });
}

}  // extern "C"
