// Rows of elements as 16-byte packs or single elements, in float32 pairs, and
// sums over warps and blocks: what the kernels that go over rows share.
#pragma once

#include <type_traits>

#include "tc_ptx.cuh"

namespace olc {

// V elements of T in one access on a boundary of its V sizeof(T) bytes: 16 bytes, the 4 of a pair
// of 16-bit elements, or one element; and the same as pairs of float32 (V = 1: the second of
// the pair is not used).
template <typename T, int V>
struct alignas(V * sizeof(T)) Pack {
    T v[V];
};
template <int V>
constexpr int pairs() {
    return V == 1 ? 1 : V / 2;
}
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load(const void* p) {
    return *static_cast<const Pack<T, V>*>(p);
}
template <typename T, int V>
__device__ __forceinline__ void widen(F2 (&out)[pairs<V>()], const Pack<T, V>& k) {
    if constexpr (V == 1) {
        out[0] = pack_f2(Num<T>::to_acc(k.v[0]), 0.f);
    } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&k);
#pragma unroll
        for (int i = 0; i < V / 2; ++i)
            out[i] = pack_f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) out[i] = pack_f2(Num<T>::to_acc(k.v[2 * i]), Num<T>::to_acc(k.v[2 * i + 1]));
    }
}
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const F2 (&in)[pairs<V>()]) {
    Pack<T, V> k;
#pragma unroll
    for (int i = 0; i < pairs<V>(); ++i) {
        float lo, hi;
        unpack_f2(in[i], lo, hi);
        if constexpr (V == 1) {
            k.v[0] = Num<T>::from_acc(lo);
        } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
            reinterpret_cast<__nv_bfloat162*>(&k)[i] = __floats2bfloat162_rn(lo, hi);
        } else if constexpr (std::is_same_v<T, __half>) {
            reinterpret_cast<__half2*>(&k)[i] = __floats2half2_rn(lo, hi);
        } else {
            k.v[2 * i] = lo;
            k.v[2 * i + 1] = hi;
        }
    }
    *reinterpret_cast<Pack<T, V>*>(p) = k;
}
template <int V>
__device__ __forceinline__ float sum_of(F2 x) {
    float lo, hi;
    unpack_f2(x, lo, hi);
    return V == 1 ? lo : lo + hi;
}
__device__ __forceinline__ F2 both(float v) { return pack_f2(v, v); }

// bytes from global to shared memory (both on 16-byte boundaries), completing on a barrier
__device__ __forceinline__ void bulk_copy(void* to, const void* from, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     tc::smem_u32(to)),
                 "l"(from), "r"(bytes), "r"(tc::smem_u32(bar))
                 : "memory");
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

// A thread's columns of a row: packs of V at (base + i stride) V on boundaries of their size, or,
// for rows of any alignment (V = 1), pairs of single elements `stride` apart: two elements
// an instruction either way.  Single elements are addressed and tested one by
// one only where the row ends: `full` tells that the i-th pair of every lane of
// the warp lies inside the row.
template <typename T, int V>
struct Columns {
    static constexpr int PER = V == 1 ? 2 : V;      // columns of one i
    static constexpr int P = PER / 2;
    struct Raw {
        T v[PER];
    };
    static __device__ __forceinline__ int at(int base, int i, int q, int stride) {
        return V == 1 ? base + (2 * i + q) * stride : (base + i * stride) * V + q;
    }
    static __device__ __forceinline__ Raw read(const T* row, int base, int i, int stride, int cols, bool live, bool full) {
        Raw r{};
        if constexpr (V == 1) {
            if (live && full) {
#pragma unroll
                for (int q = 0; q < 2; ++q) r.v[q] = row[at(base, i, q, stride)];
            } else if (live) {
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    if (at(base, i, q, stride) < cols) r.v[q] = row[at(base, i, q, stride)];
            }
        } else {
            if (live && at(base, i, 0, stride) < cols) {
                const Pack<T, V> k = load<T, V>(row + at(base, i, 0, stride));
#pragma unroll
                for (int q = 0; q < V; ++q) r.v[q] = k.v[q];
            }
        }
        return r;
    }
    static __device__ __forceinline__ bool in(int base, int i, int q, int stride, int cols) {
        return at(base, i, q, stride) < cols;
    }
    static __device__ __forceinline__ void write(T* row, int base, int i, int stride, int cols, const F2 (&o)[P], bool full) {
        if constexpr (V == 1) {
            float lo, hi;
            unpack_f2(o[0], lo, hi);
            if (full || in(base, i, 0, stride, cols)) row[at(base, i, 0, stride)] = Num<T>::from_acc(lo);
            if (full || in(base, i, 1, stride, cols)) row[at(base, i, 1, stride)] = Num<T>::from_acc(hi);
        } else if (in(base, i, 0, stride, cols)) {
            store<T, V>(row + at(base, i, 0, stride), o);
        }
    }
    // a pair of columns, zeros where the row has ended
    static __device__ __forceinline__ F2 inside(F2 v, int base, int i, int q, int stride, int cols, bool full) {
        if constexpr (V == 1) {
            if (full) return v;
            float lo, hi;
            unpack_f2(v, lo, hi);
            return pack_f2(in(base, i, 0, stride, cols) ? lo : 0.f, in(base, i, 1, stride, cols) ? hi : 0.f);
        } else {
            return in(base, i, 0, stride, cols) ? v : 0;
        }
    }
    static __device__ __forceinline__ void pairs_of(F2 (&out)[P], const Raw& r) {
#pragma unroll
        for (int q = 0; q < P; ++q) out[q] = pack_f2(Num<T>::to_acc(r.v[2 * q]), Num<T>::to_acc(r.v[2 * q + 1]));
    }
};

template <typename F>
olc_status by_type(olc_dtype dt, F&& f) {
    switch (dt) {
        case OLC_FLOAT: return f(float{});
        case OLC_FLOAT16: return f(__half{});
        case OLC_BFLOAT16: return f(__nv_bfloat16{});
        default: return OLC_ERR_DTYPE;
    }
}

}  // namespace olc
