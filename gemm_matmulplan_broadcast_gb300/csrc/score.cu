// Log probabilities of given tokens from logits [rows, vocab], with the
// entropy of each row's distribution and its k most likely tokens, and the
// gradient.
//
//   m = max_j z_j,  s = sum_j e^(z_j - m),  a = sum_j (z_j - m) e^(z_j - m)
//   lse = m + log s,  logprob = (z_token - m) - log s,  H = log s - a / s
//   (the sums in units of log 2, which is what the exponential unit takes)
//   dz_j = dlogprob (1[j = token] - p_j) - dH p_j (log p_j + H)
//
// (a <= 0 <= log s but for a residue below 2^-8, so the entropy's two terms never
// cancel.)  About six
// operations and one exponential an element against one element read: the
// bytes bound it, with the exponential unit close behind for 16-bit logits.
// Measured, BF16 [4096, 50257] in rows of 50264: forward 81 us with five
// alternatives (5.1 TB/s; 71 us, 5.8 TB/s without: what follows a row's sums
// shares issue slots with the next row; 125 us where 99 of 100 logits are masks of
// -inf or -1e9, whose stretches take the longer form), backward 120 us (6.9 TB/s,
// a copy's rate).  One row [1, 50257] FP16 with 20 alternatives: 11.3 us, a chain of
// loads, sums and picks that nothing else can fill.
//
// Forward.  One pass: each thread keeps a running m, s and a, rescaled when a
// later group of its elements brings a larger maximum.  A row is one block,
// or, where there are fewer rows than blocks fit, a cluster of blocks that
// each take a slice of it; the first block joins the slices' sums in slice
// order through distributed shared memory.
//
// The k largest need no second pass over the row.  k threads whose own maximum
// is at least t hold at least k elements >= t; so the k-th largest of the
// threads' maxima is a bound that every one of the k largest elements reaches.
// Only stretches of a thread's elements whose maximum reaches it are read
// again: a few packs of the row.  Order is by value, then by the lower index.
#include <new>
#include <type_traits>

#include "plan_state.h"
#include "tc_ptx.cuh"

namespace olc {
namespace score {

constexpr int kThreads = 128;               // consumers; one more warp issues the loads, two finish rows
constexpr int kWarps = kThreads / 32;
constexpr int kBlockThreads = kThreads + 96;
constexpr int kMaxTop = 32;
constexpr int kMaxCluster = 8;
constexpr int kBuffer = 256;                // candidates above the bound, and as many at it
constexpr int kUnroll = 8;                  // 16-byte packs a thread takes of a chunk
constexpr int kChunk = kThreads * kUnroll;  // packs of a chunk: 16 KiB
constexpr int kStages = 3;                  // chunks in flight or in use a block
constexpr int kBlocksPerSm = 3;
constexpr int kSlots = 8;                   // stretches of a slice whose maxima each thread keeps
constexpr int kGradPacks = 4;               // backward: packs a thread

struct Params {
    const void* logits;
    const int64_t* tokens;
    float* logprob;
    float* entropy;         // may be null
    float* lse;             // may be null
    float* top_logprob;     // [rows][top], may be null
    int64_t* top_index;     // [rows][top], may be null
    int64_t pitch;
    int vocab;
    int top;
    int cluster;            // blocks a row
    int64_t units;          // rows x cluster
    unsigned int* err;
};

struct GradParams {
    const void* logits;
    const int64_t* tokens;
    const float* lse;
    const float* entropy;
    const float* dlogprob;  // may be null: 0
    const float* dentropy;  // may be null: 0
    void* dlogits;
    int64_t pitch, d_pitch;
    int64_t rows;
    int vocab;
    int chunks;             // blocks a row
};

// Unsigned order of the values: -inf lowest, -0 equal to +0, NaN above all.
__device__ __forceinline__ uint32_t order_key(float z) {
    const uint32_t b = __float_as_uint(z + 0.0f);
    if (z != z) return 0xFFFFFFFFu;
    return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    if (k == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
    return __uint_as_float((k >> 31) ? k & 0x7FFFFFFFu : ~k);
}

// max(a, b), NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.69314718055994531f;

// Distances below this one weigh nothing (2^-150 is 0 in float32), and their
// product with a zero weight has to be 0 for masks of -inf and of the type's
// lowest value alike.
constexpr float kFar = -1.0e4f;

// the exponential unit, good to 2^-22 of the result
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// the same without the flush of results below 2^-126
__device__ __forceinline__ float exp2_small(float x) {
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// A running softmax over some elements of a row, in units of log 2: with a
// distance d_j from the largest element m, s = sum 2^d_j and a = sum d_j 2^d_j.
// Near zero, where most logits are, d_j = z_j log2(e) - R with the rounded
// R = m log2(e): one fused operation an element.  All distances then have R's
// rounding, residue(m), too much, at most 2^-8 there.  Farther out (logits or
// finite masks of any size; R's rounding would grow with them) m is subtracted
// first, which is exact for elements close to it: d_j = (z_j - m) log2(e).
struct Sums {
    float m, s, a;
};
constexpr float kNear = 49152.f;        // and kNear - kFar is a value that FLOAT16 holds
__device__ __forceinline__ bool near_zero(float m) { return fabsf(m) < kNear; }
__device__ __forceinline__ float residue(float m) {
    return near_zero(m) ? fmaf(m, kLog2e, -__fmul_rn(m, kLog2e)) : 0.f;
}
// what elements are taken from: -inf, the maximum of nothing, keeps them as they are
__device__ __forceinline__ float origin(float m) { return m == -INFINITY ? 0.f : m; }
// an element's distance, not below kFar
__device__ __forceinline__ float distance(float z, float m) {
    return max_nan(near_zero(m) ? fmaf(z, kLog2e, -__fmul_rn(m, kLog2e)) : (z - origin(m)) * kLog2e, kFar);
}

// the same sums around another maximum (m >= q.m)
__device__ __forceinline__ void move_to(Sums& q, float m) {
    if (q.m != -INFINITY) {          // else nothing but zeros, or a NaN to keep
        const float d = max_nan(fmaf(q.m - m, kLog2e, residue(m) - residue(q.m)), kFar);
        const float c = exp2_fast(d);
        q.a = c * fmaf(d, q.s, q.a);
        q.s *= c;
    }
    q.m = m;
}

// the sums of both sets of elements, in this order
__device__ __forceinline__ Sums join(Sums x, Sums y) {
    const float m = fmaxf(x.m, y.m);
    move_to(x, m);
    move_to(y, m);
    return Sums{m, x.s + y.s, x.a + y.a};
}

// Operations on a 16-byte pack of elements as loaded: 16-bit types compare
// two elements an instruction.
template <typename T>
__device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b) {      // NaN loses
    if constexpr (sizeof(T) == 4) return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    uint32_t r;
    if constexpr (std::is_same_v<T, __half>) asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <typename T>
__device__ __forceinline__ uint32_t floor_word(uint32_t a, uint32_t b) {    // max(a, b), NaN stays
    if constexpr (sizeof(T) == 4) return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
    uint32_t r;
    if constexpr (std::is_same_v<T, __half>) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// both halves of a word hold `v` (float32: the word is v)
template <typename T>
__device__ __forceinline__ uint32_t splat(float v) {
    if constexpr (sizeof(T) == 4) return __float_as_uint(v);
    const T e = Num<T>::from_acc(v);
    const uint32_t b = *reinterpret_cast<const unsigned short*>(&e);
    return b | (b << 16);
}
// the larger of a word's elements
template <typename T>
__device__ __forceinline__ float word_max(uint32_t w) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w);
    const unsigned short lo = (unsigned short)w, hi = (unsigned short)(w >> 16);
    return fmaxf(Num<T>::to_acc(*reinterpret_cast<const T*>(&lo)), Num<T>::to_acc(*reinterpret_cast<const T*>(&hi)));
}
// the elements of words 2i, 2i + 1 (float32) or of word i (16-bit): one pair
template <typename T>
__device__ __forceinline__ F2 pair_of(const uint32_t (&w)[4], int i) {
    if constexpr (sizeof(T) == 4) return pack_f2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    if constexpr (std::is_same_v<T, __half>) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        return pack_f2(f.x, f.y);
    } else {
        return pack_f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
}
// A row's values that lie kFar below a `top` near zero weigh nothing and are
// raised to that floor, so that no infinity meets a zero: a value of every
// type, rounded by 128 at most.
template <typename T>
__device__ __forceinline__ uint32_t floor_of(float top) {
    return splat<T>(top + kFar);
}

template <typename T>
struct Slice {
    static constexpr int V = 16 / sizeof(T);
    const T* row;
    int head;           // elements before the row's first 16-byte boundary (first slice)
    int v0, v1;         // 16-byte packs of this slice, counted from that boundary
    int body;           // index of the row's element at that boundary
    int tail0, tail1;   // elements after the last whole pack (last slice)
};

template <typename T>
__device__ __forceinline__ Slice<T> slice_of(const T* row, int vocab, int part, int parts) {
    constexpr int V = Slice<T>::V;
    Slice<T> s;
    s.row = row;
    const int off = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    const int lead = off ? min(V - off, vocab) : 0;
    const int packs = (vocab - lead) / V;
    s.body = lead;
    s.head = part == 0 ? lead : 0;
    const int each = parts == 1 ? packs : packs / parts, extra = packs - each * parts;
    s.v0 = each * part + min(part, extra);          // the first `extra` slices take one more
    s.v1 = s.v0 + each + (part < extra ? 1 : 0);
    s.tail0 = part == parts - 1 ? lead + packs * V : vocab;
    s.tail1 = vocab;
    return s;
}

template <typename T>
__device__ __forceinline__ void unpack(const uint4& k, float (&z)[16 / sizeof(T)]) {
    const T* e = reinterpret_cast<const T*>(&k);
#pragma unroll
    for (int i = 0; i < (int)(16 / sizeof(T)); ++i) z[i] = Num<T>::to_acc(e[i]);
}

// bit i: element i of the pack is at least the word's (NaN: no)
template <typename T>
__device__ __forceinline__ unsigned reaching(const uint4& k, uint32_t least) {
    const uint32_t w[4] = {k.x, k.y, k.z, k.w};
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            m |= (unsigned)(__uint_as_float(w[i]) >= __uint_as_float(least)) << i;
        } else {
            unsigned r;
            if constexpr (std::is_same_v<T, __half>)
                r = __hge2_mask(*reinterpret_cast<const __half2*>(&w[i]), *reinterpret_cast<const __half2*>(&least));
            else
                r = __hge2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w[i]),
                                *reinterpret_cast<const __nv_bfloat162*>(&least));
            m |= ((r & 1u) | ((r >> 16) & 2u)) << (2 * i);
        }
    }
    return m;
}

// chunks a thread's stretch of the slice spans
template <typename T>
__device__ __forceinline__ int chunks_a_slot(const Slice<T>& s) {
    const int chunks = (s.v1 - s.v0 + kChunk - 1) / kChunk;
    return (chunks + kSlots - 1) / kSlots;
}

// one element, any values
__device__ __forceinline__ void take(Sums& q, float z) {
    if (z > q.m) move_to(q, z);
    const float d = distance(z, q.m);
    const float e = exp2_fast(d);
    q.s += e;
    q.a = fmaf(d, e, q.a);
}

// N packs at once: the maximum first (returned), then the sums around it, two
// elements an instruction
template <typename T, int N>
__device__ __forceinline__ float take(Sums& q, const uint4 (&k)[N]) {
    uint32_t top = max_word<T>(max_word<T>(k[0].x, k[0].y), max_word<T>(k[0].z, k[0].w));
#pragma unroll
    for (int i = 1; i < N; ++i)
        top = max_word<T>(top, max_word<T>(max_word<T>(k[i].x, k[i].y), max_word<T>(k[i].z, k[i].w)));
    const float m = word_max<T>(top);
    if (m > q.m) move_to(q, m);
    const F2 scale = pack_f2(kLog2e, kLog2e);
    F2 s = pack_f2(0.f, 0.f), a = s;
    if (near_zero(q.m)) {
        const uint32_t low = floor_of<T>(q.m);
        const float r = -__fmul_rn(q.m, kLog2e);
        const F2 shift = pack_f2(r, r);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t w[4] = {floor_word<T>(k[i].x, low), floor_word<T>(k[i].y, low), floor_word<T>(k[i].z, low),
                                   floor_word<T>(k[i].w, low)};
#pragma unroll
            for (int j = 0; j < (int)(8 / sizeof(T)); ++j) {
                const F2 d = fma2(pair_of<T>(w, j), scale, shift);
                float lo, hi;
                unpack_f2(d, lo, hi);
                const F2 e = pack_f2(exp2_fast(lo), exp2_fast(hi));
                s = add2(s, e);
                a = fma2(d, e, a);
            }
        }
    } else {
        // masks alone so far, or logits far from zero
        const float r = -origin(q.m);
        const F2 shift = pack_f2(r, r);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t w[4] = {k[i].x, k[i].y, k[i].z, k[i].w};
#pragma unroll
            for (int j = 0; j < (int)(8 / sizeof(T)); ++j) {
                float lo, hi;
                unpack_f2(mul2(add2(pair_of<T>(w, j), shift), scale), lo, hi);
                lo = max_nan(lo, kFar);
                hi = max_nan(hi, kFar);
                const F2 e = pack_f2(exp2_fast(lo), exp2_fast(hi));
                s = add2(s, e);
                a = fma2(pack_f2(lo, hi), e, a);
            }
        }
    }
    float lo, hi;
    unpack_f2(s, lo, hi);
    q.s += lo + hi;
    unpack_f2(a, lo, hi);
    q.a += lo + hi;
    return m;
}

// What the consumers leave of a row (or slice) to the finishing warp.
struct Row {
    float m[kThreads], s[kThreads], a[kThreads];
    float slot_max[kSlots][kThreads];        // each thread's maxima over stretches of its packs
};

// A finishing warp's search for the largest elements.
struct Best {
    alignas(16) unsigned long long above[kBuffer + 1];   // elements above the bound (key_index), as they came
    int at_index[kBuffer];                   // elements at it
    unsigned short hot[kSlots * kThreads];   // (slot, thread) whose maximum reaches the bound
    uint32_t best_key[kMaxTop];              // the slice's best, in order
    int best_index[kMaxTop];
    int best_count;
};

struct Shared {
    uint64_t full[kStages], empty[kStages];  // the ring's chunks
    uint64_t row_full[2], row_empty[2];
    int abort_flag;
    alignas(16) Row row[2];
    Best best[2];
    Sums slice_sums[kMaxCluster];            // the first block: every slice's
    uint32_t all_key[kMaxCluster * kMaxTop];
    int all_index[kMaxCluster * kMaxTop];
};

__device__ __forceinline__ bool better(uint32_t ka, int ia, uint32_t kb, int ib) {
    return ka > kb || (ka == kb && ia < ib);
}

// an element's key and index in one word: larger goes first; below ~0 for
// any element, above 0
__device__ __forceinline__ unsigned long long key_index(uint32_t key, int i) {
    return ((unsigned long long)key << 32) | (0x7FFFFFFFu - (uint32_t)i);
}
__device__ __forceinline__ int index_of(unsigned long long c) { return (int)(0x7FFFFFFFu - (uint32_t)c); }

// the consumers' barrier, by whole warps
__device__ __forceinline__ void sync() {
    __syncwarp();
    asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
}

// The functions below run on one warp.

template <typename T>
__device__ __forceinline__ float element(const Slice<T>& s, int i) {
    return Num<T>::to_acc(s.row[i]);
}

// k rounds, each the best element after the last one: right for any values,
// taken where more elements than the buffer holds exceed the bound, or where
// a NaN hides what the maxima say.
template <typename T>
__device__ __noinline__ void top_by_rounds(const Slice<T>& s, int k, Best& sh) {
    const int lane = threadIdx.x & 31;
    unsigned long long last = ~0ull;
    int n = 0;
    for (; n < k; ++n) {
        unsigned long long best = 0;
        auto see = [&](float z, int i) {
            const unsigned long long c = key_index(order_key(z), i);
            if (c < last && c > best) best = c;
        };
        if (lane < s.head) see(element(s, lane), lane);
        const uint4* body = reinterpret_cast<const uint4*>(s.row + s.body);
#pragma unroll 4
        for (int v = s.v0 + lane; v < s.v1; v += 32) {
            float z[Slice<T>::V];
            unpack<T>(__ldg(body + v), z);
#pragma unroll
            for (int i = 0; i < Slice<T>::V; ++i) see(z[i], s.body + v * Slice<T>::V + i);
        }
        if (s.tail0 + lane < s.tail1) see(element(s, s.tail0 + lane), s.tail0 + lane);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            const unsigned long long o = __shfl_xor_sync(0xffffffffu, best, d);
            best = o > best ? o : best;
        }
        if (best == 0) break;                        // the slice holds no more elements
        if (lane == 0) {
            sh.best_key[n] = (uint32_t)(best >> 32);
            sh.best_index[n] = index_of(best);
        }
        last = best;
    }
    if (lane == 0) sh.best_count = n;
    __syncwarp();
}

// the k lowest indices of elements with this key, in order, into at_index;
// their number
template <typename T>
__device__ __noinline__ int lowest_at(const Slice<T>& s, uint32_t key, int k, Best& sh) {
    const int lane = threadIdx.x & 31;
    int found = 0;
    auto scan = [&](int begin, int end) {
        for (int base = begin; base < end && found < k; base += 32) {
            const int i = base + lane;
            const bool hit = i < end && order_key(element(s, i)) == key;
            const unsigned b = __ballot_sync(0xffffffffu, hit);
            const int at = found + __popc(b & ((1u << lane) - 1u));
            if (hit && at < k) sh.at_index[at] = i;
            found += __popc(b);
        }
    };
    scan(0, s.head);
    scan(s.body + s.v0 * Slice<T>::V, s.body + s.v1 * Slice<T>::V);
    scan(s.tail0, s.tail1);
    __syncwarp();
    return min(found, k);
}

// The slice's k best elements in order, into best_*.  `plain`: no NaN was met.
template <typename T>
__device__ __forceinline__ void top_of_slice(const Slice<T>& s, const Row& r, bool plain, int k, Best& sh) {
    constexpr int V = Slice<T>::V;
    if (!plain) {                                    // uniform over the warp
        top_by_rounds(s, k, sh);
        return;
    }
    const int lane = threadIdx.x & 31;
    // the bound: the k-th largest of the maxima of 64 pairs of threads
    const float4 m4 = reinterpret_cast<const float4*>(r.m)[lane];
    const uint32_t m0 = order_key(fmaxf(m4.x, m4.y)), m1 = order_key(fmaxf(m4.z, m4.w));
    int larger0 = 0, larger1 = 0;
#pragma unroll 8
    for (int i = 0; i < 32; ++i) {
        const uint32_t o0 = __shfl_sync(0xffffffffu, m0, i), o1 = __shfl_sync(0xffffffffu, m1, i);
        larger0 += (o0 > m0) + (o1 > m0);
        larger1 += (o0 > m1) + (o1 > m1);
    }
    const uint32_t bound = __reduce_min_sync(
        0xffffffffu, min(larger0 < k ? m0 : 0xFFFFFFFFu, larger1 < k ? m1 : 0xFFFFFFFFu));
    const float least = key_value(bound);

    // the stretches of threads' packs that reach it
    const int chunks = (s.v1 - s.v0 + kChunk - 1) / kChunk;
    const int a_slot = chunks_a_slot(s);
    const int slots = chunks ? (chunks + a_slot - 1) / a_slot : 0;
    int n = 0;
    for (int slot = 0; slot < slots; ++slot) {
        const float4 x = reinterpret_cast<const float4*>(r.slot_max[slot])[lane];
        const float q[4] = {x.x, x.y, x.z, x.w};
        if (!__any_sync(0xffffffffu, fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)) >= least)) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // (a thread without packs in the stretch has the maximum -inf)
            const bool hit = q[j] >= least && s.v0 + slot * a_slot * kChunk + lane * 4 + j < s.v1;
            const unsigned b = __ballot_sync(0xffffffffu, hit);
            if (hit) sh.hot[n + __popc(b & ((1u << lane) - 1u))] = (unsigned short)(slot * kThreads + lane * 4 + j);
            n += __popc(b);
        }
    }
    __syncwarp();

    int above = 0, at = 0;
    auto collect = [&](bool have, float z, int i) {  // the whole warp calls it
        const uint32_t key = order_key(z);
        const unsigned low = (1u << lane) - 1u;
        const unsigned ba = __ballot_sync(0xffffffffu, have && key > bound);
        const unsigned be = __ballot_sync(0xffffffffu, have && key == bound);
        if (have && key > bound) {
            const int q = above + __popc(ba & low);
            if (q < kBuffer) sh.above[q] = key_index(key, i);
        } else if (have && key == bound) {
            const int q = at + __popc(be & low);
            if (q < kBuffer) sh.at_index[q] = i;
        }
        above += __popc(ba);
        at += __popc(be);
    };
    const int ends = s.head + s.tail1 - s.tail0;     // at most 2 (V - 1) elements
    if (ends > 0) {
        const int i = lane < s.head ? lane : s.tail0 + lane - s.head;
        collect(lane < ends, lane < ends ? element(s, i) : 0.f, i);
    }
    // every pack of those stretches, four loads in flight a lane
    const uint32_t word = splat<T>(least);           // one of the row's own values: exact
    const uint4* body = reinterpret_cast<const uint4*>(s.row + s.body);
    const int items = n * a_slot * kUnroll;
    for (int base = 0; base < items; base += 128) {
        uint4 k4[4];
        int v4[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int item = base + j * 32 + lane;
            v4[j] = s.v1;
            if (item < items) {
                int entry = item / kUnroll, pack = item % kUnroll;
                if (a_slot > 1) {
                    pack += entry % a_slot * kUnroll;
                    entry /= a_slot;
                }
                const int h = sh.hot[entry];
                v4[j] = s.v0 + h / kThreads * a_slot * kChunk + h % kThreads + pack * kThreads;
            }
            if (v4[j] < s.v1) k4[j] = __ldg(body + v4[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            unsigned m = v4[j] < s.v1 ? reaching<T>(k4[j], word) : 0u;
            while (__any_sync(0xffffffffu, m != 0)) {
                const bool have = m != 0;
                const int i = have ? __ffs(m) - 1 : 0;
                m &= m - 1;
                const int w4 = i * (int)sizeof(T) / 4;
                const uint32_t w = w4 < 2 ? (w4 ? k4[j].y : k4[j].x) : (w4 == 2 ? k4[j].z : k4[j].w);
                float z;
                if constexpr (sizeof(T) == 4) {
                    z = __uint_as_float(w);
                } else {
                    const unsigned short b = (unsigned short)(w >> (16 * (i & 1)));
                    z = Num<T>::to_acc(*reinterpret_cast<const T*>(&b));
                }
                collect(have, z, s.body + v4[j] * V + i);
            }
        }
    }
    __syncwarp();
    if (above > kBuffer) {
        top_by_rounds(s, k, sh);
        return;
    }
    if (at > kBuffer) at = lowest_at(s, bound, k, sh);
    if (lane == 0) sh.best_count = min(k, above + at);
    if (lane == 0) sh.above[above] = 0;              // two at a time: below every element
    __syncwarp();
    for (int c = lane; c < above; c += 32) {
        const unsigned long long me = sh.above[c];
        int rank = 0;
#pragma unroll 4
        for (int i = 0; i < above; i += 2) {
            const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(&sh.above[i]);
            rank += (o.x > me) + (o.y > me);
        }
        if (rank < k) {
            sh.best_key[rank] = (uint32_t)(me >> 32);
            sh.best_index[rank] = index_of(me);
        }
    }
    for (int c = lane; c < at; c += 32) {
        const int me = sh.at_index[c];
        int rank = above;
        for (int i = 0; i < at; ++i) rank += sh.at_index[i] < me;
        if (rank < k) {
            sh.best_key[rank] = bound;
            sh.best_index[rank] = me;
        }
    }
    __syncwarp();
}

// the threads' sums joined: every lane gets them
__device__ __forceinline__ Sums join_row(const Row& r) {
    const int lane = threadIdx.x & 31;
    const float4 m4 = reinterpret_cast<const float4*>(r.m)[lane], s4 = reinterpret_cast<const float4*>(r.s)[lane],
                 a4 = reinterpret_cast<const float4*>(r.a)[lane];
    const float ms[4] = {m4.x, m4.y, m4.z, m4.w}, ss[4] = {s4.x, s4.y, s4.z, s4.w}, as[4] = {a4.x, a4.y, a4.z, a4.w};
    const uint32_t w = __reduce_max_sync(0xffffffffu, order_key(fmaxf(fmaxf(ms[0], ms[1]), fmaxf(ms[2], ms[3]))));
    Sums q{key_value(w), 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        Sums x{ms[i], ss[i], as[i]};
        move_to(x, q.m);
        q.s += x.s;
        q.a += x.a;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        q.s += __shfl_xor_sync(0xffffffffu, q.s, d);
        q.a += __shfl_xor_sync(0xffffffffu, q.a, d);
    }
    return q;
}

// A row's token and its logit, asked for before the row's sums are there.
struct Given {
    int64_t token;
    float logit;
};
template <typename T>
__device__ __forceinline__ Given given_of(const Params& p, int64_t row) {
    Given g;
    g.token = p.tokens[row];
    const T* z = static_cast<const T*>(p.logits) + row * p.pitch;
    g.logit = g.token >= 0 && g.token < p.vocab ? Num<T>::to_acc(z[g.token]) : 0.f;
    return g;
}

// a row's results, by threads t = 0, 1, ... of at least kMaxTop
__device__ __forceinline__ void write_row(const Params& p, int64_t row, const Given& g, const Sums& q, const Best& sh,
                                          int t) {
    const bool nothing = q.m == -INFINITY && q.s == 0.f;         // every logit is -inf
    const float log2_s = log2f(q.s);
    // log s with the distances' common residue taken out again: lse and the log
    // probabilities start from m itself, not from m scaled there and back
    const float log_s = (log2_s - residue(q.m)) * kLn2;
    const float lse = nothing ? -INFINITY : q.m + log_s;
    if (t < p.top) {
        const float v = key_value(sh.best_key[t]);
        if (p.top_logprob) p.top_logprob[row * p.top + t] = nothing ? -INFINITY : (v - q.m) - log_s;
        if (p.top_index) p.top_index[row * p.top + t] = sh.best_index[t];
    }
    if (t == 0) {
        float lp;
        if (g.token < 0) lp = 0.f;                               // ignored
        else if (g.token >= p.vocab) lp = __uint_as_float(0x7FC00000u);
        else lp = nothing ? -INFINITY : (g.logit - q.m) - log_s;
        p.logprob[row] = lp;
        if (p.lse) p.lse[row] = lse;
        if (p.entropy) p.entropy[row] = nothing ? 0.f : (log2_s - q.a / q.s) * kLn2;
    }
}

// store into the first block of the cluster
__device__ __forceinline__ void give_first(const void* local, uint32_t value) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(local)));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(value) : "memory");
}
// (by whole warps: one lane's work may come before either)
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Persistent blocks (a row cut over a cluster: one unit each) of three roles.
// The loading warp copies chunk after chunk of the block's rows into a ring,
// whatever the others are at; the consumers sum them up; the finishing warp
// joins a row's sums and finds its largest elements while the consumers are
// at the next row.
template <typename T>
__global__ void __launch_bounds__(kBlockThreads, kBlocksPerSm) forward_kernel(const Params p) {
    extern __shared__ __align__(128) unsigned char ring[];
    __shared__ Shared sh;
    const int parts = p.cluster;
    const int t = threadIdx.x;
    volatile int* abort_flag = &sh.abort_flag;
    if (t == 0) {
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(&sh.full[i], 1);
            tc::mbar_init(&sh.empty[i], kWarps);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&sh.row_full[i], kWarps);
            tc::mbar_init(&sh.row_empty[i], 1);
        }
        sh.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();
    if (parts > 1) cluster_arrive();

    if (t >= kThreads + 32) {
        // the finishing warps: every other row each, from the row buffer of its own
        const int lane = t & 31, buf = (t - kThreads - 32) >> 5;
        Best& best = sh.best[buf];
        uint32_t phase = 0;
        for (int64_t u = blockIdx.x + (int64_t)buf * gridDim.x; u < p.units; u += 2 * (int64_t)gridDim.x, phase ^= 1) {
            const int64_t row = u / parts;
            const int part = (int)(u % parts);       // = the block's rank in its cluster
            const Slice<T> slice = slice_of(static_cast<const T*>(p.logits) + row * p.pitch, p.vocab, part, parts);
            const Given given = parts == 1 ? given_of<T>(p, row) : Given{0, 0.f};
            if (!tc::warp_wait(&sh.row_full[buf], phase, abort_flag, p.err)) break;
            const Sums q = join_row(sh.row[buf]);
            if (p.top > 0) top_of_slice(slice, sh.row[buf], q.s == q.s, p.top, best);
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sh.row_empty[buf]);
            if (parts == 1) {
                write_row(p, row, given, q, best, lane);
                __syncwarp();
            } else {
                // every slice's results go to the first block
                cluster_wait();                      // all blocks of the cluster run
                if (lane == 0) {
                    give_first(&sh.slice_sums[part].m, __float_as_uint(q.m));
                    give_first(&sh.slice_sums[part].s, __float_as_uint(q.s));
                    give_first(&sh.slice_sums[part].a, __float_as_uint(q.a));
                }
                if (p.top > 0) {
                    const bool some = lane < best.best_count;
                    give_first(&sh.all_key[part * kMaxTop + lane], some ? best.best_key[lane] : 0u);      // 0: below every element
                    give_first(&sh.all_index[part * kMaxTop + lane], some ? (uint32_t)best.best_index[lane] : 0u);
                }
                cluster_arrive();
                cluster_wait();
                return;                              // a cluster's block has one unit
            }
        }
        if (parts > 1) {                             // the other warp, or a wait that ran out
            cluster_wait();
            cluster_arrive();
            cluster_wait();
        }
        return;
    }
    if (t >= kThreads) {
        if (t == kThreads) {
            uint32_t stage = 0, phase = 0, armed = 0, parity = 0;
            bool ok = true;
            for (int64_t u = blockIdx.x; u < p.units && ok; u += gridDim.x) {
                const T* z = static_cast<const T*>(p.logits) + u / parts * p.pitch;
                const Slice<T> s = slice_of(z, p.vocab, (int)(u % parts), parts);
                const uint4* body = reinterpret_cast<const uint4*>(z + s.body);
                for (int v = s.v0; v < s.v1; v += kChunk) {
                    if (!tc::mbar_wait(&sh.empty[stage], phase ^ 1, abort_flag, p.err)) {
                        ok = false;
                        break;
                    }
                    const uint32_t bytes = (uint32_t)min(kChunk, s.v1 - v) * 16;
                    tc::mbar_arrive_expect_tx(&sh.full[stage], bytes);
                    armed |= 1u << stage;
                    parity = (parity & ~(1u << stage)) | (phase << stage);
                    asm volatile(
                        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                            tc::smem_u32(ring) + stage * (kChunk * 16)),
                        "l"(body + v), "r"(bytes), "r"(tc::smem_u32(&sh.full[stage]))
                        : "memory");
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            if (*abort_flag)                         // nothing may land after the block has left
                for (int i = 0; i < kStages; ++i)
                    if ((armed >> i) & 1u) tc::mbar_wait_drain(&sh.full[i], (parity >> i) & 1u);
        }
        __syncwarp();
        if (parts > 1) {
            cluster_wait();
            cluster_arrive();
            cluster_wait();
        }
        return;
    }

    uint32_t stage = 0, phase = 0, buf = 0, row_phase = 0;
    const uint32_t none = splat<T>(-INFINITY);
    const Given given = parts > 1 && blockIdx.x % parts == 0 ? given_of<T>(p, blockIdx.x / parts) : Given{0, 0.f};
    for (int64_t u = blockIdx.x; u < p.units; u += gridDim.x) {
        const T* z = static_cast<const T*>(p.logits) + u / parts * p.pitch;
        const Slice<T> slice = slice_of(z, p.vocab, (int)(u % parts), parts);
        Sums q{-INFINITY, 0.f, 0.f};
        if (t < slice.head) take(q, Num<T>::to_acc(z[t]));
        if (slice.tail0 + t < slice.tail1) take(q, Num<T>::to_acc(z[slice.tail0 + t]));
        const int a_slot = p.top > 0 ? chunks_a_slot(slice) : 0;
        int left = a_slot, slot = 0;
        float slot_top = -INFINITY;
        // the buffer's last row has been finished
        const bool ok = tc::warp_wait(&sh.row_empty[buf], row_phase ^ 1, abort_flag, p.err);
        Row& r = sh.row[buf];
        for (int v = slice.v0; v < slice.v1 && ok; v += kChunk) {
            if (tc::warp_wait(&sh.full[stage], phase, abort_flag, p.err)) {
                const uint4* chunk = reinterpret_cast<const uint4*>(ring + stage * (kChunk * 16)) + t;
                const int mine = slice.v1 - v - t;   // this thread's packs: at 0, kThreads, ... below this
                uint4 k[kUnroll];
                if (mine > (kUnroll - 1) * kThreads) {
#pragma unroll
                    for (int i = 0; i < kUnroll; ++i) k[i] = chunk[i * kThreads];
                } else {
                    // -inf past the slice's end: it weighs nothing
#pragma unroll
                    for (int i = 0; i < kUnroll; ++i)
                        k[i] = i * kThreads < mine ? chunk[i * kThreads] : make_uint4(none, none, none, none);
                }
                if (mine > 0) slot_top = fmaxf(slot_top, take<T>(q, k));
            }
            __syncwarp();
            if ((t & 31) == 0) tc::mbar_arrive(&sh.empty[stage]);
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1;
            }
            if (--left == 0 || (p.top > 0 && v + kChunk >= slice.v1)) {
                r.slot_max[slot++][t] = slot_top;
                slot_top = -INFINITY;
                left = a_slot;
            }
        }
        r.m[t] = q.m;
        r.s[t] = q.s;
        r.a[t] = q.a;
        __syncwarp();
        if ((t & 31) == 0) tc::mbar_arrive(&sh.row_full[buf]);
        if (++buf == 2) {
            buf = 0;
            row_phase ^= 1;
        }
    }
    if (parts == 1) return;
    cluster_wait();
    cluster_arrive();
    cluster_wait();
    if (blockIdx.x % parts != 0) return;
    // the first block's consumers join the slices
    Sums q = sh.slice_sums[0];
    for (int r = 1; r < parts; ++r) q = join(q, sh.slice_sums[r]);
    if (p.top > 0) {
        // an element's rank: its place in its own slice, and in each other slice the elements that go before it
        for (int e = t; e < parts * kMaxTop; e += kThreads) {
            const int r = e / kMaxTop;
            const uint32_t key = sh.all_key[e];
            const int index = sh.all_index[e];
            if (key == 0) continue;
            int rank = e % kMaxTop;
#pragma unroll
            for (int o = 0; o < kMaxCluster; ++o) {
                if (o >= parts || o == r) continue;
                int n = 0;                           // in order: the count is a place, found by halving
                const int b = o * kMaxTop;
#pragma unroll
                for (int step = kMaxTop / 2; step > 0; step >>= 1)
                    if (n + step <= p.top && better(sh.all_key[b + n + step - 1], sh.all_index[b + n + step - 1], key, index))
                        n += step;
                if (n + 1 <= p.top && better(sh.all_key[b + n], sh.all_index[b + n], key, index)) ++n;
                rank += n;
            }
            if (rank < p.top) {
                sh.best[0].best_key[rank] = key;
                sh.best[0].best_index[rank] = index;
            }
        }
        sync();
    }
    write_row(p, blockIdx.x / parts, given, q, sh.best[0], t);
}

// One block takes a stretch of a row.  Every element is read and written by
// the same thread, so dlogits may be the logits.  With log p = z - lse and c =
// dlogprob + dH H, dz = -p (c + dH log p), and dlogprob more at the token: lse is
// subtracted first, so that errors are of the size of log p and not of lse.  p is
// formed 2^24 times too large and the bracket as much too small: log p, some -90
// where p passes 2^-126, lifts such gradients back into the normal range.
template <typename T>
__global__ void __launch_bounds__(256) backward_kernel(const GradParams p) {
    constexpr int V = 16 / sizeof(T);
    const int64_t row = blockIdx.x / p.chunks;
    const int part = (int)(blockIdx.x % p.chunks);
    const T* z = static_cast<const T*>(p.logits) + row * p.pitch;
    T* d = static_cast<T*>(p.dlogits) + row * p.d_pitch;
    const Slice<T> s = slice_of(z, p.vocab, part, p.chunks);
    const int t = threadIdx.x;
    const uint4* body = reinterpret_cast<const uint4*>(z + s.body);
    uint4 k4[kGradPacks];
#pragma unroll
    for (int i = 0; i < kGradPacks; ++i)
        if (s.v0 + t + i * 256 < s.v1) k4[i] = body[s.v0 + t + i * 256];
    const float lse = p.lse[row];
    const int64_t token64 = p.dlogprob ? p.tokens[row] : -1;
    const int token = token64 < 0 || token64 >= p.vocab ? -1 : (int)token64;
    float dlp = token64 >= 0 ? p.dlogprob[row] : 0.f;
    if (token64 >= p.vocab) dlp = __uint_as_float(0x7FC00000u);
    const float dh = p.dentropy ? p.dentropy[row] : 0.f;
    const float h = p.dentropy ? p.entropy[row] : 0.f;
    const bool nothing = lse == -INFINITY;
    const float c = fmaf(dh, h, dlp);
    auto grad = [&](float v, int i) -> float {           // any values
        if (nothing) return 0.f;
        const float logp = v - lse, q = exp2_small(logp * kLog2e);
        // a probability of zero contributes nothing, whatever its logarithm
        float g = q == 0.f && dlp == dlp ? 0.f : -q * fmaf(dh, logp + h, dlp);
        if (i == token) g += dlp;
        return g;
    };
    if (t < s.head) d[t] = Num<T>::from_acc(grad(Num<T>::to_acc(z[t]), t));
    const bool same = ((reinterpret_cast<uintptr_t>(d) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
    constexpr float LARGER = 16777216.f, LEAST = 0x1p-100f;      // (brackets that 2^-24 leaves all their digits)
    const bool digits = (fabsf(c) >= LEAST || c == 0.f) && (fabsf(dh) >= LEAST || dh == 0.f);
    const bool quick = near_zero(lse) && same && (digits || c != c);
    const uint32_t low = floor_of<T>(quick ? lse : 0.f);
    const float c_less = -c / LARGER, dh_less = -dh / LARGER;
    const F2 scale2 = pack_f2(kLog2e, kLog2e), larger2 = pack_f2(24.f, 24.f), minus_lse2 = pack_f2(-lse, -lse),
             c2 = pack_f2(c_less, c_less), dh2 = pack_f2(dh_less, dh_less);
#pragma unroll
    for (int pack = 0; pack < kGradPacks; ++pack) {
        const int v = s.v0 + t + pack * 256;
        if (v >= s.v1) break;
        const uint4 k = k4[pack];
        const int at = s.body + v * V;
        if (quick) {
            const uint32_t w[4] = {floor_word<T>(k.x, low), floor_word<T>(k.y, low), floor_word<T>(k.z, low),
                                   floor_word<T>(k.w, low)};
            F2 g[V / 2];
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                const F2 logp = add2(pair_of<T>(w, j), minus_lse2);
                float lo, hi;
                unpack_f2(fma2(logp, scale2, larger2), lo, hi);
                g[j] = mul2(pack_f2(exp2_fast(lo), exp2_fast(hi)), fma2(logp, dh2, c2));
            }
            if ((unsigned)(token - at) < (unsigned)V) {
#pragma unroll
                for (int j = 0; j < V / 2; ++j) {
                    float lo, hi;
                    unpack_f2(g[j], lo, hi);
                    if (token == at + 2 * j) lo += dlp;
                    if (token == at + 2 * j + 1) hi += dlp;
                    g[j] = pack_f2(lo, hi);
                }
            }
            uint4 o;
            uint32_t* e = reinterpret_cast<uint32_t*>(&o);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                float lo, hi;
                unpack_f2(g[j], lo, hi);
                if constexpr (sizeof(T) == 4) {
                    e[2 * j] = __float_as_uint(lo);
                    e[2 * j + 1] = __float_as_uint(hi);
                } else if constexpr (std::is_same_v<T, __half>) {
                    const __half2 y = __floats2half2_rn(lo, hi);
                    e[j] = *reinterpret_cast<const uint32_t*>(&y);
                } else {
                    const __nv_bfloat162 y = __floats2bfloat162_rn(lo, hi);
                    e[j] = *reinterpret_cast<const uint32_t*>(&y);
                }
            }
            *reinterpret_cast<uint4*>(d + at) = o;
        } else {
            float x[V];
            unpack<T>(k, x);
#pragma unroll
            for (int i = 0; i < V; ++i) d[at + i] = Num<T>::from_acc(grad(x[i], at + i));
        }
    }
    if (s.tail0 + t < s.tail1) d[s.tail0 + t] = Num<T>::from_acc(grad(Num<T>::to_acc(z[s.tail0 + t]), s.tail0 + t));
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

// Blocks on one row: where fewer rows than two blocks an SM, a row is cut so
// that the blocks fill them, as long as a slice keeps 12288 elements: joining
// more slices costs more than they save ([1, 50264] FP16 with 20 alternatives:
// 14.4 us in 8 slices, 11.1 in 4, 10.7 in 2; without alternatives 4.0, 4.2 and
// 5.2).
inline int cluster_of(int64_t rows, int64_t vocab, int sm_count) {
    int c = 1;
    while (c < kMaxCluster && rows * c * 2 <= 2 * (int64_t)sm_count && vocab / (2 * c) >= 12288) c *= 2;
    return c;
}

template <typename T>
cudaError_t launch_forward(const Params& p, int sm_count, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    const int smem = kStages * kChunk * 16;
    const cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(forward_kernel<T>), smem);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(p.cluster > 1 ? p.units : min64(p.units, (int64_t)sm_count * kBlocksPerSm)));
    cfg.blockDim = dim3(kBlockThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, forward_kernel<T>, p);
}

}  // namespace score
}  // namespace olc

using namespace olc;

struct olc_token_log_probs_plan {
    PlanState state;
    olc_dtype dtype;
    int64_t rows, vocab;
    int top;
};

extern "C" {

olc_status olc_token_log_probs_plan_create(int64_t rows, int64_t vocab, int top, olc_dtype dtype,
                                           olc_token_log_probs_plan** out) {
    if (!out) return OLC_ERR_NULL;
    *out = nullptr;
    if (!plan_dtype_ok(dtype)) return OLC_ERR_DTYPE;
    if (rows < 0 || vocab < 0) return OLC_ERR_NEGATIVE_DIM;
    if (vocab == 0 || vocab >= (int64_t(1) << 31) - 65536 || rows >= (int64_t(1) << 27)) return OLC_ERR_INVALID;
    if (top < 0 || top > OLC_MAX_TOP || top > vocab) return OLC_ERR_INVALID;
    olc_token_log_probs_plan* p = new (std::nothrow) olc_token_log_probs_plan;
    if (!p) return OLC_ERR_OOM;
    p->state.init();
    p->dtype = dtype;
    p->rows = rows;
    p->vocab = vocab;
    p->top = top;
    *out = p;
    return OLC_OK;
}

void olc_token_log_probs_plan_destroy(olc_token_log_probs_plan* plan) {
    if (!plan) return;
    plan->state.destroy();
    delete plan;
}

olc_status olc_token_log_probs_forward(olc_token_log_probs_plan* plan, const void* logits, int64_t pitch,
                                       const int64_t* tokens, float* logprob, float* entropy, float* lse,
                                       float* top_logprob, int64_t* top_index, void* stream) {
    static_assert(score::kMaxTop == OLC_MAX_TOP, "");
    if (!plan) return OLC_ERR_NULL;
    if (plan->rows == 0) return OLC_OK;
    if (!logits || !tokens || !logprob) return OLC_ERR_NULL;
    const int64_t eb = plan_elem_bytes(plan->dtype);
    if (plan->rows > 1 && (pitch < plan->vocab || !plan_fits(plan->rows, pitch, eb))) return OLC_ERR_INVALID;
    if (plan_misaligned(logits, eb) || plan_misaligned(tokens, 8) || plan_misaligned(logprob, 4) ||
        plan_misaligned(entropy, 4) || plan_misaligned(lse, 4) || plan_misaligned(top_logprob, 4) ||
        plan_misaligned(top_index, 8))
        return OLC_ERR_INVALID;
    const olc_status st = plan->state.bind();
    if (st != OLC_OK) return st;
    const int cluster = score::cluster_of(plan->rows, plan->vocab, plan->state.sm_count);
    score::Params p{logits, tokens, logprob, entropy, lse, top_logprob, top_index, pitch, (int)plan->vocab,
                    top_logprob || top_index ? plan->top : 0, cluster, plan->rows * cluster, device_error_word()};
    return score::by_type(plan->dtype, [&](auto tag) {
        return plan_status(score::launch_forward<decltype(tag)>(p, plan->state.sm_count, static_cast<cudaStream_t>(stream)));
    });
}

olc_status olc_token_log_probs_backward(olc_token_log_probs_plan* plan, const void* logits, int64_t pitch,
                                        const int64_t* tokens, const float* lse, const float* entropy,
                                        const float* dlogprob, const float* dentropy, void* dlogits, int64_t d_pitch,
                                        void* stream) {
    if (!plan) return OLC_ERR_NULL;
    if (plan->rows == 0) return OLC_OK;
    if (!logits || !lse || !dlogits || (dlogprob && !tokens) || (dentropy && !entropy)) return OLC_ERR_NULL;
    const int64_t eb = plan_elem_bytes(plan->dtype);
    if (plan->rows > 1 && (pitch < plan->vocab || d_pitch < plan->vocab || !plan_fits(plan->rows, pitch, eb) ||
                           !plan_fits(plan->rows, d_pitch, eb)))
        return OLC_ERR_INVALID;
    if (plan_misaligned(logits, eb) || plan_misaligned(dlogits, eb) || plan_misaligned(tokens, 8) ||
        plan_misaligned(lse, 4) || plan_misaligned(entropy, 4) || plan_misaligned(dlogprob, 4) ||
        plan_misaligned(dentropy, 4))
        return OLC_ERR_INVALID;
    const olc_status st = plan->state.bind();
    if (st != OLC_OK) return st;
    // slices of at most kGradPacks packs a thread
    const int64_t packs = plan->vocab / (16 / eb);
    const int64_t chunks = max64(1, ceil_div(packs, 256 * score::kGradPacks));
    if (plan->rows * chunks > 0x7fffffffLL) return OLC_ERR_INVALID;
    score::GradParams p{logits, tokens, lse, entropy, dlogprob, dentropy, dlogits, pitch, d_pitch, plan->rows,
                        (int)plan->vocab, (int)chunks};
    return score::by_type(plan->dtype, [&](auto tag) {
        using T = decltype(tag);
        return plan_status(plan_launch(score::backward_kernel<T>, dim3((unsigned)(plan->rows * chunks)), dim3(256), 0,
                                      static_cast<cudaStream_t>(stream), p));
    });
}

}  // extern "C"
