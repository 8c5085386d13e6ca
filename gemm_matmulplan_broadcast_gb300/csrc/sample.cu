// One token for each row of logits [rows, vocab] from one uniform number u a row:
// temperature, top-k, top-p and min-p, then the inverse of the distribution that is left.
//
//   w_j = e^((z_j - m) / T),  m = max_j z_j
//   kept: a prefix of the order (value, then the lower index); where it ends is the
//         strictest of the k-th token, the first whose prefix weighs top_p of the k
//         tokens' weight, and the last with w_j >= min_p
//   token: the lowest kept j with  sum_{kept i <= j} w_i > u sum_kept w
//
// Choices hang on sums next to borders, so the weights are 64-bit integers
// (2^43 for the largest): their sums are the same in any order, across warps, blocks
// and passes.  Tokens within 12 octaves of the largest are heavy: weights good to 2^-38 of
// themselves (x = (z - m) log2(e) / T in two float32s, a table of 2^(i/64), the rest of the
// exponential in two parts).  The light ones have float32's rounding, 2^-23 of themselves, so
// 2^-35 of the largest weight.  A row with more than 512 heavy tokens counts fewer of them as heavy,
// down to those within 0.75 octaves; its light weights are scaled to stay within 32 bits, so that their
// unit is up to 2^-31 of the largest weight: they have half of that on top, and those below it are 0.
//
// A row is a cluster of blocks, each with a slice of it, read again by each pass, from L2:
//   the maximum; then
//   top-k: a bound that the k largest reach (the k-th largest of the threads' own maxima),
//     the list of the tokens that reach it, and everything else on that list;
//   or the list of the heavy tokens with the light weights' sum, for top-p alone by the
//     exponential unit, good to 2^-16 of it (2^-12 with 4096 terms a thread).  If what is kept ends
//     among the heavy tokens wherever the sum lies within that, the list gives the token.  Otherwise the sum again, as
//     accurate as the weights, with a histogram of counts over 4096 equal steps of x, 45
//     octaves: it shows to a fraction of a percent in which steps the light
//     weights reach top-p, a second list takes those steps' tokens, the weights above
//     them are summed, and the cut is found exactly;
//   without a list that holds all that is kept, sums by slices, warps and packs,
//     the listed tokens added to each, lead to the token.
// Rows that none of this fits (far from zero in units of the temperature, many equal logits,
// large k) go element by element: a histogram, or bisection over values.
//
// Rows that nothing cuts need no order: every block's list stays its own.
//
// Bound by instructions and, with few rows, by the passes' latency: about 25 issue slots an
// element for the accurate sum, 12 for the rough one.  Measured: BF16 [1024, 50257] with
// top-p 173 us (the logits' bytes: 15.5; one row in eight has its cut among the light
// tokens and takes 90 us of its SM's quarter), FLOAT [64, 131072] unfiltered 40 us, BF16
// [256, 50257] of mixed settings 82 us (the SM that gets the most such rows), one
// row of 50257 16 us.
#include <cmath>
#include <cstring>
#include <new>
#include <type_traits>

#include "plan_state.h"
#include "row_packs.cuh"

namespace olc {
namespace sample {

using u64 = unsigned long long;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBlocksPerSm = 4;
constexpr int kMaxCluster = 8;
constexpr int kBins = 4096;
constexpr int kOctaves = 45;            // below 2^-45 of the largest a weight is 0
constexpr int kList = 1024;
constexpr int kMostHeavy = 512;         // of a row: the list is ordered, so that more cost more than the cuts they decide save
constexpr int kSmall = 128;             // entries up to which a list is ordered by counting
constexpr int kBracket = 512;           // tokens of the steps in which top-p's cut lies
constexpr int kTurns = 6;               // tries to find the steps of a cut
constexpr int kMostK = kThreads * 7 / 8;    // the largest top_k that the threads' maxima bound
constexpr int kOne = 43;                // the largest weight is 2^43; vocab <= 2^20
constexpr float kHeavy = -12.f;         // x from which on weights are formed in two parts (or nearer to 0: Scale)

struct Power {                          // 2^(i/64)
    u64 fixed;                          // scaled by 2^43
    float hi, lo;
};

struct Params {
    const void* logits;
    const float* uniforms;
    const float* temperature;   // may be null: 1
    const int* top_k;           // may be null: all
    const float* top_p;         // may be null: 1
    const float* min_p;         // may be null: 0
    int64_t* tokens;
    float* logprob;             // may be null
    int64_t pitch;
    int vocab;
    int cluster;
    Power powers[64];
};

// The row's scale: x = (z - m) c with c = log2(e) / T in two parts
struct Scale {
    float m, hi, lo;
    float least;            // z - m is not taken below this one (x = -64, where weights are 0)
    int exact;              // the light weights' differences z - m in two parts
    float heavy;            // x from which on tokens are heavy: kHeavy, nearer to 0 in rows with too many of those
    int shift;              // light weights are scaled by 2^(43 - shift): 2^31 at the limit of the heavy ones
};

// what one block tells the others of its cluster
struct Found {
    u64 a, b, c;
    int i, j;
};

struct Shared {
    Power powers[64];
    u64 warp[kWarps], warp2[kWarps];
    u64 exchange[2][2];         // [parity]: sums of this block
    Found found[2];             // of the first block: [parity]
    int listed;                 // entries of this block's list
    int listed2;
    u64 light[kWarps];          // sums of the warps' parts without the listed entries
    Scale scale;
    double min_distance;
    unsigned min_key;
    alignas(16) unsigned bins[kBins];   // counts of this block, then (its share of the bins) of the cluster; later
                                        // weights by rank
    alignas(16) u64 list[kList];        // key above ~index; the first block's takes the others' in
    u64 weight[kList];
    alignas(16) u64 list2[kBracket];
    u64 weight2[kBracket];
};

// ---- values and weights -------------------------------------------------------

// Unsigned order of the values: -inf lowest, -0 equal to +0 (no NaN comes here)
__device__ __forceinline__ unsigned order_key(float z) {
    const unsigned b = __float_as_uint(z + 0.0f);
    return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(unsigned k) { return __uint_as_float((k >> 31) ? k & 0x7FFFFFFFu : ~k); }
__device__ __forceinline__ u64 entry_of(float z, int i) { return ((u64)order_key(z) << 32) | (unsigned)~i; }
__device__ __forceinline__ int index_of(u64 entry) { return (int)~(unsigned)entry; }
__device__ __forceinline__ float value_of(u64 entry) { return key_value((unsigned)(entry >> 32)); }

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// By one thread: double precision costs 64 times as much.  `min_distance`: w >= min_p
// <=> z - m >= it.
__device__ __forceinline__ Scale scale_of(float temperature, float min_p, double& min_distance) {
    Scale s;
    s.m = 0.f;
    const double heat = (double)fminf(fmaxf(temperature, 0x1p-96f), 0x1p96f);
    const double c = 1.4426950408889634 / heat;
    s.hi = (float)c;
    s.lo = (float)(c - (double)s.hi);
    s.least = -64.f / s.hi;
    s.exact = 1;
    s.heavy = kHeavy;
    s.shift = 0;
    min_distance = min_p > 0.f ? heat * log((double)min_p) : 0.0;
    return s;
}

// steps of x, 0 at the maximum (an infinity for z = -inf)
constexpr float kStepsPerOctave = (float)kBins / kOctaves;
__device__ __forceinline__ float step_of(float z, const Scale& s) { return (z - s.m) * -s.hi * kStepsPerOctave; }

// the exponential unit, good to 2^-22 of the result
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

constexpr float kMagic = 12582912.f;            // 1.5 2^23: adding it rounds to an integer in the low bits
constexpr float kLn2 = 0.69314718055994531f, kLn2Lo = 0.69314718055994531 - (double)0.69314718055994531f;

// 2^x, x = hi + lo in [kHeavy, 0]: 2^(i/64) (1 + e), e = 2^r - 1 with |r| <= 2^-7
__device__ __forceinline__ u64 heavy_weight(float hi, float lo, const Power* powers) {
    const float rounded = fmaf(hi, 64.f, kMagic);
    const int k = __float_as_int(rounded) - __float_as_int(kMagic);
    const float r = fmaf(rounded - kMagic, -0x1p-6f, hi);       // exact
    const Power t = powers[k & 63];
    // r ln 2 in two parts, and the higher terms of the exponential's series
    const float ph = r * kLn2;
    const float pl = fmaf(lo, kLn2, fmaf(r, kLn2Lo, fmaf(r, kLn2, -ph)));
    const float s = ph + pl;
    const float q = s * s * fmaf(s, fmaf(s, 1.f / 24.f, 1.f / 6.f), 0.5f);
    // 2^(i/64) e: its upper part as an integer of 2^-28, then what is left of it
    const float a = t.hi * ph;
    const float upper = fmaf(a, 0x1p28f, kMagic);
    const float rest = fmaf(upper - kMagic, -0x1p-28f, a) +
                       fmaf(t.lo, ph, fmaf(t.hi, pl + q, fmaf(t.hi, ph, -a)));
    const long long w = (long long)t.fixed + ((long long)(__float_as_int(upper) - __float_as_int(kMagic)) << (kOne - 28)) +
                        __float2int_rn(rest * 0x1p43f);
    const int down = -(k >> 6);
    return (u64)(w + ((1ll << down) >> 1)) >> down;
}

// 2^x below 2^-12, scaled by 2^43: 2^f by a polynomial fitted to it on [-1/2, 1/2]
// (Remez' exchange, relative error 2^-29 before its roundings) and the integer part added to the exponent
__device__ __forceinline__ constexpr float poly(int i) {
    constexpr float c[7] = {0x1.000000p+0f, 0x1.62e430p-1f, 0x1.ebfbdap-3f, 0x1.c6aed4p-5f,
                            0x1.3b2dbcp-7f, 0x1.5f456ap-10f, 0x1.41d334p-13f};
    return c[i] * 0x1p43f;
}
// (d = z - m, e what it lost; x - n is one fused operation's rounding of 2^-26)
template <bool EXACT>
__device__ __forceinline__ unsigned light_weight(float d, float e, const Scale& s) {
    const float magic = kMagic - (float)s.shift, rounded = fmaf(d, s.hi, magic);
    float f = fmaf(d, s.lo, fmaf(d, s.hi, magic - rounded));
    if constexpr (EXACT) f = fmaf(e, s.hi, f);
    float p = poly(6);
#pragma unroll
    for (int i = 5; i >= 0; --i) p = fmaf(p, f, poly(i));
    return __float2uint_rn(__int_as_float(__float_as_int(p) + (__float_as_int(rounded) << 23)));
}
// z - m, and what that lost (Knuth's two-sum)
__device__ __forceinline__ float difference(float z, float m, float& lost) {
    const float d = z - m, b = z - d;
    lost = (z - (d + b)) + (b - m);
    return d;
}

__device__ __forceinline__ u64 weight_of(float z, const Scale& s, const Power* powers) {
    float e;
    const float d = difference(z, s.m, e), hi = d * s.hi;
    if (hi >= s.heavy) return heavy_weight(hi, fmaf(e, s.hi, fmaf(d, s.lo, fmaf(d, s.hi, -hi))), powers);
    if (!(d >= s.least)) return 0;
    return (u64)(s.exact ? light_weight<true>(d, e, s) : light_weight<false>(d, 0.f, s)) << s.shift;
}

// ---- words of a pack ----------------------------------------------------------------

template <typename T>
__device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b) {
    if constexpr (sizeof(T) == 4) return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    uint32_t r;
    if constexpr (std::is_same_v<T, __half>) asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <typename T>
__device__ __forceinline__ uint32_t max_nan_word(uint32_t a, uint32_t b) {
    if constexpr (sizeof(T) == 4) return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
    uint32_t r;
    if constexpr (std::is_same_v<T, __half>) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// an element of a word (float32: the word)
template <typename T>
__device__ __forceinline__ float of_word(uint32_t w, int half) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w);
    if constexpr (std::is_same_v<T, __nv_bfloat16>) return __uint_as_float(half ? w & 0xFFFF0000u : w << 16);
    const unsigned short b = (unsigned short)(half ? w >> 16 : w);
    return Num<T>::to_acc(*reinterpret_cast<const T*>(&b));
}
// the largest of a word's elements, NaN if one is
template <typename T>
__device__ __forceinline__ float word_max(uint32_t w) {
    return sizeof(T) == 4 ? __uint_as_float(w) : max_nan(of_word<T>(w, 0), of_word<T>(w, 1));
}
// both halves of a word hold the largest value that is not above v (float32: v)
template <typename T>
__device__ __forceinline__ uint32_t splat_down(float v) {
    if constexpr (sizeof(T) == 4) return __float_as_uint(v);
    unsigned short b;
    if constexpr (std::is_same_v<T, __half>) b = __half_as_ushort(__float2half_rd(v));
    else b = __bfloat16_as_ushort(__float2bfloat16_rd(v));
    return b | ((uint32_t)b << 16);
}
// whether an element of the word reaches the other's
template <typename T>
__device__ __forceinline__ bool reaches(uint32_t w, uint32_t least) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w) >= __uint_as_float(least);
    else if constexpr (std::is_same_v<T, __half>)
        return __hge2_mask(*reinterpret_cast<const __half2*>(&w), *reinterpret_cast<const __half2*>(&least)) != 0;
    else
        return __hge2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w), *reinterpret_cast<const __nv_bfloat162*>(&least)) != 0;
}
// all bits of the elements of w that reach least's
template <typename T>
__device__ __forceinline__ uint32_t reach_mask(uint32_t w, uint32_t least) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w) >= __uint_as_float(least) ? 0xFFFFFFFFu : 0u;
    else if constexpr (std::is_same_v<T, __half>)
        return __hge2_mask(*reinterpret_cast<const __half2*>(&w), *reinterpret_cast<const __half2*>(&least));
    else
        return __hge2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w), *reinterpret_cast<const __nv_bfloat162*>(&least));
}
// The least value of the type that is heavy, as a word (by one warp): by a search
// over the order of the type's values, in which what is heavy grows.
template <typename T>
__device__ __forceinline__ uint32_t heavy_word(const Scale& s) {
    constexpr uint32_t SIGN = sizeof(T) == 4 ? 0x80000000u : 0x8000u, ALL = SIGN | (SIGN - 1);
    auto place = [](uint32_t b) { return b & SIGN ? ~b & ALL : b | SIGN; };
    auto bits = [](uint32_t k) { return k & SIGN ? k & ~SIGN : ~k & ALL; };
    const uint32_t lane = threadIdx.x & 31;
    uint32_t lo = place(splat_down<T>(__fadd_rd(s.m, 1.01f * s.heavy / s.hi)) & ALL), hi = place(splat_down<T>(s.m) & ALL);
    while (lo < hi) {                                   // hi is heavy, lo may be
        const uint32_t each = (hi - lo) / 32 + 1, mine = min(lo + lane * each, hi);
        const unsigned heavy = __ballot_sync(0xffffffffu, (of_word<T>(bits(mine), 0) - s.m) * s.hi >= s.heavy);
        const int first = heavy ? __ffs(heavy) - 1 : 32;
        const uint32_t from = lo;
        if (first < 32) hi = min(hi, from + first * each);
        if (first > 0) lo = min(hi, from + (first - 1) * each + 1);
    }
    return sizeof(T) == 4 ? bits(lo) : bits(lo) * 0x10001u;
}
// light_weight of two elements, the same operations in the same order; MASKED: those of
// steps below `low`.  11 paired FP32 operations, 17 with EXACT differences.
template <bool EXACT, bool MASKED>
__device__ __forceinline__ u64 light_weights(F2 z, const Scale& s, float low) {
    const F2 minus = both(-1.f), minus_m = both(-s.m), c = both(s.hi), magic = both(kMagic - (float)s.shift);
    const F2 d = add2(z, minus_m), rounded = fma2(d, c, magic);
    F2 f = fma2(d, both(s.lo), fma2(d, c, fma2(rounded, minus, magic)));
    if constexpr (EXACT) {
        const F2 b = fma2(d, minus, z);
        f = fma2(add2(fma2(add2(d, b), minus, z), add2(b, minus_m)), c, f);
    }
    F2 p = both(poly(6));
#pragma unroll
    for (int i = 5; i >= 0; --i) p = fma2(p, f, both(poly(i)));
    float p0, p1, r0, r1;
    unpack_f2(p, p0, p1);
    unpack_f2(rounded, r0, r1);
    unsigned w0 = __float2uint_rn(__int_as_float(__float_as_int(p0) + (__float_as_int(r0) << 23)));
    unsigned w1 = __float2uint_rn(__int_as_float(__float_as_int(p1) + (__float_as_int(r1) << 23)));
    if constexpr (MASKED) {
        float d0, d1;
        unpack_f2(d, d0, d1);
        if (!(d0 * -s.hi * kStepsPerOctave < low)) w0 = 0;
        if (!(d1 * -s.hi * kStepsPerOctave < low)) w1 = 0;
    }
    return (u64)w0 + w1;                        // (next to the limit of the heavy tokens both may round to 2^31)
}

// Rows whose maximum is so far from zero, in units of the temperature, that the type's steps
// there span several octaves are not worked on by words.
template <typename T>
__device__ __forceinline__ bool by_words(const Scale& s) {
    if (std::is_same_v<T, __half> && s.m + s.least < -60000.f) return false;       // no value for a weight of 0
    return fabsf(s.m) * s.hi < (sizeof(T) == 4 ? 0x1p24f : 0x1p9f);
}

// ---- a block's part of the row --------------------------------------------------

// The row as 16-byte packs from the boundary at or before its start; places
// outside of the row read as -inf.
template <typename T>
struct Row {
    static constexpr int V = 16 / sizeof(T);
    const T* row;
    int off, vocab, packs;
    int v0, v1;             // this block's
    __device__ __forceinline__ Row(const Params& p, int64_t r, int rank) {
        row = static_cast<const T*>(p.logits) + r * p.pitch;
        vocab = p.vocab;
        off = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
        packs = (off + vocab + V - 1) / V;
        v0 = (int)((int64_t)packs * rank / p.cluster);
        v1 = (int)((int64_t)packs * (rank + 1) / p.cluster);
    }
    __device__ __forceinline__ int first_index(int v) const { return v * V - off; }
    __device__ __forceinline__ uint4 words(int v) const {
        const int i = first_index(v);
        if (i >= 0 && i + V <= vocab) return __ldg(reinterpret_cast<const uint4*>(row + i));
        alignas(16) T e[V];
#pragma unroll
        for (int q = 0; q < V; ++q) e[q] = i + q >= 0 && i + q < vocab ? row[i + q] : Num<T>::from_acc(-INFINITY);
        return *reinterpret_cast<const uint4*>(e);
    }
    __device__ __forceinline__ void get(int v, float (&z)[V]) const {
        const int i = first_index(v);
        if (i >= 0 && i + V <= vocab) {
            const uint4 k = __ldg(reinterpret_cast<const uint4*>(row + i));
            const T* e = reinterpret_cast<const T*>(&k);
#pragma unroll
            for (int q = 0; q < V; ++q) z[q] = Num<T>::to_acc(e[q]);
        } else {
#pragma unroll
            for (int q = 0; q < V; ++q)
                z[q] = i + q >= 0 && i + q < vocab ? Num<T>::to_acc(row[i + q]) : -INFINITY;
        }
    }
};

// ---- the cluster ------------------------------------------------------------------

__device__ __forceinline__ unsigned remote(const void* local, int rank) {
    unsigned at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(tc::smem_u32(local)), "r"(rank));
    return at;
}
__device__ __forceinline__ u64 read64(const u64* local, int rank) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote(local, rank)) : "memory");
    return v;
}
__device__ __forceinline__ unsigned read32(const void* local, int rank) {
    unsigned v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote(local, rank)) : "memory");
    return v;
}
__device__ __forceinline__ void write64(u64* local, int rank, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(remote(local, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void write32(int* local, int rank, int v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(remote(local, rank)), "r"(v) : "memory");
}
// A block's view of its cluster.  Every call is made by all threads of all blocks.
struct Team {
    Shared& sh;
    int rank, size;
    int parity;

    // all blocks' writes to shared memory before it are seen after it
    __device__ __forceinline__ void barrier() {
        if (size == 1) {
            __syncthreads();
            return;
        }
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        __syncwarp();
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    static __device__ __forceinline__ u64 warp_add(u64 v) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        return v;
    }
    // Sums over the cluster; `before`: over the lower ranks.  The warps' sums stay in
    // sh.warp (and warp2) until the next call.
    __device__ __forceinline__ void sum(u64& a, u64& b, u64& a_before, u64& b_before) {
        const u64 wa = warp_add(a), wb = warp_add(b);
        __syncthreads();                        // the last call's sh.warp has been read
        if ((threadIdx.x & 31) == 0) {
            sh.warp[threadIdx.x >> 5] = wa;
            sh.warp2[threadIdx.x >> 5] = wb;
        }
        __syncthreads();
        a = b = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            a += sh.warp[w];
            b += sh.warp2[w];
        }
        a_before = b_before = 0;
        if (size == 1) return;
        parity ^= 1;
        if (threadIdx.x == 0) {
            sh.exchange[parity][0] = a;
            sh.exchange[parity][1] = b;
        }
        barrier();
        // a block a lane: one trip to the others' memory
        const int r = threadIdx.x & 31;
        u64 x = 0, y = 0;
        if (r < size) {
            x = read64(&sh.exchange[parity][0], r);
            y = read64(&sh.exchange[parity][1], r);
        }
        a = warp_add(x);
        b = warp_add(y);
        a_before = warp_add(r < rank ? x : 0);
        b_before = warp_add(r < rank ? y : 0);
    }
    __device__ __forceinline__ u64 sum(u64 a) {
        u64 b = 0, x, y;
        sum(a, b, x, y);
        return a;
    }
    __device__ __forceinline__ float maximum(float v) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, d));
        if ((threadIdx.x & 31) == 0) sh.warp[threadIdx.x >> 5] = __float_as_uint(v);
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v = max_nan(v, __uint_as_float((unsigned)sh.warp[w]));
        if (size == 1) return v;
        parity ^= 1;
        if (threadIdx.x == 0) sh.exchange[parity][0] = __float_as_uint(v);
        barrier();
        const int r = threadIdx.x & 31;
        if (r < size) v = __uint_as_float((unsigned)read64(&sh.exchange[parity][0], r));
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, d));
        return v;
    }
    // One thread of the cluster has told what it found (below); all get it.
    __device__ __forceinline__ Found told() {
        barrier();
        Found f;
        const Found& at = sh.found[parity];
        f.a = read64(&at.a, 0);
        f.b = read64(&at.b, 0);
        f.c = read64(&at.c, 0);
        f.i = (int)read32(&at.i, 0);
        f.j = (int)read32(&at.j, 0);
        parity ^= 1;                            // the next one goes elsewhere
        return f;
    }
    __device__ __forceinline__ void tell(Found f) {
        Found& at = sh.found[parity];
        write64(&at.a, 0, f.a);
        write64(&at.b, 0, f.b);
        write64(&at.c, 0, f.c);
        write32(&at.i, 0, f.i);
        write32(&at.j, 0, f.j);
    }
};

// inclusive sum over the lanes below and this one
__device__ __forceinline__ u64 warp_scan(u64 v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const u64 o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// Exclusive sums over the block's threads in order, and over `slot`'s warps.
__device__ __forceinline__ u64 block_scan(u64 v, u64* slot) {
    const u64 inclusive = warp_scan(v);
    // (Lane 0 stores a total that all lanes have.  With the store in lane 31, of its own sum, calls
    // ended with a misaligned address here; what made it so is not known.  This form has not.)
    const u64 total = __shfl_sync(0xffffffffu, inclusive, 31);
    const int warp = threadIdx.x >> 5;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) slot[warp] = total;
    __syncthreads();
    u64 before = inclusive - v;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const u64 other = slot[w];
        before += w < warp ? other : 0;
    }
    return before;
}

// The sum of value(z, index) over the row.
template <typename T, typename F>
__device__ __forceinline__ u64 row_sum(const Row<T>& row, Team& team, F&& value) {
    u64 s = 0;
    for (int v = row.v0 + (int)threadIdx.x; v < row.v1; v += kThreads) {
        float z[Row<T>::V];
        row.get(v, z);
#pragma unroll
        for (int q = 0; q < Row<T>::V; ++q) s += value(z[q], row.first_index(v) + q);
    }
    return team.sum(s);
}

// One warp: the element of packs [begin, end) at which the running sum of value(z,
// index) exceeds `target`; tells its index, the value there, `total` and z (-1, 0 and NaN
// where the sum never does).
template <typename T, typename F>
__device__ __forceinline__ void find_in(const Row<T>& row, Team& team, int begin, int end, u64 target, u64 total,
                                        F&& value) {
    constexpr int V = Row<T>::V;
    const int lane = threadIdx.x & 31;
    for (int base = begin; base < end; base += 32) {
        // a pack a lane
        float z[V];
        u64 w[V], s = 0;
#pragma unroll
        for (int q = 0; q < V; ++q) z[q] = -INFINITY;
        if (base + lane < end) row.get(base + lane, z);
#pragma unroll
        for (int q = 0; q < V; ++q) {
            w[q] = base + lane < end ? value(z[q], row.first_index(base + lane) + q) : 0;
            s += w[q];
        }
        const u64 sums = warp_scan(s);
        const unsigned past = __ballot_sync(0xffffffffu, sums > target);
        if (past && lane == __ffs(past) - 1) {
            u64 reach = sums - s;
            bool found = false;
#pragma unroll
            for (int q = 0; q < V; ++q) {
                reach += w[q];
                if (!found && reach > target) {
                    found = true;
                    team.tell(Found{w[q], total, 0, row.first_index(base + lane) + q, (int)__float_as_uint(z[q])});
                }
            }
        }
        if (past) return;
        target -= __shfl_sync(0xffffffffu, sums, 31);
    }
    if (lane == 0) team.tell(Found{0, total, 0, -1, 0x7FC00000});
}

// The lowest index at which the running sum of value(z, index) exceeds `target`
// (below the total): i, the value there: a, the total: b, and j, the bits of z.
// target_of(total) gives the target.
template <typename T, typename F, typename G>
__device__ __forceinline__ Found locate(const Row<T>& row, Team& team, F&& value, G&& target_of) {
    constexpr int V = Row<T>::V;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto part = [&](int begin, int end) {       // of packs, by one warp
        u64 s = 0;
        for (int v = begin + lane; v < end; v += 32) {
            float z[V];
            row.get(v, z);
#pragma unroll
            for (int q = 0; q < V; ++q) s += value(z[q], row.first_index(v) + q);
        }
        return s;
    };
    auto cut = [](int begin, int end, int k) { return begin + (int)((int64_t)(end - begin) * k / kWarps); };
    u64 own = part(cut(row.v0, row.v1, warp), cut(row.v0, row.v1, warp + 1));
    u64 sum = own, none = 0, before, none_before;
    team.sum(sum, none, before, none_before);
    const u64 total = sum;
    u64 target = target_of(total);
    u64 mine = 0;
    for (int w = 0; w < kWarps; ++w) mine += team.sh.warp[w];
    if (target >= before && target < before + mine) {        // the whole block
        target -= before;
        int at = 0;
        while (at < kWarps - 1 && target >= team.sh.warp[at]) target -= team.sh.warp[at++];
        const int b1 = cut(row.v0, row.v1, at), e1 = cut(row.v0, row.v1, at + 1);
        __syncthreads();
        own = Team::warp_add(part(cut(b1, e1, warp), cut(b1, e1, warp + 1)));
        if (lane == 0) team.sh.warp[warp] = own;
        __syncthreads();
        at = 0;
        while (at < kWarps - 1 && target >= team.sh.warp[at]) target -= team.sh.warp[at++];
        if (warp == 0) find_in(row, team, cut(b1, e1, at), cut(b1, e1, at + 1), target, total, value);
    }
    return team.told();
}

// ---- the list ----------------------------------------------------------------------

// Descending order of n entries (n <= E kThreads), by the block: a bitonic sort of E
// entries a thread, i = t + e kThreads.  Partners are in the thread, in the warp, or meet in
// `list` and `other` by turns.
template <int E>
__device__ __forceinline__ void sort_entries(u64* list, u64* other, int n) {
    const int t = threadIdx.x;
    u64 x[E];
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = t + e * kThreads < n ? list[t + e * kThreads] : 0;
    __syncthreads();
    u64* buffer = other;
    for (int k = 2; k <= E * kThreads; k *= 2)
        for (int j = k / 2; j > 0; j /= 2) {
            if (j >= kThreads) {
                if constexpr (E > 1) {
#pragma unroll
                    for (int e = 0; e < E; ++e)
#pragma unroll
                        for (int o = e + 1; o < E; ++o)
                            if ((e ^ o) * kThreads == j) {
                                const u64 a = max(x[e], x[o]), b = min(x[e], x[o]);
                                const bool down = ((t + e * kThreads) & k) == 0;
                                x[e] = down ? a : b;
                                x[o] = down ? b : a;
                            }
                }
                continue;
            }
            u64 y[E];
            if (j < 32) {
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] = __shfl_xor_sync(0xffffffffu, x[e], j);
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) buffer[t + e * kThreads] = x[e];
                __syncthreads();
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] = buffer[(t ^ j) + e * kThreads];
                buffer = buffer == list ? other : list;
            }
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const bool down = ((t + e * kThreads) & k) == 0, low = (t & j) == 0;
                x[e] = down == low ? max(x[e], y[e]) : min(x[e], y[e]);
            }
        }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) list[t + e * kThreads] = x[e];
    __syncthreads();
}
// (lists and the buffers beside them are whole numbers of kThreads long)
__device__ __noinline__ void sort_list(u64* list, u64* other, int n) {
    static_assert(kList == 4 * kThreads && kBracket == 2 * kThreads, "");
    if (n <= kThreads) sort_entries<1>(list, other, n);
    else if (n <= 2 * kThreads) sort_entries<2>(list, other, n);
    else sort_entries<4>(list, other, n);
}

// running sums of the first n
__device__ __forceinline__ void scan_weights(u64* weight, int n, u64* slot) {
    constexpr int PER = kList / kThreads;
    const int first = threadIdx.x * PER;
    u64 w[PER], s = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        w[i] = first + i < n ? weight[first + i] : 0;
        s += w[i];
    }
    u64 before = block_scan(s, slot);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        before += w[i];
        if (first + i < n) weight[first + i] = before;
    }
    __syncthreads();
}

// the first of n running sums that is at least `least` (n if none)
__device__ __forceinline__ int first_reaching(const u64* sums, int n, u64 least) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (sums[mid] >= least) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// ---- shares -------------------------------------------------------------------------

// p = mantissa 2^-shift, 0 < p < 1
__device__ __forceinline__ void parts_of(float p, u64& mantissa, int& shift) {
    const unsigned b = __float_as_uint(p);
    const int e = (int)(b >> 23);
    mantissa = e ? (b & 0x7FFFFFu) | 0x800000u : b & 0x7FFFFFu;
    shift = 150 - (e ? e : 1);
}
// floor(p s) and ceil(p s)
__device__ __forceinline__ u64 share_floor(float p, u64 s) {
    if (!(p > 0.f)) return 0;
    u64 m;
    int shift;
    parts_of(fminf(p, 0x1.fffffep-1f), m, shift);
    return shift >= 128 ? 0 : (u64)(((unsigned __int128)m * s) >> shift);
}
__device__ __forceinline__ u64 share_ceil(float p, u64 s) {
    u64 m;
    int shift;
    parts_of(p, m, shift);
    if (shift >= 100) return s ? 1 : 0;         // m s is below 2^87
    const unsigned __int128 v = (unsigned __int128)m * s, one = (unsigned __int128)1 << shift;
    return (u64)((v + one - 1) >> shift);
}

__device__ __forceinline__ void write_result(const Params& p, int64_t row, int token, float z, u64 w, u64 total,
                                             const Scale& s) {
    p.tokens[row] = token;
    if (!p.logprob) return;
    const float other = (float)(total - w) / (float)total;
    float lp;
    if (other < 0.5f) {
        lp = log1pf(-other);
    } else {
        // x - log2(total), each in two parts
        float lost;
        const float d = difference(z, s.m, lost), hi = d * s.hi, lo = fmaf(lost, s.hi, fmaf(d, s.lo, fmaf(d, s.hi, -hi)));
        const int e = 63 - __clzll((long long)total);
        const float mantissa = (float)total * __int_as_float((127 - e) << 23);
        lp = ((hi - (float)(e - kOne)) + (lo - log2f(mantissa))) * kLn2;
    }
    p.logprob[row] = lp;
}

// ---- the list, by the first block ------------------------------------------------------

// takes in the other blocks' entries, which are `most` together at most; their number
__device__ __forceinline__ int gather(Team& team, u64* list, const int* listed, int most) {
    if (team.size == 1) return min(*listed, most);
    // every block's number, a block a lane, and where its entries go
    const int lane = threadIdx.x & 31;
    const int own = lane < team.size ? min((int)read32(listed, lane), most) : 0;
    int after = own;
#pragma unroll
    for (int d = 1; d < kMaxCluster; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, after, d);
        if (lane >= d) after += o;
    }
    const int size = min(__shfl_sync(0xffffffffu, after, kMaxCluster - 1), most);
    const int first = __shfl_sync(0xffffffffu, own, 0);     // this block's own stay where they are
    for (int base = first; base < size; base += kThreads) {
        const int i = base + (int)threadIdx.x;
        int block = 0, start = 0;
#pragma unroll
        for (int k = 0; k < kMaxCluster; ++k) {
            const int end = __shfl_sync(0xffffffffu, after, k);
            if (i >= end) {
                block = k + 1;
                start = end;
            }
        }
        if (i < size) list[i] = read64(&list[i - start], block);
    }
    return size;
}

// threads that share one of `size` entries: 2^this, within a warp
__device__ __forceinline__ int log_share(int size) {
    int log = 5;
    while (log > 0 && (size << log) > kThreads) --log;
    return log;
}

// the list's order, and the weights' running sums in it
__device__ __forceinline__ void order_list(u64* list, u64* weight, int size, const Scale& s, Shared& sh) {
    const int t = threadIdx.x;
    if (size <= kSmall) {
        // each entry's place is the number of larger ones (their weights are summed on the way)
        const int log = log_share(size), each = 1 << log, i = t >> log;
        __syncthreads();
        if (t < size) weight[t] = weight_of(value_of(list[t]), s, sh.powers);
        __syncthreads();
        const u64 own = i < size ? list[i] : 0;
        u64 before = 0;
        int place = 0;
        if (i < size)
            for (int j = t & (each - 1); j < size; j += each)
                if (list[j] > own) {
                    before += weight[j];
                    ++place;
                }
        for (int d = 1; d < each; d <<= 1) {
            before += __shfl_xor_sync(0xffffffffu, before, d);
            place += __shfl_xor_sync(0xffffffffu, place, d);
        }
        if (i < size) before += weight[i];
        __syncthreads();
        if (i < size && (t & (each - 1)) == 0) {
            list[place] = own;
            weight[place] = before;
        }
        __syncthreads();
        return;
    }
    sort_list(list, weight, size);
    for (int i = t; i < size; i += kThreads) weight[i] = weight_of(value_of(list[i]), s, sh.powers);
    __syncthreads();
    scan_weights(weight, size, sh.warp);
}

// The list's first `size` entries, in order, are all that is kept: the token.
template <typename T>
__device__ __forceinline__ void choose(const Params& p, int64_t r, const Row<T>& row, float u, int size, const Scale& s,
                                       Shared& sh) {
    const int t = threadIdx.x;
    const u64 total = sh.weight[size - 1];
    const u64 target = share_floor(u, total);
    if (size <= kSmall) {
        // the entry whose weight, behind those of lower indices, reaches over the target
        const int log = log_share(size), each = 1 << log, i = t >> log;
        u64 before = 0, own = 0;
        unsigned mine = 0;
        if (i < size) {
            mine = (unsigned)sh.list[i];                // ~index
            own = sh.weight[i] - (i ? sh.weight[i - 1] : 0);
            for (int j = t & (each - 1); j < size; j += each)
                if ((unsigned)sh.list[j] > mine) before += sh.weight[j] - (j ? sh.weight[j - 1] : 0);
        }
        for (int d = 1; d < each; d <<= 1) before += __shfl_xor_sync(0xffffffffu, before, d);
        if (i < size && (t & (each - 1)) == 0 && before <= target && target < before + own)
            write_result(p, r, (int)~mine, value_of(sh.list[i]), own, total, s);
        return;
    }
    // single weights again, and the entries by index
    u64 w[kList / kThreads];
#pragma unroll
    for (int k = 0; k < kList / kThreads; ++k) {
        const int i = t + k * kThreads;
        w[k] = i < size ? sh.weight[i] - (i ? sh.weight[i - 1] : 0) : 0;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kList / kThreads; ++k) {
        const int i = t + k * kThreads;
        if (i < size) sh.list[i] = (sh.list[i] << 32) | (unsigned)i;
    }
    __syncthreads();
    u64* const by_rank = reinterpret_cast<u64*>(sh.bins);        // the counts are done with
    static_assert(sizeof(sh.bins) >= sizeof(sh.weight), "");
#pragma unroll
    for (int k = 0; k < kList / kThreads; ++k)
        if (t + k * kThreads < size) by_rank[t + k * kThreads] = w[k];
    sort_list(sh.list, sh.weight, size);
    for (int i = t; i < size; i += kThreads) sh.weight[i] = by_rank[(int)(sh.list[i] & 0xFFFFFFFFu)];
    __syncthreads();
    scan_weights(sh.weight, size, sh.warp);
    if (t == 0) {
        const int at = first_reaching(sh.weight, size, target + 1);
        const int token = (int)~(unsigned)(sh.list[at] >> 32);
        const u64 weight = sh.weight[at] - (at ? sh.weight[at - 1] : 0);
        write_result(p, r, token, Num<T>::to_acc(row.row[token]), weight, total, s);
    }
}

// how many of the first `size` entries of an ordered list are not below `cut`
__device__ __forceinline__ int kept_of(const u64* list, int size, u64 cut) {
    int lo = 0, hi = size;                                  // descending order
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (list[mid] < cut) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// ---- the histogram ---------------------------------------------------------------------

// Counts of tokens by steps.  Each block takes a share of the bins when they are counted, each
// thread `each` in a row; bin b lies where the threads' b-th bins are side by side.
struct Bins {
    Team& team;
    int log_each, each, stride, mine;
    u64 before_count, before_mass;      // this thread's bins'
    u64 count, mass;                    // the cluster's

    __device__ __forceinline__ explicit Bins(Team& t) : team(t) {
        log_each = 31 - __clz(kBins / kThreads / team.size);
        each = 1 << log_each;
        stride = kBins >> log_each;
        mine = team.rank * kThreads + threadIdx.x;
    }
    __device__ __forceinline__ void clear() {
        for (int i = threadIdx.x; i < kBins; i += kThreads) team.sh.bins[i] = 0;
        __syncthreads();
    }
    static __device__ __forceinline__ void add(Shared& sh, float step, int log_each) {
        const int b = (int)step;
        atomicAdd(&sh.bins[(b & ((1 << log_each) - 1)) * (kBins >> log_each) + (b >> log_each)], 1u);
    }
    // the weight in a step's middle, at least 1
    static __device__ __forceinline__ u64 weight(int b) {
        return ((u64)__float2uint_rz(exp2f((b + 0.5f) * (-1.f / kStepsPerOctave)) * 0x1p31f) << 12) + 1;
    }
    __device__ __forceinline__ void sum() {
        team.barrier();
        u64 c = 0, w = 0;
        for (int i = 0; i < each; ++i) {
            unsigned* const at = &team.sh.bins[i * stride + mine];
            unsigned k = *at;
            if (team.size > 1) {
                for (int other = 1; other < team.size; ++other) k += read32(at, (team.rank + other) & (team.size - 1));
                *at = k;                        // only this block reads its share of its bins
            }
            c += k;
            w += k * weight(mine * each + i);
        }
        count = c;
        mass = w;
        team.sum(count, mass, before_count, before_mass);
        before_count += block_scan(c, team.sh.warp);
        before_mass += block_scan(w, team.sh.warp2);
    }
    // f(bin, count before it, weight before it, its count) for this thread's bins in order
    template <typename F>
    __device__ __forceinline__ void in_order(F&& f) {
        u64 c = before_count, w = before_mass;
        for (int i = 0; i < each; ++i) {
            const unsigned k = team.sh.bins[i * stride + mine];
            const int b = mine * each + i;
            f(b, c, w, k);
            c += k;
            w += k * weight(b);
        }
    }
    // the bin in which the estimated weight reaches over `target`: i, the counts before it and
    // up to its end: a, b, the estimate before it: c
    __device__ __forceinline__ Found reaching(u64 target) {
        target = min(target, mass - 1);
        in_order([&](int b, u64 c, u64 w, unsigned k) {
            if (w <= target && target < w + k * weight(b)) team.tell(Found{c, c + k, w, b, 0});
        });
        return team.told();
    }
    // the bins around the one that reaches over `near`, 2^-13 of the weight on either side, or that one
    // where those hold more than `most` tokens; false where it does, too
    __device__ __forceinline__ bool bracket(u64 near, u64 most, Found& low, Found& high) {
        const u64 off = mass >> 13;
        low = reaching(near > off ? near - off : 0);
        high = reaching(near + off);
        if (high.b - low.a <= most) return true;
        low = high = reaching(near);
        return high.b - low.a <= most;
    }
    // where to look next: the exact weight above the bracket is known now
    static __device__ __forceinline__ u64 corrected(const Found& low, u64 target, u64 above) {
        const long long near = (long long)low.c + (long long)(target - above);
        return near > 0 ? (u64)near : 0;
    }
};

// ---- any row ---------------------------------------------------------------------------

struct Settings {
    float u, top_p;
    int top_k;              // 0: all
    unsigned max_key;
    u64 min_cut;            // the last entry that min_p keeps
};

// Single elements, whatever their values: rows far from zero, rows with more tokens at
// a cut than the lists hold, k beyond the threads' maxima.
template <typename T>
__device__ __noinline__ void any_row(const Params& p, int64_t r, const Row<T> row, Team team, const Scale s,
                                     const Settings o) {
    constexpr int V = Row<T>::V;
    Shared& sh = team.sh;
    const int t = threadIdx.x;
    if (t == 0) sh.listed = 0;
    u64 cut = 0;                                            // the last entry that is kept so far
    // Tokens of steps [from, to) that `cut` keeps go into the block's list; the
    // weights of all that it keeps are added to `all`, those of lower steps to `above`.
    auto collect = [&](float from, float to, bool weigh, u64& all, u64& above) {
        for (int v = row.v0 + t; v < row.v1; v += kThreads) {
            float z[V];
            row.get(v, z);
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float f = step_of(z[q], s);
                const u64 entry = entry_of(z[q], row.first_index(v) + q);
                if (!(f < (float)kBins) || entry < cut) continue;
                if (f >= from && f < to) {
                    const int at = atomicAdd(&sh.listed, 1);
                    if (at < kList) sh.list[at] = entry;
                }
                if (!weigh) continue;
                const u64 w = weight_of(z[q], s, sh.powers);
                all += w;
                if (f < from) above += w;
            }
        }
    };
    // The cut at which the sum of value(z) over kept entries reaches `least`, by
    // bisection over keys, then among equal ones by index.
    auto bisect = [&](auto&& value, u64 least) {
        unsigned lo = 0, hi = o.max_key;                    // sum(key >= lo) >= least
        while (lo < hi) {
            const unsigned mid = hi - (hi - lo) / 2;
            const u64 sum = row_sum(row, team, [&](float z, int i) -> u64 {
                return order_key(z) >= mid && entry_of(z, i) >= cut ? value(z) : 0;
            });
            if (sum >= least) lo = mid;
            else hi = mid - 1;
        }
        const u64 above = row_sum(row, team, [&](float z, int i) -> u64 {
            return order_key(z) > lo && entry_of(z, i) >= cut ? value(z) : 0;
        });
        const Found f = locate(
            row, team, [&](float z, int i) -> u64 { return order_key(z) == lo && entry_of(z, i) >= cut ? value(z) : 0; },
            [&](u64) -> u64 { return least - above - 1; });
        cut = ((u64)lo << 32) | (unsigned)~f.i;
    };
    auto weight = [&](float z) { return weight_of(z, s, sh.powers); };
    // the first block is done with the list; `entry` is the new cut.  Every block hears of it,
    // and empties its list for the next collection.
    auto cut_told = [&](u64 entry, bool good) {
        __syncthreads();                                    // the block has read what it needs
        if (team.rank == 0 && t == 0) team.tell(Found{entry, 0, 0, good, 0});
        const Found f = team.told();
        if (t == 0) sh.listed = 0;
        return f;
    };
    if (o.top_k > 0 || o.top_p < 1.f) {
        Bins bins(team);
        bins.clear();
        for (int v = row.v0 + t; v < row.v1; v += kThreads) {
            float z[V];
            row.get(v, z);
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float f = step_of(z[q], s);
                if (f < (float)kBins) Bins::add(sh, f, bins.log_each);
            }
        }
        bins.sum();
        u64 unused = 0;
        u64 known = bins.mass;                              // estimate of the k tokens' weight
        if (o.top_k && bins.count > (u64)o.top_k) {
            bins.in_order([&](int b, u64 c, u64 w, unsigned k) {
                if (c < (u64)o.top_k && c + k >= (u64)o.top_k)
                    team.tell(Found{c, c + k, w + ((u64)o.top_k - c) * Bins::weight(b), b, 0});
            });
            const Found f = team.told();
            known = f.c;
            if (f.b - f.a <= (u64)kList) {
                collect((float)f.i, (float)(f.i + 1), false, unused, unused);
                team.barrier();
                u64 last = 0;
                if (team.rank == 0) {
                    order_list(sh.list, sh.weight, gather(team, sh.list, &sh.listed, kList), s, sh);
                    last = sh.list[o.top_k - 1 - (int)f.a];
                }
                cut = cut_told(last, true).a;
            } else {
                bisect([](float) -> u64 { return 1; }, (u64)o.top_k);
            }
        }
        if (o.top_p < 1.f) {
            // the steps around the estimate, then around what the sums above them say
            u64 near = (u64)((float)known * o.top_p);
            for (int turn = 0;; ++turn) {
                Found low, high;
                if (!bins.bracket(near, kList, low, high) || turn == kTurns) {
                    const u64 all = row_sum(row, team, [&](float z, int i) -> u64 { return entry_of(z, i) >= cut ? weight(z) : 0; });
                    bisect(weight, share_ceil(o.top_p, all));
                    break;
                }
                u64 all = 0, above = 0, b1, b2, last_kept = 0;
                collect((float)low.i, (float)(high.i + 1), true, all, above);
                team.sum(all, above, b1, b2);
                const u64 target = share_ceil(o.top_p, all);
                near = Bins::corrected(low, target, above);
                bool good = false;
                if (team.rank == 0) {
                    const int size = gather(team, sh.list, &sh.listed, kList);
                    order_list(sh.list, sh.weight, size, s, sh);
                    good = size > 0 && above < target && target - above <= sh.weight[size - 1];
                    if (good) last_kept = sh.list[first_reaching(sh.weight, size, target - above)];
                }
                const Found f = cut_told(last_kept, good);
                if (!f.i) continue;
                cut = f.a;
                break;
            }
        }
    }
    // the token by sums over all that is kept
    cut = max(cut, o.min_cut);
    const Found f = locate(
        row, team, [&](float z, int i) -> u64 { return entry_of(z, i) >= cut ? weight(z) : 0; },
        [&](u64 sum) -> u64 { return share_floor(o.u, sum); });
    if (team.rank == 0 && t == 0) write_result(p, r, f.i, __int_as_float(f.j), f.a, f.b, s);
    team.barrier();                                         // nobody leaves while others read its memory
}

// ---- rows near zero, by words ------------------------------------------------------------

// What a pass over the light elements does beside summing their weights.
struct Pass {
    bool heavy_to_list;     // lists the heavy tokens
    bool histogram;         // counts the light tokens by their steps
    bool roughly;           // (with heavy_to_list) sums by the exponential unit alone, at a third of the cost
    bool masked;            // sums the steps below `low` only
    bool steps_to_list2;    // lists the light tokens of steps [low, high)
    int log_each;           // of the histogram (Bins)
    float low, high;
    uint32_t least, heavy;  // words: what elements are raised to, the least heavy value
};

// One warp's packs [begin, end): the sum of the light weights.
template <typename T, bool EXACT, bool MASKED>
__device__ __noinline__ u64 light_part(const Row<T> row, Shared& sh, int begin, int end, const Pass what) {
    constexpr int V = Row<T>::V, PER = 4 / sizeof(T);
    const Scale s = sh.scale;
    u64 sum = 0;
    float rough = 0.f;
    int v = begin + (int)(threadIdx.x & 31);
    uint4 next[2]{};                                        // on their way
    if (v < end) next[0] = row.words(v);
    if (v + 32 < end) next[1] = row.words(v + 32);
    for (; v < end; v += 32) {
        uint32_t w[4] = {next[0].x, next[0].y, next[0].z, next[0].w};
        next[0] = next[1];
        if (v + 64 < end) next[1] = row.words(v + 64);
        uint32_t heavy[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            heavy[i] = reach_mask<T>(w[i], what.heavy);
            if (MASKED || !what.heavy_to_list) w[i] = (w[i] & ~heavy[i]) | (what.least & heavy[i]);
        }
        if (!MASKED && what.heavy_to_list && (heavy[0] | heavy[1] | heavy[2] | heavy[3])) {
#pragma unroll
            for (int q = 0; q < V; ++q) {
                if (!(heavy[q / PER] >> (q % PER * 16) & 1)) continue;
                const int at = atomicAdd(&sh.listed, 1);
                if (at < kList) sh.list[at] = entry_of(of_word<T>(w[q / PER], q % PER), row.first_index(v) + q);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = (w[i] & ~heavy[i]) | (what.least & heavy[i]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = max_word<T>(w[i], what.least);
        if (!MASKED && what.roughly) {
#pragma unroll
            for (int q = 0; q < V; ++q) rough += exp2_fast((of_word<T>(w[q / PER], q % PER) - s.m) * s.hi);
            continue;
        }
        if (!MASKED && what.histogram) {
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float step = step_of(of_word<T>(w[q / PER], q % PER), s);
                if (step < (float)kBins) Bins::add(sh, step, what.log_each);
            }
        }
        if (MASKED && what.steps_to_list2) {
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float z = of_word<T>(w[q / PER], q % PER), f = step_of(z, s);
                if (f < what.low || !(f < what.high)) continue;
                const int at = atomicAdd(&sh.listed2, 1);
                if (at < kBracket) sh.list2[at] = entry_of(z, row.first_index(v) + q);
            }
        }
#pragma unroll
        for (int q = 0; q < V; q += 2)
            sum += light_weights<EXACT, MASKED>(
                pack_f2(of_word<T>(w[q / PER], q % PER), of_word<T>(w[(q + 1) / PER], (q + 1) % PER)), s, what.low);
    }
    return Team::warp_add(!MASKED && what.roughly ? (u64)__float2ull_rz(rough * 0x1p43f) : sum << s.shift);
}

// The kth largest of the threads' maxima or a little less: k elements or more are not
// below it.
__device__ __forceinline__ float bound_of(unsigned key, unsigned max_key, int k) {
    unsigned lo = 0, hi = max_key;                          // k threads or more reach lo
    while (lo < hi) {
        const unsigned mid = hi - (hi - lo) / 2;
        const int n = __syncthreads_count(key >= mid);
        if (n >= k) lo = mid;
        else hi = mid - 1;
        if (n >= k && n <= k + k / 8) break;
    }
    return key_value(lo);
}

// ---- the kernel ----------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) sample_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(128) unsigned char memory[];
    Shared& sh = *reinterpret_cast<Shared*>(memory);
    constexpr int V = Row<T>::V;
    const int64_t r = blockIdx.x / (unsigned)p.cluster;
    Team team{sh, (int)(blockIdx.x % (unsigned)p.cluster), p.cluster, 0};
    const Row<T> row(p, r, team.rank);
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const float temperature = p.temperature ? p.temperature[r] : 1.f, u = p.uniforms[r];
    const float top_p = p.top_p ? p.top_p[r] : 1.f, min_p = p.min_p ? p.min_p[r] : 0.f;
    const int given_k = p.top_k ? p.top_k[r] : 0;
    const int top_k = given_k > 0 && given_k < p.vocab ? given_k : 0;
    if (t < 64) sh.powers[t] = p.powers[t];
    if (t == 0) {
        sh.listed = sh.listed2 = 0;
        sh.scale = scale_of(temperature, min_p, sh.min_distance);
    }
    float m = -INFINITY;
    {
        uint32_t top = splat_down<T>(-INFINITY);
#pragma unroll 2
        for (int v = row.v0 + t; v < row.v1; v += kThreads) {
            const uint4 k = row.words(v);
            top = max_nan_word<T>(top, max_nan_word<T>(max_nan_word<T>(k.x, k.y), max_nan_word<T>(k.z, k.w)));
        }
        m = word_max<T>(top);
    }
    const float own_max = m;
    m = team.maximum(m);
    const bool wrong = !(m < INFINITY) || !(temperature >= 0.f && temperature < INFINITY) || u != u || top_p != top_p ||
                       min_p != min_p;
    if (wrong || m == -INFINITY) {                           // the whole cluster
        if (team.rank == 0 && t == 0) {
            p.tokens[r] = -1;
            if (p.logprob) p.logprob[r] = wrong ? __uint_as_float(0x7FC00000u) : -INFINITY;
        }
        team.barrier();                                      // nobody leaves while others read its memory
        return;
    }
    if (t == 0) {
        sh.scale.m = m;
        // differences z - m lose bits that count where m is small beside them, or in 32 bits
        sh.scale.exact = sizeof(T) == 4 || fabsf(m) * sh.scale.hi < 0x1p-5f;
        sh.min_key = min_p > 0.f ? order_key(__double2float_ru((double)m + sh.min_distance)) : 0;
    }
    __syncthreads();
    Scale s = sh.scale;
    const unsigned max_key = order_key(m);
    if (temperature == 0.f || top_k == 1 || !(top_p > 0.f) || min_p > 1.f) {
        // the first of the order
        const Found f = locate(row, team, [&](float z, int) -> u64 { return order_key(z) == max_key; }, [](u64) -> u64 { return 0; });
        if (team.rank == 0 && t == 0) {
            p.tokens[r] = f.i;
            if (p.logprob) p.logprob[r] = 0.f;
        }
        team.barrier();
        return;
    }
    const Settings o{u, top_p, top_k, max_key, (u64)sh.min_key << 32};
    if (!by_words<T>(s) || top_k > kMostK) {
        any_row(p, r, row, team, s, o);
        return;
    }
    const uint32_t least = splat_down<T>(__fadd_rd(m, s.least));
    if (top_k > 0) {
        // The list takes every token that may be among the k (or has no weight): all that
        // follows is about it.
        // A bound below which none of them lies: in every block its share of k threads reach it.
        const int share = (top_k + team.size - 1) / team.size;
        float bound = fmaxf(bound_of(order_key(own_max), max_key, share), __fadd_rd(m, s.least));
        if (team.size > 1) bound = -team.maximum(-bound);
        const uint32_t from = splat_down<T>(bound);
#pragma unroll 2
        for (int v = row.v0 + t; v < row.v1; v += kThreads) {
            const uint4 k = row.words(v);
            const uint32_t w[4] = {k.x, k.y, k.z, k.w};
            if (!reaches<T>(max_word<T>(max_word<T>(w[0], w[1]), max_word<T>(w[2], w[3])), from)) continue;
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float z = of_word<T>(w[q * (int)sizeof(T) / 4], q % (4 / (int)sizeof(T)));
                if (!(z >= bound)) continue;
                const int at = atomicAdd(&sh.listed, 1);
                if (at < kList) sh.list[at] = entry_of(z, row.first_index(v) + q);
            }
        }
        __syncthreads();
        const u64 listed = team.sum(t == 0 ? sh.listed : 0);
        if (listed > (u64)kList) {
            any_row(p, r, row, team, s, o);
            return;
        }
        if (team.rank == 0) {
            const int size = gather(team, sh.list, &sh.listed, kList);
            order_list(sh.list, sh.weight, size, s, sh);
            int keep = min(top_k, size);
            if (top_p < 1.f) keep = min(keep, first_reaching(sh.weight, keep, share_ceil(top_p, sh.weight[keep - 1])) + 1);
            choose(p, r, row, u, min(keep, kept_of(sh.list, size, o.min_cut)), s, sh);
        }
        team.barrier();                                      // nobody leaves while others read its memory
        return;
    }
    // FLOAT16's values are 2^-24 apart near zero.  Where that is four octaves or more, a word that is
    // raised to `least` may lie far below x = -64, out of the light weights' range.
    if (std::is_same_v<T, __half> && s.hi >= 0x1p26f) {
        any_row(p, r, row, team, s, o);
        return;
    }
    // A flat row: kMostHeavy tokens are heavy at most, those within 6, 3, 1.5 or 0.75 octaves
    // of the largest.  (Weights below 2^heavy are then good to 2^-23 of themselves and half a unit
    // of 2^(shift - 43), 2^-32 at most.)
    // False where more tokens are, or equal ones.
    auto fewer_heavy = [&] {
        auto packed = [](bool a, bool b, bool c) { return (u64)a + ((u64)b << 21) + ((u64)c << 42); };
        auto few = [](u64 counts, int k) { return (unsigned)(counts >> (21 * k) & 0x1FFFFF) <= kMostHeavy; };
        u64 n12_6_3 = 0, n2_1 = 0, b1, b2;
#pragma unroll 2
        for (int v = row.v0 + t; v < row.v1; v += kThreads) {
            const uint4 k = row.words(v);
            const uint32_t w[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const float x = (of_word<T>(w[q * (int)sizeof(T) / 4], q % (4 / (int)sizeof(T))) - m) * s.hi;
                n12_6_3 += packed(x >= -12.f, x >= -6.f, x >= -3.f);
                n2_1 += packed(x >= -1.5f, x >= -0.75f, false);
            }
        }
        team.sum(n12_6_3, n2_1, b1, b2);
        const float heavy = few(n12_6_3, 0) ? kHeavy : few(n12_6_3, 1) ? -6.f : few(n12_6_3, 2) ? -3.f
                          : few(n2_1, 0) ? -1.5f : few(n2_1, 1) ? -0.75f : 0.f;
        if (heavy == 0.f) return false;
        __syncthreads();
        s.heavy = heavy;
        s.shift = 12 - (int)-heavy;
        if (t == 0) {
            sh.listed = 0;
            sh.scale = s;
        }
        __syncthreads();
        return true;
    };
    // Flat rows are mostly known from the share of the threads whose maximum is heavy
    // (1 - e^-x of them where x tokens a thread are): those are counted before the list is
    // made.  Otherwise the first sum is in vain: FLOAT [106, 96364] with top-p 100 us, so 91
    // (BF16 [1024, 50257] 184 and 171; with up to 1024 heavy tokens 182, with 128 174).
    // (The counts alone decide what is heavy, so that a row's token does not depend on how many
    // blocks share the row.)
    const int most = (int)(kThreads * (1.f - __expf(-0.75f * kMostHeavy / (float)(kThreads * team.size))));
    bool flat = __syncthreads_count((own_max - m) * s.hi >= kHeavy) > most;
    if (team.size > 1) flat = team.maximum(flat) > 0.f;
    if (flat && !fewer_heavy()) {
        any_row(p, r, row, team, s, o);
        return;
    }
    // The light weights' sum, and a list of the heavy tokens.
    Pass pass{true, false, top_p < 1.f, false, false, 0, 0.f, 0.f, least, heavy_word<T>(s)};
    auto part_of = [](int begin, int end, int k) { return begin + (int)((int64_t)(end - begin) * k / kWarps); };
    auto light_sum = [&](int begin, int end) {              // of the block's warps' parts, into sh.light
        const int b = part_of(begin, end, warp), e = part_of(begin, end, warp + 1);
        constexpr bool MAY = sizeof(T) == 4;                  // FLOAT: exact always
        const u64 sum = pass.masked ? (MAY || s.exact ? light_part<T, true, true>(row, sh, b, e, pass)
                                                      : light_part<T, MAY, true>(row, sh, b, e, pass))
                                    : (MAY || s.exact ? light_part<T, true, false>(row, sh, b, e, pass)
                                                      : light_part<T, MAY, false>(row, sh, b, e, pass));
        __syncthreads();
        if (lane == 0) sh.light[warp] = sum;
        __syncthreads();
        u64 all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) all += sh.light[w];
        return t == 0 ? all : 0;
    };
    u64 light = light_sum(row.v0, row.v1), listed = t == 0 ? sh.listed : 0, b1, b2;
    team.sum(light, listed, b1, b2);
    if (listed > (u64)kMostHeavy) {
        if (!fewer_heavy()) {
            any_row(p, r, row, team, s, o);
            return;
        }
        pass.heavy = heavy_word<T>(s);
        light = team.sum(light_sum(row.v0, row.v1));
    }
    // Nothing is cut: the blocks' lists stay where they are, and need no order.
    const bool all = !(top_p < 1.f) && o.min_cut == 0;
    // What is kept may end within the list.  For that the light weights' sum need be known
    // so well only that the place of the cut is.
    enum { DONE, TOP_P, OTHER, ROUGH };
    // How far it may be off when formed roughly.  A thread adds up `terms` of float32; each is off by
    // 2^-22 by the exponential unit and by three roundings of an x down to -44, together and with the
    // weights' own error below 128 2^-24; what lies below that x is less than a unit of the weights each.
    const u64 terms = V * ((row.packs - 1) / (kThreads * team.size) + 1);
    auto rough_off = [&] { return ((light >> 24) + 1) * (terms + 128) + ((u64)p.vocab << s.shift); };
    Bins bins(team);
    Found f{};
    while (!all) {
        if (team.rank == 0) {
            int size = sh.listed;
            if (pass.heavy_to_list) {                        // the first time
                size = gather(team, sh.list, &sh.listed, kList);
                order_list(sh.list, sh.weight, size, s, sh);
                if (t == 0) sh.listed = size;
            }
            const u64 heavy = sh.weight[size - 1], off = pass.roughly ? rough_off() : 0;
            const u64 target = top_p < 1.f ? share_ceil(top_p, heavy + light - min(light, off)) : ~0ull;
            const int reach = first_reaching(sh.weight, size, target), least_p = kept_of(sh.list, size, o.min_cut);
            const int keep = min(reach + 1, least_p < size ? least_p : size + 1);
            int what = keep <= size ? DONE : (o.min_cut > 0 ? OTHER : TOP_P);
            if (pass.roughly && (what == TOP_P || (keep == reach + 1 &&
                                                   first_reaching(sh.weight, size, share_ceil(top_p, heavy + light + off)) != reach)))
                what = ROUGH;
            if (what == DONE) choose(p, r, row, u, keep, s, sh);
            __syncthreads();
            if (t == 0) team.tell(Found{heavy, target, 0, what, 0});
        }
        f = team.told();
        if (f.i != ROUGH) break;
        // as well as the weights then, with a histogram of the light tokens' steps: the cut may lie among them
        bins.clear();
        pass.heavy_to_list = pass.roughly = false;
        pass.histogram = true;
        pass.log_each = bins.log_each;
        light = team.sum(light_sum(row.v0, row.v1));
        pass.histogram = false;
    }
    if (!all && f.i == DONE) {
        team.barrier();                                      // nobody leaves while others read its memory
        return;
    }
    if (f.i == OTHER) {
        any_row(p, r, row, team, s, o);
        return;
    }
    u64 cut = 0;
    pass.heavy_to_list = false;
    if (!all) {
        // The cut lies among the light tokens: the histogram shows where, to a fraction of a percent
        // of their weight; the tokens of those steps go into a second list.
        const u64 target = f.b - f.a;                        // of the light weights
        bins.sum();
        u64 near = (u64)((float)target / (float)light * (float)bins.mass);
        for (int turn = 0;; ++turn) {
            Found low, high;
            if (!bins.bracket(near, kBracket, low, high) || turn == kTurns) {
                any_row(p, r, row, team, s, o);
                return;
            }
            pass.masked = pass.steps_to_list2 = true;
            pass.low = (float)low.i;
            pass.high = (float)(high.i + 1);
            u64 above = light_sum(row.v0, row.v1);
            above = team.sum(above);
            near = Bins::corrected(low, target, above);
            if (team.rank == 0) {
                const int size = gather(team, sh.list2, &sh.listed2, kBracket);
                order_list(sh.list2, sh.weight2, size, s, sh);
                const bool good = size > 0 && above < target && target - above <= sh.weight2[size - 1];
                const int at = good ? first_reaching(sh.weight2, size, target - above) : 0;
                __syncthreads();
                if (t == 0) {
                    sh.listed2 = size;
                    team.tell(Found{good ? sh.list2[at] : 0, 0, 0, good, 0});
                }
            }
            const Found g = team.told();
            if (g.i) {
                cut = g.a;
                break;
            }
            if (t == 0) sh.listed2 = 0;
        }
        pass.steps_to_list2 = false;
    }
    // The token by sums over the row: the light sums of its parts, and the listed tokens of each.
    auto add_listed = [&](int begin, int end) {              // sh.warp: by sixteenths of [begin, end)
        auto add = [&](const u64* list, int size, u64 least_entry) {
            for (int i = t; i < size; i += kThreads) {
                const u64 entry = list[i];
                const int v = (index_of(entry) + row.off) / V;
                if (entry < least_entry || v < begin || v >= end) continue;
                int k = (int)((int64_t)(v - begin) * kWarps / (end - begin));
                while (k > 0 && v < part_of(begin, end, k)) --k;
                while (k < kWarps - 1 && v >= part_of(begin, end, k + 1)) ++k;
                atomicAdd(&sh.warp[k], weight_of(value_of(entry), s, sh.powers));
            }
        };
        __syncthreads();
        if (t < kWarps) sh.warp[t] = sh.light[t];
        __syncthreads();
        add(sh.list, sh.listed, 0);
        add(sh.list2, sh.listed2, cut);
        __syncthreads();
        const u64 part = lane < kWarps ? sh.warp[lane] : 0;
        __syncthreads();
        return part;
    };
    u64 part = add_listed(row.v0, row.v1);
    const u64 mine = Team::warp_add(part);
    u64 total = t == 0 ? mine : 0, none = 0, before, none_before;
    team.sum(total, none, before, none_before);
    u64 target = share_floor(u, total);
    if (target >= before && target < before + mine) {         // the whole block
        target -= before;
        int begin = row.v0, end = row.v1;
        for (int level = 0;; ++level) {
            int at = 0;
            for (; at < kWarps - 1; ++at) {
                const u64 w = __shfl_sync(0xffffffffu, part, at);
                if (target < w) break;
                target -= w;
            }
            const int b = part_of(begin, end, at), e = part_of(begin, end, at + 1);
            begin = b;
            end = e;
            if (level == 1) break;
            light_sum(begin, end);
            part = add_listed(begin, end);
        }
        if (warp == 0)
            find_in(row, team, begin, end, target, total,
                    [&](float z, int i) -> u64 { return entry_of(z, i) >= cut ? weight_of(z, s, sh.powers) : 0; });
    }
    const Found at = team.told();
    if (team.rank == 0 && t == 0) write_result(p, r, at.i, __int_as_float(at.j), at.a, at.b, s);
    team.barrier();
}

// ---- host side -------------------------------------------------------------

// Blocks a row: as many as keep every block resident, with two rounds of packs each
// or more; twice as many where each still has eight rounds, so that rows with more passes
// than others hold fewer SMs up (us, resident and twice: FP16 [334, 51426] top-p 110 and 93,
// FLOAT [106, 96364] 91 and 81; with fewer rounds FLOAT [243, 9822] 48 and 55; four times as
// many: BF16 [1024, 50257] 182, twice 169).
inline int cluster_of(int64_t rows, int64_t packs, int sm_count) {
    const int64_t resident = kBlocksPerSm * (int64_t)sm_count;
    int c = 1;
    while (c < kMaxCluster) {
        const int64_t blocks = rows * c * 2, rounds = packs / ((int64_t)c * 2 * kThreads);
        if (blocks > 2 * resident || rounds < (blocks > resident ? 8 : 2)) break;
        c *= 2;
    }
    return c;
}

struct Powers {
    Power of[64];
    Powers() {
        for (int i = 0; i < 64; ++i) {
            const double v = std::exp2(i / 64.0);
            of[i].fixed = (u64)std::llrint(std::ldexp(v, kOne));
            of[i].hi = (float)v;
            of[i].lo = (float)(v - (double)of[i].hi);
        }
    }
};

template <typename T>
cudaError_t forward_as(Params p, int64_t rows, int sm_count, cudaStream_t s) {
    p.cluster = cluster_of(rows, ceil_div(p.vocab, 16 / sizeof(T)), sm_count);
    static const Powers powers;
    std::memcpy(p.powers, powers.of, sizeof powers.of);
    const cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(sample_kernel<T>), (int)sizeof(Shared));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * p.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sample_kernel<T>, p);
}

}  // namespace sample
}  // namespace olc

using namespace olc;

struct olc_sample_plan {
    PlanState state;
    olc_dtype dtype;
    int64_t rows, vocab;
};

extern "C" {

olc_status olc_sample_plan_create(int64_t rows, int64_t vocab, olc_dtype dtype, olc_sample_plan** out) {
    if (!out) return OLC_ERR_NULL;
    *out = nullptr;
    if (!plan_dtype_ok(dtype)) return OLC_ERR_DTYPE;
    if (rows < 0 || vocab < 0) return OLC_ERR_NEGATIVE_DIM;
    if (rows >= (int64_t(1) << 27) || vocab == 0 || vocab > (int64_t(1) << 20)) return OLC_ERR_INVALID;
    olc_sample_plan* p = new (std::nothrow) olc_sample_plan;
    if (!p) return OLC_ERR_OOM;
    p->state.init();
    p->dtype = dtype;
    p->rows = rows;
    p->vocab = vocab;
    *out = p;
    return OLC_OK;
}

void olc_sample_plan_destroy(olc_sample_plan* plan) {
    if (!plan) return;
    plan->state.destroy();
    delete plan;
}

olc_status olc_sample_forward(olc_sample_plan* plan, const void* logits, int64_t pitch, const float* uniforms,
                              const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                              int64_t* tokens, float* logprob, void* stream) {
    if (!plan) return OLC_ERR_NULL;
    if (plan->rows == 0) return OLC_OK;
    if (!logits || !uniforms || !tokens) return OLC_ERR_NULL;
    const int64_t eb = plan_elem_bytes(plan->dtype);
    if (plan->rows > 1 && (pitch < plan->vocab || !plan_fits(plan->rows, pitch, eb))) return OLC_ERR_INVALID;
    if (plan_misaligned(logits, eb) || plan_misaligned(uniforms, 4) || plan_misaligned(temperature, 4) ||
        plan_misaligned(top_k, 4) || plan_misaligned(top_p, 4) || plan_misaligned(min_p, 4) ||
        plan_misaligned(tokens, 8) || plan_misaligned(logprob, 4))
        return OLC_ERR_INVALID;
    const olc_status st = plan->state.bind();
    if (st != OLC_OK) return st;
    sample::Params p{};
    p.logits = logits;
    p.uniforms = uniforms;
    p.temperature = temperature;
    p.top_k = top_k;
    p.top_p = top_p;
    p.min_p = min_p;
    p.tokens = tokens;
    p.logprob = logprob;
    p.pitch = pitch;
    p.vocab = (int)plan->vocab;
    return by_type(plan->dtype, [&](auto tag) {
        return plan_status(sample::forward_as<decltype(tag)>(p, plan->rows, plan->state.sm_count,
                                                             static_cast<cudaStream_t>(stream)));
    });
}

}  // extern "C"
