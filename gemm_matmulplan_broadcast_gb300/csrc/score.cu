// Log probabilities of given tokens from logits [rows, vocab], with the
// entropy of each row's distribution and its k most likely tokens, and the
// gradient.
//
//   m = max_j z_j,  s = sum_j e^(z_j - m),  a = sum_j (z_j - m) e^(z_j - m)
//   lse = m + log s,  logprob = z_token - lse,  H = log s - a / s
//   dz_j = dlogprob (1[j = token] - p_j) - dH p_j (log p_j + H)
//
// (a <= 0 <= log s, so the entropy's two terms never cancel.)  About six
// operations and one exponential an element against one element read: the
// bytes bound it, with the exponential unit close behind for 16-bit logits.
//
// Forward.  One pass: each thread keeps a running m, s and a, rescaled when a
// later group of its elements brings a larger maximum.  A row is one block,
// or, where there are fewer rows than blocks fit, a cluster of blocks that
// each take a slice of it; the first block joins the slices' sums in slice
// order through distributed shared memory.
//
// The k largest need no second pass over the row.  k groups of threads whose
// own maximum is at least t hold at least k elements >= t; so the k-th
// largest of the groups' maxima is a bound that every one of the k largest
// elements reaches, and only the few threads whose maximum reaches it read
// their elements again.  Order is by value, then by the lower index.
#include <new>

#include "common.cuh"
#include "plan_state.h"

namespace olc {
namespace score {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kGroups = kThreads / 4;       // four neighbouring threads share a maximum
constexpr int kMaxTop = 32;
constexpr int kMaxCluster = 8;
constexpr int kBuffer = 1024;               // candidates above the bound, and as many at it
constexpr int kUnroll = 4;                  // 16-byte loads in flight a thread

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

// Distances below this one weigh nothing (e^-104 is 0 in float32), and their
// product with a zero weight has to be 0 for masks of -inf and of the type's
// lowest value alike.
constexpr float kFar = -1.0e4f;

// A running softmax over some elements of a row.
struct Sums {
    float m, s, a;
};
__device__ __forceinline__ float reference_of(float m) { return m == -INFINITY ? 0.f : m; }

// the sums of both sets of elements, in this order
__device__ __forceinline__ Sums join(const Sums& x, const Sums& y) {
    const float m = fmaxf(x.m, y.m);
    const float r = reference_of(m);
    const float dx = x.m - r, dy = y.m - r;         // 0 or negative; -inf where a side is empty
    const float cx = __expf(dx), cy = __expf(dy);
    Sums o;
    o.m = m;
    o.s = cx * x.s + cy * y.s;
    o.a = cx * (x.a + max_nan(dx, kFar) * x.s) + cy * (y.a + max_nan(dy, kFar) * y.s);
    return o;
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
    s.v0 = (int)((int64_t)packs * part / parts);
    s.v1 = (int)((int64_t)packs * (part + 1) / parts);
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

// every element of the slice that this thread owns: f(value, index)
template <typename T, typename F>
__device__ __forceinline__ void own_elements(const Slice<T>& s, F&& f) {
    constexpr int V = Slice<T>::V;
    const int t = threadIdx.x;
    if (t < s.head) f(Num<T>::to_acc(s.row[t]), t);
    const uint4* body = reinterpret_cast<const uint4*>(s.row + s.body);
    for (int v = s.v0 + t; v < s.v1; v += kThreads) {
        float z[V];
        unpack<T>(__ldg(body + v), z);
#pragma unroll
        for (int i = 0; i < V; ++i) f(z[i], s.body + v * V + i);
    }
    if (s.tail0 + t < s.tail1) f(Num<T>::to_acc(s.row[s.tail0 + t]), s.tail0 + t);
}

template <int N>
__device__ __forceinline__ void take(Sums& q, const float (&z)[N]) {
    float cm = z[0];
#pragma unroll
    for (int i = 1; i < N; ++i) cm = fmaxf(cm, z[i]);
    if (cm > q.m) {
        if (q.m == -INFINITY) {
            // nothing but -inf (0) or NaN (kept) so far
        } else {
            const float d = q.m - cm, c = __expf(d);
            q.a = c * fmaf(max_nan(d, kFar), q.s, q.a);
            q.s *= c;
        }
        q.m = cm;
    }
    const float r = reference_of(q.m);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float d = max_nan(z[i] - r, kFar);
        const float e = __expf(d);
        q.s += e;
        q.a = fmaf(d, e, q.a);
    }
}

template <typename T>
__device__ __forceinline__ Sums read_slice(const Slice<T>& s) {
    constexpr int V = Slice<T>::V;
    Sums q{-INFINITY, 0.f, 0.f};
    const int t = threadIdx.x;
    if (t < s.head) {
        const float z[1] = {Num<T>::to_acc(s.row[t])};
        take(q, z);
    }
    const uint4* body = reinterpret_cast<const uint4*>(s.row + s.body);
    int v = s.v0 + t;
    for (; v + (kUnroll - 1) * kThreads < s.v1; v += kUnroll * kThreads) {
        uint4 k[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) k[i] = __ldg(body + v + i * kThreads);
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            float z[V];
            unpack<T>(k[i], z);
            take(q, z);
        }
    }
    for (; v < s.v1; v += kThreads) {
        float z[V];
        unpack<T>(__ldg(body + v), z);
        take(q, z);
    }
    if (s.tail0 + t < s.tail1) {
        const float z[1] = {Num<T>::to_acc(s.row[s.tail0 + t])};
        take(q, z);
    }
    return q;
}

struct Shared {
    Sums warp_sums[kWarps];
    Sums sums;                               // of this block's slice
    uint32_t group_max[kGroups];
    uint32_t bound;
    int above, at;
    uint32_t above_key[kBuffer];
    int above_index[kBuffer];
    int at_index[kBuffer];
    unsigned long long warp_best[kWarps];
    int warp_count[kWarps];
    uint32_t best_key[kMaxTop];              // this slice's best, in order
    int best_index[kMaxTop];
    int best_count;
    uint32_t all_key[kMaxCluster * kMaxTop]; // the first block: every slice's
    int all_index[kMaxCluster * kMaxTop];
    int all_count;
};

__device__ __forceinline__ bool better(uint32_t ka, int ia, uint32_t kb, int ib) {
    return ka > kb || (ka == kb && ia < ib);
}

// k rounds, each the best element after the last one: right for any values,
// taken where more elements than the buffer holds exceed the bound, or where
// a NaN hides what the maxima say.
template <typename T>
__device__ void top_by_rounds(const Slice<T>& s, int k, Shared& sh) {
    unsigned long long last = ~0ull;
    int n = 0;
    for (; n < k; ++n) {
        unsigned long long best = 0;
        own_elements(s, [&](float z, int i) {
            // (key, lower index first); below ~0 whatever the key
            const unsigned long long c = ((unsigned long long)order_key(z) << 32) | (0x7FFFFFFFu - (uint32_t)i);
            if (c < last && c > best) best = c;
        });
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            const unsigned long long o = __shfl_xor_sync(0xffffffffu, best, d);
            best = o > best ? o : best;
        }
        __syncthreads();
        if ((threadIdx.x & 31) == 0) sh.warp_best[threadIdx.x >> 5] = best;
        __syncthreads();
        for (int w = 0; w < kWarps; ++w) best = sh.warp_best[w] > best ? sh.warp_best[w] : best;
        if (best == 0) break;                        // the slice holds no more elements
        if (threadIdx.x == 0) {
            sh.best_key[n] = (uint32_t)(best >> 32);
            sh.best_index[n] = (int)(0x7FFFFFFFu - (uint32_t)best);
        }
        last = best;
    }
    if (threadIdx.x == 0) sh.best_count = n;
}

// the k lowest indices of elements with this key, in order, into at_index
template <typename T>
__device__ void lowest_at(const Slice<T>& s, uint32_t key, int k, Shared& sh) {
    int found = 0;
    auto scan = [&](int begin, int end) {
        for (int base = begin; base < end && found < k; base += kThreads) {
            const int i = base + (int)threadIdx.x;
            const bool hit = i < end && order_key(Num<T>::to_acc(s.row[i])) == key;
            const unsigned b = __ballot_sync(0xffffffffu, hit);
            __syncthreads();
            if ((threadIdx.x & 31) == 0) sh.warp_count[threadIdx.x >> 5] = __popc(b);
            __syncthreads();
            int before = found, all = found;
            for (int w = 0; w < kWarps; ++w) {
                if (w < (int)(threadIdx.x >> 5)) before += sh.warp_count[w];
                all += sh.warp_count[w];
            }
            before += __popc(b & ((1u << (threadIdx.x & 31)) - 1u));
            if (hit && before < k) sh.at_index[before] = i;
            found = all;
        }
    };
    scan(0, s.head);
    scan(s.body + s.v0 * Slice<T>::V, s.body + s.v1 * Slice<T>::V);
    scan(s.tail0, s.tail1);
    __syncthreads();
    if (threadIdx.x == 0) sh.at = min(found, k);
    __syncthreads();
}

// The slice's k best elements in order, into best_*.  `mine`: this thread's
// maximum; `plain`: no NaN was met.
template <typename T>
__device__ void top_of_slice(const Slice<T>& s, float mine, bool plain, int k, Shared& sh) {
    if (!plain) {                                    // uniform over the block
        top_by_rounds(s, k, sh);
        return;
    }
    const int t = threadIdx.x;
    const uint32_t own_key = order_key(mine);
    uint32_t g = own_key;
    g = max(g, __shfl_xor_sync(0xffffffffu, g, 1));
    g = max(g, __shfl_xor_sync(0xffffffffu, g, 2));
    if ((t & 3) == 0) sh.group_max[t >> 2] = g;
    if (t == 0) sh.above = sh.at = 0;
    __syncthreads();
    if (t < kGroups) {
        const uint32_t me = sh.group_max[t];
        int rank = 0;
#pragma unroll 8
        for (int i = 0; i < kGroups; ++i) {
            const uint32_t o = sh.group_max[i];
            rank += o > me || (o == me && i < t);
        }
        if (rank == k - 1) sh.bound = me;
    }
    __syncthreads();
    const uint32_t bound = sh.bound;
    if (own_key >= bound)
        own_elements(s, [&](float z, int i) {
            const uint32_t key = order_key(z);
            if (key > bound) {
                const int at = atomicAdd(&sh.above, 1);
                if (at < kBuffer) {
                    sh.above_key[at] = key;
                    sh.above_index[at] = i;
                }
            } else if (key == bound) {
                const int at = atomicAdd(&sh.at, 1);
                if (at < kBuffer) sh.at_index[at] = i;
            }
        });
    __syncthreads();
    const int above = sh.above;
    if (above > kBuffer) {
        top_by_rounds(s, k, sh);
        return;
    }
    if (sh.at > kBuffer) lowest_at(s, bound, k, sh);
    const int at = sh.at;
    if (t == 0) sh.best_count = min(k, above + at);
    for (int c = t; c < above + at; c += kThreads) {
        const uint32_t key = c < above ? sh.above_key[c] : bound;
        const int index = c < above ? sh.above_index[c] : sh.at_index[c - above];
        int rank = 0;
        for (int i = 0; i < above; ++i) rank += better(sh.above_key[i], sh.above_index[i], key, index);
        if (c >= above)
            for (int i = 0; i < at; ++i) rank += sh.at_index[i] < index;
        if (rank < k) {
            sh.best_key[rank] = key;
            sh.best_index[rank] = index;
        }
    }
}

__device__ __forceinline__ uint32_t remote(const void* local, int rank) {
    uint32_t out;
    asm("mapa.shared::cluster.u32 %0, %1, %2;"
        : "=r"(out)
        : "r"((uint32_t)__cvta_generic_to_shared(local)), "r"(rank));
    return out;
}
__device__ __forceinline__ uint32_t remote_u32(const void* local, int rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote(local, rank)) : "memory");
    return v;
}
__device__ __forceinline__ float remote_f32(const float* local, int rank) {
    return __uint_as_float(remote_u32(local, rank));
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) forward_kernel(const Params p) {
    __shared__ Shared sh;
    const int parts = p.cluster;
    const int64_t row = blockIdx.x / parts;
    const int part = (int)(blockIdx.x % parts);      // = the block's rank in its cluster
    const int t = threadIdx.x;
    grid_dependency_wait();
    grid_launch_dependents();
    const T* z = static_cast<const T*>(p.logits) + row * p.pitch;
    const Slice<T> slice = slice_of(z, p.vocab, part, parts);
    Sums q = read_slice(slice);
    const float mine = q.m;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        Sums o;
        o.m = __shfl_xor_sync(0xffffffffu, q.m, d);
        o.s = __shfl_xor_sync(0xffffffffu, q.s, d);
        o.a = __shfl_xor_sync(0xffffffffu, q.a, d);
        q = (t & d) ? join(o, q) : join(q, o);
    }
    if ((t & 31) == 0) sh.warp_sums[t >> 5] = q;
    __syncthreads();
    if (t < 32) {
        q = t < kWarps ? sh.warp_sums[t] : Sums{-INFINITY, 0.f, 0.f};
#pragma unroll
        for (int d = 1; d < kWarps; d <<= 1) {
            Sums o;
            o.m = __shfl_xor_sync(0xffffffffu, q.m, d);
            o.s = __shfl_xor_sync(0xffffffffu, q.s, d);
            o.a = __shfl_xor_sync(0xffffffffu, q.a, d);
            q = (t & d) ? join(o, q) : join(q, o);
        }
        if (t == 0) sh.sums = q;
    }
    __syncthreads();
    if (p.top > 0) {
        top_of_slice(slice, mine, sh.sums.s == sh.sums.s, p.top, sh);
        __syncthreads();
    }
    if (parts > 1) {
        cluster_barrier();                           // every slice's results are in its block's memory
        if (part == 0) {
            if (t == 0) {
                q = sh.sums;
                for (int r = 1; r < parts; ++r)
                    q = join(q, Sums{remote_f32(&sh.sums.m, r), remote_f32(&sh.sums.s, r), remote_f32(&sh.sums.a, r)});
                sh.warp_sums[0] = q;
            }
            if (p.top > 0) {
                const int r = t / kMaxTop, i = t % kMaxTop;
                if (t == 0) sh.all_count = 0;
                __syncthreads();
                if (r < parts && i < (int)remote_u32(&sh.best_count, r)) {
                    const int at = atomicAdd(&sh.all_count, 1);
                    sh.all_key[at] = remote_u32(&sh.best_key[i], r);
                    sh.all_index[at] = (int)remote_u32(&sh.best_index[i], r);
                }
                __syncthreads();
                const int n = sh.all_count;
                if (t < n) {
                    const uint32_t key = sh.all_key[t];
                    const int index = sh.all_index[t];
                    int rank = 0;
                    for (int c = 0; c < n; ++c) rank += better(sh.all_key[c], sh.all_index[c], key, index);
                    if (rank < p.top) {
                        sh.best_key[rank] = key;
                        sh.best_index[rank] = index;
                    }
                }
            }
            __syncthreads();
        }
        cluster_barrier();                           // no block leaves while its memory is read
        if (part != 0) return;
        q = sh.warp_sums[0];
    } else {
        q = sh.sums;
    }
    const float log_s = logf(q.s);
    const bool nothing = q.m == -INFINITY && q.s == 0.f;     // every logit is -inf
    const float lse = nothing ? -INFINITY : q.m + log_s;
    if (t == 0) {
        const int64_t token = p.tokens[row];
        float lp;
        if (token < 0) lp = 0.f;                             // ignored
        else if (token >= p.vocab) lp = __uint_as_float(0x7FC00000u);
        else lp = nothing ? -INFINITY : Num<T>::to_acc(z[token]) - lse;
        p.logprob[row] = lp;
        if (p.lse) p.lse[row] = lse;
        if (p.entropy) p.entropy[row] = nothing ? 0.f : log_s - q.a / q.s;
    }
    if (t < p.top) {
        const float v = key_value(sh.best_key[t]);
        if (p.top_logprob) p.top_logprob[row * p.top + t] = nothing ? -INFINITY : v - lse;
        if (p.top_index) p.top_index[row * p.top + t] = sh.best_index[t];
    }
}

// One block takes a stretch of a row.  Every element is read and written by
// the same thread, so dlogits may be the logits.
template <typename T>
__global__ void __launch_bounds__(256) backward_kernel(const GradParams p) {
    constexpr int V = 16 / sizeof(T);
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t row = blockIdx.x / p.chunks;
    const int part = (int)(blockIdx.x % p.chunks);
    const T* z = static_cast<const T*>(p.logits) + row * p.pitch;
    T* d = static_cast<T*>(p.dlogits) + row * p.d_pitch;
    const Slice<T> s = slice_of(z, p.vocab, part, p.chunks);
    const float lse = p.lse[row];
    const int64_t token = p.dlogprob ? p.tokens[row] : -1;
    float dlp = p.dlogprob && token >= 0 ? p.dlogprob[row] : 0.f;
    if (token >= p.vocab) dlp = __uint_as_float(0x7FC00000u);
    const float dh = p.dentropy ? p.dentropy[row] : 0.f;
    const float h = p.dentropy ? p.entropy[row] : 0.f;
    const bool nothing = lse == -INFINITY;
    auto grad = [&](float v, int i) -> float {
        if (nothing) return 0.f;
        const float logp = v - lse;
        const float q = __expf(logp);
        // a probability of zero contributes nothing, whatever its logarithm
        float g = q == 0.f && dlp == dlp ? 0.f : -q * fmaf(dh, logp + h, dlp);
        if (i == token) g += dlp;
        return g;
    };
    const int t = threadIdx.x;
    if (t < s.head) d[t] = Num<T>::from_acc(grad(Num<T>::to_acc(z[t]), t));
    const uint4* body = reinterpret_cast<const uint4*>(z + s.body);
    const bool same = ((reinterpret_cast<uintptr_t>(d) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
    for (int v = s.v0 + t; v < s.v1; v += 256) {
        float k[V];
        unpack<T>(body[v], k);
        uint4 o;
        T* e = reinterpret_cast<T*>(&o);
#pragma unroll
        for (int i = 0; i < V; ++i) e[i] = Num<T>::from_acc(grad(k[i], s.body + v * V + i));
        if (same) {
            *reinterpret_cast<uint4*>(d + s.body + v * V) = o;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) d[s.body + v * V + i] = e[i];
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
// that the blocks fill them, as long as a slice keeps a few packs a thread.
inline int cluster_of(int64_t rows, int64_t vocab, int sm_count) {
    int c = 1;
    while (c < kMaxCluster && rows * c * 2 <= 2 * (int64_t)sm_count && vocab / (2 * c) >= 4096) c *= 2;
    return c;
}

template <typename T>
cudaError_t launch_forward(const Params& p, int64_t rows, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * p.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
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
    score::Params p{logits, tokens, logprob, entropy, lse, top_logprob, top_index, pitch, (int)plan->vocab,
                    top_logprob || top_index ? plan->top : 0,
                    score::cluster_of(plan->rows, plan->vocab, plan->state.sm_count)};
    return score::by_type(plan->dtype, [&](auto tag) {
        return plan_status(score::launch_forward<decltype(tag)>(p, plan->rows, static_cast<cudaStream_t>(stream)));
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
    // four packs a thread
    const int64_t stretch = 256 * 4 * (16 / eb);
    const int64_t chunks = ceil_div(plan->vocab, stretch);
    if (plan->rows * chunks > 0x7fffffffLL) return OLC_ERR_INVALID;
    score::GradParams p{logits, tokens, lse, entropy, dlogprob, dentropy, dlogits, pitch, d_pitch, plan->rows,
                        (int)plan->vocab, (int)chunks};
    return score::by_type(plan->dtype, [&](auto tag) {
        using T = decltype(tag);
        return plan_status(launch_pdl(score::backward_kernel<T>, dim3((unsigned)(plan->rows * chunks)), dim3(256), 0,
                                      static_cast<cudaStream_t>(stream), p));
    });
}

}  // extern "C"
