// Rows of a table by token id, scaled, and the table's gradient.
//
//   y_i = s E[t_i]                       (t_i < 0: zeros, a place without a token)
//   dE_v = s sum_{i: t_i = v} dy_i       (zeros, or what is there, for tokens that do not occur)
//
// One multiplication an element moved: the bytes bound both directions.
//
// Forward.  Loads of 16 bytes by as many threads as a row takes, four on their way each:
// BF16 16384 ids, 50257 x 4096 31.5 us = 0.86 of the copy rate (the rows that ids share
// are read once from memory).  One id: 1.7 us, a launch.
//
// Backward.  Sums in an order that does not change from run to run need the
// places of each token together and in order: a stable counting sort by token
// (sort_kernel, one launch: a block owns every 128th token, or fewer, and reads all
// ids).  The sums then go over chunks of equal length of the sorted places, so that a
// token that fills half of the batch costs no block more than any other
// (sum_kernel); a token whose places cross chunks leaves partial sums that
// join_kernel adds in chunk order.  The rows of tokens that do not occur are
// cleared by further blocks of sum_kernel while its chunks are summed.  BF16 16384 ids,
// 50257 x 4096: 106 us, of which the sort takes 18, the sums and the clearing 75 (546 MB:
// the copy rate), the joining 12; 0.77 of the copy rate altogether.  With few bytes the
// three launches and the sort's passes over the ids bound it: 9001 ids, 1001 x 333 FLOAT
// 30 us; with few ids the clearing: 14 ids, 32735 x 5473 BF16 75 us (floor 54).
#include <initializer_list>
#include <new>

#include "plan_state.h"
#include "row_packs.cuh"

namespace olc {
namespace embedding {

constexpr int kThreads = 256;
constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kMaxBins = 1536;          // tokens of a sort block: a counter for each and each warp, 202 KB
constexpr int kClearRows = 8;           // rows a group of threads clears
constexpr int kJoinLogTx = 5;           // threads of a join block's group
constexpr int kJoinChunks = kThreads >> kJoinLogTx;     // groups, and chunks whose ends it looks at

struct Tile {
    int log_tx;             // threads on a row: 1 << log_tx; the block's others take further rows
    int64_t packs;          // of a row
    int64_t col_tiles;
};

struct FwdParams {
    const void* table;
    const int64_t* tokens;
    void* Y;
    int64_t table_pitch, y_pitch;
    int64_t n, vocab;
    float scale;
    Tile tile;
    int64_t units;
};

// What the sort leaves: each token's places together, in order.
struct Sorted {
    int2* range;            // [vocab]: where each token's places begin and end
    int* total;             // of all tokens
    int* place;             // [n]
    int* token;             // [n]
};

struct BwdParams {
    const void* dY;
    void* dE;
    float* partial;         // [chunks][2][cols]: of the run that began before the chunk, of the one that goes on after it
    int64_t dy_pitch, e_pitch;
    int64_t vocab, cols;
    float scale;
    int accumulate;
    int length;             // places of a chunk, a multiple of 4
    int64_t chunks;
    Sorted s;
    Tile tile, clear;       // (of the rows that are cleared: 16 bytes a pack)
    int64_t sum_units, units;
};

template <typename T, int V>
__device__ __forceinline__ void fill(T* to, float v) {
    F2 o[pairs<V>()];
#pragma unroll
    for (int q = 0; q < pairs<V>(); ++q) o[q] = both(v);
    store<T, V>(to, o);
}

// PK packs a thread, all of them on their way at once
template <typename T, int V, int PK>
__global__ void __launch_bounds__(kThreads) forward_kernel(const FwdParams p) {
    const int tx = threadIdx.x & ((1 << p.tile.log_tx) - 1), ty = threadIdx.x >> p.tile.log_tx;
    const int rows = kThreads >> p.tile.log_tx;
    for (int64_t unit = blockIdx.x; unit < p.units; unit += gridDim.x) {
        const int64_t row_tile = unit / p.tile.col_tiles;
        const int64_t row = row_tile * rows + ty;
        const int64_t first = ((unit - row_tile * p.tile.col_tiles) * PK << p.tile.log_tx) + tx;
        if (row >= p.n) continue;
        const int64_t token = p.tokens[row];
        T* y = static_cast<T*>(p.Y) + row * p.y_pitch;
        if (token < 0 || token >= p.vocab) {
#pragma unroll
            for (int i = 0; i < PK; ++i) {
                const int64_t c = first + ((int64_t)i << p.tile.log_tx);
                if (c < p.tile.packs) fill<T, V>(y + c * V, token < 0 ? 0.f : __uint_as_float(0x7FC00000u));
            }
            continue;
        }
        const T* e = static_cast<const T*>(p.table) + token * p.table_pitch;
        Pack<T, V> k[PK];
#pragma unroll
        for (int i = 0; i < PK; ++i) {
            const int64_t c = first + ((int64_t)i << p.tile.log_tx);
            if (c < p.tile.packs) k[i] = load<T, V>(e + c * V);
        }
#pragma unroll
        for (int i = 0; i < PK; ++i) {
            const int64_t c = first + ((int64_t)i << p.tile.log_tx);
            if (c >= p.tile.packs) continue;
            F2 v[pairs<V>()];
            widen<T, V>(v, k[i]);
#pragma unroll
            for (int q = 0; q < pairs<V>(); ++q) v[q] = mul2(v[q], both(p.scale));
            store<T, V>(y + c * V, v);
        }
    }
}

// A block sorts the places of every 2^log_blocks-th token from blockIdx.x on (frequent
// tokens often have low ids: they are shared out): each warp
// counts its own stretch of the ids by token, a scan over warps and tokens turns
// the counts into positions, and the warps go over their stretches again.  Within
// 32 ids the lanes with the same token take consecutive positions.
__global__ void __launch_bounds__(kSortThreads)
sort_kernel(const int64_t* __restrict__ tokens, int n, int64_t vocab, int log_blocks, int bins, Sorted s) {
    extern __shared__ int counts[];                 // [kSortWarps][bins]
    __shared__ int scan[kSortWarps + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int residue = (int)blockIdx.x, mask = (1 << log_blocks) - 1;
    const int own = (int)((vocab - residue + mask) >> log_blocks);      // tokens; at least 1, at most bins
    for (int i = threadIdx.x; i < kSortWarps * bins; i += kSortThreads) counts[i] = 0;
    __syncthreads();
    const int stretch = (int)(ceil_div(ceil_div(n, kSortWarps), 32) * 32);      // at most n + 31
    const int64_t begin = min64((int64_t)warp * stretch, n), end = min64(begin + stretch, n);
    int* const mine = counts + warp * bins;
    // 512 ids at a time, all on their way at once: the block's tokens among them, as its
    // first, second, ... one, or -1
    constexpr int EACH = 16;
    int own_ids[EACH], below = 0;
    auto read = [&](int64_t base, bool count) {
        int64_t id[EACH];
#pragma unroll
        for (int u = 0; u < EACH; ++u) {
            const int64_t i = base + u * 32 + lane;
            id[u] = i < end ? tokens[i] : -1;
        }
#pragma unroll
        for (int u = 0; u < EACH; ++u) {
            const bool known = id[u] >= 0 && id[u] < vocab;
            const int r = (int)id[u] & mask;
            own_ids[u] = known && r == residue ? (int)(id[u] >> log_blocks) : -1;
            if (count) below += known && r < residue;
        }
    };
    for (int64_t base = begin; base < end; base += 32 * EACH) {
        read(base, true);
#pragma unroll
        for (int u = 0; u < EACH; ++u)
            if (own_ids[u] >= 0) atomicAdd(&mine[own_ids[u]], 1);
    }
    below = __reduce_add_sync(0xffffffffu, below);
    if (lane == 0) scan[warp] = below;
    __syncthreads();
    int position = 0;                               // where the block's first place goes
    for (int w = 0; w < kSortWarps; ++w) position += scan[w];
    __syncthreads();
    // a thread's consecutive tokens (one, where they suffice): their totals over the
    // warps, the sum of those over the tokens before, then every warp's first position
    const int per = (own + kSortThreads - 1) / kSortThreads;
    auto over_warps = [&](int b, int first, bool write) {
        int c[kSortWarps];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) c[w] = counts[w * bins + b];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            if (write) counts[w * bins + b] = first;
            first += c[w];
        }
        return first;
    };
    int sum = 0;
    for (int j = 0; j < per; ++j)
        if (threadIdx.x * per + j < own) sum = over_warps(threadIdx.x * per + j, sum, false);
    int before = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, before, d);
        if (lane >= d) before += o;
    }
    const int warps_sum = __shfl_sync(0xffffffffu, before, 31);
    if (lane == 0) scan[warp] = warps_sum;
    __syncthreads();
    position += before - sum;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
        const int c = scan[w];
        position += w < warp ? c : 0;
    }
    for (int j = 0; j < per; ++j) {
        const int b = threadIdx.x * per + j;
        if (b >= own) continue;
        const int begin = position;
        position = over_warps(b, position, true);
        s.range[((int64_t)b << log_blocks) + residue] = make_int2(begin, position);
        if (residue == (int)gridDim.x - 1 && b == own - 1) *s.total = position;
    }
    __syncthreads();
    for (int64_t base = begin; base < end; base += 32 * EACH) {
        if (end - begin > 32 * EACH) read(base, false);     // (else they are still there)
#pragma unroll
        for (int u = 0; u < EACH; ++u) {
            const int b = own_ids[u];
            if (!__any_sync(0xffffffffu, b >= 0)) continue;
            const unsigned same = __match_any_sync(0xffffffffu, b);
            int at = 0;
            if (b >= 0) at = mine[b] + __popc(same & ((1u << lane) - 1u));
            __syncwarp();
            if (b >= 0) {
                s.place[at] = (int)(base + u * 32 + lane);
                s.token[at] = (b << log_blocks) + residue;
                if ((same >> lane) == 1u) mine[b] = at + 1;         // the last of them
            }
            __syncwarp();
        }
    }
}

template <typename T, int V>
__device__ __forceinline__ void add_pack(F2 (&acc)[pairs<V>()], const Pack<T, V>& k) {
    F2 v[pairs<V>()];
    widen<T, V>(v, k);
#pragma unroll
    for (int q = 0; q < pairs<V>(); ++q) acc[q] = add2(acc[q], v[q]);
}

// float32 partial sums of V columns
template <int V>
__device__ __forceinline__ void put_partial(float* to, const F2 (&acc)[pairs<V>()]) {
    if constexpr (V == 1) {
        float lo, hi;
        unpack_f2(acc[0], lo, hi);
        *to = lo;
    } else {
        if constexpr (V == 2) *reinterpret_cast<F2*>(to) = acc[0];
        else
#pragma unroll
            for (int q = 0; q < V / 2; q += 2) *reinterpret_cast<ulonglong2*>(to + 2 * q) = make_ulonglong2(acc[q], acc[q + 1]);
    }
}
template <int V>
__device__ __forceinline__ void add_partial(F2 (&acc)[pairs<V>()], const float* from) {
    if constexpr (V == 1) {
        acc[0] = add2(acc[0], pack_f2(*from, 0.f));
    } else {
        if constexpr (V == 2) acc[0] = add2(acc[0], *reinterpret_cast<const F2*>(from));
        else
#pragma unroll
        for (int q = 0; q < V / 2; q += 2) {
            const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(from + 2 * q);
            acc[q] = add2(acc[q], v.x);
            acc[q + 1] = add2(acc[q + 1], v.y);
        }
    }
}

// a token's finished sum
template <typename T, int V>
__device__ __forceinline__ void finish(const BwdParams& p, int64_t token, int64_t c, F2 (&acc)[pairs<V>()]) {
    T* to = static_cast<T*>(p.dE) + token * p.e_pitch + c;
    if (p.accumulate) {
        F2 old[pairs<V>()];
        widen<T, V>(old, load<T, V>(to));
#pragma unroll
        for (int q = 0; q < pairs<V>(); ++q) acc[q] = fma2(acc[q], both(p.scale), old[q]);
    } else {
#pragma unroll
        for (int q = 0; q < pairs<V>(); ++q) acc[q] = mul2(acc[q], both(p.scale));
    }
    store<T, V>(to, acc);
}

// Zeros for the 16 bytes of a row that lie in the pack-th 16 bytes from the boundary at
// or before its start: one store where all of them are the row's, whatever the row's alignment (by
// single elements 32735 x 5473 BF16 take 219 us, so 75).
template <typename T, int V>
__device__ __forceinline__ void clear_pack(T* row, int64_t pack, int64_t cols) {
    constexpr int E = 16 / sizeof(T);
    if constexpr (V == E) {
        fill<T, V>(row + pack * V, 0.f);
    } else {
        const int64_t first = pack * E - (int64_t)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
        if (first >= 0 && first + E <= cols) {
            fill<T, E>(row + first, 0.f);
        } else {
            for (int64_t c = first < 0 ? 0 : first; c < first + E && c < cols; ++c) fill<T, 1>(row + c, 0.f);
        }
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) sum_kernel(const BwdParams p) {
    const T* dY = static_cast<const T*>(p.dY);
    const int tx = threadIdx.x & ((1 << p.tile.log_tx) - 1), ty = threadIdx.x >> p.tile.log_tx;
    const int groups = kThreads >> p.tile.log_tx;
    for (int64_t unit = blockIdx.x; unit < p.units; unit += gridDim.x) {
        if (unit >= p.sum_units) {
            const int64_t u = unit - p.sum_units;
            const int64_t group = u / p.clear.col_tiles * (kThreads >> p.clear.log_tx) + (threadIdx.x >> p.clear.log_tx);
            const int64_t pack = ((u % p.clear.col_tiles) << p.clear.log_tx) + (threadIdx.x & ((1 << p.clear.log_tx) - 1));
            const int64_t v0 = group * kClearRows;
            if (pack >= p.clear.packs || v0 >= p.vocab) continue;
            int2 range[kClearRows];
#pragma unroll
            for (int i = 0; i < kClearRows; ++i) range[i] = p.s.range[min64(v0 + i, p.vocab - 1)];
            unsigned untouched = 0;
#pragma unroll
            for (int i = 0; i < kClearRows; ++i) untouched |= (unsigned)(v0 + i < p.vocab && range[i].x == range[i].y) << i;
            T* const row = static_cast<T*>(p.dE) + v0 * p.e_pitch;
#pragma unroll 1
            for (; untouched; untouched &= untouched - 1) clear_pack<T, V>(row + (__ffs(untouched) - 1) * p.e_pitch, pack, p.cols);
            continue;
        }
        const int64_t group = unit / p.tile.col_tiles * groups + ty;
        const int64_t pack = ((unit % p.tile.col_tiles) << p.tile.log_tx) + tx;
        if (pack >= p.tile.packs) continue;
        const int64_t c = pack * V;
        const int64_t n = *p.s.total, p0 = group * p.length, p1 = min64(p0 + p.length, n);
        if (p0 >= n) continue;
        F2 acc[pairs<V>()];
        auto clear = [&] {
#pragma unroll
            for (int q = 0; q < pairs<V>(); ++q) acc[q] = both(0.f);
        };
        clear();
        int current = p.s.token[p0];
        auto leave = [&] {
            const int2 range = p.s.range[current];
            if (range.x >= p0 && range.y <= p1) finish<T, V>(p, current, c, acc);
            else put_partial<V>(p.partial + (group * 2 + (range.x >= p0)) * p.cols + c, acc);
        };
        for (int64_t at = p0; at < p1; at += 4) {
            // (the arrays' lengths are multiples of 4; what lies past the last place is not used)
            const int4 token = *reinterpret_cast<const int4*>(p.s.token + at);
            const int4 place = *reinterpret_cast<const int4*>(p.s.place + at);
            const int tokens[4] = {token.x, token.y, token.z, token.w}, places[4] = {place.x, place.y, place.z, place.w};
            Pack<T, V> k[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (at + j < p1) k[j] = load<T, V>(dY + (int64_t)places[j] * p.dy_pitch + c);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (at + j >= p1) break;
                if (tokens[j] != current) {
                    leave();
                    clear();
                    current = tokens[j];
                }
                add_pack<T, V>(acc, k[j]);
            }
        }
        leave();
    }
}

// Tokens whose places cross a chunk's end: the partial sums of the chunk in which
// they begin and of those after it, in order.  A block looks at the ends of kJoinChunks
// chunks, one for each of its groups of threads; a group alone adds up to kAlone
// partial sums, of more of them every group takes every kJoinChunks-th, and those are added
// in group order.  (A third of 16384 places one token, BF16 4096 columns: 108 us with the
// gradient, 161 where one group adds all; between 2 and 64 the limit does not tell.)
constexpr int kAlone = 16;
template <typename T, int V>
__global__ void __launch_bounds__(kThreads) join_kernel(const BwdParams p) {
    constexpr int LOG_TX = kJoinLogTx, GROUPS = kThreads >> LOG_TX;
    static_assert(GROUPS == kJoinChunks, "");
    __shared__ int shared_by_all[kJoinChunks];
    __shared__ alignas(16) float sums[GROUPS - 1][1 << LOG_TX][V];
    const int tx = threadIdx.x & ((1 << LOG_TX) - 1), group = threadIdx.x >> LOG_TX;
    const int64_t tiles = ceil_div(p.tile.packs, 1 << LOG_TX);
    for (int64_t unit = blockIdx.x; unit < p.units; unit += gridDim.x) {
        const int64_t c0 = unit / tiles * kJoinChunks;
        const int64_t pack = (unit % tiles << LOG_TX) + tx, c = pack * V;
        const bool in = pack < p.tile.packs;
        F2 acc[pairs<V>()];
        auto clear = [&] {
#pragma unroll
            for (int q = 0; q < pairs<V>(); ++q) acc[q] = both(0.f);
        };
        const int64_t chunk = c0 + group, next = (chunk + 1) * p.length;
        int token = -1;
        int64_t last = 0;
        if (next < *p.s.total) {
            const int t = p.s.token[next - 1];
            const int2 range = p.s.range[t];
            if (range.x >= next - p.length && range.y > next) {
                token = t;
                last = (range.y - 1) / p.length;
            }
        }
        const bool alone = last - chunk < kAlone;
        if (tx == 0) shared_by_all[group] = alone ? -1 : token;
        if (token >= 0 && alone && in) {
            clear();
            add_partial<V>(acc, p.partial + (chunk * 2 + 1) * p.cols + c);
#pragma unroll 4
            for (int64_t k = chunk + 1; k <= last; ++k) add_partial<V>(acc, p.partial + k * 2 * p.cols + c);
            finish<T, V>(p, token, c, acc);
        }
        __syncthreads();
        for (int i = 0; i < kJoinChunks; ++i) {
            const int t = shared_by_all[i];
            if (t < 0) continue;                            // the whole block
            const int64_t from = c0 + i, to = (p.s.range[t].y - 1) / p.length;
            clear();
            if (in) {
                if (group == 0) add_partial<V>(acc, p.partial + (from * 2 + 1) * p.cols + c);
#pragma unroll 4
                for (int64_t k = from + 1 + group; k <= to; k += GROUPS) add_partial<V>(acc, p.partial + k * 2 * p.cols + c);
                if (group > 0) put_partial<V>(&sums[group - 1][tx][0], acc);
            }
            __syncthreads();
            if (in && group == 0) {
                for (int g = 1; g < GROUPS; ++g) add_partial<V>(acc, &sums[g - 1][tx][0]);
                finish<T, V>(p, t, c, acc);
            }
            __syncthreads();
        }
        __syncthreads();
    }
}

// ---- host side -------------------------------------------------------------

constexpr int64_t kMaxGrid = 0x7fffffff;

// 2^log threads on a row of `packs`, `each` packs a thread, at most a block
inline Tile tile_of(int64_t packs, int each) {
    int log = 0;
    while ((1 << log) < kThreads && ((int64_t)each << log) < packs) ++log;
    return Tile{log, packs, ceil_div(packs, (int64_t)each << log)};
}

inline dim3 grid_of(int64_t units) { return dim3((unsigned)min64(units, kMaxGrid)); }

// Four packs a thread where one each would be two blocks an SM or more; else one (BF16,
// one pack and four: [2400, 4096] 8.2 and 4.9 us, [300, 4096] 2.4 and 2.2, [1000, 64] 1.9
// and 2.3).  Eight of the small packs of 16-bit rows off 16-byte boundaries (BF16, four and
// eight: [16384, 1001] 24.7 and 21.9, [16384, 2050] 46.9 and 38.1; not of FLOAT elements:
// [16384, 4097] 130 and 168).
template <typename T, int V>
cudaError_t forward_as(FwdParams p, int64_t cols, int sm_count, cudaStream_t s) {
    const int64_t packs = cols / V;
    auto run = [&](auto kernel, int each) {
        p.tile = tile_of(packs, each);
        p.units = ceil_div(p.n, kThreads >> p.tile.log_tx) * p.tile.col_tiles;
        return plan_launch(kernel, grid_of(p.units), dim3(kThreads), 0, s, p);
    };
    constexpr int EACH = sizeof(T) == 2 && V <= 2 ? 8 : 4;
    return p.n * packs >= (int64_t)sm_count * 2 * kThreads ? run(forward_kernel<T, V, EACH>, EACH)
                                                           : run(forward_kernel<T, V, 1>, 1);
}

// Places of a chunk.  A thread adds a chunk's rows one after the other: with few places
// short chunks end sooner.  A token that occurs often leaves a partial sum for each
// chunk: with many places long chunks leave less to join.  BF16, us, at 8, 16, 32 and 64
// places: [2048, 1024] into 50257 rows, a third of them one token, 32.5, 34.5, 41.6, 58.6;
// [9001, 333] 24, 22.0, 21.7, 24.6; [16384, 4096] 130, 119, 108, 105; [16384, 512] 45, 37,
// 37, 47; [78462, 64] 141, 100, 76, 75.
inline int chunk_length(int64_t n) { return n <= 4096 ? 8 : (n <= 12288 ? 16 : 32); }

// Sort blocks: a power of two, 128 (nearly one an SM), more where their counters hold no more
// tokens, no more than there are tokens.
inline int sort_log_blocks(int64_t vocab) {
    int log = 7;
    while (ceil_div(vocab, int64_t(1) << log) > kMaxBins) ++log;
    while (log > 0 && (int64_t(1) << log) > vocab) --log;
    return log;
}

struct Layout {
    size_t total, place, token, partial, bytes;
};
inline Layout layout_of(int64_t n, int64_t vocab, int64_t cols, int64_t chunks) {
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    Layout l;
    l.total = up((size_t)vocab * 8);
    l.place = l.total + 256;
    l.token = l.place + up((size_t)n * 4);
    l.partial = l.token + up((size_t)n * 4);
    l.bytes = l.partial + (size_t)chunks * 2 * (size_t)cols * 4;
    return l;
}

// Elements of eb bytes in a pack: 16 bytes of them, a pair of 16-bit ones, or one, on a boundary of
// whose size every row starts and ends.
inline int pack_elements(int64_t eb, int64_t cols, std::initializer_list<const void*> pointers,
                         std::initializer_list<int64_t> pitches) {
    uint64_t all = (uint64_t)(cols * eb);
    for (const void* p : pointers) all |= (uint64_t)reinterpret_cast<uintptr_t>(p);
    for (int64_t p : pitches) all |= (uint64_t)(p * eb);
    return all % 16 == 0 ? (int)(16 / eb) : (eb == 2 && all % 4 == 0 ? 2 : 1);
}

template <typename T, int V>
cudaError_t backward_as(BwdParams p, const int64_t* tokens, int64_t n, cudaStream_t s) {
    const int log_blocks = sort_log_blocks(p.vocab), bins = (int)ceil_div(p.vocab, int64_t(1) << log_blocks);
    const size_t smem = (size_t)kSortWarps * bins * 4;
    cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(sort_kernel), kSortWarps * kMaxBins * 4);
    if (e == cudaSuccess)
        e = plan_launch(sort_kernel, dim3(1u << log_blocks), dim3(kSortThreads), smem, s, tokens, (int)n, p.vocab,
                        log_blocks, bins, p.s);
    if (e != cudaSuccess) return e;
    p.tile = tile_of(p.cols / V, 1);
    const int groups = kThreads >> p.tile.log_tx;
    p.sum_units = ceil_div(p.chunks, groups) * p.tile.col_tiles;
    const int64_t bytes = p.cols * (int64_t)sizeof(T);
    p.clear = V * sizeof(T) == 16 ? p.tile : tile_of((bytes + 30) / 16, 1);
    p.units = p.sum_units + (p.accumulate ? 0 : ceil_div(p.vocab, (kThreads >> p.clear.log_tx) * kClearRows) * p.clear.col_tiles);
    e = plan_launch(sum_kernel<T, V>, grid_of(p.units), dim3(kThreads), 0, s, p);
    if (e != cudaSuccess || p.chunks <= 1) return e;
    p.units = ceil_div(p.chunks - 1, kJoinChunks) * ceil_div(p.tile.packs, 1 << kJoinLogTx);
    return plan_launch(join_kernel<T, V>, grid_of(p.units), dim3(kThreads), 0, s, p);
}

}  // namespace embedding
}  // namespace olc

using namespace olc;

struct olc_embedding_plan {
    PlanState state;
    olc_dtype dtype;
    int64_t n, vocab, cols;
    float scale;
};

extern "C" {

olc_status olc_embedding_plan_create(int64_t tokens, int64_t vocab, int64_t cols, double scale, olc_dtype dtype,
                                     olc_embedding_plan** out) {
    if (!out) return OLC_ERR_NULL;
    *out = nullptr;
    if (!plan_dtype_ok(dtype)) return OLC_ERR_DTYPE;
    if (tokens < 0 || vocab < 0 || cols < 0) return OLC_ERR_NEGATIVE_DIM;
    // places and tokens are 32-bit in the kernels
    constexpr int64_t most = (int64_t(1) << 31) - 65536;
    if (tokens >= most || vocab >= most || cols >= most || !(scale >= -3e38 && scale <= 3e38)) return OLC_ERR_INVALID;
    if (!plan_fits(tokens, cols, 4) || !plan_fits(vocab, cols, 4)) return OLC_ERR_INVALID;
    olc_embedding_plan* p = new (std::nothrow) olc_embedding_plan;
    if (!p) return OLC_ERR_OOM;
    p->state.init();
    p->dtype = dtype;
    p->n = tokens;
    p->vocab = vocab;
    p->cols = cols;
    p->scale = (float)scale;
    *out = p;
    return OLC_OK;
}

void olc_embedding_plan_destroy(olc_embedding_plan* plan) {
    if (!plan) return;
    plan->state.destroy();
    delete plan;
}

olc_status olc_embedding_forward(olc_embedding_plan* plan, const void* table, int64_t table_pitch,
                                 const int64_t* tokens, void* Y, int64_t y_pitch, void* stream) {
    if (!plan) return OLC_ERR_NULL;
    const int64_t eb = plan_elem_bytes(plan->dtype), n = plan->n, cols = plan->cols;
    if (n == 0 || cols == 0) return OLC_OK;
    if ((!table && plan->vocab > 0) || !tokens || !Y) return OLC_ERR_NULL;
    if ((plan->vocab > 1 && (table_pitch < cols || !plan_fits(plan->vocab, table_pitch, eb))) ||
        (n > 1 && (y_pitch < cols || !plan_fits(n, y_pitch, eb))))
        return OLC_ERR_INVALID;
    if (plan_misaligned(table, eb) || plan_misaligned(tokens, 8) || plan_misaligned(Y, eb)) return OLC_ERR_INVALID;
    const olc_status st = plan->state.bind();
    if (st != OLC_OK) return st;
    const embedding::FwdParams p{table, tokens, Y, table_pitch, y_pitch, n, plan->vocab, plan->scale, {}, 0};
    const int elements = embedding::pack_elements(eb, cols, {table, Y},
                                                  {plan->vocab <= 1 ? 0 : table_pitch, n == 1 ? 0 : y_pitch});
    return by_type(plan->dtype, [&](auto tag) {
        using T = decltype(tag);
        const cudaStream_t s = static_cast<cudaStream_t>(stream);
        const int sms = plan->state.sm_count;
        if (elements == 16 / (int)sizeof(T)) return plan_status(embedding::forward_as<T, 16 / sizeof(T)>(p, cols, sms, s));
        if constexpr (sizeof(T) == 2)
            if (elements == 2) return plan_status(embedding::forward_as<T, 2>(p, cols, sms, s));
        return plan_status(embedding::forward_as<T, 1>(p, cols, sms, s));
    });
}

olc_status olc_embedding_backward(olc_embedding_plan* plan, const void* dY, int64_t dy_pitch, const int64_t* tokens,
                                  void* dtable, int64_t dtable_pitch, int accumulate, void* stream) {
    if (!plan) return OLC_ERR_NULL;
    const int64_t eb = plan_elem_bytes(plan->dtype), n = plan->n, vocab = plan->vocab, cols = plan->cols;
    if (vocab == 0 || cols == 0 || (accumulate && n == 0)) return OLC_OK;
    if (!dtable || (n > 0 && (!dY || !tokens))) return OLC_ERR_NULL;
    if ((n > 1 && (dy_pitch < cols || !plan_fits(n, dy_pitch, eb))) ||
        (vocab > 1 && (dtable_pitch < cols || !plan_fits(vocab, dtable_pitch, eb))))
        return OLC_ERR_INVALID;
    if (plan_misaligned(dY, eb) || plan_misaligned(tokens, 8) || plan_misaligned(dtable, eb)) return OLC_ERR_INVALID;
    olc_status st = plan->state.bind();
    if (st != OLC_OK) return st;
    const int elements = embedding::pack_elements(eb, cols, {dY, dtable},
                                                  {n <= 1 ? 0 : dy_pitch, vocab == 1 ? 0 : dtable_pitch});
    const int length = embedding::chunk_length(n);
    const int64_t chunks = ceil_div(n, length);
    const embedding::Layout l = embedding::layout_of(n, vocab, cols, chunks);
    st = plan->state.ensure(l.bytes);
    if (st != OLC_OK) return st;
    char* const m = static_cast<char*>(plan->state.memory);
    const embedding::BwdParams p{dY, dtable, reinterpret_cast<float*>(m + l.partial), dy_pitch, dtable_pitch, vocab, cols,
                                 plan->scale, accumulate != 0, length, chunks,
                                 {reinterpret_cast<int2*>(m), reinterpret_cast<int*>(m + l.total),
                                  reinterpret_cast<int*>(m + l.place), reinterpret_cast<int*>(m + l.token)},
                                 {}, {}, 0, 0};
    return by_type(plan->dtype, [&](auto tag) {
        using T = decltype(tag);
        const cudaStream_t s = static_cast<cudaStream_t>(stream);
        return plan_status(plan->state.use(s, [&] {
            if (elements == 16 / (int)sizeof(T)) return embedding::backward_as<T, 16 / sizeof(T)>(p, tokens, n, s);
            if constexpr (sizeof(T) == 2)
                if (elements == 2) return embedding::backward_as<T, 2>(p, tokens, n, s);
            return embedding::backward_as<T, 1>(p, tokens, n, s);
        }));
    });
}

}  // extern "C"
