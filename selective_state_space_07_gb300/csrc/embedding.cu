// Scaled embedding lookup and its gradient on sm_103a (include/embedding.h
// holds the formulas and the boundary).
//
// Both are bound by HBM: the lookup reads a row and writes one for each token;
// the gradient writes all of dW, most rows as zeros, and reads dy once.
//
// The gradient sorts first. One kernel does it, without one CTA waiting for
// another: each CTA owns a range of ids, and its 32 warps read all ids (from
// L2), a 32nd of the tokens each: once to count the range's ids, and how many
// tokens have smaller ones, which is where the CTA's part of the sorted list
// begins; and once more to put each token of the range in its place, in token
// order. (Reading all ids in every CTA costs more than it saves where they are
// many: then two kernels before it give each range its own tokens.) A second
// kernel adds: a group of lanes takes a row of dW (256 columns of it) and its
// run of tokens, at most 32 of them.
// Longer runs (frequent ids) are cut where the sorted list's pieces of 32 end;
// a piece holds at most the end of one such run and the start of another, and
// leaves their partial sums for a third kernel, which adds them in order.
//
// Measured, in percent of the HBM copy rate: the lookup of 16384 ids of
// 50001 x 2048 bf16 21 us (79%; 16 when its rows are in L2 from the call
// before), fp32 43 (77%); the gradient of the first 103 us (67%): 11 the sort, 82 the rows (86% of the copy rate by themselves, most of
// them zeros written), the rest the joined sums. 64 ids of the same table:
// 64 us (94%). Many tokens for narrow rows are bound by the sort: 65536 ids of
// 50001 x 64 bf16 31 us (10%).
#include <cmath>

#include "../../include/embedding.h"
#include "rows.cuh"
#include "ssm_common.cuh"
#include "ssm_internal.h"

namespace ssm {
namespace {

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kMostIds = 1024;   // ids of a CTA's range
constexpr int kPiece = 32;       // tokens of a piece of the sorted list
constexpr int kRowThreads = 256;

// More tokens than kDirect are divided among the ranges first, by CTAs of
// kChunk tokens or a multiple, at most kMostChunks; ranges then are at most
// kMostRanges. The whole gradient of 50001 x 64, tokens sorted straight and
// divided first: 16384 21.0 and 22.8 us, 24576 25.3 and 26.1, 32768 29.1 and
// 27.4, 65536 43.6 and 32.3, 262144 120 and 55.
constexpr int64_t kDirect = 28 * 1024;
constexpr int kChunk = 1024, kMostChunks = 128, kMostRanges = 512;

struct EmbedWs {
    size_t off, order, sid, part, pairs, counts, starts, total;
};
EmbedWs embed_ws(int64_t tokens, int64_t V, int64_t D) {
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    EmbedWs w;
    w.off = 0;
    w.order = w.off + up((size_t)(V + 1) * 4);
    w.sid = w.order + up((size_t)tokens * 4);
    w.part = w.sid + up((size_t)tokens * 4);
    w.pairs = w.part + up((size_t)((tokens + kPiece - 1) / kPiece) * 2 * D * sizeof(float));
    w.counts = w.pairs + up(tokens > kDirect ? (size_t)tokens * 8 : 0);
    w.starts = w.counts + up(tokens > kDirect ? (size_t)kMostChunks * kMostRanges * 4 : 0);
    w.total = w.starts + up(tokens > kDirect ? (size_t)(kMostRanges + 1) * 4 : 0);
    return w;
}

// Exclusive prefix of v over the CTA's threads, and the sum of all.
__device__ __forceinline__ int cta_prefix(int v, int* warps, int& all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    __syncthreads();  // the last call's sums have been read
    if (lane == 31) warps[warp] = s;
    __syncthreads();
    int t = warps[lane], w = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += u;
    }
    all = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w - t, warp);
    return before + s - v;
}

// The id at place i of the warp's share: kNoId where there is none, or one
// that has no gradient (the padding id, or outside the table: then `wrong`).
constexpr unsigned kNoId = 0xffffffffu;
__device__ __forceinline__ unsigned load_id(const int64_t* __restrict__ ids, int i) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(ids + i));
    return v.y == 0 ? v.x : kNoId;
}
__device__ __forceinline__ unsigned load_id(const int32_t* __restrict__ ids, int i) { return (unsigned)__ldg(ids + i); }
template <typename ID>
__device__ __forceinline__ unsigned valid_id(const ID* __restrict__ ids, int i, int to, unsigned V, unsigned padding, bool& wrong) {
    if (i >= to) return kNoId;
    const unsigned v = load_id(ids, i);
    wrong = wrong || v >= V;
    return v >= V || v == padding ? kNoId : v;
}

// Where a CTA of the sort finds its range's tokens: among all, or in its part
// of the pairs (id, token) divided by range before.
template <typename ID> struct AllTokens {
    static constexpr bool kDivided = false;
    const ID* ids;
    int n;
    unsigned V, padding;
    __device__ __forceinline__ int2 places() const { return make_int2(0, n); }
    __device__ __forceinline__ unsigned id(int i, int to, bool& wrong) const { return valid_id(ids, i, to, V, padding, wrong); }
    __device__ __forceinline__ int token(int i) const { return i; }
};
struct RangeTokens {
    static constexpr bool kDivided = true;
    const int2* pairs;
    const int* starts;
    __device__ __forceinline__ int2 places() const { return make_int2(__ldg(starts + blockIdx.x), __ldg(starts + blockIdx.x + 1)); }
    __device__ __forceinline__ unsigned id(int i, int to, bool&) const { return i < to ? (unsigned)__ldg(&pairs[i].x) : kNoId; }
    __device__ __forceinline__ int token(int i) const { return __ldg(&pairs[i].y); }
};

// The range of an id: v / range, exactly, for ids below 2^21 and ranges of at
// most 2^10 (per = 2^32 / range + 1 in 32 bits; 0 where range is 1).
__device__ __forceinline__ int range_of(unsigned v, unsigned per) { return per ? (int)__umulhi(v, per) : (int)v; }

// How many of a chunk's tokens each range has: counts[chunk][range].
template <typename ID>
__global__ void __launch_bounds__(kSortThreads) embed_count_kernel(const AllTokens<ID> src, int chunk, int ranges, unsigned per, int* counts,
                                                                 unsigned* status) {
    __shared__ int count[kMostRanges];
    begin_kernel();
    for (int r = threadIdx.x; r < ranges; r += kSortThreads) count[r] = 0;
    __syncthreads();
    const int from = blockIdx.x * chunk, to = min(src.n, from + chunk);
    bool wrong = false;
    for (int j = from + (int)threadIdx.x; j < to; j += kSortThreads) {
        const unsigned v = src.id(j, to, wrong);
        if (v != kNoId) atomicAdd(count + range_of(v, per), 1);
    }
    if (wrong && status) atomicOr(status, kStatusIndex);
    __syncthreads();
    for (int r = threadIdx.x; r < ranges; r += kSortThreads) counts[blockIdx.x * ranges + r] = count[r];
}

// The chunk's pairs (id, token) to their ranges' parts, in token order; starts[r] is where range r's part begins.
template <typename ID>
__global__ void __launch_bounds__(kSortThreads) embed_divide_kernel(const AllTokens<ID> src, int chunk, int ranges, unsigned per,
                                                                  const int* __restrict__ counts, int2* pairs, int* starts) {
    extern __shared__ int next[];  // [kSortWarps][ranges]: a warp's next place in each range
    __shared__ int warps[32];
    __shared__ int sums[2][kSortThreads];
    begin_kernel();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, chunks = gridDim.x;
    int* mine = next + warp * ranges;
    for (int j = threadIdx.x; j < kSortWarps * ranges; j += kSortThreads) next[j] = 0;
    // a range's tokens in all chunks and in those before this one: threads side by side over the ranges, each a share of
    // the chunks
    const int shares = kSortThreads / ranges, r = threadIdx.x % ranges, share = threadIdx.x / ranges;
    int all = 0, before = 0;
    if (share < shares) {
#pragma unroll 16
        for (int c = share; c < chunks; c += shares) {
            const int n = __ldg(counts + c * ranges + r);
            all += n, before += c < (int)blockIdx.x ? n : 0;
        }
    }
    sums[0][threadIdx.x] = all, sums[1][threadIdx.x] = before;
    __syncthreads();
    const int from = blockIdx.x * chunk + warp * (chunk / kSortWarps), to = min(src.n, from + chunk / kSortWarps);
    bool wrong = false;
    for (int j = from + lane; j < to; j += 32) {
        const unsigned v = src.id(j, to, wrong);
        if (v != kNoId) atomicAdd(mine + range_of(v, per), 1);
    }
    if ((int)threadIdx.x < ranges)
        for (int k = 1; k < shares; ++k) all += sums[0][k * ranges + r], before += sums[1][k * ranges + r];
    int total;
    const int start = cta_prefix((int)threadIdx.x < ranges ? all : 0, warps, total);  // (its barriers end the counting, too)
    if ((int)threadIdx.x < ranges) {
        int at = start + before;
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w) {
            const int n = next[w * ranges + r];
            next[w * ranges + r] = at;
            at += n;
        }
        if (blockIdx.x == 0) starts[r] = start;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) starts[ranges] = total;
    __syncthreads();
    for (int j0 = from; j0 < to; j0 += 32) {
        const unsigned v = src.id(j0 + lane, to, wrong);
        const int k = v != kNoId ? range_of(v, per) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, k);
        int p = 0;
        if (k >= 0) p = mine[k] + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (k >= 0 && lane == __ffs(same) - 1) mine[k] += __popc(same);
        __syncwarp();
        if (k >= 0) pairs[p] = make_int2((int)v, j0 + lane);
    }
}

// off[v] for the ids of the range, and their tokens in order[off[v]..): by
// id, tokens of one id in their own order; sid the id at each place.
template <typename SRC>
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(const SRC src, int V, int range, int* off, int* order, int* sid,
                                                                unsigned* status) {
    extern __shared__ int counts[];  // [kSortWarps][range], then the first place of each id [range]
    __shared__ int warps[32];
    constexpr int U = 8;  // tokens of a lane in flight
    begin_kernel();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int lo = blockIdx.x * range, hi = min(V, lo + range);
    const int2 in = src.places();
    const int share = (in.y - in.x + kSortThreads - 1) / kSortThreads * 32, from = min(in.y, in.x + warp * share), to = min(in.y, from + share);
    int *cnt = counts + warp * range, *place = counts + kSortWarps * range;
    for (int j = threadIdx.x; j < kSortWarps * range; j += kSortThreads) counts[j] = 0;
    __syncthreads();
    const unsigned len = hi - lo;  // an id of the range, less lo, is below it; all others wrap or are above
    int less = 0;
    bool wrong = false;
    for (int j0 = from; j0 < to; j0 += 32 * U) {
        unsigned id[U];
#pragma unroll
        for (int u = 0; u < U; ++u) id[u] = src.id(j0 + 32 * u + lane, to, wrong);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!SRC::kDivided) less += id[u] < (unsigned)lo;
            if (id[u] - lo < len) atomicAdd(cnt + (id[u] - lo), 1);
        }
    }
    if (blockIdx.x == 0 && wrong && status) atomicOr(status, kStatusIndex);
    int base = in.x, total;
    if (!SRC::kDivided) cta_prefix(less, warps, base);  // (its barriers stand between the counts and their reading, too)
    else __syncthreads();
    int c[kSortWarps], sum = 0;
    if ((int)threadIdx.x < range) {
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) c[w] = counts[w * range + threadIdx.x];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            counts[w * range + threadIdx.x] = sum;
            sum += c[w];
        }
    }
    const int start = base + cta_prefix(sum, warps, total);
    if ((int)threadIdx.x < range) {
        place[threadIdx.x] = start;
        if (lo + (int)threadIdx.x < hi) off[lo + threadIdx.x] = start;
    }
    if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) off[V] = base + total;
    if (total == 0) return;
    __syncthreads();
    for (int j0 = from; j0 < to; j0 += 32 * U) {
        unsigned ids_[U];
#pragma unroll
        for (int u = 0; u < U; ++u) ids_[u] = src.id(j0 + 32 * u + lane, to, wrong);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const unsigned id = ids_[u] - lo;
            const bool mine = id < len;
            if (!__any_sync(0xffffffffu, mine)) continue;
            const unsigned same = __match_any_sync(0xffffffffu, mine ? id : kNoId);
            int p = 0;
            if (mine) p = place[id] + cnt[id] + __popc(same & ((1u << lane) - 1));
            __syncwarp();
            if (mine && lane == __ffs(same) - 1) cnt[id] += __popc(same);
            __syncwarp();
            if (mine) order[p] = src.token(j0 + 32 * u + lane), sid[p] = lo + (int)id;
        }
    }
}

struct EmbedParams {
    int V;
    int64_t D;
    float scale;
    const void* dy;
    const int *off, *order, *sid;
    float *dW, *part;
    int across_log2;  // groups of a CTA side by side over the columns
    int pieces;
};

// The sum of dy over order[from..to), columns of block cb.
template <typename IO, Layout L, int T, int NC>
__device__ __forceinline__ void add_tokens(const EmbedParams& p, int from, int to, int64_t c0, int t, float (&s)[NC][8]) {
    using C = Chunk<IO, L, T>;
    const IO* dy = static_cast<const IO*>(p.dy);
    constexpr int U = 4;  // tokens in flight
    for (int j = from; j < to; j += U) {
        C in[U][NC];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool there = j + u < to;
            const IO* row = dy + (int64_t)(there ? __ldg(p.order + j + u) : 0) * p.D;
#pragma unroll
            for (int k = 0; k < NC; ++k) in[u][k].load(row, there ? p.D : 0, c0 + (int64_t)k * 8 * T, t);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                float f[8];
                in[u][k].get(f);
#pragma unroll
                for (int i = 0; i < 8; ++i) s[k][i] += f[i];
            }
    }
}
template <Layout L, int T, int NC>
__device__ __forceinline__ void store_row(float* row, int64_t D, int64_t c0, int t, float scale, const float (&s)[NC][8]) {
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = s[k][i] * scale;
        Chunk<float, L, T>::store(row, D, c0 + (int64_t)k * 8 * T, t, f);
    }
}

// Groups of T lanes take pieces first (the longest work), then rows. A CTA's
// groups lie side by side over the columns of a row, as many as it has blocks
// of 8 T NC (at most all of them: then each takes every so many blocks), and
// over rows beyond that, so that what a CTA writes at a time is one run.
template <typename IO, Layout L, int T, int NC>
__global__ void __launch_bounds__(kRowThreads) embed_rows_kernel(const EmbedParams p) {
    constexpr int kGroups = kRowThreads / T, kSpan = 8 * T * NC;
    const int t = threadIdx.x % T, group = threadIdx.x / T;
    const int across = 1 << p.across_log2, down = kGroups >> p.across_log2;
    const int64_t c_first = (int64_t)(group & (across - 1)) * kSpan, c_step = (int64_t)across * kSpan;
    const int step = gridDim.x * down, own = blockIdx.x * down + (group >> p.across_log2);
    begin_kernel();
    const int valid = __ldg(p.off + p.V);
    int piece = own;
    for (; piece < p.pieces; piece += step) {
        const int first = piece * kPiece, last = min(valid, first + kPiece) - 1;
        if (first > last) continue;
        const int va = __ldg(p.sid + first), vb = __ldg(p.sid + last);
        const int ea = __ldg(p.off + va + 1), sb = __ldg(p.off + vb);
        const bool head = ea - __ldg(p.off + va) > kPiece, tail = vb != va && __ldg(p.off + vb + 1) - sb > kPiece;
        for (int64_t c0 = c_first; c0 < p.D; c0 += c_step) {
            if (head) {
                float s[NC][8] = {};
                add_tokens<IO, L, T, NC>(p, first, min(ea, last + 1), c0, t, s);
                store_row<L, T, NC>(p.part + (int64_t)piece * 2 * p.D, p.D, c0, t, 1.f, s);
            }
            if (tail) {
                float s[NC][8] = {};
                add_tokens<IO, L, T, NC>(p, sb, last + 1, c0, t, s);
                store_row<L, T, NC>(p.part + ((int64_t)piece * 2 + 1) * p.D, p.D, c0, t, 1.f, s);
            }
        }
    }
    // (the rows go round from where the pieces ended)
    int v = piece - p.pieces;
    int from = 0, to = 0;
    if (v < p.V) from = __ldg(p.off + v), to = __ldg(p.off + v + 1);
    while (v < p.V) {
        const int next = v + step;  // its run is looked up while this row is added
        int nfrom = 0, nto = 0;
        if (next < p.V) nfrom = __ldg(p.off + next), nto = __ldg(p.off + next + 1);
        if (to - from <= kPiece) {
            for (int64_t c0 = c_first; c0 < p.D; c0 += c_step) {
                float s[NC][8] = {};
                add_tokens<IO, L, T, NC>(p, from, to, c0, t, s);
                store_row<L, T, NC>(p.dW + (int64_t)v * p.D, p.D, c0, t, p.scale, s);
            }
        }
        v = next, from = nfrom, to = nto;
    }
}

// Rows whose run is longer than a piece: the CTA of the piece that such a run
// starts in adds its partial sums, 32 x 8 columns, each warp a share of them
// in order.
__global__ void __launch_bounds__(kRowThreads) embed_join_kernel(const EmbedParams p) {
    constexpr int kW = kRowThreads / 32;
    __shared__ float sums[kW][256];
    begin_kernel();
    const int first = blockIdx.x * kPiece, valid = __ldg(p.off + p.V), last = min(valid, first + kPiece) - 1;
    if (first > last) return;
    const int v = __ldg(p.sid + last), from = __ldg(p.off + v), to = __ldg(p.off + v + 1);
    if (to - from <= kPiece || from < first) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c0 = (int64_t)blockIdx.y * 256;
    const int a = from / kPiece, n = (to - 1) / kPiece - a + 1;  // partial sums: of the first piece, then of each after it
    const int share = (n + kW - 1) / kW;
    float s[8] = {};
#pragma unroll 2
    for (int j = warp * share; j < min(n, (warp + 1) * share); ++j) {
        const int slot = 2 * (a + j) + (j == 0 && from % kPiece != 0);
        const float* row = p.part + (int64_t)slot * p.D + c0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c0 + 32 * i + lane < p.D) s[i] += __ldg(row + 32 * i + lane);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[warp][32 * i + lane] = s[i];
    __syncthreads();
    if (c0 + threadIdx.x < p.D) {
        float f = 0.f;
#pragma unroll
        for (int w = 0; w < kW; ++w) f += sums[w][threadIdx.x];
        p.dW[(int64_t)v * p.D + c0 + threadIdx.x] = f * p.scale;
    }
}

// out = scale * W[id]: groups of T lanes take a token each.
template <typename IO, Layout L, int T, int NC, typename ID>
__global__ void __launch_bounds__(kRowThreads) embed_fwd_kernel(const ID* __restrict__ ids, int64_t n, int64_t V, int64_t D,
                                                              float scale, const IO* __restrict__ W, IO* out, int blocks,
                                                              unsigned* status) {
    using C = Chunk<IO, L, T>;
    begin_kernel();
    const int t = threadIdx.x % T;
    const int64_t groups = (int64_t)gridDim.x * (kRowThreads / T), units = n * blocks;
    bool wrong = false;
    for (int64_t unit = (int64_t)blockIdx.x * (kRowThreads / T) + threadIdx.x / T; unit < units; unit += groups) {
        const int64_t row = unit / blocks, c0 = (unit - row * blocks) * (8 * T * NC), v = __ldg(ids + row);
        const bool there = v >= 0 && v < V;
        wrong = wrong || !there;
        C in[NC];
#pragma unroll
        for (int k = 0; k < NC; ++k) in[k].load(W + (there ? v : 0) * D, there ? D : 0, c0 + (int64_t)k * 8 * T, t);
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            float f[8];
            in[k].get(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= scale;
            C::store(out + row * D, D, c0 + (int64_t)k * 8 * T, t, f);
        }
    }
    if (wrong && status) atomicOr(status, kStatusIndex);
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool off(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// As many CTAs of a grid-striding kernel as are resident.
template <typename K> int64_t slots(K kern, int (&per_sm)[64]) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -1;
    int& n = per_sm[dev & 63];
    if (n == 0 && (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, kRowThreads, 0) != cudaSuccess || n < 1)) {
        n = 0;
        return -1;
    }
    return (int64_t)n * sm_count();
}

template <typename IO, Layout L, int T, int NC> int launch_rows(EmbedParams p, cudaStream_t s) {
    static int per_sm[64] = {};
    auto kern = embed_rows_kernel<IO, L, T, NC>;
    const int64_t most = slots(kern, per_sm);
    if (most < 1) return -1;
    constexpr int kGroups = kRowThreads / T, kSpan = 8 * T * NC;
    p.across_log2 = 0;
    while (1 << p.across_log2 < kGroups && (kSpan << p.across_log2) < p.D) ++p.across_log2;
    const int64_t down = kGroups >> p.across_log2, want = (p.pieces + (int64_t)p.V + down - 1) / down;
    if (launch_next(kern, dim3((unsigned)(want < most ? want : most)), kRowThreads, 0, s, p) < 0) return -1;
    if (p.pieces < 2) return 1;  // no run is longer than the whole list
    return launch_next(embed_join_kernel, dim3((unsigned)p.pieces, (unsigned)((p.D + 255) / 256)), kRowThreads, 0, s, p) < 0 ? -1 : 2;
}
template <typename IO, Layout L, int T, int NC, typename ID>
int launch_lookup(const ssm_embed_args& a, cudaStream_t s) {
    static int per_sm[64] = {};
    auto kern = embed_fwd_kernel<IO, L, T, NC, ID>;
    const int64_t most = slots(kern, per_sm);
    if (most < 1) return -1;
    const int blocks = (int)((a.D + 8 * T * NC - 1) / (8 * T * NC));
    const int64_t want = (a.tokens * blocks + kRowThreads / T - 1) / (kRowThreads / T);
    return launch_next(kern, dim3((unsigned)(want < most ? want : most)), kRowThreads, 0, s, static_cast<const ID*>(a.ids), a.tokens, a.V,
                       a.D, a.scale, static_cast<const IO*>(a.W), static_cast<IO*>(a.out), blocks, static_cast<unsigned*>(a.status));
}
// Lanes and chunks by the row's width: at most 1024 columns a group in the
// lookup (16384 of 50001 x 2048 bf16, the same ids again: 17.3 us; at most 512 18.9, 256 26.6);
// 256 in the gradient, whose sums then take few enough registers for 48 warps
// an SM. Rows of up to 32 and 128 elements take 4 and 16 lanes (65536 of
// 50001 x 32: 6.4 us, with a warp 12.6; the gradient 42.5 and 48.7).
#define EMBED_GROUP(D, F)          \
    do {                           \
        if ((D) <= 32) F(4, 1);    \
        if ((D) <= 128) F(16, 1);  \
        if ((D) <= 256) F(32, 1);  \
        if ((D) <= 512) F(32, 2);  \
        F(32, 4);                  \
    } while (0)
template <typename IO, Layout L> int rows_by_width(const EmbedParams& p, cudaStream_t s) {
    if (p.D <= 32) return launch_rows<IO, L, 4, 1>(p, s);
    if (p.D <= 128) return launch_rows<IO, L, 16, 1>(p, s);
    return launch_rows<IO, L, 32, 1>(p, s);
}
template <typename IO, Layout L, typename ID> int lookup_by_width(const ssm_embed_args& a, cudaStream_t s) {
#define EMBED_F(T, NC) return launch_lookup<IO, L, T, NC, ID>(a, s)
    EMBED_GROUP(a.D, EMBED_F);
#undef EMBED_F
}
template <typename IO> int lookup(const ssm_embed_args& a, cudaStream_t s) {
    const bool vec = a.D * (int64_t)sizeof(IO) % 16 == 0 && on16(a.W) && on16(a.out);
    if (a.ids64) return vec ? lookup_by_width<IO, kVector<IO>, int64_t>(a, s) : lookup_by_width<IO, Layout::kEach, int64_t>(a, s);
    return vec ? lookup_by_width<IO, kVector<IO>, int32_t>(a, s) : lookup_by_width<IO, Layout::kEach, int32_t>(a, s);
}

int check_embed(int64_t tokens, int64_t V, int64_t D, int io, int ids64, float scale, const void* ids) {
    if (tokens < 0 || V < 0 || D < 0) return SSM_ERR_INVALID_ARG;
    if (io != SSM_F32 && io != SSM_BF16) return SSM_ERR_UNSUPPORTED;
    if ((ids64 != 0 && ids64 != 1) || !std::isfinite(scale)) return SSM_ERR_INVALID_ARG;
    if (tokens > 0x3fffffff || V > 0x3fffffff || D > (int64_t(1) << 20)) return SSM_ERR_UNSUPPORTED;
    if (tokens > 0 && D > 0 && !ids) return SSM_ERR_INVALID_ARG;
    return off(ids, ids64 ? 8 : 4) ? SSM_ERR_ALIGNMENT : SSM_OK;
}

}  // namespace
}  // namespace ssm

extern "C" {

size_t ssm_embed_workspace_bytes(int64_t tokens, int64_t V, int64_t D) {
    if (tokens <= 0 || V <= 0 || D <= 0) return 0;
    return ssm::embed_ws(tokens, V, D).total;
}

int ssm_embed_fwd(const ssm_embed_args* a, void* stream) {
    ssm::reset_launches();
    if (!a) return SSM_ERR_INVALID_ARG;
    const int rc = ssm::check_embed(a->tokens, a->V, a->D, a->io_dtype, a->ids64, a->scale, a->ids);
    if (rc != SSM_OK) return rc;
    const bool work = a->tokens > 0 && a->D > 0;
    if (work && (!a->out || (a->V > 0 && !a->W))) return SSM_ERR_INVALID_ARG;
    const unsigned es = a->io_dtype == SSM_BF16 ? 2 : 4;
    if (ssm::off(a->W, es) || ssm::off(a->out, es) || ssm::off(a->status, 16)) return SSM_ERR_ALIGNMENT;
    if (!work) return SSM_OK;
    cudaStream_t s = (cudaStream_t)stream;
    return ssm::count_launches(a->io_dtype == SSM_BF16 ? ssm::lookup<__nv_bfloat16>(*a, s) : ssm::lookup<float>(*a, s));
}

int ssm_embed_bwd(const ssm_embed_bwd_args* a, void* stream) {
    ssm::reset_launches();
    if (!a) return SSM_ERR_INVALID_ARG;
    int rc = ssm::check_embed(a->tokens, a->V, a->D, a->io_dtype, a->ids64, a->scale, a->ids);
    if (rc != SSM_OK) return rc;
    const bool work = a->tokens > 0 && a->V > 0 && a->D > 0;
    if (a->V > 0 && a->D > 0 && !a->dW) return SSM_ERR_INVALID_ARG;
    if (work && !a->dy) return SSM_ERR_INVALID_ARG;
    const unsigned es = a->io_dtype == SSM_BF16 ? 2 : 4;
    if (ssm::off(a->dy, es) || ssm::off(a->dW, 4) || ssm::off(a->workspace, 16) || ssm::off(a->status, 16)) return SSM_ERR_ALIGNMENT;
    if (work && (!a->workspace || a->workspace_bytes < ssm_embed_workspace_bytes(a->tokens, a->V, a->D))) return SSM_ERR_WORKSPACE;
    cudaStream_t s = (cudaStream_t)stream;
    if (a->V == 0 || a->D == 0) return SSM_OK;
    if (!work)
        return cudaMemsetAsync(a->dW, 0, (size_t)a->V * a->D * sizeof(float), s) == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
    const ssm::EmbedWs w = ssm::embed_ws(a->tokens, a->V, a->D);
    char* ws = static_cast<char*>(a->workspace);
    const int sms = ssm::sm_count();
    int range = (int)((a->V + sms - 1) / sms);
    if (range > ssm::kMostIds) range = ssm::kMostIds;
    const unsigned grid = (unsigned)((a->V + range - 1) / range);
    int* off = reinterpret_cast<int*>(ws + w.off);
    int *order = reinterpret_cast<int*>(ws + w.order), *sid = reinterpret_cast<int*>(ws + w.sid);
    const int smem = (ssm::kSortWarps + 1) * range * (int)sizeof(int), most = (ssm::kSortWarps + 1) * ssm::kMostIds * (int)sizeof(int);
    auto sort = [&](auto tag) {
        using ID = decltype(tag);
        static unsigned long long all_mask = 0, part_mask = 0, divide_mask = 0;
        const ssm::AllTokens<ID> all{static_cast<const ID*>(a->ids), (int)a->tokens, (unsigned)a->V,
                                     a->padding_id < 0 || a->padding_id >= a->V ? ssm::kNoId : (unsigned)a->padding_id};
        unsigned* status = static_cast<unsigned*>(a->status);
        if (a->tokens <= ssm::kDirect || grid > (unsigned)ssm::kMostRanges) {
            if (!ssm::ensure_smem(ssm::embed_sort_kernel<ssm::AllTokens<ID>>, most, all_mask)) return -1;
            return ssm::launch_next(ssm::embed_sort_kernel<ssm::AllTokens<ID>>, dim3(grid), ssm::kSortThreads, smem, s, all, (int)a->V, range,
                                    off, order, sid, status);
        }
        int2* pairs = reinterpret_cast<int2*>(ws + w.pairs);
        int *counts = reinterpret_cast<int*>(ws + w.counts), *starts = reinterpret_cast<int*>(ws + w.starts);
        const int64_t each = (a->tokens + ssm::kMostChunks - 1) / ssm::kMostChunks;
        const int chunk = (int)((each + ssm::kChunk - 1) / ssm::kChunk * ssm::kChunk);
        const unsigned chunks = (unsigned)((a->tokens + chunk - 1) / chunk);
        const unsigned per = range == 1 ? 0u : (unsigned)((1ull << 32) / (unsigned)range + 1);
        const int next = ssm::kSortWarps * (int)grid * (int)sizeof(int);
        if (!ssm::ensure_smem(ssm::embed_sort_kernel<ssm::RangeTokens>, most, part_mask) ||
            !ssm::ensure_smem(ssm::embed_divide_kernel<ID>, ssm::kSortWarps * ssm::kMostRanges * (int)sizeof(int), divide_mask))
            return -1;
        if (ssm::launch_next(ssm::embed_count_kernel<ID>, dim3(chunks), ssm::kSortThreads, 0, s, all, chunk, (int)grid, per, counts, status) < 0 ||
            ssm::launch_next(ssm::embed_divide_kernel<ID>, dim3(chunks), ssm::kSortThreads, next, s, all, chunk, (int)grid, per,
                             static_cast<const int*>(counts), pairs, starts) < 0 ||
            ssm::launch_next(ssm::embed_sort_kernel<ssm::RangeTokens>, dim3(grid), ssm::kSortThreads, smem, s,
                             ssm::RangeTokens{pairs, starts}, (int)a->V, range, off, order, sid, status) < 0)
            return -1;
        return 3;
    };
    rc = ssm::count_launches(a->ids64 ? sort(int64_t{}) : sort(int32_t{}));
    if (rc != SSM_OK) return rc;
    ssm::EmbedParams p{};
    p.V = (int)a->V; p.D = a->D; p.scale = a->scale; p.dy = a->dy;
    p.off = off; p.order = order; p.sid = sid; p.dW = a->dW; p.part = reinterpret_cast<float*>(ws + w.part);
    p.pieces = (int)((a->tokens + ssm::kPiece - 1) / ssm::kPiece);
    // Vectors where rows and sums allow them: four elements in bf16, two in fp32 (16384 ids of 50001 x 1024 fp32: 70 us
    // in twos, 80 in fours, 71 singly; of 50001 x 2048 bf16: 106, 105 and 113).
    const unsigned n = a->io_dtype == SSM_BF16 ? 4 : 2;
    const bool vec = a->D % n == 0 && !ssm::off(a->dy, n * es) && !ssm::off(a->dW, n * 4);
    if (a->io_dtype == SSM_BF16)
        return ssm::count_launches(vec ? ssm::rows_by_width<__nv_bfloat16, ssm::Layout::kQuad>(p, s)
                                       : ssm::rows_by_width<__nv_bfloat16, ssm::Layout::kEach>(p, s));
    return ssm::count_launches(vec ? ssm::rows_by_width<float, ssm::Layout::kPair>(p, s) : ssm::rows_by_width<float, ssm::Layout::kEach>(p, s));
}

}  // extern "C"
