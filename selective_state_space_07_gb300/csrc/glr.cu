// Gated linear recurrence on sm_103a: forward, backward and single-token step
// (include/glr.h holds the formulas and the boundary).
//
// The recurrence h_t = a_t h_{t-1} + b_t is a composition of affine maps, one
// per token: (a2, b2) o (a1, b1) = (a1 a2, a2 b1 + b2). It streams x and two
// gates in and y out once, so HBM bounds it, if the work along L can be cut
// finely enough to fill the GPU without reading anything twice.
//
// Work is cut into tiles of 64 tokens x 64 channels (32 tokens in fp32: as
// many bytes), one CTA of four warps each: a warp takes a run of 16 (8) of a
// tile's tokens, a lane two neighbouring channels, so that its arithmetic is
// in pairs. A warp scans its run from a zero state, keeping h_j and the
// running product P_j; the four warps' maps meet in shared memory; and
// y_j = h_j + P_j * (state before the run). (Eight warps of 8 tokens: 126 us
// where four of 16 take 105.)
//
// The state before a tile comes from the tiles before it in one pass over the
// data (the published single-pass scan with look-back): every tile publishes its map (P, H), and every 16th the state after
// it; a tile takes the last such state and applies the at most 15 maps in
// between, in order. (Where few columns make the chain of those states count,
// the state comes after every 256th tile, and the map of each block of 16,
// which waits for no state.) Which values are combined, and in which order,
// depends on the tile's place alone, so results do not depend on timing. The
// words published start as a pattern that no arithmetic gives (all ones), so a
// reader polls the values themselves: no flags, no fences.
//
// CTAs are persistent. Tiles are numbered chunk by chunk and handed out by a
// ticket; a CTA holds the tickets of its next tiles, whose copies (TMA, one
// box per input) fill its other stages meanwhile, and works on them in order.
// A tile only waits for lower tickets, and the lowest one unfinished is
// always being worked on, so every wait ends; all the same each is bounded.
//
// The backward runs the same scheme from the last chunk to the first over
// v = a g (what a token hands to the one before it): per warp (P, V), the
// same products P. The states h_{t-1} that the gradients need are recomputed
// in fp32 from the state that the forward saved before the tile's first token,
// so no bf16 copy of them enters the gradients. (States are saved every 32
// tokens for either type; a bf16 tile has 64 and takes every other one.)
//
// Measured, bf16 unless said, in percent of the HBM copy rate, for slow decays
// (c softplus(lam) < 1/4): 4 x 4096 x 4096 forward with checkpoints 101 us
// (79%), backward 200 (69%), other decays 108 and 223; 4 x 2048 x 4096 fp32 89
// (88%) and 157 (88%). 1 x 65536 x 2048: 267 us (59%) and 481, other decays 281
// and 553; each of its 19 chunks at work at a time waits for those before it.
// Registers allow 16 warps an SM forward and 12 backward, which issue in half
// of the slots (32 and 59 instructions an element). 2 x 509 x 256 fp32, both
// passes 22 us: launches.
#include <cmath>
#include <type_traits>

#include "../../include/glr.h"
#include "ssm_common.cuh"
#include "ssm_internal.h"

namespace ssm {
namespace {

constexpr int kWarps = 4;
constexpr int kCols = 64;                // channels of a tile
constexpr int kThreads = 32 * kWarps;
// Chunks of a block, and of a span, between published states: a block, or 16
// blocks whose maps are published too. Long spans where a sequence has few
// columns, so that many of its chunks are at work at a time and would wait for
// one state after the other: 1 x 65536 x 64 bf16 16 us forward and 31 backward
// (47 and 62 with short spans), 8 columns of 704 chunks 55 and 118 (55 and
// 126); where there are many columns the second look costs more than it saves
// (32 columns of 1024 chunks 268 and 519, with short spans 264 and 511).
constexpr int kBlock = 16, kLongSpan = 16 * kBlock;
constexpr unsigned kFewColumns = 8;
constexpr int kCkptTokens = 32;          // tokens between saved states
constexpr int kRedThreads = 256;
constexpr unsigned kEmpty = 0xffffffffu; // a word not yet published

// Tokens of a warp and of a tile (a chunk of the sequence), by I/O type: a
// tile of one input is 8 KB either way.
template <typename IO> constexpr int kTok = 32 / (int)sizeof(IO);
template <typename IO> constexpr int kChunk = kTok<IO> * kWarps;
template <typename IO> constexpr int kBoxBytes = kChunk<IO> * kCols * (int)sizeof(IO);
constexpr int chunk_tokens(int io) { return io == SSM_BF16 ? kChunk<__nv_bfloat16> : kChunk<float>; }

struct GlrParams {
    int64_t B, L, D;
    int64_t sx, sr, si;  // elements from one token's row to the next
    float c;
    const void *x, *r, *i, *dy;
    const float *lam, *start;  // start: h0 (forward) or dh_last (backward), nullable
    void *y, *dx, *dr, *di;
    float *end, *ckpt;  // end: h_last (forward) or dh0 (backward), nullable
    float* part;        // backward: [chunks * B, D] partial sums of dloga * r
    unsigned* status;
    unsigned* sync;     // [0] the last ticket taken, [1] kEmpty until a wait runs out
    float4* maps;       // [tiles, 32]: (P, H) of two channels a lane
    float4* blocks;     // [blocks * columns, 32]: the maps of whole blocks
    float2* states;     // [spans * columns, 32]: the states behind them
    float* cs;          // [D]: c * softplus(lam)
    float* held;        // [B, D]: a copy of start, where end is written in its place
    unsigned columns, chunks, per_row;  // columns = B * per_row
    int64_t fault_chunk1;
    unsigned long long wait_ns;
};
// TMA descriptors of the inputs as [B*L, D] in boxes of a tile; what lies
// past the last row or channel reads as zero.
struct GlrBoxes {
    CUtensorMap x, r, i, dy;
};

// The workspace behind the status word: what tiles publish comes first, in
// one piece that starts as all ones. For the larger of the two tile counts
// (fp32's), so that one size serves both types.
struct GlrWs {
    size_t sync, publish_bytes, maps, blocks, states, cs, held, part, total;
};
GlrWs glr_ws(int64_t B, int64_t L, int64_t D, int chunk) {
    const size_t columns = (size_t)B * ((D + kCols - 1) / kCols), chunks = (size_t)((L + chunk - 1) / chunk);
    const size_t blocks = (chunks + kBlock - 1) / kBlock, tiles = columns * chunks;
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    const bool multi = chunks > 1;
    GlrWs w;
    w.sync = 256;
    w.maps = w.sync + (multi ? 256 : 0);
    w.blocks = w.maps + (multi ? tiles * 32 * sizeof(float4) : 0);
    w.states = w.blocks + (multi ? blocks * columns * 32 * sizeof(float4) : 0);
    w.cs = w.states + (multi ? blocks * columns * 32 * sizeof(float2) : 0);
    w.publish_bytes = w.cs - w.sync;
    w.held = w.cs + (multi ? up((size_t)D * sizeof(float)) : 0);
    w.part = w.held + (multi ? up((size_t)B * D * sizeof(float)) : 0);
    w.total = w.part + up((size_t)B * chunks * D * sizeof(float));
    return w;
}

// Published words: each 32-bit word is written once, and is its own message.
__device__ __forceinline__ float4 ld_word4(const float4* p) {
    float4 v;
    asm volatile("ld.relaxed.gpu.global.v4.f32 {%0, %1, %2, %3}, [%4];\n"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_word2(const float2* p) {
    float2 v;
    asm volatile("ld.relaxed.gpu.global.v2.f32 {%0, %1}, [%2];\n" : "=f"(v.x), "=f"(v.y) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ unsigned ld_word(const unsigned* p) {
    unsigned v;
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];\n" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ float word(float v) {  // a NaN that happens to be the empty pattern becomes another NaN
    return __float_as_uint(v) == kEmpty ? __uint_as_float(0x7fffffffu) : v;
}
__device__ __forceinline__ void st_words(float4* p, float4 v) {
    asm volatile("st.relaxed.gpu.global.v4.f32 [%0], {%1, %2, %3, %4};\n" ::"l"(p), "f"(word(v.x)), "f"(word(v.y)),
                 "f"(word(v.z)), "f"(word(v.w)) : "memory");
}
__device__ __forceinline__ void st_words(float2* p, float2 v) {
    asm volatile("st.relaxed.gpu.global.v2.f32 [%0], {%1, %2};\n" ::"l"(p), "f"(word(v.x)), "f"(word(v.y)) : "memory");
}
// kEmpty, the greatest word, if any word of a value is empty
__device__ __forceinline__ unsigned greatest(float2 v) { return max(__float_as_uint(v.x), __float_as_uint(v.y)); }
__device__ __forceinline__ unsigned greatest(float4 v) { return max(greatest(pk(v.x, v.y)), greatest(pk(v.z, v.w))); }
__device__ __forceinline__ float sqrt_approx(float x) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 dup(float v) { return pk(v, v); }

// Two channels of one token as loaded, and as fp32.
template <typename IO> struct Pair;
template <> struct Pair<float> {
    using T = float2;
    __device__ static T ld(const float* p) { return __ldg(reinterpret_cast<const float2*>(p)); }
    __device__ static T lds(const char* p) { return *reinterpret_cast<const float2*>(p); }
    __device__ static float2 f(T v) { return v; }
    __device__ static T none() { return pk(0.f, 0.f); }
};
template <> struct Pair<__nv_bfloat16> {
    using T = unsigned;
    __device__ static T ld(const __nv_bfloat16* p) { return __ldg(reinterpret_cast<const unsigned*>(p)); }
    __device__ static T lds(const char* p) { return *reinterpret_cast<const unsigned*>(p); }
    __device__ static float2 f(T w) { return pk(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
    __device__ static T none() { return 0u; }
};

__device__ __forceinline__ float softplus_full(float v) { return fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v))); }

// The gates of two channels, cs = c * softplus(lam): of t = cs r = -log a come
// a = exp(-t) and w = 1 - a, each with all its digits, so that neither slow
// decays (w, and 1 - a^2 = w (2 - w)) nor fast ones (a) cancel. Below t = 1/4,
// w = t (1 - t/2 + t^2/6 - ...), the terms left out below 5e-8 of the sum, and
// a = 1 - w; above, a = 2^(-t log2e) and w = 1 - a.
// The exponential of -t is the MUFU form for both I/O types: its relative error
// (2^-22, and as much as t's own rounding) is that of fp32 sums. The sigmoid's
// would grow with |z|, as n = -z log2e is rounded (6e-7 at z = -10, 4e-6 at
// -70): in fp32 I/O its e = 2^n gets what n lacks (Cody and Waite's reduction),
// e + e (-z - n ln 2). (4 x 2048 x 4096 fp32 with expf and divisions instead:
// forward 118 us, backward 187 to 226.)
// SERIES: every t of the warp is known to be below 1/4 (t = cs r <= cs).
template <typename IO> __device__ __forceinline__ float2 gate2(float2 z) { return sigmoid2<true>(z); }
__device__ __forceinline__ float within(float v, float most) {  // (a NaN stays one)
    float u;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(u) : "f"(v), "f"(-most));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(u) : "f"(u), "f"(most));
    return u;
}
template <> __device__ __forceinline__ float2 gate2<float>(float2 z) {
    const float2 x = pk(within(-z.x, 88.0f), within(-z.y, 88.0f));  // (e^88 is finite, and its reciprocal flushed to 0)
    const float2 n = __fmul2_rn(x, dup(kLog2e));
    const float2 d = __ffma2_rn(n, dup(1.904654290e-9f), __ffma2_rn(n, dup(-kLn2), x));  // x - n ln 2, with ln 2 in two parts
    float2 e = pk(ex2(n.x), ex2(n.y));
    e = __ffma2_rn(e, d, e);
    const float2 w = __fadd2_rn(dup(1.0f), e);
    return pk(rcp(w.x), rcp(w.y));
}
struct Decay {
    float2 a, w;
};
__device__ __forceinline__ float2 one_minus(float2 v) { return __ffma2_rn(v, dup(-1.f), dup(1.f)); }
template <bool SERIES> __device__ __forceinline__ Decay decay(float2 t) {
    float2 p = __ffma2_rn(t, dup(-1.0f / 720), dup(1.0f / 120));
    p = __ffma2_rn(p, t, dup(-1.0f / 24));
    p = __ffma2_rn(p, t, dup(1.0f / 6));
    p = __ffma2_rn(p, t, dup(-0.5f));
    p = __ffma2_rn(p, t, dup(1.0f));
    p = __fmul2_rn(p, t);
    const float2 q = one_minus(p);
    if (SERIES) return {q, p};
    const float2 z = __fmul2_rn(t, dup(-kLog2e)), e = pk(ex2(z.x), ex2(z.y)), f = one_minus(e);
    return {pk(t.x < 0.25f ? q.x : e.x, t.y < 0.25f ? q.y : e.y), pk(t.x < 0.25f ? p.x : f.x, t.y < 0.25f ? p.y : f.y)};
}
// Both in one word, for the backward, which keeps them for each token: v = w
// near 1, else v = -a (never -0). With n = 1 where v >= 0 and 0 elsewhere,
// a = n - v and 1 - a^2 = v (a + n) + 1 - n.
template <bool SERIES> __device__ __forceinline__ float2 hold(const Decay& d) {
    if (SERIES) return d.w;
    const float2 v = __ffma2_rn(d.a, dup(-1.f), dup(-1.17549435e-38f));
    return pk(d.w.x < 0.2211f ? d.w.x : v.x, d.w.y < 0.2211f ? d.w.y : v.y);
}
__device__ __forceinline__ float not_negative(float v) {
    float n;
    asm("set.ge.f32.f32 %0, %1, 0f00000000;" : "=f"(n) : "f"(v));
    return n;
}
struct Held {
    float2 n, a;
};
template <bool SERIES> __device__ __forceinline__ Held held_decay(float2 v) {
    if (SERIES) return {dup(1.f), one_minus(v)};
    const float2 n = pk(not_negative(v.x), not_negative(v.y));
    return {n, __ffma2_rn(v, dup(-1.f), n)};
}
// Whether the series is enough for all of a warp's channels. (It alone: 101 us
// forward, 200 backward at 4 x 4096 x 4096 bf16; with the choice for each
// element 108 and 223.)
__device__ __forceinline__ bool all_series(float2 cs) { return __all_sync(0xffffffffu, cs.x < 0.25f && cs.y < 0.25f); }
// 1 - a^2 of w = 1 - a
__device__ __forceinline__ float2 input_power(float2 w) { return __fmul2_rn(w, __ffma2_rn(w, dup(-1.f), dup(2.f))); }
__device__ __forceinline__ float2 sqrt2(float2 v) { return pk(sqrt_approx(v.x), sqrt_approx(v.y)); }
__device__ __forceinline__ float rsqrt_approx(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 apply(float4 f, float2 h) { return __ffma2_rn(pk(f.x, f.y), h, pk(f.z, f.w)); }
// g after f
__device__ __forceinline__ float4 compose(float4 f, float4 g) {
    const float2 P = __fmul2_rn(pk(f.x, f.y), pk(g.x, g.y)), H = apply(g, pk(f.z, f.w));
    return make_float4(P.x, P.y, H.x, H.y);
}
constexpr float4 kIdentity = {1.f, 1.f, 0.f, 0.f};

// Where a tile lies: tk counts in the order of the scan, columns fastest,
// then chunks (from the last in the backward). One thread works it out for
// the CTA.
struct Tile {
    unsigned tk, k, col, chunk, b;
    int c0, rows;   // the column's first channel; the chunk's tokens
    int64_t out;    // element of the tile's first row and channel in a dense [B, L, D]
    int64_t state;  // ... in a [B, D]
    int64_t saved;  // ... in the saved states, of the chunk's first
};
template <typename IO> __device__ __forceinline__ Tile find_tile(const GlrParams& p, unsigned tk, bool reverse) {
    Tile t;
    t.tk = tk;
    t.k = tk / p.columns;
    t.col = tk - t.k * p.columns;
    t.chunk = reverse ? p.chunks - 1 - t.k : t.k;
    t.b = t.col / p.per_row;
    t.c0 = (int)(t.col - t.b * p.per_row) * kCols;
    const int64_t first = (int64_t)t.chunk * kChunk<IO>, per = (p.L + kCkptTokens - 1) / kCkptTokens;
    t.rows = (int)min64(kChunk<IO>, p.L - first);
    t.out = (t.b * p.L + first) * p.D + t.c0;
    t.state = t.b * p.D + t.c0;
    t.saved = (t.b * per + first / kCkptTokens) * p.D + t.c0;
    return t;
}
// A lane's place in any tile: its channels, its warp's run of tokens.
template <typename IO> struct Lane {
    int ch, t0;       // the lane's first channel within the column, the run's first token within the chunk
    int64_t row_off;  // elements from the tile's first to the lane's first in a dense [B, L, D]
    __device__ explicit Lane(const GlrParams& p)
        : ch(2 * (threadIdx.x & 31)), t0((threadIdx.x >> 5) * kTok<IO>), row_off((int64_t)t0 * p.D + ch) {}
    __device__ bool live(const GlrParams& p, const Tile& t) const { return t.c0 + ch < p.D; }
    // how many of the run's tokens exist (0 past the last channel)
    __device__ int tokens(const GlrParams& p, const Tile& t) const {
        return live(p, t) ? max(0, min(kTok<IO>, t.rows - t0)) : 0;
    }
};

// What a tile's warps hand one another. Read between a tile's two barriers
// only, so the next tile may write it after the second.
struct TileMaps {
    float4 run[kWarps][32];  // (P, H) of a warp's run; P shared by both directions
    float2 back[kWarps][32]; // V of the reverse scan (backward only)
};
struct Look {
    float4 four[4][32];    // published maps of the block's chunks, four composed
    float4 blocks[4][32];  // published maps of the span's blocks, four composed
    float2 state[32];      // the state they start from
    int failed;
};

// Polls until every word of f[0..n) is there. False when the wait ran out,
// here or in another tile. Between polls the warp sleeps a little, so that it
// leaves the issue slots to warps with work; the clock and the abort word are
// looked at every 16th time.
template <int N, typename V, typename Load>
__device__ __forceinline__ bool poll(const GlrParams& p, V (&f)[N], int n, Load load) {
    unsigned long long t0 = 0;
    for (unsigned round = 0;; ++round) {
        unsigned most = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (j < n) f[j] = load(j);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (j < n) most = max(most, greatest(f[j]));
        }
        if (__all_sync(0xffffffffu, most != kEmpty)) return true;
        __nanosleep(20);
        if (round % 16 == 0) {
            const unsigned long long now = global_ns();
            if (round == 0) t0 = now;
            const bool late = now - t0 > p.wait_ns, stop = ld_word(p.sync + 1) != kEmpty;
            if (__any_sync(0xffffffffu, late)) {
                if ((threadIdx.x & 31) == 0) {
                    atomicExch(p.sync + 1, 0u);
                    atomicOr(p.status, kStatusTimeout);
                }
                return false;
            }
            if (__any_sync(0xffffffffu, stop)) return false;
        }
    }
}

// Gathers what the tile's carry is made of, by the whole CTA: each of the
// four warps up to four maps of the block's chunks before the tile's, then up
// to four maps of the span's blocks before that, the last one the state that
// the span starts from too. The caller synchronises, then reads the carry with
// look_carry.
static_assert(kWarps == 4 && kBlock == 16 && kLongSpan == 16 * kBlock, "four maps a warp");
__device__ __forceinline__ bool look_four(const GlrParams& p, float4 (&to)[4][32], const float4* maps, unsigned first, unsigned n, unsigned col) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (4 * warp >= n) return true;
    float4 f[4] = {kIdentity, kIdentity, kIdentity, kIdentity};
    const float4* from = maps + (size_t)((first + 4 * warp) * p.columns + col) * 32 + lane;
    const size_t step = (size_t)p.columns * 32;
    const bool ok = poll(p, f, (int)n - 4 * warp, [&](int j) { return ld_word4(from + j * step); });
    to[warp][lane] = compose(compose(f[0], f[1]), compose(f[2], f[3]));
    return ok;
}
__device__ __forceinline__ void look_chunks(const GlrParams& p, Look& look, unsigned k, unsigned col) {
    if (!look_four(p, look.four, p.maps, k / kBlock * kBlock, k % kBlock, col) && (threadIdx.x & 31) == 0) look.failed = 1;
}
template <int SPAN> __device__ __forceinline__ void look_blocks(const GlrParams& p, Look& look, unsigned k, unsigned col, const float* start) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned span = k / SPAN;
    bool ok = true;
    if (SPAN > kBlock) ok = look_four(p, look.blocks, p.blocks, span * (SPAN / kBlock), k % SPAN / kBlock, col);
    if (warp == kWarps - 1) {
        float2 f[1] = {start ? __ldg(reinterpret_cast<const float2*>(start)) : dup(0.f)};
        if (span) {
            const float2* from = p.states + (size_t)((span - 1) * p.columns + col) * 32 + lane;
            ok = poll(p, f, 1, [&](int) { return ld_word2(from); }) && ok;
        }
        look.state[lane] = f[0];
    }
    if (!ok && lane == 0) look.failed = 1;
}
template <int SPAN> __device__ __forceinline__ float2 look_carry(const Look& look, unsigned k) {
    const int lane = threadIdx.x & 31, n = (int)(k % kBlock), m = (int)(k % SPAN / kBlock);
    float2 h = look.state[lane];
#pragma unroll
    for (int w = 0; w < 4; ++w)
        if (4 * w < m) h = apply(look.blocks[w][lane], h);
#pragma unroll
    for (int w = 0; w < 4; ++w)
        if (4 * w < n) h = apply(look.four[w][lane], h);
    return h;
}
// Whether a tile ends a block (a span) that others follow.
__device__ __forceinline__ bool closes(const GlrParams& p, unsigned k, int chunks) {
    return k % chunks == chunks - 1 && k + 1 < p.chunks;
}
// By the warp that has the tile's map. A block's map needs no state, so blocks do not wait for one another; it is
// composed from look_chunks' maps, behind a barrier.
__device__ __forceinline__ void publish_map(const GlrParams& p, const Tile& t, float4 map) {
    if (t.k % kBlock != kBlock - 1 && t.k + 1 < p.chunks) st_words(p.maps + (size_t)t.tk * 32 + (threadIdx.x & 31), map);
}
__device__ __forceinline__ void publish_block(const GlrParams& p, const Look& look, const Tile& t, float4 map) {
    if (closes(p, t.k, kLongSpan)) return;  // (the state behind it says it all)
    const int lane = threadIdx.x & 31;
    const float4 before = compose(compose(look.four[0][lane], look.four[1][lane]), compose(look.four[2][lane], look.four[3][lane]));
    st_words(p.blocks + (size_t)(t.k / kBlock * p.columns + t.col) * 32 + lane, compose(before, map));
}
template <int SPAN> __device__ __forceinline__ void publish_state(const GlrParams& p, const Tile& t, float2 h) {
    st_words(p.states + (size_t)(t.k / SPAN * p.columns + t.col) * 32 + (threadIdx.x & 31), h);
}

// A warp's run past the sequence's end must be the identity map: its inputs
// there are set to x = dy = 0 and a closed recurrence gate (a = 1 exactly).
// One warp's run forwards from a zero state: h_j and the running product.
template <typename IO, bool SERIES, typename Load>
__device__ __forceinline__ float4 run_forward(float2 cs, Load load, float2 (&h)[kTok<IO>], float2 (&pr)[kTok<IO>]) {
    float2 hh = dup(0.f), pp = dup(1.f);
#pragma unroll
    for (int j = 0; j < kTok<IO>; ++j) {
        float2 x, rg, ig;
        load(j, x, rg, ig);
        const Decay d = decay<SERIES>(__fmul2_rn(cs, gate2<IO>(rg)));
        hh = __ffma2_rn(d.a, hh, __fmul2_rn(__fmul2_rn(sqrt2(input_power(d.w)), gate2<IO>(ig)), x));
        pp = __fmul2_rn(pp, d.a);
        h[j] = hh;
        pr[j] = pp;
    }
    return make_float4(pp.x, pp.y, hh.x, hh.y);
}
// The warp's outputs once its carry is known. Saved states: before tokens 0,
// 32, ... of the sequence. Returns 0 if they are finite, NaN if not: a state
// that is not finite stays so, so the run's last one tells.
template <typename IO>
__device__ __forceinline__ float finish_forward(const GlrParams& p, const Tile& t, const Lane<IO>& at, float2 carry,
                                                const float2 (&h)[kTok<IO>], const float2 (&pr)[kTok<IO>]) {
    constexpr int T = kTok<IO>;
    const int nt = at.tokens(p, t);
    if (nt == 0) return 0.f;
    if (p.ckpt && at.t0 % kCkptTokens == 0)
        *reinterpret_cast<float2*>(p.ckpt + t.saved + at.t0 / kCkptTokens * p.D + at.ch) = carry;
    IO* yp = static_cast<IO*>(p.y) + t.out + at.row_off;
    const unsigned D = (unsigned)p.D;
    float2 y;
    if (nt == T) {
#pragma unroll
        for (int j = 0; j < T; ++j, yp += D) st2<IO>(yp, y = __ffma2_rn(pr[j], carry, h[j]));
    } else {
#pragma unroll
        for (int j = 0; j < T; ++j, yp += D)
            if (j < nt) st2<IO>(yp, y = __ffma2_rn(pr[j], carry, h[j]));
    }
    if (p.end && t.chunk + 1 == p.chunks && at.t0 + nt == t.rows)
        *reinterpret_cast<float2*>(p.end + t.state + at.ch) = y;
    return __fmaf_rn(y.x, 0.f, y.y * 0.f);
}

// The warp's run in the backward, before the carries are known: the decays (w,
// held in one word each) and the gates (kept; the input gates in the series
// only), the run's map (P, H) forwards and V backwards.
template <typename IO, bool SERIES, typename Load>
__device__ __forceinline__ float4 run_backward(float2 cs, Load load, float2 (&w)[kTok<IO>], float2 (&r)[kTok<IO>],
                                               float2 (&i)[kTok<IO>], float2& back) {
    float2 hh = dup(0.f), pp = dup(1.f), vv = dup(0.f);
#pragma unroll
    for (int j = 0; j < kTok<IO>; ++j) {
        float2 x, rg, ig, dy;
        load(j, x, rg, ig, dy);
        r[j] = gate2<IO>(rg);
        const float2 iv = gate2<IO>(ig);
        if (SERIES) i[j] = iv;
        const Decay d = decay<SERIES>(__fmul2_rn(cs, r[j]));
        w[j] = hold<SERIES>(d);
        hh = __ffma2_rn(d.a, hh, __fmul2_rn(__fmul2_rn(sqrt2(input_power(d.w)), iv), x));
        pp = __fmul2_rn(pp, d.a);
        vv = __ffma2_rn(pp, dy, vv);  // V = sum_j (a_0 ... a_j) dy_j
    }
    back = vv;
    return make_float4(pp.x, pp.y, hh.x, hh.y);
}
// The warp's gradients once the state before its run and the gradient that
// comes in from behind it are known. Returns what its first token hands on;
// `sum` is the run's sum of dloga * r, which is not finite where a gradient
// or a state is not.
template <typename IO, bool SERIES, typename Load>
__device__ __forceinline__ float2 finish_backward(const GlrParams& p, const Tile& t, const Lane<IO>& at, float2 cs, float2 h, float2 v,
                                                  Load load, const float2 (&w)[kTok<IO>], const float2 (&r)[kTok<IO>],
                                                  const float2 (&i)[kTok<IO>], float2& sum) {
    float2 g[kTok<IO>];
#pragma unroll
    for (int j = kTok<IO> - 1; j >= 0; --j) {
        float2 x, ig, dy;
        load(j, x, ig, dy);
        g[j] = __fadd2_rn(dy, v);
        v = __fmul2_rn(held_decay<SERIES>(w[j]).a, g[j]);
    }
    const float2 ncs = pk(-cs.x, -cs.y);
    const unsigned D = (unsigned)p.D;
    const int nt = at.tokens(p, t);
    const int64_t base = t.out + at.row_off;
    IO *dxp = static_cast<IO*>(p.dx) + base, *drp = static_cast<IO*>(p.dr) + base, *dip = static_cast<IO*>(p.di) + base;
    sum = dup(0.f);
#pragma unroll
    for (int j = 0; j < kTok<IO>; ++j) {
        float2 x, ig, dy;
        load(j, x, ig, dy);
        const float2 iv = SERIES ? i[j] : gate2<IO>(ig);
        float2 wj = w[j];
        asm volatile("" : "+f"(wj.x), "+f"(wj.y));  // (a is taken from it again: kept from above it would cost registers)
        const Held d = held_decay<SERIES>(wj);
        const float2 a = d.a, m2 = SERIES ? input_power(wj) : __ffma2_rn(wj, __fadd2_rn(a, d.n), one_minus(d.n));
        // 1/m; where a = 1 the floor keeps it finite, and r or cs makes the product below 0
        const float2 inv = pk(rsqrt_approx(fmaxf(m2.x, 1e-36f)), rsqrt_approx(fmaxf(m2.y, 1e-36f)));
        const float2 ix = __fmul2_rn(iv, x), m = __fmul2_rn(m2, inv);
        const float2 dx = __fmul2_rn(g[j], __fmul2_rn(m, iv));
        const float2 di = __fmul2_rn(__fmul2_rn(dx, x), one_minus(iv));
        const float2 ah = __fmul2_rn(a, h);
        const float2 nai = __fmul2_rn(__fmul2_rn(a, inv), __fmul2_rn(a, dup(-1.f)));  // -a^2/m
        const float2 dlr = __fmul2_rn(__fmul2_rn(g[j], __ffma2_rn(nai, ix, ah)), r[j]);
        const float2 dr = __fmul2_rn(__fmul2_rn(dlr, ncs), one_minus(r[j]));
        h = __ffma2_rn(m, ix, ah);
        sum = __fadd2_rn(sum, dlr);
        if (j < nt) {
            st2<IO>(dxp, dx);
            st2<IO>(dip, di);
            st2<IO>(drp, dr);
        }
        dxp += D, dip += D, drp += D;
    }
    return v;
}
// A lane's two channels of a [B, D] (or of the saved states), where they exist.
__device__ __forceinline__ float2 ldg2(const float* p, bool live) {
    return p && live ? __ldg(reinterpret_cast<const float2*>(p)) : dup(0.f);
}
// ... of p.start, by a kernel that may write p.end in its place behind a barrier.
__device__ __forceinline__ float2 ld_start(const GlrParams& p, const Tile& t, int ch, bool live) {
    return p.start && live ? *reinterpret_cast<const float2*>(p.start + t.state + ch) : dup(0.f);
}

// ---------------------------------------------------------------- one chunk
// A sequence of at most one tile: one CTA a column, no carries, inputs
// straight into registers.
__device__ __forceinline__ float2 own_cs(const GlrParams& p, float (&cs)[kCols], int c0) {
    if (threadIdx.x < kCols) {
        const int64_t d = c0 + (int64_t)threadIdx.x;
        cs[threadIdx.x] = d < p.D ? p.c * softplus_full(__ldg(p.lam + d)) : 0.f;
    }
    __syncthreads();
    return *reinterpret_cast<const float2*>(&cs[2 * (threadIdx.x & 31)]);
}

// The run's inputs; past the end x = dy = 0 and the recurrence gate closed.
template <typename IO> struct Raw {
    typename Pair<IO>::T v[kTok<IO>];
    __device__ void load(const void* base, int64_t stride, int64_t L, const Tile& t, const Lane<IO>& at, int nt) {
        const IO* q = static_cast<const IO*>(base) + (t.b * L + at.t0) * stride + t.c0 + at.ch;
#pragma unroll
        for (int j = 0; j < kTok<IO>; ++j) v[j] = j < nt ? Pair<IO>::ld(q + j * stride) : Pair<IO>::none();
    }
    __device__ float2 f(int j) const { return Pair<IO>::f(v[j]); }
};
__device__ __forceinline__ float2 closed() { return dup(__int_as_float(0xff800000)); }

template <typename IO> __global__ void __launch_bounds__(kThreads) glr_fwd_short_kernel(const GlrParams p) {
    __shared__ float css[kCols];
    __shared__ float4 run[kWarps][32];
    begin_kernel();
    const Tile t = find_tile<IO>(p, blockIdx.x, false);
    const Lane<IO> at(p);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nt = at.tokens(p, t);
    Raw<IO> x, rg, ig;
    rg.load(p.r, p.sr, p.L, t, at, nt);
    ig.load(p.i, p.si, p.L, t, at, nt);
    x.load(p.x, p.sx, p.L, t, at, nt);
    float2 carry = ld_start(p, t, at.ch, at.live(p, t));
    const float2 cs = own_cs(p, css, t.c0);
    float2 h[kTok<IO>], pr[kTok<IO>];
    run[warp][lane] = run_forward<IO, false>(
        cs, [&](int j, float2& xv, float2& rv, float2& iv) { xv = x.f(j), rv = j < nt ? rg.f(j) : closed(), iv = ig.f(j); },
        h, pr);
    __syncthreads();
    for (int w = 0; w < warp; ++w) carry = apply(run[w][lane], carry);
    flag_nonfinite(p.status, finish_forward<IO>(p, t, at, carry, h, pr));
}

template <typename IO> __global__ void __launch_bounds__(kThreads) glr_bwd_short_kernel(const GlrParams p) {
    __shared__ float css[kCols];
    __shared__ TileMaps maps;
    __shared__ float2 red[kWarps][32];
    begin_kernel();
    const Tile t = find_tile<IO>(p, blockIdx.x, true);
    const Lane<IO> at(p);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nt = at.tokens(p, t);
    const bool live = at.live(p, t);
    Raw<IO> x, rg, ig, dy;
    rg.load(p.r, p.sr, p.L, t, at, nt);
    ig.load(p.i, p.si, p.L, t, at, nt);
    x.load(p.x, p.sx, p.L, t, at, nt);
    dy.load(p.dy, p.D, p.L, t, at, nt);
    float2 h = ldg2(p.ckpt + t.saved + at.ch, live), v = ld_start(p, t, at.ch, live);
    const float2 cs = own_cs(p, css, t.c0);
    float2 w[kTok<IO>], r[kTok<IO>], i[kTok<IO>], back, sum;
    maps.run[warp][lane] = run_backward<IO, false>(
        cs,
        [&](int j, float2& xv, float2& rv, float2& iv, float2& gv) {
            xv = x.f(j), rv = j < nt ? rg.f(j) : closed(), iv = ig.f(j), gv = dy.f(j);
        },
        w, r, i, back);
    maps.back[warp][lane] = back;
    __syncthreads();
    for (int u = 0; u < warp; ++u) h = apply(maps.run[u][lane], h);
    for (int u = kWarps - 1; u > warp; --u) {
        const float4 f = maps.run[u][lane];
        v = __ffma2_rn(pk(f.x, f.y), v, maps.back[u][lane]);
    }
    v = finish_backward<IO, false>(
        p, t, at, cs, h, v, [&](int j, float2& xv, float2& iv, float2& gv) { xv = x.f(j), iv = ig.f(j), gv = dy.f(j); }, w, r, i, sum);
    if (p.end && warp == 0 && live) *reinterpret_cast<float2*>(p.end + t.state + at.ch) = v;
    flag_nonfinite(p.status, live ? (sum.x + sum.y + v.x + v.y) * 0.f : 0.f);
    red[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && live) {
#pragma unroll
        for (int u = 1; u < kWarps; ++u) sum = __fadd2_rn(sum, red[u][lane]);
        *reinterpret_cast<float2*>(p.part + t.state + at.ch) = sum;
    }
}

// ---------------------------------------------------------------- many chunks
// Sets the published words to empty and c * softplus(lam) down for the tiles;
// and copies the start (held: nullable) where the end is written over it: a
// tile of the first span may read it after the last tile has written that.
__global__ void __launch_bounds__(256) glr_prepare_kernel(uint4* publish, int64_t n16, const float* __restrict__ lam,
                                                        float c, float* cs, int64_t D, const float* start, float* held, int64_t states) {
    begin_kernel();
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t j = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; j < n16; j += step)
        publish[j] = make_uint4(kEmpty, kEmpty, kEmpty, kEmpty);
    for (int64_t j = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; j < D; j += step)
        cs[j] = c * softplus_full(__ldg(lam + j));
    if (!held) return;
    for (int64_t j = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; j < states; j += step) held[j] = start[j];
}

// The ring of staged tiles of a CTA. A stage holds a tile's boxes of rgate,
// igate, x and (backward) dy, as [tokens][64 channels] each.
template <typename IO, int STREAMS, int STAGES> struct Ring {
    static constexpr int kStage = STREAMS * kBoxBytes<IO>;
    static constexpr int kSmem = STAGES * kStage + 128;
    uint64_t full[STAGES];
    Tile tile[STAGES];
};
__device__ __forceinline__ unsigned take_ticket(const GlrParams& p) { return atomicAdd(p.sync, 1u) + 1u; }

template <typename IO, int STREAMS>
__device__ __forceinline__ void issue_tile(const GlrParams& p, const GlrBoxes& bx, const Tile& t, char* to, uint64_t* full) {
    const int x = t.c0, y = (int)((int64_t)t.b * p.L + (int64_t)t.chunk * kChunk<IO>);
    const unsigned bar = smem_u32(full);
    mbar_expect_tx(bar, STREAMS * kBoxBytes<IO>);
    tma_load_2d(to, &bx.r, x, y, bar);
    tma_load_2d(to + kBoxBytes<IO>, &bx.i, x, y, bar);
    tma_load_2d(to + 2 * kBoxBytes<IO>, &bx.x, x, y, bar);
    if (STREAMS == 4) tma_load_2d(to + 3 * kBoxBytes<IO>, &bx.dy, x, y, bar);
}
// Rows of a staged tile past the sequence's end (they belong to the next
// batch row, or read as zero): each lane closes its own two channels.
template <typename IO, int STREAMS> __device__ __forceinline__ void close_rows(const Tile& t, const Lane<IO>& at, char* in) {
    const float2 shut = closed(), zero = dup(0.f);
#pragma unroll
    for (int j = 0; j < kTok<IO>; ++j) {
        if (at.t0 + j < t.rows) continue;
        IO* q = reinterpret_cast<IO*>(in + j * kCols * sizeof(IO));
        st2<IO>(q, shut);
#pragma unroll
        for (int u = 1; u < STREAMS; ++u) st2<IO>(q + u * kChunk<IO> * kCols, zero);
    }
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");  // before the stage's next copies
}

// A wait ran out: the CTA lets its copies in flight land (bounded) and stops.
template <int STAGES, typename R>
__device__ __forceinline__ void drain(const R& ring, unsigned from, unsigned to, unsigned total) {
    for (unsigned j = from; j <= to; ++j)
        if (ring.tile[j % STAGES].tk < total) mbar_wait_bounded(smem_u32(&ring.full[j % STAGES]), j / STAGES & 1);
}

template <typename IO, int STREAMS, int STAGES>
__device__ __forceinline__ void open_ring(const GlrParams& p, const GlrBoxes& bx, Ring<IO, STREAMS, STAGES>& ring, Look& look,
                                          char* buf, unsigned total, bool reverse) {
    if (threadIdx.x == 0) {
        look.failed = 0;
        for (int s = 0; s < STAGES; ++s) mbar_init(smem_u32(&ring.full[s]), 1);
        mbar_fence_init();
        for (int s = 0; s < STAGES; ++s) {
            const Tile t = find_tile<IO>(p, take_ticket(p), reverse);
            ring.tile[s] = t;
            if (t.tk < total)
                issue_tile<IO, STREAMS>(p, bx, t, buf + s * Ring<IO, STREAMS, STAGES>::kStage, &ring.full[s]);
        }
    }
    __syncthreads();
}

constexpr int kFwdStages = 2, kBwdStages = 2;
// CTAs an SM, by registers: 128 a thread and 168. (At three and two, 110 and
// 213 us instead of 102 and 203 for 4 x 4096 x 4096; at five and four the
// registers spill.)
constexpr int kFwdCtas = 4, kBwdCtas = 3;

template <typename IO, int SPAN>
__global__ void __launch_bounds__(kThreads, kFwdCtas) glr_fwd_kernel(const GlrParams p, const __grid_constant__ GlrBoxes bx) {
    constexpr int ST = kFwdStages, T = kTok<IO>;
    using R = Ring<IO, 3, ST>;
    extern __shared__ __align__(128) char raw[];
    char* buf = raw + ((128u - (smem_u32(raw) & 127u)) & 127u);
    __shared__ R ring;
    __shared__ float4 run[kWarps][32];
    __shared__ Look look;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned total = p.columns * p.chunks;
    const Lane<IO> at(p);
    begin_kernel();
    open_ring(p, bx, ring, look, buf, total, false);
    float acc = 0.f;
    for (unsigned it = 0;; ++it) {
        const int s = it % ST;
        const Tile t = ring.tile[s];
        if (t.tk >= total) break;
        unsigned next = 0;
        if (threadIdx.x == 0) next = take_ticket(p);
        const float2 cs = ldg2(p.cs + t.c0 + at.ch, at.live(p, t));
        char* in = buf + s * R::kStage + (at.t0 * kCols + at.ch) * sizeof(IO);
        if (!mbar_wait_bounded(smem_u32(&ring.full[s]), it / ST & 1))
            look.failed = 1, atomicOr(p.status, kStatusTimeout), atomicExch(p.sync + 1, 0u);
        if (t.rows < kChunk<IO>) close_rows<IO, 3>(t, at, in);
        const auto load = [&](int j, float2& x, float2& rg, float2& ig) {
            const char* q = in + j * kCols * sizeof(IO);
            rg = Pair<IO>::f(Pair<IO>::lds(q));
            ig = Pair<IO>::f(Pair<IO>::lds(q + kBoxBytes<IO>));
            x = Pair<IO>::f(Pair<IO>::lds(q + 2 * kBoxBytes<IO>));
        };
        float2 h[T], pr[T];
        const float4 mine = all_series(cs) ? run_forward<IO, true>(cs, load, h, pr) : run_forward<IO, false>(cs, load, h, pr);
        run[warp][lane] = mine;
        __syncthreads();
        const bool failed = look.failed;
        if (threadIdx.x == 0) {  // the stage has been read: its next tile
            const Tile u = find_tile<IO>(p, failed ? total : next, false);
            if (failed) mbar_wait_bounded(smem_u32(&ring.full[s]), it / ST & 1);
            ring.tile[s] = u;
            if (u.tk < total) issue_tile<IO, 3>(p, bx, u, buf + s * R::kStage, &ring.full[s]);
        }
        const bool withhold = p.fault_chunk1 == (int64_t)t.chunk + 1;
        float4 before = kIdentity;  // the tile's tokens before the warp's
#pragma unroll
        for (int w = 0; w < kWarps - 1; ++w)
            if (w < warp) before = compose(before, run[w][lane]);
        const float4 whole = compose(before, mine);  // the last warp's: the tile's map
        if (warp == kWarps - 1 && !withhold) publish_map(p, t, whole);
        if (!failed) look_chunks(p, look, t.k, t.col);
        if (SPAN > kBlock && closes(p, t.k, kBlock)) {
            __syncthreads();
            if (warp == kWarps - 1 && !withhold) publish_block(p, look, t, whole);
        }
        if (!failed) look_blocks<SPAN>(p, look, t.k, t.col, p.start && at.live(p, t) ? p.start + t.state + at.ch : nullptr);
        __syncthreads();
        if (look.failed) {
            drain<ST>(ring, it + 1, it + ST, total);
            return;
        }
        const float2 carry = look_carry<SPAN>(look, t.k);
        if (warp == kWarps - 1 && closes(p, t.k, SPAN) && !withhold) publish_state<SPAN>(p, t, apply(whole, carry));
        acc += finish_forward<IO>(p, t, at, apply(before, carry), h, pr);
    }
    flag_nonfinite(p.status, acc);
}

template <typename IO, int SPAN>
__global__ void __launch_bounds__(kThreads, kBwdCtas) glr_bwd_kernel(const GlrParams p, const __grid_constant__ GlrBoxes bx) {
    constexpr int ST = kBwdStages, T = kTok<IO>;
    using R = Ring<IO, 4, ST>;
    extern __shared__ __align__(128) char raw[];
    char* buf = raw + ((128u - (smem_u32(raw) & 127u)) & 127u);
    __shared__ R ring;
    __shared__ TileMaps run;
    __shared__ float2 red[kWarps][32];
    __shared__ Look look;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned total = p.columns * p.chunks;
    const Lane<IO> at(p);
    begin_kernel();
    open_ring(p, bx, ring, look, buf, total, true);
    float acc = 0.f;
    for (unsigned it = 0;; ++it) {
        const int s = it % ST;
        const Tile t = ring.tile[s];
        if (t.tk >= total) break;
        unsigned next = 0;
        if (threadIdx.x == 0) next = take_ticket(p);
        const bool live = at.live(p, t);
        const float2 cs = ldg2(p.cs + t.c0 + at.ch, live);
        float2 h = ldg2(p.ckpt + t.saved + at.ch, live);
        char* in = buf + s * R::kStage + (at.t0 * kCols + at.ch) * sizeof(IO);
        if (!mbar_wait_bounded(smem_u32(&ring.full[s]), it / ST & 1))
            look.failed = 1, atomicOr(p.status, kStatusTimeout), atomicExch(p.sync + 1, 0u);
        if (t.rows < kChunk<IO>) close_rows<IO, 4>(t, at, in);
        const auto load = [&](int j, float2& x, float2& rg, float2& ig, float2& dy) {
            const char* q = in + j * kCols * sizeof(IO);
            rg = Pair<IO>::f(Pair<IO>::lds(q));
            ig = Pair<IO>::f(Pair<IO>::lds(q + kBoxBytes<IO>));
            x = Pair<IO>::f(Pair<IO>::lds(q + 2 * kBoxBytes<IO>));
            dy = Pair<IO>::f(Pair<IO>::lds(q + 3 * kBoxBytes<IO>));
        };
        float2 sum;
        // A body for each way to the decays (the warps of a CTA have the same channels, and so take the same one): with
        // one for both, or with the input gates kept outside the series too, registers spill (4 x 4096 x 4096 bf16:
        // 200 us in the series and 223 outside, otherwise 250 to 320).
        auto work = [&](auto way) {
            constexpr bool SERIES = decltype(way)::value;
            float2 w[T], r[T], i[T], back;
            const float4 mine = run_backward<IO, SERIES>(cs, load, w, r, i, back);
            run.run[warp][lane] = mine;
            run.back[warp][lane] = back;
            __syncthreads();
            const bool failed = look.failed;
            // the tile's tokens behind the warp's, composed from the last one on, and the state before the warp's
            float4 behind = kIdentity;
#pragma unroll
            for (int u = kWarps - 1; u > 0; --u) {
                if (u > warp) {
                    const float4 f = run.run[u][lane];
                    const float2 v = run.back[u][lane];
                    behind = compose(behind, make_float4(f.x, f.y, v.x, v.y));
                }
            }
            const float4 whole = compose(behind, make_float4(mine.x, mine.y, back.x, back.y));  // warp 0: the tile's map
            const bool publishes = warp == 0 && p.fault_chunk1 != (int64_t)t.chunk + 1;
            if (publishes) publish_map(p, t, whole);
#pragma unroll
            for (int u = 0; u < kWarps - 1; ++u)
                if (u < warp) h = apply(run.run[u][lane], h);
            if (!failed) look_chunks(p, look, t.k, t.col);
            if (SPAN > kBlock && closes(p, t.k, kBlock)) {
                __syncthreads();
                if (publishes) publish_block(p, look, t, whole);
            }
            if (!failed) look_blocks<SPAN>(p, look, t.k, t.col, p.start && live ? p.start + t.state + at.ch : nullptr);
            __syncthreads();
            if (look.failed) {
                drain<ST>(ring, it, it + ST - 1, total);
                return false;
            }
            const float2 carry = look_carry<SPAN>(look, t.k);
            if (publishes && closes(p, t.k, SPAN)) publish_state<SPAN>(p, t, apply(whole, carry));
            const auto again = [&](int j, float2& x, float2& ig, float2& dy) {
                const char* q = in + j * kCols * sizeof(IO);
                ig = Pair<IO>::f(Pair<IO>::lds(q + kBoxBytes<IO>));
                x = Pair<IO>::f(Pair<IO>::lds(q + 2 * kBoxBytes<IO>));
                dy = Pair<IO>::f(Pair<IO>::lds(q + 3 * kBoxBytes<IO>));
            };
            const float2 v = finish_backward<IO, SERIES>(p, t, at, cs, h, apply(behind, carry), again, w, r, i, sum);
            acc += live ? (sum.x + sum.y + v.x + v.y) * 0.f : 0.f;
            if (p.end && t.chunk == 0 && warp == 0 && live) *reinterpret_cast<float2*>(p.end + t.state + at.ch) = v;
            return true;
        };
        if (!(all_series(cs) ? work(std::true_type{}) : work(std::false_type{}))) return;
        red[warp][lane] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {  // the stage has been read for the last time: its next tile
            const Tile u = find_tile<IO>(p, next, true);
            ring.tile[s] = u;
            if (next < total) issue_tile<IO, 4>(p, bx, u, buf + s * R::kStage, &ring.full[s]);
        }
        // the tile's sum of dloga * r, in warp order (red is written again behind the next tile's barriers)
        if (warp == 1 && live) {
            sum = red[0][lane];
#pragma unroll
            for (int u = 1; u < kWarps; ++u) sum = __fadd2_rn(sum, red[u][lane]);
            *reinterpret_cast<float2*>(p.part + ((int64_t)t.b * p.chunks + t.chunk) * p.D + t.c0 + at.ch) = sum;
        }
    }
    flag_nonfinite(p.status, acc);
}

// dlam[d] = -c sigmoid(lam[d]) * sum of the rows of part: a CTA takes 32
// channels, its eight warps the rows in turn, folded in warp order.
__global__ void __launch_bounds__(kRedThreads) glr_dlam_kernel(const float* __restrict__ part, int64_t rows, int64_t D,
                                                             const float* __restrict__ lam, float c, float* dlam) {
    __shared__ float red[8][32];
    begin_kernel();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t d = (int64_t)blockIdx.x * 32 + lane;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (d < D) {
        int64_t r = warp;
        for (; r + 24 < rows; r += 32) {
#pragma unroll
            for (int u = 0; u < 4; ++u) s[u] += __ldg(part + (r + 8 * u) * D + d);
        }
        for (; r < rows; r += 8) s[0] += __ldg(part + r * D + d);
    }
    red[warp][lane] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    if (warp == 0 && d < D) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t += red[w][lane];
        dlam[d] = -c * sigmoid<false>(lam[d]) * t;
    }
}

// One token for every channel: a thread takes two neighbouring channels of
// one batch row.
template <typename IO>
__global__ void __launch_bounds__(128) glr_step_kernel(int64_t B, int64_t D, int64_t sx, int64_t sr, int64_t si, float c,
                                                       const IO* __restrict__ x, const IO* __restrict__ rg,
                                                       const IO* __restrict__ ig, const float* __restrict__ lam,
                                                       float* state, IO* y, unsigned* status) {
    const int64_t half = D / 2, idx = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    begin_kernel();
    float acc = 0.f;
    if (idx < B * half) {
        const int64_t b = idx / half, d = 2 * (idx - b * half);
        using P2 = Pair<IO>;
        const float2 xv = P2::f(P2::ld(x + b * sx + d)), rv = P2::f(P2::ld(rg + b * sr + d)),
                     iv = P2::f(P2::ld(ig + b * si + d));
        float2* hp = reinterpret_cast<float2*>(state + b * D + d);
        const float2 h0 = *hp, lv = __ldg(reinterpret_cast<const float2*>(lam + d));
        const float2 cs = pk(c * softplus_full(lv.x), c * softplus_full(lv.y));
        const Decay f = decay<false>(__fmul2_rn(cs, gate2<IO>(rv)));
        const float2 u = __fmul2_rn(__fmul2_rn(sqrt2(input_power(f.w)), gate2<IO>(iv)), xv);
        const float2 h = __ffma2_rn(f.a, h0, u);
        *hp = h;
        st2<IO>(y + b * D + d, h);
        acc = __fmaf_rn(h.x, 0.f, h.y * 0.f);
    }
    flag_nonfinite(status, acc);
}

// A missing carry armed for a thread's next call (the test hook): taken by that call, whatever becomes of it.
struct WaitFault {
    int64_t chunk1 = 0;
    unsigned long long wait_ns = 0;
};
thread_local WaitFault g_fault;
WaitFault take_fault() {
    const WaitFault f = g_fault;
    g_fault = WaitFault{};
    return f;
}
void set_fault(GlrParams& p, const WaitFault& f) {
    p.fault_chunk1 = f.chunk1;
    if (f.wait_ns) p.wait_ns = f.wait_ns;
}

bool off16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

int check_stride(int64_t s, int64_t D, int io) {
    if (s == 0) return SSM_OK;
    if (s < D || s > (int64_t(1) << 32)) return SSM_ERR_INVALID_ARG;
    return s * (io == SSM_BF16 ? 2 : 4) % 16 == 0 ? SSM_OK : SSM_ERR_ALIGNMENT;
}

int check_common(int64_t B, int64_t D, int io, float c, int64_t sx, int64_t sr, int64_t si) {
    if (B < 0 || D < 0 || B > (int64_t(1) << 31) || D > (int64_t(1) << 31)) return SSM_ERR_INVALID_ARG;
    if (io != SSM_F32 && io != SSM_BF16) return SSM_ERR_UNSUPPORTED;
    if (!std::isfinite(c) || c <= 0.f) return SSM_ERR_INVALID_ARG;
    if (D % 8 != 0) return SSM_ERR_ALIGNMENT;
    for (int64_t s : {sx, sr, si}) {
        const int rc = check_stride(s, D, io);
        if (rc != SSM_OK) return rc;
    }
    return SSM_OK;
}

int check_seq(const ssm_glr_args* a) {
    if (!a) return SSM_ERR_INVALID_ARG;
    int rc = check_common(a->B, a->D, a->io_dtype, a->c, a->x_stride, a->r_stride, a->i_stride);
    if (rc != SSM_OK) return rc;
    if (a->L < 0 || a->L > (int64_t(1) << 40)) return SSM_ERR_INVALID_ARG;
    if (a->L > 0 && a->B > (int64_t(0x7fffffff) - 64) / a->L) return SSM_ERR_UNSUPPORTED;  // rows of the copies
    const int64_t chunks = (a->L + kChunk<float> - 1) / kChunk<float>, per_row = (a->D + kCols - 1) / kCols;
    // (each product is bounded before the next factor, so none passes 64 bits)
    if (chunks > 0 && per_row > 0 && a->B > 0 &&
        (chunks > 0x7fffffff / per_row || chunks * per_row > 0x7fffffff / a->B))
        return SSM_ERR_UNSUPPORTED;
    const bool work = a->B > 0 && a->L > 0 && a->D > 0;
    if (work && (!a->x || !a->rgate || !a->igate || !a->lam)) return SSM_ERR_INVALID_ARG;
    for (const void* p : {a->x, a->rgate, a->igate, (const void*)a->lam, (const void*)a->h0, (const void*)a->y,
                          (const void*)a->h_last, (const void*)a->ckpt, (const void*)a->workspace})
        if (off16(p)) return SSM_ERR_ALIGNMENT;
    if (!a->workspace || a->workspace_bytes < ssm_glr_workspace_bytes(a->B, a->L, a->D)) return SSM_ERR_WORKSPACE;
    return SSM_OK;
}

GlrParams base_params(const ssm_glr_args& a) {
    GlrParams p{};
    const int chunk = chunk_tokens(a.io_dtype);
    const GlrWs w = glr_ws(a.B, a.L, a.D, chunk);
    char* ws = static_cast<char*>(a.workspace);
    p.B = a.B; p.L = a.L; p.D = a.D;
    p.sx = a.x_stride ? a.x_stride : a.D;
    p.sr = a.r_stride ? a.r_stride : a.D;
    p.si = a.i_stride ? a.i_stride : a.D;
    p.c = a.c; p.x = a.x; p.r = a.rgate; p.i = a.igate; p.lam = a.lam; p.ckpt = a.ckpt;
    p.status = reinterpret_cast<unsigned*>(ws);
    p.sync = reinterpret_cast<unsigned*>(ws + w.sync);
    p.maps = reinterpret_cast<float4*>(ws + w.maps);
    p.blocks = reinterpret_cast<float4*>(ws + w.blocks);
    p.states = reinterpret_cast<float2*>(ws + w.states);
    p.cs = reinterpret_cast<float*>(ws + w.cs);
    p.held = reinterpret_cast<float*>(ws + w.held);
    p.part = reinterpret_cast<float*>(ws + w.part);
    p.chunks = (unsigned)((a.L + chunk - 1) / chunk);
    p.per_row = (unsigned)((a.D + kCols - 1) / kCols);
    p.columns = (unsigned)a.B * p.per_row;
    p.wait_ns = kWaitNs;
    return p;
}


// One kernel for the forward or backward of a sequence of more than one
// chunk: as many CTAs as are resident at once (they take tiles by ticket).
template <auto KERN, int SMEM> int launch_tiles(const GlrParams& p, const GlrBoxes& bx, cudaStream_t s) {
    static unsigned long long mask = 0;
    static int per_sm[64] = {};
    if (!ensure_smem(KERN, SMEM, mask)) return -1;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -1;
    int& n = per_sm[dev & 63];
    if (n == 0 && (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, KERN, kThreads, SMEM) != cudaSuccess || n < 1)) {
        n = 0;
        return -1;
    }
    const int64_t tiles = (int64_t)p.columns * p.chunks, slots = (int64_t)n * sm_count();
    return launch_next(KERN, dim3((unsigned)(tiles < slots ? tiles : slots)), kThreads, SMEM, s, p, bx);
}

template <typename IO> bool encode_boxes(const GlrParams& p, bool bwd, GlrBoxes& bx) {
    const CUtensorMapDataType t = sizeof(IO) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
    auto enc = [&](CUtensorMap* m, const void* base, int64_t stride) {
        return encode_2d(m, t, base, p.D, p.B * p.L, stride * (int64_t)sizeof(IO), kCols, kChunk<IO>, CU_TENSOR_MAP_SWIZZLE_NONE);
    };
    return enc(&bx.x, p.x, p.sx) && enc(&bx.r, p.r, p.sr) && enc(&bx.i, p.i, p.si) && (!bwd || enc(&bx.dy, p.dy, p.D));
}

template <typename IO> int launch_seq(bool bwd, GlrParams p, size_t publish_bytes, cudaStream_t s) {
    if (p.chunks == 1) {
        return launch_next(bwd ? glr_bwd_short_kernel<IO> : glr_fwd_short_kernel<IO>, dim3(p.columns), kThreads, 0, s, p);
    }
    GlrBoxes bx;
    if (!encode_boxes<IO>(p, bwd, bx)) return -1;
    const int64_t n16 = (int64_t)(publish_bytes / 16), want = (n16 + 1023) / 1024 + (p.D + 255) / 256;
    const int64_t cap = 8 * (int64_t)sm_count();
    const bool in_place = p.start && p.start == p.end;
    if (launch_next(glr_prepare_kernel, dim3((unsigned)(want < cap ? want : cap)), 256, 0, s, reinterpret_cast<uint4*>(p.sync), n16,
                    p.lam, p.c, p.cs, p.D, p.start, in_place ? p.held : nullptr, p.B * p.D) < 0)
        return -1;
    if (in_place) p.start = p.held;
    const bool few = p.columns <= kFewColumns && p.chunks > kBlock;
    constexpr int kFwdSmem = Ring<IO, 3, kFwdStages>::kSmem, kBwdSmem = Ring<IO, 4, kBwdStages>::kSmem;
    int r;
    if (bwd)
        r = few ? launch_tiles<glr_bwd_kernel<IO, kLongSpan>, kBwdSmem>(p, bx, s) : launch_tiles<glr_bwd_kernel<IO, kBlock>, kBwdSmem>(p, bx, s);
    else
        r = few ? launch_tiles<glr_fwd_kernel<IO, kLongSpan>, kFwdSmem>(p, bx, s) : launch_tiles<glr_fwd_kernel<IO, kBlock>, kFwdSmem>(p, bx, s);
    return r < 0 ? -1 : 1 + r;
}

// [B, D] fp32 state handed through (or zeroed) when there are no tokens.
int copy_state(float* out, const float* in, int64_t B, int64_t D, cudaStream_t s) {
    if (!out || B == 0 || D == 0 || out == in) return SSM_OK;
    const size_t bytes = (size_t)B * D * sizeof(float);
    const cudaError_t e = in ? cudaMemcpyAsync(out, in, bytes, cudaMemcpyDeviceToDevice, s)
                             : cudaMemsetAsync(out, 0, bytes, s);
    return e == cudaSuccess ? SSM_OK : SSM_ERR_CUDA;
}

}  // namespace
}  // namespace ssm

extern "C" {

size_t ssm_glr_workspace_bytes(int64_t B, int64_t L, int64_t D) {
    if (B <= 0 || L <= 0 || D <= 0) return 256;
    return ssm::glr_ws(B, L, D, ssm::kChunk<float>).total;
}

int64_t ssm_glr_ckpt_elems(int64_t B, int64_t L, int64_t D) {
    if (B < 0 || L < 0 || D < 0) return 0;
    return B * ((L + ssm::kCkptTokens - 1) / ssm::kCkptTokens) * D;
}

int ssm_glr_debug_arm_wait_fault(int64_t chunk, uint64_t wait_ns) {
    if (wait_ns > 10000000000ull) return SSM_ERR_INVALID_ARG;
    ssm::g_fault = chunk < 0 ? ssm::WaitFault{} : ssm::WaitFault{chunk + 1, wait_ns};
    return SSM_OK;
}

int ssm_glr_fwd(const ssm_glr_args* a, void* stream) {
    ssm::reset_launches();
    const ssm::WaitFault fault = ssm::take_fault();
    int rc = ssm::check_seq(a);
    if (rc != SSM_OK) return rc;
    cudaStream_t s = (cudaStream_t)stream;
    if (a->B == 0 || a->D == 0 || a->L == 0) return ssm::copy_state(a->h_last, a->h0, a->B, a->D, s);
    if (!a->y) return SSM_ERR_INVALID_ARG;
    ssm::GlrParams p = ssm::base_params(*a);
    p.start = a->h0; p.end = a->h_last; p.y = a->y;
    ssm::set_fault(p, fault);
    const size_t pub = ssm::glr_ws(a->B, a->L, a->D, ssm::chunk_tokens(a->io_dtype)).publish_bytes;
    return ssm::count_launches(a->io_dtype == SSM_BF16 ? ssm::launch_seq<__nv_bfloat16>(false, p, pub, s)
                                                       : ssm::launch_seq<float>(false, p, pub, s));
}

int ssm_glr_bwd(const ssm_glr_bwd_args* a, void* stream) {
    ssm::reset_launches();
    const ssm::WaitFault fault = ssm::take_fault();
    if (!a) return SSM_ERR_INVALID_ARG;
    const ssm_glr_args& f = a->f;
    int rc = ssm::check_seq(&f);
    if (rc != SSM_OK) return rc;
    const bool work = f.B > 0 && f.L > 0 && f.D > 0;
    if (work && (!f.ckpt || !a->dy || !a->dx || !a->drgate || !a->digate)) return SSM_ERR_INVALID_ARG;
    if (f.D > 0 && !a->dlam) return SSM_ERR_INVALID_ARG;
    for (const void* q : {a->dy, (const void*)a->dh_last, (const void*)a->dx, (const void*)a->drgate,
                          (const void*)a->digate, (const void*)a->dlam, (const void*)a->dh0})
        if (ssm::off16(q)) return SSM_ERR_ALIGNMENT;
    cudaStream_t s = (cudaStream_t)stream;
    if (!work) {
        if (f.D > 0 && cudaMemsetAsync(a->dlam, 0, (size_t)f.D * sizeof(float), s) != cudaSuccess) return SSM_ERR_CUDA;
        return ssm::copy_state(a->dh0, a->dh_last, f.B, f.D, s);
    }
    ssm::GlrParams p = ssm::base_params(f);
    p.start = a->dh_last; p.end = a->dh0;
    p.dy = a->dy; p.dx = a->dx; p.dr = a->drgate; p.di = a->digate;
    ssm::set_fault(p, fault);
    const size_t pub = ssm::glr_ws(f.B, f.L, f.D, ssm::chunk_tokens(f.io_dtype)).publish_bytes;
    rc = ssm::count_launches(f.io_dtype == SSM_BF16 ? ssm::launch_seq<__nv_bfloat16>(true, p, pub, s)
                                                    : ssm::launch_seq<float>(true, p, pub, s));
    if (rc != SSM_OK) return rc;
    return ssm::count_launches(ssm::launch_next(ssm::glr_dlam_kernel, dim3((unsigned)((f.D + 31) / 32)), ssm::kRedThreads, 0, s,
                                                static_cast<const float*>(p.part), f.B * (int64_t)p.chunks, f.D, f.lam, f.c,
                                                a->dlam));
}

int ssm_glr_step(const ssm_glr_step_args* a, void* stream) {
    ssm::reset_launches();
    if (!a) return SSM_ERR_INVALID_ARG;
    int rc = ssm::check_common(a->B, a->D, a->io_dtype, a->c, a->x_stride, a->r_stride, a->i_stride);
    if (rc != SSM_OK) return rc;
    const bool work = a->B > 0 && a->D > 0;
    if (work && (!a->x_t || !a->rgate_t || !a->igate_t || !a->lam || !a->state || !a->y_t)) return SSM_ERR_INVALID_ARG;
    for (const void* q : {a->x_t, a->rgate_t, a->igate_t, (const void*)a->lam, (const void*)a->state,
                          (const void*)a->y_t, (const void*)a->workspace})
        if (ssm::off16(q)) return SSM_ERR_ALIGNMENT;
    if (!work) return SSM_OK;
    const int64_t half = a->D / 2;
    if (a->B > int64_t(0x7fffffff) * 128 / half) return SSM_ERR_UNSUPPORTED;
    const unsigned grid = (unsigned)((a->B * half + 127) / 128);
    const int64_t sx = a->x_stride ? a->x_stride : a->D, sr = a->r_stride ? a->r_stride : a->D,
                  si = a->i_stride ? a->i_stride : a->D;
    cudaStream_t s = (cudaStream_t)stream;
    auto go = [&](auto tag) {
        using IO = decltype(tag);
        return ssm::launch_next(ssm::glr_step_kernel<IO>, dim3(grid), 128, 0, s, a->B, a->D, sx, sr, si, a->c,
                                static_cast<const IO*>(a->x_t), static_cast<const IO*>(a->rgate_t), static_cast<const IO*>(a->igate_t),
                                a->lam, a->state, static_cast<IO*>(a->y_t), static_cast<unsigned*>(a->workspace));
    };
    return ssm::count_launches(a->io_dtype == SSM_BF16 ? go(__nv_bfloat16{}) : go(float{}));
}

}  // extern "C"
