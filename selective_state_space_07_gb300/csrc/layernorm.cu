// Layer norm on sm_103a: forward, and backward with the sums for weight and
// bias (include/layernorm.h holds the formulas and the boundary).
//
// Both passes read each row once and are bound by HBM. A row belongs to a
// group of T threads (4 lanes of a warp up to 512 threads), which holds it in
// registers: NC chunks of eight elements a thread, so that the mean, the
// centred sum of squares and the output come from one read. Groups walk the
// rows in steps of the grid.
//
// At two bytes an element the instructions count as much as the bytes: the
// arithmetic is in pairs (f32x2), and a lane takes up to 64 elements of a row
// in the forward, so that a row's two sums, ten steps of a warp each, cost
// little beside them; the backward, which keeps column sums besides, takes up
// to 32, and reads both rows twice from shared memory.
//
// Groups of a warp or more have a ring in shared memory that bulk copies fill,
// a row (the backward: of x and of dy) each, several rows ahead. The copies
// take whole 16-byte words: of a row that starts or ends elsewhere (an odd
// width, an odd slice) with a few of its neighbours' bytes, except where those
// would lie outside the tensor; such rows, the first and last, are read
// directly. Rows of at most 128 elements (in the forward 256) go through
// registers, one ahead, with 4 or 16 lanes each (262144 x 128 bf16: 28 us
// forward and 55 backward; with a warp and a ring 66 and 84).
//
// Column sums leave once a CTA: its groups add theirs in shared memory, in
// group order, and a second kernel adds the CTAs', in CTA order.
//
// Measured, in percent of the HBM copy rate: 65536 x 2048 bf16 forward 95 us
// (83%), backward 135 (88%); 16384 x 2048 24 (83%) and 39 (76%); 65537 x 1023
// fp32 93 (86%) and 129 (92%), bf16 51 (77%) and 109 (55%: single elements,
// instructions); 65536 x 512 33 (60%) and 41 (72%); 4096 x 16384 58 (69%) and
// 98 (61%: one row an SM at a time), 2048 x 16384 fp32 59 (67%) and 98 (61%).
// Wider rows are read from L2 again (4096 x 16384 bf16 that way: 153 and 214).
#include <cmath>

#include "../../include/layernorm.h"
#include "rows.cuh"
#include "ssm_common.cuh"
#include "ssm_internal.h"

namespace ssm {
namespace {

struct LnParams {
    int64_t rows, D, xs;
    float eps, inv_d;
    const void *x, *dy;
    const float *w, *b;
    float *mean, *rstd;
    void *y, *dx;
    float* part;  // backward: [CTAs, 2, D], nullable
    int stages, stage_bytes;  // of a group's ring: rows, and bytes of one row of one tensor
    unsigned* status;
};

template <Layout L, int T, int NC>
__device__ __forceinline__ void load_columns(const float* p, float none, int64_t D, int t, float (&f)[NC][8]) {
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t c = column<L, T>((int64_t)k * 8 * T, t, i);
            f[k][i] = p && c < D ? __ldg(p + c) : none;
        }
}

// Sums of N values over a group of T threads, the same on every one.
template <int T, int N, int R> struct GroupSum {
    static constexpr int kWarpsPer = T > 32 ? T / 32 : 1;
    float part[2][R][kWarpsPer][N];  // in turn, so that one barrier a sum is enough
};
template <int T, int N, int R>
__device__ __forceinline__ void group_sum(GroupSum<T, N, R>& sh, int turn, int group, int t, float (&v)[N]) {
#pragma unroll
    for (int o = (T < 32 ? T : 32) / 2; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if constexpr (T > 32) {
        constexpr int W = T / 32;
        if ((t & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) sh.part[turn & 1][group][t >> 5][i] = v[i];
        asm volatile("bar.sync %0, %1;\n" ::"r"(group + 1), "n"(T) : "memory");
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) s += sh.part[turn & 1][group][w][i];
            v[i] = s;
        }
    }
}

template <typename IO, Layout L, int T, int NC, int R>
__global__ void __launch_bounds__(T* R) ln_fwd_kernel(const LnParams p) {
    __shared__ GroupSum<T, 1, R> sh;
    begin_kernel();
    const int group = threadIdx.x / T, t = threadIdx.x % T;
    float w[NC][8], b[NC][8];
    load_columns<L, T, NC>(p.w, 1.f, p.D, t, w);
    load_columns<L, T, NC>(p.b, 0.f, p.D, t, b);
    const int64_t step = (int64_t)gridDim.x * R;
    using C = Chunk<IO, L, T>;
    C in[NC];
    int64_t row = (int64_t)blockIdx.x * R + group;
    const int64_t base = (int64_t)blockIdx.x * R;  // the CTA's first row: its groups make as many turns
    auto fetch = [&](int64_t r) {
        const IO* from = static_cast<const IO*>(p.x) + r * p.xs;
        const int64_t D = r < p.rows ? p.D : 0;  // past the last row nothing is read
#pragma unroll
        for (int k = 0; k < NC; ++k) in[k].load(from, D, (int64_t)k * 8 * T, t);
    };
    fetch(row);
    float bad = 0.f;
    int turn = 0;
    for (int64_t r0 = base; r0 < p.rows; r0 += step, row += step) {
        float v[NC][8];
#pragma unroll
        for (int k = 0; k < NC; ++k) in[k].get(v[k]);
        fetch(row + step);
        float s[1] = {0.f};
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) s[0] += v[k][i];
        group_sum<T, 1, R>(sh, turn++, group, t, s);
        const float mean = s[0] * p.inv_d;
        float q[1] = {0.f};
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[k][i] -= mean;
                if (column<L, T>((int64_t)k * 8 * T, t, i) >= p.D) v[k][i] = 0.f;
                q[0] = __fmaf_rn(v[k][i], v[k][i], q[0]);
            }
        group_sum<T, 1, R>(sh, turn++, group, t, q);
        const float rstd = 1.0f / sqrtf(__fmaf_rn(q[0], p.inv_d, p.eps));
        if (row < p.rows) {
            if (t == 0 && p.mean) p.mean[row] = mean;
            if (t == 0 && p.rstd) p.rstd[row] = rstd;
            IO* to = static_cast<IO*>(p.y) + row * p.D;
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    y[i] = __fmaf_rn(v[k][i] * rstd, w[k][i], b[k][i]);
                    bad = __fmaf_rn(y[i], 0.f, bad);
                }
                C::store(to, p.D, (int64_t)k * 8 * T, t, y);
            }
        }
    }
    flag_nonfinite(p.status, bad);
}

// The CTA's column sums, groups that share a warp first, then group after
// group in shared memory (sums, [2][D]), to its place in p.part.
template <Layout L, int T, int NC, int R>
__device__ __forceinline__ void leave_sums(const LnParams& p, float* sums, float (&dw)[NC][8], float (&db)[NC][8]) {
    const int t = threadIdx.x % T;
    if constexpr (T < 32) {
#pragma unroll
        for (int o = 16; o >= T; o >>= 1)
#pragma unroll
            for (int k = 0; k < NC; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dw[k][i] += __shfl_xor_sync(0xffffffffu, dw[k][i], o);
                    db[k][i] += __shfl_xor_sync(0xffffffffu, db[k][i], o);
                }
    }
    constexpr int TT = T < 32 ? 32 : T, RR = T * R / TT;  // threads that add together, and how many sets of them
    for (int u = 0; u < RR; ++u) {
        if ((int)threadIdx.x / TT == u && (int)threadIdx.x % TT < T) {
#pragma unroll
            for (int k = 0; k < NC; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int64_t c = column<L, T>((int64_t)k * 8 * T, t, i);
                    if (c < p.D) {
                        sums[c] = u ? sums[c] + dw[k][i] : dw[k][i];
                        sums[p.D + c] = u ? sums[p.D + c] + db[k][i] : db[k][i];
                    }
                }
        }
        __syncthreads();
    }
    for (int64_t c = threadIdx.x; c < 2 * p.D; c += T * R) p.part[blockIdx.x * 2 * p.D + c] = sums[c];
}

template <typename IO, Layout L, int T, int NC, int R>
__global__ void __launch_bounds__(T* R) ln_bwd_kernel(const LnParams p) {
    __shared__ GroupSum<T, 2, R> sh;
    extern __shared__ float sums[];  // [2][D]
    begin_kernel();
    const int group = threadIdx.x / T, t = threadIdx.x % T;
    float w[NC][8], dw[NC][8] = {}, db[NC][8] = {};
    load_columns<L, T, NC>(p.w, 1.f, p.D, t, w);
    const int64_t step = (int64_t)gridDim.x * R, base = (int64_t)blockIdx.x * R;
    using C = Chunk<IO, L, T>;
    C xin[NC], gin[NC];
    float mean = 0.f, rstd = 0.f;
    auto fetch = [&](int64_t r) {
        const bool there = r < p.rows;
        const IO* x = static_cast<const IO*>(p.x) + r * p.xs;
        const IO* g = static_cast<const IO*>(p.dy) + r * p.D;
        const int64_t D = there ? p.D : 0;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            xin[k].load(x, D, (int64_t)k * 8 * T, t);
            gin[k].load(g, D, (int64_t)k * 8 * T, t);
        }
        mean = there ? __ldg(p.mean + r) : 0.f;
        rstd = there ? __ldg(p.rstd + r) : 0.f;
    };
    int64_t row = base + group;
    fetch(row);
    float bad = 0.f;
    int turn = 0;
    for (int64_t r0 = base; r0 < p.rows; r0 += step, row += step) {
        float xh[NC][8], g[NC][8], s[2] = {0.f, 0.f};
        const float m = mean, rs = rstd;
#pragma unroll
        for (int k = 0; k < NC; ++k) xin[k].get(xh[k]), gin[k].get(g[k]);
        fetch(row + step);
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // elements past the row are 0 in g, and in xh, too: -m rs could be infinite
                xh[k][i] = column<L, T>((int64_t)k * 8 * T, t, i) < p.D ? (xh[k][i] - m) * rs : 0.f;
                dw[k][i] = __fmaf_rn(g[k][i], xh[k][i], dw[k][i]);
                db[k][i] += g[k][i];
                g[k][i] *= w[k][i];
                s[0] += g[k][i];
                s[1] = __fmaf_rn(g[k][i], xh[k][i], s[1]);
            }
        group_sum<T, 2, R>(sh, turn++, group, t, s);
        const float c1 = s[0] * p.inv_d, c2 = s[1] * p.inv_d;
        if (row < p.rows) {
            IO* to = static_cast<IO*>(p.dx) + row * p.D;
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    y[i] = rs * __fmaf_rn(-xh[k][i], c2, g[k][i] - c1);
                    bad = __fmaf_rn(y[i], 0.f, bad);
                }
                C::store(to, p.D, (int64_t)k * 8 * T, t, y);
            }
        }
    }
    flag_nonfinite(p.status, bad);
    if (p.part) leave_sums<L, T, NC, R>(p, sums, dw, db);
}

// ---------------------------------------------------------------- rings
constexpr int kMostStages = 6;

__device__ __forceinline__ void bulk_copy(void* dst, uintptr_t src, unsigned bytes, unsigned bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
// A group's ring: `N` tensors' rows r, r + step, ... into its part of the
// shared memory, p.stages rows ahead. ALIGNED: every row starts and ends on 16
// bytes; else a row's copy takes the 16-byte words that it lies in, unless the
// tensor does not have all of them: then it is read where it is.
template <int N, bool ALIGNED> struct Feed {
    uintptr_t lo[N], hi[N];          // the tensor: its first byte, and past its last
    uintptr_t ahead[N], now[N];      // the next row to copy, the row to work on
    uintptr_t pitch[N];              // from one of the group's rows to the next
    char* buf;
    unsigned bars, row_bytes;
    int64_t next, step, rows;
    int stages, bytes, stage = 0, phase = 0, fstage = 0;
    bool first, late = false;
    __device__ __forceinline__ bool words(int i, uintptr_t a, uintptr_t& from, unsigned& n) const {
        if (ALIGNED) {
            from = a, n = row_bytes;
            return true;
        }
        const uintptr_t to = (a + row_bytes + 15) & ~uintptr_t(15);
        from = a & ~uintptr_t(15);
        n = (unsigned)(to - from);
        return from >= lo[i] && to <= hi[i];
    }
    // The group's first thread: the next row's copies into the next stage.
    __device__ __forceinline__ void fetch() {
        if (first && next < rows) {
            const unsigned bar = bars + 8 * fstage;
            uintptr_t from[N];
            unsigned n[N], all = 0;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (!words(i, ahead[i], from[i], n[i])) n[i] = 0;
                all += n[i];
                ahead[i] += pitch[i];
            }
            mbar_expect_tx(bar, all);
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (n[i]) bulk_copy(buf + (fstage * N + i) * bytes, from[i], n[i], bar);
        }
        next += step;
        fstage = fstage + 1 == stages ? 0 : fstage + 1;
    }
    // Waits for the stage of the group's row; a wait that ran out stays so.
    __device__ __forceinline__ void wait() {
        if (!late && !mbar_wait_bounded(bars + 8 * stage, phase)) late = true;
    }
    // Where the row of tensor i is: in the stage, or (not copied) in global memory.
    __device__ __forceinline__ const char* row(int i) const {
        uintptr_t from;
        unsigned n;
        const char* to = buf + (stage * N + i) * bytes;
        if (ALIGNED) return to;
        if (!words(i, now[i], from, n)) return reinterpret_cast<const char*>(now[i]);
        return to + (now[i] - from);
    }
    __device__ __forceinline__ void leave() {
        if (!ALIGNED) {
#pragma unroll
            for (int i = 0; i < N; ++i) now[i] += pitch[i];
        }
        if (++stage == stages) stage = 0, phase ^= 1;
    }
    // A wait ran out: copies still in flight get some time more before the shared memory is given back.
    __device__ __forceinline__ void drain(unsigned* status) {
        if (!late) return;
        if (status) atomicOr(status, kStatusTimeout);
        for (int j = 0; j < stages; ++j) {
            mbar_wait_bounded(bars + 8 * stage, phase, kWaitNs / 16);
            leave();
        }
    }
};
// All threads of the CTA: barriers, then the first rows.
template <int N, bool ALIGNED, typename IO, int T, int R>
__device__ __forceinline__ Feed<N, ALIGNED> open_feed(const LnParams& p, uint64_t (&full)[R][kMostStages], char* smem, int group, int t) {
    Feed<N, ALIGNED> f;
    f.next = (int64_t)blockIdx.x * R + group, f.step = (int64_t)gridDim.x * R, f.rows = p.rows;
    f.row_bytes = (unsigned)(p.D * sizeof(IO));
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uintptr_t row = (uintptr_t)(i ? p.D : p.xs) * sizeof(IO);
        f.lo[i] = reinterpret_cast<uintptr_t>(i ? p.dy : p.x);
        f.hi[i] = f.lo[i] + (uintptr_t)(p.rows - 1) * row + f.row_bytes;
        f.ahead[i] = f.now[i] = f.lo[i] + (uintptr_t)f.next * row;
        f.pitch[i] = (uintptr_t)f.step * row;
    }
    f.stages = p.stages, f.bytes = p.stage_bytes;
    f.buf = smem + (size_t)group * p.stages * N * p.stage_bytes;
    f.bars = smem_u32(&full[group][0]);
    f.first = t == 0;
    if (t == 0) {
        for (int j = 0; j < p.stages; ++j) mbar_init(f.bars + 8 * j, 1);
        mbar_fence_init();
    }
    __syncthreads();
    for (int j = 0; j < p.stages; ++j) f.fetch();
    return f;
}

// Elements of a chunk that lie past the row, as zeros.
template <Layout L, int T> __device__ __forceinline__ void keep_row(float2 (&v)[4], int D, int c0, int t) {
    if (c0 + 8 * T <= D) return;
    if constexpr (L == Layout::kOct) {
        if (c0 + 8 * t >= D) v[0] = v[1] = v[2] = v[3] = pk(0.f, 0.f);
    } else if constexpr (L == Layout::kQuad) {
        if (c0 + 4 * t >= D) v[0] = v[1] = pk(0.f, 0.f);
        if (c0 + 4 * t + 4 * T >= D) v[2] = v[3] = pk(0.f, 0.f);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (c0 + 2 * i * T + t >= D) v[i].x = 0.f;
            if (c0 + (2 * i + 1) * T + t >= D) v[i].y = 0.f;
        }
    }
}
// A thread's eight elements of a chunk in shared memory, as pairs.
template <typename IO, Layout L, int T> __device__ __forceinline__ void take_pairs(const IO* row, int D, int c0, int t, float2 (&v)[4]) {
    Chunk<IO, L, T> in;
    in.take(row, D, c0, t);
    float f[8];
    in.get(f);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pk(f[2 * i], f[2 * i + 1]);
}
// The same with `fill` past the row, but where rows are read in eights.
template <typename IO, Layout L, int T>
__device__ __forceinline__ void take_pairs(const IO* row, int D, int c0, int t, IO fill, float2 (&v)[4]) {
    if constexpr (L == Layout::kOct) {
        take_pairs<IO, L, T>(row, D, c0, t, v);
    } else {
        Chunk<IO, L, T> in;
        in.take(row, D, c0, t, fill);
        float f[8];
        in.get(f);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = pk(f[2 * i], f[2 * i + 1]);
    }
}
// ... and normalised, (x + c) a. What has passed the row must be finite there, also where c a is not (a row of equal
// elements far from zero): it is read as -c, rounded to the row's type (equal elements are of that type), or a taken as 0.
template <typename IO, Layout L, int T>
__device__ __forceinline__ void take_normalised(const IO* row, int D, int c0, int t, float2 c, float2 a, IO fill, float2 (&v)[4]) {
    take_pairs<IO, L, T>(row, D, c0, t, fill, v);
    if (L == Layout::kOct && c0 + 8 * t >= D) a = pk(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __fmul2_rn(__fadd2_rn(v[i], c), a);
}
template <typename IO, Layout L, int T> __device__ __forceinline__ void store_pairs(IO* row, int64_t D, int c0, int t, const float2 (&v)[4]) {
    const float f[8] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
    Chunk<IO, L, T>::store(row, D, c0, t, f);
}
__device__ __forceinline__ float2 splat(float v) { return pk(v, v); }

// A column parameter in shared memory as the threads read it: a thread's
// eight of a chunk as two float4, [chunk][half][thread].
template <Layout L, int T, int NC> __device__ __forceinline__ void stage_columns(float4* to, const float* p, float none, int D) {
    float* f = reinterpret_cast<float*>(to);
    for (int j = threadIdx.x; j < 8 * T * NC; j += blockDim.x) {
        const int k = j / (8 * T), i = j / (4 * T) % 2 * 4 + j % 4, t = j / 4 % T;
        const int c = (int)column<L, T>((int64_t)k * 8 * T, t, i);
        f[j] = p && c < D ? __ldg(p + c) : none;
    }
}
template <int T> __device__ __forceinline__ void column_pairs(const float4* from, int k, int t, float2 (&v)[4]) {
    const float4 a = from[k * 2 * T + t], b = from[(k * 2 + 1) * T + t];
    v[0] = pk(a.x, a.y), v[1] = pk(a.z, a.w), v[2] = pk(b.x, b.y), v[3] = pk(b.z, b.w);
}

template <typename IO, Layout L, int T, int NC, int R>
__global__ void __launch_bounds__(T* R, NC > 4 ? 2 : 3) ln_fwd_ring_kernel(const LnParams p) {
    __shared__ GroupSum<T, 1, R> sh;
    __shared__ uint64_t full[R][kMostStages];
    extern __shared__ __align__(16) char smem[];
    const int group = threadIdx.x / T, t = threadIdx.x % T, D = (int)p.D;
    float4 *w = reinterpret_cast<float4*>(smem), *b = w + 2 * T * NC;
    begin_kernel();
    auto feed = open_feed<1, L != Layout::kEach, IO, T, R>(p, full, reinterpret_cast<char*>(b + 2 * T * NC), group, t);
    stage_columns<L, T, NC>(w, p.w, 1.f, D);
    stage_columns<L, T, NC>(b, p.b, 0.f, D);
    __syncthreads();
    float2 bad = pk(0.f, 0.f);
    int turn = 0;
    IO* to = static_cast<IO*>(p.y) + ((int64_t)blockIdx.x * R + group) * p.D;
    for (int64_t row = (int64_t)blockIdx.x * R + group; row < p.rows; row += feed.step, to += feed.step * p.D) {
        feed.wait();
        const IO* x = reinterpret_cast<const IO*>(feed.row(0));
        float2 v[NC][4], s2 = pk(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            take_pairs<IO, L, T>(x, D, k * 8 * T, t, v[k]);
#pragma unroll
            for (int i = 0; i < 4; ++i) s2 = __fadd2_rn(s2, v[k][i]);
        }
        float s[1] = {s2.x + s2.y};
        group_sum<T, 1, R>(sh, turn++, group, t, s);  // (every thread of the group has read the stage)
        feed.leave();
        if (!feed.late) feed.fetch();
        const float mean = s[0] * p.inv_d;
        float2 q2 = pk(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < NC; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[k][i] = __fadd2_rn(v[k][i], splat(-mean));
            keep_row<L, T>(v[k], D, k * 8 * T, t);
#pragma unroll
            for (int i = 0; i < 4; ++i) q2 = __ffma2_rn(v[k][i], v[k][i], q2);
        }
        float q[1] = {q2.x + q2.y};
        group_sum<T, 1, R>(sh, turn++, group, t, q);
        const float rstd = 1.0f / sqrtf(__fmaf_rn(q[0], p.inv_d, p.eps));
        if (t == 0 && p.mean) p.mean[row] = mean;
        if (t == 0 && p.rstd) p.rstd[row] = rstd;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            if (k * 8 * T >= D) break;
            float2 wk[4], bk[4];
            column_pairs<T>(w, k, t, wk);
            column_pairs<T>(b, k, t, bk);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                bk[i] = __ffma2_rn(__fmul2_rn(v[k][i], splat(rstd)), wk[i], bk[i]);
                bad = __ffma2_rn(bk[i], splat(0.f), bad);
            }
            store_pairs<IO, L, T>(to, p.D, k * 8 * T, t, bk);
        }
    }
    feed.drain(p.status);
    flag_nonfinite(p.status, bad.x + bad.y);
}

// The sums over a group of two values a thread, the same on every one: the
// half warps take one each at the first exchange.
template <int T, int R>
__device__ __forceinline__ float2 group_sum2(GroupSum<T, 2, R>& sh, int turn, int group, int t, float a, float b) {
    const int lane = threadIdx.x & 31;
    const bool up = lane & 16;
    float c = (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    if constexpr (T == 32) {
        return pk(__shfl_sync(0xffffffffu, c, 0), __shfl_sync(0xffffffffu, c, 16));
    } else {
        if ((lane & 15) == 0) sh.part[turn & 1][group][t >> 5][lane >> 4] = c;
        asm volatile("bar.sync %0, %1;\n" ::"r"(group + 1), "n"(T) : "memory");
        float2 s = *reinterpret_cast<const float2*>(sh.part[turn & 1][group][0]);
#pragma unroll
        for (int w = 1; w < T / 32; ++w) s = __fadd2_rn(s, *reinterpret_cast<const float2*>(sh.part[turn & 1][group][w]));
        return s;
    }
}

template <typename IO, Layout L, int T, int NC, int R>
__global__ void __launch_bounds__(T* R, 1) ln_bwd_ring_kernel(const LnParams p) {
    __shared__ __align__(16) GroupSum<T, 2, R> sh;
    __shared__ uint64_t full[R][kMostStages];
    extern __shared__ __align__(16) char smem[];
    const int group = threadIdx.x / T, t = threadIdx.x % T, D = (int)p.D;
    float4* w = reinterpret_cast<float4*>(smem);
    begin_kernel();
    auto feed = open_feed<2, L != Layout::kEach, IO, T, R>(p, full, reinterpret_cast<char*>(w + 2 * T * NC), group, t);
    stage_columns<L, T, NC>(w, p.w, 1.f, D);
    __syncthreads();
    float2 dw[NC][4], db[NC][4];
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[k][i] = db[k][i] = pk(0.f, 0.f);
    float2 bad = pk(0.f, 0.f);
    int turn = 0;
    const int64_t row0 = (int64_t)blockIdx.x * R + group;
    const float *mp = p.mean + row0, *rp = p.rstd + row0;
    float mean = row0 < p.rows ? __ldg(mp) : 0.f, rstd = row0 < p.rows ? __ldg(rp) : 0.f;
    IO* to = static_cast<IO*>(p.dx) + row0 * p.D;
    for (int64_t row = row0; row < p.rows; row += feed.step, to += feed.step * p.D) {
        const float2 a = splat(rstd), c = splat(-mean);
        const IO fill = IOT<IO>::from_f(mean), zero = IOT<IO>::from_f(0.f);
        mp += feed.step, rp += feed.step;
        if (row + feed.step < p.rows) mean = __ldg(mp), rstd = __ldg(rp);
        feed.wait();
        const IO* x = reinterpret_cast<const IO*>(feed.row(0));
        const IO* dy = reinterpret_cast<const IO*>(feed.row(1));
        float2 s0 = pk(0.f, 0.f), s1 = pk(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            float2 xh[4], g[4], wk[4];
            take_normalised<IO, L, T>(x, D, k * 8 * T, t, c, a, fill, xh);
            take_pairs<IO, L, T>(dy, D, k * 8 * T, t, zero, g);  // (so what lies past the row takes no part)
            column_pairs<T>(w, k, t, wk);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dw[k][i] = __ffma2_rn(g[i], xh[i], dw[k][i]);
                db[k][i] = __fadd2_rn(db[k][i], g[i]);
                const float2 h = __fmul2_rn(g[i], wk[i]);
                s0 = __fadd2_rn(s0, h);
                s1 = __ffma2_rn(h, xh[i], s1);
            }
        }
        const float2 s = group_sum2<T, R>(sh, turn++, group, t, s0.x + s0.y, s1.x + s1.y);
        // dx = rstd (h - c1 - xh c2) = h rstd + (xh (-c2 rstd) - c1 rstd)
        const float2 c1 = splat(-s.x * p.inv_d * a.x), c2 = splat(-s.y * p.inv_d * a.x);
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            if (k * 8 * T >= D) break;
            float2 xh[4], g[4], wk[4];
            take_normalised<IO, L, T>(x, D, k * 8 * T, t, c, a, fill, xh);
            take_pairs<IO, L, T>(dy, D, k * 8 * T, t, zero, g);
            column_pairs<T>(w, k, t, wk);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                g[i] = __ffma2_rn(__fmul2_rn(g[i], wk[i]), a, __ffma2_rn(xh[i], c2, c1));
                bad = __ffma2_rn(g[i], splat(0.f), bad);
            }
            store_pairs<IO, L, T>(to, p.D, k * 8 * T, t, g);
        }
        // every thread of the group has read the stage: its next row
        if constexpr (T == 32) __syncwarp();
        else asm volatile("bar.sync %0, %1;\n" ::"r"(group + 1), "n"(T) : "memory");
        feed.leave();
        if (!feed.late) feed.fetch();
    }
    feed.drain(p.status);
    flag_nonfinite(p.status, bad.x + bad.y);
    if (!p.part) return;
    // the groups' column sums side by side in shared memory (where the rings were), then added in group order
    __syncthreads();
    constexpr int kHalf = 2 * T * NC;  // float4 of a group's dw
    float4* sums = reinterpret_cast<float4*>(smem);
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int j = group * 2 * kHalf + (2 * k + h) * T + t;
            sums[j] = make_float4(dw[k][2 * h].x, dw[k][2 * h].y, dw[k][2 * h + 1].x, dw[k][2 * h + 1].y);
            sums[j + kHalf] = make_float4(db[k][2 * h].x, db[k][2 * h].y, db[k][2 * h + 1].x, db[k][2 * h + 1].y);
        }
    __syncthreads();
    float* part = p.part + (int64_t)blockIdx.x * 2 * p.D;
    for (int j = threadIdx.x; j < 2 * kHalf; j += T * R) {
        float4 v = sums[j];
#pragma unroll
        for (int u = 1; u < R; ++u) {
            const float4 f = sums[j + u * 2 * kHalf];
            v.x += f.x, v.y += f.y, v.z += f.z, v.w += f.w;
        }
        const int i = j % kHalf, k = i / (2 * T), h = i / T % 2;
        const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t col = column<L, T>((int64_t)k * 8 * T, i % T, 4 * h + e);
            if (col < p.D) part[(j / kHalf) * p.D + col] = f[e];
        }
    }
}

// Rows too wide for registers: a CTA a row, which it reads three times (the
// second and third from L2).
constexpr int kWideThreads = 512;
__device__ __forceinline__ float cta_sum(float v, float* sh) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWideThreads / 32; ++w) s += sh[w];
    return s;
}
template <typename IO, Layout L> __global__ void __launch_bounds__(kWideThreads) ln_fwd_wide_kernel(const LnParams p) {
    __shared__ float sh[kWideThreads / 32];
    constexpr int T = kWideThreads;
    using C = Chunk<IO, L, T>;
    const int t = threadIdx.x;
    begin_kernel();
    float bad = 0.f, v[8];
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const IO* x = static_cast<const IO*>(p.x) + row * p.xs;
        IO* y = static_cast<IO*>(p.y) + row * p.D;
        float s = 0.f, q = 0.f;
        C in;
#pragma unroll 4
        for (int64_t c0 = 0; c0 < p.D; c0 += 8 * T) {
            in.load(x, p.D, c0, t);
            in.get(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) s += v[i];
        }
        const float mean = cta_sum(s, sh) * p.inv_d;
#pragma unroll 4
        for (int64_t c0 = 0; c0 < p.D; c0 += 8 * T) {
            in.load(x, p.D, c0, t);
            in.get(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = column<L, T>(c0, t, i) < p.D ? v[i] - mean : 0.f;
                q = __fmaf_rn(d, d, q);
            }
        }
        const float rstd = 1.0f / sqrtf(__fmaf_rn(cta_sum(q, sh), p.inv_d, p.eps));
        if (t == 0 && p.mean) p.mean[row] = mean;
        if (t == 0 && p.rstd) p.rstd[row] = rstd;
#pragma unroll 4
        for (int64_t c0 = 0; c0 < p.D; c0 += 8 * T) {
            in.load(x, p.D, c0, t);
            in.get(v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t c = column<L, T>(c0, t, i);
                if (c < p.D) {
                    v[i] = __fmaf_rn((v[i] - mean) * rstd, p.w ? __ldg(p.w + c) : 1.f, p.b ? __ldg(p.b + c) : 0.f);
                    bad = __fmaf_rn(v[i], 0.f, bad);
                }
            }
            C::store(y, p.D, c0, t, v);
        }
    }
    flag_nonfinite(p.status, bad);
}
template <typename IO, Layout L> __global__ void __launch_bounds__(kWideThreads) ln_bwd_wide_kernel(const LnParams p) {
    __shared__ float sh[kWideThreads / 32];
    constexpr int T = kWideThreads;
    using C = Chunk<IO, L, T>;
    const int t = threadIdx.x;
    begin_kernel();
    float bad = 0.f, v[8], g[8];
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const IO *x = static_cast<const IO*>(p.x) + row * p.xs, *dy = static_cast<const IO*>(p.dy) + row * p.D;
        IO* dx = static_cast<IO*>(p.dx) + row * p.D;
        const float mean = __ldg(p.mean + row), rstd = __ldg(p.rstd + row);
        float s0 = 0.f, s1 = 0.f;
        C a, b;
#pragma unroll 4
        for (int64_t c0 = 0; c0 < p.D; c0 += 8 * T) {
            a.load(x, p.D, c0, t), b.load(dy, p.D, c0, t);
            a.get(v), b.get(g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t c = column<L, T>(c0, t, i);
                const float h = g[i] * (p.w && c < p.D ? __ldg(p.w + c) : 1.f);
                s0 += h;
                if (c < p.D) s1 = __fmaf_rn(h, (v[i] - mean) * rstd, s1);
            }
        }
        const float c1 = cta_sum(s0, sh) * p.inv_d, c2 = cta_sum(s1, sh) * p.inv_d;
#pragma unroll 4
        for (int64_t c0 = 0; c0 < p.D; c0 += 8 * T) {
            a.load(x, p.D, c0, t), b.load(dy, p.D, c0, t);
            a.get(v), b.get(g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int64_t c = column<L, T>(c0, t, i);
                const float h = g[i] * (p.w && c < p.D ? __ldg(p.w + c) : 1.f);
                v[i] = rstd * __fmaf_rn(-(v[i] - mean) * rstd, c2, h - c1);
                if (c < p.D) bad = __fmaf_rn(v[i], 0.f, bad);
            }
            C::store(dx, p.D, c0, t, v);
        }
    }
    flag_nonfinite(p.status, bad);
}
// The column sums of wide rows, before dx overwrites what it may alias: a CTA
// takes 1024 columns and a share of the rows.
constexpr int kColumnThreads = 128;
template <typename IO, Layout L> __global__ void __launch_bounds__(kColumnThreads) ln_columns_wide_kernel(const LnParams p) {
    constexpr int T = kColumnThreads;
    const int t = threadIdx.x;
    const int64_t c0 = (int64_t)blockIdx.x * 8 * T;
    begin_kernel();
    float dw[8] = {}, db[8] = {};
#pragma unroll 4
    for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
        Chunk<IO, L, T> a, b;
        a.load(static_cast<const IO*>(p.x) + row * p.xs, p.D, c0, t);
        b.load(static_cast<const IO*>(p.dy) + row * p.D, p.D, c0, t);
        const float mean = __ldg(p.mean + row), rstd = __ldg(p.rstd + row);
        float v[8], g[8];
        a.get(v), b.get(g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            dw[i] = __fmaf_rn(g[i], (v[i] - mean) * rstd, dw[i]);
            db[i] += g[i];
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t c = column<L, T>(c0, t, i);
        if (c < p.D) {
            p.part[(int64_t)blockIdx.y * 2 * p.D + c] = dw[i];
            p.part[((int64_t)blockIdx.y * 2 + 1) * p.D + c] = db[i];
        }
    }
}

// dw and db from the CTAs' sums [n, 2, D], in CTA order: 32 columns a CTA,
// 32 warps that take every 32nd row, folded in warp order.
__global__ void __launch_bounds__(1024) ln_columns_kernel(const float* __restrict__ part, int64_t n, int64_t D, float* dw, float* db) {
    __shared__ float red[32][33];
    begin_kernel();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < 2 * D) {
#pragma unroll 8
        for (int64_t r = warp; r < n; r += 32) s += __ldg(part + r * 2 * D + c);
    }
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < 2 * D) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < 32; ++w) t += red[w][lane];
        float* to = c < D ? dw : db;
        if (to) to[c < D ? c : c - D] = t;
    }
}

// The widest row that a group holds (a row of x and dy and the weight fit in
// shared memory), and the most CTAs that write sums: one an SM.
constexpr int64_t kWidest = 16384;
constexpr int kWideShares = 64, kMostCtas = 160;
int64_t most_ctas(int64_t rows, int64_t D) {
    const int64_t n = D > kWidest ? kWideShares : kMostCtas;
    return rows < n ? rows : n;
}


// Stages of a group's ring: as many rows as fit `budget` bytes a CTA, at least
// `least`: two, or one where beside the columns that is all that fits.
template <typename IO, int T, int NC> constexpr int least_stages(int tensors, int groups, int columns) {
    return columns + 2 * tensors * groups * (8 * T * NC * (int)sizeof(IO) + 32) <= 226 * 1024 ? 2 : 1;
}
void set_ring(LnParams& p, int tensors, int groups, int es, int budget, int least) {
    // a row and what its first and last 16-byte words may hold beside it
    p.stage_bytes = (int)((p.D * es + 15 + 15) / 16 * 16);
    const int n = budget / (groups * tensors * p.stage_bytes);
    p.stages = n < least ? least : n > kMostStages ? kMostStages : n;
}
// Bytes of shared memory of a CTA's rings, for the widest row of a group size.
template <typename IO, int T, int NC> constexpr int most_ring(int tensors, int groups, int budget, int least) {
    const int rows = least * tensors * groups * (8 * T * NC * (int)sizeof(IO) + 32);
    return rows > budget ? rows : budget;
}
template <typename IO, Layout L, int T, int NC> int launch_fwd_group(LnParams p, cudaStream_t s) {
    constexpr int R = T < 256 ? 256 / T : 1, kBudget = 48 * 1024;
    const int64_t want = (p.rows + R - 1) / R;
    int dev = 0, n = 1, smem = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -1;
    auto go = [&](auto kern) {
        const int64_t slots = (int64_t)n * sm_count();
        return launch_next(kern, dim3((unsigned)(want < slots ? want : slots)), T * R, smem, s, p);
    };
    if constexpr (T < 32) {
        static int per_sm[64] = {};
        auto kern = ln_fwd_kernel<IO, L, T, NC, R>;
        int& m = per_sm[dev & 63];
        if (m == 0 && (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&m, kern, T * R, 0) != cudaSuccess || m < 1)) return m = 0, -1;
        n = m;
        return go(kern);
    } else {
        static unsigned long long mask = 0;
        auto kern = ln_fwd_ring_kernel<IO, L, T, NC, R>;
        constexpr int kColumns = 2 * 8 * T * NC * (int)sizeof(float);  // weight and bias
        constexpr int kLeast = least_stages<IO, T, NC>(1, R, kColumns);
        if (!ensure_smem(kern, kColumns + most_ring<IO, T, NC>(1, R, kBudget, kLeast), mask)) return -1;
        set_ring(p, 1, R, sizeof(IO), kBudget, kLeast);
        smem = kColumns + p.stages * R * p.stage_bytes;
        n = smem > 110 * 1024 ? 1 : NC > 4 ? 2 : 3;  // (or by the kernel's launch bounds)
        return go(kern);
    }
}
template <typename IO, Layout L, int T, int NC> int launch_bwd_group(LnParams p, unsigned& ctas, cudaStream_t s) {
    // In fp32 half the groups where rows are long, so that three of them still fit (65537 x 1023: 130 us, with all 138;
    // 65536 x 256 with all 39, with half 48).
    constexpr int kThreads = T < 32 || sizeof(IO) == 2 || 8 * T * NC <= 512 ? 512 : 256, R = T < kThreads ? kThreads / T : 1;
    constexpr int kBudget = (8 * T * NC > 8192 ? 160 : 192) * 1024;  // (what the weight leaves)
    const int64_t want = (p.rows + R - 1) / R, slots = sm_count() < kMostCtas ? sm_count() : kMostCtas;
    ctas = (unsigned)(want < slots ? want : slots);
    static unsigned long long mask = 0;
    if constexpr (T < 32) {
        const int sums = p.part ? (int)(2 * p.D * sizeof(float)) : 0;
        auto kern = ln_bwd_kernel<IO, L, T, NC, R>;
        if (!ensure_smem(kern, 2 * 8 * T * NC * (int)sizeof(float), mask)) return -1;
        return launch_next(kern, dim3(ctas), T * R, sums, s, p);
    } else {
        auto kern = ln_bwd_ring_kernel<IO, L, T, NC, R>;
        constexpr int kColumns = 8 * T * NC * (int)sizeof(float);  // the weight
        constexpr int kSums = R * 2 * kColumns;                    // the groups' column sums, in the end
        constexpr int kLeast = least_stages<IO, T, NC>(2, R, kColumns), kRing = most_ring<IO, T, NC>(2, R, kBudget, kLeast);
        if (!ensure_smem(kern, kColumns + (kRing > kSums ? kRing : kSums), mask)) return -1;
        set_ring(p, 2, R, sizeof(IO), kBudget, kLeast);
        const int ring = kColumns + p.stages * 2 * R * p.stage_bytes;
        return launch_next(kern, dim3(ctas), T * R, ring > kSums ? ring : kSums, s, p);
    }
}

template <typename IO, Layout L> int launch_wide(bool bwd, const LnParams& p, unsigned& ctas, cudaStream_t s) {
    const int64_t cap = 4 * (int64_t)sm_count();
    const unsigned grid = (unsigned)(p.rows < cap ? p.rows : cap);
    if (!bwd) {
        return launch_next(ln_fwd_wide_kernel<IO, L>, dim3(grid), kWideThreads, 0, s, p);
    }
    int n = 0;
    if (p.part) {
        ctas = (unsigned)(p.rows < kWideShares ? p.rows : kWideShares);
        const unsigned across = (unsigned)((p.D + 8 * kColumnThreads - 1) / (8 * kColumnThreads));
        if (launch_next(ln_columns_wide_kernel<IO, L>, dim3(across, ctas), kColumnThreads, 0, s, p) < 0) return -1;
        ++n;
    }
    return launch_next(ln_bwd_wide_kernel<IO, L>, dim3(grid), kWideThreads, 0, s, p) < 0 ? -1 : n + 1;
}

// The group for a row: half a warp for up to 256 elements in the forward
// (65536 x 256 bf16 14 us, in a warp 22; in the backward 34 and 28), a warp for
// up to 2048 (64 a lane; 65536 x 2048 bf16 97 us, in two warps 99), in the
// backward for up to 512 (16 a lane; 65536 x 1024 in two warps of 16 a lane
// 74 us, in one of 32 a lane 87); beyond, the fewest warps with at most 64 (32)
// a lane.
template <typename IO, Layout L> int launch_rows(bool bwd, const LnParams& p, unsigned& ctas, cudaStream_t s) {
    if (p.D > kWidest) return launch_wide<IO, L>(bwd, p, ctas, s);
#define LN_GROUP(T, NC, FT, FNC) return bwd ? launch_bwd_group<IO, L, T, NC>(p, ctas, s) : launch_fwd_group<IO, L, FT, FNC>(p, s)
    if (p.D <= 32) LN_GROUP(4, 1, 4, 1);
    if (p.D <= 128) LN_GROUP(16, 1, 16, 1);
    if (p.D <= 256) LN_GROUP(32, 1, 16, 2);
    if (p.D <= 512) LN_GROUP(32, 2, 32, 2);
    if (p.D <= 1024) LN_GROUP(64, 2, 32, 4);
    if (p.D <= 2048) LN_GROUP(64, 4, 32, 8);
    if (p.D <= 4096) LN_GROUP(128, 4, 64, 8);
    if (p.D <= 8192) LN_GROUP(256, 4, 128, 8);
    LN_GROUP(512, 4, 256, 8);
#undef LN_GROUP
}
bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool off(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

int launch_layernorm(bool bwd, const LnParams& p, int io, unsigned& ctas, cudaStream_t s) {
    const int64_t es = io == SSM_BF16 ? 2 : 4;
    // Vectors where every row starts on 16 bytes (65536 x 768 bf16: 37 us forward and 67 backward; singly 49 and 105).
    const bool vec = p.D * es % 16 == 0 && p.xs * es % 16 == 0 && on16(p.x) && on16(p.y) && on16(p.dy) && on16(p.dx);
    if (io == SSM_BF16)
        return vec ? launch_rows<__nv_bfloat16, kVector<__nv_bfloat16>>(bwd, p, ctas, s)
                   : launch_rows<__nv_bfloat16, Layout::kEach>(bwd, p, ctas, s);
    return vec ? launch_rows<float, kVector<float>>(bwd, p, ctas, s) : launch_rows<float, Layout::kEach>(bwd, p, ctas, s);
}

int check_layernorm(const ssm_layernorm_args* a) {
    if (!a) return SSM_ERR_INVALID_ARG;
    if (a->rows < 0 || a->D < 0 || a->x_stride < 0 || (a->x_stride && a->x_stride < a->D)) return SSM_ERR_INVALID_ARG;
    if (a->io_dtype != SSM_F32 && a->io_dtype != SSM_BF16) return SSM_ERR_UNSUPPORTED;
    if (!std::isfinite(a->eps) || a->eps < 0.f) return SSM_ERR_INVALID_ARG;
    // every element count stays far inside 64 bits, and a CTA's columns inside 32
    if (a->rows > (int64_t(1) << 40) || a->D > (int64_t(1) << 30) || a->x_stride > (int64_t(1) << 32)) return SSM_ERR_UNSUPPORTED;
    if (a->rows > 0 && a->D > 0 && !a->x) return SSM_ERR_INVALID_ARG;
    const unsigned es = a->io_dtype == SSM_BF16 ? 2 : 4;
    if (off(a->x, es) || off(a->y, es)) return SSM_ERR_ALIGNMENT;
    for (const void* q : {(const void*)a->w, (const void*)a->b, (const void*)a->mean, (const void*)a->rstd})
        if (off(q, 4)) return SSM_ERR_ALIGNMENT;
    if (off(a->status, 16)) return SSM_ERR_ALIGNMENT;
    return SSM_OK;
}

LnParams ln_params(const ssm_layernorm_args& a) {
    LnParams p{};
    p.rows = a.rows; p.D = a.D; p.xs = a.x_stride ? a.x_stride : a.D;
    p.eps = a.eps; p.inv_d = a.D ? (float)(1.0 / (double)a.D) : 0.f;
    p.x = a.x; p.w = a.w; p.b = a.b; p.mean = a.mean; p.rstd = a.rstd; p.y = a.y;
    p.status = static_cast<unsigned*>(a.status);
    return p;
}

}  // namespace
}  // namespace ssm

extern "C" {

size_t ssm_layernorm_workspace_bytes(int64_t rows, int64_t D) {
    if (rows <= 0 || D <= 0) return 0;
    return (size_t)ssm::most_ctas(rows, D) * 2 * (size_t)D * sizeof(float);
}

int ssm_layernorm_fwd(const ssm_layernorm_args* a, void* stream) {
    ssm::reset_launches();
    const int rc = ssm::check_layernorm(a);
    if (rc != SSM_OK) return rc;
    if (a->rows == 0 || a->D == 0) return SSM_OK;
    if (!a->y) return SSM_ERR_INVALID_ARG;
    unsigned ctas = 0;
    return ssm::count_launches(ssm::launch_layernorm(false, ssm::ln_params(*a), a->io_dtype, ctas, (cudaStream_t)stream));
}

int ssm_layernorm_bwd(const ssm_layernorm_bwd_args* a, void* stream) {
    ssm::reset_launches();
    if (!a) return SSM_ERR_INVALID_ARG;
    const ssm_layernorm_args& f = a->f;
    int rc = ssm::check_layernorm(&f);
    if (rc != SSM_OK) return rc;
    const bool work = f.rows > 0 && f.D > 0;
    if (work && (!a->dy || !a->dx || !f.mean || !f.rstd)) return SSM_ERR_INVALID_ARG;
    const unsigned es = f.io_dtype == SSM_BF16 ? 2 : 4;
    if (ssm::off(a->dy, es) || ssm::off(a->dx, es) || ssm::off(a->dw, 4) || ssm::off(a->db, 4) || ssm::off(a->workspace, 16))
        return SSM_ERR_ALIGNMENT;
    const bool sums = a->dw || a->db;
    if (sums && work && (!a->workspace || a->workspace_bytes < ssm_layernorm_workspace_bytes(f.rows, f.D))) return SSM_ERR_WORKSPACE;
    cudaStream_t s = (cudaStream_t)stream;
    if (!work) {
        for (float* q : {a->dw, a->db})
            if (q && f.D > 0 && cudaMemsetAsync(q, 0, (size_t)f.D * sizeof(float), s) != cudaSuccess) return SSM_ERR_CUDA;
        return SSM_OK;
    }
    ssm::LnParams p = ssm::ln_params(f);
    p.y = nullptr;
    p.dy = a->dy; p.dx = a->dx;
    p.part = sums ? static_cast<float*>(a->workspace) : nullptr;
    unsigned ctas = 0;
    rc = ssm::count_launches(ssm::launch_layernorm(true, p, f.io_dtype, ctas, s));
    if (rc != SSM_OK || !sums) return rc;
    return ssm::count_launches(ssm::launch_next(ssm::ln_columns_kernel, dim3((unsigned)((2 * f.D + 31) / 32)), 1024, 0, s,
                                                static_cast<const float*>(p.part), (int64_t)ctas, f.D, a->dw, a->db));
}

}  // extern "C"
