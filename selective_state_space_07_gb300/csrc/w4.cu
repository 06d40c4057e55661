// Matrix-vector products with 4-bit weights on sm_103a (include/w4.h holds
// the formula and the boundary).
//
// A decoding step reads each weight once for a handful of rows of x, so HBM
// bounds it: half a byte a weight. Sixteen rows of W are one tensor-core
// operand (mma.sync m16n8k16: the weights as A, eight rows of x as B): the
// larger tcgen05 tiles want the weights widened in TMEM or shared memory first,
// at four times their bytes.
//
// A warp takes 16 rows of W and units of 512 k, two TMA boxes of 2 KB each in a
// ring of the warp's own: its copies run two or four boxes ahead, across
// tiles, without holding registers for them. (Loaded straight into registers,
// the units came too late whatever the source's order: 42 us for 1 x 4096 x
// 65536.) A CTA's warps split K as far as that evens out the last round of
// tiles, and rows beyond that; their sums are added in warp order.
//
// Which k a fragment's places stand for does not matter as long as both
// operands agree, so nibbles stay where they are: a lane's 8, 16 or 32
// consecutive weights of a row and group are one load from the box, four masks
// and three shifts turn a word into four bf16 pairs (128 + q as bits, less
// 136: exact), and x lies in shared memory in the order that those pairs come
// in. Boxes are swizzled and the fragment's rows are taken in an order that
// makes the loads free of bank conflicts. A group's sum gets its scale in fp32.
//
// Measured, in percent of the HBM copy rate: 1 x 4096 x 65536 31 us (65%),
// groups of 32 38 (59%); there the instructions bound it, 165 a KB of weights,
// 88 of which take the nibbles apart. 1 x 2048 x 8192: 4.5 us, a launch. More
// rows of x add products and reads of x: 16 x 2048 x 50001 24 us (33%),
// 32 x 4096 x 65536 80 (26%). (Those with tcgen05, the widened weights as
// operand A in TMEM: 27 and 64 us. Writing 4 bytes of TMEM for each byte of
// weights bounds that, whatever the number of rows; it is slower for up to 16,
// and for fewer weights: 16 x 2048 x 2048 12 us, here 5.8.)
#include <cuda_bf16.h>

#include "../../include/w4.h"
#include "ssm_common.cuh"
#include "ssm_internal.h"

namespace ssm {
namespace {

constexpr int kUnitK = 512, kBoxK = 256, kBox = 16 * kBoxK / 2;  // a unit of k, and of its two boxes of 16 rows: 2 KB
constexpr int kMostRows = 32;       // rows of x a pass
// Of x in shared memory, at most. What does not fit there makes shares of K
// with sums through memory, so x comes before the rings: two boxes a warp and
// 128 KB of x take 80 us for 32 x 4096 x 65536, three and 96 KB 116.
constexpr int kXBytes = 128 * 1024;

struct W4Params {
    int64_t N, K, xs;
    int M;           // rows of x of this pass
    int groups;      // K / group
    int per;         // groups of a K share
    int tiles;       // of rows of W, a CTA's at a time
    int split;       // warps that split K (the others take other rows): a power of two
    int rows_log2;   // rows of W of a CTA's tile
    bool wide_scales;  // a unit's scales of a row start on 8 bytes
    const __nv_bfloat16* x;
    const uint8_t* q;
    const __nv_bfloat16* s;
    const float* bias;
    void* y;
    float* part;     // [shares, M, N], nullable
    unsigned* status;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same onto zero.
__device__ __forceinline__ void mma_first(float (&c)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// Nibbles 0 and 4 of v as q - 8 in bf16: 0x4300 | q is 128 + q. (One three-input
// logic operation: with both constants as immediates it would be two.)
__device__ __forceinline__ unsigned two_weights(unsigned v) {
    unsigned u, r;
    asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(u) : "r"(v), "r"(0x43004300u));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(u), "r"(0x43084308u));  // 136
    return r;
}
// A unit's scales of one row: bf16 pairs, for G groups from s on; zero for
// groups past the last, the `left` th (x is zero there, too, and an infinite
// scale must not meet it). The loads stay in front of the waits that follow them.
template <int G> struct Scales {
    unsigned v[G / 2];
    __device__ __forceinline__ void load(bool wide, const unsigned short* s, int left) {
        if (wide) {  // (whole units only)
#pragma unroll
            for (int j = 0; j < G; j += 4)
                asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];\n" : "=r"(v[j / 2]), "=r"(v[j / 2 + 1]) : "l"(s + j));
        } else {
#pragma unroll
            for (int j = 0; j < G; j += 2)
                v[j / 2] = (j < left ? __ldg(s + j) : 0u) | (j + 1 < left ? (unsigned)__ldg(s + j + 1) : 0u) << 16;
        }
    }
    __device__ __forceinline__ float get(int j) const {
        return __uint_as_float(j & 1 ? v[j / 2] & 0xffff0000u : v[j / 2] << 16);
    }
};

// W words of a box.
template <int W> __device__ __forceinline__ void read_words(const char* p, unsigned (&v)[W]) {
    if constexpr (W == 4) {
        const uint4 q = *reinterpret_cast<const uint4*>(p);
        v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
    } else if constexpr (W == 2) {
        const uint2 q = *reinterpret_cast<const uint2*>(p);
        v[0] = q.x, v[1] = q.y;
    } else {
        v[0] = *reinterpret_cast<const unsigned*>(p);
    }
}

// What a kernel of WARPS warps and MT tiles of eight rows of x keeps beside x:
// the ring, and two sets of the warps' sums (one where two would not fit).
template <int MT, int WARPS> struct W4Smem {
    static constexpr int kStages = WARPS == 8 ? 4 : 2;
    static constexpr int kSets = MT > 2 ? 1 : 2;
    static constexpr int kRing = WARPS * kStages * kBox, kSum = WARPS * MT * 16 * 8 * 4;
    static constexpr int kOwn = kRing + kSets * kSum + 1024;  // (1024: the boxes' alignment)
};

// W: words of 8 weights a lane holds of a row's group (group = 32 W).
template <int W, int MT, int WARPS, typename OUT>
__global__ void __launch_bounds__(32 * WARPS, 1) w4_kernel(const W4Params p, const __grid_constant__ CUtensorMap weights) {
    using S = W4Smem<MT, WARPS>;
    constexpr int G = 16 / W, ST = S::kStages, kThreads = 32 * WARPS;  // groups of a unit
    extern __shared__ __align__(16) char raw[];
    let_next_start();
    char* base = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    float(*red)[WARPS][MT][16][8] = reinterpret_cast<float(*)[WARPS][MT][16][8]>(base + S::kRing);
    uint4* xs = reinterpret_cast<uint4*>(base + S::kRing + S::kSets * S::kSum);
    __shared__ uint64_t bars[WARPS][ST];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    char* ring = base + warp * ST * kBox;
    const int k0 = blockIdx.y * p.per, groups = min(p.per, p.groups - k0);  // the CTA's share of K
    const int units = (groups + G - 1) / G, ks = warp & (p.split - 1), rg = warp / p.split;
    // fragment row g is row 0 4 2 6 1 5 3 7 of the box: lanes that load together then differ in the swizzled bits
    const int r = (g & 1) * 4 + (g & 2) + (g >> 2);
    const int from = r * 128 + ((((t * W) / 4) ^ r) * 16 + (t * W % 4) * 4);

    // the boxes of the warp's units of all the CTA's tiles, as one sequence: what is copied next
    const int rows_log2 = p.rows_log2, row_step = gridDim.x << rows_log2;
    int frow = (blockIdx.x << rows_log2) + rg * 16, fu = ks, fhalf = 0, fstage = 0;
    const int row_end = p.tiles << rows_log2;
    const bool idle = ks >= units;  // (K = 0, or a last share of fewer units: nothing to copy)
    auto fetch = [&]() {
        if (frow >= row_end) return;
        if (lane == 0) {
            const unsigned bar = smem_u32(&bars[warp][fstage]);
            mbar_expect_tx(bar, kBox);
            tma_load_2d(ring + fstage * kBox, &weights, k0 * (16 * W) + fu * (kUnitK / 2) + fhalf * (kBoxK / 2), frow, bar);
        }
        fstage = fstage + 1 == ST ? 0 : fstage + 1;
        fhalf ^= 1;
        if (fhalf == 0) {
            fu += p.split;
            if (fu >= units) fu = ks, frow += row_step;
        }
    };
    if (lane == 0) {
        for (int j = 0; j < ST; ++j) mbar_init(smem_u32(&bars[warp][j]), 1);
        mbar_fence_init();
    }
    __syncwarp();
    wait_for_previous();
    if (!idle)
        for (int j = 0; j < ST; ++j) fetch();

    // x of the share, eight k at a time in the order that a word's nibbles come in: 0 4 1 5 2 6 3 7; zero in the groups
    // that fill the last unit
    const int blocks = groups * 4 * W, all = units * G * 4 * W;
    const unsigned per_row = 0xffffffffu / (unsigned)max(all, 1) + 1;  // u / all is u * this / 2^32: both are at most 2^13
#pragma unroll 4
    for (int u = threadIdx.x; u < all * p.M; u += kThreads) {
        const int m = (int)__umulhi(u, per_row), b = u - m * all;  // b: (group, lane t, word w)
        uint4 v = make_uint4(0, 0, 0, 0);
        if (b < blocks) v = __ldg(reinterpret_cast<const uint4*>(p.x + m * p.xs + ((int64_t)k0 * 4 * W + b) * 8));
        const int gr = b / (4 * W), bt = b / W % 4, bw = b % W;
        xs[((gr * W + bw) * p.M + m) * 4 + bt] = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                                                            __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
    }
    // the scales of the lane's two rows in a tile, from the share's first group on
    auto scale_row = [&](int tile, int half) {
        const int64_t row = min64(((int64_t)tile << rows_log2) + rg * 16 + r + 8 * half, p.N - 1);
        return reinterpret_cast<const unsigned short*>(p.s) + row * p.groups + k0;
    };
    const unsigned short *plo = scale_row(blockIdx.x, 0), *phi = scale_row(blockIdx.x, 1);
    Scales<G> slo, shi;
    if (!idle) {
        slo.load(p.wide_scales, plo + ks * G, groups - ks * G);
        shi.load(p.wide_scales, phi + ks * G, groups - ks * G);
    }
    __syncthreads();

    // rows of x past the last: the last again; those columns are not written
    int mrow[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) mrow[j] = min(8 * j + g, p.M - 1) * 4 + t;
    const int step = p.M * 4;  // from one word's fragments to the next's
    float bad = 0.f;
    int stage = 0, phase = 0, set = 0;
    bool late = false;
    for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
        float acc[MT][4] = {};
        for (int u = ks; u < units; u += p.split) {
            // the next unit's scales, while this one is worked on
            Scales<G> nlo, nhi;
            int nu = u + p.split;
            if (nu >= units) {
                nu = ks;
                plo = scale_row(tile + gridDim.x, 0), phi = scale_row(tile + gridDim.x, 1);
            }
            nlo.load(p.wide_scales, plo + nu * G, groups - nu * G);
            nhi.load(p.wide_scales, phi + nu * G, groups - nu * G);
            const uint4* xg = xs + u * G * W * step;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const bool came = late || mbar_wait_bounded(smem_u32(&bars[warp][stage]), phase);
                late = __any_sync(0xffffffffu, !came) || late;
                unsigned lo[G / 2][W], hi[G / 2][W];
                const char* box = ring + stage * kBox;
#pragma unroll
                for (int j = 0; j < G / 2; ++j) {
                    read_words<W>(box + (from ^ (j * 16 * W)), lo[j]);
                    read_words<W>(box + 1024 + (from ^ (j * 16 * W)), hi[j]);
                }
                __syncwarp();
                if (!late) {
                    if (++stage == ST) stage = 0, phase ^= 1;
                    fetch();
                }
#pragma unroll
                for (int j = 0; j < G / 2; ++j) {
                    float c[MT][4];
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        const unsigned l = lo[j][w], h = hi[j][w];
                        const unsigned a0[4] = {two_weights(l), two_weights(h), two_weights(l >> 4), two_weights(h >> 4)};
                        const unsigned a1[4] = {two_weights(l >> 8), two_weights(h >> 8), two_weights(l >> 12), two_weights(h >> 12)};
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const uint4 b = xg[mrow[m]];
                            if (w == 0) mma_first(c[m], a0, b.x, b.y);
                            else mma_bf16(c[m], a0, b.x, b.y);
                            mma_bf16(c[m], a1, b.z, b.w);
                        }
                        xg += step;
                    }
                    const float s0 = slo.get(half * (G / 2) + j), s1 = shi.get(half * (G / 2) + j);
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        acc[m][0] = __fmaf_rn(s0, c[m][0], acc[m][0]);
                        acc[m][1] = __fmaf_rn(s0, c[m][1], acc[m][1]);
                        acc[m][2] = __fmaf_rn(s1, c[m][2], acc[m][2]);
                        acc[m][3] = __fmaf_rn(s1, c[m][3], acc[m][3]);
                    }
                }
            }
            slo = nlo, shi = nhi;
        }
        if (S::kSets == 1) __syncthreads();  // the last tile's sums have been read
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            *reinterpret_cast<float2*>(&red[set][warp][m][r][2 * t]) = make_float2(acc[m][0], acc[m][1]);
            *reinterpret_cast<float2*>(&red[set][warp][m][r + 8][2 * t]) = make_float2(acc[m][2], acc[m][3]);
        }
        __syncthreads();
        for (int o = threadIdx.x; o < p.M << rows_log2; o += kThreads) {
            const int m = o >> rows_log2, row = o & ((1 << rows_log2) - 1);
            const int64_t n = ((int64_t)tile << rows_log2) + row;
            if (n >= p.N) continue;
            const int w0 = row / 16 * p.split;
            float v = 0.f;
            for (int w = 0; w < p.split; ++w) v += red[set][w0 + w][m >> 3][row & 15][m & 7];
            if (p.part) {
                p.part[((int64_t)blockIdx.y * p.M + m) * p.N + n] = v;
            } else {
                if (p.bias) v += __ldg(p.bias + n);
                static_cast<OUT*>(p.y)[(int64_t)m * p.N + n] = IOT<OUT>::from_f(v);
                bad = __fmaf_rn(v, 0.f, bad);
            }
        }
        if (S::kSets == 2) set ^= 1;  // (the next tile's sums go beside these)
    }
    if (late) {
        // a copy did not come in time (none was made after that): those in flight get some time more before the ring is
        // given back
        if (lane == 0 && p.status) atomicOr(p.status, kStatusTimeout);
        for (int j = 0; j < ST; ++j) {
            mbar_wait_bounded(smem_u32(&bars[warp][stage]), phase, kWaitNs / 16);
            if (++stage == ST) stage = 0, phase ^= 1;
        }
    }
    flag_nonfinite(p.status, bad);
}

// y from the K shares' sums, in their order: four values of a row a thread, side by side over the CTA.
constexpr int kJoin = 4 * 256;
template <typename OUT>
__global__ void __launch_bounds__(256) w4_join_kernel(const float* __restrict__ part, int shares, int64_t M, int64_t N,
                                                    const float* __restrict__ bias, OUT* y, unsigned* status) {
    const int64_t m = blockIdx.y, n0 = (int64_t)blockIdx.x * kJoin + threadIdx.x;
    float v[4] = {}, bad = 0.f;
    begin_kernel();
#pragma unroll 4
    for (int s = 0; s < shares; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n0 + 256 * j < N) v[j] += __ldg(part + (s * M + m) * N + n0 + 256 * j);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t n = n0 + 256 * j;
        if (n >= N) break;
        const float o = bias ? v[j] + __ldg(bias + n) : v[j];
        y[m * N + n] = IOT<OUT>::from_f(o);
        bad = __fmaf_rn(o, 0.f, bad);
    }
    flag_nonfinite(status, bad);
}

// One warp a group: scale and nibbles. Done once for weights, and so left simple: a byte stored a lane bounds it (65536 x
// 4096 with groups of 128 from bf16 340 us, 29% of the copy rate, from fp32 345; with groups of 32 993).
template <typename IN>
__global__ void __launch_bounds__(256) w4_quantize_kernel(int64_t count, int group, const IN* __restrict__ w, uint8_t* q,
                                                        __nv_bfloat16* s) {
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * 8;
    for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < count; i += step) {
        const IN* from = w + i * group;
        float v[2][2] = {}, most = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (2 * lane + 64 * h < group) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    v[h][j] = IOT<IN>::to_f(from[2 * lane + 64 * h + j]);
                    most = fmaxf(most, fabsf(v[h][j]));
                }
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(most, 7.0f));
        const float sf = __bfloat162float(sb);
        if (lane == 0) s[i] = sb;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (2 * lane + 64 * h < group) {
                int n[2];
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    n[j] = sf > 0.f ? 8 + (int)fminf(fmaxf(rintf(__fdiv_rn(v[h][j], sf)), -8.f), 7.f) : 8;
                q[(i * group) / 2 + lane + 32 * h] = (uint8_t)(n[0] | n[1] << 4);
            }
    }
}

int launched() { return cudaGetLastError() == cudaSuccess ? 1 : -1; }
bool off(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// Groups of a share of K for M rows of x: as many whole units as keep the share of x in shared memory.
int64_t share_groups(int64_t M, int group) { return kXBytes / (M * kUnitK * 2) * (kUnitK / group); }

template <int W, int MT, int WARPS, typename OUT> int launch_w4(W4Params p, int shares, cudaStream_t s) {
    using S = W4Smem<MT, WARPS>;
    auto kern = w4_kernel<W, MT, WARPS, OUT>;
    constexpr int G = 16 / W;
    static unsigned long long mask = 0;
    if (!ensure_smem(kern, S::kOwn + kXBytes, mask)) return -1;
    const int units = p.per > 0 ? (p.per + G - 1) / G : 1;
    const int64_t slots = sm_count() / shares > 0 ? sm_count() / shares : 1;
    // Warps that split K: of the powers of two that leave each a unit, the smallest (fewest sums to join) whose rounds
    // of tiles take the fewest rows of W in all (1 x 4096 x 4096: 4.8 us; unsplit 11.6; 16 x 2048 x 50001 24 and 29).
    int64_t least = 0;
    for (int split = 1; split <= WARPS && split <= units; split *= 2) {
        const int64_t rows = WARPS / split * 16, tiles = (p.N + rows - 1) / rows, cost = (tiles + slots - 1) / slots * rows;
        if (split == 1 || cost < least) least = cost, p.split = split;
    }
    p.wide_scales = p.groups % G == 0 && p.per % G == 0 && (reinterpret_cast<uintptr_t>(p.s) & 7u) == 0;
    const int rows = WARPS / p.split * 16;
    p.rows_log2 = 4;
    while (1 << p.rows_log2 < rows) ++p.rows_log2;
    p.tiles = (int)((p.N + rows - 1) / rows);
    CUtensorMap weights{};
    if (p.K > 0 && !encode_2d(&weights, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.q, p.K / 2, p.N, p.K / 2, kBoxK / 2, 16, CU_TENSOR_MAP_SWIZZLE_128B))
        return -1;
    return launch_next(kern, dim3((unsigned)(p.tiles < slots ? p.tiles : slots), (unsigned)shares), 32 * WARPS,
                       S::kOwn + units * kUnitK * p.M * 2, s, p, weights);
}
// One CTA an SM, of sixteen warps: x comes to shared memory once for all of
// them (1 x 4096 x 65536: 31.3 us; two CTAs of eight 33.4). Of eight, for
// half the rows of W at a time, where those would not fill half of the SMs
// (1 x 2048 x 2048: 3.8 us, as sixteen 4.8; 5 x 1536 x 768 5.7 and 7.5).
template <int W, typename OUT> int launch_rows(const W4Params& p, int shares, cudaStream_t s) {
    const int units = p.per > 0 ? (p.per * 2 * W + 31) / 32 : 1;
    int split = 1;  // the most warps that K can be split over
    while (split < 16 && 2 * split <= units) split *= 2;
    const bool few = (p.N + 256 / split - 1) / (256 / split) * 2 < sm_count();
#define W4_GO(MT) return few ? launch_w4<W, MT, 8, OUT>(p, shares, s) : launch_w4<W, MT, 16, OUT>(p, shares, s)
    if (p.M <= 8) W4_GO(1);
    if (p.M <= 16) W4_GO(2);
    W4_GO(4);
#undef W4_GO
}
template <typename OUT> int run_w4(const ssm_w4_args& a, cudaStream_t s) {
    int n = 0;
    for (int64_t m0 = 0; m0 < a.M; m0 += kMostRows) {
        W4Params p{};
        p.N = a.N; p.K = a.K; p.xs = a.x_stride ? a.x_stride : a.K;
        p.M = (int)min64(kMostRows, a.M - m0);
        p.groups = (int)(a.K / a.group);
        const int per = (int)min64(p.groups, share_groups(p.M, a.group));
        const int shares = p.groups > 0 ? (p.groups + per - 1) / per : 1;  // (K = 0: one share of nothing)
        const int unit = kUnitK / a.group;
        p.per = min(per, ((p.groups + shares - 1) / shares + unit - 1) / unit * unit);
        p.x = static_cast<const __nv_bfloat16*>(a.x) + m0 * p.xs;
        p.q = static_cast<const uint8_t*>(a.q);
        p.s = static_cast<const __nv_bfloat16*>(a.s);
        p.bias = a.bias;
        OUT* y = static_cast<OUT*>(a.y) + m0 * a.N;
        p.y = y;
        p.status = static_cast<unsigned*>(a.workspace);
        p.part = shares > 1 ? reinterpret_cast<float*>(static_cast<char*>(a.workspace) + 256) : nullptr;
        const int r = a.group == 128 ? launch_rows<4, OUT>(p, shares, s)
                                     : a.group == 64 ? launch_rows<2, OUT>(p, shares, s) : launch_rows<1, OUT>(p, shares, s);
        if (r < 0) return -1;
        n += r;
        if (shares > 1) {
            if (launch_next(w4_join_kernel<OUT>, dim3((unsigned)((a.N + kJoin - 1) / kJoin), (unsigned)p.M), 256, 0, s,
                            static_cast<const float*>(p.part), shares, (int64_t)p.M, a.N, a.bias, y, p.status) < 0)
                return -1;
            ++n;
        }
    }
    return n;
}

bool group_ok(int g) { return g == 32 || g == 64 || g == 128; }

}  // namespace
}  // namespace ssm

extern "C" {

size_t ssm_w4_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || K <= 0) return 256;
    const int64_t m = M < ssm::kMostRows ? M : ssm::kMostRows;
    // the most shares any group size gives
    int64_t shares = 1;
    for (int g : {32, 64, 128}) {
        const int64_t per = ssm::share_groups(m, g), n = ((K + g - 1) / g + per - 1) / per;
        if (n > shares) shares = n;
    }
    return 256 + (shares > 1 ? (size_t)shares * m * N * sizeof(float) : 0);
}

int ssm_w4_matvec(const ssm_w4_args* a, void* stream) {
    ssm::reset_launches();
    if (!a) return SSM_ERR_INVALID_ARG;
    if (a->M < 0 || a->N < 0 || a->K < 0 || a->x_stride < 0 || (a->x_stride && a->x_stride < a->K)) return SSM_ERR_INVALID_ARG;
    if (!ssm::group_ok(a->group) || a->K % a->group != 0) return SSM_ERR_UNSUPPORTED;
    if (a->y_dtype != SSM_F32 && a->y_dtype != SSM_BF16) return SSM_ERR_UNSUPPORTED;
    // tiles and groups are counted in 32 bits
    if (a->M > (int64_t(1) << 31) || a->N > (int64_t(1) << 30) || a->K > (int64_t(1) << 24) || a->x_stride > (int64_t(1) << 32))
        return SSM_ERR_UNSUPPORTED;
    const bool work = a->M > 0 && a->N > 0;
    if (work && (!a->y || (a->K > 0 && (!a->x || !a->q || !a->s)))) return SSM_ERR_INVALID_ARG;
    if (ssm::off(a->x, 16) || ssm::off(a->q, 16) || a->x_stride % 8 || ssm::off(a->s, 2) || ssm::off(a->bias, 4) ||
        ssm::off(a->y, a->y_dtype == SSM_BF16 ? 2 : 4) || ssm::off(a->workspace, 16))
        return SSM_ERR_ALIGNMENT;
    const size_t need = ssm_w4_workspace_bytes(a->M, a->N, a->K);
    if (a->workspace ? a->workspace_bytes < need : need > 256) return SSM_ERR_WORKSPACE;
    if (!work) return SSM_OK;
    cudaStream_t s = (cudaStream_t)stream;
    return ssm::count_launches(a->y_dtype == SSM_BF16 ? ssm::run_w4<__nv_bfloat16>(*a, s) : ssm::run_w4<float>(*a, s));
}

int ssm_w4_quantize(int64_t N, int64_t K, int32_t group, int32_t w_dtype, const void* w, void* q, void* s, void* stream) {
    ssm::reset_launches();
    if (N < 0 || K < 0) return SSM_ERR_INVALID_ARG;
    if (!ssm::group_ok(group) || K % group != 0) return SSM_ERR_UNSUPPORTED;
    if (w_dtype != SSM_F32 && w_dtype != SSM_BF16) return SSM_ERR_UNSUPPORTED;
    if (N > (int64_t(1) << 31) || K > (int64_t(1) << 24)) return SSM_ERR_UNSUPPORTED;
    if (N == 0 || K == 0) return SSM_OK;
    if (!w || !q || !s) return SSM_ERR_INVALID_ARG;
    if (ssm::off(w, 16) || ssm::off(q, 16) || ssm::off(s, 2)) return SSM_ERR_ALIGNMENT;
    const int64_t count = N * (K / group), want = (count + 7) / 8, most = 16 * (int64_t)ssm::sm_count();
    const unsigned grid = (unsigned)(want < most ? want : most);
    cudaStream_t st = (cudaStream_t)stream;
    if (w_dtype == SSM_BF16)
        ssm::w4_quantize_kernel<<<grid, 256, 0, st>>>(count, group, static_cast<const __nv_bfloat16*>(w), static_cast<uint8_t*>(q),
                                                    static_cast<__nv_bfloat16*>(s));
    else
        ssm::w4_quantize_kernel<<<grid, 256, 0, st>>>(count, group, static_cast<const float*>(w), static_cast<uint8_t*>(q),
                                                    static_cast<__nv_bfloat16*>(s));
    return ssm::count_launches(ssm::launched());
}

}  // extern "C"
