// Rows of fp32 or bf16 values read and written by groups of T threads, eight
// elements a thread at a time: shared by layer norm and the embedding.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ssm_common.cuh"

namespace ssm {

// Which elements of a chunk of 8 T are a thread's, so that a warp's access is
// one run of memory: eight in a row (bf16, 16 bytes), four in a row and four
// more 4 T further on (fp32, 16 bytes; bf16 beside fp32), two in a row and so
// on (fp32, 8 bytes), or every T-th.
enum class Layout { kOct, kQuad, kPair, kEach };
template <typename IO> constexpr Layout kVector = sizeof(IO) == 2 ? Layout::kOct : Layout::kQuad;

template <Layout L, int T> __device__ __forceinline__ int64_t column(int64_t c0, int t, int i) {
    return L == Layout::kOct ? c0 + 8 * t + i : L == Layout::kQuad ? c0 + 4 * t + (i & 3) + (i >> 2) * (4 * T) : c0 + i * T + t;
}

__device__ __forceinline__ void unpack2(unsigned u, float& a, float& b) {
    a = __uint_as_float(u << 16);
    b = __uint_as_float(u & 0xffff0000u);
}
__device__ __forceinline__ unsigned pack2(float a, float b) {
    const __nv_bfloat162 q = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const unsigned*>(&q);
}

// A thread's eight elements of the chunk that starts at column c0 of a row of
// D; elements from D on read as zero (by the second form of take as `fill`) and
// are not written. load reads global memory, take a row in shared memory (or,
// element by element, either).
template <typename IO, Layout L, int T> struct Chunk;
template <int T> struct Chunk<__nv_bfloat16, Layout::kOct, T> {
    uint4 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* row, int64_t D, int64_t c0, int t) {
        const int64_t e = c0 + 8 * t;
        v = e < D ? __ldg(reinterpret_cast<const uint4*>(row + e)) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void take(const __nv_bfloat16* row, int D, int c0, int t) {
        const int e = c0 + 8 * t;
        v = e < D ? *reinterpret_cast<const uint4*>(row + e) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        unpack2(v.x, f[0], f[1]), unpack2(v.y, f[2], f[3]), unpack2(v.z, f[4], f[5]), unpack2(v.w, f[6], f[7]);
    }
    __device__ __forceinline__ static void store(__nv_bfloat16* row, int64_t D, int64_t c0, int t, const float (&f)[8]) {
        const int64_t e = c0 + 8 * t;
        if (e < D)
            *reinterpret_cast<uint4*>(row + e) = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
    }
};
template <int T> struct Chunk<__nv_bfloat16, Layout::kQuad, T> {
    uint2 v[2];
    __device__ __forceinline__ void load(const __nv_bfloat16* row, int64_t D, int64_t c0, int t) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t e = c0 + 4 * t + 4 * T * i;
            v[i] = e < D ? __ldg(reinterpret_cast<const uint2*>(row + e)) : make_uint2(0, 0);
        }
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        unpack2(v[0].x, f[0], f[1]), unpack2(v[0].y, f[2], f[3]), unpack2(v[1].x, f[4], f[5]), unpack2(v[1].y, f[6], f[7]);
    }
};
template <int T> struct Chunk<float, Layout::kQuad, T> {
    float4 v[2];
    __device__ __forceinline__ void load(const float* row, int64_t D, int64_t c0, int t) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t e = c0 + 4 * t + 4 * T * i;
            v[i] = e < D ? __ldg(reinterpret_cast<const float4*>(row + e)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    __device__ __forceinline__ void take(const float* row, int D, int c0, int t) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = c0 + 4 * t + 4 * T * i;
            v[i] = e < D ? *reinterpret_cast<const float4*>(row + e) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    __device__ __forceinline__ void take(const float* row, int D, int c0, int t, float fill) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = c0 + 4 * t + 4 * T * i;
            v[i] = e < D ? *reinterpret_cast<const float4*>(row + e) : make_float4(fill, fill, fill, fill);
        }
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) f[4 * i] = v[i].x, f[4 * i + 1] = v[i].y, f[4 * i + 2] = v[i].z, f[4 * i + 3] = v[i].w;
    }
    __device__ __forceinline__ static void store(float* row, int64_t D, int64_t c0, int t, const float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t e = c0 + 4 * t + 4 * T * i;
            if (e < D) *reinterpret_cast<float4*>(row + e) = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
        }
    }
};
template <int T> struct Chunk<float, Layout::kPair, T> {
    float2 v[4];
    __device__ __forceinline__ void load(const float* row, int64_t D, int64_t c0, int t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t e = c0 + 2 * t + 2 * T * i;
            v[i] = e < D ? __ldg(reinterpret_cast<const float2*>(row + e)) : make_float2(0.f, 0.f);
        }
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[2 * i] = v[i].x, f[2 * i + 1] = v[i].y;
    }
    __device__ __forceinline__ static void store(float* row, int64_t D, int64_t c0, int t, const float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t e = c0 + 2 * t + 2 * T * i;
            if (e < D) *reinterpret_cast<float2*>(row + e) = make_float2(f[2 * i], f[2 * i + 1]);
        }
    }
};
template <typename IO, int T> struct Chunk<IO, Layout::kEach, T> {
    IO v[8];
    __device__ __forceinline__ void load(const IO* row, int64_t D, int64_t c0, int t) {
        const IO* q = row + c0 + t;
        const int left = (int)min64(D - c0 - t, 8 * T);  // element i is there if i T < left
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i * T < left ? q[i * T] : IOT<IO>::from_f(0.f);
    }
    __device__ __forceinline__ void take(const IO* row, int D, int c0, int t) { load(row, D, c0, t); }
    __device__ __forceinline__ void take(const IO* row, int D, int c0, int t, IO fill) {
        const IO* q = row + c0 + t;
        const int left = (int)min64((int64_t)D - c0 - t, 8 * T);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i * T < left ? q[i * T] : fill;
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = IOT<IO>::to_f(v[i]);
    }
    __device__ __forceinline__ static void store(IO* row, int64_t D, int64_t c0, int t, const float (&f)[8]) {
        IO* q = row + c0 + t;
        const int left = (int)min64(D - c0 - t, 8 * T);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i * T < left) q[i * T] = IOT<IO>::from_f(f[i]);
    }
};

}  // namespace ssm
