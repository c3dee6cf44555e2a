// attn_vec.cuh -- arithmetic on pairs of floats (one instruction for two on sm_100), and the 16-byte chunks of rows that
// lanes of the query / key prologue hold.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace gdr2 {

// Two floats in one 64-bit register pair.
struct F2 {
    uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void split(F2 x, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v)); }
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 neg(F2 x) {
    F2 r;
    r.v = x.v ^ 0x8000000080000000ull;
    return r;
}
__device__ __forceinline__ float sum2(F2 x) {
    float a, b;
    split(x, a, b);
    return a + b;
}

// Two 16-byte chunks of a row in the order in which a rotation takes them: u[i], v[i] are rotated into one another.
// Half layout: u is the first chunk, v the second. Interleaved: u has the even elements of both chunks and v the odd ones
// (a bf16 element is taken out of its word one by one anyway, so the order is free; with neighbours kept together and
// swapped in registers the backward of 16 + 16 interleaved bf16 heads of 128, 150 MB of rows, took 87 us instead of 71).
template <typename T, bool kInter> struct Chunks {
    static constexpr int kElems = 16 / sizeof(T), kPairs = kElems / 2, kHalf = kPairs / 2;  // of one chunk
    static __device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
    static __device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
    static __device__ __forceinline__ uint32_t bf16_pack(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ void get(uint4 a, uint4 b, F2 (&u)[kPairs], F2 (&v)[kPairs]) {
        const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            if constexpr (kInter) {
                const uint32_t *w = (i < kHalf ? x : y) + (sizeof(T) == 2 ? 2 * (i % kHalf) : 0);
                if constexpr (sizeof(T) == 2)
                    u[i] = f2(bf16_lo(w[0]), bf16_lo(w[1])), v[i] = f2(bf16_hi(w[0]), bf16_hi(w[1]));
                else
                    u[i] = f2(__uint_as_float(w[0]), __uint_as_float(w[2])), v[i] = f2(__uint_as_float(w[1]), __uint_as_float(w[3]));
            } else if constexpr (sizeof(T) == 2) {
                u[i] = f2(bf16_lo(x[i]), bf16_hi(x[i])), v[i] = f2(bf16_lo(y[i]), bf16_hi(y[i]));
            } else {
                u[i] = f2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
                v[i] = f2(__uint_as_float(y[2 * i]), __uint_as_float(y[2 * i + 1]));
            }
        }
    }
    static __device__ __forceinline__ void put(T *p, T *q, const F2 (&u)[kPairs], const F2 (&v)[kPairs]) {
        uint32_t x[4], y[4];
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            float u0, u1, v0, v1;
            split(u[i], u0, u1);
            split(v[i], v0, v1);
            if constexpr (kInter) {
                uint32_t *w = (i < kHalf ? x : y) + (sizeof(T) == 2 ? 2 * (i % kHalf) : 0);
                if constexpr (sizeof(T) == 2) {
                    w[0] = bf16_pack(u0, v0), w[1] = bf16_pack(u1, v1);
                } else {
                    w[0] = __float_as_uint(u0), w[1] = __float_as_uint(v0);
                    w[2] = __float_as_uint(u1), w[3] = __float_as_uint(v1);
                }
            } else if constexpr (sizeof(T) == 2) {
                x[i] = bf16_pack(u0, u1), y[i] = bf16_pack(v0, v1);
            } else {
                x[2 * i] = __float_as_uint(u0), x[2 * i + 1] = __float_as_uint(u1);
                y[2 * i] = __float_as_uint(v0), y[2 * i + 1] = __float_as_uint(v1);
            }
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<uint4 *>(q) = make_uint4(y[0], y[1], y[2], y[3]);
    }
    // Where element e of a row's table of floats stands so that u and v of a chunk are runs of it (`pairs` below).
    static __device__ __forceinline__ int place(int e) {
        return kInter ? (e & ~(kElems - 1)) + (e & 1) * (kElems / 2) + (e & (kElems - 1)) / 2 : e;
    }
    // u and v out of a table of floats in that order, the chunks at p and q (16-byte aligned).
    static __device__ __forceinline__ void pairs(const float *p, const float *q, F2 (&u)[kPairs], F2 (&v)[kPairs]) {
        if constexpr (kInter) {
            load<kHalf>(p, u), load<kHalf>(q, u + kHalf);
            load<kHalf>(p + kPairs, v), load<kHalf>(q + kPairs, v + kHalf);
        } else {
            load<kPairs>(p, u), load<kPairs>(q, v);
        }
    }
    template <int M> static __device__ __forceinline__ void load(const float *p, F2 *w) {  // p: 8 M-byte aligned, 16 at most
        if constexpr (M == 1) {
            const float2 a = *reinterpret_cast<const float2 *>(p);
            w[0] = f2(a.x, a.y);
        } else {
#pragma unroll
            for (int i = 0; i < M; i += 2) {
                const float4 a = *reinterpret_cast<const float4 *>(p + 2 * i);
                w[i] = f2(a.x, a.y), w[i + 1] = f2(a.z, a.w);
            }
        }
    }
    // The element of the row that component k of u[i] (v: odd) stands for, the chunks at elements at0 and at1.
    static __device__ __forceinline__ int element(int i, int k, bool odd, int at0, int at1) {
        if constexpr (kInter) return (i < kHalf ? at0 : at1) + 4 * (i % kHalf) + 2 * k + odd;
        return (odd ? at1 : at0) + 2 * i + k;
    }
};

}  // namespace gdr2
