// attn_vec.cuh -- arithmetic on pairs of floats (one instruction for two on sm_100), and the 16-byte chunks of rows that
// lanes of the query / key prologue hold, kept as loaded (bf16 packed two to a register) until they are converted.
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
__device__ __forceinline__ F2 swap(F2 x) {
    float a, b;
    split(x, a, b);
    return f2(b, a);
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

// One 16-byte chunk of a row: kPairs pairs of consecutive elements.
template <typename T> struct Chunk {
    static constexpr int kElems = 16 / sizeof(T), kPairs = kElems / 2;
    uint4 v;
    __device__ __forceinline__ void put(T *p) const { *reinterpret_cast<uint4 *>(p) = v; }
    __device__ __forceinline__ void get(F2 (&x)[kPairs]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            if constexpr (sizeof(T) == 2)
                x[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
            else
                x[i] = f2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        }
    }
    static __device__ __forceinline__ void store(T *p, const F2 (&x)[kPairs]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            float a, b;
            split(x[i], a, b);
            if constexpr (sizeof(T) == 2) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                w[2 * i] = __float_as_uint(a), w[2 * i + 1] = __float_as_uint(b);
            }
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

}  // namespace gdr2
