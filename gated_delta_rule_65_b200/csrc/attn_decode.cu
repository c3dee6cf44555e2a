// attn_decode.cu -- softmax attention of one new token per sequence over the paged key-value cache (sm_100a).
//
// Per query head j of sequence n, over the tokens i of its window that are on a page of the cache:
//   s_i = scale q.k_i,  m = max s_i,  p_i = exp(s_i - m),  l = sum p_i,  o = sum p_i v_i / l,  lse = m + ln l;
// o = 0 and lse = -inf where no token is left. All statistics, sums and the output's accumulator are fp32; scores are
// kept in units of log2 (scale log2(e)) so that p is one exp2.
//
// Bound: each K and V element is read once and used 2 G times (G = Hq / Hk query heads of a KV head), G operations a
// byte of bf16 against the 250 of the GPU's balance, so HBM bounds the step for every head layout and the M = 128
// tiles of tcgen05 would be at most an eighth full. The products run on warp-level m16n8k16 matrix instructions
// instead, whose sixteen rows hold the query heads of a KV head; at 6.5 TB/s they are busy less than a tenth of the
// time. Up to 8 heads leave half the rows free: there the eight upper rows carry the low halves of p (p = hi + lo in
// bf16), so that rounding p costs 2^-17 and no further instruction. 9 to 16 heads take a second product for lo.
// fp32 caches run the same schedule on fp32 multiply-adds (tf32 products would lose 13 bits).
//
// Work split: the tiles (64 tokens for bf16, 32 for fp32) of all (sequence, KV head) rows lie on one line, and each
// CTA takes an equal run of it, whatever the lengths: one long sequence spreads over the whole GPU, a ragged batch
// leaves no CTA idle, and a row that lies in one CTA is finished there. Rows cut by a border leave (m, l, o) in the
// workspace, and a second kernel joins them in the order of the line: no atomics, the same bits every call. The split
// depends on the lengths alone, which only the GPU reads (a captured graph stays valid as sequences grow).
//
// Inside a CTA each of 4 warps takes a quarter of every tile through its own ring of cp.async stages (24 KB) with its
// own (m, l, o), so the main loop has no barrier; the warps' results meet at the end of a row.
#include <math.h>

#include "attn.h"
#include "common.cuh"
#include "kernels.h"

namespace gdr2 {
namespace {

constexpr int kCtas = 2 * kAttnSms;  // CTAs of the line: two resident per SM
constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kRing = 24 * 1024;     // bytes of a warp's stages
constexpr int kMaxRows = 16;         // query heads of a row of the line
constexpr float kLn2 = 0.69314718055994530942f, kLog2e = 1.4426950408889634074f;

// Workspace: per CTA two partial rows (0: a row begun by an earlier CTA, 1: a row that goes on in the next) with their
// (m, l) pairs, and the ids of those rows (-1: none).
struct Partials {
    float *o, *ml;
    int *row;
};
__host__ __device__ inline size_t partial_floats(int d) { return (size_t)kCtas * 2 * kMaxRows * d; }
inline Partials partials(void *ws, int d) {
    Partials w;
    w.o = static_cast<float *>(ws);
    w.ml = w.o + partial_floats(d);
    w.row = reinterpret_cast<int *>(w.ml + (size_t)kCtas * 2 * kMaxRows * 2);
    return w;
}

__device__ __forceinline__ uint32_t sptr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int bytes) {  // bytes 0: zeros, nothing is read
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&b);
}
__device__ __forceinline__ float2 unpack2(uint32_t w) { return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w)); }
// 2^(x - m) with m = -inf standing for "no token yet" (then x = -inf too, and the result is 0, not NaN).
__device__ __forceinline__ float pow2_rel(float x, float m) { return exp2f(x - (m == -INFINITY ? 0.f : m)); }

// What the line is made of. A row: (sequence n, KV head h, block of up to `rows` of its query heads).
struct Line {
    int G, nb, HG, rows;  // query heads of a KV head, blocks of them, rows of a sequence, heads of a block
};

// The span of sequence n that is attended: tokens [start, len); false for a slot without a sequence.
__device__ __forceinline__ bool span_of(const AttnDecodeArgs &p, int n, int &s, int &start, int &len) {
    s = p.seq ? p.seq[n] : n;
    start = len = 0;
    if (s < 0 || s >= p.R) return false;
    const long long cap = (long long)p.P * p.page_size;
    long long x = p.lens[s];
    x = x < 0 ? 0 : x > cap ? cap : x;
    len = (int)x;
    start = p.window > 0 && len > p.window ? len - p.window : 0;
    return true;
}

// A place on the line: tile t of the nt tiles of row hg of sequence n.
template <int TILE> struct Place {
    int n, hg, t, nt, start, len;
    const int *pages;
    __device__ __forceinline__ void enter(const AttnDecodeArgs &p) {
        int s;
        span_of(p, n, s, start, len);
        nt = (len - start + TILE - 1) / TILE;
        pages = p.table + (size_t)(nt > 0 ? s : 0) * p.P;
    }
    __device__ __forceinline__ void next(const AttnDecodeArgs &p, int HG) {  // not past the line's end
        if (++t < nt) return;
        t = 0;
        if (++hg < HG) return;
        hg = 0;
        do {
            ++n;
            if (n >= p.N) return;
            enter(p);
        } while (nt == 0);
    }
};

// The products of one warp's tile, bf16: rows of 16 query heads against 16 tokens.
template <int D, bool kPacked> struct Bf16Math {
    using T = __nv_bfloat16;
    static constexpr int kTok = 16, kRows = kPacked ? 8 : 16, kRowBytes = 2 * D;
    uint32_t a[D / 16][4];
    float o[D / 8][4], m[2], l[2];
    static __device__ __forceinline__ int swizzle(int row) { return row & 7; }
    __device__ __forceinline__ void begin(const T *q, int heads, float *, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int row = g + (x & 1) * 8, k = ks * 16 + (x >> 1) * 8 + 2 * t;
                a[ks][x] = row < heads ? *reinterpret_cast<const uint32_t *>(q + (size_t)row * D + k) : 0u;
            }
#pragma unroll
        for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
    }
    __device__ __forceinline__ void step(uint32_t sk, uint32_t sv, uint32_t on, float sc, const float *, float *, int lane) {
        const int t = lane & 3, mi = lane >> 3, r = lane & 7;
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        {
            const int tok = (mi >> 1) * 8 + r;
            const uint32_t base = sk + tok * kRowBytes;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t b[4];
                ldsm4(base + (((2 * ks + (mi & 1)) ^ swizzle(tok)) << 4), b);
                mma(s[0], a[ks], b[0], b[1]);
                mma(s[1], a[ks], b[2], b[3]);
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                s[j][x] *= sc;
                if (!(on >> (8 * j + 2 * t + (x & 1)) & 1)) s[j][x] = -INFINITY;
            }
        uint32_t hi[4], lo[4];
        float al[2];
#pragma unroll
        for (int h = 0; h < (kPacked ? 1 : 2); ++h) {
            float mx = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            mx = fmaxf(mx, m[h]);
            al[h] = pow2_rel(m[h], mx);
            m[h] = mx;
            float pr[4];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int x = 0; x < 2; ++x) pr[2 * j + x] = pow2_rel(s[j][2 * h + x], mx);
            l[h] = l[h] * al[h] + ((pr[0] + pr[1]) + (pr[2] + pr[3]));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t u = pack2(pr[2 * j], pr[2 * j + 1]);
                const float2 f = unpack2(u);
                hi[2 * j + h] = u;
                lo[2 * j + h] = pack2(pr[2 * j] - f.x, pr[2 * j + 1] - f.y);
            }
        }
        if constexpr (kPacked) {
            al[1] = al[0];
            hi[1] = lo[0];  // the upper eight rows carry the low halves
            hi[3] = lo[2];
        }
        if (__any_sync(0xffffffffu, al[0] != 1.f || al[1] != 1.f)) {
#pragma unroll
            for (int j = 0; j < D / 8; ++j) {
                o[j][0] *= al[0], o[j][1] *= al[0];
                o[j][2] *= al[1], o[j][3] *= al[1];
            }
        }
        const int tok = (mi & 1) * 8 + r;
        const uint32_t base = sv + tok * kRowBytes;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            uint32_t b[4];
            ldsm4t(base + (((2 * j + (mi >> 1)) ^ swizzle(tok)) << 4), b);
            mma(o[2 * j], hi, b[0], b[1]);
            mma(o[2 * j + 1], hi, b[2], b[3]);
            if constexpr (!kPacked) {
                mma(o[2 * j], lo, b[0], b[1]);
                mma(o[2 * j + 1], lo, b[2], b[3]);
            }
        }
    }
    // The warp's statistics and columns [c0, c0 + D / 2) of its output, for the merge: wo [kRows][D / 2].
    __device__ __forceinline__ void stats(float *wm, float *wl, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int h = 0; h < (kPacked ? 1 : 2); ++h) {
            float x = l[h];
            x += __shfl_xor_sync(0xffffffffu, x, 1);
            x += __shfl_xor_sync(0xffffffffu, x, 2);
            if (t == 0) wm[g + 8 * h] = m[h], wl[g + 8 * h] = x;
        }
    }
    template <int HALF> __device__ __forceinline__ void put(float *wo, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            const float(&c)[4] = o[HALF * (D / 16) + j];
            if constexpr (kPacked) {
                *reinterpret_cast<float2 *>(wo + g * (D / 2) + 8 * j + 2 * t) = make_float2(c[0] + c[2], c[1] + c[3]);
            } else {
                *reinterpret_cast<float2 *>(wo + g * (D / 2) + 8 * j + 2 * t) = make_float2(c[0], c[1]);
                *reinterpret_cast<float2 *>(wo + (g + 8) * (D / 2) + 8 * j + 2 * t) = make_float2(c[2], c[3]);
            }
        }
    }
};

// The products of one warp's tile, fp32: GB query heads against 8 tokens. Scores: four lanes of a token take 16-byte
// chunks t, t + 4, ... of its row. Output: a lane owns four channels (d = 64: for every other token).
template <int D, int GB> struct F32Math {
    using T = float;
    static constexpr int kTok = 8, kRows = GB, kRowBytes = 4 * D;
    static constexpr int kPer = (GB + 3) / 4;   // heads whose statistics a lane keeps: t, t + 4
    static constexpr int kLanes = D / 4;        // lanes of an output row
    float4 o[GB];
    float m[kPer], l[kPer];
    // rows 2 i and 2 i + 1 share a quarter-warp's access to four neighbouring chunks: bit 2 keeps them apart
    static __device__ __forceinline__ int swizzle(int row) { return ((row & 1) << 2) | ((row >> 1) & 3); }
    __device__ __forceinline__ void begin(const T *q, int heads, float *sq, int) {
        for (int x = threadIdx.x; x < GB * D; x += kThreads) sq[x] = x / D < heads ? q[x] : 0.f;
#pragma unroll
        for (int h = 0; h < GB; ++h) o[h] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kPer; ++i) m[i] = -INFINITY, l[i] = 0.f;
        __syncthreads();
    }
    // sp: the warp's [GB][8] probabilities and [GB] factors
    __device__ __forceinline__ void step(uint32_t sk, uint32_t sv, uint32_t on, float sc, const float *sq, float *sp, int lane) {
        const int g = lane >> 2, t = lane & 3;
        const char *k = reinterpret_cast<const char *>(__cvta_shared_to_generic(sk)) + g * kRowBytes;
        const char *v = reinterpret_cast<const char *>(__cvta_shared_to_generic(sv));
        float s[GB];
#pragma unroll
        for (int h = 0; h < GB; ++h) s[h] = 0.f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const float4 kk = *reinterpret_cast<const float4 *>(k + (((t + 4 * i) ^ swizzle(g)) << 4));
#pragma unroll
            for (int h = 0; h < GB; ++h) {
                const float4 qq = *reinterpret_cast<const float4 *>(sq + h * D + 4 * (t + 4 * i));
                s[h] = fmaf(qq.x, kk.x, fmaf(qq.y, kk.y, fmaf(qq.z, kk.z, fmaf(qq.w, kk.w, s[h]))));
            }
        }
#pragma unroll
        for (int h = 0; h < GB; ++h) {
            s[h] += __shfl_xor_sync(0xffffffffu, s[h], 1);
            s[h] += __shfl_xor_sync(0xffffffffu, s[h], 2);
        }
        const bool seen = on >> g & 1;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            float x = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (4 * i + c < GB && t == c) x = s[4 * i + c < GB ? 4 * i + c : 0] * sc;
            if (!seen) x = -INFINITY;
            float mx = x;
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            mx = fmaxf(mx, m[i]);
            const float al = pow2_rel(m[i], mx), pr = pow2_rel(x, mx);
            m[i] = mx;
            l[i] = l[i] * al + pr;
            if (4 * i + t < GB) {
                sp[(4 * i + t) * 8 + g] = pr;
                if (g == 0) sp[GB * 8 + 4 * i + t] = al;
            }
        }
        __syncwarp();
        const int c = lane % kLanes, sub = lane / kLanes;
#pragma unroll
        for (int h = 0; h < GB; ++h) {
            const float al = sp[GB * 8 + h];
            o[h].x *= al, o[h].y *= al, o[h].z *= al, o[h].w *= al;
        }
#pragma unroll
        for (int i = 0; i < 8; i += 32 / kLanes) {
            const int tok = i + sub;
            const float4 vv = *reinterpret_cast<const float4 *>(v + tok * kRowBytes + ((c ^ swizzle(tok)) << 4));
#pragma unroll
            for (int h = 0; h < GB; ++h) {
                const float pr = sp[h * 8 + tok];
                o[h].x = fmaf(pr, vv.x, o[h].x), o[h].y = fmaf(pr, vv.y, o[h].y);
                o[h].z = fmaf(pr, vv.z, o[h].z), o[h].w = fmaf(pr, vv.w, o[h].w);
            }
        }
        __syncwarp();
    }
    __device__ __forceinline__ void stats(float *wm, float *wl, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            float x = l[i];
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
            if (g == 0 && 4 * i + t < GB) wm[4 * i + t] = m[i], wl[4 * i + t] = x;
        }
        if constexpr (D == 64) {
#pragma unroll
            for (int h = 0; h < GB; ++h) {
                o[h].x += __shfl_xor_sync(0xffffffffu, o[h].x, 16);
                o[h].y += __shfl_xor_sync(0xffffffffu, o[h].y, 16);
                o[h].z += __shfl_xor_sync(0xffffffffu, o[h].z, 16);
                o[h].w += __shfl_xor_sync(0xffffffffu, o[h].w, 16);
            }
        }
    }
    template <int HALF> __device__ __forceinline__ void put(float *wo, int lane) {
        const int c = lane - HALF * (D / 8);
        if (c < 0 || c >= D / 8) return;
#pragma unroll
        for (int h = 0; h < GB; ++h) *reinterpret_cast<float4 *>(wo + h * (D / 2) + 4 * c) = o[h];
    }
};

template <int D, typename M> struct Shared {
    static constexpr int kStage = 2 * M::kTok * M::kRowBytes, kStages = kRing / kStage;
    alignas(128) uint8_t ring[kWarps][kStages][kStage];
    float merge[kWarps][M::kRows][D / 2];
    float wm[kWarps][M::kRows], wl[kWarps][M::kRows];
    uint32_t on[kWarps][kStages];
    float q[sizeof(typename M::T) == 4 ? M::kRows * D : 4];
    float p[sizeof(typename M::T) == 4 ? kWarps : 1][sizeof(typename M::T) == 4 ? M::kRows * 9 : 1];
    long long scan[kWarps];
    long long at;
    int n0;
};

template <typename T> __device__ __forceinline__ void store_out(T *p, float4 v) { store4(p, v); }

// One row's result in this CTA from its warps' parts: finished (whole) or left in the workspace (slot).
template <int D, typename M, int HALF>
__device__ __forceinline__ void merge_half(Shared<D, M> &sh, M &math, typename M::T *o, float *lse, int heads,
                                           bool whole, float *part, float *ml, int warp, int lane) {
    if (HALF == 0) math.stats(sh.wm[warp], sh.wl[warp], lane);
    math.template put<HALF>(&sh.merge[warp][0][0], lane);
    __syncthreads();
    for (int x = threadIdx.x; x < M::kRows * (D / 8); x += kThreads) {
        const int row = x / (D / 8), c = 4 * (x % (D / 8));
        if (row >= heads) break;
        float mx = sh.wm[0][row];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, sh.wm[w][row]);
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = pow2_rel(sh.wm[w][row], mx);
            const float4 y = *reinterpret_cast<const float4 *>(&sh.merge[w][row][c]);
            s.x = fmaf(f, y.x, s.x), s.y = fmaf(f, y.y, s.y), s.z = fmaf(f, y.z, s.z), s.w = fmaf(f, y.w, s.w);
            l = fmaf(f, sh.wl[w][row], l);
        }
        const int col = HALF * (D / 2) + c;
        if (whole) {
            const float i = l == 0.f ? 0.f : 1.f / l;  // no token left: zeros
            store_out(o + (size_t)row * D + col, make_float4(s.x * i, s.y * i, s.z * i, s.w * i));
            if (HALF == 0 && c == 0 && lse) lse[row] = (mx + log2f(l)) * kLn2;
        } else {
            *reinterpret_cast<float4 *>(part + (size_t)row * D + col) = s;
            if (HALF == 0 && c == 0) ml[2 * row] = mx, ml[2 * row + 1] = l;
        }
    }
    __syncthreads();
}

template <int D, typename M>
__global__ void __launch_bounds__(kThreads, 2) attn_decode_kernel(AttnDecodeArgs p, Line ln, Partials w) {
    using T = typename M::T;
    using S = Shared<D, M>;
    constexpr int TILE = M::kTok * kWarps, CH = M::kRowBytes / 16;
    extern __shared__ __align__(128) uint8_t raw[];
    S &sh = *reinterpret_cast<S *>(raw);
    cudaTriggerProgrammaticLaunchCompletion();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // this CTA's run [begin, end) of the line: a prefix sum of the sequences' tiles, each thread a run of sequences
    const int per = (p.N + kThreads - 1) / kThreads;
    const int na = min(p.N, tid * per), ne = min(p.N, na + per);
    long long mine = 0;
    for (int n = na; n < ne; ++n) {
        int s, a, b;
        if (span_of(p, n, s, a, b)) mine += (b - a + TILE - 1) / TILE;
    }
    mine *= ln.HG;
    long long pre = mine;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, pre, x);
        if (lane >= x) pre += y;
    }
    if (lane == 31) sh.scan[warp] = pre;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int x = 0; x < kWarps; ++x) {
        if (x < warp) pre += sh.scan[x];
        total += sh.scan[x];
    }
    // (with fewer tiles than CTAs the first ones take one each: the join expects no empty CTA between two parts)
    const long long parts = min((long long)gridDim.x, total);
    const long long begin = blockIdx.x < parts ? total * blockIdx.x / parts : total;
    const long long end = blockIdx.x < parts ? total * (blockIdx.x + 1) / parts : total;
    if (begin < end && begin < pre && begin >= pre - mine) {
        long long at = pre - mine;
        for (int n = na; n < ne; ++n) {
            int s, a, b;
            if (!span_of(p, n, s, a, b)) continue;
            const long long nt = (long long)((b - a + TILE - 1) / TILE) * ln.HG;
            if (begin < at + nt) {
                sh.n0 = n;
                sh.at = begin - at;
                break;
            }
            at += nt;
        }
    }
    // sequences with nothing to attend
    for (int n = blockIdx.x; n < p.N; n += gridDim.x) {
        int s, a, b;
        if (!span_of(p, n, s, a, b) || b > a) continue;
        for (int x = tid; x < p.Hq * D / 4; x += kThreads)
            store_out(static_cast<T *>(p.o) + (size_t)n * p.Hq * D + 4 * x, make_float4(0.f, 0.f, 0.f, 0.f));
        if (p.lse)
            for (int x = tid; x < p.Hq; x += kThreads) p.lse[(size_t)n * p.Hq + x] = -INFINITY;
    }
    __syncthreads();
    if (begin >= end) {
        if (tid < 2) w.row[2 * blockIdx.x + tid] = -1;
        return;
    }

    Place<TILE> cur;
    cur.n = sh.n0;
    cur.enter(p);
    cur.hg = (int)(sh.at / cur.nt);
    cur.t = (int)(sh.at - (long long)cur.hg * cur.nt);
    Place<TILE> ahead = cur;
    long long xa = begin;  // the next tile to load
    int page = 0;          // the page of this lane's token of that tile, fetched one tile early
    auto fetch = [&]() {
        page = -1;
        if (xa < end && lane < M::kTok) {
            const int tok = ahead.start + ahead.t * TILE + warp * M::kTok + lane;
            if (tok < ahead.len) page = __ldg(ahead.pages + tok / p.page_size);
        }
    };
    const T *kp = static_cast<const T *>(p.k_pages), *vp = static_cast<const T *>(p.v_pages);
    auto issue = [&](int stage) {
        if (xa < end) {
            const int tok = ahead.start + ahead.t * TILE + warp * M::kTok + lane;
            const bool on = page >= 0 && page < p.num_pages;
            const uint32_t mask = __ballot_sync(0xffffffffu, on);
            if (lane == 0) sh.on[warp][stage] = mask;
            const int h = ahead.hg / ln.nb;
            const long long row = on ? ((long long)page * p.Hk + h) * p.page_size + tok % p.page_size : 0;
            const uint32_t dst = sptr(&sh.ring[warp][stage][0]);
#pragma unroll
            for (int i = 0; i < M::kTok * CH / 32; ++i) {
                const int x = i * 32 + lane, r = x / CH, c = x % CH;
                const long long rr = __shfl_sync(0xffffffffu, row, r);
                const int bytes = mask >> r & 1 ? 16 : 0;
                const size_t off = (size_t)rr * D + c * (16 / sizeof(T));
                const uint32_t d = dst + r * M::kRowBytes + ((c ^ M::swizzle(r)) << 4);
                cp16(d, kp + off, bytes);
                cp16(d + M::kTok * M::kRowBytes, vp + off, bytes);
            }
            ++xa;
            if (xa < end) ahead.next(p, ln.HG);
            fetch();
        }
        cp_commit();
    };
    fetch();
#pragma unroll 1
    for (int s = 0; s < S::kStages; ++s) issue(s);

    M math;
    const float sc = p.scale * kLog2e;
    int stage = 0, row0 = -1, row1 = -1, t0 = cur.t;
    bool fresh = true;
    for (long long x = begin; x < end; ++x) {
        const int h = cur.hg / ln.nb, blk = cur.hg - h * ln.nb;
        const int heads = min(ln.rows, ln.G - blk * ln.rows), j0 = h * ln.G + blk * ln.rows;
        if (fresh) {
            math.begin(static_cast<const T *>(p.q) + ((size_t)cur.n * p.Hq + j0) * D, heads, sh.q, lane);
            t0 = cur.t;
            fresh = false;
        }
        cp_wait<S::kStages - 1>();
        __syncwarp();
        const uint32_t sk = sptr(&sh.ring[warp][stage][0]);
        math.step(sk, sk + M::kTok * M::kRowBytes, sh.on[warp][stage], sc, sh.q,
                  sh.p[sizeof(T) == 4 ? warp : 0], lane);
        __syncwarp();
        issue(stage);
        if (++stage == S::kStages) stage = 0;
        if (cur.t + 1 == cur.nt || x + 1 == end) {
            const bool whole = t0 == 0 && cur.t + 1 == cur.nt;
            const int slot = 2 * blockIdx.x + (t0 == 0);
            if (!whole) (t0 == 0 ? row1 : row0) = cur.n * ln.HG + cur.hg;
            T *o = static_cast<T *>(p.o) + ((size_t)cur.n * p.Hq + j0) * D;
            float *lse = p.lse ? p.lse + (size_t)cur.n * p.Hq + j0 : nullptr;
            float *part = w.o + (size_t)slot * kMaxRows * D, *ml = w.ml + (size_t)slot * kMaxRows * 2;
            merge_half<D, M, 0>(sh, math, o, lse, heads, whole, part, ml, warp, lane);
            merge_half<D, M, 1>(sh, math, o, lse, heads, whole, part, ml, warp, lane);
            fresh = true;
        }
        if (x + 1 < end) cur.next(p, ln.HG);
    }
    cp_wait<0>();
    if (tid == 0) {
        w.row[2 * blockIdx.x] = row0;
        w.row[2 * blockIdx.x + 1] = row1;
    }
}

// Joins the parts of the row that begins in CTA blockIdx.x of the line and goes on in the next ones; block y takes
// one of its query heads. 256 threads: D / 4 lanes of four channels, 1024 / D groups that share the parts.
template <int D, typename T>
__global__ void __launch_bounds__(256) attn_decode_join_kernel(AttnDecodeArgs p, Line ln, Partials w, int ctas) {
    constexpr int LN = D / 4, NG = 256 / LN;
    __shared__ float4 so[NG][LN];
    __shared__ float sm[NG], sl[NG];
    __shared__ int last;
    cudaGridDependencySynchronize();
    const int c = blockIdx.x, head = blockIdx.y;
    const int row = __ldcg(w.row + 2 * c + 1);
    if (row < 0) return;
    const int n = row / ln.HG, hg = row - n * ln.HG, h = hg / ln.nb, blk = hg - h * ln.nb;
    if (head >= min(ln.rows, ln.G - blk * ln.rows)) return;
    // the parts: CTA c's second slot, then the first slots of the CTAs that follow with the same row
    if (threadIdx.x == 0) last = ctas;
    __syncthreads();
    for (int k = c + 1 + threadIdx.x; k < ctas; k += 256)
        if (__ldcg(w.row + 2 * k) != row) {
            atomicMin(&last, k);
            break;
        }
    __syncthreads();
    const int cnt = last - c, lane = threadIdx.x % LN, grp = threadIdx.x / LN;
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float m1, float l1, const float4 &o1) {
        const float mx = fmaxf(m, m1), f = pow2_rel(m, mx), g = pow2_rel(m1, mx);
        o.x = o.x * f + o1.x * g, o.y = o.y * f + o1.y * g, o.z = o.z * f + o1.z * g, o.w = o.w * f + o1.w * g;
        l = l * f + l1 * g;
        m = mx;
    };
#pragma unroll 4
    for (int i = grp; i < cnt; i += NG) {
        const size_t slot = (size_t)2 * (c + i) + (i == 0);
        const float2 ml = __ldcg(reinterpret_cast<const float2 *>(w.ml + (slot * kMaxRows + head) * 2));
        add(ml.x, ml.y, __ldcg(reinterpret_cast<const float4 *>(w.o + (slot * kMaxRows + head) * D + 4 * lane)));
    }
    so[grp][lane] = o;
    if (lane == 0) sm[grp] = m, sl[grp] = l;
    __syncthreads();
    if (grp != 0) return;
#pragma unroll
    for (int g = 1; g < NG; ++g) add(sm[g], sl[g], so[g][lane]);
    const size_t j = (size_t)n * p.Hq + h * ln.G + blk * ln.rows + head;
    const float i = l == 0.f ? 0.f : 1.f / l;
    store_out(static_cast<T *>(p.o) + j * D + 4 * lane, make_float4(o.x * i, o.y * i, o.z * i, o.w * i));
    if (lane == 0 && p.lse) p.lse[j] = (m + log2f(l)) * kLn2;
}

template <int D, typename M> cudaError_t run(const AttnDecodeArgs &a, cudaStream_t st) {
    using T = typename M::T;
    constexpr int TILE = M::kTok * kWarps;
    constexpr int smem = (int)sizeof(Shared<D, M>);
    static_assert(smem <= 113 * 1024, "two CTAs on an SM");
    Line ln;
    ln.G = a.Hq / a.Hk;
    ln.rows = M::kRows;
    ln.nb = (ln.G + M::kRows - 1) / M::kRows;
    ln.HG = a.Hk * ln.nb;
    cudaError_t e = cudaFuncSetAttribute(attn_decode_kernel<D, M>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // no more CTAs than the largest possible line has tiles
    long long span = (long long)a.P * a.page_size;
    if (a.window > 0 && a.window < span) span = a.window;
    const long long tiles = (long long)a.N * ln.HG * ((span + TILE - 1) / TILE);
    const int ctas = tiles < kCtas ? (int)tiles : kCtas;
    const Partials w = partials(a.workspace, D);
    GDR2_LAUNCH("attn_decode", st, (attn_decode_kernel<D, M><<<ctas, kThreads, smem, st>>>(a, ln, w)));
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int heads = ln.G < ln.rows ? ln.G : ln.rows;
    GDR2_LAUNCH("attn_decode_join", st,
                e = launch_dependent(attn_decode_join_kernel<D, T>, dim3(ctas, heads), dim3(256), 0, st, a, ln, w, ctas));
    return e;
}

template <int D> cudaError_t dispatch(const AttnDecodeArgs &a, cudaStream_t st) {
    const int G = a.Hq / a.Hk;
    if (a.dtype == 1) return G <= 8 ? run<D, Bf16Math<D, true>>(a, st) : run<D, Bf16Math<D, false>>(a, st);
    if (G == 1) return run<D, F32Math<D, 1>>(a, st);
    if (G == 2) return run<D, F32Math<D, 2>>(a, st);
    if (G <= 4) return run<D, F32Math<D, 4>>(a, st);
    return run<D, F32Math<D, 8>>(a, st);
}

}  // namespace

size_t attn_decode_workspace_bytes(int d) {
    return (partial_floats(d) + (size_t)kCtas * 2 * kMaxRows * 2) * sizeof(float) + (size_t)kCtas * 2 * sizeof(int);
}

cudaError_t launch_attn_decode(const AttnDecodeArgs &a, cudaStream_t st) {
    return a.d == 128 ? dispatch<128>(a, st) : dispatch<64>(a, st);
}

}  // namespace gdr2
