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
// instead, whose sixteen rows hold the query heads of a KV head; at 6.2 TB/s they are busy a fifth of the time. Up to 8
// heads leave half the rows free: there the eight upper rows carry the low halves of p (p = hi + lo in bf16), so that
// rounding p costs 2^-17 and no further instruction. 9 to 16 heads take a second product for lo.
// fp32 caches run the same schedule on fp32 multiply-adds (single tf32 products would lose 13 bits).
//
// Work split: the tiles (64 tokens; 32 for fp32 heads of 128) of all (sequence, KV head) rows lie on one line, and each
// CTA takes an equal run of it, whatever the lengths: one long sequence spreads over the whole GPU, a ragged batch
// leaves no CTA idle, and a row that lies in one CTA is finished there. More query heads of a KV head than one CTA holds
// go to neighbouring CTAs with the same run, which find each other's tiles in L2 (each block costs its own way of the
// tiles into the SM: 400 MB take 70 us with 16 bf16 heads of 128 on a KV head and 98 with 32). Rows cut by a border
// leave (m, l, o) in the workspace, and a second kernel joins them in the order of the line: no atomics, the same bits
// every call. The split depends on the lengths alone, which only the GPU reads (a captured graph stays valid as
// sequences grow).
//
// Inside a CTA each of 4 warps takes a quarter of every tile through its own ring of cp.async stages (16 KB) with its
// own (m, l, o), so the main loop has no barrier; the warps' results meet at the end of a row. Two CTAs to an SM for
// bf16 (three: 140 us against 133 below; a ring of 24 KB: 137), three for fp32, whose products leave more latency to
// cover (27 us against 29 below). Rows of at most 8 tiles are not cut: a single sequence of 333 tokens takes 9.0 us
// with its rows whole and 8.4 us cut and joined, but the second launch costs the host 3 us.
//
// Measured on one B200, back to back: 256 sequences of 100 to 4,096 tokens in a window of 2,048 (16 / 4 heads of 128,
// bf16, pages of 16) in 133 us (829 MB, 6.2 TB/s, 95% of the measured copy; 135 from call to call); 3 sequences of
// 50,001 to 65,536 tokens (16 / 2 heads) in 37 us (183 MB, 75%: about 7 us of it are the start, the end and the join);
// 33 ragged fp32 sequences of up to 2,000 tokens (12 / 6 heads of 64) in 26 us (107 MB, 63%).
#include <math.h>

#include "attn.h"
#include "attn_vec.cuh"
#include "common.cuh"
#include "kernels.h"

namespace gdr2 {
namespace {

constexpr int kMaxCtas = 3 * kAttnSms;  // CTAs of the line: two or three resident on an SM
constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kRing = 16 * 1024;        // bytes of a warp's stages
constexpr int kMaxRows = 16;            // query heads of a row of the line
constexpr int kWholeTiles = 8;          // rows of at most so many tiles are not cut
constexpr float kLn2 = 0.69314718055994530942f, kLog2e = 1.4426950408889634074f;

// Workspace: per CTA two partial rows (0: a row begun by an earlier CTA, 1: a row that goes on in the next) with their
// (m, l) pairs; and the rows that borders cut, (row, CTA where it begins, its runs), row -1: none. Their list is kept
// by row where the line has fewer rows than CTAs, else by the CTA where a row begins (at most one each).
struct Partials {
    float *o, *ml;
    int4 *cut;
    int by_row;
};
__host__ __device__ inline size_t partial_floats(int d) { return (size_t)kMaxCtas * 2 * kMaxRows * d; }
inline Partials partials(void *ws, int d) {
    Partials w;
    w.o = static_cast<float *>(ws);
    w.ml = w.o + partial_floats(d);
    w.cut = reinterpret_cast<int4 *>(w.ml + (size_t)kMaxCtas * 2 * kMaxRows * 2);
    w.by_row = 0;
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
// 2^x for the main loop: 2 steps of fp32, results below 2^-126 are zero (next to a maximum of 1 they are nothing).
__device__ __forceinline__ float pow2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What the line is made of: rows (sequence n, KV head h). CTA x takes run x / nb of it for block x % nb of up to `rows`
// of the row's query heads.
struct Line {
    int G, nb, rows;        // query heads of a KV head, blocks of them, heads of a block
    int whole;              // no row is cut
    Divisor by_page;
};

// The span of sequence n that is attended: tokens [start, len); false for a slot without a sequence.
__device__ __forceinline__ bool span_of(const AttnDecodeArgs &p, int n, int &s, int &start, int &len) {
    s = p.seq ? p.seq[n] : n;
    start = len = 0;
    if (s < 0 || s >= p.R) return false;
    len = min(max(p.lens[s], 0), p.P * p.page_size);
    start = p.window > 0 && len > p.window ? len - p.window : 0;
    return true;
}

// A place on the line: the tile of tokens [first, first + TILE) of KV head h of sequence n.
template <int TILE> struct Place {
    int n, h, first, start, len;
    const int *pages;
    __device__ __forceinline__ void enter(const AttnDecodeArgs &p) {
        int s;
        span_of(p, n, s, start, len);
        pages = p.table + (len > start ? (size_t)s * p.P : 0);
        first = start;
    }
    __device__ __forceinline__ bool last() const { return first + TILE >= len; }
    __device__ __forceinline__ void next(const AttnDecodeArgs &p) {  // not past the line's end
        first += TILE;
        if (first < len) return;
        first = start;
        if (++h < p.Hk) return;
        h = 0;
        do {
            if (++n >= p.N) return;
            enter(p);
        } while (len == start);
    }
};

// The products of one warp's tile, bf16: rows of 16 query heads against 16 tokens. m is the largest q.k so far (of the
// queries with the scale's sign), ms = m sc, p = 2^(q.k sc - ms) with sc = |scale| log2(e).
template <int D, bool kPacked> struct Bf16Math {
    using T = __nv_bfloat16;
    static constexpr int kTok = 16, kRows = kPacked ? 8 : 16, kRowBytes = 2 * D, kStats = kPacked ? 1 : 2, kPerSm = 2;
    static constexpr int kCols = D;  // columns merged at a time
    uint32_t a[D / 16][4];
    float o[D / 8][4], m[kStats], ms[kStats], l[kStats];
    static __device__ __forceinline__ int swizzle(int row) { return row & 7; }
    __device__ __forceinline__ void begin(const T *q, int heads, float scale, float *, int lane) {
        const int g = lane >> 2, t = lane & 3;
        const uint32_t sign = scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int row = g + (x & 1) * 8, k = ks * 16 + (x >> 1) * 8 + 2 * t;
                a[ks][x] = 0u;
                if (!(kPacked && (x & 1)) && row < heads && scale != 0.f)
                    a[ks][x] = *reinterpret_cast<const uint32_t *>(q + (size_t)row * D + k) ^ sign;
            }
#pragma unroll
        for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
#pragma unroll
        for (int h = 0; h < kStats; ++h) m[h] = -INFINITY, ms[h] = 0.f, l[h] = 0.f;
    }
    __device__ __forceinline__ void step(uint32_t stage, uint32_t on, float sc, const float *, float *, int lane) {
        const int t = lane & 3, mi = lane >> 3, r = lane & 7;
        // stages start at multiples of 256 bytes, so a chunk's place is an exclusive or away from the lane's first one
        const uint32_t ka = stage + ((mi >> 1) * 8 + r) * kRowBytes + (((mi & 1) ^ r) << 4);
        const uint32_t va = stage + kTok * kRowBytes + ((mi & 1) * 8 + r) * kRowBytes + (((mi >> 1) ^ r) << 4);
        float s[2][4], s2[2][4];  // two chains of products: their latency, not their rate, would show
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int x = 0; x < 4; ++x) s[j][x] = s2[j][x] = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            uint32_t b[4];
            ldsm4(ka ^ (ks << 5), b);
            mma(ks & 1 ? s2[0] : s[0], a[ks], b[0], b[1]);
            mma(ks & 1 ? s2[1] : s[1], a[ks], b[2], b[3]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int x = 0; x < 2 * kStats; ++x) s[j][x] += s2[j][x];
        if (on != 0xffffu) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int x = 0; x < 2 * kStats; ++x)
                    if (!(on >> (8 * j + 2 * t + (x & 1)) & 1)) s[j][x] = -INFINITY;
        }
        uint32_t hi[4], lo[4];
        float al[2];
#pragma unroll
        for (int h = 0; h < kStats; ++h) {
            float mx = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            mx = fmaxf(mx, m[h]);
            const float was = m[h] == -INFINITY ? -INFINITY : ms[h];
            m[h] = mx;
            ms[h] = mx == -INFINITY ? 0.f : mx * sc;
            al[h] = pow2(was - ms[h]);
            float pr[4];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int x = 0; x < 2; ++x) pr[2 * j + x] = pow2(fmaf(s[j][2 * h + x], sc, -ms[h]));
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
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
            uint32_t b[4];
            ldsm4t(va ^ (j << 5), b);
            mma(o[2 * j], hi, b[0], b[1]);
            mma(o[2 * j + 1], hi, b[2], b[3]);
            if constexpr (!kPacked) {
                mma(o[2 * j], lo, b[0], b[1]);
                mma(o[2 * j + 1], lo, b[2], b[3]);
            }
        }
    }
    // The warp's statistics (m in units of log2), and columns [C0, C0 + kCols) of its output, for the merge: wo [kRows][kCols].
    __device__ __forceinline__ void stats(float *wm, float *wl, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int h = 0; h < kStats; ++h) {
            float x = l[h];
            x += __shfl_xor_sync(0xffffffffu, x, 1);
            x += __shfl_xor_sync(0xffffffffu, x, 2);
            if (t == 0) wm[g + 8 * h] = m[h] == -INFINITY ? -INFINITY : ms[h], wl[g + 8 * h] = x;
        }
    }
    template <int C0> __device__ __forceinline__ void put(float *wo, int lane) {
        const int g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int j = 0; j < kCols / 8; ++j) {
            const float(&c)[4] = o[C0 / 8 + j];
            if constexpr (kPacked) {
                *reinterpret_cast<float2 *>(wo + g * kCols + 8 * j + 2 * t) = make_float2(c[0] + c[2], c[1] + c[3]);
            } else {
                *reinterpret_cast<float2 *>(wo + g * kCols + 8 * j + 2 * t) = make_float2(c[0], c[1]);
                *reinterpret_cast<float2 *>(wo + (g + 8) * kCols + 8 * j + 2 * t) = make_float2(c[2], c[3]);
            }
        }
    }
};

// The products of one warp's tile, fp32: GB <= 4 query heads against kTok tokens (4 KB of K), on pairs of floats. Scores:
// four lanes of a token take 16-byte chunks t, t + 4, ... of its row, each lane one token of every eight, and the exchange
// that adds their parts leaves lane t with head t. Output: a lane owns four channels (d = 64: of every other
// token).
template <int D, int GB> struct F32Math {
    using T = float;
    static constexpr int kTok = 1024 / D, kRows = GB, kRowBytes = 4 * D, kPer = kTok / 8, kPerSm = 3;
    static constexpr int kCols = D / 2;  // columns merged at a time: all of them leave no room for a third CTA
    static constexpr int kLanes = D / 4;   // lanes of an output row
    static_assert(GB <= 4, "a lane keeps the statistics of one head");
    F2 o[GB][2];
    float m, ms, l;
    // rows 2 i and 2 i + 1 share a quarter-warp's access to four neighbouring chunks: bit 2 keeps them apart
    static __device__ __forceinline__ int swizzle(int row) { return ((row & 1) << 2) | ((row >> 1) & 3); }
    static __device__ __forceinline__ void load(const void *p, F2 (&x)[2]) {
        const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(p);
        x[0].v = v.x, x[1].v = v.y;
    }
    __device__ __forceinline__ void begin(const T *q, int heads, float scale, float *sq, int) {
        const float sign = scale < 0.f ? -1.f : scale == 0.f ? 0.f : 1.f;
        for (int x = threadIdx.x; x < GB * D; x += kThreads) sq[x] = x / D < heads && scale != 0.f ? sign * q[x] : 0.f;
#pragma unroll
        for (int h = 0; h < GB; ++h) o[h][0] = o[h][1] = f2(0.f, 0.f);
        m = -INFINITY, ms = 0.f, l = 0.f;
        __syncthreads();
    }
    // Sums over the four lanes of a token of four heads' parts; lane t gets head t's.
    static __device__ __forceinline__ float spread(float a0, float a1, float a2, float a3, int t) {
        const bool b0 = t & 1, b1 = t & 2;
        float x = b0 ? a1 : a0, y = b0 ? a3 : a2;
        x += __shfl_xor_sync(0xffffffffu, b0 ? a0 : a1, 1);
        y += __shfl_xor_sync(0xffffffffu, b0 ? a2 : a3, 1);
        const float z = b1 ? y : x;
        return z + __shfl_xor_sync(0xffffffffu, b1 ? x : y, 2);
    }
    // sp: the warp's probabilities [kTok][GB] and factors [GB], each twice side by side
    __device__ __forceinline__ void step(uint32_t stage, uint32_t on, float sc, const float *sq, float *sp, int lane) {
        const int g = lane >> 2, t = lane & 3;
        const char *k = reinterpret_cast<const char *>(__cvta_shared_to_generic(stage)) + g * kRowBytes;
        const char *v = reinterpret_cast<const char *>(__cvta_shared_to_generic(stage)) + kTok * kRowBytes;
        float2 *pp = reinterpret_cast<float2 *>(sp);
        F2 s[kPer][GB];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            F2 kk[kPer][2];
#pragma unroll
            for (int y = 0; y < kPer; ++y) load(k + y * 8 * kRowBytes + (((t + 4 * i) ^ swizzle(g)) << 4), kk[y]);
#pragma unroll
            for (int h = 0; h < GB; ++h) {
                F2 qq[2];
                load(sq + h * D + 4 * (t + 4 * i), qq);
#pragma unroll
                for (int y = 0; y < kPer; ++y)
                    s[y][h] = fma(qq[1], kk[y][1], i ? fma(qq[0], kk[y][0], s[y][h]) : mul(qq[0], kk[y][0]));
            }
        }
        float x[kPer], mx = m;
#pragma unroll
        for (int y = 0; y < kPer; ++y) {
            float a[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) a[c] = c < GB ? sum2(s[y][c < GB ? c : 0]) : 0.f;
            x[y] = spread(a[0], a[1], a[2], a[3], t);
            if (t >= GB || !(on >> (8 * y + g) & 1)) x[y] = -INFINITY;
            mx = fmaxf(mx, x[y]);
        }
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
        const float was = m == -INFINITY ? -INFINITY : ms;
        m = mx;
        ms = mx == -INFINITY ? 0.f : mx * sc;
        const float al = pow2(was - ms);
        l *= al;
#pragma unroll
        for (int y = 0; y < kPer; ++y) {
            const float pr = pow2(fmaf(x[y], sc, -ms));
            l += pr;
            if (t < GB) pp[(8 * y + g) * GB + t] = make_float2(pr, pr);
        }
        if (t < GB && g == 0) pp[kTok * GB + t] = make_float2(al, al);
        __syncwarp();
        if (__any_sync(0xffffffffu, t < GB && al != 1.f)) {
#pragma unroll
            for (int h = 0; h < GB; ++h) {
                F2 f;
                f.v = *reinterpret_cast<const unsigned long long *>(pp + kTok * GB + h);
                o[h][0] = mul(o[h][0], f), o[h][1] = mul(o[h][1], f);
            }
        }
        const int c = lane % kLanes, sub = lane / kLanes;
#pragma unroll
        for (int i = 0; i < kTok; i += 32 / kLanes) {
            const int tok = i + sub;
            F2 vv[2], pr[GB];
            load(v + tok * kRowBytes + ((c ^ swizzle(tok & 7)) << 4), vv);
            if constexpr (GB == 1) {
                pr[0].v = *reinterpret_cast<const unsigned long long *>(pp + tok);
            } else {
#pragma unroll
                for (int h = 0; h < GB; h += 2) {
                    F2 two[2];
                    load(pp + tok * GB + h, two);
                    pr[h] = two[0], pr[h + 1] = two[1];
                }
            }
#pragma unroll
            for (int h = 0; h < GB; ++h) o[h][0] = fma(pr[h], vv[0], o[h][0]), o[h][1] = fma(pr[h], vv[1], o[h][1]);
        }
        __syncwarp();
    }
    __device__ __forceinline__ void stats(float *wm, float *wl, int lane) {
        const int g = lane >> 2, t = lane & 3;
        float x = l;
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
        if (g == 0 && t < GB) wm[t] = m == -INFINITY ? -INFINITY : ms, wl[t] = x;
        if constexpr (D == 64) {
#pragma unroll
            for (int h = 0; h < GB; ++h)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    F2 y;
                    y.v = __shfl_xor_sync(0xffffffffu, o[h][x].v, 16);
                    o[h][x] = add(o[h][x], y);
                }
        }
    }
    template <int C0> __device__ __forceinline__ void put(float *wo, int lane) {
        const int c = lane - C0 / 4;
        if (c < 0 || c >= kCols / 4) return;
#pragma unroll
        for (int h = 0; h < GB; ++h)
            *reinterpret_cast<ulonglong2 *>(wo + h * kCols + 4 * c) = make_ulonglong2(o[h][0].v, o[h][1].v);
    }
};

// The same for eight query heads: eight lanes of a token instead of four, so that a lane's part of all eight queries
// stays in registers (with four lanes they come from shared memory again for every tile, a load for each two products:
// 98 us against 79 for 400 MB, heads of 128), and lane t keeps the statistics of head t.
template <int D> struct F32Math<D, 8> {
    using T = float;
    static constexpr int GB = 8, kTok = 1024 / D, kRows = GB, kRowBytes = 4 * D, kPer = kTok / 4, kPerSm = 2;
    static constexpr int kCols = D / 2, kLanes = D / 4, kChunks = D / 32;
    F2 o[GB][2], q[GB][kChunks][2];
    float m, ms, l;
    static __device__ __forceinline__ int swizzle(int row) { return row & 7; }
    static __device__ __forceinline__ void load(const void *p, F2 (&x)[2]) {
        const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(p);
        x[0].v = v.x, x[1].v = v.y;
    }
    __device__ __forceinline__ void begin(const T *qp, int heads, float scale, float *, int lane) {
        const F2 sign = f2(scale < 0.f ? -1.f : 1.f, scale < 0.f ? -1.f : 1.f);
#pragma unroll
        for (int h = 0; h < GB; ++h) {
            o[h][0] = o[h][1] = f2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                q[h][i][0] = q[h][i][1] = f2(0.f, 0.f);
                if (h < heads && scale != 0.f) {
                    load(qp + (size_t)h * D + 4 * ((lane & 7) + 8 * i), q[h][i]);
                    q[h][i][0] = mul(q[h][i][0], sign), q[h][i][1] = mul(q[h][i][1], sign);
                }
            }
        }
        m = -INFINITY, ms = 0.f, l = 0.f;
    }
    // Sums over the eight lanes of a token of eight heads' parts; lane t gets head t's.
    static __device__ __forceinline__ float spread(const float (&a)[8], int t) {
        float x[4], y[2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = (t & 1 ? a[2 * i + 1] : a[2 * i]) + __shfl_xor_sync(0xffffffffu, t & 1 ? a[2 * i] : a[2 * i + 1], 1);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            y[i] = (t & 2 ? x[2 * i + 1] : x[2 * i]) + __shfl_xor_sync(0xffffffffu, t & 2 ? x[2 * i] : x[2 * i + 1], 2);
        return (t & 4 ? y[1] : y[0]) + __shfl_xor_sync(0xffffffffu, t & 4 ? y[0] : y[1], 4);
    }
    __device__ __forceinline__ void step(uint32_t stage, uint32_t on, float sc, const float *, float *sp, int lane) {
        const int g = lane >> 3, t = lane & 7;
        const char *k = reinterpret_cast<const char *>(__cvta_shared_to_generic(stage));
        const char *v = k + kTok * kRowBytes;
        float2 *pp = reinterpret_cast<float2 *>(sp);
        float x[kPer], mx = m;
#pragma unroll
        for (int y = 0; y < kPer; ++y) {
            const int tok = 4 * y + g;
            F2 s[GB];
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {
                F2 kk[2];
                load(k + tok * kRowBytes + (((t + 8 * i) ^ swizzle(tok)) << 4), kk);
#pragma unroll
                for (int h = 0; h < GB; ++h) s[h] = fma(q[h][i][1], kk[1], i ? fma(q[h][i][0], kk[0], s[h]) : mul(q[h][i][0], kk[0]));
            }
            float a[GB];
#pragma unroll
            for (int h = 0; h < GB; ++h) a[h] = sum2(s[h]);
            x[y] = spread(a, t);
            if (!(on >> tok & 1)) x[y] = -INFINITY;
            mx = fmaxf(mx, x[y]);
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        const float was = m == -INFINITY ? -INFINITY : ms;
        m = mx;
        ms = mx == -INFINITY ? 0.f : mx * sc;
        const float al = pow2(was - ms);
        l *= al;
#pragma unroll
        for (int y = 0; y < kPer; ++y) {
            const float pr = pow2(fmaf(x[y], sc, -ms));
            l += pr;
            pp[(4 * y + g) * GB + t] = make_float2(pr, pr);
        }
        if (g == 0) pp[kTok * GB + t] = make_float2(al, al);
        __syncwarp();
        if (__any_sync(0xffffffffu, al != 1.f)) {
#pragma unroll
            for (int h = 0; h < GB; ++h) {
                F2 f;
                f.v = *reinterpret_cast<const unsigned long long *>(pp + kTok * GB + h);
                o[h][0] = mul(o[h][0], f), o[h][1] = mul(o[h][1], f);
            }
        }
        const int c = lane % kLanes, sub = lane / kLanes;
#pragma unroll
        for (int i = 0; i < kTok; i += 32 / kLanes) {
            const int tok = i + sub;
            F2 vv[2], pr[GB];
            load(v + tok * kRowBytes + ((c ^ swizzle(tok & 7)) << 4), vv);
#pragma unroll
            for (int h = 0; h < GB; h += 2) {
                F2 two[2];
                load(pp + tok * GB + h, two);
                pr[h] = two[0], pr[h + 1] = two[1];
            }
#pragma unroll
            for (int h = 0; h < GB; ++h) o[h][0] = fma(pr[h], vv[0], o[h][0]), o[h][1] = fma(pr[h], vv[1], o[h][1]);
        }
        __syncwarp();
    }
    __device__ __forceinline__ void stats(float *wm, float *wl, int lane) {
        float x = l;
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (lane < 8) wm[lane] = m == -INFINITY ? -INFINITY : ms, wl[lane] = x;
        if constexpr (D == 64) {
#pragma unroll
            for (int h = 0; h < GB; ++h)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    F2 y;
                    y.v = __shfl_xor_sync(0xffffffffu, o[h][i].v, 16);
                    o[h][i] = add(o[h][i], y);
                }
        }
    }
    template <int C0> __device__ __forceinline__ void put(float *wo, int lane) {
        const int c = lane - C0 / 4;
        if (c < 0 || c >= kCols / 4) return;
#pragma unroll
        for (int h = 0; h < GB; ++h)
            *reinterpret_cast<ulonglong2 *>(wo + h * kCols + 4 * c) = make_ulonglong2(o[h][0].v, o[h][1].v);
    }
};

template <int D, typename M> struct Shared {
    static constexpr int kStage = 2 * M::kTok * M::kRowBytes, kStages = kRing / kStage;
    alignas(1024) uint8_t ring[kWarps][kStages][kStage];
    alignas(16) float merge[kWarps][M::kRows][M::kCols];
    float wm[kWarps][M::kRows], wl[kWarps][M::kRows];
    uint32_t on[kWarps][kStages];
    alignas(16) float q[sizeof(typename M::T) == 4 ? M::kRows * D : 4];
    alignas(16) float p[sizeof(typename M::T) == 4 ? kWarps : 1][sizeof(typename M::T) == 4 ? 2 * M::kRows * (M::kTok + 2) : 4];
    long long scan[kWarps];
    long long at[2];
    int n0[2], nt0[2];
};

template <typename T> __device__ __forceinline__ void store_out(T *p, float4 v) { store4(p, v); }

// One row's result in this CTA from its warps' parts: finished (whole) or left in the workspace (slot).
template <int D, typename M, int C0>
__device__ __forceinline__ void merge_columns(Shared<D, M> &sh, M &math, typename M::T *o, float *lse, int heads,
                                           bool whole, float *part, float *ml, int warp, int lane) {
    if (C0 == 0) math.stats(sh.wm[warp], sh.wl[warp], lane);
    math.template put<C0>(&sh.merge[warp][0][0], lane);
    __syncthreads();
    for (int x = threadIdx.x; x < M::kRows * (M::kCols / 4); x += kThreads) {
        const int row = x / (M::kCols / 4), c = 4 * (x % (M::kCols / 4));
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
        const int col = C0 + c;
        if (whole) {
            const float i = l == 0.f ? 0.f : 1.f / l;  // no token left: zeros
            store_out(o + (size_t)row * D + col, make_float4(s.x * i, s.y * i, s.z * i, s.w * i));
            if (C0 == 0 && c == 0 && lse) lse[row] = (mx + log2f(l)) * kLn2;
        } else {
            *reinterpret_cast<float4 *>(part + (size_t)row * D + col) = s;
            if (C0 == 0 && c == 0) ml[2 * row] = mx, ml[2 * row + 1] = l;
        }
    }
    __syncthreads();
}

template <int D, typename M>
__global__ void __launch_bounds__(kThreads, M::kPerSm) attn_decode_kernel(AttnDecodeArgs p, Line ln, Partials w) {
    using T = typename M::T;
    using S = Shared<D, M>;
    constexpr int TILE = M::kTok * kWarps, CH = M::kRowBytes / 16;
    extern __shared__ __align__(1024) uint8_t raw[];
    S &sh = *reinterpret_cast<S *>(raw);
    follow();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    {  // the table's way to L2 overlaps that of the lengths, which say where in it a CTA begins
        const size_t line = ((size_t)blockIdx.x * kThreads + tid) * 32;
        if (line < (size_t)p.R * p.P) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.table + line));
    }

    // this CTA's run [begin, end) of the line: a prefix sum of the sequences' tiles, each thread a run of sequences
    const int per = (p.N + kThreads - 1) / kThreads;
    const int na = min(p.N, tid * per), ne = min(p.N, na + per);
    long long mine = 0;
    for (int n = na; n < ne; ++n) {
        int s, a, b;
        if (span_of(p, n, s, a, b)) mine += (b - a + TILE - 1) / TILE;
    }
    mine *= p.Hk;
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
    const int run = blockIdx.x / ln.nb, blk = blockIdx.x - run * ln.nb;
    const long long parts = min((long long)gridDim.x / ln.nb, total);
    long long edge[2];
    const bool small = total < (1 << 22);  // then a product with a CTA's number fits 32 bits, whose divisions are short
    edge[0] = edge[1] = total;
    if (run < parts) {
        edge[0] = small ? (uint32_t)total * run / (uint32_t)parts : total * run / parts;
        edge[1] = small ? (uint32_t)total * (run + 1) / (uint32_t)parts : total * (run + 1) / parts;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        if (edge[x] < total && edge[x] < pre && edge[x] >= pre - mine) {
            long long at = pre - mine;
            for (int n = na; n < ne; ++n) {
                int s, a, b;
                if (!span_of(p, n, s, a, b)) continue;
                const int nt = (b - a + TILE - 1) / TILE;
                if (edge[x] < at + (long long)nt * p.Hk) {
                    sh.n0[x] = n, sh.nt0[x] = nt, sh.at[x] = edge[x] - at;
                    break;
                }
                at += (long long)nt * p.Hk;
            }
        }
        if (x == 0 && !ln.whole) break;  // the end of the run is looked up only to be moved
    }
    // sequences with nothing to attend, and slots without a sequence
    for (int n = blockIdx.x; n < p.N; n += gridDim.x) {
        int s, a, b;
        const bool any = span_of(p, n, s, a, b);
        if (b > a) continue;
        if (w.by_row)
            for (int x = tid; x < p.Hk * ln.nb; x += kThreads) w.cut[n * p.Hk * ln.nb + x].x = -1;
        if (!any) continue;
        for (int x = tid; x < p.Hq * D / 4; x += kThreads)
            store_out(static_cast<T *>(p.o) + (size_t)n * p.Hq * D + 4 * x, make_float4(0.f, 0.f, 0.f, 0.f));
        if (p.lse)
            for (int x = tid; x < p.Hq; x += kThreads) p.lse[(size_t)n * p.Hq + x] = -INFINITY;
    }
    __syncthreads();
    // the row that the run begins in, and its tiles before the run
    int first_row = 0, head_start = 0;
    if (edge[0] < total) {
        first_row = small ? (int)((uint32_t)sh.at[0] / (uint32_t)sh.nt0[0]) : (int)(sh.at[0] / sh.nt0[0]);
        head_start = (int)(sh.at[0] - (long long)first_row * sh.nt0[0]);
    }
    if (ln.whole) {  // a row belongs to the run that its first tile lies in
#pragma unroll
        for (int x = 0; x < 2; ++x)
            if (edge[x] < total) {
                const int before = (int)(sh.at[x] % sh.nt0[x]);
                if (before) edge[x] += sh.nt0[x] - before;
            }
    }
    const long long begin = edge[0], end = edge[1];
    if (begin >= end) {
        if (tid == 0 && !ln.whole && !w.by_row) w.cut[blockIdx.x].x = -1;
        return;
    }

    Place<TILE> cur;
    cur.n = sh.n0[0];
    cur.enter(p);
    {
        cur.h = first_row;
        cur.first = cur.start + head_start * TILE;
        if (ln.whole && head_start) {
            cur.first = cur.len - 1;  // past the row that belongs to the run before
            cur.next(p);
            head_start = 0;
        }
    }
    Place<TILE> ahead = cur;
    long long xa = begin;  // the next tile to load
    int page = -1, off = 0;  // the page of this lane's token of that tile, fetched one tile early, and its place there
    auto fetch = [&]() {
        page = -1;
        const int tok = ahead.first + warp * M::kTok + lane;
        if (xa < end && lane < M::kTok && tok < ahead.len) {
            const uint32_t j = ln.by_page.divide(tok);
            page = ahead.pages[j];
            off = tok - (int)j * p.page_size;
        }
    };
    // a lane copies chunk cl of rows r0, r0 + 32 / CH, ...: their places in a stage differ by constants
    const int cl = lane % CH, r0 = lane / CH;
    const uint8_t *kp = static_cast<const uint8_t *>(p.k_pages) + cl * 16, *vp = static_cast<const uint8_t *>(p.v_pages) + cl * 16;
    const uint32_t ring = sptr(&sh.ring[warp][0][0]) + r0 * M::kRowBytes;
    auto issue = [&](int stage) {
        if (xa < end) {
            const bool on = page >= 0 && page < p.num_pages;
            const uint32_t mask = __ballot_sync(0xffffffffu, on);
            if (lane == 0) sh.on[warp][stage] = mask;
            const uint32_t row = on ? ((uint32_t)page * p.Hk + ahead.h) * p.page_size + off : 0u;  // below 2^32: checked
            const uint32_t dst = ring + stage * S::kStage;
            GDR2_DCHECK(stage >= 0 && stage < S::kStages && ahead.n >= 0 && ahead.n < p.N && ahead.h >= 0 && ahead.h < p.Hk);
            GDR2_DCHECK((uint64_t)row < (uint64_t)p.num_pages * p.Hk * p.page_size);
#pragma unroll
            for (int i = 0; i < M::kTok * CH / 32; ++i) {
                constexpr int kStep = 32 / CH;
                const int r = i * kStep + r0;
                const uint32_t rr = __shfl_sync(0xffffffffu, row, r);
                const int bytes = mask >> r & 1 ? 16 : 0;
                const uint32_t d = dst + i * kStep * M::kRowBytes + ((cl ^ M::swizzle(r & 7)) << 4);
                cp16(d, kp + (uint64_t)rr * M::kRowBytes, bytes);
                cp16(d + M::kTok * M::kRowBytes, vp + (uint64_t)rr * M::kRowBytes, bytes);
            }
            ++xa;
            if (xa < end) ahead.next(p);
            fetch();
        }
        cp_commit();
    };
    fetch();
#pragma unroll 1
    for (int s = 0; s < S::kStages; ++s) issue(s);

    M math;
    const float sc = p.scale == 0.f ? 1.f : fabsf(p.scale) * kLog2e;
    const int heads = min(ln.rows, ln.G - blk * ln.rows);
    int stage = 0, j0 = 0;
    int4 cut = make_int4(-1, 0, 0, 0);
    bool fresh = true, head_of_row = false;
    for (long long x = begin; x < end; ++x) {
        if (fresh) {
            j0 = cur.h * ln.G + blk * ln.rows;
            head_of_row = cur.first == cur.start;
            math.begin(static_cast<const T *>(p.q) + ((size_t)cur.n * p.Hq + j0) * D, heads, p.scale, sh.q, lane);
            fresh = false;
        }
        cp_wait<S::kStages - 1>();
        __syncwarp();
        math.step(sptr(&sh.ring[warp][0][0]) + stage * S::kStage, sh.on[warp][stage], sc, sh.q,
                  sh.p[sizeof(T) == 4 ? warp : 0], lane);
        __syncwarp();
        issue(stage);
        if (++stage == S::kStages) stage = 0;
        if (cur.last() || x + 1 == end) {
            const bool whole = head_of_row && cur.last();
            GDR2_DCHECK(cur.n < p.N && j0 >= 0 && j0 + heads <= p.Hq && heads > 0 && (whole || !ln.whole));
            const int slot = 2 * blockIdx.x + head_of_row;
            const int row = (cur.n * p.Hk + cur.h) * ln.nb + blk;
            if (head_of_row && !whole && tid == 0) {
                // the run that its last tile falls to: the smallest k with total (k + 1) / parts >= the row's end
                const int done = (cur.first - cur.start) / TILE, nt = (cur.len - cur.start + TILE - 1) / TILE;
                const long long e = (x - done + nt) * parts, k = (e + total - 1) / total - 1;
                cut = make_int4(row, blockIdx.x, (int)(k - run) + 1, 0);
                GDR2_DCHECK(k > run && k < parts);
            }
            if (head_of_row && w.by_row && tid == 0) w.cut[row] = whole ? make_int4(-1, 0, 0, 0) : cut;
            T *o = static_cast<T *>(p.o) + ((size_t)cur.n * p.Hq + j0) * D;
            float *lse = p.lse ? p.lse + (size_t)cur.n * p.Hq + j0 : nullptr;
            float *part = w.o + (size_t)slot * kMaxRows * D, *ml = w.ml + (size_t)slot * kMaxRows * 2;
            merge_columns<D, M, 0>(sh, math, o, lse, heads, whole, part, ml, warp, lane);
            if constexpr (M::kCols < D) merge_columns<D, M, D / 2>(sh, math, o, lse, heads, whole, part, ml, warp, lane);
            fresh = true;
        }
        if (x + 1 < end) cur.next(p);
    }
    cp_wait<0>();
    if (tid == 0 && !ln.whole && !w.by_row) w.cut[blockIdx.x] = cut;
}

// Joins the rows of the line that borders of CTAs cut: block (x, y) takes query heads y hb .. of entry x of their list;
// the row's parts are the second slot of the CTA where it begins and the first slots of the CTAs that follow. D / 4
// lanes of four channels for each of hb heads, the parts shared by the groups of lanes that remain.
constexpr int kJoinThreads = 512;

template <int D, typename T>
__global__ void __launch_bounds__(kJoinThreads) attn_decode_join_kernel(AttnDecodeArgs p, Line ln, Partials w, int hb) {
    constexpr int LN = D / 4, NG = kJoinThreads / LN;
    __shared__ float4 so[NG][LN];
    __shared__ float sm[NG], sl[NG];
    const int tid = threadIdx.x, lane = tid % LN, rest = tid / LN, grp = rest / hb, ng = NG / hb;
    const int head = blockIdx.y * hb + rest - grp * hb;
    follow();
    const int4 cut = __ldcg(w.cut + blockIdx.x);
    const int row = cut.x, c = cut.y, cnt = cut.z;
    if (row < 0) return;
    const int nh = row / ln.nb, blk = row - nh * ln.nb, n = nh / p.Hk, h = nh - n * p.Hk;
    GDR2_DCHECK(n < p.N && c >= 0 && cnt > 1 && c + (cnt - 1) * ln.nb < kMaxCtas);
    const bool on = head < min(ln.rows, ln.G - blk * ln.rows);
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = grp; on && i0 < cnt; i0 += 4 * ng) {
        float2 ml[4];
        float4 v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * ng;
            const size_t at = ((size_t)2 * (c + i * ln.nb) + (i == 0)) * kMaxRows + head;
            ml[u] = make_float2(-INFINITY, 0.f);
            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < cnt) {
                ml[u] = __ldcg(reinterpret_cast<const float2 *>(w.ml) + at);
                v[u] = __ldcg(reinterpret_cast<const float4 *>(w.o + at * D) + lane);
            }
        }
        const float mx = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), m), f = pow2_rel(m, mx);
        o.x *= f, o.y *= f, o.z *= f, o.w *= f, l *= f;
        m = mx;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float g = pow2_rel(ml[u].x, mx);
            o.x = fmaf(v[u].x, g, o.x), o.y = fmaf(v[u].y, g, o.y), o.z = fmaf(v[u].z, g, o.z), o.w = fmaf(v[u].w, g, o.w);
            l = fmaf(ml[u].y, g, l);
        }
    }
    so[rest][lane] = o;
    if (lane == 0) sm[rest] = m, sl[rest] = l;
    __syncthreads();
    if (grp != 0 || !on) return;
    const int parts = min(ng, cnt);
    for (int g = 1; g < parts; ++g) m = fmaxf(m, sm[g * hb + rest]);
    o = make_float4(0.f, 0.f, 0.f, 0.f);
    l = 0.f;
#pragma unroll 4
    for (int g = 0; g < parts; ++g) {
        const float f = pow2_rel(sm[g * hb + rest], m);
        const float4 v = so[g * hb + rest][lane];
        o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y), o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
        l = fmaf(sl[g * hb + rest], f, l);
    }
    const size_t j = (size_t)n * p.Hq + h * ln.G + blk * ln.rows + head;
    const float i = l == 0.f ? 0.f : 1.f / l;
    store_out(static_cast<T *>(p.o) + j * D + 4 * lane, make_float4(o.x * i, o.y * i, o.z * i, o.w * i));
    if (lane == 0 && p.lse) p.lse[j] = (m + log2f(l)) * kLn2;
}

// How a call's line is cut: from its sizes alone, so that a workspace query and the call agree.
struct Plan {
    Line ln;
    long long rows;
    int ctas;
};
template <int D, typename M> Plan plan(const AttnDecodeArgs &a) {
    constexpr int TILE = M::kTok * kWarps, full = M::kPerSm * kAttnSms;
    Plan p;
    p.ln.G = a.Hq / a.Hk;
    p.ln.rows = M::kRows;
    p.ln.nb = (p.ln.G + M::kRows - 1) / M::kRows;
    p.ln.by_page = Divisor(a.page_size);
    // no more CTAs than the largest possible line has tiles, or rows if they stay whole: short ones do, as there is
    // nothing to join then, and a few tiles more or less make no CTA late
    long long span = (long long)a.P * a.page_size;
    if (a.window > 0 && a.window < span) span = a.window;
    const long long each = (span + TILE - 1) / TILE;
    const long long rows = (long long)a.N * a.Hk;
    p.rows = rows * p.ln.nb;
    p.ln.whole = each <= kWholeTiles;
    const long long most = p.ln.whole ? rows : rows * each, runs = full / p.ln.nb;  // at least one: checked
    p.ctas = (int)(most < runs ? most : runs) * p.ln.nb;
    return p;
}

template <int D, typename M> cudaError_t run(const AttnDecodeArgs &a, cudaStream_t st) {
    using T = typename M::T;
    constexpr int smem = (int)sizeof(Shared<D, M>);
    static_assert(smem * M::kPerSm <= (227 - M::kPerSm) * 1024, "they fit an SM together");
    static Allowed allowed;
    cudaError_t e = allowed(attn_decode_kernel<D, M>, smem);
    if (e != cudaSuccess) return e;
    const Plan pl = plan<D, M>(a);
    const Line ln = pl.ln;
    const long long rows = pl.rows;
    const int ctas = pl.ctas;
    Partials w = partials(a.workspace, D);
    w.by_row = !ln.whole && rows < ctas;
    GDR2_LAUNCH("attn_decode", st, e = launch(attn_decode_kernel<D, M>, dim3(ctas), dim3(kThreads), smem, 0, st, a, ln, w));
    if (e != cudaSuccess || ln.whole || ctas == ln.nb) return e;  // a single run cuts nothing
    const int entries = w.by_row ? (int)rows : ctas, heads = ln.G < ln.rows ? ln.G : ln.rows;
    // few rows have many parts: a block for each head, all its groups on the parts. Many rows have few: one block a row.
    int hb = 1;
    if (entries * heads > kAttnSms)
        while (hb < heads) hb *= 2;
    GDR2_LAUNCH("attn_decode_join", st,
                e = launch(attn_decode_join_kernel<D, T>, dim3(entries, (heads + hb - 1) / hb), dim3(kJoinThreads), 0, 0, st,
                           a, ln, w, hb));
    return e;
}

// f.template operator()<D, Math>() for the call's types and heads
template <int D, typename F> auto dispatch(const AttnDecodeArgs &a, F f) {
    const int G = a.Hq / a.Hk;
    if (a.dtype == 1) return G <= 8 ? f.template operator()<D, Bf16Math<D, true>>() : f.template operator()<D, Bf16Math<D, false>>();
    if (G == 1) return f.template operator()<D, F32Math<D, 1>>();
    if (G == 2) return f.template operator()<D, F32Math<D, 2>>();
    if (G <= 4) return f.template operator()<D, F32Math<D, 4>>();
    // 16 heads of 64 / 128, 400 MB: 141 / 142 us in blocks of 8, 133 / 158 at once: one form for both, at 6% for 64
    return f.template operator()<D, F32Math<D, 8>>();  // more in blocks of 8
}

struct Run {
    const AttnDecodeArgs &a;
    cudaStream_t st;
    template <int D, typename M> cudaError_t operator()() const { return run<D, M>(a, st); }
};
struct Bytes {
    const AttnDecodeArgs &a;
    template <int D, typename M> size_t operator()() const {
        return plan<D, M>(a).ln.whole ? 0
                                      : (partial_floats(D) + (size_t)kMaxCtas * 2 * kMaxRows * 2) * sizeof(float) +
                                            (size_t)kMaxCtas * sizeof(int4);
    }
};

}  // namespace

size_t attn_decode_workspace_bytes(const AttnDecodeArgs &a) {
    return a.d == 128 ? dispatch<128>(a, Bytes{a}) : dispatch<64>(a, Bytes{a});
}

int status_take_attn_decode() { return take_status(); }

cudaError_t launch_attn_decode(const AttnDecodeArgs &a, cudaStream_t st) {
    return a.d == 128 ? dispatch<128>(a, Run{a, st}) : dispatch<64>(a, Run{a, st});
}

}  // namespace gdr2
