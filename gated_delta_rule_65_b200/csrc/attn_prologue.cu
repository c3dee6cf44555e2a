// attn_prologue.cu -- the query / key prologue of the hybrid cell's attention layer (sm_100a): per-head RMS norm and
// rotary positions in one pass over HBM, forward, backward, and the serving form that writes K and V into pages.
//
// Per (token t, head), with x the projection's row of d channels:
//   n = rsqrt(mean(x^2) + eps),  u = n x (.) g            (norm = 0: u = x)
//   the first rot channels are rotated pairwise by theta_i = pos_t * freq_i, i < rot / 2, and scaled by mag:
//     y_a = mag (u_a cos - u_b sin),  y_b = mag (u_a sin + u_b cos)
//   with (a, b) = (i, i + rot / 2) in the half layout and (2 i, 2 i + 1) in the interleaved one.
// Backward: dz = the transposed rotation of dy; dg = sum over tokens and heads of n x (.) dz;
//   dx = n (g (.) dz - n^2 x mean(x (.) g (.) dz)).
//
// Angles: pos * freq reaches 10^5 turns, where an fp32 product is off by whole percents of a turn. The product is
// formed in fp64 in units of turns, its whole turns are dropped there, and the rest (exact to 2^-24 of a turn) goes
// to sincospif.
//
// Both directions are bound by HBM: 2 (forward) or 3 (backward) rows of d elements moved per (token, head), about 50
// fp32 operations per lane and row. A lane holds 8 consecutive channels of a row (16 bytes of bf16), d / 8 lanes make
// a row, and a group of d / 8 lanes keeps ONE token and walks its heads: cos and sin stay in registers for all of
// them (read per row from shared memory they cost 16 wavefronts per two rows, more than a third of the time that the
// rows' bytes take). The angles of a CTA's tokens are formed once by all its threads.
#include "attn.h"
#include "attn_vec.cuh"
#include "common.cuh"
#include "kernels.h"

namespace gdr2 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 16;                  // tokens of a CTA at a time
constexpr int kBwdCtas = 2 * kAttnSms;       // CTAs of the backward (a partial sum of dg each)

// cos and sin of the CTA's tokens t0 .. t0 + tb - 1, scaled by mag.
template <int D>
__device__ __forceinline__ void make_angles(const AttnPrologueArgs &p, int t0, int tb, float (*sc)[D / 2],
                                            float (*ss)[D / 2]) {
    const int half = p.rot / 2;
    for (int x = threadIdx.x; x < tb * half; x += kThreads) {
        const int tok = x / half, i = x - tok * half;
        if (t0 + tok >= p.T) break;
        const double turns = (double)p.pos[t0 + tok] * (p.freqs[i] * 0.15915494309189533577);
        float s, c;
        sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
        sc[tok][i] = p.mag * c;
        ss[tok][i] = p.mag * s;
    }
}

// What a lane multiplies its 8 channels and their partners with: y = c x + s partner(x).
struct Turn {
    float c[8], s[8];
    int partner;  // lane of the row (half layout)
    bool on;      // the lane's channels are rotated
};

template <int D, bool kInter>
__device__ __forceinline__ void load_turn(const AttnPrologueArgs &p, int l, const float *sc, const float *ss, Turn &t) {
    t.on = 8 * l < p.rot;
    t.partner = l;
    if (!t.on) return;
    if constexpr (kInter) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            t.c[e] = sc[4 * l + e / 2];
            t.s[e] = (e & 1) ? ss[4 * l + e / 2] : -ss[4 * l + e / 2];
        }
    } else {
        const int hl = p.rot / 16;  // lanes of a half
        const bool low = l < hl;
        const int i0 = 8 * (low ? l : l - hl);
        t.partner = low ? l + hl : l - hl;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            t.c[e] = sc[i0 + e];
            t.s[e] = low ? -ss[i0 + e] : ss[i0 + e];
        }
    }
}

// y = the rotation (kBack: its transpose) of x. Every lane of the warp takes part.
template <int L, bool kInter, bool kBack>
__device__ __forceinline__ void turn(const Turn &t, const float (&x)[8], float (&y)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float o = kInter ? x[e ^ 1] : __shfl_sync(0xffffffffu, x[e], t.partner, L);
        const float s = kBack ? -t.s[e] : t.s[e];
        y[e] = t.on ? fmaf(x[e], t.c[e], o * s) : x[e];
    }
}

template <int L> __device__ __forceinline__ float sum_row(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ void load_gain(const float *g, int l, float (&w)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = g ? __ldg(g + 8 * l + e) : 1.f;
}

// One token's H rows of x, heads h0, h0 + step, ... (this group's share), normed, rotated and stored at out + h hs.
// Trip counts are the same for every group of the CTA: a group without a row left works on zeros and stores nothing.
template <int D, typename T, bool kInter>
__device__ __forceinline__ void fwd_rows(const AttnPrologueArgs &p, const T *x, const float *gain, T *out,
                                         long long hs, int H, int h0, int step, bool live, int l, const Turn &t) {
    constexpr int L = D / 8, U = 4;
    float g[8];
    load_gain(gain, l, g);
    const int iters = (H + step - 1) / step;
    for (int i0 = 0; i0 < iters; i0 += U) {
        Vec8<T> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + (i0 + u) * step;
            if (live && h < H)
                raw[u].load_stream(x + (size_t)h * D + 8 * l);
            else
                raw[u].zero();
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u < iters) {
                const int h = h0 + (i0 + u) * step;
                float v[8], y[8];
                raw[u].get(v);
                if (p.norm) {
                    float q = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) q = fmaf(v[e], v[e], q);
                    const float n = rsqrtf(sum_row<L>(q) * (1.f / D) + p.eps);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] *= n * g[e];
                }
                turn<L, kInter, false>(t, v, y);
                if (live && h < H) Vec8<T>::store(out + h * hs + 8 * l, y);
            }
        }
    }
}

// tb: tokens of a CTA, a power of two of at most kMaxTok and at most the CTA's groups.
template <int D, typename T, bool kInter, bool kCache>
__global__ void __launch_bounds__(kThreads) attn_prologue_fwd_kernel(AttnPrologueArgs p, int tb) {
    constexpr int L = D / 8, NG = kThreads / L;
    __shared__ float sc[kMaxTok][D / 2], ss[kMaxTok][D / 2];
    const int grp = threadIdx.x / L, l = threadIdx.x % L;
    const int t0 = blockIdx.x * tb, step = NG / tb, tok = grp / step, h0 = grp % step;
    make_angles<D>(p, t0, tb, sc, ss);
    __syncthreads();
    const int tt = t0 + tok;
    bool live = tt < p.T;
    int page = -1, off = 0;
    if constexpr (kCache) {
        const int s = live ? p.seq[tt] : -1;
        live = s >= 0 && s < p.R;
        if (live) {
            const int pos = p.pos[tt], j = pos / p.page_size;
            if (pos >= 0 && j < p.P) {
                page = p.table[(size_t)s * p.P + j];
                off = pos - j * p.page_size;
                if (page >= p.num_pages) page = -1;
            }
        }
    }
    Turn t;
    load_turn<D, kInter>(p, l, sc[tok], ss[tok], t);
    const size_t tr = live ? (size_t)tt : 0;
    fwd_rows<D, T, kInter>(p, static_cast<const T *>(p.xq) + tr * p.sxq, p.gq,
                           static_cast<T *>(p.q) + tr * p.Hq * D, D, p.Hq, h0, step, live, l, t);
    if constexpr (!kCache) {
        fwd_rows<D, T, kInter>(p, static_cast<const T *>(p.xk) + tr * p.sxk, p.gk,
                               static_cast<T *>(p.k) + tr * p.Hk * D, D, p.Hk, h0, step, live, l, t);
    } else {
        const bool put = live && page >= 0;
        const long long hs = (long long)p.page_size * D;
        const size_t slot = put ? (size_t)page * p.Hk * hs + (size_t)off * D : 0;
        fwd_rows<D, T, kInter>(p, static_cast<const T *>(p.xk) + tr * p.sxk, p.gk,
                               static_cast<T *>(p.k_pages) + slot, hs, p.Hk, h0, step, put, l, t);
        if (put) {
            const T *v = static_cast<const T *>(p.xv) + tr * p.sxv + 8 * l;
            T *dst = static_cast<T *>(p.v_pages) + slot + 8 * l;
            for (int h = h0; h < p.Hk; h += step) {
                Vec8<T> raw;
                raw.load_stream(v + (size_t)h * D);
                raw.put(dst + h * hs);
            }
        }
    }
}

template <int D, typename T, bool kInter>
__device__ __forceinline__ void bwd_rows(const AttnPrologueArgs &p, const T *x, const T *dy, const float *gain, T *dx,
                                         int H, int h0, int step, bool live, int l, const Turn &t, float (&acc)[8]) {
    constexpr int L = D / 8, U = sizeof(T) == 2 ? 4 : 2;
    float g[8];
    load_gain(gain, l, g);
    const int iters = (H + step - 1) / step;
    for (int i0 = 0; i0 < iters; i0 += U) {
        Vec8<T> rx[U], rd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + (i0 + u) * step;
            if (live && h < H) {
                rd[u].load_stream(dy + (size_t)h * D + 8 * l);
                if (p.norm) rx[u].load_stream(x + (size_t)h * D + 8 * l);
            } else {
                rd[u].zero();
                rx[u].zero();
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u < iters) {
                const int h = h0 + (i0 + u) * step;
                float v[8], dz[8];
                rd[u].get(v);
                turn<L, kInter, true>(t, v, dz);
                if (p.norm) {
                    rx[u].get(v);
                    float q = 0.f, m = 0.f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        q = fmaf(v[e], v[e], q);
                        m = fmaf(v[e] * g[e], dz[e], m);
                    }
                    q = sum_row<L>(q);
                    m = sum_row<L>(m);
                    const float n = rsqrtf(q * (1.f / D) + p.eps), c = m * (1.f / D) * n * n;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        acc[e] = fmaf(dz[e] * n, v[e], acc[e]);
                        dz[e] = n * fmaf(-c, v[e], g[e] * dz[e]);
                    }
                }
                if (live && h < H) Vec8<T>::store(dx + (size_t)h * D + 8 * l, dz);
            }
        }
    }
}

// A CTA takes the token blocks b, b + gridDim, ...: a fixed assignment, so the sums over tokens have a fixed order.
template <int D, typename T, bool kInter>
__global__ void __launch_bounds__(kThreads, 2) attn_prologue_bwd_kernel(AttnPrologueArgs p, int tb,
                                                                        float *__restrict__ partial) {
    constexpr int L = D / 8, NG = kThreads / L;
    __shared__ float sc[kMaxTok][D / 2], ss[kMaxTok][D / 2];
    __shared__ float red[NG][D];
    cudaTriggerProgrammaticLaunchCompletion();
    const int grp = threadIdx.x / L, l = threadIdx.x % L;
    const int step = NG / tb, tok = grp / step, h0 = grp % step;
    float aq[8], ak[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) aq[e] = ak[e] = 0.f;
    const int blocks = (p.T + tb - 1) / tb;
    for (int b = blockIdx.x; b < blocks; b += gridDim.x) {
        const int t0 = b * tb, tt = t0 + tok;
        __syncthreads();  // the block before has been read
        make_angles<D>(p, t0, tb, sc, ss);
        __syncthreads();
        const bool live = tt < p.T;
        const size_t tr = live ? (size_t)tt : 0;
        Turn t;
        load_turn<D, kInter>(p, l, sc[tok], ss[tok], t);
        bwd_rows<D, T, kInter>(p, static_cast<const T *>(p.xq) + tr * p.sxq, static_cast<const T *>(p.dq) + tr * p.Hq * D,
                               p.gq, static_cast<T *>(p.dxq) + tr * p.sdxq, p.Hq, h0, step, live, l, t, aq);
        bwd_rows<D, T, kInter>(p, static_cast<const T *>(p.xk) + tr * p.sxk, static_cast<const T *>(p.dk) + tr * p.Hk * D,
                               p.gk, static_cast<T *>(p.dxk) + tr * p.sdxk, p.Hk, h0, step, live, l, t, ak);
    }
    if (partial == nullptr) return;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) red[grp][8 * l + e] = which ? ak[e] : aq[e];
        __syncthreads();
        if (threadIdx.x < D) {
            float v = 0.f;
#pragma unroll
            for (int x = 0; x < NG; ++x) v += red[x][threadIdx.x];
            partial[((size_t)blockIdx.x * 2 + which) * D + threadIdx.x] = v;
        }
    }
}

// dg[c] = the CTAs' partial sums: slice s adds the CTAs s, s + 32, ... in order, then the slices are added in order.
template <int D>
__global__ void __launch_bounds__(1024) attn_prologue_reduce_kernel(const float *__restrict__ partial, int ctas,
                                                                    float *dgq, float *dgk) {
    __shared__ float red[32][33];
    const int which = blockIdx.x, c = blockIdx.y * 32 + threadIdx.x % 32, sl = threadIdx.x / 32;
    cudaGridDependencySynchronize();
    float v = 0.f;
#pragma unroll 4
    for (int i = sl; i < ctas; i += 32) v += __ldcg(partial + ((size_t)i * 2 + which) * D + c);
    red[sl][threadIdx.x % 32] = v;
    __syncthreads();
    if (sl == 0) {
        float s = 0.f;
#pragma unroll
        for (int x = 0; x < 32; ++x) s += red[x][threadIdx.x];
        float *out = which ? dgk : dgq;
        if (out) out[c] = s;
    }
}

// Tokens of a CTA: about 8 rows for a group of lanes (fewer leave its loads uncovered, more leave SMs idle at the
// end), fewer tokens while the grid would not fill the GPU twice.
int tokens_per_cta(int T, int rows, int groups) {
    int tb = kMaxTok < groups ? kMaxTok : groups;
    while (tb > 1 && (tb * rows > 8 * groups || (T + tb - 1) / tb < 8 * kAttnSms)) tb /= 2;
    return tb;
}

template <int D, typename T, bool kInter>
cudaError_t run_fwd(const AttnPrologueArgs &a, bool cache, cudaStream_t st) {
    const int tb = tokens_per_cta(a.T, a.Hq + a.Hk, kThreads / (D / 8));
    const int grid = (a.T + tb - 1) / tb;
    if (cache)
        GDR2_LAUNCH("attn_prologue_cache", st,
                    (attn_prologue_fwd_kernel<D, T, kInter, true><<<grid, kThreads, 0, st>>>(a, tb)));
    else
        GDR2_LAUNCH("attn_prologue_fwd", st,
                    (attn_prologue_fwd_kernel<D, T, kInter, false><<<grid, kThreads, 0, st>>>(a, tb)));
    return cudaGetLastError();
}

template <int D, typename T, bool kInter>
cudaError_t run_bwd(const AttnPrologueArgs &a, cudaStream_t st) {
    const int tb = tokens_per_cta(a.T, a.Hq + a.Hk, kThreads / (D / 8));
    const int blocks = (a.T + tb - 1) / tb, grid = blocks < kBwdCtas ? blocks : kBwdCtas;
    float *partial = a.dgq || a.dgk ? static_cast<float *>(a.workspace) : nullptr;
    GDR2_LAUNCH("attn_prologue_bwd", st,
                (attn_prologue_bwd_kernel<D, T, kInter><<<grid, kThreads, 0, st>>>(a, tb, partial)));
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || partial == nullptr) return e;
    GDR2_LAUNCH("attn_prologue_reduce", st,
                e = launch_dependent(attn_prologue_reduce_kernel<D>, dim3(2, D / 32), dim3(1024), 0, st,
                                     (const float *)partial, grid, a.dgq, a.dgk));
    return e;
}

template <typename F> cudaError_t dispatch(const AttnPrologueArgs &a, F f) {
    // without a rotation the interleaved form runs: it needs no exchange between lanes
    const bool inter = a.interleaved || a.rot == 0;
    if (a.dtype == 1) {
        if (a.d == 128) return inter ? f.template operator()<128, __nv_bfloat16, true>() : f.template operator()<128, __nv_bfloat16, false>();
        return inter ? f.template operator()<64, __nv_bfloat16, true>() : f.template operator()<64, __nv_bfloat16, false>();
    }
    if (a.d == 128) return inter ? f.template operator()<128, float, true>() : f.template operator()<128, float, false>();
    return inter ? f.template operator()<64, float, true>() : f.template operator()<64, float, false>();
}

struct Fwd {
    const AttnPrologueArgs &a;
    bool cache;
    cudaStream_t st;
    template <int D, typename T, bool I> cudaError_t operator()() const { return run_fwd<D, T, I>(a, cache, st); }
};
struct Bwd {
    const AttnPrologueArgs &a;
    cudaStream_t st;
    template <int D, typename T, bool I> cudaError_t operator()() const { return run_bwd<D, T, I>(a, st); }
};

}  // namespace

size_t attn_prologue_workspace_bytes(int d) { return (size_t)kBwdCtas * 2 * d * sizeof(float); }

cudaError_t launch_attn_prologue_fwd(const AttnPrologueArgs &a, cudaStream_t st) { return dispatch(a, Fwd{a, false, st}); }
cudaError_t launch_attn_prologue_cache(const AttnPrologueArgs &a, cudaStream_t st) { return dispatch(a, Fwd{a, true, st}); }
cudaError_t launch_attn_prologue_bwd(const AttnPrologueArgs &a, cudaStream_t st) { return dispatch(a, Bwd{a, st}); }

}  // namespace gdr2
