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
// Bound: HBM moves 2 (forward) or 3 (backward) rows of d elements per (token, head); next to it stands the issue of
// instructions. So a lane holds two 16-byte chunks of a row, in the half layout the two that are rotated into one
// another: the rotation needs no exchange between lanes, a warp takes four bf16 rows of 128 channels at once, and all
// arithmetic runs on pairs of floats. A lane keeps ONE token and walks its heads, so the coefficients (gain, cosine and
// sine folded together) stay in registers for all of them and the token's angles are formed once, by the whole warp. All
// lane groups of a warp share a token where its heads fill them, else several tokens share the warp. Every lane feeds
// itself: cp.async into shared memory that only it reads, several rows deep and running on into the next token, so that
// nothing but a warp's own exchange of angles ever waits.
//
// Measured on one B200, back to back: 32,768 tokens of 16 + 16 bf16 heads of 128 channels forward in 89 us (537 MB,
// 6.0 TB/s, 92% of the measured copy) and backward in 138 us (805 MB, 5.8 TB/s, 89%); 17,820 new tokens of 16 packed
// prompts (16 + 4 + 4 heads) into the pages in 42 us (219 MB, 5.2 TB/s, 80%: 7.5 tokens for a warp, so the last round is
// half empty). 150 MB of fp32 rows (16 + 16 heads of 128) take 53 and 77 us (86% and 90%).
#include "attn.h"
#include "attn_vec.cuh"
#include "common.cuh"
#include "kernels.h"

namespace gdr2 {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
// CTAs on an SM and rows of a lane in flight, measured on the training batch (B = 8, T = 4096, 16 + 16 heads of 128
// channels, bf16), kernel times with their events (about 3 us). Forward, 2 CTAs: 92 us with 4 to 8 rows (and 16 packed
// prompts into the cache 49.1 us with 4, 49.9 with 8); 3 CTAs: 118 to 130 us with 4 to 8 rows (spills, and more warps on
// more tokens scatter the requests). Backward, 2 CTAs: 173 us fetching row by row (4 rows ahead), 141 in bursts of 2 and
// 145 of 3; 1 CTA: 149 row by row, 143 and 146 in bursts of 2 and 4.
constexpr int kFwdCtas = 2, kFwdDepth = 4;
constexpr int kBwdCtas = 2, kBwdBurst = 2, kBwdDepth = 2 * kBwdBurst;
constexpr int kBwdGrid = kBwdCtas * kAttnSms;  // CTAs of the backward (a partial sum of dgq or dgk each)

// How lanes hold a row: kLanes lanes of two chunks each, kRows rows in a warp.
template <int D, typename T> struct Layout {
    static constexpr int kElems = 16 / sizeof(T), kPairs = kElems / 2;
    static constexpr int kLanes = D / (2 * kElems), kRows = 32 / kLanes;
    static constexpr int kRowsLog = kRows == 8 ? 3 : kRows == 4 ? 2 : 1;
    static_assert(1 << kRowsLog == kRows, "2, 4 or 8 rows");
};

// The two channels at which lane l's chunks start, and which of them are rotated. Half layout: lanes below
// rot / (2 kElems) hold chunk l and the one rotated with it; the rest of the row is split in two runs, so that each
// access of the lanes is contiguous.
template <int D, typename T, bool kInter> struct Slot {
    using Y = Layout<D, T>;
    int at0, at1;
    bool on0, on1;
    __device__ __forceinline__ bool on(int i) const { return kInter && i >= Y::kPairs / 2 ? on1 : on0; }  // u[i], v[i] rotated
    __device__ __forceinline__ Slot(int l, int rot) {
        if constexpr (kInter) {
            at0 = l * Y::kElems, at1 = (l + Y::kLanes) * Y::kElems;
            on0 = at0 < rot, on1 = at1 < rot;
        } else {
            const int hp = rot / (2 * Y::kElems);
            on0 = on1 = l < hp;
            at0 = (on0 ? l : l + hp) * Y::kElems;
            at1 = (on0 ? l + hp : l + Y::kLanes) * Y::kElems;
        }
    }
};

// Radians per position of the two pairs whose angles a lane forms, in turns.
struct Freqs {
    double f[2];
    __device__ __forceinline__ void load(const AttnPrologueArgs &p, int lane) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            f[i] = lane + 32 * i < p.rot / 2 ? p.freqs[lane + 32 * i] * 0.15915494309189533577 : 0.0;
    }
    // cos and sin of the warp's `tokens` tokens, scaled by mag: cs[k][0 .. D / 2) and cs[k][D / 2 .. D). pos: the position
    // of the lane's token; token k's first lane is k 32 / tokens.
    template <int D, bool kOne>
    __device__ __forceinline__ void angles(const AttnPrologueArgs &p, int pos, int tokens, float (*cs)[D], int lane) const {
        __syncwarp();  // the tokens before have been read
        // two tokens at a time, for their chains to overlap (1 + 1 heads of 64, half of it rotated, backward: 160 us for
        // 150 MB of rows, 181 one by one, 155 four at a time, which the 4 + 4 heads' registers pay for: 111 against 102)
        constexpr int G = kOne ? 1 : 2;
#pragma unroll 1
        for (int k = 0; k < tokens; k += G) {
            float sn[G][D / 64], cn[G][D / 64];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int at = kOne ? pos : __shfl_sync(0xffffffffu, pos, (k + g) * (32 / tokens) & 31);
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                    const double turns = (double)at * f[i];
                    sincospif(2.f * (float)(turns - rint(turns)), &sn[g][i], &cn[g][i]);
                }
            }
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int i = 0; i < D / 64; ++i) {
                    const int x = lane + 32 * i;
                    if (x < p.rot / 2 && k + g < tokens) {
                        cs[k + g][x] = p.mag * cn[g][i];
                        cs[k + g][D / 2 + x] = p.mag * sn[g][i];
                    }
                }
        }
        __syncwarp();
    }
};

// A token's rotation as a lane applies it to u and v (partners, Chunks): cosines and sines, 1 and 0 where nothing is
// rotated.
template <int D, typename T, bool kInter>
__device__ __forceinline__ void load_turn(const Slot<D, T, kInter> &w, const float *sc, const float *ss, F2 (&c)[Chunks<T, kInter>::kPairs],
                                          F2 (&s)[Chunks<T, kInter>::kPairs]) {
    using C = Chunks<T, kInter>;
    if constexpr (kInter) {
        C::template load<C::kHalf>(sc + w.at0 / 2, c), C::template load<C::kHalf>(sc + w.at1 / 2, c + C::kHalf);
        C::template load<C::kHalf>(ss + w.at0 / 2, s), C::template load<C::kHalf>(ss + w.at1 / 2, s + C::kHalf);
    } else {
        const int at = w.on0 ? w.at0 : 0;
        C::template load<C::kPairs>(sc + at, c), C::template load<C::kPairs>(ss + at, s);
    }
#pragma unroll
    for (int i = 0; i < C::kPairs; ++i)
        if (!w.on(i)) c[i] = f2(1.f, 1.f), s[i] = f2(0.f, 0.f);
}

// y = cu u + sv v, z = cv v + su u. An infinity in an unrotated channel must not reach another one as 0 * inf: without a
// rotation the partner's place is taken by a zero (kAll: the whole row is rotated).
template <bool kAll>
__device__ __forceinline__ void turn(bool on, F2 cu, F2 sv, F2 cv, F2 su, F2 u, F2 v, F2 &y, F2 &z) {
    F2 pu = u, pv = v;
    if (!kAll) {
        pu.v = on ? pu.v : 0;
        pv.v = on ? pv.v : 0;
    }
    y = fma(cu, u, mul(sv, pv));
    z = fma(cv, v, mul(su, pu));
}

template <int L> __device__ __forceinline__ float sum_row(float v) {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A row's gain in shared memory, in the lanes' order (ones where there is none).
template <int D, typename C> __device__ __forceinline__ void stage_gain(const float *g, float *sg) {
    for (int i = threadIdx.x; i < D; i += kThreads) sg[C::place(i)] = g ? g[i] : 1.f;
}

// The work of a warp: units u = warp, warp + warps, ... of (block of tokens, part). groups = 2^gl lane groups share a
// token, so that a block has kRows / groups tokens and lane group grp works on token grp / groups of it; there are
// parts = 2^log parts, and part k of a token takes the heads k groups + grp % groups, + parts groups, ... of each
// tensor. All powers of two: no division in a unit's few rows. kOne: all groups on one token, known to the compiler.
struct Units {
    int log, gl, count, stride;
};
template <typename Y, bool kOne> struct Walk : Units {
    __device__ __forceinline__ explicit Walk(const Units &u) : Units(u) {}
    __device__ __forceinline__ int groups_log() const { return kOne ? Y::kRowsLog : gl; }
    __device__ __forceinline__ int tokens() const { return kOne ? 1 : Y::kRows >> gl; }
    __device__ __forceinline__ int slot(int grp) const { return kOne ? 0 : grp >> gl; }  // which token of the block
    __device__ __forceinline__ int token(int u, int grp) const { return (u >> log) * tokens() + slot(grp); }
    __device__ __forceinline__ int head(int u, int grp) const {
        return ((u & ((1 << log) - 1)) << groups_log()) + (kOne ? grp : grp & ((1 << gl) - 1));
    }
    __device__ __forceinline__ int step() const { return 1 << (log + groups_log()); }
};

__device__ __forceinline__ void cp16(void *dst, const void *src, bool on) {  // off: zeros, nothing is read
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(on ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// ---- forward and cache form ----------------------------------------------------------------------------------

template <int D, typename T> struct FwdShared {
    uint4 ring[kFwdDepth][2][kThreads];
    alignas(16) float gain[2][D];
    alignas(16) float cs[kWarps][Layout<D, T>::kRows][D];
};

template <int D, typename T, bool kInter, bool kAll, bool kCache, bool kOne>
__global__ void __launch_bounds__(kThreads, kFwdCtas) attn_prologue_fwd_kernel(AttnPrologueArgs p, Units units) {
    using Y = Layout<D, T>;
    const Walk<Y, kOne> un(units);
    using C = Chunks<T, kInter>;
    constexpr int N = Y::kPairs;
    extern __shared__ __align__(16) uint8_t raw[];
    FwdShared<D, T> &sh = *reinterpret_cast<FwdShared<D, T> *>(raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, grp = lane / Y::kLanes, l = lane % Y::kLanes;
    const Slot<D, T, kInter> w(l, p.rot);
    const int step = un.step(), tokens = un.tokens();
    const float *cs = sh.cs[warp][un.slot(grp)];
    const int tq = (p.Hq + step - 1) / step, tk = (p.Hk + step - 1) / step;
    int u = blockIdx.x * kWarps + warp;
    follow();

    // the ring: what this lane fetches next is row `src` (head ha of ea) of tensor seg of unit ua, `left` rows of it
    // remaining, its own the first of each step
    int ua = u, seg = -1, left = 0, ha = 0, ea = 0;
    const T *src = nullptr;
    auto enter = [&]() {
        const int tok = un.token(ua, grp);
        ha = un.head(ua, grp);
        ++seg;
        const T *x = static_cast<const T *>(seg == 0 ? p.xq : seg == 1 ? p.xk : p.xv);
        src = x + (size_t)tok * (seg == 0 ? p.sxq : seg == 1 ? p.sxk : p.sxv) + (size_t)ha * D;
        ea = !kOne && tok >= p.T ? 0 : seg == 0 ? p.Hq : p.Hk;
        left = seg == 0 ? tq : tk;
    };
    if (ua < un.count) enter();
    auto fetch = [&](int slot) {
        GDR2_DCHECK(slot >= 0 && slot < kFwdDepth);
        if (ua < un.count) {
            const bool on = ha < ea;
            const T *x = on ? src : static_cast<const T *>(p.xq);
            cp16(&sh.ring[slot][0][threadIdx.x], x + w.at0, on);
            cp16(&sh.ring[slot][1][threadIdx.x], x + w.at1, on);
            src += step * D, ha += step;
            if (--left == 0) {
                if (seg == (kCache ? 2 : 1)) seg = -1, ua += un.stride;
                if (ua < un.count) enter();
            }
        }
        cp_commit();
    };
#pragma unroll
    for (int i = 0; i < kFwdDepth; ++i) fetch(i);
    // the lane's token of a unit (0 behind the last), its position and its sequence read two units ahead
    auto token = [&](int v) {
        const int tok = v < un.count ? un.token(v, grp) : 0;
        return kOne || tok < p.T ? tok : 0;
    };
    int pos = 0, seq = 0, page = -1, npos = 0, nseq = 0;
    auto find_page = [&](int q, int s) {
        if (s < 0 || s >= p.R || q < 0) return -1;
        const int j = (int)p.by_page.divide(q);
        return j < p.P ? p.table[(size_t)s * p.P + j] : -1;
    };
    if (p.rot || kCache) {
        pos = p.pos[token(u)];
        npos = p.pos[token(u + un.stride)];
    }
    if constexpr (kCache) {
        seq = p.seq[token(u)];
        nseq = p.seq[token(u + un.stride)];
        page = find_page(pos, seq);
    }
    Freqs fr;
    fr.load(p, lane);
    stage_gain<D, C>(p.gq, sh.gain[0]);
    stage_gain<D, C>(p.gk, sh.gain[1]);
    __syncthreads();
    int slot = 0;
    for (; u < un.count; u += un.stride) {
        const int tok = un.token(u, grp), h0 = un.head(u, grp);
        const bool real = kOne || tok < p.T;
        GDR2_DCHECK(tok >= 0 && tok < p.T + tokens - 1);
        int fpos = 0, fseq = 0, npage = -1;
        if (p.rot || kCache) fpos = p.pos[token(u + 2 * un.stride)];
        if constexpr (kCache) {
            fseq = p.seq[token(u + 2 * un.stride)];
            npage = find_page(npos, nseq);
        }
        fr.angles<D, kOne>(p, pos, tokens, sh.cs[warp], lane);
        const bool live = real && (!kCache || (seq >= 0 && seq < p.R));
        const bool put = live && (!kCache || (page >= 0 && page < p.num_pages));
        GDR2_DCHECK(!kCache || !put || (pos >= 0 && pos - p.by_page.divide(pos) * p.page_size < (uint32_t)p.page_size));
        const long long hs = kCache ? (long long)p.page_size * D : D;  // from head to head where keys go
        const size_t at = kCache ? (put ? ((size_t)page * p.Hk * p.page_size + (pos - p.by_page.divide(pos) * p.page_size)) * D : 0) : (size_t)tok * p.Hk * D;
#pragma unroll 1
        for (int which = 0; which < 2; ++which) {
            // the gain folded into the rotation: the partner's goes with its sine
            F2 cu[N], sv[N], cv[N], su[N];
            {
                F2 c[N], s[N], gu[N], gv[N];
                load_turn<D, T, kInter>(w, cs, cs + D / 2, c, s);
                C::pairs(sh.gain[which] + w.at0, sh.gain[which] + w.at1, gu, gv);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    cu[i] = mul(c[i], gu[i]), sv[i] = mul(neg(s[i]), gv[i]);
                    cv[i] = mul(c[i], gv[i]), su[i] = mul(s[i], gu[i]);
                }
            }
            const int H = (which ? put : live) ? (which ? p.Hk : p.Hq) : 0, trips = which ? tk : tq;  // H: heads to store
            const long long os = which ? hs : D, inc = os * step;
            T *out = (which == 0 ? static_cast<T *>(p.q) + (size_t)tok * p.Hq * D : static_cast<T *>(kCache ? p.k_pages : p.k) + at) +
                     h0 * os;
#pragma unroll 1
            for (int i = 0, h = h0; i < trips; ++i, h += step, out += inc) {
                cp_wait<kFwdDepth - 1>();
                F2 u[N], v[N], y[N], z[N];
                C::get(sh.ring[slot][0][threadIdx.x], sh.ring[slot][1][threadIdx.x], u, v);
#pragma unroll
                for (int i = 0; i < N; ++i) turn<kAll>(w.on(i), cu[i], sv[i], cv[i], su[i], u[i], v[i], y[i], z[i]);
                if (p.norm) {
                    F2 q = mul(u[0], u[0]);
#pragma unroll
                    for (int i = 1; i < N; ++i) q = fma(u[i], u[i], q);
#pragma unroll
                    for (int i = 0; i < N; ++i) q = fma(v[i], v[i], q);
                    const float n = rsqrtf(sum_row<Y::kLanes>(sum2(q)) * (1.f / D) + p.eps);
                    const F2 nn = f2(n, n);
#pragma unroll
                    for (int i = 0; i < N; ++i) y[i] = mul(y[i], nn), z[i] = mul(z[i], nn);
                }
                fetch(slot);
                if (++slot == kFwdDepth) slot = 0;
                if (h < H) C::put(out + w.at0, out + w.at1, y, z);
            }
        }
        if constexpr (kCache) {
            T *v = static_cast<T *>(p.v_pages) + at;
#pragma unroll 1
            for (int i = 0, h = h0; i < tk; ++i, h += step) {
                cp_wait<kFwdDepth - 1>();
                if (put && h < p.Hk) {
                    *reinterpret_cast<uint4 *>(v + h * hs + w.at0) = sh.ring[slot][0][threadIdx.x];
                    *reinterpret_cast<uint4 *>(v + h * hs + w.at1) = sh.ring[slot][1][threadIdx.x];
                }
                fetch(slot);
                if (++slot == kFwdDepth) slot = 0;
            }
        }
        pos = npos, npos = fpos;
        seq = nseq, nseq = fseq;
        page = npage;
    }
    cp_wait<0>();
}

// ---- backward --------------------------------------------------------------------------------------------------

template <int D, typename T> struct BwdShared {
    uint4 ring[kBwdDepth][4][kThreads];
    alignas(16) float gain[D];
    alignas(16) float cs[kWarps][Layout<D, T>::kRows][D];
};

// The first `cq` CTAs take the queries, the others the keys (one set of sums in a lane's registers), each warp a fixed
// set of units: the sums over tokens have a fixed order.
template <int D, typename T, bool kInter, bool kAll, bool kOne>
__global__ void __launch_bounds__(kThreads, kBwdCtas) attn_prologue_bwd_kernel(AttnPrologueArgs p, Units uq, Units uk, int cq,
                                                                               float *__restrict__ partial) {
    using Y = Layout<D, T>;
    using C = Chunks<T, kInter>;
    constexpr int N = Y::kPairs;
    extern __shared__ __align__(16) uint8_t raw[];
    BwdShared<D, T> &sh = *reinterpret_cast<BwdShared<D, T> *>(raw);
    const bool keys = blockIdx.x >= cq;
    const Walk<Y, kOne> un(keys ? uk : uq);
    const T *x = static_cast<const T *>(keys ? p.xk : p.xq), *dy = static_cast<const T *>(keys ? p.dk : p.dq);
    T *dx = static_cast<T *>(keys ? p.dxk : p.dxq);
    const long long sx = keys ? p.sxk : p.sxq, sdx = keys ? p.sdxk : p.sdxq;
    const int H = keys ? p.Hk : p.Hq;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, grp = lane / Y::kLanes, l = lane % Y::kLanes;
    const Slot<D, T, kInter> w(l, p.rot);
    const int step = un.step(), tokens = un.tokens(), rows = (H + step - 1) / step;
    const float *cs = sh.cs[warp][un.slot(grp)];
    int u = (blockIdx.x - (keys ? cq : 0)) * kWarps + warp;
    follow();
    int ua = u, left = 0, ha = 0;  // as in the forward: the row this lane fetches next
    const T *sd = nullptr, *sr = nullptr;
    auto enter = [&]() {
        const int tok = un.token(ua, grp);
        ha = kOne || tok < p.T ? un.head(ua, grp) : H;
        sd = dy + ((size_t)tok * H + ha) * D;
        sr = x + (size_t)tok * sx + (size_t)ha * D;
        left = rows;
    };
    if (ua < un.count) enter();
    auto fetch = [&](int slot) {
        GDR2_DCHECK(slot >= 0 && slot < kBwdDepth);
        if (ua < un.count) {
            const bool on = ha < H, ox = on && p.norm;
            const T *g = on ? sd : dy, *r = on ? sr : x;
            cp16(&sh.ring[slot][0][threadIdx.x], g + w.at0, on);
            cp16(&sh.ring[slot][1][threadIdx.x], g + w.at1, on);
            cp16(&sh.ring[slot][2][threadIdx.x], r + w.at0, ox);
            cp16(&sh.ring[slot][3][threadIdx.x], r + w.at1, ox);
            sd += step * D, sr += step * D, ha += step;
            if (--left == 0) {
                ua += un.stride;
                if (ua < un.count) enter();
            }
        }
        cp_commit();
    };
#pragma unroll
    for (int i = 0; i < kBwdDepth; ++i) fetch(i);
    auto position = [&](int v) {
        const int tok = v < un.count ? un.token(v, grp) : 0;
        return p.rot ? p.pos[kOne || tok < p.T ? tok : 0] : 0;
    };
    int pos = position(u);
    Freqs fr;
    fr.load(p, lane);
    stage_gain<D, C>(keys ? p.gk : p.gq, sh.gain);
    __syncthreads();
    F2 gu[N], gv[N], au[N], av[N];
    C::pairs(sh.gain + w.at0, sh.gain + w.at1, gu, gv);
#pragma unroll
    for (int i = 0; i < N; ++i) au[i] = av[i] = f2(0.f, 0.f);
    int slot = 0;
    for (; u < un.count; u += un.stride) {
        const int tok = un.token(u, grp), h0 = kOne || tok < p.T ? un.head(u, grp) : H;
        GDR2_DCHECK(tok >= 0 && tok < p.T + tokens - 1 && slot % kBwdBurst >= 0 && slot < kBwdDepth);
        const int npos = position(u + un.stride);
        fr.angles<D, kOne>(p, pos, tokens, sh.cs[warp], lane);
        F2 tc[N], ts[N];
        load_turn<D, T, kInter>(w, cs, cs + D / 2, tc, ts);
        T *out = dx + (size_t)tok * sdx + (size_t)h0 * D;
#pragma unroll 1
        for (int i = 0, h = h0; i < rows; ++i, h += step, out += step * D) {
            if (slot % kBwdBurst == 0) cp_wait<kBwdBurst>();
            F2 u[N], v[N], y[N], z[N];
            C::get(sh.ring[slot][0][threadIdx.x], sh.ring[slot][1][threadIdx.x], u, v);
#pragma unroll
            for (int i = 0; i < N; ++i)  // the transposed rotation
                turn<kAll>(w.on(i), tc[i], ts[i], tc[i], neg(ts[i]), u[i], v[i], y[i], z[i]);
            if (p.norm) {
                F2 xu[N], xv[N];
                C::get(sh.ring[slot][2][threadIdx.x], sh.ring[slot][3][threadIdx.x], xu, xv);
                F2 q = f2(0.f, 0.f), m = q;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    q = fma(xu[i], xu[i], q);
                    q = fma(xv[i], xv[i], q);
                    u[i] = mul(xu[i], y[i]);
                    v[i] = mul(xv[i], z[i]);
                    m = fma(gu[i], u[i], m);
                    m = fma(gv[i], v[i], m);
                }
                const float qs = sum_row<Y::kLanes>(sum2(q)), ms = sum_row<Y::kLanes>(sum2(m));
                const float n = rsqrtf(qs * (1.f / D) + p.eps), c = -ms * (1.f / D) * n * n;
                const F2 nn = f2(n, n), cc = f2(c, c);
                if (h < H) {  // a lane without a row has n = eps^-1/2, infinite for eps = 0
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        au[i] = fma(u[i], nn, au[i]);
                        av[i] = fma(v[i], nn, av[i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    y[i] = mul(fma(cc, xu[i], mul(gu[i], y[i])), nn);
                    z[i] = mul(fma(cc, xv[i], mul(gv[i], z[i])), nn);
                }
            }
            if (++slot % kBwdBurst == 0) {
#pragma unroll
                for (int x = kBwdBurst; x > 0; --x) fetch(slot - x);
                if (slot == kBwdDepth) slot = 0;
            }
            if (h < H) C::put(out + w.at0, out + w.at1, y, z);
        }
        pos = npos;
    }
    cp_wait<0>();
    if (partial == nullptr) return;
    __syncthreads();  // the ring becomes the table of the lanes' sums
    constexpr int kGroups = kWarps * Y::kRows;
    static_assert(sizeof(sh.ring) >= kGroups * D * sizeof(float), "sums fit the ring");
    float *red = reinterpret_cast<float *>(&sh.ring[0][0][0]), *mine = red + (warp * Y::kRows + grp) * D;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        split(au[i], mine[C::element(i, 0, false, w.at0, w.at1)], mine[C::element(i, 1, false, w.at0, w.at1)]);
        split(av[i], mine[C::element(i, 0, true, w.at0, w.at1)], mine[C::element(i, 1, true, w.at0, w.at1)]);
    }
    __syncthreads();
    if (threadIdx.x < D) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < kGroups; ++i) v += red[i * D + threadIdx.x];
        partial[(size_t)blockIdx.x * D + threadIdx.x] = v;
    }
}

// dg[c] = the partial sums of its CTAs: slice s adds the CTAs s, s + 32, ... in order, then the slices in order.
template <int D>
__global__ void __launch_bounds__(1024) attn_prologue_reduce_kernel(const float *partial, int cq, int ctas,
                                                                    float *dgq, float *dgk) {
    __shared__ float red[32][33];
    const int which = blockIdx.x, c = blockIdx.y * 32 + threadIdx.x % 32, sl = threadIdx.x / 32;
    float *out = which ? dgk : dgq;
    follow();
    if (out == nullptr) return;
    const int a = which ? cq : 0, e = which ? ctas : cq;
    float v = 0.f;
#pragma unroll 4
    for (int i = a + sl; i < e; i += 32) v += __ldcg(partial + (size_t)i * D + c);
    red[sl][threadIdx.x % 32] = v;
    __syncthreads();
    if (sl == 0) {
        float s = 0.f;
#pragma unroll
        for (int x = 0; x < 32; ++x) s += red[x][threadIdx.x];
        out[c] = s;
    }
}

// Lane groups of a token: as many as leave no lane idle (bf16, 2 + 1 heads of 64 with all eight groups on one token: 309
// us forward and 455 backward for 150 MB of rows; with one group a token 77 and 148), more while that leaves fewer than
// two units for each warp of the grid.
// Parts of a token: one warp for all its heads while there are two units for each warp of the grid (a part repeats the
// token's angles; with fewer units the last round leaves most warps idle: 16 packed prompts took 69 us with eight units
// asked for, 51 with two), more below, up to one row a lane.
Units split_units(int T, int Hq, int Hk, int rows, int warps) {
    Units un{};
    const int most = Hq > Hk ? Hq : Hk;
    auto even = [&](int groups) { return Hq % groups == 0 && Hk % groups == 0; };
    auto blocks = [&] { return (((long long)T << un.gl) + rows - 1) / rows; };
    while ((2 << un.gl) <= rows && even(2 << un.gl)) ++un.gl;
    while ((2 << un.gl) <= rows && blocks() < 2LL * warps) ++un.gl;
    while ((1 << (un.log + un.gl)) < most && (blocks() << un.log) < 2LL * warps) ++un.log;
    un.count = (int)(blocks() << un.log);
    un.stride = warps;
    return un;
}

template <int D, typename T, bool kInter, bool kAll, bool kCache>
cudaError_t run_fwd(const AttnPrologueArgs &a, cudaStream_t st) {
    constexpr int smem = sizeof(FwdShared<D, T>), full = kFwdCtas * kAttnSms;
    Units un = split_units(a.T, a.Hq, a.Hk, Layout<D, T>::kRows, full * kWarps);
    const int need = (int)(((long long)un.count + kWarps - 1) / kWarps), grid = need < full ? need : full;
    un.stride = grid * kWarps;
    const bool whole = un.gl == Layout<D, T>::kRowsLog;
    const auto kernel = whole ? attn_prologue_fwd_kernel<D, T, kInter, kAll, kCache, true>
                              : attn_prologue_fwd_kernel<D, T, kInter, kAll, kCache, false>;
    static Allowed allowed[2];
    cudaError_t e = allowed[whole](kernel, smem);
    if (e != cudaSuccess) return e;
    GDR2_LAUNCH(kCache ? "attn_prologue_cache" : "attn_prologue_fwd", st, e = launch(kernel, dim3(grid), dim3(kThreads), smem, 0, st, a, un));
    return e;
}

template <int D, typename T, bool kInter, bool kAll>
cudaError_t run_bwd(const AttnPrologueArgs &a, cudaStream_t st) {
    constexpr int smem = sizeof(BwdShared<D, T>);
    // CTAs in proportion to the heads and a token's angles, which take about the time of kAngles rows; at least one each
    // (7 + 1 bf16 heads of 128, 150 MB of rows: 93 us with 2, 99 with 4, 180 by the heads alone)
    constexpr int kAngles = 2;
    const long long heads = (long long)a.Hq + a.Hk + 2 * kAngles;
    int cq = (int)((kBwdGrid * (long long)(a.Hq + kAngles) + heads / 2) / heads);
    cq = cq < 1 ? 1 : cq > kBwdGrid - 1 ? kBwdGrid - 1 : cq;
    int ck = kBwdGrid - cq;
    auto part = [&](int H, int &ctas) {
        Units un = split_units(a.T, H, 0, Layout<D, T>::kRows, ctas * kWarps);
        const int need = (int)(((long long)un.count + kWarps - 1) / kWarps);
        ctas = need < ctas ? need : ctas;
        un.stride = ctas * kWarps;
        return un;
    };
    const Units uq = part(a.Hq, cq), uk = part(a.Hk, ck);
    const bool whole = uq.gl == Layout<D, T>::kRowsLog && uk.gl == uq.gl;
    const auto kernel = whole ? attn_prologue_bwd_kernel<D, T, kInter, kAll, true> : attn_prologue_bwd_kernel<D, T, kInter, kAll, false>;
    static Allowed allowed[2];
    cudaError_t e = allowed[whole](kernel, smem);
    if (e != cudaSuccess) return e;
    float *partial = a.dgq || a.dgk ? static_cast<float *>(a.workspace) : nullptr;
    GDR2_LAUNCH("attn_prologue_bwd", st, e = launch(kernel, dim3(cq + ck), dim3(kThreads), smem, 0, st, a, uq, uk, cq, partial));
    if (e != cudaSuccess || partial == nullptr) return e;
    GDR2_LAUNCH("attn_prologue_reduce", st,
                e = launch(attn_prologue_reduce_kernel<D>, dim3(2, D / 32), dim3(1024), 0, 0, st,
                                     (const float *)partial, cq, cq + ck, a.dgq, a.dgk));
    return e;
}

// f.template operator()<D, T, interleaved, the whole row rotated>() for the call
template <int D, typename T, typename F> cudaError_t dispatch_rot(const AttnPrologueArgs &a, F f) {
    if (a.interleaved) return a.rot == D ? f.template operator()<D, T, true, true>() : f.template operator()<D, T, true, false>();
    return a.rot == D ? f.template operator()<D, T, false, true>() : f.template operator()<D, T, false, false>();
}
template <typename F> cudaError_t dispatch(const AttnPrologueArgs &a, F f) {
    if (a.dtype == 1) return a.d == 128 ? dispatch_rot<128, __nv_bfloat16>(a, f) : dispatch_rot<64, __nv_bfloat16>(a, f);
    return a.d == 128 ? dispatch_rot<128, float>(a, f) : dispatch_rot<64, float>(a, f);
}

struct Fwd {
    const AttnPrologueArgs &a;
    bool cache;
    cudaStream_t st;
    template <int D, typename T, bool I, bool A> cudaError_t operator()() const {
        return cache ? run_fwd<D, T, I, A, true>(a, st) : run_fwd<D, T, I, A, false>(a, st);
    }
};
struct Bwd {
    const AttnPrologueArgs &a;
    cudaStream_t st;
    template <int D, typename T, bool I, bool A> cudaError_t operator()() const { return run_bwd<D, T, I, A>(a, st); }
};

}  // namespace

size_t attn_prologue_workspace_bytes(int d) { return (size_t)kBwdGrid * d * sizeof(float); }

int status_take_attn_prologue() { return take_status(); }

cudaError_t launch_attn_prologue_fwd(const AttnPrologueArgs &a, cudaStream_t st) { return dispatch(a, Fwd{a, false, st}); }
cudaError_t launch_attn_prologue_cache(const AttnPrologueArgs &a, cudaStream_t st) {
    AttnPrologueArgs b = a;
    b.by_page = Divisor(a.page_size);
    return dispatch(b, Fwd{b, true, st});
}
cudaError_t launch_attn_prologue_bwd(const AttnPrologueArgs &a, cudaStream_t st) { return dispatch(a, Bwd{a, st}); }

}  // namespace gdr2
