// kv_pages.cu -- bookkeeping of the paged key-value cache on the device (sm_100a): reserving pages for new tokens,
// forking (and reordering and releasing) sequences, compacting the pool, and the page copies these need.
//
// A cache: pools k_pages, v_pages [num_pages, Hk, page_size, d]; table [R, P], entry (r, j) the page of tokens
// j page_size ... of sequence r (anything outside [0, num_pages) means none); lens [R]; ref [num_pages], how many
// entries name a page (plus what the caller adds to pin one); a page with ref <= 0 is free. Pages are handed out
// lowest number first, to the entries in (r, j) order, so every call has one possible result.
//
// The bookkeeping moves 8 (R P + num_pages) bytes or so, a microsecond of HBM time at most; its cost is the few
// dependent passes (count, rank, assign). It runs as one kernel on one cluster of up to 8 CTAs whose barriers separate
// the passes: a kernel for each pass would pay a launch for each, a single CTA the loads of one SM. Every warp owns a
// contiguous strip of the items (pages, entries or sequences) and counts by ballots, so a rank is the sum of the
// strips before (a scan over at most 256 numbers) plus a population count. Integer atomics only, whose order does
// not show. The copies follow in a kernel over the whole GPU, one warp for each 4 KB of a page's rows of one head.
#include <cooperative_groups.h>

#include "attn.h"
#include "common.cuh"
#include "kernels.h"

namespace gdr2 {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kMaxCluster = 8;
constexpr int kMaxWarps = kMaxCluster * kThreads / 32;
constexpr int kOwners = 4096;

// Workspace, ints: strip totals of three counts, numbers for the copies, then lists.
struct Lists {
    int *ta, *tb, *tc;  // [kMaxWarps] strip totals
    int *ncopy;      // [4] copies; compact: the live pages
    int *pages;      // [num_pages] each strip's free pages from its start on (compact: those below the live count, by rank)
    int *high;       // [num_pages] compact: live pages at or above the live count, by rank
    int *rank;       // [num_pages] compact: rank of such a page
    int *needs;      // [R P / 32] reserve: which of 32 entries need a page, a bit each
    int *owner;      // [R] fork: who keeps a sequence's partly filled page
    int *src, *dst, *rows;  // [R] fork: copies
};

size_t need_words(int R, int P) { return ((size_t)R * P + 31) / 32; }

Lists lists(void *ws, int R, int P, int num_pages) {
    Lists w;
    int *p = static_cast<int *>(ws);
    auto take = [&](size_t n) {
        int *x = p;
        p += (n + 3) / 4 * 4;
        return x;
    };
    w.ta = take(kMaxWarps), w.tb = take(kMaxWarps), w.tc = take(kMaxWarps), w.ncopy = take(4);
    w.pages = take(num_pages), w.high = take(num_pages), w.rank = take(num_pages);
    w.needs = take(need_words(R, P));
    w.owner = take(R), w.src = take(R), w.dst = take(R), w.rows = take(R);
    return w;
}

// A warp's strip of n items: [first, last), whole multiples of 32 long.
struct Strip {
    int first, last;
};
__device__ __forceinline__ int strip_length(int n, int warps) { return ((n + warps - 1) / warps + 31) / 32 * 32; }
__device__ __forceinline__ Strip strip(int n, int warp, int warps) {
    const int len = strip_length(n, warps);
    Strip s;
    s.first = (int)min((long long)n, (long long)len * warp);
    s.last = (int)min((long long)n, (long long)s.first + len);
    return s;
}

constexpr int kAhead = 8;  // items of a lane whose loads are in flight together

// The place (r, j) of a lane's entries i, i + 32, ... of the table: a division only where the row changes. (Divided at
// every entry, with the two by the page size that the comparisons of tokens below do without, the instructions of the
// passes outweighed their loads: 23 us for a reservation of 256 sequences and 66,304 entries.)
struct Cell {
    int r, j;
    __device__ __forceinline__ Cell(int i, int P) : r(i / P), j(i - r * P) {}
    __device__ __forceinline__ void next(int P) {
        j += 32;
        if (j >= P) {
            const int q = j / P;
            r += q, j -= q * P;
        }
    }
};

__device__ __forceinline__ int valid(int e, int num_pages) { return e >= 0 && e < num_pages ? e : -1; }
__device__ __forceinline__ int entry(const int *table, int at, int num_pages) { return valid(__ldcg(table + at), num_pages); }

// The number of free pages in a strip.
__device__ __forceinline__ int count_free(const int *ref, Strip s, int lane) {
    int c = 0;
    for (int b = s.first; b < s.last; b += 32 * kAhead) {
        int n[kAhead];
#pragma unroll
        for (int x = 0; x < kAhead; ++x) n[x] = b + 32 * x + lane < s.last ? __ldcg(ref + b + 32 * x + lane) : 1;
#pragma unroll
        for (int x = 0; x < kAhead; ++x) c += n[x] <= 0;
    }
    return __reduce_add_sync(0xffffffffu, c);
}
// The same, and the free pages listed at list[s.first ...]; the counts are copied to `copy` unless it is null.
__device__ __forceinline__ int list_free(const int *ref, Strip s, int *list, int *copy, int lane) {
    int c = 0;
    for (int b = s.first; b < s.last; b += 32 * kAhead) {
        int n[kAhead];
#pragma unroll
        for (int x = 0; x < kAhead; ++x) n[x] = b + 32 * x + lane < s.last ? __ldcg(ref + b + 32 * x + lane) : 1;
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            const int i = b + 32 * x + lane;
            const unsigned m = __ballot_sync(0xffffffffu, n[x] <= 0);
            if (n[x] <= 0) list[s.first + c + __popc(m & ((1u << lane) - 1))] = i;
            if (copy && i < s.last) copy[i] = n[x];
            c += __popc(m);
        }
    }
    return c;
}

// pre[i] = t[0] + ... + t[i - 1], i <= warps (a multiple of 32); by one warp. t: global memory, or shared memory where
// the cluster is one CTA.
__device__ __forceinline__ void prefix(const int *t, int warps, int *pre, int lane) {
    const int each = warps / 32;
    int v[kMaxWarps / 32], sum = 0;
#pragma unroll
    for (int i = 0; i < kMaxWarps / 32; ++i) {
        v[i] = i < each ? *static_cast<const volatile int *>(t + lane * each + i) : 0;
        sum += v[i];
    }
    int at = sum;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, at, x);
        if (lane >= x) at += y;
    }
    at -= sum;
#pragma unroll
    for (int i = 0; i < kMaxWarps / 32; ++i)
        if (i < each) {
            pre[lane * each + i] = at;
            at += v[i];
        }
    if (lane == 31) pre[warps] = at;
}
// The warp's total. It is zero in nearly every call: then one vote tells.
__device__ __forceinline__ long long total(long long x) {
    if (!__any_sync(0xffffffffu, x != 0)) return 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
constexpr long long kMost = 0x7fffffff;  // counts are held to it
// The free page of a rank: the strip whose list holds it, and its place there.
__device__ __forceinline__ int free_page(const int *pages, const int *pre, int rank, int warps, int length) {
    int a = 0, e = warps;  // pre[a] <= rank < pre[e]
    while (e - a > 1) {
        const int mid = (a + e) / 2;
        if (pre[mid] <= rank)
            a = mid;
        else
            e = mid;
    }
    GDR2_DCHECK(rank >= pre[a] && rank < pre[a + 1]);
    return __ldcg(pages + a * length + rank - pre[a]);
}

struct Place {
    int gid, threads, warp, warps, lane;
};
__device__ __forceinline__ Place place() {
    Place t;
    t.gid = blockIdx.x * kThreads + threadIdx.x;
    t.threads = gridDim.x * kThreads;
    t.warp = t.gid >> 5, t.warps = t.threads >> 5, t.lane = threadIdx.x & 31;
    return t;
}

// The blocks that copies move: the rows of one head of a page, page_size of them of row_bytes each, in both pools.
struct Blocks {
    uint8_t *k, *v;
    int Hk, page_size, row_bytes;
};

// Copies the first rows[i] (null: all) token rows of every head of page src[i] to page dst[i], i < n. A warp moves up to
// 4 KB of one block, eight 16-byte loads a lane in flight; the caller's warps are warp, warp + warps, ...
__device__ __forceinline__ void copy_rows(int n, const int *src, const int *dst, const int *rows, const Blocks &bl, uint32_t warp,
                                          uint32_t warps, int lane) {
    constexpr int kPiece = 4096;
    const long long block = (long long)bl.page_size * bl.row_bytes;
    const uint32_t pieces = (uint32_t)((block + kPiece - 1) / kPiece), heads = 2 * bl.Hk;
    const uint32_t items = (uint32_t)n * heads * pieces;  // below 2^32: checked for the whole pool
    for (uint32_t x = warp; x < items; x += warps) {
        const uint32_t y = x / pieces, piece = x - y * pieces, i = y / heads, hh = y - i * heads, h = hh >> 1;
        const long long bytes = rows ? (long long)__ldcg(rows + i) * bl.row_bytes : block;
        uint8_t *pool = hh & 1 ? bl.v : bl.k;
        GDR2_DCHECK(i < (uint32_t)n && h < (uint32_t)bl.Hk && bytes <= block && __ldcg(src + i) != __ldcg(dst + i));
        const uint8_t *s = pool + ((long long)__ldcg(src + i) * bl.Hk + h) * block;
        uint8_t *d = pool + ((long long)__ldcg(dst + i) * bl.Hk + h) * block;
        const long long base = (long long)piece * kPiece + lane * 16;
        uint4 r[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (base + u * 512 < bytes) r[u] = __ldcs(reinterpret_cast<const uint4 *>(s + base + u * 512));
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (base + u * 512 < bytes) *reinterpret_cast<uint4 *>(d + base + u * 512) = r[u];
    }
}

// Pages for tokens [lens[r], want[r]) of every sequence: its entries from the one of token lens[r] to the one of token
// want[r] - 1 that are empty get a page. Before that, pages wholly behind the window of the token at lens[r] are
// released. The grid is one cluster.
__global__ void __launch_bounds__(kThreads) kv_reserve_kernel(KvPagesArgs a, Lists w) {
    cg::cluster_group cl = cg::this_cluster();
    const Place t = place();
    const int E = a.R * a.P, ps = a.page_size;
    follow();
    __shared__ int need[kMaxWarps + 1], free[kMaxWarps + 1], sums[3][kThreads / 32];
    __shared__ long long past;
    const bool one = gridDim.x == 1;
    int *ta = one ? sums[0] : w.ta, *tb = one ? sums[1] : w.tb, *tc = one ? sums[2] : w.tc;
    const Strip es = strip(E, t.warp, t.warps), pg = strip(a.num_pages, t.warp, t.warps);
    if (es.first + t.lane * 32 < es.last) {  // the entries' way to L2 overlaps that of the counts
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.table + es.first + t.lane * 32));
        const int r = (es.first + t.lane * 32) / a.P;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.lens + r));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.want + r));
    }
    // the counts are copied and free pages listed on the way; a window's releases change them, so then list later
    int nfree = list_free(a.ref, pg, w.pages, a.ref_out, t.lane);
    if (a.window > 0) cl.sync();
    // entries: released, copied, and counted where a page is needed
    int c = 0;
    Cell at(es.first + t.lane, a.P);
    for (int b = es.first; b < es.last; b += 32 * kAhead) {
        int e[kAhead], len[kAhead], want[kAhead], tok[kAhead];  // tok: the first token of the entry's page
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            const int i = b + 32 * x + t.lane;
            const bool in = i < es.last;
            tok[x] = at.j * ps;
            e[x] = in ? __ldcg(a.table + i) : 0;
            len[x] = in ? a.lens[at.r] : 0;
            want[x] = in ? a.want[at.r] : 0;
            at.next(a.P);
        }
        int words = 0;
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            const int i = b + 32 * x + t.lane;
            bool is = false;
            if (i < es.last) {
                e[x] = valid(e[x], a.num_pages);
                len[x] = max(len[x], 0);
                if (e[x] >= 0 && a.window > 0 && tok[x] + ps <= len[x] - (a.window - 1)) {
                    atomicSub(a.ref_out + e[x], 1);
                    e[x] = -1;
                }
                a.table_out[i] = e[x];
                is = e[x] < 0 && tok[x] + ps > len[x] && tok[x] < want[x];
            }
            const int m = (int)__ballot_sync(0xffffffffu, is);
            c += __popc(m);
            words = t.lane == x ? m : words;
        }
        if (t.lane < kAhead && b + 32 * t.lane < es.last) w.needs[b / 32 + t.lane] = words;  // strips start at whole words
    }
    long long over = 0;  // entries past the table's end: from the one of token lens[r] on, if that lies there too
    for (int r = t.gid; r < a.R; r += t.threads) {
        const int want = a.want[r], last = want > 0 ? (want - 1) / ps + 1 : 0;
        if (last > a.P) over += max(0, last - max(a.P, a.lens[r] / ps));
    }
    over = min(total(over), kMost);
    if (a.window > 0) {
        cl.sync();
        nfree = list_free(a.ref_out, pg, w.pages, nullptr, t.lane);
    }
    if (t.lane == 0) ta[t.warp] = c, tb[t.warp] = nfree, tc[t.warp] = (int)over;
    cl.sync();
    if (threadIdx.x < 32) prefix(ta, t.warps, need, t.lane);
    if (threadIdx.x / 32 == 1) prefix(tb, t.warps, free, t.lane);
    if (threadIdx.x / 32 == 2) {
        long long x = 0;
        for (int i = t.lane; i < t.warps; i += 32) x += *static_cast<const volatile int *>(tc + i);
        x = total(x);
        if (t.lane == 0) past = x;
    }
    __syncthreads();
    const int all = free[t.warps], length = strip_length(a.num_pages, t.warps);
    int rank0 = need[t.warp];
    if (t.gid == 0) *a.count_out = (int)min(past + max(0, need[t.warps] - all), kMost);
    if (c == 0) return;
    for (int g = es.first / 32; g * 32 < es.last; g += 32) {
        const int mine = (g + t.lane) * 32 < es.last ? __ldcg(w.needs + g + t.lane) : 0;
        for (unsigned some = __ballot_sync(0xffffffffu, mine != 0); some; some &= some - 1) {
            const int x = __ffs(some) - 1;
            const unsigned m = (unsigned)__shfl_sync(0xffffffffu, mine, x);
            const int rank = rank0 + __popc(m & ((1u << t.lane) - 1));
            if ((m >> t.lane & 1) && rank < all) {
                const int page = free_page(w.pages, free, rank, t.warps, length);
                GDR2_DCHECK(page >= 0 && page < a.num_pages && (g + x) * 32 + t.lane < es.last);
                a.table_out[(g + x) * 32 + t.lane] = page;
                a.ref_out[page] = 1;
            }
            rank0 += __popc(m);
        }
    }
}

// Every sequence r takes over the content of sequence parent[r] as it was before the call (r itself: stays; outside
// [0, R): released). Full pages are shared. The partly filled last page stays with one taker, the parent itself if it
// is one, else the first; every other taker gets a copy of its tokens on a fresh page. The grid is one cluster.
__global__ void __launch_bounds__(kThreads) kv_fork_kernel(KvPagesArgs a, Lists w, Blocks bl, int copy) {
    cg::cluster_group cl = cg::this_cluster();
    const Place t = place();
    const int E = a.R * a.P, ps = a.page_size;
    follow();
    const Strip es = strip(E, t.warp, t.warps), pg = strip(a.num_pages, t.warp, t.warps), rs = strip(a.R, t.warp, t.warps);
    // who keeps a sequence's last page: up to kOwners sequences each CTA finds it for itself
    __shared__ int need[kMaxWarps + 1], free[kMaxWarps + 1], owner_here[kOwners], sums[2][kThreads / 32];
    const bool one = gridDim.x == 1;
    int *ta = one ? sums[0] : w.ta, *tb = one ? sums[1] : w.tb;
    const bool here = a.R <= kOwners;
    int *owner = here ? owner_here : w.owner;
    const int r0 = here ? threadIdx.x : t.gid, rn = here ? kThreads : t.threads;
    for (int r = r0; r < a.R; r += rn) owner[r] = a.R;
    if (here)
        __syncthreads();
    else
        cl.sync();
    for (int r = r0; r < a.R; r += rn) {
        const int p = a.parent[r];
        if (p >= 0 && p < a.R) atomicMin(owner + p, r == p ? -1 : r);
    }
    for (int b = pg.first; b < pg.last; b += 32 * kAhead) {
        int n[kAhead];
#pragma unroll
        for (int x = 0; x < kAhead; ++x) n[x] = b + 32 * x + t.lane < pg.last ? __ldcg(a.ref + b + 32 * x + t.lane) : 0;
#pragma unroll
        for (int x = 0; x < kAhead; ++x)
            if (b + 32 * x + t.lane < pg.last) a.ref_out[b + 32 * x + t.lane] = n[x];
    }
    cl.sync();
    auto length = [&](int p) { return (int)min((long long)max(a.lens[p], 0), (long long)a.P * ps); };
    auto owns = [&](int r, int p) { return (here ? owner_here[p] : __ldcg(w.owner + p)) == (r == p ? -1 : r); };
    constexpr int kFew = 4;
    Cell at(es.first + t.lane, a.P);
    for (int b = es.first; b < es.last; b += 32 * kFew) {
        int was[kFew], took[kFew], r[kFew], j[kFew], p[kFew], len[kFew];
        bool own[kFew];
#pragma unroll
        for (int x = 0; x < kFew; ++x) {
            const int i = b + 32 * x + t.lane;
            r[x] = at.r, j[x] = at.j;
            at.next(a.P);
            p[x] = i < es.last ? a.parent[r[x]] : -1;
            was[x] = i < es.last ? __ldcg(a.table + i) : -1;
            if (p[x] >= a.R) p[x] = -1;
        }
#pragma unroll
        for (int x = 0; x < kFew; ++x) {
            took[x] = p[x] >= 0 ? __ldcg(a.table + p[x] * a.P + j[x]) : -1;
            len[x] = p[x] >= 0 ? length(p[x]) : 0;
            own[x] = p[x] >= 0 && owns(r[x], p[x]);
        }
#pragma unroll
        for (int x = 0; x < kFew; ++x) {
            const int i = b + 32 * x + t.lane;
            if (i < es.last) {
                const int o = valid(was[x], a.num_pages);
                const int e = own[x] || (j[x] + 1) * ps <= len[x] ? valid(took[x], a.num_pages) : -1;
                if (p[x] != r[x]) {
                    if (o >= 0) atomicSub(a.ref_out + o, 1);
                    if (e >= 0) atomicAdd(a.ref_out + e, 1);
                }
                a.table_out[i] = e;
                if (j[x] == 0) a.lens_out[r[x]] = p[x] >= 0 ? a.lens[p[x]] : 0;  // as it is, inside the table or not
            }
        }
    }
    // sequences that need a copy: its source, or -1
    auto source = [&](int r) {
        if (r >= rs.last) return -1;
        const int p = a.parent[r];
        if (p < 0 || p >= a.R || owns(r, p)) return -1;
        const int len = length(p);
        return len % ps ? entry(a.table, p * a.P + len / ps, a.num_pages) : -1;
    };
    int c = 0;
    for (int b = rs.first; b < rs.last; b += 32) c += __popc(__ballot_sync(0xffffffffu, source(b + t.lane) >= 0));
    cl.sync();
    const int nfree = list_free(a.ref_out, pg, w.pages, nullptr, t.lane);
    if (t.lane == 0) ta[t.warp] = c, tb[t.warp] = nfree;
    cl.sync();
    if (threadIdx.x < 32) prefix(ta, t.warps, need, t.lane);
    if (threadIdx.x / 32 == 1) prefix(tb, t.warps, free, t.lane);
    __syncthreads();
    const int all = free[t.warps], needed = need[t.warps], each = strip_length(a.num_pages, t.warps);
    int rank0 = need[t.warp];
    if (t.gid == 0) {
        w.ncopy[0] = min(needed, all);
        *a.count_out = max(0, needed - all);
    }
    for (int b = rs.first; b < rs.last; b += 32) {
        const int r = b + t.lane, src = source(r);
        const unsigned m = __ballot_sync(0xffffffffu, src >= 0);
        const int rank = rank0 + __popc(m & ((1u << t.lane) - 1));
        if (src >= 0) {
            const int len = length(a.parent[r]), j = len / ps;
            if (rank < all) {
                const int page = free_page(w.pages, free, rank, t.warps, each);
                GDR2_DCHECK(page >= 0 && page < a.num_pages && j < a.P && rank < a.R);
                a.table_out[r * a.P + j] = page;
                a.ref_out[page] = 1;
                w.src[rank] = src, w.dst[rank] = page, w.rows[rank] = len - j * ps;
            } else {
                a.lens_out[r] = j * ps;
            }
        }
        rank0 += __popc(m);
    }
    if (copy) {
        cl.sync();
        copy_rows(min(needed, all), w.src, w.dst, w.rows, bl, t.warp, t.warps, t.lane);
    }
}

// The rest of a compaction, once the lists are there: counts and pages move, the table follows.
__device__ __forceinline__ void move_pages(const KvPagesArgs &a, const Lists &w, const Blocks &bl, int moves, int live, const Place &t) {
    for (int k = t.gid; k < moves; k += t.threads) {
        const int src = __ldcg(w.high + k), dst = __ldcg(w.pages + k);
        const int n = __ldcg(a.ref + src);
        a.ref_out[dst] = n;
        a.ref_out[src] = 0;
    }
    const uint32_t E = (uint32_t)a.R * a.P, th = t.threads;  // E < 2^31 and a step over the grid behind it: unsigned holds both
    for (uint32_t b = t.gid; b < E; b += 4 * th) {
        int e[4], k[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) e[x] = b + x * th < E ? entry(a.table, b + x * th, a.num_pages) : -1;
#pragma unroll
        for (int x = 0; x < 4; ++x) k[x] = e[x] >= live ? __ldcg(w.rank + e[x]) : -1;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (k[x] >= 0) e[x] = __ldcg(w.pages + k[x]);
            if (b + x * th < E) a.table_out[b + x * th] = e[x];
        }
    }
    copy_rows(moves, w.high, w.pages, nullptr, bl, t.warp, t.warps, t.lane);
}

// Live pages numbered live or above move to the free numbers below, in order; table and counts follow (here if `copy`,
// else in kv_move_kernel).
__global__ void __launch_bounds__(kThreads) kv_compact_kernel(KvPagesArgs a, Lists w, Blocks bl, int copy) {
    cg::cluster_group cl = cg::this_cluster();
    const Place t = place();
    follow();
    const Strip pg = strip(a.num_pages, t.warp, t.warps);
    __shared__ int pre[kMaxWarps + 1], sums[kThreads / 32];
    int *ta = gridDim.x == 1 ? sums : w.ta;
    const int nf = count_free(a.ref, pg, t.lane);
    if (t.lane == 0) ta[t.warp] = pg.last - pg.first - nf;
    cl.sync();
    if (threadIdx.x < 32) prefix(ta, t.warps, pre, t.lane);
    __syncthreads();
    int live0 = pre[t.warp];          // live pages before this strip
    const int live = pre[t.warps];
    // live pages below number `live`: those of the strips before the one that holds it, and of its first part
    const int len = strip_length(a.num_pages, t.warps), mid = live / len;
    const Strip part{mid * len, live};
    const int below = pre[mid] + live - part.first - count_free(a.ref, part, t.lane);
    const int moves = live - below;  // as many live above as free below
    for (int b = pg.first; b < pg.last; b += 32 * kAhead) {
        int n[kAhead];
#pragma unroll
        for (int x = 0; x < kAhead; ++x) n[x] = b + 32 * x + t.lane < pg.last ? __ldcg(a.ref + b + 32 * x + t.lane) : 0;
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            const int i = b + 32 * x + t.lane;
            const bool is = n[x] > 0;
            const unsigned m = __ballot_sync(0xffffffffu, is);
            const int lb = live0 + __popc(m & ((1u << t.lane) - 1));  // live pages before i
            if (i < pg.last) {
                if (i < live) {
                    GDR2_DCHECK(lb <= i);
                    if (is)
                        a.ref_out[i] = n[x];
                    else
                        w.pages[i - lb] = i;
                } else {
                    w.rank[i] = is ? lb - below : -1;
                    GDR2_DCHECK(!is || (lb >= below && lb - below < moves));
                    if (is)
                        w.high[lb - below] = i;
                    else
                        a.ref_out[i] = 0;
                }
            }
            live0 += __popc(m);
        }
    }
    if (t.gid == 0) {
        w.ncopy[0] = moves, w.ncopy[1] = live;
        *a.count_out = live;
    }
    if (copy) {
        cl.sync();
        move_pages(a, w, bl, moves, live, t);
    }
}

__global__ void __launch_bounds__(256) kv_move_kernel(KvPagesArgs a, Lists w, Blocks bl) {
    follow();
    Place t;
    t.gid = blockIdx.x * 256 + threadIdx.x, t.threads = gridDim.x * 256;
    t.warp = t.gid >> 5, t.warps = t.threads >> 5, t.lane = threadIdx.x & 31;
    const int2 n = __ldcg(reinterpret_cast<const int2 *>(w.ncopy));
    move_pages(a, w, bl, n.x, n.y, t);
}

// Copies by a kernel of its own over the whole GPU.
__global__ void __launch_bounds__(256) kv_copy_kernel(const int *ncopy, const int *src, const int *dst, const int *rows, Blocks bl) {
    follow();
    copy_rows(__ldcg(ncopy), src, dst, rows, bl, blockIdx.x * 8 + (threadIdx.x >> 5), gridDim.x * 8, threadIdx.x & 31);
}

// CTAs of the cluster: one while each of its threads has a few items, the largest portable cluster above that, or when
// it copies pages too.
int cluster_size(const KvPagesArgs &a, bool copy) {
    const long long items = (long long)a.R * a.P + a.num_pages;
    int c = copy ? kMaxCluster : 1;
    while (c < kMaxCluster && items > 4LL * c * kThreads) c *= 2;
    return c;
}

Blocks blocks(const KvPagesArgs &a) {
    return Blocks{(uint8_t *)a.k_pages, (uint8_t *)a.v_pages, a.Hk, a.page_size, a.d * (a.dtype == 1 ? 2 : 4)};
}

// Whether the cluster copies the pages itself, which saves the host the second launch, 2.3 us a call, but has eight SMs
// to copy with. By the bytes really moved, us of a call from Python and of the device alone, inside / by a kernel of
// their own:
//                           0.25 MB              1 MB                 2 MB                 4 MB
//   fork, call              15.8 / 18.1          15.8 / 18.1          17.3 / 18.3          21.5 / 18.1
//   fork, device            11.5 / 10.6          12.7 / 11.0          16.9 / 12.1          21.2 / 11.1
//   compaction, call        13.6 / 15.8          13.7 / 15.8          13.8 / 16.1          16.1 / 15.8
//   compaction, device       6.2 / 5.1            8.0 / 5.9           10.9 / 5.7           15.8 / 5.5
// (32, 32, 256 and 32 forks; 64, 512, 512 and 64 pages.) So a call that the host makes copies inside up to 2 MB. The
// border is on what a call can move at most, and that is about twice what it moves: a partly filled page is half full,
// and of num_pages / 2 pages a compaction moves live (1 - live / num_pages), at most half of them, where the live ones
// are spread evenly. A captured call, whose launches cost the host nothing, always leaves the copies to the other kernel.
constexpr long long kOwnCopy = 4 << 20;
bool own_copy(const Blocks &bl, long long most, cudaStream_t st) {
    const long long page = 2LL * bl.Hk * bl.page_size * bl.row_bytes;  // below 2^43: copies_fit
    if (most > kOwnCopy / page) return false;
    cudaStreamCaptureStatus s = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(st, &s) != cudaSuccess) {  // s is not set then; the launch will say what is wrong
        (void)cudaGetLastError();
        return true;
    }
    return s == cudaStreamCaptureStatusNone;
}

// CTAs of a copy over the whole GPU: a warp for each 4 KB that may move, eight CTAs an SM at most.
int copy_grid(const Blocks &bl, long long most) {
    const long long pieces = ((long long)bl.page_size * bl.row_bytes + 4095) / 4096;
    const long long want = (most * bl.Hk * 2 * pieces + 7) / 8, full = 8LL * kAttnSms;
    return (int)(want < full ? want : full);
}

}  // namespace

size_t kv_workspace_bytes(int R, int P, int num_pages) {
    auto whole = [](size_t n) { return (n + 3) / 4 * 4; };
    return (3 * (size_t)kMaxWarps + 4 + 3 * whole(num_pages) + whole(need_words(R, P)) + 4 * whole(R)) * sizeof(int);
}

int status_take_kv_pages() { return take_status(); }

cudaError_t launch_kv_reserve(const KvPagesArgs &a, cudaStream_t st) {
    const int c = cluster_size(a, false);
    cudaError_t e;
    GDR2_LAUNCH("kv_reserve", st,
                e = launch(kv_reserve_kernel, dim3(c), dim3(kThreads), 0, c, st, a, lists(a.workspace, a.R, a.P, a.num_pages)));
    return e;
}

cudaError_t launch_kv_fork(const KvPagesArgs &a, cudaStream_t st) {
    const Lists w = lists(a.workspace, a.R, a.P, a.num_pages);
    const Blocks bl = blocks(a);
    const bool own = own_copy(bl, a.R, st);
    const int c = cluster_size(a, own);
    cudaError_t e;
    GDR2_LAUNCH("kv_fork", st, e = launch(kv_fork_kernel, dim3(c), dim3(kThreads), 0, c, st, a, w, bl, (int)own));
    if (e != cudaSuccess || own) return e;
    GDR2_LAUNCH("kv_copy", st,
                e = launch(kv_copy_kernel, dim3(copy_grid(bl, a.R)), dim3(256), 0, 0, st, (const int *)w.ncopy,
                           (const int *)w.src, (const int *)w.dst, (const int *)w.rows, bl));
    return e;
}

cudaError_t launch_kv_compact(const KvPagesArgs &a, cudaStream_t st) {
    const Lists w = lists(a.workspace, a.R, a.P, a.num_pages);
    const Blocks bl = blocks(a);
    const long long most = a.num_pages / 2;  // a live page above for each free one below
    const bool own = own_copy(bl, most, st);
    const int c = cluster_size(a, own);
    cudaError_t e;
    GDR2_LAUNCH("kv_compact", st, e = launch(kv_compact_kernel, dim3(c), dim3(kThreads), 0, c, st, a, w, bl, (int)own));
    if (e != cudaSuccess || own) return e;
    GDR2_LAUNCH("kv_move", st, e = launch(kv_move_kernel, dim3(copy_grid(bl, most)), dim3(256), 0, 0, st, a, w, bl));
    return e;
}

}  // namespace gdr2
