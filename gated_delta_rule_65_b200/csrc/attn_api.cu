// attn_api.cu -- the extern "C" boundary of the attention half of the hybrid cell (declared in include/gdr2.h).
//
// As in gdr2_api.cu: arguments are validated on the host before anything is launched, kernels go to the caller's
// stream, and nothing here allocates, frees or synchronises.
#include <math.h>
#include <stdint.h>

#include "attn.h"
#include "gdr2.h"

namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool ok_ptr(const void *p) { return p != nullptr && aligned(p, 16); }
bool ok_num(const void *p) { return p != nullptr && aligned(p, 4); }  // arrays of ints and gains: their own alignment
bool opt_num(const void *p) { return p == nullptr || aligned(p, 4); }

int check_heads(int Hq, int Hk, int d, int dtype) {
    if (Hq <= 0 || Hk <= 0 || d <= 0) return GDR2_ERR_INVALID_ARG;
    if (dtype != GDR2_F32 && dtype != GDR2_BF16) return GDR2_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return GDR2_ERR_UNSUPPORTED;
    if (Hq > 65535 || Hk > 65535) return GDR2_ERR_UNSUPPORTED;
    return GDR2_OK;
}

// A token's rows of H heads, `stride` elements from token to token; 16-byte accesses at every row.
bool ok_stride(long long stride, int H, int d, int dtype) {
    return stride >= (long long)H * d && stride % (dtype == GDR2_BF16 ? 8 : 4) == 0;
}

int check_prologue(int T, int Hq, int Hk, int d, int dtype, int norm, const float *gq, const float *gk, float eps,
                   const int *pos, const double *freqs, int rot) {
    const int st = check_heads(Hq, Hk, d, dtype);
    if (st != GDR2_OK) return st;
    if (T <= 0 || rot < 0 || rot > d || (norm != 0 && norm != 1)) return GDR2_ERR_INVALID_ARG;
    if (rot % 16 != 0) return GDR2_ERR_UNSUPPORTED;
    if (norm ? !(eps >= 0.f) : gq != nullptr || gk != nullptr) return GDR2_ERR_INVALID_ARG;
    if (!opt_num(gq) || !opt_num(gk)) return GDR2_ERR_INVALID_ARG;
    if (rot > 0 && (!ok_num(pos) || freqs == nullptr || !aligned(freqs, 8))) return GDR2_ERR_INVALID_ARG;
    return GDR2_OK;
}

int check_pages(int R, int P, int page_size, int num_pages) {
    if (R <= 0 || P <= 0 || page_size <= 0 || num_pages <= 0) return GDR2_ERR_INVALID_ARG;
    // token numbers and places in the table are 32-bit
    if ((long long)P * page_size > 0x7fff0000LL || (long long)R * P > 0x7fff0000LL || num_pages > 0x7fff0000)
        return GDR2_ERR_UNSUPPORTED;
    return GDR2_OK;
}

int check_decode(const gdr2::AttnDecodeArgs &a, int R) {
    int st = check_heads(a.Hq, a.Hk, a.d, a.dtype);
    if (st == GDR2_OK) st = check_pages(R, a.P, a.page_size, a.num_pages);
    if (st != GDR2_OK) return st;
    if (a.N <= 0 || a.Hq % a.Hk != 0 || a.window < 0) return GDR2_ERR_INVALID_ARG;
    if (a.Hq / a.Hk > 1024) return GDR2_ERR_UNSUPPORTED;  // a CTA for each block of a KV head's query heads
    // rows of the work and token rows of the pool are counted in 32 bits
    if ((long long)a.N * a.Hq > 0x7fffffffLL || (long long)a.Hk * a.page_size > 0x7fffffffLL ||
        (long long)a.Hk * a.page_size * a.num_pages > 0xffffffffLL)
        return GDR2_ERR_UNSUPPORTED;
    return GDR2_OK;
}

// The copies of kv_fork and kv_compact count 4 KB pieces of a page's heads in 32 bits.
bool copies_fit(int Hk, int page_size, int d, int num_pages, int dtype) {
    const long long pieces = ((long long)page_size * d * (dtype == GDR2_BF16 ? 2 : 4) + 4095) / 4096;
    return pieces < (1LL << 31) && pieces * 2 * Hk < (1LL << 31) && pieces * 2 * Hk * num_pages < 0xffff0000LL;
}

int done(cudaError_t e) { return e == cudaSuccess ? GDR2_OK : GDR2_ERR_CUDA; }

// The record of a call, if it is one.
template <typename A> const A *record(const void *args, size_t bytes) {
    return args != nullptr && aligned(args, 8) && bytes == sizeof(A) ? static_cast<const A *>(args) : nullptr;
}

}  // namespace

extern "C" {

int gdr2_rope_freqs(double *freqs, double *mag, int rot, double base, int scaling, double factor, double orig_len,
                    double turns_low, double turns_high) {
    if (freqs == nullptr || rot <= 0 || rot % 2 != 0 || !(base > 0.0) || !isfinite(base)) return GDR2_ERR_INVALID_ARG;
    if (scaling < GDR2_ROPE_PLAIN || scaling > GDR2_ROPE_PARTS) return GDR2_ERR_INVALID_ARG;
    if (scaling != GDR2_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return GDR2_ERR_INVALID_ARG;
    if (scaling == GDR2_ROPE_BASE && rot == 2) return GDR2_ERR_INVALID_ARG;
    if (scaling == GDR2_ROPE_PARTS &&
        (!(orig_len > 0.0) || !isfinite(orig_len) || !(turns_low >= 0.0) || !(turns_high > turns_low) || !isfinite(turns_high)))
        return GDR2_ERR_INVALID_ARG;
    if (scaling == GDR2_ROPE_BASE) base *= pow(factor, (double)rot / (rot - 2));
    for (int i = 0; i < rot / 2; ++i) {
        double f = pow(base, -2.0 * i / rot);
        if (scaling == GDR2_ROPE_LINEAR) f /= factor;
        if (scaling == GDR2_ROPE_PARTS) {
            const double turns = orig_len * f / (2.0 * 3.14159265358979323846);
            double keep = (turns - turns_low) / (turns_high - turns_low);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            f *= keep + (1.0 - keep) / factor;
        }
        freqs[i] = f;
    }
    if (mag) *mag = scaling == GDR2_ROPE_PARTS ? 0.1 * log(factor) + 1.0 : 1.0;
    return GDR2_OK;
}

int gdr2_attn_prologue_fwd(const void *xq, const void *xk, const float *gq, const float *gk, int norm, float eps,
                           const int *pos, const double *freqs, float mag, int rot, int interleaved, void *q, void *k,
                           int T, int Hq, int Hk, int d, int dtype, long long xq_stride, long long xk_stride,
                           void *stream) {
    const int st = check_prologue(T, Hq, Hk, d, dtype, norm, gq, gk, eps, pos, freqs, rot);
    if (st != GDR2_OK) return st;
    if (!ok_ptr(xq) || !ok_ptr(xk) || !ok_ptr(q) || !ok_ptr(k) || !ok_stride(xq_stride, Hq, d, dtype) ||
        !ok_stride(xk_stride, Hk, d, dtype))
        return GDR2_ERR_INVALID_ARG;
    gdr2::AttnPrologueArgs a{};
    a.xq = xq; a.xk = xk; a.gq = gq; a.gk = gk; a.norm = norm; a.eps = eps;
    a.pos = pos; a.freqs = freqs; a.mag = mag; a.rot = rot; a.interleaved = interleaved != 0;
    a.q = q; a.k = k;
    a.T = T; a.Hq = Hq; a.Hk = Hk; a.d = d; a.dtype = dtype; a.sxq = xq_stride; a.sxk = xk_stride;
    return done(gdr2::launch_attn_prologue_fwd(a, (cudaStream_t)stream));
}

size_t gdr2_attn_prologue_workspace_bytes(int d) {
    return d == 64 || d == 128 ? gdr2::attn_prologue_workspace_bytes(d) : 0;
}

int gdr2_attn_prologue_bwd(const void *xq, const void *xk, const float *gq, const float *gk, int norm, float eps,
                           const int *pos, const double *freqs, float mag, int rot, int interleaved, const void *dq,
                           const void *dk, void *dxq, void *dxk, float *dgq, float *dgk, int T, int Hq, int Hk, int d,
                           int dtype, long long xq_stride, long long xk_stride, long long dxq_stride,
                           long long dxk_stride, void *workspace, size_t workspace_bytes, void *stream) {
    const int st = check_prologue(T, Hq, Hk, d, dtype, norm, gq, gk, eps, pos, freqs, rot);
    if (st != GDR2_OK) return st;
    if (!ok_ptr(xq) || !ok_ptr(xk) || !ok_ptr(dq) || !ok_ptr(dk) || !ok_ptr(dxq) || !ok_ptr(dxk) || !opt_num(dgq) ||
        !opt_num(dgk) || (!norm && (dgq || dgk)) || !ok_stride(xq_stride, Hq, d, dtype) ||
        !ok_stride(xk_stride, Hk, d, dtype) || !ok_stride(dxq_stride, Hq, d, dtype) || !ok_stride(dxk_stride, Hk, d, dtype))
        return GDR2_ERR_INVALID_ARG;
    if ((dgq || dgk) && (!ok_ptr(workspace) || workspace_bytes < gdr2::attn_prologue_workspace_bytes(d)))
        return GDR2_ERR_WORKSPACE;
    gdr2::AttnPrologueArgs a{};
    a.xq = xq; a.xk = xk; a.gq = gq; a.gk = gk; a.norm = norm; a.eps = eps;
    a.pos = pos; a.freqs = freqs; a.mag = mag; a.rot = rot; a.interleaved = interleaved != 0;
    a.dq = dq; a.dk = dk; a.dxq = dxq; a.dxk = dxk; a.dgq = dgq; a.dgk = dgk;
    a.T = T; a.Hq = Hq; a.Hk = Hk; a.d = d; a.dtype = dtype;
    a.sxq = xq_stride; a.sxk = xk_stride; a.sdxq = dxq_stride; a.sdxk = dxk_stride;
    a.workspace = workspace;
    return done(gdr2::launch_attn_prologue_bwd(a, (cudaStream_t)stream));
}

int gdr2_attn_prologue_cache(const void *xq, const void *xk, const void *xv, const float *gq, const float *gk, int norm,
                             float eps, const int *seq, const int *pos, const double *freqs, float mag, int rot,
                             int interleaved, void *q, void *k_pages, void *v_pages, const int *table, int T, int Hq,
                             int Hk, int d, int R, int P, int page_size, int num_pages, int dtype, long long xq_stride,
                             long long xk_stride, long long xv_stride, void *stream) {
    int st = check_prologue(T, Hq, Hk, d, dtype, norm, gq, gk, eps, pos, freqs, rot);
    if (st == GDR2_OK) st = check_pages(R, P, page_size, num_pages);
    if (st != GDR2_OK) return st;
    if (!ok_ptr(xq) || !ok_ptr(xk) || !ok_ptr(xv) || !ok_ptr(q) || !ok_ptr(k_pages) || !ok_ptr(v_pages) ||
        !ok_num(seq) || !ok_num(pos) || !ok_num(table) || !ok_stride(xq_stride, Hq, d, dtype) ||
        !ok_stride(xk_stride, Hk, d, dtype) || !ok_stride(xv_stride, Hk, d, dtype))
        return GDR2_ERR_INVALID_ARG;
    gdr2::AttnPrologueArgs a{};
    a.xq = xq; a.xk = xk; a.xv = xv; a.gq = gq; a.gk = gk; a.norm = norm; a.eps = eps;
    a.pos = pos; a.freqs = freqs; a.mag = mag; a.rot = rot; a.interleaved = interleaved != 0;
    a.q = q; a.seq = seq; a.table = table; a.k_pages = k_pages; a.v_pages = v_pages;
    a.R = R; a.P = P; a.page_size = page_size; a.num_pages = num_pages;
    a.T = T; a.Hq = Hq; a.Hk = Hk; a.d = d; a.dtype = dtype; a.sxq = xq_stride; a.sxk = xk_stride; a.sxv = xv_stride;
    return done(gdr2::launch_attn_prologue_cache(a, (cudaStream_t)stream));
}

size_t gdr2_attn_decode_workspace_bytes(int N, int Hq, int Hk, int d, int P, int page_size, int window, int dtype) {
    gdr2::AttnDecodeArgs a{};
    a.N = N; a.Hq = Hq; a.Hk = Hk; a.d = d; a.P = P; a.page_size = page_size; a.num_pages = 1; a.window = window;
    a.dtype = dtype;
    return check_decode(a, 1) == GDR2_OK ? gdr2::attn_decode_workspace_bytes(a) : 0;  // R: any, slots may share sequences
}

int gdr2_attn_decode(const void *q, const void *k_pages, const void *v_pages, const int *table, const int *lens,
                     const int *seq, float scale, int window, void *o, float *lse, int N, int Hq, int Hk, int d, int R,
                     int P, int page_size, int num_pages, int dtype, void *workspace, size_t workspace_bytes,
                     void *stream) {
    gdr2::AttnDecodeArgs a{};
    a.q = q; a.k_pages = k_pages; a.v_pages = v_pages; a.table = table; a.lens = lens; a.seq = seq;
    a.scale = scale; a.window = window; a.o = o; a.lse = lse;
    a.N = N; a.Hq = Hq; a.Hk = Hk; a.d = d; a.R = R; a.P = P; a.page_size = page_size; a.num_pages = num_pages;
    a.dtype = dtype; a.workspace = workspace;
    const int st = check_decode(a, R);
    if (st != GDR2_OK) return st;
    if (seq == nullptr && N > R) return GDR2_ERR_INVALID_ARG;
    if (!ok_ptr(q) || !ok_ptr(k_pages) || !ok_ptr(v_pages) || !ok_num(table) || !ok_num(lens) || !opt_num(seq) ||
        !ok_ptr(o) || !opt_num(lse))
        return GDR2_ERR_INVALID_ARG;
    const size_t need = gdr2::attn_decode_workspace_bytes(a);
    if (need > 0 && (!ok_ptr(workspace) || workspace_bytes < need)) return GDR2_ERR_WORKSPACE;
    return done(gdr2::launch_attn_decode(a, (cudaStream_t)stream));
}

size_t gdr2_kv_workspace_bytes(int R, int P, int num_pages) {
    return check_pages(R, P, 1, num_pages) == GDR2_OK ? gdr2::kv_workspace_bytes(R, P, num_pages) : 0;
}

int gdr2_kv_reserve(const int *table, const int *lens, const int *want, const int *ref, int *table_out, int *ref_out,
                    int *missing, int R, int P, int page_size, int num_pages, int window, void *workspace,
                    size_t workspace_bytes, void *stream) {
    const int st = check_pages(R, P, page_size, num_pages);
    if (st != GDR2_OK) return st;
    if (window < 0 || !ok_num(table) || !ok_num(lens) || !ok_num(want) || !ok_num(ref) || !ok_num(table_out) ||
        !ok_num(ref_out) || !ok_num(missing))
        return GDR2_ERR_INVALID_ARG;
    if (!ok_ptr(workspace) || workspace_bytes < gdr2::kv_workspace_bytes(R, P, num_pages)) return GDR2_ERR_WORKSPACE;
    gdr2::KvPagesArgs a{};
    a.table = table; a.lens = lens; a.want = want; a.ref = ref;
    a.table_out = table_out; a.ref_out = ref_out; a.count_out = missing;
    a.R = R; a.P = P; a.page_size = page_size; a.num_pages = num_pages; a.window = window; a.workspace = workspace;
    return done(gdr2::launch_kv_reserve(a, (cudaStream_t)stream));
}

int gdr2_kv_fork(const int *table, const int *lens, const int *ref, const int *parent, int *table_out, int *lens_out,
                 int *ref_out, int *missing, void *k_pages, void *v_pages, int R, int P, int Hk, int page_size, int d,
                 int num_pages, int dtype, void *workspace, size_t workspace_bytes, void *stream) {
    int st = check_heads(Hk, Hk, d, dtype);
    if (st == GDR2_OK) st = check_pages(R, P, page_size, num_pages);
    if (st == GDR2_OK && !copies_fit(Hk, page_size, d, num_pages, dtype)) st = GDR2_ERR_UNSUPPORTED;
    if (st != GDR2_OK) return st;
    if (!ok_num(table) || !ok_num(lens) || !ok_num(ref) || !ok_num(parent) || !ok_num(table_out) || !ok_num(lens_out) ||
        !ok_num(ref_out) || !ok_num(missing) || !ok_ptr(k_pages) || !ok_ptr(v_pages) || table_out == table ||
        lens_out == lens)
        return GDR2_ERR_INVALID_ARG;
    if (!ok_ptr(workspace) || workspace_bytes < gdr2::kv_workspace_bytes(R, P, num_pages)) return GDR2_ERR_WORKSPACE;
    gdr2::KvPagesArgs a{};
    a.table = table; a.lens = lens; a.ref = ref; a.parent = parent;
    a.table_out = table_out; a.lens_out = lens_out; a.ref_out = ref_out; a.count_out = missing;
    a.k_pages = k_pages; a.v_pages = v_pages;
    a.R = R; a.P = P; a.page_size = page_size; a.num_pages = num_pages; a.Hk = Hk; a.d = d; a.dtype = dtype;
    a.workspace = workspace;
    return done(gdr2::launch_kv_fork(a, (cudaStream_t)stream));
}

int gdr2_kv_compact(const int *table, const int *ref, int *table_out, int *ref_out, int *live, void *k_pages,
                    void *v_pages, int R, int P, int Hk, int page_size, int d, int num_pages, int dtype,
                    void *workspace, size_t workspace_bytes, void *stream) {
    int st = check_heads(Hk, Hk, d, dtype);
    if (st == GDR2_OK) st = check_pages(R, P, page_size, num_pages);
    if (st == GDR2_OK && !copies_fit(Hk, page_size, d, num_pages, dtype)) st = GDR2_ERR_UNSUPPORTED;
    if (st != GDR2_OK) return st;
    if (!ok_num(table) || !ok_num(ref) || !ok_num(table_out) || !ok_num(ref_out) || !ok_num(live) || !ok_ptr(k_pages) ||
        !ok_ptr(v_pages))
        return GDR2_ERR_INVALID_ARG;
    if (!ok_ptr(workspace) || workspace_bytes < gdr2::kv_workspace_bytes(R, P, num_pages)) return GDR2_ERR_WORKSPACE;
    gdr2::KvPagesArgs a{};
    a.table = table; a.ref = ref; a.table_out = table_out; a.ref_out = ref_out; a.count_out = live;
    a.k_pages = k_pages; a.v_pages = v_pages;
    a.R = R; a.P = P; a.page_size = page_size; a.num_pages = num_pages; a.Hk = Hk; a.d = d; a.dtype = dtype;
    a.workspace = workspace;
    return done(gdr2::launch_kv_compact(a, (cudaStream_t)stream));
}

int gdr2_attn_call(int call, const void *args, size_t bytes) {
    switch (call) {
    case GDR2_CALL_ATTN_PROLOGUE_FWD:
        if (const auto *r = record<gdr2_attn_prologue_fwd_args>(args, bytes))
            return gdr2_attn_prologue_fwd(
                r->xq, r->xk, r->gq, r->gk, r->norm, r->eps, r->pos, r->freqs, r->mag, r->rot, r->interleaved,
                r->q, r->k, r->T, r->Hq, r->Hk, r->d, r->dtype, r->xq_stride, r->xk_stride, r->stream);
        break;
    case GDR2_CALL_ATTN_PROLOGUE_BWD:
        if (const auto *r = record<gdr2_attn_prologue_bwd_args>(args, bytes))
            return gdr2_attn_prologue_bwd(
                r->xq, r->xk, r->gq, r->gk, r->norm, r->eps, r->pos, r->freqs, r->mag, r->rot, r->interleaved,
                r->dq, r->dk, r->dxq, r->dxk, r->dgq, r->dgk, r->T, r->Hq, r->Hk, r->d, r->dtype, r->xq_stride,
                r->xk_stride, r->dxq_stride, r->dxk_stride, r->workspace, r->workspace_bytes, r->stream);
        break;
    case GDR2_CALL_ATTN_PROLOGUE_CACHE:
        if (const auto *r = record<gdr2_attn_prologue_cache_args>(args, bytes))
            return gdr2_attn_prologue_cache(
                r->xq, r->xk, r->xv, r->gq, r->gk, r->norm, r->eps, r->seq, r->pos, r->freqs, r->mag, r->rot,
                r->interleaved, r->q, r->k_pages, r->v_pages, r->table, r->T, r->Hq, r->Hk, r->d, r->R, r->P,
                r->page_size, r->num_pages, r->dtype, r->xq_stride, r->xk_stride, r->xv_stride, r->stream);
        break;
    case GDR2_CALL_ATTN_DECODE:
        if (const auto *r = record<gdr2_attn_decode_args>(args, bytes))
            return gdr2_attn_decode(
                r->q, r->k_pages, r->v_pages, r->table, r->lens, r->seq, r->scale, r->window, r->o, r->lse, r->N,
                r->Hq, r->Hk, r->d, r->R, r->P, r->page_size, r->num_pages, r->dtype, r->workspace,
                r->workspace_bytes, r->stream);
        break;
    case GDR2_CALL_KV_RESERVE:
        if (const auto *r = record<gdr2_kv_reserve_args>(args, bytes))
            return gdr2_kv_reserve(
                r->table, r->lens, r->want, r->ref, r->table_out, r->ref_out, r->missing, r->R, r->P, r->page_size,
                r->num_pages, r->window, r->workspace, r->workspace_bytes, r->stream);
        break;
    case GDR2_CALL_KV_FORK:
        if (const auto *r = record<gdr2_kv_fork_args>(args, bytes))
            return gdr2_kv_fork(
                r->table, r->lens, r->ref, r->parent, r->table_out, r->lens_out, r->ref_out, r->missing,
                r->k_pages, r->v_pages, r->R, r->P, r->Hk, r->page_size, r->d, r->num_pages, r->dtype,
                r->workspace, r->workspace_bytes, r->stream);
        break;
    case GDR2_CALL_KV_COMPACT:
        if (const auto *r = record<gdr2_kv_compact_args>(args, bytes))
            return gdr2_kv_compact(
                r->table, r->ref, r->table_out, r->ref_out, r->live, r->k_pages, r->v_pages, r->R, r->P, r->Hk,
                r->page_size, r->d, r->num_pages, r->dtype, r->workspace, r->workspace_bytes, r->stream);
        break;
    }
    return GDR2_ERR_INVALID_ARG;
}

}  // extern "C"
