// attn.h -- internal launcher interface of the attention half of the hybrid cell: the query / key prologue, the
// attention of one new token over the paged key-value cache, and the cache's page bookkeeping.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace gdr2 {

// SMs the persistent grids below are sized for. A constant, so that a workspace query and the launch agree.
constexpr int kAttnSms = 148;

struct AttnPrologueArgs {
    const void *xq, *xk, *xv;             // [T, H, d], token strides sxq, sxk, sxv; xv only for the cache form
    const float *gq, *gk;                 // [d] or null
    int norm;                             // 0: no norm, 1: RMS norm over the head
    float eps;
    const int *pos;                       // [T]; null when rot = 0
    const double *freqs;                  // [rot / 2]
    float mag;
    int rot, interleaved;
    void *q, *k;                          // forward outputs, contiguous
    const void *dq, *dk;                  // backward inputs, contiguous
    void *dxq, *dxk;                      // backward outputs, token strides sdxq, sdxk
    float *dgq, *dgk;                     // [d] or null
    const int *seq, *table;               // cache form
    void *k_pages, *v_pages;              // [num_pages, Hk, page_size, d]
    int R, P, page_size, num_pages;
    int T, Hq, Hk, d, dtype;
    long long sxq, sxk, sxv, sdxq, sdxk;  // elements
    void *workspace;
};
size_t attn_prologue_workspace_bytes(int d);
cudaError_t launch_attn_prologue_fwd(const AttnPrologueArgs &a, cudaStream_t st);
cudaError_t launch_attn_prologue_cache(const AttnPrologueArgs &a, cudaStream_t st);
cudaError_t launch_attn_prologue_bwd(const AttnPrologueArgs &a, cudaStream_t st);

struct AttnDecodeArgs {
    const void *q, *k_pages, *v_pages;
    const int *table, *lens, *seq;        // seq may be null
    float scale;
    int window;                           // 0: the whole sequence
    void *o;
    float *lse;                           // may be null
    int N, Hq, Hk, d, R, P, page_size, num_pages, dtype;
    void *workspace;
};
size_t attn_decode_workspace_bytes(int d);
cudaError_t launch_attn_decode(const AttnDecodeArgs &a, cudaStream_t st);

struct KvPagesArgs {
    const int *table, *lens, *want, *ref, *parent;
    int *table_out, *lens_out, *ref_out, *count_out;  // count_out: pages missing, or pages live
    void *k_pages, *v_pages;
    int R, P, num_pages, page_size, window, Hk, d, dtype;
    void *workspace;
};
size_t kv_workspace_bytes(int R, int num_pages);
cudaError_t launch_kv_reserve(const KvPagesArgs &a, cudaStream_t st);
cudaError_t launch_kv_fork(const KvPagesArgs &a, cudaStream_t st);
cudaError_t launch_kv_compact(const KvPagesArgs &a, cudaStream_t st);

// A launch whose blocks may become resident while the kernel before it on the stream still runs; the kernel
// waits for that kernel's results with cudaGridDependencySynchronize() before it reads or writes anything.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace gdr2
