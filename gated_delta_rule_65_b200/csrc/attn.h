// attn.h -- internal launcher interface of the attention half of the hybrid cell: the query / key prologue, the
// attention of one new token over the paged key-value cache, and the cache's page bookkeeping.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

namespace gdr2 {

// SMs the persistent grids below are sized for. A constant, so that a workspace query and the launch agree.
constexpr int kAttnSms = 148;

// Division of numbers below 2^31 by d >= 1: x d' >> shift with d' = floor(2^(31 + s) / d) + 1, 2^s >= d, is exact.
struct Divisor {
    uint32_t magic, shift;
    Divisor() : magic(0), shift(0) {}
    explicit Divisor(uint32_t d) {
        uint32_t s = 0;
        while ((1ull << s) < d) ++s;
        shift = 31 + s;
        magic = (uint32_t)((1ull << shift) / d + 1);
    }
#ifdef __CUDACC__
    __device__ __forceinline__ uint32_t divide(uint32_t x) const { return (uint32_t)((uint64_t)x * magic >> shift); }
#endif
};

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
    Divisor by_page;                      // page_size, set by the launch
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
size_t attn_decode_workspace_bytes(const AttnDecodeArgs &a);  // of the sizes in it; 0 where nothing is cut
cudaError_t launch_attn_decode(const AttnDecodeArgs &a, cudaStream_t st);

struct KvPagesArgs {
    const int *table, *lens, *want, *ref, *parent;
    int *table_out, *lens_out, *ref_out, *count_out;  // count_out: pages missing, or pages live
    void *k_pages, *v_pages;
    int R, P, num_pages, page_size, window, Hk, d, dtype;
    void *workspace;
};
size_t kv_workspace_bytes(int R, int P, int num_pages);
cudaError_t launch_kv_reserve(const KvPagesArgs &a, cudaStream_t st);
cudaError_t launch_kv_fork(const KvPagesArgs &a, cudaStream_t st);
cudaError_t launch_kv_compact(const KvPagesArgs &a, cudaStream_t st);

// As in kernels.h; only failed index checks of the debug build set a bit here.
int status_take_attn_prologue();
int status_take_attn_decode();
int status_take_kv_pages();

// The launch of every kernel here: its blocks may become resident while the kernel before it on the stream still runs.
// So each kernel begins with follow(), which lets the next one do the same and waits until everything before it on
// the stream has finished and can be read; nothing of global memory is touched before. What a kernel before may have
// written (tables, lengths, workspaces) is read by ordinary loads, which that wait orders, not by __ldg, which asks that
// nobody writes the data while the kernel is resident. (Two launches of a pair are 1.3 us apart this way, measured on an
// empty second kernel. __ldcg for the table costs an attention of one short sequence 0.2 us of 6.8 and 16 packed
// prompts 0.8 of 47.3: a page's tokens look their entry up one by one, and find it in L1.) Shared memory above 48 KB is
// allowed to the kernel on its first launch on a device; a launch refused later (the device was reset since) allows it
// again.
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 0 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
    if (smem <= 48 * 1024 || e != cudaErrorInvalidValue) return e;
    (void)cudaGetLastError();
    const cudaError_t f = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    return f != cudaSuccess ? f : cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// A kernel's allowance of shared memory, asked for once on each device.
struct Allowed {
    std::atomic<unsigned long long> devices{0};
    template <typename... P> cudaError_t operator()(void (*kernel)(P...), size_t smem) {
        int dev = 0;
        const cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const unsigned long long bit = 1ull << (dev & 63);
        if (dev < 64 && (devices.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
        const cudaError_t f = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (f == cudaSuccess && dev < 64) devices.fetch_or(bit, std::memory_order_relaxed);
        return f;
    }
};

#ifdef __CUDACC__
__device__ __forceinline__ void follow() {
    cudaTriggerProgrammaticLaunchCompletion();
    cudaGridDependencySynchronize();
}
#endif

}  // namespace gdr2
