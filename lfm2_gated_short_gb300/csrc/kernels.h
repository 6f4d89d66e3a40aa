// kernels.h -- internal launchers behind the C ABI (api.cu). Arguments are
// already validated by the caller; these only pick a template instance and
// enqueue on the stream. All return the cudaError_t of the launch.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace sc {

// Prefill: rows_per_thread 0 selects the TMA-streamed kernel (one CTA per SM),
// 4/8/16/32 the register-tiled kernel with that many rows per thread.
// bias (here and below) is the optional per-channel conv bias, NULL for none.
cudaError_t launch_prefill(int dtype, int H, int K, const void *bcx, int64_t T, const void *w,
                           const void *bias, const int32_t *cu_seqlens, int N,
                           const int32_t *slot_ids, void *pool, int n_slots, void *y,
                           int rows_per_thread, int sm_count, cudaStream_t stream);

cudaError_t launch_decode(int dtype, int H, int K, const void *bcx, int N, const void *w,
                          const void *bias, const int32_t *slot_ids, void *pool, int n_slots,
                          void *y, cudaStream_t stream);

cudaError_t launch_verify(int dtype, int H, int K, const void *bcx, int N, int D,
                          const void *w, const void *bias, const int32_t *slot_ids,
                          const void *pool, int n_slots, void *win, void *y,
                          cudaStream_t stream);

// L layers at once: win [L, N, D, H, K], pool [L, n_slots, H, K].
cudaError_t launch_rollback(int dtype, int H, int K, int L, int N, int D, const void *win,
                            const int32_t *accepted, const int32_t *slot_ids, void *pool,
                            int n_slots, cudaStream_t stream);

// Bytes of fp32 partials the backward writes: one H*K dW block per row range,
// plus H dbias entries per row range when dbias is wanted.
size_t backward_partial_bytes(int H, int K, int64_t T, bool with_dbias);
// The caller-workspace size: room for both.
size_t backward_workspace_bytes(int H, int K, int64_t T);

// dbias (fp32 [H]) is written when non-NULL.
cudaError_t launch_backward(int dtype, int H, int K, const void *bcx, int64_t T,
                            const void *w, const void *bias, const void *dy, void *dbcx,
                            float *dw, float *dbias, void *workspace, cudaStream_t stream);

// Packed varlen backward with initial states (NULL: zeros), an optional
// final-state gradient (NULL: zeros) and an optional initial-state gradient
// output (NULL: not written). Same workspace size as launch_backward.
cudaError_t launch_backward_varlen(int dtype, int H, int K, const void *bcx, int64_t T,
                                   const void *w, const void *bias, const int32_t *cu_seqlens,
                                   int N, const void *init, const void *dy,
                                   const float *d_final, void *dbcx, float *dw, float *dbias,
                                   float *d_init, void *workspace, cudaStream_t stream);

// The bias-free backward kernels with their dW partials in the library's
// fixed device scratch (kNoAllocScratchBytes) instead of a caller workspace.
// The caller checks backward_partial_bytes(H, K, T, false) <=
// kNoAllocScratchBytes first.
constexpr size_t kNoAllocScratchBytes = (size_t)8 << 20;
cudaError_t launch_backward_noalloc(int dtype, int H, int K, const void *bcx, int64_t T,
                                    const void *w, const void *dy, void *dbcx, float *dw,
                                    cudaStream_t stream);

// The layer's projections (bf16): in_proj fused with the ShortConv, writing y
// and, through k_commit_states, the slots' new states (workspace: the last K
// values of u per sequence, in_proj_workspace_bytes); out_proj a plain GEMM.
size_t in_proj_workspace_bytes(int H, int K, int N);
cudaError_t launch_in_proj_prefill(int D, int H, int K, const void *hidden, int64_t T,
                                   const void *w_in, const void *w, const void *bias,
                                   const int32_t *cu_seqlens, int N, const int32_t *slot_ids,
                                   void *pool, int n_slots, void *y, void *workspace,
                                   int sm_count, cudaStream_t stream);
cudaError_t launch_out_proj(int H, int D, const void *y, int64_t T, const void *w_out, void *out,
                            int sm_count, cudaStream_t stream);
// in_proj fused with the decode of N one-token sequences (bf16): y [N, H] and
// the slots' new states, in one launch.
cudaError_t launch_in_proj_decode(int D, int H, int K, const void *hidden, int N,
                                  const void *w_in, const void *w, const void *bias,
                                  const int32_t *slot_ids, void *pool, int n_slots, void *y,
                                  int sm_count, cudaStream_t stream);
cudaError_t take_error_proj(cudaStream_t stream, unsigned int *sum);

// Enqueue: take (read and clear) a translation unit's error word and OR it into
// *sum (device memory). Likewise take_error_proj, _slots, _pages, _draft, _attention.
cudaError_t take_error_backward(cudaStream_t stream, unsigned int *sum);

// Slot pool: claim n_claim free slots (lowest first, all-or-nothing) and
// zero their states when pool != NULL; release slots; copy states.
cudaError_t launch_slots_claim(uint32_t *in_use, int n_slots, int n_claim, int32_t *out,
                               void *pool, int64_t state_bytes, cudaStream_t stream);
cudaError_t launch_slots_release(uint32_t *in_use, int n_slots, const int32_t *slots, int n,
                                 cudaStream_t stream);
cudaError_t launch_pool_copy(const int32_t *src, const int32_t *dst, int n, int64_t state_bytes,
                             void *pool, int n_slots, cudaStream_t stream);
cudaError_t take_error_slots(cudaStream_t stream, unsigned int *sum);
// A one-thread kernel whose bounded wait must run out and set SC_DEV_TIMEOUT.
cudaError_t launch_wait_limit_check(cudaStream_t stream);

// The paged cache (pages.cu). `pools`: L stacked layers of k and v pages of
// page_size * token_bytes bytes each.
struct PageTable {
    int32_t *refs;   // [n_pages] table entries that name the page (0: free)
    int32_t *table;  // [n_slots, max_pages]
    int32_t *lens;   // [n_slots]
    int n_pages, n_slots, max_pages, page_size;
};
struct PagePools {
    void *k, *v;
    int L;
    int64_t token_bytes;
    float *k_scales, *v_scales;  // of an 8-bit cache: page_scales a page and layer
    int page_scales;             // 0: none
};
size_t pages_workspace_bytes(int n_pages, int n);
cudaError_t launch_pages_resize(const PageTable &pt, const int32_t *slots, const int32_t *new_lens,
                                int n, const PagePools &pools, void *workspace, int sm_count,
                                cudaStream_t stream);
cudaError_t launch_pages_fork(const PageTable &pt, const int32_t *src, const int32_t *dst, int n,
                              const PagePools &pools, void *workspace, int sm_count,
                              cudaStream_t stream);
cudaError_t launch_pages_compact(const PageTable &pt, const PagePools &pools, int32_t *n_used,
                                 void *workspace, int sm_count, cudaStream_t stream);
cudaError_t launch_pages_append(const PageTable &pt, const void *k, int64_t k_stride,
                                const void *v, int64_t v_stride, const int32_t *slots, int N,
                                int D, const PagePools &pools, cudaStream_t stream);
cudaError_t take_error_pages(cudaStream_t stream, unsigned int *sum);

// The 8-bit cache (cache8.cu): pools of e4m3 codes, [n_pages, page_size, Hkv, Dh], and scales,
// [n_pages, page_size / 2^block_log2, Hkv].
struct Cache8 {
    void *k, *v;
    float *k_scales, *v_scales;
    int Hkv, Dh, block_log2;
};
cudaError_t launch_append8(int dtype, const PageTable &pt, const void *k, int64_t k_stride,
                           const void *v, int64_t v_stride, const int32_t *slots, int N, int D,
                           const Cache8 &c, cudaStream_t stream);
cudaError_t launch_read8(int dtype, const PageTable &pt, const int32_t *slots, const int32_t *cu,
                         const int32_t *starts, int N, int64_t rows, const Cache8 &c, void *k,
                         void *v, int sm_count, cudaStream_t stream);
cudaError_t take_error_cache8(cudaStream_t stream, unsigned int *sum);

// Rotary positions (rope.cu). Strides in elements; positions, or D newest tokens of slots.
struct RopeArgs {
    const void *q, *k;
    void *q_out, *k_out;
    int64_t q_stride, k_stride, q_out_stride, k_out_stride;
    const double *freqs;
    const int32_t *positions, *lens, *slots;
    int64_t T;
    int Hq, Hkv, Dh, R, D, n_slots;
    float amplitude;
    int half_layout, inverse, copy;  // copy: the values behind R, from in to out
};
cudaError_t launch_rope(int dtype, const RopeArgs &a, int sm_count, cudaStream_t stream);
cudaError_t take_error_rope(cudaStream_t stream, unsigned int *sum);

// Draft acceptance (draft.cu). draft NULL: the drafts were certain.
cudaError_t launch_draft_accept(int dtype, int V, int N, int D, const void *target,
                                int64_t target_stride, const void *draft, int64_t draft_stride,
                                const int32_t *tokens, const int32_t *n_drafts,
                                const float *uniforms, int32_t *accepted, int32_t *out_tokens,
                                int sm_count, cudaStream_t stream);
cudaError_t take_error_draft(cudaStream_t stream, unsigned int *sum);

// Attention over the paged cache (attention.cu), bf16, or e4m3 codes with scales of 2^block_log2
// tokens and a head (NULL: bf16).
struct AttnShape {
    int Hq, Hkv, Dh, N, D, shared_pages;
};
struct Scales8 {
    const float *k, *v;
    int block_log2;
};
size_t attention_workspace_bytes(const AttnShape &s);
size_t attention8_workspace_bytes(const AttnShape &s, int page_size);
cudaError_t launch_prefix_attention(const AttnShape &s, const void *q, int64_t q_stride,
                                    const void *k_pages, const void *v_pages,
                                    const Scales8 *scales, const PageTable &pt,
                                    const int32_t *slots, float scale, void *out, void *workspace,
                                    int sm_count, cudaStream_t stream);
cudaError_t take_error_attention(cudaStream_t stream, unsigned int *sum);

// Read and clear the device error word of the current device (synchronous
// with respect to `stream`).
cudaError_t read_and_clear_error(cudaStream_t stream, unsigned int *code);

// The bounds-checked build (-DSC_BOUNDS_CHECK): a buffer a call may touch,
// [base, base + bytes), writable or read only. The entry points install the
// call's buffers in the table of each translation unit they launch into.
struct BoundsRegion {
    uint64_t base;
    uint64_t bytes;
    uint32_t writable;
    uint32_t pad;
};
constexpr int kMaxBoundsRegions = 16;
#ifdef SC_BOUNDS_CHECK
enum BoundsUnit {
    kUnitForward = 0,
    kUnitBackward = 1,
    kUnitProj = 2,
    kUnitSlots = 3,
    kUnitPages = 4,
    kUnitDraft = 5,
    kUnitAttention = 6,
    kUnitCache8 = 7,
    kUnitRope = 8
};
cudaError_t bounds_install(int unit, const BoundsRegion *r, int n, cudaStream_t stream);
// The first address any unit refused since the last call (0 when none), cleared.
cudaError_t bounds_take_first_bad(cudaStream_t stream, unsigned long long *addr);
cudaError_t bounds_install_backward(const BoundsRegion *r, int n, cudaStream_t stream);
cudaError_t bounds_install_proj(const BoundsRegion *r, int n, cudaStream_t stream);
cudaError_t bounds_install_slots(const BoundsRegion *r, int n, cudaStream_t stream);
cudaError_t bounds_install_pages(const BoundsRegion *r, int n, cudaStream_t stream);
cudaError_t bounds_install_draft(const BoundsRegion *r, int n, cudaStream_t stream);
void bounds_starve_next_attention();
cudaError_t bounds_install_attention(const BoundsRegion *r, int n, cudaStream_t stream);
cudaError_t bounds_install_cache8(const BoundsRegion *r, int n, cudaStream_t stream);
cudaError_t bounds_install_rope(const BoundsRegion *r, int n, cudaStream_t stream);
cudaError_t bounds_take_backward(cudaStream_t stream, unsigned long long *addr);
cudaError_t bounds_take_proj(cudaStream_t stream, unsigned long long *addr);
cudaError_t bounds_take_slots(cudaStream_t stream, unsigned long long *addr);
cudaError_t bounds_take_pages(cudaStream_t stream, unsigned long long *addr);
cudaError_t bounds_take_draft(cudaStream_t stream, unsigned long long *addr);
cudaError_t bounds_take_attention(cudaStream_t stream, unsigned long long *addr);
cudaError_t bounds_take_cache8(cudaStream_t stream, unsigned long long *addr);
cudaError_t bounds_take_rope(cudaStream_t stream, unsigned long long *addr);
#endif

}  // namespace sc
