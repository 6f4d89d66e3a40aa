// pages.cu -- the paged key/value cache: resize, fork, compact, append.
//
// A sequence (a slot, the same id as its conv state's) holds its tokens on
// pages of page_size tokens named by its row of the page table; refs counts
// the table entries that name a page, so branches of one prompt share its
// full pages. A partly filled last page is never shared: fork and a
// truncation into a shared page copy it, so an append writes no page that
// another sequence reads.
//
// Claims take the lowest free pages in listed order, so every call's result
// is a function of its inputs alone. The metadata of a call (a few table
// rows and the refs array, read once) is worked out by one CTA, which leaves
// a list of page copies; a second kernel over the whole GPU copies the data
// of every layer.
#include "common.cuh"
#include "errors.cuh"
#include "kernels.h"
#include "launch.h"
#include "shortconv.h"
#include "tma.cuh"

namespace sc {

constexpr int kMetaThreads = 1024;
constexpr int kCopyThreads = 256;

// One page copy: the first `rows` tokens of page src to page dst.
struct PageCopy {
    int32_t src, dst, rows, pad;
};

// Workspace: the copy count, then the copies, then the claimed page ids.
struct PageWork {
    int32_t *n_copies;
    PageCopy *copies;
    int32_t *claimed;  // [n_pages]: the free pages taken, lowest first
    int32_t *offset;   // [n]: first claim of listed sequence i, or -1 - it with a copy
};

static __host__ __device__ PageWork page_work(void *ws, int n_pages, int n_copies) {
    PageWork w;
    w.n_copies = (int32_t *)ws;
    w.copies = (PageCopy *)((char *)ws + 16);
    w.claimed = (int32_t *)(w.copies + n_copies);
    w.offset = w.claimed + n_pages;
    return w;
}

// refs is changed by atomics, which act in L2: read it there.
__device__ __forceinline__ int ld_refs(const int32_t *p) {
    if (!SC_RD_OK(p, 4)) return 1;
    return __ldcg(p);
}
__device__ __forceinline__ void add_refs(const PageTable &pt, int id, int by) {
    if (SC_WR_OK(pt.refs + id, 4)) atomicAdd(pt.refs + id, by);
}
__device__ __forceinline__ bool page_ok(const PageTable &pt, int id) {
    return id >= 0 && id < pt.n_pages;
}
__device__ __forceinline__ int pages_of(const PageTable &pt, int len) {
    return (len + pt.page_size - 1) / pt.page_size;
}
__device__ __forceinline__ int32_t *table_row(const PageTable &pt, int slot) {
    return pt.table + (int64_t)slot * pt.max_pages;
}
// The length of a valid slot, or -1 (and an error bit).
__device__ __forceinline__ int slot_len(const PageTable &pt, int slot, bool report) {
    if (slot < 0 || slot >= pt.n_slots) {
        if (report) raise_error(SC_DEV_BAD_SLOT);
        return -1;
    }
    const int len = gld(pt.lens + slot);
    if (len < 0 || len > (int64_t)pt.max_pages * pt.page_size) {
        if (report) raise_error(SC_DEV_BAD_LENGTH);
        return -1;
    }
    return len;
}

// Exclusive sum of v over the CTA's threads; *total the whole sum.
__device__ __forceinline__ int block_scan(int v, int *total) {
    __shared__ int s_warp[kMetaThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(~0u, inc, o);
        if (lane >= o) inc += up;
    }
    __syncthreads();  // s_warp of a previous call
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        int w = s_warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(~0u, w, o);
            if (lane >= o) w += up;
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    *total = s_warp[kMetaThreads / 32 - 1];
    return inc - v + (warp > 0 ? s_warp[warp - 1] : 0);
}

// The `want` lowest free pages into claimed[]; false with fewer free.
__device__ bool claim_lowest(const PageTable &pt, int want, int32_t *claimed) {
    int found = 0;
    for (int p0 = 0; p0 < pt.n_pages && found < want; p0 += kMetaThreads) {
        const int p = p0 + threadIdx.x;
        const int is_free = p < pt.n_pages && ld_refs(pt.refs + p) <= 0;
        int here;
        const int rank = found + block_scan(is_free, &here);
        if (is_free && rank < want) gst(claimed + rank, p);
        found += here;
    }
    __syncthreads();  // claimed[] is read by other threads
    return found >= want;
}

// Release (sign -1) or take back (+1) table entries [from, to) of a slot, one warp.
__device__ __forceinline__ void count_entries(const PageTable &pt, int slot, int from, int to,
                                              int sign) {
    for (int e = from + (int)(threadIdx.x & 31); e < to; e += 32) {
        const int id = gld(table_row(pt, slot) + e);
        if (page_ok(pt, id))
            add_refs(pt, id, sign);
        else if (sign < 0)
            raise_error(SC_DEV_BAD_PAGE);
    }
}

__global__ void __launch_bounds__(kMetaThreads)
    k_pages_resize(PageTable pt, const int32_t *__restrict__ slots,
                   const int32_t *__restrict__ new_lens, int n, PageWork w) {
    __shared__ int s_copies;
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t cap = (int64_t)pt.max_pages * pt.page_size;
    if (tid == 0) s_copies = 0;
    // Old and new length of listed sequence i; false (reported once) when either is bad.
    auto lengths = [&](int i, int *slot, int *old, int *now, bool report) {
        *slot = gld(slots + i);
        *now = gld(new_lens + i);
        *old = slot_len(pt, *slot, report);
        if (*old >= 0 && (*now < 0 || *now > cap)) {
            if (report) raise_error(SC_DEV_BAD_LENGTH);
            return false;
        }
        return *old >= 0;
    };
    int slot, old, now;
    for (int i = warp; i < n; i += kMetaThreads / 32)  // released entries
        if (lengths(i, &slot, &old, &now, lane == 0))
            count_entries(pt, slot, pages_of(pt, now), pages_of(pt, old), -1);
    __syncthreads();
    int want = 0;
    for (int i0 = 0; i0 < n; i0 += kMetaThreads) {  // claims, in listed order
        const int i = i0 + tid;
        int claims = 0, copy = 0;
        if (i < n && lengths(i, &slot, &old, &now, false)) {
            const int need = pages_of(pt, now), have = pages_of(pt, old);
            if (now < old && now % pt.page_size != 0) {
                const int id = gld(table_row(pt, slot) + need - 1);
                copy = page_ok(pt, id) && ld_refs(pt.refs + id) > 1;
            }
            claims = copy + max(0, need - have);
        }
        int here;
        const int at = want + block_scan(claims, &here);
        if (i < n) gst(w.offset + i, copy ? -1 - at : at);
        want += here;
    }
    const bool enough = want <= pt.n_pages && claim_lowest(pt, want, w.claimed);
    __syncthreads();
    for (int i = warp; i < n; i += kMetaThreads / 32) {
        if (!lengths(i, &slot, &old, &now, false)) continue;
        const int need = pages_of(pt, now), have = pages_of(pt, old);
        if (!enough) {
            count_entries(pt, slot, need, have, 1);
            continue;
        }
        int32_t *row = table_row(pt, slot);
        for (int e = need + lane; e < have; e += 32) gst(row + e, -1);
        int at = gld(w.offset + i);
        if (at < 0) {
            at = -1 - at;
            if (lane == 0) {
                const int from = gld(row + need - 1), to = gld(w.claimed + at);
                add_refs(pt, from, -1);
                add_refs(pt, to, 1);
                gst(row + need - 1, to);
                gst(w.copies + atomicAdd(&s_copies, 1),
                    PageCopy{from, to, now % pt.page_size, 0});
            }
            ++at;
        }
        for (int e = have + lane; e < need; e += 32) {
            const int id = gld(w.claimed + at + e - have);
            add_refs(pt, id, 1);
            gst(row + e, id);
        }
        if (lane == 0) gst(pt.lens + slot, now);
    }
    __syncthreads();
    if (tid == 0) {
        if (!enough) raise_error(SC_DEV_NO_PAGE);
        gst(w.n_copies, enough ? s_copies : 0);
    }
}

__global__ void __launch_bounds__(kMetaThreads)
    k_pages_fork(PageTable pt, const int32_t *__restrict__ src, const int32_t *__restrict__ dst,
                 int n, PageWork w) {
    __shared__ int s_copies;
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) s_copies = 0;
    auto pair = [&](int i, int *s, int *d, int *ls, int *ld, bool report) {
        *s = gld(src + i);
        *d = gld(dst + i);
        *ls = slot_len(pt, *s, report);
        *ld = slot_len(pt, *d, report);
        if (*s == *d && *ls >= 0) {
            if (report) raise_error(SC_DEV_BAD_SLOT);
            return false;
        }
        return *ls >= 0 && *ld >= 0;
    };
    int s, d, ls, ld;
    for (int i = warp; i < n; i += kMetaThreads / 32)  // the destinations' old pages
        if (pair(i, &s, &d, &ls, &ld, lane == 0)) count_entries(pt, d, 0, pages_of(pt, ld), -1);
    __syncthreads();
    int want = 0;
    for (int i0 = 0; i0 < n; i0 += kMetaThreads) {
        const int i = i0 + tid;
        const int claims =
            i < n && pair(i, &s, &d, &ls, &ld, false) && ls % pt.page_size != 0 ? 1 : 0;
        int here;
        const int at = want + block_scan(claims, &here);
        if (i < n) gst(w.offset + i, at);
        want += here;
    }
    const bool enough = want <= pt.n_pages && claim_lowest(pt, want, w.claimed);
    __syncthreads();
    for (int i = warp; i < n; i += kMetaThreads / 32) {
        if (!pair(i, &s, &d, &ls, &ld, false)) continue;
        if (!enough) {
            count_entries(pt, d, 0, pages_of(pt, ld), 1);
            continue;
        }
        const int full = ls / pt.page_size, rows = ls % pt.page_size;
        const int32_t *from = table_row(pt, s);
        int32_t *to = table_row(pt, d);
        for (int e = lane; e < pt.max_pages; e += 32) {
            int id = -1;
            if (e < full) {
                id = gld(from + e);
                if (page_ok(pt, id))
                    add_refs(pt, id, 1);
                else
                    raise_error(SC_DEV_BAD_PAGE);
            } else if (e == full && rows) {
                const int old = gld(from + e);
                id = gld(w.claimed + gld(w.offset + i));
                add_refs(pt, id, 1);
                if (page_ok(pt, old))
                    gst(w.copies + atomicAdd(&s_copies, 1), PageCopy{old, id, rows, 0});
                else
                    raise_error(SC_DEV_BAD_PAGE);
            }
            gst(to + e, id);
        }
        if (lane == 0) gst(pt.lens + d, ls);
    }
    __syncthreads();
    if (tid == 0) {
        if (!enough) raise_error(SC_DEV_NO_PAGE);
        gst(w.n_copies, enough ? s_copies : 0);
    }
}

// U = used pages; the i-th used page >= U moves to the i-th free page < U.
// claimed[p] becomes the new id of moved page p.
__global__ void __launch_bounds__(kMetaThreads)
    k_pages_compact_plan(PageTable pt, PageWork w, int32_t *__restrict__ n_used) {
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    int used = 0, here;
    for (int p0 = 0; p0 < pt.n_pages; p0 += kMetaThreads) {
        const int p = p0 + tid;
        block_scan(p < pt.n_pages && ld_refs(pt.refs + p) > 0, &here);
        used += here;
    }
    int holes = 0, moved = 0;
    for (int p0 = 0; p0 < pt.n_pages; p0 += kMetaThreads) {
        const int p = p0 + tid;
        const bool in = p < pt.n_pages;
        const bool busy = in && ld_refs(pt.refs + p) > 0;
        const int hole = in && p < used && !busy, move = busy && p >= used;
        const int rh = holes + block_scan(hole, &here);
        holes += here;
        const int rm = moved + block_scan(move, &here);
        moved += here;
        if (hole) gst(&w.copies[rh].dst, p);
        if (move) gst(&w.copies[rm].src, p);
        if (in && p >= used && !busy) gst(w.claimed + p, -1);  // a table may not name it
    }
    __syncthreads();
    for (int i = tid; i < moved; i += kMetaThreads) {
        const int from = gld(&w.copies[i].src);
        gst(&w.copies[i].rows, pt.page_size);
        gst(w.claimed + from, gld(&w.copies[i].dst));
    }
    if (tid == 0) {
        gst(w.n_copies, moved);
        gst(n_used, used);
    }
}

__device__ __forceinline__ void copy_pages(const PageWork &w, const PageTable &pt,
                                           const PagePools &pools) {
    const int n = gld(w.n_copies);
    const int64_t page_bytes = pt.page_size * pools.token_bytes;
    for (int64_t u = blockIdx.x; u < (int64_t)n * pools.L * 2; u += gridDim.x) {
        const PageCopy c = gld(w.copies + u / (2 * pools.L));
        const int rest = (int)(u % (2 * pools.L));
        char *base = (char *)(rest & 1 ? pools.v : pools.k) +
                     (int64_t)(rest >> 1) * pt.n_pages * page_bytes;
        const uint4 *from = (const uint4 *)(base + c.src * page_bytes);
        uint4 *to = (uint4 *)(base + c.dst * page_bytes);
        const int q = (int)(c.rows * pools.token_bytes / 16);
        for (int i = threadIdx.x; i < q; i += blockDim.x) st_plain(to + i, ld_plain(from + i));
    }
}

__global__ void __launch_bounds__(kCopyThreads)
    k_pages_copy(PageTable pt, PagePools pools, PageWork w) {
    pdl_wait();
    pdl_launch_dependents();
    copy_pages(w, pt, pools);
}

// The moved pages' data, their refs, and every table entry that names one.
__global__ void __launch_bounds__(kCopyThreads)
    k_pages_compact_move(PageTable pt, PagePools pools, PageWork w, const int32_t *n_used) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t tid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t threads = (int64_t)gridDim.x * blockDim.x;
    const int n = gld(w.n_copies), used = gld(n_used);
    for (int64_t i = tid; i < n; i += threads) {
        const PageCopy c = gld(w.copies + i);
        gst(pt.refs + c.dst, gld(pt.refs + c.src));
        gst(pt.refs + c.src, 0);
    }
    const int lane = threadIdx.x & 31;
    for (int64_t s = tid >> 5; s < pt.n_slots; s += threads >> 5) {
        const int len = slot_len(pt, (int)s, lane == 0);
        int32_t *row = table_row(pt, (int)s);
        for (int e = lane; len > 0 && e < pages_of(pt, len); e += 32) {
            const int id = gld(row + e);
            const int to = !page_ok(pt, id) ? -1 : id >= used ? gld(w.claimed + id) : id;
            if (to < 0)
                raise_error(SC_DEV_BAD_PAGE);
            else if (to != id)
                gst(row + e, to);
        }
    }
    copy_pages(w, pt, pools);
}

// One warp copies a token's K (or V) row; the token's position is lens - D + j.
__global__ void __launch_bounds__(kCopyThreads)
    k_pages_append(PageTable pt, const char *__restrict__ k, int64_t k_stride,
                   const char *__restrict__ v, int64_t v_stride, const int32_t *__restrict__ slots,
                   int N, int D, PagePools pools) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t unit = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (unit >= (int64_t)N * D * 2) return;
    const int64_t token = unit >> 1;
    const int i = (int)(token / D), j = (int)(token % D);
    const int slot = gld(slots + i);
    const int len = slot_len(pt, slot, lane == 0);
    if (len < 0) return;
    const int pos = len - D + j;
    if (pos < 0) {
        if (lane == 0) raise_error(SC_DEV_BAD_LENGTH);
        return;
    }
    const int id = gld(table_row(pt, slot) + pos / pt.page_size);
    if (!page_ok(pt, id)) {
        if (lane == 0) raise_error(SC_DEV_BAD_PAGE);
        return;
    }
    const bool is_v = unit & 1;
    const uint4 *from = (const uint4 *)(is_v ? v + token * v_stride : k + token * k_stride);
    uint4 *to = (uint4 *)((char *)(is_v ? pools.v : pools.k) +
                          ((int64_t)id * pt.page_size + pos % pt.page_size) * pools.token_bytes);
    for (int64_t q = lane; q < pools.token_bytes / 16; q += 32) st_plain(to + q, ld_plain(from + q));
}

// ------------------------------------------------------------ host side

size_t pages_workspace_bytes(int n_pages, int n) {
    // n: listed sequences of a resize or fork (a copy each); 0: a compaction (up to half the pages)
    const size_t copies = n > 0 ? (size_t)n : (size_t)n_pages / 2 + 1;
    return 16 + copies * sizeof(PageCopy) + ((size_t)n_pages + n) * 4;
}

cudaError_t launch_pages_resize(const PageTable &pt, const int32_t *slots, const int32_t *new_lens,
                                int n, const PagePools &pools, void *workspace, int sm_count,
                                cudaStream_t stream) {
    const PageWork w = page_work(workspace, pt.n_pages, n);
    cudaError_t e = launch_pdl(k_pages_resize, dim3(1), dim3(kMetaThreads), 0, stream, pt, slots,
                               new_lens, n, w);
    if (e != cudaSuccess || pools.L == 0) return e;
    return launch_pdl(k_pages_copy, dim3((unsigned)(4 * sm_count)), dim3(kCopyThreads), 0, stream,
                      pt, pools, w);
}

cudaError_t launch_pages_fork(const PageTable &pt, const int32_t *src, const int32_t *dst, int n,
                              const PagePools &pools, void *workspace, int sm_count,
                              cudaStream_t stream) {
    const PageWork w = page_work(workspace, pt.n_pages, n);
    cudaError_t e =
        launch_pdl(k_pages_fork, dim3(1), dim3(kMetaThreads), 0, stream, pt, src, dst, n, w);
    if (e != cudaSuccess || pools.L == 0) return e;
    return launch_pdl(k_pages_copy, dim3((unsigned)(4 * sm_count)), dim3(kCopyThreads), 0, stream,
                      pt, pools, w);
}

cudaError_t launch_pages_compact(const PageTable &pt, const PagePools &pools, int32_t *n_used,
                                 void *workspace, int sm_count, cudaStream_t stream) {
    const PageWork w = page_work(workspace, pt.n_pages, pt.n_pages / 2 + 1);
    cudaError_t e = launch_pdl(k_pages_compact_plan, dim3(1), dim3(kMetaThreads), 0, stream, pt, w,
                               n_used);
    if (e != cudaSuccess) return e;
    return launch_pdl(k_pages_compact_move, dim3((unsigned)(4 * sm_count)), dim3(kCopyThreads), 0,
                      stream, pt, pools, w, (const int32_t *)n_used);
}

cudaError_t launch_pages_append(const PageTable &pt, const void *k, int64_t k_stride,
                                const void *v, int64_t v_stride, const int32_t *slots, int N,
                                int D, const PagePools &pools, cudaStream_t stream) {
    const int64_t warps = (int64_t)N * D * 2;
    const int64_t blocks = (warps * 32 + kCopyThreads - 1) / kCopyThreads;
    return launch_pdl(k_pages_append, dim3((unsigned)blocks), dim3(kCopyThreads), 0, stream, pt,
                      (const char *)k, k_stride, (const char *)v, v_stride, slots, N, D, pools);
}

cudaError_t take_error_pages(cudaStream_t stream, unsigned int *sum) {
    return take_error_here(stream, sum);
}

#ifdef SC_BOUNDS_CHECK
cudaError_t bounds_install_pages(const BoundsRegion *r, int n, cudaStream_t stream) {
    return bounds_install_here(r, n, stream);
}
cudaError_t bounds_take_pages(cudaStream_t stream, unsigned long long *addr) {
    return bounds_take_first_bad_here(stream, addr);
}
#endif

}  // namespace sc
