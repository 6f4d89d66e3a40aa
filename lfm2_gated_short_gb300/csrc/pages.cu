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
// is a function of its inputs alone. The metadata of a call (the listed table
// rows, and the refs array read once) is worked out by one CTA or a cluster,
// which leaves a list of page copies; a second kernel over the whole GPU
// copies the data of every layer, unless it is little.
//
// Metadata is bound by chains of dependent reads, a compaction's copy by DRAM (1.06 GB
// read and written in 161 us, 6.6 TB/s).
#include "common.cuh"
#include "errors.cuh"
#include "kernels.h"
#include "launch.h"
#include "shortconv.h"
#include "tcgen05.cuh"
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
// page_size is a power of two: its logarithm, and the divisions by it.
__device__ __forceinline__ int page_log2(const PageTable &pt) { return __ffs(pt.page_size) - 1; }
__device__ __forceinline__ int pages_of(const PageTable &pt, int len) {
    return (len + pt.page_size - 1) >> page_log2(pt);
}
__device__ __forceinline__ int full_pages(const PageTable &pt, int len) {
    return len >> page_log2(pt);
}
__device__ __forceinline__ int part_of(const PageTable &pt, int len) {
    return len & (pt.page_size - 1);
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

// refs of the 16 pages from p0 + 16 t on, for thread t (pages past the end: in use).
constexpr int kScanPages = 16;
__device__ __forceinline__ void load_refs(const PageTable &pt, int p0, int (&r)[kScanPages]) {
    const int p = p0 + (int)threadIdx.x * kScanPages;
    if (p + kScanPages <= pt.n_pages && (reinterpret_cast<uintptr_t>(pt.refs) & 15) == 0 &&
        SC_RD_OK(pt.refs + p, 4 * kScanPages)) {
#pragma unroll
        for (int k = 0; k < kScanPages; k += 4) {
            const int4 v = __ldcg(reinterpret_cast<const int4 *>(pt.refs + p + k));
            r[k] = v.x, r[k + 1] = v.y, r[k + 2] = v.z, r[k + 3] = v.w;
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < kScanPages; ++k) r[k] = p + k < pt.n_pages ? ld_refs(pt.refs + p + k) : 1;
}

// The `want` lowest free pages into claimed[]; false with fewer free.
__device__ bool claim_lowest(const PageTable &pt, int want, int32_t *claimed) {
    int found = 0;
    for (int p0 = 0; p0 < pt.n_pages && found < want; p0 += kMetaThreads * kScanPages) {
        int r[kScanPages], mine = 0, here;
        load_refs(pt, p0, r);
#pragma unroll
        for (int k = 0; k < kScanPages; ++k) mine += r[k] <= 0;
        int rank = found + block_scan(mine, &here);
#pragma unroll
        for (int k = 0; k < kScanPages; ++k)
            if (r[k] <= 0) {
                if (rank < want) gst(claimed + rank, p0 + (int)threadIdx.x * kScanPages + k);
                ++rank;
            }
        found += here;
    }
    __syncthreads();  // claimed[] is read by other threads
    return found >= want;
}

// Up to kMetaThreads listed sequences in shared memory: entries [lo, hi) of each one's
// table row are the call's business (lo == hi for one that is skipped).
struct Rows {
    int n;
    int4 q[kMetaThreads];  // slot, lo, hi, and what the call keeps of it
};

// Threads as (row group, column): a thread walks its group's rows, so that
// branches of one prompt, next to each other in the list, meet in one thread and
// their equal page ids become one atomic; the CTAs of the cluster take the
// columns in turn. f(first row, end row, column) for every column.
template <typename F>
__device__ __forceinline__ void for_entries(const Rows &rows, F &&f) {
    __shared__ int s_width;
    int width = 0;
    for (int r = threadIdx.x; r < rows.n; r += kMetaThreads)
        width = max(width, rows.q[r].z - rows.q[r].y);
    __syncthreads();
    if (threadIdx.x == 0) s_width = 0;
    __syncthreads();
    width = __reduce_max_sync(~0u, width);
    if ((threadIdx.x & 31) == 0) atomicMax(&s_width, width);
    __syncthreads();
    width = s_width;
    const int ctas = (int)cluster_ctas(), rank = (int)cluster_ctarank();
    int shift = 5;  // 2^shift columns a CTA at once
    while ((1 << shift) * ctas < width && (1 << shift) < kMetaThreads) ++shift;
    const int groups = kMetaThreads >> shift, col = threadIdx.x & ((1 << shift) - 1);
    const int per = (rows.n + groups - 1) / groups;
    const int r0 = min(rows.n, (int)(threadIdx.x >> shift) * per), r1 = min(rows.n, r0 + per);
    for (int c = (rank << shift) + col; c < width; c += ctas << shift) f(r0, r1, c);
}

// refs += sign for every listed entry.
__device__ __forceinline__ void count_entries(const PageTable &pt, const Rows &rows, int sign) {
    for_entries(rows, [&](int r0, int r1, int c) {
        int id = -1, run = 0;
        constexpr int kAhead = 8;  // entries in flight
        for (int r = r0; r < r1; r += kAhead) {
            int e[kAhead], in = 0;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int4 q = rows.q[min(r + k, r1 - 1)];
                const bool live = r + k < r1 && q.y + c < q.z;
                e[k] = live ? gld(table_row(pt, q.x) + q.y + c) : id;
                in |= (int)live << k;
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (!(in >> k & 1)) continue;
                if (e[k] != id) {
                    if (run) add_refs(pt, id, sign * run);
                    id = e[k];
                    run = 0;
                }
                if (page_ok(pt, id))
                    ++run;
                else if (sign < 0)
                    raise_error(SC_DEV_BAD_PAGE);
            }
        }
        if (run) add_refs(pt, id, sign * run);
    });
}

// Written by one CTA of a cluster and read, after a cluster barrier, by the others.
template <typename V>
__device__ __forceinline__ V ld_shared_word(const V *p) {
    if (!SC_RD_OK(p, sizeof(V))) return V{};
    return __ldcg(p);
}

// Copies 0 .. n - 1 in every layer and pool. A unit is up to 4 KB of one page copy,
// one warp's; `worker` of `workers` warps.
__device__ __forceinline__ void copy_pages(const PageWork &w, int n, const PageTable &pt,
                                           const PagePools &pools, int worker, int workers) {
    constexpr int kWords = 8;  // 16-byte words a lane
    const int lane = threadIdx.x & 31;
    const int64_t page_bytes = pt.page_size * pools.token_bytes;
    const uint32_t chunks = (uint32_t)((page_bytes / 16 + 32 * kWords - 1) / (32 * kWords));
    const uint32_t per_copy = chunks * 2 * (uint32_t)pools.L;
    for (int64_t u = worker; u < (int64_t)n * per_copy; u += workers) {
        const uint32_t ci = u <= UINT32_MAX ? (uint32_t)u / per_copy : (uint32_t)(u / per_copy);
        const uint32_t rest = (uint32_t)(u - (int64_t)ci * per_copy), lp = rest / chunks;
        const int4 c = ld_shared_word(reinterpret_cast<const int4 *>(w.copies + ci));
        char *base =
            (char *)(lp & 1 ? pools.v : pools.k) + (int64_t)(lp >> 1) * pt.n_pages * page_bytes;
        const uint4 *from = (const uint4 *)(base + c.x * page_bytes);
        uint4 *to = (uint4 *)(base + c.y * page_bytes);
        const int q = (int)(c.z * pools.token_bytes / 16);
        const int i0 = (int)(rest - lp * chunks) * 32 * kWords + lane;
        uint4 v[kWords];
#pragma unroll
        for (int k = 0; k < kWords; ++k)
            if (i0 + 32 * k < q) v[k] = ld_plain(from + i0 + 32 * k);
#pragma unroll
        for (int k = 0; k < kWords; ++k)
            if (i0 + 32 * k < q) st_plain(to + i0 + 32 * k, v[k]);
    }
    // A page's scales go whole: those of blocks without a copied token are nobody's.
    if (pools.page_scales == 0) return;
    for (int64_t u = worker; u < (int64_t)n * 2 * pools.L; u += workers) {
        const uint32_t ci = (uint32_t)(u / (2 * pools.L)), lp = (uint32_t)(u - (int64_t)ci * 2 * pools.L);
        const int4 c = ld_shared_word(reinterpret_cast<const int4 *>(w.copies + ci));
        float *base = (lp & 1 ? pools.v_scales : pools.k_scales) +
                      (int64_t)(lp >> 1) * pt.n_pages * pools.page_scales;
        const float *from = base + (int64_t)c.x * pools.page_scales;
        float *to = base + (int64_t)c.y * pools.page_scales;
        for (int i = lane; i < pools.page_scales; i += 32) gst(to + i, gld(from + i));
    }
}

// The end of a resize or fork: the number of copies for the copy kernel, or the copies
// themselves, by the cluster's warps, where they are few.
__device__ __forceinline__ void finish_copies(const PageWork &w, int n, bool enough,
                                              const PageTable &pt, const PagePools &pools,
                                              int inline_copy) {
    const int rank = (int)cluster_ctarank();
    if (rank == 0 && threadIdx.x == 0) {
        if (!enough) raise_error(SC_DEV_NO_PAGE);
        gst(w.n_copies, enough ? n : 0);
    }
    cluster_sync();
    if (inline_copy)
        copy_pages(w, ld_shared_word(w.n_copies), pt, pools,
                   rank * (kMetaThreads / 32) + (int)(threadIdx.x >> 5),
                   (int)cluster_ctas() * (kMetaThreads / 32));
}

// A cluster works a resize or fork out: entries are spread over its CTAs, what
// needs an order (claims) or is one item a sequence is CTA 0's. The
// barriers between the steps are the cluster's. `inline_copy`: the copies are
// few enough to be made here (else k_pages_copy follows).
__global__ void __launch_bounds__(kMetaThreads)
    k_pages_resize(PageTable pt, const int32_t *__restrict__ slots,
                   const int32_t *__restrict__ new_lens, int n, PageWork w, PagePools pools,
                   int inline_copy) {
    __shared__ int s_copies;
    __shared__ Rows rows;
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    const bool first = cluster_ctarank() == 0;
    const int64_t cap = (int64_t)pt.max_pages * pt.page_size;
    if (tid == 0) s_copies = 0;
    // This thread's listed sequence of those from i0 on: slot, old and new length. With at
    // most kMetaThreads listed it is read once and stays in registers.
    int slot = 0, old = 0, now = 0;
    bool ok = false;
    auto read = [&](int i0, bool report) {
        const int i = i0 + tid;
        if (n <= kMetaThreads && !report) return;
        ok = false;
        if (i >= n) return;
        slot = gld(slots + i);
        now = gld(new_lens + i);
        old = slot_len(pt, slot, report && first);
        ok = old >= 0;
        if (ok && (now < 0 || now > cap)) {
            if (report && first) raise_error(SC_DEV_BAD_LENGTH);
            ok = false;
        }
    };
    // The claims of the sequences from i0 on, as this thread's first one (-1 - it where the
    // sequence gets a copy of its last page), and the number of all so far.
    auto claims = [&](int want, int *at) {
        int mine = 0, copy = 0;
        if (ok) {
            const int need = pages_of(pt, now), have = pages_of(pt, old);
            if (now < old && part_of(pt, now) != 0) {
                const int id = gld(table_row(pt, slot) + need - 1);
                copy = page_ok(pt, id) && ld_refs(pt.refs + id) > 1;
            }
            mine = copy + max(0, need - have);
        }
        int here;
        const int begin = want + block_scan(mine, &here);
        *at = copy ? -1 - begin : begin;
        return want + here;
    };
    // The sequences as rows: released entries, or with `all` the claimed ones too; .w is
    // the first claim of a growing one, else -1.
    auto list = [&](int i0, bool all, int at) {
        __syncthreads();
        if (tid == 0) rows.n = min(n - i0, kMetaThreads);
        if (i0 + tid < n) {
            const int need = pages_of(pt, now), have = pages_of(pt, old);
            const bool grows = all && need > have;
            rows.q[tid] = make_int4(slot, ok ? (grows ? have : need) : 0,
                                    ok ? (grows ? need : max(need, have)) : 0,
                                    ok && grows ? at : -1);
        }
        __syncthreads();
    };
    for (int i0 = 0; i0 < n; i0 += kMetaThreads) {
        read(i0, true);
        list(i0, false, 0);
        count_entries(pt, rows, -1);
    }
    cluster_sync();
    // Every CTA counts the claims; CTA 0 looks the pages up.
    int want = 0, at = 0;
    for (int i0 = 0; i0 < n; i0 += kMetaThreads) {
        read(i0, false);
        want = claims(want, &at);
        if (n > kMetaThreads && first && i0 + tid < n) gst(w.offset + i0 + tid, at);
    }
    if (first) {
        const bool found = want <= pt.n_pages && claim_lowest(pt, want, w.claimed);
        if (tid == 0) gst(w.n_copies, found ? 1 : 0);  // until the copies are counted
    }
    cluster_sync();
    const bool enough = ld_shared_word(w.n_copies) != 0;
    for (int i0 = 0; i0 < n; i0 += kMetaThreads) {
        read(i0, false);
        if (n > kMetaThreads && i0 + tid < n) at = ld_shared_word(w.offset + i0 + tid);
        list(i0, enough, at);
        if (!enough) {  // take the releases back
            count_entries(pt, rows, 1);
            continue;
        }
        if (first && ok && at < 0) {
            int32_t *entry = table_row(pt, slot) + pages_of(pt, now) - 1;
            const int from = gld(entry), to = gld(w.claimed + (-1 - at));
            add_refs(pt, from, -1);
            add_refs(pt, to, 1);
            gst(entry, to);
            gst(w.copies + atomicAdd(&s_copies, 1), PageCopy{from, to, part_of(pt, now), 0});
        }
        for_entries(rows, [&](int r0, int r1, int c) {
            for (int r = r0; r < r1; ++r) {
                const int4 q = rows.q[r];
                if (q.y + c >= q.z) continue;
                int id = -1;
                if (q.w >= 0) {
                    id = ld_shared_word(w.claimed + q.w + c);
                    add_refs(pt, id, 1);
                }
                gst(table_row(pt, q.x) + q.y + c, id);
            }
        });
    }
    cluster_sync();  // every CTA has read the old lengths
    for (int i0 = 0; first && enough && i0 < n; i0 += kMetaThreads) {
        read(i0, false);
        if (ok) gst(pt.lens + slot, now);
    }
    finish_copies(w, s_copies, enough, pt, pools, inline_copy);
}

__global__ void __launch_bounds__(kMetaThreads)
    k_pages_fork(PageTable pt, const int32_t *__restrict__ src, const int32_t *__restrict__ dst,
                 int n, PageWork w, PagePools pools, int inline_copy) {
    __shared__ int s_copies;
    __shared__ Rows rows;
    __shared__ int2 s_share[kMetaThreads];  // of a pair: full pages, the page after them (-1: none)
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    const bool first = cluster_ctarank() == 0;
    if (tid == 0) s_copies = 0;
    // This thread's pair of those from i0 on. With at most kMetaThreads it is read once.
    int s = 0, d = 0, ls = 0, ld = 0;
    bool ok = false;
    auto read = [&](int i0, bool report) {
        const int i = i0 + tid;
        if (n <= kMetaThreads && !report) return;
        ok = false;
        if (i >= n) return;
        s = gld(src + i);
        d = gld(dst + i);
        ls = slot_len(pt, s, report && first);
        ld = slot_len(pt, d, report && first);
        ok = ls >= 0 && ld >= 0 && s != d;
        if (s == d && ls >= 0 && report && first) raise_error(SC_DEV_BAD_SLOT);
    };
    // The pairs as rows: the destination's own entries, or with `share` its whole row (.w:
    // the source).
    auto list = [&](int i0, bool share) {
        __syncthreads();
        if (tid == 0) rows.n = min(n - i0, kMetaThreads);
        if (i0 + tid < n)
            rows.q[tid] = make_int4(d, 0, !ok ? 0 : share ? pt.max_pages : pages_of(pt, ld), s);
        __syncthreads();
    };
    for (int i0 = 0; i0 < n; i0 += kMetaThreads) {
        read(i0, true);
        list(i0, false);
        count_entries(pt, rows, -1);
    }
    cluster_sync();
    // Every CTA counts the claims; CTA 0 looks the pages up.
    int want = 0, at = 0;
    for (int i0 = 0; i0 < n; i0 += kMetaThreads) {
        read(i0, false);
        int here;
        at = want + block_scan(ok && part_of(pt, ls) != 0, &here);
        if (n > kMetaThreads && first && i0 + tid < n) gst(w.offset + i0 + tid, at);
        want += here;
    }
    if (first) {
        const bool found = want <= pt.n_pages && claim_lowest(pt, want, w.claimed);
        if (tid == 0) gst(w.n_copies, found ? 1 : 0);  // until the copies are counted
    }
    cluster_sync();
    const bool enough = ld_shared_word(w.n_copies) != 0;
    for (int i0 = 0; i0 < n; i0 += kMetaThreads) {
        read(i0, false);
        if (n > kMetaThreads && i0 + tid < n) at = ld_shared_word(w.offset + i0 + tid);
        __syncthreads();  // s_share of the pairs before
        if (enough && i0 + tid < n) {
            int last = -1;
            if (ok && part_of(pt, ls)) {
                last = ld_shared_word(w.claimed + at);
                if (first) {
                    const int from = gld(table_row(pt, s) + full_pages(pt, ls));
                    add_refs(pt, last, 1);
                    if (page_ok(pt, from))
                        gst(w.copies + atomicAdd(&s_copies, 1),
                            PageCopy{from, last, part_of(pt, ls), 0});
                    else
                        raise_error(SC_DEV_BAD_PAGE);
                }
            }
            s_share[tid] = make_int2(full_pages(pt, ls), last);
        }
        list(i0, enough);
        if (!enough) {
            count_entries(pt, rows, 1);
            continue;
        }
        for_entries(rows, [&](int r0, int r1, int c) {
            int from = -1, entry = -1, run = 0;  // of the last source, and its run of shares
            auto flush = [&]() {
                if (run == 0) return;
                if (page_ok(pt, entry))
                    add_refs(pt, entry, run);
                else
                    raise_error(SC_DEV_BAD_PAGE);
                run = 0;
            };
            for (int r = r0; r < r1; ++r) {
                const int4 q = rows.q[r];
                const int2 share = s_share[r];
                if (q.z == 0) continue;
                int v = c == share.x ? share.y : -1;
                if (c < share.x) {
                    if (q.w != from) {
                        flush();
                        from = q.w;
                        entry = gld(table_row(pt, from) + c);
                    }
                    ++run;
                    v = entry;
                }
                gst(table_row(pt, q.x) + c, v);
            }
            flush();
        });
    }
    cluster_sync();  // every CTA has read the old lengths
    for (int i0 = 0; first && enough && i0 < n; i0 += kMetaThreads) {
        read(i0, false);
        if (ok) gst(pt.lens + d, ls);
    }
    finish_copies(w, s_copies, enough, pt, pools, inline_copy);
}

// U = used pages; the i-th used page >= U moves to the i-th free page < U.
// claimed[p] becomes the new id of moved page p.
__global__ void __launch_bounds__(kMetaThreads)
    k_pages_compact_plan(PageTable pt, PageWork w, int32_t *__restrict__ n_used) {
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    constexpr int kStep = kMetaThreads * kScanPages;
    int used = 0, here, r[kScanPages];
    for (int p0 = 0; p0 < pt.n_pages; p0 += kStep) {
        load_refs(pt, p0, r);
        int mine = 0;
#pragma unroll
        for (int k = 0; k < kScanPages; ++k)
            mine += r[k] > 0 && p0 + tid * kScanPages + k < pt.n_pages;
        block_scan(mine, &here);
        used += here;
    }
    int holes = 0, moved = 0;
    for (int p0 = 0; p0 < pt.n_pages; p0 += kStep) {
        if (pt.n_pages > kStep) load_refs(pt, p0, r);  // else they are still here
        const int p = p0 + tid * kScanPages;
        int hole = 0, move = 0;
#pragma unroll
        for (int k = 0; k < kScanPages; ++k) {
            hole += p + k < used && r[k] <= 0;
            move += p + k >= used && p + k < pt.n_pages && r[k] > 0;
        }
        int rh = holes + block_scan(hole, &here);
        holes += here;
        int rm = moved + block_scan(move, &here);
        moved += here;
#pragma unroll
        for (int k = 0; k < kScanPages; ++k) {
            if (p + k < used && r[k] <= 0) gst(&w.copies[rh++].dst, p + k);
            if (p + k >= used && p + k < pt.n_pages) {
                if (r[k] > 0)
                    gst(&w.copies[rm++].src, p + k);
                else
                    gst(w.claimed + p + k, -1);  // a table may not name it
            }
        }
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

__global__ void __launch_bounds__(kCopyThreads)
    k_pages_copy(PageTable pt, PagePools pools, PageWork w) {
    pdl_wait();
    pdl_launch_dependents();
    const int warps = kCopyThreads / 32;
    copy_pages(w, gld(w.n_copies), pt, pools, blockIdx.x * warps + (threadIdx.x >> 5),
               gridDim.x * warps);
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
    copy_pages(w, n, pt, pools, (int)(tid >> 5), (int)(threads >> 5));
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
    const int id = gld(table_row(pt, slot) + full_pages(pt, pos));
    if (!page_ok(pt, id)) {
        if (lane == 0) raise_error(SC_DEV_BAD_PAGE);
        return;
    }
    const bool is_v = unit & 1;
    const uint4 *from = (const uint4 *)(is_v ? v + token * v_stride : k + token * k_stride);
    uint4 *to = (uint4 *)((char *)(is_v ? pools.v : pools.k) +
                          ((int64_t)id * pt.page_size + part_of(pt, pos)) * pools.token_bytes);
    for (int64_t q = lane; q < pools.token_bytes / 16; q += 32) st_plain(to + q, ld_plain(from + q));
}

// ------------------------------------------------------------ host side

size_t pages_workspace_bytes(int n_pages, int n) {
    // n: listed sequences of a resize or fork (a copy each); 0: a compaction (up to half the pages)
    const size_t copies = n > 0 ? (size_t)n : (size_t)n_pages / 2 + 1;
    return 16 + copies * sizeof(PageCopy) + ((size_t)n_pages + n) * 4;
}

// The plan of a resize or fork. One CTA is enough for a few thousand table entries; with
// more, 8 share them. Forks of 2 to 64 branches, us with one CTA and with eight: 2100 entries
// 11.5-12.0 and 11.6-12.9, 4100 entries 12.1-12.7 and 11.3-12.9, 8200 entries 13.4-14.0 and
// 12.4-12.8, 16400 entries 16.9-17.1 and 13.0-13.4; a fork and a resize of 64 sequences of 1025
// pages 49 and 26. Copies of up to 128 KB a CTA, were every listed sequence to need one, are
// made in the same launch. Where few or none are needed, as in a resize, that spares one (a
// fork and a resize of 2 sequences: 14.0 us, 15.0 with the copy kernel). Where all are: one CTA
// 9.9 us with 64 KB, 11.0 with 128 and 14.5 with 384 (10.2, 10.4 and 10.5 with the copy kernel),
// eight CTAs 13.2 with 64 KB each, 13.4 with 128 and 15.1 with 192 (11.9, 12.2 and 11.9).
struct MetaPlan {
    unsigned ctas;
    int inline_copy;
};
static MetaPlan meta_plan(const PageTable &pt, const PagePools &pools, int n) {
    MetaPlan m;
    m.ctas = (int64_t)n * pt.max_pages > 4096 ? 8 : 1;
    m.inline_copy = (int64_t)n * pools.L * 2 * pt.page_size * pools.token_bytes <=
                    (int64_t)m.ctas * (128 << 10);
    return m;
}

template <typename F>
static cudaError_t launch_meta(F kernel, const PageTable &pt, const int32_t *a, const int32_t *b,
                               int n, const PagePools &pools, void *workspace, int sm_count,
                               cudaStream_t stream) {
    const PageWork w = page_work(workspace, pt.n_pages, n);
    const MetaPlan m = meta_plan(pt, pools, n);
    const cudaError_t e = launch_pdl_cluster(kernel, dim3(m.ctas), dim3(kMetaThreads), 0, stream,
                                             m.ctas, pt, a, b, n, w, pools, m.inline_copy);
    if (e != cudaSuccess || m.inline_copy) return e;
    return launch_pdl(k_pages_copy, dim3((unsigned)(4 * sm_count)), dim3(kCopyThreads), 0, stream,
                      pt, pools, w);
}

cudaError_t launch_pages_resize(const PageTable &pt, const int32_t *slots, const int32_t *new_lens,
                                int n, const PagePools &pools, void *workspace, int sm_count,
                                cudaStream_t stream) {
    return launch_meta(k_pages_resize, pt, slots, new_lens, n, pools, workspace, sm_count, stream);
}

cudaError_t launch_pages_fork(const PageTable &pt, const int32_t *src, const int32_t *dst, int n,
                              const PagePools &pools, void *workspace, int sm_count,
                              cudaStream_t stream) {
    return launch_meta(k_pages_fork, pt, src, dst, n, pools, workspace, sm_count, stream);
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
