// draft.cu -- verification of drafted tokens against the target's probabilities.
//
// Sequence i drafted n <= D tokens x_j from distributions q_j (or with
// certainty); the target gives p_j at each of them and p_n after the last.
// Draft j is accepted while u_j q_j(x_j) < p_j(x_j), in order; a is the
// number accepted. The next token is then drawn from the rest
// max(p_a - q_a, 0) at the rejected draft, or from p_n when none was
// rejected, by the cumulative sum: the lowest token whose inclusive sum
// exceeds u_D times the whole.
//
// Which token that is must not depend on the order of a sum of V terms, so
// the weights are whole numbers: a probability in units of 2^-40 (truncated),
// sums in 64 bits. V <= 2^22 keeps every sum below 2^62. The accept test is a
// product of two 32-bit floats in 64 bits, which is exact.
//
// Only row a of p and q is read whole: 2 V values a sequence. 256 sequences x 130051 in
// bf16: 35 us, 3.8 TB/s, 57 % of the measured copy rate (129 us with conversions to 64-bit
// integers, 54 without packed pairs). No unit is full: the ALU pipe is busy half the time,
// issue slots 46 %, but 58 % on the fullest SM and 36 % on the emptiest. The 512 CTAs lie
// unevenly on 152 SMs that hold four each, and the call takes as long as the full ones.
#include <atomic>

#include "common.cuh"
#include "errors.cuh"
#include "kernels.h"
#include "launch.h"
#include "shortconv.h"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace sc {

constexpr int kDraftThreads = 256;
constexpr int kDraftWarps = kDraftThreads / 32;
constexpr int kMaxDraftCluster = 8;
typedef unsigned long long u64;

__device__ __forceinline__ float prob_of(const float *p) { return gld(p); }
__device__ __forceinline__ float prob_of(const __nv_bfloat16 *p) {
    return __bfloat162float(gld(p));
}

// trunc(2^40 p) = 2^20 hi + lo for 0 <= p <= 1, hi and lo whole and below 2^20 (hi
// 2^20 for p = 1), as the bit patterns of 2^23 + hi and 2^23 + lo: adding 2^23
// rounded towards zero leaves a number's whole part in the low mantissa bits,
// and what is left of 2^20 p after it is exact. Equal exponents make a
// difference of patterns the difference of the numbers. Two numbers at once.
__device__ __forceinline__ f32x2 f2_fma_rz(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 d;
    asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
struct Weights {
    f32x2 hi, lo;
};
__device__ __forceinline__ Weights weights_of(float p0, float p1) {
    const f32x2 scale = f2_make(1048576.0f, 1048576.0f), whole = f2_make(8388608.0f, 8388608.0f);
    const f32x2 p = f2_make(p0, p1);
    const f32x2 h = f2_fma_rz(p, scale, whole);
    const f32x2 rest = f2_fma(p, scale, f2_fma(h, f2_make(-1.0f, -1.0f), whole));
    return {h, f2_fma_rz(rest, scale, whole)};
}
// (hi, lo) += max(weight(p) - weight(q), 0) of two elements, all in [0, 1]:
// truncation keeps the order of p and q, so q is lowered to p where it is larger.
__device__ __forceinline__ void add_rest(float p0, float p1, float q0, float q1, int &hi, int &lo) {
    const Weights p = weights_of(p0, p1), q = weights_of(fminf(p0, q0), fminf(p1, q1));
    hi += (int)p.hi - (int)q.hi;
    hi += (int)(p.hi >> 32) - (int)(q.hi >> 32);
    lo += (int)p.lo - (int)q.lo;
    lo += (int)(p.lo >> 32) - (int)(q.lo >> 32);
}
// One element of any value: clamped, a NaN 0.
__device__ __forceinline__ void add_rest(float p, float q, int &hi, int &lo) {
    add_rest(__saturatef(p), 0.0f, __saturatef(q), 0.0f, hi, lo);
}
__device__ __forceinline__ u64 whole_of(int hi, int lo) {
    return (u64)((long long)hi * 1048576 + lo);
}

// floor(total m / 2^31) for total < 2^62, m < 2^31.
__device__ __forceinline__ u64 scaled_mark(u64 total, u64 m) {
    return ((total >> 32) * m << 1) + (((total & 0xFFFFFFFFull) * m) >> 31);
}

// The kVec = 16 / sizeof(T) probabilities of a row from element t on (a
// multiple of kVec), zeros past V. A row may start anywhere (an odd V moves every
// row): the two aligned 16-byte words that hold them are loaded and shifted;
// a word that reaches outside the row is read by elements.
constexpr int kPer = 2;  // vectors of a lane in a chunk, 32 vectors apart

// Elements are numbered from `skip` before the row's start, where p's row has a 16-byte
// boundary: every vector of p then is one aligned word, and q's is shifted by
// the rows' difference only.
template <typename T>
struct Row16 {
    static constexpr int kVec = 16 / sizeof(T);
    const T *row;    // element 0: not read below `lo`
    int lo, V, mis;  // valid elements [lo, V); bytes that element 0 lies past a boundary

    __device__ __forceinline__ Row16(const T *p, int v, int skip)
        : row(p - skip), lo(skip), V(v + skip),
          mis((int)(reinterpret_cast<uintptr_t>(p - skip) & 15)) {}

    // Whether the words of [t, t + n) lie inside the row.
    __device__ __forceinline__ bool inside(int t, int n) const {
        return t - mis / (int)sizeof(T) >= lo && t + n + (mis ? kVec : 0) <= V;
    }
    // Start copying a warp's words of its chunk from element t on to `dst`, and the one
    // after them that a row off alignment ends in.
    __device__ __forceinline__ void copy(int t, uint32_t dst) const {
        const int lane = threadIdx.x & 31;
        const char *at = reinterpret_cast<const char *>(row + t) - mis + lane * 16;
#pragma unroll
        for (int k = 0; k < kPer; ++k) copy16(dst + (lane + 32 * k) * 16, at + 32 * 16 * k);
        if (mis && lane == 0) copy16(dst + 32 * kPer * 16, at + 32 * kPer * 16);
    }
    static __device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
        if (!SC_RD_OK(src, 16)) {  // refused: zeros
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(0) : "memory");
            return;
        }
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    }
    // The two words that hold this lane's k-th vector of what copy() brought.
    __device__ __forceinline__ void take(const uint4 *at, int k, uint4 (&w)[2]) const {
        w[0] = at[(threadIdx.x & 31) + 32 * k];
        if (mis) w[1] = at[(threadIdx.x & 31) + 32 * k + 1];
    }
    // The kVec elements as 4 words.
    __device__ __forceinline__ void align(const uint4 (&v)[2], uint32_t (&out)[4]) const {
        uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
        if (mis & 8) {  // mis is the same for the whole row
#pragma unroll
            for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
        }
        if (mis & 4) {
#pragma unroll
            for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
        }
        if (mis & 2) {
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 16);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) out[k] = w[k];
    }
    static __device__ __forceinline__ void unpack(const uint32_t (&w)[4], float (&f)[kVec]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (sizeof(T) == 4) {
                f[k] = __uint_as_float(w[k]);
            } else {
                f[2 * k] = bf16_lo(w[k]);
                f[2 * k + 1] = bf16_hi(w[k]);
            }
        }
    }
    // Whether all elements of p and q are in [0, 1]: as whole numbers, larger bit patterns
    // are larger numbers, infinity, NaN and everything negative.
    static __device__ __forceinline__ bool plain(const uint32_t (&p)[4], const uint32_t (&q)[4]) {
        if constexpr (sizeof(T) == 4) {
            const uint32_t m = __vimax3_u32(__vimax3_u32(p[0], p[1], p[2]),
                                            __vimax3_u32(p[3], q[0], q[1]), max(q[2], q[3]));
            return m <= 0x3F800000u;
        } else {
            const uint32_t m = __vimax3_u16x2(__vimax3_u16x2(p[0], p[1], p[2]),
                                              __vimax3_u16x2(p[3], q[0], q[1]),
                                              __vmaxu2(q[2], q[3]));
            return (m & 0xFFFFu) <= 0x3F80u && (m >> 16) <= 0x3F80u;
        }
    }
    // At the row's ends: element by element, zeros outside.
    __device__ __forceinline__ void get(int t, float (&f)[kVec]) const {
#pragma unroll
        for (int e = 0; e < kVec; ++e)
            f[e] = t + e >= lo && t + e < V ? prob_of(row + t + e) : 0.0f;
    }
};

__device__ __forceinline__ u64 warp_scan(u64 v, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 up = __shfl_up_sync(~0u, v, o);
        if (lane >= o) v += up;
    }
    return v;
}

// A warp's copies in flight: kRing chunks of both rows.
constexpr int kRing = 3;
constexpr int kRingWords = 32 * kPer + 1;
constexpr size_t kRingBytes = (size_t)kDraftWarps * kRing * 2 * kRingWords * 16;

// A cluster of CTAs shares a sequence's row of V, one run of chunks each; a chunk is
// kPer vectors a thread. Each warp streams its part of the chunks through a ring of its own
// (4 CTAs an SM: 192 KB in flight, where loads into registers left 50; 256 x 130051 in bf16
// 42 us with those, 35 so). The sums of every (chunk, warp) stay in shared memory, so the row is
// read once and then only the 32 kPer vectors that hold the token again.
// `sums` holds chunks * kDraftWarps entries.
template <typename T>
__global__ void __launch_bounds__(kDraftThreads, 4)
    k_draft_accept(int V, int D, int chunks, const T *__restrict__ target, int64_t target_stride,
                   const T *__restrict__ draft, int64_t draft_stride,
                   const int32_t *__restrict__ tokens, const int32_t *__restrict__ n_drafts,
                   const float *__restrict__ uniforms, int32_t *__restrict__ accepted,
                   int32_t *__restrict__ out_tokens) {
    using R = Row16<T>;
    constexpr int kVec = R::kVec;
    extern __shared__ uint4 dyn[];
    const uint4 *ring = dyn + (threadIdx.x >> 5) * kRing * 2 * kRingWords;  // this warp's
    const uint32_t ring_a = smem_addr(ring);
    u64 *sums = reinterpret_cast<u64 *>(dyn + kRingBytes / 16);
    __shared__ int s_a, s_n;
    __shared__ u64 s_warp[kDraftWarps];
    __shared__ u64 s_total[2][kMaxDraftCluster];  // every CTA's sum, by pass
    __shared__ u64 s_found[kMaxDraftCluster];     // and what it found: a, and whether a < n
    pdl_wait();
    pdl_launch_dependents();
    cluster_arrive();  // every CTA of the cluster runs before one stores to another
    const int C = (int)cluster_ctas(), rank = (int)cluster_ctarank();
    const int64_t i = blockIdx.x / C;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float *u = uniforms + i * (D + 1);
    int32_t *out = out_tokens + i * (D + 1);

    if (warp == 0) {  // the first rejected draft
        int n = n_drafts ? gld(n_drafts + i) : D;
        bool bad = n < 0 || n > D;
        if (bad && lane == 0 && rank == 0) raise_error(SC_DEV_BAD_ACCEPTED);
        int a = bad ? 0 : n;
        for (int j0 = 0; !bad && j0 < n; j0 += 32) {
            const int j = j0 + lane;
            bool ok = true, wrong = false;
            if (j < n) {
                const int x = gld(tokens + i * D + j);
                const float r = gld(u + j);
                wrong = x < 0 || x >= V;
                if (!wrong) {
                    const double p = prob_of(target + (i * (D + 1) + j) * target_stride + x);
                    const double q = draft ? prob_of(draft + (i * D + j) * draft_stride + x) : 1.0;
                    ok = (double)r * q < p;
                }
            }
            if (__any_sync(~0u, wrong)) {
                if (lane == 0 && rank == 0) raise_error(SC_DEV_BAD_TOKEN);
                bad = true;
            }
            const unsigned no = __ballot_sync(~0u, !ok);
            if (no && a == n) a = j0 + __ffs(no) - 1;
        }
        if (lane == 0) {
            s_a = bad ? -1 : a;
            s_n = n;
        }
    }
    __syncthreads();
    const int a = s_a;
    cluster_wait();
    // No CTA leaves before all know what each found: a store to one that has left faults.
    if (tid < C)
        st_cluster_u64(cluster_map(smem_addr(&s_found[rank]), tid),
                       (u64)(uint32_t)a << 1 | (a < s_n));
    if (a < 0) {  // bad drafts
        cluster_sync();
        if (rank == 0) {  // nothing accepted, no token
            for (int j = tid; j <= D; j += kDraftThreads) gst(out + j, -1);
            if (tid == 0) gst(accepted + i, 0);
        }
        return;
    }
    const float r = gld(u + D);
    const T *p_row = target + (i * (D + 1) + a) * target_stride;
    const int skip = (int)(reinterpret_cast<uintptr_t>(p_row) & 15) / (int)sizeof(T);
    const bool with_q = draft && a < s_n;
    const R p(p_row, V, skip);
    const R q(with_q ? draft + (i * D + a) * draft_stride : p_row, V, skip);
    const int sure = !draft && a < s_n ? gld(tokens + i * D + a) + skip : -1;
    bool rest = a < s_n;
    constexpr int kWarpStep = 32 * kPer * kVec, kStep = kDraftWarps * kWarpStep;  // of a chunk
    const int run = chunks * kStep;              // elements of a CTA (V <= 2^22, C <= 8: fits)
    u64 total = 0, before = 0, here = 0;
    for (int pass = 0; pass < 2; ++pass) {  // the rest; the whole of p where nothing is left
        u64 mine = 0;
        const bool use_q = rest && with_q;
        // One chunk's sum over the warp: at most 32 kPer kVec 2^20 = 2^29 in hi, as much in lo.
        auto store = [&](int c, int hi, int lo) {
            const u64 s = whole_of(__reduce_add_sync(~0u, hi), __reduce_add_sync(~0u, lo));
            if (lane == 0) sums[c * kDraftWarps + warp] = s;
            mine += s;
        };
        auto each = [&](const float (&fp)[kVec], const float (&fq)[kVec], int t, int &hi, int &lo) {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                add_rest(fp[e], rest && t + e == sure ? 1.0f : fq[e], hi, lo);
        };
        // This warp's chunks [c0, c1) are whole; the rest, at the row's ends, is read by elements.
        const int tw = rank * run + warp * kWarpStep;
        int c0 = 0, c1 = chunks;
        auto whole = [&](int c) {
            return p.inside(tw + c * kStep, kWarpStep) &&
                   (!use_q || q.inside(tw + c * kStep, kWarpStep));
        };
        while (c0 < chunks && tw + c0 * kStep < V && !whole(c0)) ++c0;
        while (c1 > c0 && !whole(c1 - 1)) --c1;
        for (int c = 0; c < chunks; ++c) {
            if (c == c0 && c1 > c0) c = c1;
            if (c == chunks) break;
            int hi = 0, lo = 0;
            for (int k = 0; k < kPer; ++k) {
                float fp[kVec], fq[kVec] = {};
                const int t = tw + c * kStep + (lane + 32 * k) * kVec;
                p.get(t, fp);
                if (use_q) q.get(t, fq);
                each(fp, fq, t, hi, lo);
            }
            store(c, hi, lo);
        }
        int put = 0, take = 0;  // ring slots
        auto start = [&](int c) {
            if (c < c1) {
                const uint32_t dst = ring_a + put * 2 * kRingWords * 16;
                p.copy(tw + c * kStep, dst);
                if (use_q) q.copy(tw + c * kStep, dst + kRingWords * 16);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            put = put + 1 == kRing ? 0 : put + 1;
        };
        for (int k = 0; k < kRing - 1; ++k) start(c0 + k);
        for (int c = c0; c < c1; ++c) {
            start(c + kRing - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
            __syncwarp();
            const uint4 *at = ring + take * 2 * kRingWords;
            take = take + 1 == kRing ? 0 : take + 1;
            int hi = 0, lo = 0;
#pragma unroll
            for (int k = 0; k < kPer; ++k) {
                float fp[kVec], fq[kVec];
                uint4 raw[2];
                uint32_t uq[4] = {0u, 0u, 0u, 0u};
                const int t = tw + c * kStep + (lane + 32 * k) * kVec;
                const uint4 pw = at[lane + 32 * k];
                const uint32_t up[4] = {pw.x, pw.y, pw.z, pw.w};
                if (use_q) {
                    q.take(at + kRingWords, k, raw);
                    q.align(raw, uq);
                }
                R::unpack(up, fp);
                R::unpack(uq, fq);
                if (R::plain(up, uq) && !(rest && (unsigned)(sure - t) < kVec)) {
#pragma unroll
                    for (int e = 0; e < kVec; e += 2)
                        add_rest(fp[e], fp[e + 1], fq[e], fq[e + 1], hi, lo);
                } else {
                    each(fp, fq, t, hi, lo);
                }
            }
            store(c, hi, lo);
            __syncwarp();  // the words are read before the slot is copied to again
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        if (lane == 0) s_warp[warp] = mine;
        __syncthreads();
        here = 0;
#pragma unroll
        for (int k = 0; k < kDraftWarps; ++k) here += s_warp[k];
        if (tid < C) st_cluster_u64(cluster_map(smem_addr(&s_total[pass][rank]), tid), here);
        cluster_sync();
        // Inputs that change under the call: the CTAs may differ, and all leave here.
        bool same = true;
        for (int k = 0; k < C; ++k) same &= s_found[k] == s_found[0];
        if (!same) return;
        total = before = 0;
        for (int k = 0; k < C; ++k) {
            if (k == rank) before = total;
            total += s_total[pass][k];
        }
        if (total > 0 || !rest) break;  // the same in every CTA
        rest = false;
    }
    if (rank == 0) {
        if (tid == 0) {
            if (total == 0) raise_error(SC_DEV_BAD_PROBS);
            gst(accepted + i, a);
        }
        for (int j = tid; j <= D; j += kDraftThreads)
            if (j != a || total == 0) gst(out + j, j < a ? gld(tokens + i * D + j) : -1);
    }
    const u64 mark = scaled_mark(
        total, (u64)__float2ull_rz(fminf(fmaxf(r, 0.0f), 0.99999994f) * 2147483648.0f));
    if (warp != 0 || mark < before || mark >= before + here) return;
    // This CTA's run holds the token: its (chunk, warp), then the vector.
    u64 sum = before;
    int at = -1;
    for (int k0 = 0; k0 < chunks * kDraftWarps; k0 += 32) {  // kDraftWarps chunks end inside
        const int k = k0 + lane;
        const u64 inc = warp_scan(k < chunks * kDraftWarps ? sums[k] : 0, lane);
        const unsigned hit = __ballot_sync(~0u, sum + inc > mark);
        if (hit) {
            const int h = __ffs(hit) - 1;
            at = k0 + h;
            const u64 up = __shfl_sync(~0u, inc, h > 0 ? h - 1 : 0);
            if (h > 0) sum += up;
            break;
        }
        sum += __shfl_sync(~0u, inc, 31);
    }
    if (at < 0) return;  // cannot be: the run's sum holds the mark
    for (int k = 0; k < kPer; ++k) {
        const int t = rank * run + at / kDraftWarps * kStep + at % kDraftWarps * kWarpStep +
                      (lane + 32 * k) * kVec;
        u64 w[kVec], mine = 0;
        float fp[kVec], fq[kVec] = {};
        p.get(t, fp);
        if (rest && with_q) q.get(t, fq);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            int hi = 0, lo = 0;
            add_rest(fp[e], rest && t + e == sure ? 1.0f : fq[e], hi, lo);
            w[e] = whole_of(hi, lo);
            mine += w[e];
        }
        const u64 inc = warp_scan(mine, lane);
        const unsigned hit = __ballot_sync(~0u, sum + inc > mark);
        if (hit) {
            if (lane == __ffs(hit) - 1) {
                u64 acc = sum + inc - mine;
                int pick = t;
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    acc += w[e];
                    if (acc <= mark) pick = t + e + 1;
                }
                gst(out + a, pick - skip);
            }
            return;
        }
        sum += __shfl_sync(~0u, inc, 31);
    }
}

template <typename T>
static cudaError_t launch_accept(int V, int N, int D, const void *target, int64_t target_stride,
                                 const void *draft, int64_t draft_stride, const int32_t *tokens,
                                 const int32_t *n_drafts, const float *uniforms, int32_t *accepted,
                                 int32_t *out_tokens, int sm_count, cudaStream_t stream) {
    constexpr int kChunk = kDraftThreads * kPer * (16 / (int)sizeof(T));
    // CTAs of a sequence: no more than give each a whole chunk, and all of them on the GPU
    // at once (4 an SM: finding the rejected draft takes three memory latencies, which
    // a second wave would pay again); but the chunk sums have to fit (512 chunks, 32 KB).
    int C = 1;
    while (C < kMaxDraftCluster && V > C * kChunk &&
           (2ll * N * C <= 4 * sm_count || V > C * kChunk * 512))
        C *= 2;
    // Up to a vector less one before the row (see Row16).
    const int chunks = (V + 16 / (int)sizeof(T) - 1 + C * kChunk - 1) / (C * kChunk);
    const size_t smem = kRingBytes + (size_t)chunks * kDraftWarps * 8;
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(done.load() & (1ull << dev))) {
        e = cudaFuncSetAttribute(k_draft_accept<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)(kRingBytes + 513 * kDraftWarps * 8));
        if (e != cudaSuccess) return e;
        if (dev < 64) done.fetch_or(1ull << dev);
    }
    return launch_pdl_cluster(k_draft_accept<T>, dim3((unsigned)(N * C)), dim3(kDraftThreads), smem,
                              stream, (unsigned)C, V, D, chunks,
                              (const T *)target, target_stride, (const T *)draft, draft_stride,
                              tokens, n_drafts, uniforms, accepted, out_tokens);
}

cudaError_t launch_draft_accept(int dtype, int V, int N, int D, const void *target,
                                int64_t target_stride, const void *draft, int64_t draft_stride,
                                const int32_t *tokens, const int32_t *n_drafts,
                                const float *uniforms, int32_t *accepted, int32_t *out_tokens,
                                int sm_count, cudaStream_t stream) {
    return (dtype == SC_BF16 ? launch_accept<__nv_bfloat16> : launch_accept<float>)(
        V, N, D, target, target_stride, draft, draft_stride, tokens, n_drafts, uniforms, accepted,
        out_tokens, sm_count, stream);
}

cudaError_t take_error_draft(cudaStream_t stream, unsigned int *sum) {
    return take_error_here(stream, sum);
}

#ifdef SC_BOUNDS_CHECK
cudaError_t bounds_install_draft(const BoundsRegion *r, int n, cudaStream_t stream) {
    return bounds_install_here(r, n, stream);
}
cudaError_t bounds_take_draft(cudaStream_t stream, unsigned long long *addr) {
    return bounds_take_first_bad_here(stream, addr);
}
#endif

}  // namespace sc
