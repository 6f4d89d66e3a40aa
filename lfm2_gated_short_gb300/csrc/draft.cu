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
// Only row a of p and q is read whole: 2 V values a sequence.
#include "common.cuh"
#include "errors.cuh"
#include "kernels.h"
#include "launch.h"
#include "shortconv.h"
#include "tma.cuh"

namespace sc {

constexpr int kDraftThreads = 512;
typedef unsigned long long u64;

__device__ __forceinline__ float prob_of(const float *p) { return gld(p); }
__device__ __forceinline__ float prob_of(const __nv_bfloat16 *p) {
    return __bfloat162float(gld(p));
}

// trunc(2^40 clamp(p, 0, 1)); fmaxf makes a NaN 0.
__device__ __forceinline__ u64 weight_of(float p) {
    return __float2ull_rz(fminf(fmaxf(p, 0.0f), 1.0f) * 1099511627776.0f);
}

// floor(total m / 2^31) for total < 2^62, m < 2^31.
__device__ __forceinline__ u64 scaled_mark(u64 total, u64 m) {
    return ((total >> 32) * m << 1) + (((total & 0xFFFFFFFFull) * m) >> 31);
}

template <typename T>
__global__ void __launch_bounds__(kDraftThreads)
    k_draft_accept(int V, int D, const T *__restrict__ target, int64_t target_stride,
                   const T *__restrict__ draft, int64_t draft_stride,
                   const int32_t *__restrict__ tokens, const int32_t *__restrict__ n_drafts,
                   const float *__restrict__ uniforms, int32_t *__restrict__ accepted,
                   int32_t *__restrict__ out_tokens) {
    constexpr int kWarps = kDraftThreads / 32;
    __shared__ int s_a, s_n, s_pick;
    __shared__ u64 s_sum[kWarps];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t i = blockIdx.x;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float *u = uniforms + i * (D + 1);
    int32_t *out = out_tokens + i * (D + 1);

    if (warp == 0) {  // the first rejected draft
        int n = n_drafts ? gld(n_drafts + i) : D;
        bool bad = n < 0 || n > D;
        if (bad && lane == 0) raise_error(SC_DEV_BAD_ACCEPTED);
        int a = bad ? 0 : n;
        for (int j0 = 0; !bad && j0 < n; j0 += 32) {
            const int j = j0 + lane;
            bool ok = true, wrong = false;
            if (j < n) {
                const int x = gld(tokens + i * D + j);
                wrong = x < 0 || x >= V;
                if (!wrong) {
                    const double p = prob_of(target + (i * (D + 1) + j) * target_stride + x);
                    const double q = draft ? prob_of(draft + (i * D + j) * draft_stride + x) : 1.0;
                    ok = (double)gld(u + j) * q < p;
                }
            }
            if (__any_sync(~0u, wrong)) {
                if (lane == 0) raise_error(SC_DEV_BAD_TOKEN);
                bad = true;
            }
            const unsigned no = __ballot_sync(~0u, !ok);
            if (no && a == n) a = j0 + __ffs(no) - 1;
        }
        if (lane == 0) {
            s_a = bad ? -1 : a;
            s_n = n;
            s_pick = -1;
        }
    }
    __syncthreads();
    const int a = s_a;
    if (a < 0) {  // bad drafts: nothing accepted, no token
        for (int j = tid; j <= D; j += kDraftThreads) gst(out + j, -1);
        if (tid == 0) gst(accepted + i, 0);
        return;
    }
    const T *p = target + (i * (D + 1) + a) * target_stride;
    const T *q = draft && a < s_n ? draft + (i * D + a) * draft_stride : nullptr;
    const int sure = !draft && a < s_n ? gld(tokens + i * D + a) : -1;
    bool rest = a < s_n;
    auto weight = [&](int t) -> u64 {
        const u64 wp = weight_of(prob_of(p + t));
        if (!rest) return wp;
        const u64 wq = q ? weight_of(prob_of(q + t)) : t == sure ? 1ull << 40 : 0ull;
        return wp > wq ? wp - wq : 0ull;
    };
    // Each warp owns a run of tokens.
    const int per = ((V + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int t0 = min(V, warp * per), t1 = min(V, t0 + per);
    u64 total = 0, before = 0, mine = 0;
    for (int pass = 0; pass < 2; ++pass) {  // the rest; the whole of p where nothing is left
        mine = 0;
        for (int t = t0 + lane; t < t1; t += 32) mine += weight(t);
#pragma unroll
        for (int o = 16; o; o >>= 1) mine += __shfl_xor_sync(~0u, mine, o);
        if (lane == 0) s_sum[warp] = mine;
        __syncthreads();
        total = before = 0;
        for (int k = 0; k < kWarps; ++k) {
            if (k == warp) before = total;
            total += s_sum[k];
        }
        __syncthreads();
        if (total > 0 || !rest) break;
        rest = false;
    }
    const float r = gld(u + D);
    const u64 mark = scaled_mark(total, (u64)__float2ull_rz(fminf(fmaxf(r, 0.0f), 0.99999994f) * 2147483648.0f));
    if (mark >= before && mark < before + mine) {  // this warp's run holds the token
        u64 sum = before;
        for (int c = t0; c < t1; c += 32) {
            const int t = c + lane;
            u64 inc = t < t1 ? weight(t) : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 up = __shfl_up_sync(~0u, inc, o);
                if (lane >= o) inc += up;
            }
            const unsigned hit = __ballot_sync(~0u, sum + inc > mark);
            if (hit) {
                if (lane == 0) s_pick = c + __ffs(hit) - 1;
                break;
            }
            sum += __shfl_sync(~0u, inc, 31);
        }
    }
    __syncthreads();
    if (tid == 0) {
        if (total == 0) raise_error(SC_DEV_BAD_PROBS);
        gst(accepted + i, a);
    }
    for (int j = tid; j <= D; j += kDraftThreads)
        gst(out + j, j < a ? gld(tokens + i * D + j) : j == a ? s_pick : -1);
}

template <typename T>
static cudaError_t launch_accept(int V, int N, int D, const void *target, int64_t target_stride,
                                 const void *draft, int64_t draft_stride, const int32_t *tokens,
                                 const int32_t *n_drafts, const float *uniforms, int32_t *accepted,
                                 int32_t *out_tokens, cudaStream_t stream) {
    return launch_pdl(k_draft_accept<T>, dim3((unsigned)N), dim3(kDraftThreads), 0, stream, V, D,
                      (const T *)target, target_stride, (const T *)draft, draft_stride, tokens,
                      n_drafts, uniforms, accepted, out_tokens);
}

cudaError_t launch_draft_accept(int dtype, int V, int N, int D, const void *target,
                                int64_t target_stride, const void *draft, int64_t draft_stride,
                                const int32_t *tokens, const int32_t *n_drafts,
                                const float *uniforms, int32_t *accepted, int32_t *out_tokens,
                                cudaStream_t stream) {
    return (dtype == SC_BF16 ? launch_accept<__nv_bfloat16> : launch_accept<float>)(
        V, N, D, target, target_stride, draft, draft_stride, tokens, n_drafts, uniforms, accepted,
        out_tokens, stream);
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
