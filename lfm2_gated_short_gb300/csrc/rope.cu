// rope.cu -- rotary positions: pairs of a head's first R values turned by position times
// frequency, and the gradient, the same turn backwards.
//
//   a' = A (a cos t - b sin t),  b' = A (b cos t + a sin t),  t = p f_i
// Pair i is (x_i, x_{i + R/2}) or (x_{2i}, x_{2i+1}).
//
// The angle is counted in turns as a 64-bit fraction: F_i = f_i / 2 pi mod 1 in units of
// 2^-64, and p F_i mod 2^64 is exact for every position, so that a far position's angle
// is as good as a near one's (an fp32 product of 10^6 radians is off by up to 0.03). Sines and
// cosines come from the fraction's distance to the nearest quarter turn.
//
// A tile is a few tokens: its sines and cosines are computed once, for all heads, into
// shared memory; the rest streams the heads through registers, bound by their bytes: 16384 tokens of
// 32 + 8 bf16 heads of 64, forward and backward (336 MB), 56.7 us, 5.9 TB/s of the 6.75 that a copy
// reaches; 5001 of 14 + 2 fp32 heads of 128 at far positions, half turned (164 MB), 30.5 us, 5.4 TB/s. A
// step's few tokens are latency, 2.8 us.
#include <cuda_bf16.h>

#include "common.cuh"
#include "errors.cuh"
#include "kernels.h"
#include "launch.h"
#include "shortconv.h"

namespace sc {

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 8;     // of a tile, at most

// Turns a position of f radians a position, mod 1, in units of 2^-64: f = m 2^(e - 1075)
// times floor(2^64 / 2 pi), whose relative error is below 2^-61.
__device__ __forceinline__ uint64_t turns_of(double f) {
    const uint64_t b = (uint64_t)__double_as_longlong(f);
    const int e = (int)(b >> 52) & 0x7FF;
    if (e == 0 || e == 0x7FF) return 0;
    const uint64_t m = (b & 0xFFFFFFFFFFFFFull) | 1ull << 52;
    constexpr uint64_t kInv2Pi = 0x28BE60DB9391054Aull;
    const uint64_t lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
    const int s = 1075 - e;  // the product's shift to the right
    uint64_t t;
    if (s <= 0)
        t = s > -64 ? lo << -s : 0;
    else if (s < 64)
        t = hi << (64 - s) | lo >> s;
    else
        t = s < 128 ? hi >> (s - 64) : 0;
    return (int64_t)b < 0 ? 0 - t : t;
}

// (cos, sin) of a 64-bit fraction of a turn.
__device__ __forceinline__ float2 cos_sin(uint64_t turns) {
    const uint64_t q = (turns + (1ull << 61)) >> 62;  // nearest quarter
    const int64_t rest = (int64_t)(turns - (q << 62));  // within an eighth of a turn
    float s, c;
    sincospif((float)rest * 0x1p-63f, &s, &c);
    const float x = q & 1 ? s : c, y = q & 1 ? c : s;
    return make_float2(((q + 1) & 2) ? -x : x, (q & 2) ? -y : y);
}

// VP values as they are stored, one access where VP fills 16 bytes.
template <typename T, int VP>
struct Part {
    static constexpr bool kFull = VP * sizeof(T) == 16;
    static constexpr int kWords = kFull ? 4 : 1;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (kFull) {
            const uint4 q = ld_plain(p);
            w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
        } else {
            static_assert(VP == 1, "one value or 16 bytes");
            w[0] = __float_as_uint((float)gld(p));
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (kFull)
            st_plain(p, make_uint4(w[0], w[1], w[2], w[3]));
        else
            gst(p, (T)__uint_as_float(w[0]));
    }
    __device__ __forceinline__ void get(float (&f)[VP]) const {
#pragma unroll
        for (int e = 0; e < VP; ++e)
            f[e] = kFull && sizeof(T) == 2 ? (e & 1 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]))
                                           : __uint_as_float(w[e < kWords ? e : 0]);
    }
    __device__ __forceinline__ void set(const float (&f)[VP]) {
        if constexpr (kFull && sizeof(T) == 2) {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = pack_bf16(f[2 * e], f[2 * e + 1]);
        } else {
#pragma unroll
            for (int e = 0; e < VP; ++e) w[e] = __float_as_uint(f[e]);
        }
    }
};

// Position of row t, or INT64_MIN for a row that is left alone.
__device__ __forceinline__ int64_t position_of(const RopeArgs &a, int64_t t, bool report) {
    if (a.positions != nullptr) return gld(a.positions + t);
    const int64_t i = t / a.D;
    const int j = (int)(t - i * a.D), slot = gld(a.slots + i);
    if (slot < 0 || slot >= a.n_slots) {
        if (report) raise_error(SC_DEV_BAD_SLOT);
        return INT64_MIN;
    }
    const int64_t p = (int64_t)gld(a.lens + slot) - a.D + j;
    if (p < 0) {
        if (report) raise_error(SC_DEV_BAD_LENGTH);
        return INT64_MIN;
    }
    return p;
}

template <typename T, int VP, bool HALF>
__global__ void __launch_bounds__(kRopeThreads, 5) k_rope(RopeArgs a, int tokens) {
    extern __shared__ float s_turn[];  // [tokens][cos of the pairs, sin of the pairs]
    __shared__ bool s_live[kRopeTokens];
    pdl_wait();
    pdl_launch_dependents();
    const int half = a.R / 2;
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int here = (int)min((int64_t)tokens, a.T - t0);
    for (int x = threadIdx.x; x < here * half; x += kRopeThreads) {
        const int t = x / half, i = x - t * half;
        const int64_t p = position_of(a, t0 + t, i == 0);
        if (i == 0) s_live[t] = p != INT64_MIN;
        float2 cs = cos_sin((uint64_t)p * turns_of(gld(a.freqs + i)));
        s_turn[t * a.R + i] = cs.x * a.amplitude;
        s_turn[t * a.R + half + i] = (a.inverse ? -cs.y : cs.y) * a.amplitude;
    }
    __syncthreads();
    // Items: VP pairs of a head, then 2 VP of the values behind them (VP of them last, where
    // they are no whole number). A thread takes every 256th, kAhead of them in flight.
    const int turned = half / VP, rest = (a.Dh - a.R) / VP;
    const int per = turned + (a.copy ? (rest + 1) / 2 : 0), heads = a.Hq + a.Hkv;
    // The step to a thread's next item: dt tokens, dh heads, dc places.
    const int dhs = kRopeThreads / per, dc = kRopeThreads - dhs * per, dt = dhs / heads;
    const int dh = dhs - dt * heads;
    int hd = threadIdx.x / per, c = threadIdx.x - hd * per, t = hd / heads;
    hd -= t * heads;
    constexpr int kAhead = VP * sizeof(T) == 16 ? 2 : 1;
    while (t < here) {
        Part<T, VP> u[kAhead], w[kAhead];
        T *to[kAhead];
        int at[kAhead][3];  // first, second (-1: none), place of its sines (-1: copied)
#pragma unroll
        for (int n = 0; n < kAhead; ++n) {
            to[n] = nullptr;
            if (t < here && s_live[t]) {
                const bool is_k = hd >= a.Hq;
                const int64_t row = t0 + t, head = (int64_t)(is_k ? hd - a.Hq : hd) * a.Dh;
                const T *from =
                    (const T *)(is_k ? a.k : a.q) + row * (is_k ? a.k_stride : a.q_stride) + head;
                to[n] = (T *)(is_k ? a.k_out : a.q_out) +
                        row * (is_k ? a.k_out_stride : a.q_out_stride) + head;
                if (c < turned) {
                    at[n][0] = HALF ? c * VP : 2 * c * VP;
                    at[n][1] = at[n][0] + (HALF ? half : VP);
                    at[n][2] = t * a.R + c * VP;
                } else {
                    at[n][0] = a.R + 2 * (c - turned) * VP;
                    at[n][1] = at[n][0] + VP < a.Dh ? at[n][0] + VP : -1;
                    at[n][2] = -1;
                }
                u[n].load(from + at[n][0]);
                if (at[n][1] >= 0) w[n].load(from + at[n][1]);
            }
            t += dt;
            hd += dh;
            c += dc;
            if (c >= per) {
                c -= per;
                ++hd;
            }
            if (hd >= heads) {
                hd -= heads;
                ++t;
            }
        }
#pragma unroll
        for (int n = 0; n < kAhead; ++n) {
            if (to[n] == nullptr) continue;
            if (at[n][2] >= 0) {
                const float *cs = s_turn + at[n][2], *sn = cs + half;
                float x[VP], y[VP];
                u[n].get(x);
                w[n].get(y);
#pragma unroll
                for (int e = 0; e < VP; ++e) {
                    // Pair e is (x_e, y_e), or values 2 e and 2 e + 1 of x and y together.
                    float &p = HALF || VP == 1 ? x[e] : (2 * e < VP ? x : y)[2 * e % VP];
                    float &q = HALF || VP == 1 ? y[e] : (2 * e + 1 < VP ? x : y)[(2 * e + 1) % VP];
                    const float p0 = p, q0 = q;
                    p = p0 * cs[e] - q0 * sn[e];
                    q = q0 * cs[e] + p0 * sn[e];
                }
                u[n].set(x);
                w[n].set(y);
            }
            u[n].store(to[n] + at[n][0]);
            if (at[n][1] >= 0) w[n].store(to[n] + at[n][1]);
        }
    }
}

// ------------------------------------------------------------ host side

template <typename T, int VP>
static cudaError_t launch_rope_vp(const RopeArgs &a, int tokens, cudaStream_t stream) {
    const dim3 grid((unsigned)((a.T + tokens - 1) / tokens));
    const size_t smem = (size_t)tokens * a.R * 4;
    return a.half_layout
               ? launch_pdl(k_rope<T, VP, true>, grid, dim3(kRopeThreads), smem, stream, a, tokens)
               : launch_pdl(k_rope<T, VP, false>, grid, dim3(kRopeThreads), smem, stream, a, tokens);
}

template <typename T>
static cudaError_t launch_rope_t(const RopeArgs &a, int tokens, cudaStream_t stream) {
    // 16-byte accesses where every row, head and half starts on 16 bytes.
    constexpr int kFull = 16 / (int)sizeof(T);
    auto fits = [](const void *p, int64_t stride) {
        return ((uintptr_t)p & 15) == 0 && stride % kFull == 0;
    };
    const bool full = a.R / 2 % kFull == 0 && a.Dh % kFull == 0 && fits(a.q, a.q_stride) &&
                      fits(a.q_out, a.q_out_stride) && fits(a.k, a.k_stride) &&
                      fits(a.k_out, a.k_out_stride);
    return full ? launch_rope_vp<T, kFull>(a, tokens, stream) : launch_rope_vp<T, 1>(a, tokens, stream);
}

cudaError_t launch_rope(int dtype, const RopeArgs &a, int sm_count, cudaStream_t stream) {
    // A tile of up to 44 KB: less pays its sines and its start too often, more leaves the GPU's
    // last wave half empty. us forward and backward, of 40 bf16 heads of 64 (5 KB a token) and 16
    // fp32 heads of 128, half turned (8 KB), with 4 and 8 tokens a tile: 16384 tokens of the
    // first 61.3 and 56.8; 9000 tokens of both 36.2 and 35.0, 49.1 and 53.7; 30000 tokens 105 and 96,
    // 146 and 150. With few tokens, four tiles an SM.
    const int64_t row = (int64_t)(a.Hq + a.Hkv) * a.Dh * (dtype == SC_BF16 ? 2 : 4);
    int tokens = kRopeTokens;
    while (tokens > 1 && (tokens * row > (44 << 10) || a.T < (int64_t)tokens * 4 * sm_count))
        tokens >>= 1;
    return dtype == SC_BF16 ? launch_rope_t<__nv_bfloat16>(a, tokens, stream)
                            : launch_rope_t<float>(a, tokens, stream);
}

cudaError_t take_error_rope(cudaStream_t stream, unsigned int *sum) {
    return take_error_here(stream, sum);
}

#ifdef SC_BOUNDS_CHECK
cudaError_t bounds_install_rope(const BoundsRegion *r, int n, cudaStream_t stream) {
    return bounds_install_here(r, n, stream);
}
cudaError_t bounds_take_rope(cudaStream_t stream, unsigned long long *addr) {
    return bounds_take_first_bad_here(stream, addr);
}
#endif

}  // namespace sc
