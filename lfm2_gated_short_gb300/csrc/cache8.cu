// cache8.cu -- the 8-bit paged cache: the quantising append, and reading back.
//
// A block is B tokens of a page under one kv head. Its scale s is the least power of two
// with which all that was written to it fits (|x| <= 448 s), a token's code e4m3(x / s). An
// append that needs a larger scale in a block that holds earlier tokens moves
// those tokens' codes to it.
#include <cuda_bf16.h>

#include "common.cuh"
#include "e4m3.cuh"
#include "errors.cuh"
#include "kernels.h"
#include "launch.h"
#include "shortconv.h"

namespace sc {

constexpr int kAppendThreads = 256;
constexpr int kReadThreads = 256;
constexpr int kReadRows = 32;  // rows of a tile

__device__ __forceinline__ int slot_length(const PageTable &pt, int slot, bool report) {
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

// Eight values of a row as fp32.
template <typename T>
struct Eight {
    Row<T> r;
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < Dt<T>::Q; ++i) r.q[i] = ld_plain(reinterpret_cast<const uint4 *>(p) + i);
    }
    // The largest magnitude's fp32 bits; infinities and NaN do not count.
    __device__ __forceinline__ uint32_t most() const {
        float f[kCh];
        Dt<T>::unpack(r.q, f);
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < kCh; ++e) {
            const uint32_t b = __float_as_uint(f[e]) & 0x7FFFFFFFu;
            m = max(m, b < 0x7F800000u ? b : 0u);
        }
        return m;
    }
    __device__ __forceinline__ uint2 codes(float inverse) const {
        float f[kCh];
        Dt<T>::unpack(r.q, f);
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = f32_e4m3x2(f[2 * e] * inverse, f[2 * e + 1] * inverse);
        return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
    }
};

// A warp takes one block of K or V: it finds the new tokens' largest magnitude, moves the
// earlier codes where the scale rises, and writes the new ones.
template <typename T>
__global__ void __launch_bounds__(kAppendThreads)
    k_append8(PageTable pt, const T *__restrict__ k, int64_t k_stride, const T *__restrict__ v,
              int64_t v_stride, const int32_t *__restrict__ slots, int N, int D, int nb,
              Cache8 c) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t unit = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
    if (unit >= (int64_t)N * nb * 2 * c.Hkv) return;
    const int h = (int)(unit % c.Hkv);
    const int64_t rest = unit / c.Hkv;
    const bool is_v = rest & 1;
    const int b = (int)((rest >> 1) % nb), i = (int)((rest >> 1) / nb);
    const int slot = gld(slots + i);
    const int len = slot_length(pt, slot, lane == 0);
    if (len < 0) return;
    const int first = len - D;  // position of the first new token
    if (first < 0 && lane == 0) raise_error(SC_DEV_BAD_LENGTH);
    const int from = max(first, 0), B = c.block, ps = pt.page_size;
    const int64_t b0 = (int64_t)(from / B + b) * B;
    if (b0 >= len) return;
    const int lo = max((int)b0, from), hi = (int)min(b0 + B, (int64_t)len);
    const int id = gld(pt.table + (int64_t)slot * pt.max_pages + (int)b0 / ps);
    if (id < 0 || id >= pt.n_pages) {
        if (lane == 0) raise_error(SC_DEV_BAD_PAGE);
        return;
    }
    const int r0 = (int)b0 % ps;
    const int64_t width = (int64_t)c.Hkv * c.Dh;
    unsigned char *codes = (unsigned char *)(is_v ? c.v : c.k) +
                           ((int64_t)id * ps + r0) * width + h * c.Dh;  // of the block's first token
    uint32_t *scale = reinterpret_cast<uint32_t *>(is_v ? c.v_scales : c.k_scales) +
                      ((int64_t)id * (ps / B) + r0 / B) * c.Hkv + h;
    const int64_t stride = is_v ? v_stride : k_stride;
    const T *x = (is_v ? v : k) + ((int64_t)i * D + (lo - first)) * stride + h * c.Dh;
    const int per = c.Dh / 8, n = (hi - lo) * per;  // eights of a row, and of the new rows
    constexpr int kKeep = 4;                        // a lane's first eights stay in registers
    Eight<T> keep[kKeep];
    uint32_t most = 0;
#pragma unroll
    for (int q = 0; q < kKeep; ++q) {
        const int e = lane + 32 * q;
        if (e < n) keep[q].load(x + (int64_t)(e / per) * stride + e % per * 8);
    }
    const uint32_t was = lo > b0 ? scale_bits(gld(scale)) : 0u;
#pragma unroll
    for (int q = 0; q < kKeep; ++q)
        if (lane + 32 * q < n) most = max(most, keep[q].most());
    for (int e = lane + 32 * kKeep; e < n; e += 32) {
        Eight<T> u;
        u.load(x + (int64_t)(e / per) * stride + e % per * 8);
        most = max(most, u.most());
    }
    const uint32_t need = scale_for(__reduce_max_sync(~0u, most));
    const uint32_t now = max(need, was);
    if (lane == 0) gst(scale, now);
    const float inverse = __uint_as_float(inverse_bits(now));
    unsigned char *to = codes + (lo - b0) * width;
#pragma unroll
    for (int q = 0; q < kKeep; ++q) {
        const int e = lane + 32 * q;
        if (e < n)
            gst(reinterpret_cast<uint2 *>(to + (e / per) * width + e % per * 8),
                keep[q].codes(inverse));
    }
    for (int e = lane + 32 * kKeep; e < n; e += 32) {
        Eight<T> u;
        u.load(x + (int64_t)(e / per) * stride + e % per * 8);
        gst(reinterpret_cast<uint2 *>(to + (e / per) * width + e % per * 8), u.codes(inverse));
    }
    if (lo == b0 || now == was) return;
    const float step = __uint_as_float(was) * inverse;  // 2^-184 at least: exact or zero
    for (int e = lane; e < (int)(lo - b0) * per; e += 32) {
        uint2 *p = reinterpret_cast<uint2 *>(codes + (e / per) * width + e % per * 8);
        const uint2 w = gld(p);
        uint32_t out[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint32_t two = q ? w.y : w.x;
            const uint32_t a = e4m3x2_f16x2(two), z = e4m3x2_f16x2_hi(two);
            out[q] = f32_e4m3x2(f16_lo(a) * step, f16_hi(a) * step) |
                     f32_e4m3x2(f16_lo(z) * step, f16_hi(z) * step) << 16;
        }
        gst(p, make_uint2(out[0], out[1]));
    }
}

// Rows cu[i] .. cu[i + 1] - 1 are sequence i's tokens from starts[i] on. A tile's rows find
// their pages first, then all threads stream 16 codes at a time.
template <typename T>
__global__ void __launch_bounds__(kReadThreads)
    k_read8(PageTable pt, const int32_t *__restrict__ slots, const int32_t *__restrict__ cu,
            const int32_t *__restrict__ starts, int N, int64_t rows, Cache8 c, T *__restrict__ k,
            T *__restrict__ v) {
    __shared__ int64_t s_row[kReadRows];    // row of the pools, or -1
    __shared__ int64_t s_block[kReadRows];  // its block
    __shared__ int s_bad;
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    if (tid == 0) s_bad = 0;
    __syncthreads();
    for (int i = tid; i <= N; i += kReadThreads) {
        const int at = gld(cu + i), before = i > 0 ? gld(cu + i - 1) : 0;
        if (at < before || (i == 0 && at != 0) || (i == N && at != rows)) s_bad = 1;
    }
    __syncthreads();
    if (s_bad) {
        if (tid == 0 && blockIdx.x == 0) raise_error(SC_DEV_BAD_SEQLENS);
        return;
    }
    const int per = c.Hkv * c.Dh / 16, ps = pt.page_size, blocks = ps / c.block;
    for (int64_t r0 = (int64_t)blockIdx.x * kReadRows; r0 < rows;
         r0 += (int64_t)gridDim.x * kReadRows) {
        const int here = (int)min((int64_t)kReadRows, rows - r0);
        __syncthreads();
        if (tid < here) {
            const int r = (int)r0 + tid;
            int i = 0, top = N;  // the last i with cu[i] <= r
            while (top - i > 1) {
                const int mid = (i + top) >> 1;
                if (gld(cu + mid) <= r) i = mid;
                else top = mid;
            }
            const int slot = gld(slots + i), begin = gld(cu + i), end = gld(cu + i + 1);
            const int len = slot_length(pt, slot, true);
            const int start = starts != nullptr ? gld(starts + i) : 0;
            int64_t at = -1, block = 0;
            if (len >= 0 && (start < 0 || (int64_t)start + end - begin > len)) {
                raise_error(SC_DEV_BAD_LENGTH);
            } else if (len >= 0) {
                const int pos = start + (r - begin);
                const int id = gld(pt.table + (int64_t)slot * pt.max_pages + pos / ps);
                if (id < 0 || id >= pt.n_pages) {
                    raise_error(SC_DEV_BAD_PAGE);
                } else {
                    at = (int64_t)id * ps + pos % ps;
                    block = (int64_t)id * blocks + pos % ps / c.block;
                }
            }
            s_row[tid] = at;
            s_block[tid] = block;
        }
        __syncthreads();
        for (int x = tid; x < here * 2 * per; x += kReadThreads) {
            const int r = x / (2 * per), y = x - r * 2 * per;
            const bool is_v = y >= per;
            const int q = is_v ? y - per : y, h = q * 16 / c.Dh;
            const int64_t at = s_row[r];
            if (at < 0) continue;
            const uint4 w = ld_plain((const uint4 *)(is_v ? c.v : c.k) + at * per + q);
            const float s = __uint_as_float(scale_bits(
                gld(reinterpret_cast<const uint32_t *>(is_v ? c.v_scales : c.k_scales) +
                    s_block[r] * c.Hkv + h)));
            T *to = (is_v ? v : k) + ((r0 + r) * per + q) * 16;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float f[kCh];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t four = e ? (u ? w.w : w.z) : (u ? w.y : w.x);
                    const uint32_t a = e4m3x2_f16x2(four), z = e4m3x2_f16x2_hi(four);
                    f[4 * u] = f16_lo(a) * s;
                    f[4 * u + 1] = f16_hi(a) * s;
                    f[4 * u + 2] = f16_lo(z) * s;
                    f[4 * u + 3] = f16_hi(z) * s;
                }
                store_row<T>(to + e * kCh, f);
            }
        }
    }
}

// ------------------------------------------------------------ host side

template <typename T>
static cudaError_t append8(const PageTable &pt, const void *k, int64_t k_stride, const void *v,
                           int64_t v_stride, const int32_t *slots, int N, int D, const Cache8 &c,
                           cudaStream_t stream) {
    const int nb = (int)(((int64_t)D + 2 * c.block - 2) / c.block);  // blocks that D tokens meet at most
    const int64_t threads = (int64_t)N * nb * 2 * c.Hkv * 32;
    return launch_pdl(k_append8<T>, dim3((unsigned)((threads + kAppendThreads - 1) / kAppendThreads)),
                      dim3(kAppendThreads), 0, stream, pt, (const T *)k, k_stride, (const T *)v,
                      v_stride, slots, N, D, nb, c);
}

cudaError_t launch_append8(int dtype, const PageTable &pt, const void *k, int64_t k_stride,
                           const void *v, int64_t v_stride, const int32_t *slots, int N, int D,
                           const Cache8 &c, cudaStream_t stream) {
    return dtype == SC_BF16
               ? append8<__nv_bfloat16>(pt, k, k_stride, v, v_stride, slots, N, D, c, stream)
               : append8<float>(pt, k, k_stride, v, v_stride, slots, N, D, c, stream);
}

cudaError_t launch_read8(int dtype, const PageTable &pt, const int32_t *slots, const int32_t *cu,
                         const int32_t *starts, int N, int64_t rows, const Cache8 &c, void *k,
                         void *v, int sm_count, cudaStream_t stream) {
    const int64_t tiles = (rows + kReadRows - 1) / kReadRows, most = 8ll * sm_count;
    const dim3 grid((unsigned)(tiles < 1 ? 1 : tiles < most ? tiles : most));
    if (dtype == SC_BF16)
        return launch_pdl(k_read8<__nv_bfloat16>, grid, dim3(kReadThreads), 0, stream, pt, slots,
                          cu, starts, N, rows, c, (__nv_bfloat16 *)k, (__nv_bfloat16 *)v);
    return launch_pdl(k_read8<float>, grid, dim3(kReadThreads), 0, stream, pt, slots, cu, starts, N,
                      rows, c, (float *)k, (float *)v);
}

cudaError_t take_error_cache8(cudaStream_t stream, unsigned int *sum) {
    return take_error_here(stream, sum);
}

#ifdef SC_BOUNDS_CHECK
cudaError_t bounds_install_cache8(const BoundsRegion *r, int n, cudaStream_t stream) {
    return bounds_install_here(r, n, stream);
}
cudaError_t bounds_take_cache8(cudaStream_t stream, unsigned long long *addr) {
    return bounds_take_first_bad_here(stream, addr);
}
#endif

}  // namespace sc
