// cache8.cu -- the 8-bit paged cache: the quantising append, and reading back.
//
// A block is B tokens of a page under one kv head. Its scale s is the least power of two
// with which all that was written to it fits (|x| <= 448 s), a token's code e4m3(x / s). An
// append that needs a larger scale in a block that holds earlier tokens moves
// those tokens' codes to it.
#include <cuda_bf16.h>

#include <limits.h>

#include "common.cuh"
#include "e4m3.cuh"
#include "errors.cuh"
#include "kernels.h"
#include "launch.h"
#include "shortconv.h"
#include "work_split.h"

namespace sc {

constexpr int kAppendThreads = 128;
// CTAs of an SM: with 6, 7, 8 and 9 (which spills) k_append8's prompt below takes 13.2, 11.0, 11.9, 13.6 us.
constexpr int kAppendCtas = 7;
constexpr int kReadThreads = 256;

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

// Eight values of a row.
template <typename T>
struct Eight {
    Row<T> r;
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < Dt<T>::Q; ++i) r.q[i] = ld_plain(reinterpret_cast<const uint4 *>(p) + i);
    }
    // The largest magnitude's bits, of bf16 in both halves of a word, without NaN (that maximum
    // gives the other operand).
    __device__ __forceinline__ uint32_t most(uint32_t m) const {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(r.q);
#pragma unroll
        for (int e = 0; e < 4 * Dt<T>::Q; ++e) {
            if constexpr (sizeof(T) == 2)
                asm("{\n\t.reg .b32 a;\n\t"
                    "abs.bf16x2 a, %1;\n\t"
                    "max.bf16x2 %0, %0, a;\n\t}"
                    : "+r"(m)
                    : "r"(w[e]));
            else
                m = __float_as_uint(fmaxf(__uint_as_float(m), fabsf(__uint_as_float(w[e]))));
        }
        return m;
    }
    // The same without them, as fp32 bits.
    __device__ __forceinline__ uint32_t most_finite(uint32_t m) const {
        float f[kCh];
        Dt<T>::unpack(r.q, f);
#pragma unroll
        for (int e = 0; e < kCh; ++e) {
            const uint32_t b = __float_as_uint(f[e]) & 0x7FFFFFFFu;
            m = max(m, b < 0x7F800000u ? b : 0u);
        }
        return m;
    }
    // `inverse`: of the scale, a power of two, so that a bf16 product is exact too (or so small that
    // its code is 0).
    __device__ __forceinline__ uint2 codes(float inverse) const {
        uint32_t w[4];
        const uint32_t both = __float_as_uint(inverse) | __float_as_uint(inverse) >> 16;
        const uint32_t *u = reinterpret_cast<const uint32_t *>(r.q);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (sizeof(T) == 2) {
                const uint32_t x = bf2_mul(u[e], both);
                w[e] = f32_e4m3x2(bf16_lo(x), bf16_hi(x));
            } else {
                w[e] = f32_e4m3x2(__uint_as_float(u[2 * e]) * inverse,
                                  __uint_as_float(u[2 * e + 1]) * inverse);
            }
        }
        return make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410));
    }
};

// A lane's places among a block's rows of `per` eights: lane, lane + 32, ... EVEN: `per` divides
// 32, so that a lane keeps its column.
template <bool EVEN>
struct Places {
    int per, row, col, drow, dcol;
    __device__ __forceinline__ Places(int per_, int lane) : per(per_) {
        row = lane / per;
        col = lane - row * per;
        drow = 32 / per;
        dcol = 32 - drow * per;
    }
    __device__ __forceinline__ void next() {
        row += drow;
        if (EVEN) return;
        col += dcol;
        if (col >= per) {
            col -= per;
            ++row;
        }
    }
};

// A warp takes one block of K or V: it finds the new tokens' largest magnitude, moves the
// earlier codes where the scale rises, and writes the new ones. The block's values stay in registers
// between the two passes over them, so that they are read once.
// 16391 bf16 tokens of 8 x 64 in blocks of 32 (50 MB read and written): 11.0 us in a graph, 4.6 TB/s of
// the 6.75 that a copy reaches; of 8 x 128 in blocks of 16, 18.1 us, 5.6 TB/s. A wave of 28 warps an
// SM loads, works and stores as one, and the last of two is not full. CTAs of 256 threads give 12.9 and
// 22 (24 warps an SM). One token a sequence is latency: 2.7 us for 64 of them.
template <typename T, bool EVEN>
__global__ void __launch_bounds__(kAppendThreads, kAppendCtas)
    k_append8(PageTable pt, const T *__restrict__ k, int64_t k_stride, const T *__restrict__ v,
              int64_t v_stride, const int32_t *__restrict__ slots, int N, int D, int nb,
              Cache8 c) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    // The call's units are below 2^29.
    const uint32_t unit = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    const uint32_t rest = unit / (uint32_t)c.Hkv, pair = rest >> 1;
    const int h = (int)(unit - rest * c.Hkv), i = (int)(pair / (uint32_t)nb);
    const int b = (int)(pair - (uint32_t)i * nb);
    const bool is_v = rest & 1;
    if (i >= N) return;
    const int slot = gld(slots + i);
    const int len = slot_length(pt, slot, lane == 0);
    if (len < 0) return;
    const int first = len - D;  // position of the first new token
    if (first < 0 && lane == 0) raise_error(SC_DEV_BAD_LENGTH);
    const int lb = c.block_log2, lp = __ffs(pt.page_size) - 1, from = max(first, 0);
    const int64_t b0 = ((int64_t)(from >> lb) + b) << lb;
    if (b0 >= len) return;
    const int lo = max((int)b0, from), hi = (int)min(b0 + (1 << lb), (int64_t)len);
    const int id = gld(pt.table + (int64_t)slot * pt.max_pages + ((int)b0 >> lp));
    const int64_t stride = is_v ? v_stride : k_stride;
    const T *x = (is_v ? v : k) + ((int64_t)i * D + (lo - first)) * stride + h * c.Dh;
    const int n = hi - lo;  // new rows
    constexpr int kKeep = sizeof(T) == 2 ? 8 : 4;  // a lane's first eights stay in registers
    Eight<T> keep[kKeep];
    const Places<EVEN> begin(c.Dh / 8, lane);
    // Places past the new rows repeat the last one's values, which changes no maximum: the kept
    // ones need no branches, four at a time.
    const bool many = n * begin.per > 128;
    {
        Places<EVEN> p = begin;
#pragma unroll
        for (int q = 0; q < kKeep; ++q, p.next()) {
            if (q == 4 && !many) break;
            keep[q].load(x + min(p.row, n - 1) * stride + p.col * 8);
        }
    }
    if (id < 0 || id >= pt.n_pages) {
        if (lane == 0) raise_error(SC_DEV_BAD_PAGE);
        return;
    }
    const int r0 = (int)b0 & (pt.page_size - 1);
    const int64_t width = (int64_t)c.Hkv * c.Dh;
    unsigned char *codes = (unsigned char *)(is_v ? c.v : c.k) +
                           (((int64_t)id << lp) + r0) * width + h * c.Dh;  // of the block's first token
    uint32_t *scale = reinterpret_cast<uint32_t *>(is_v ? c.v_scales : c.k_scales) +
                      (((int64_t)id << (lp - lb)) + (r0 >> lb)) * c.Hkv + h;
    // Every eight of the block, the kept ones first: f(eight, row, column).
    auto each = [&](auto &&f) {
        Places<EVEN> p = begin;
#pragma unroll
        for (int q = 0; q < kKeep; ++q, p.next()) {
            if (q == 4 && !many) return;
            f(keep[q], p.row, p.col);
        }
        for (; p.row < n; p.next()) {
            Eight<T> u;
            u.load(x + p.row * stride + p.col * 8);
            f(u, p.row, p.col);
        }
    };
    const uint32_t was = lo > b0 ? scale_bits(gld(scale)) : 0u;
    uint32_t most = 0;
    each([&](const Eight<T> &u, int, int) { most = u.most(most); });
    if (sizeof(T) == 2) most = max(most & 0xFFFF0000u, most << 16);
    most = __reduce_max_sync(~0u, most);
    if (most >= 0x7F800000u) {
        most = 0;
        each([&](const Eight<T> &u, int, int) { most = u.most_finite(most); });
        most = __reduce_max_sync(~0u, most);
    }
    const uint32_t now = max(scale_for(most), was);
    if (lane == 0) gst(scale, now);
    const float inverse = __uint_as_float(inverse_bits(now));
    unsigned char *to = codes + (lo - b0) * width;
    each([&](const Eight<T> &u, int row, int col) {
        const uint2 w = u.codes(inverse);
        if (row < n) gst(reinterpret_cast<uint2 *>(to + row * width + col * 8), w);
    });
    if (lo == b0 || now == was) return;
    const float step = __uint_as_float(was) * inverse;  // 2^-184 at least: exact or zero
    for (Places<EVEN> p = begin; p.row < (int)(lo - b0); p.next()) {
        uint2 *q = reinterpret_cast<uint2 *>(codes + p.row * width + p.col * 8);
        const uint2 w = gld(q);
        uint32_t out[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t four = e ? w.y : w.x;
            const uint32_t a = e4m3x2_f16x2(four), z = e4m3x2_f16x2_hi(four);
            out[e] = f32_e4m3x2(f16_lo(a) * step, f16_hi(a) * step) |
                     f32_e4m3x2(f16_lo(z) * step, f16_hi(z) * step) << 16;
        }
        gst(q, make_uint2(out[0], out[1]));
    }
}

// A word of codes is what becomes 16 bytes of values: 8 codes in bf16, 4 in fp32.
template <typename T>
struct Codes;
template <>
struct Codes<__nv_bfloat16> {
    static constexpr int kN = 8;
    typedef uint2 Word;
    static __device__ __forceinline__ uint4 values(uint2 w, uint32_t scale) {
        return e4m3_bf16x8(w, scale);
    }
};
template <>
struct Codes<float> {
    static constexpr int kN = 4;
    typedef uint32_t Word;
    static __device__ __forceinline__ uint4 values(uint32_t w, uint32_t scale) {
        const float s = __uint_as_float(scale);
        const uint32_t a = e4m3x2_f16x2(w), z = e4m3x2_f16x2_hi(w);
        return make_uint4(__float_as_uint(f16_lo(a) * s), __float_as_uint(f16_hi(a) * s),
                          __float_as_uint(f16_lo(z) * s), __float_as_uint(f16_hi(z) * s));
    }
};

// Rows cu[i] .. cu[i + 1] - 1 are sequence i's tokens from starts[i] on. A warp takes units of R
// rows of both pools; its lanes find the places of its next 32 rows (a chain of dependent
// reads) at once. Bound by DRAM: 16 sequences of 2001-9000 tokens of 8 x 64 from somewhere inside on, to
// bf16 (203 MB read and written): 35.4 us, 5.7 TB/s of 6.75. With the places found one row after the
// other it was 49.6.
template <typename T>
__global__ void __launch_bounds__(kReadThreads, 4)
    k_read8(PageTable pt, const int32_t *__restrict__ slots, const int32_t *__restrict__ cu,
            const int32_t *__restrict__ starts, int N, int rows, int R, uint32_t head_magic,
            Cache8 c, T *__restrict__ k, T *__restrict__ v) {
    typedef typename Codes<T>::Word Word;
    constexpr int kN = Codes<T>::kN;
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31;
    bool bad = false;
    for (int i = tid; i <= N; i += kReadThreads) {
        const int at = gld(cu + i), before = i > 0 ? gld(cu + i - 1) : 0;
        bad |= at < before || (i == 0 && at != 0) || (i == N && at != rows);
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0 && blockIdx.x == 0) raise_error(SC_DEV_BAD_SEQLENS);
        return;
    }
    const int per = c.Hkv * c.Dh / kN;  // words of a row
    const int lb = c.block_log2, lp = __ffs(pt.page_size) - 1;
    const int64_t step = (int64_t)gridDim.x * (kReadThreads / 32) * R;
    // The row of the pools of row r, -1 for one that is left alone.
    auto find = [&](int64_t r64) {
        if (r64 >= rows) return -1;
        const int r = (int)r64;
        int i = 0, top = N;  // the last i with cu[i] <= r
        while (top - i > 1) {
            const int mid = (i + top) >> 1;
            if (gld(cu + mid) <= r) i = mid;
            else top = mid;
        }
        const int slot = gld(slots + i), begin = gld(cu + i), end = gld(cu + i + 1);
        const int start = starts != nullptr ? gld(starts + i) : 0;
        const int len = slot_length(pt, slot, true);
        if (len < 0) return -1;
        if (start < 0 || (int64_t)start + end - begin > len) {
            raise_error(SC_DEV_BAD_LENGTH);
            return -1;
        }
        const int pos = start + (r - begin);
        const int id = gld(pt.table + (int64_t)slot * pt.max_pages + (pos >> lp));
        if (id < 0 || id >= pt.n_pages) {
            raise_error(SC_DEV_BAD_PAGE);
            return -1;
        }
        return (id << lp) + (pos & (pt.page_size - 1));  // n_pages * page_size < 2^31
    };
    // A unit's words of each pool go by in rounds of 64, two a lane; several rows make one round.
    const int ahead = 32 / R;  // units whose places the lanes hold: lane u R + r unit u's row r
    const int rounds = (R * per + 63) / 64;
    int w_row[2], w_x[2];  // the lane's words in round 0
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int w = 32 * q + lane;
        w_row[q] = R == 1 ? 0 : w / per;
        w_x[q] = w - w_row[q] * per;
    }
    int64_t r0 = ((int64_t)blockIdx.x * (kReadThreads / 32) + (tid >> 5)) * R;
    int place = -1, unit = ahead, round = 0;
    struct Batch {
        Word k[2], v[2];
        uint32_t ks[2], vs[2];
        int64_t to[2];  // word of the outputs, -1: none
    };
    auto load = [&](Batch &b) {
        if (round == 0 && unit == ahead) {
            unit = 0;
            place = lane < ahead * R ? find(r0 + lane / R * step + lane % R) : -1;
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int x = w_x[q] + 64 * round;
            const int row = __shfl_sync(~0u, place, unit * R + w_row[q] & 31);
            b.to[q] = -1;
            if (x >= per || w_row[q] >= R || row < 0) continue;
            const int64_t at = (int64_t)row * per + x;
            const int64_t scale =
                (int64_t)(row >> lb) * c.Hkv + __umulhi((uint32_t)x, head_magic);
            b.k[q] = gld((const Word *)c.k + at);
            b.v[q] = gld((const Word *)c.v + at);
            b.ks[q] = gld(reinterpret_cast<const uint32_t *>(c.k_scales) + scale);
            b.vs[q] = gld(reinterpret_cast<const uint32_t *>(c.v_scales) + scale);
            b.to[q] = (r0 + w_row[q]) * per + x;
        }
        if (++round == rounds) {
            round = 0;
            ++unit;
            r0 += step;
        }
    };
    auto put = [&](const Batch &b) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            if (b.to[q] < 0) continue;
            st_stream(k + b.to[q] * kN, Codes<T>::values(b.k[q], scale_bits(b.ks[q])));
            st_stream(v + b.to[q] * kN, Codes<T>::values(b.v[q], scale_bits(b.vs[q])));
        }
    };
    // One batch is on its way while the one before becomes values.
    Batch even, odd;
    if (r0 >= rows) return;
    load(even);
    while (true) {
        const bool more = r0 < rows;
        if (more) load(odd);
        put(even);
        if (!more) return;
        const bool more2 = r0 < rows;
        if (more2) load(even);
        put(odd);
        if (!more2) return;
    }
}

// ------------------------------------------------------------ host side

template <typename T>
static cudaError_t append8(const PageTable &pt, const void *k, int64_t k_stride, const void *v,
                           int64_t v_stride, const int32_t *slots, int N, int D, const Cache8 &c,
                           cudaStream_t stream) {
    // Blocks that D tokens meet at most.
    const int nb = (int)(((int64_t)D + 2 * (1 << c.block_log2) - 2) >> c.block_log2);
    const int64_t threads = (int64_t)N * nb * 2 * c.Hkv * 32;
    const auto kernel = 256 % c.Dh == 0 ? k_append8<T, true> : k_append8<T, false>;
    return launch_pdl(kernel, dim3((unsigned)((threads + kAppendThreads - 1) / kAppendThreads)),
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

template <typename T>
static cudaError_t read8(const PageTable &pt, const int32_t *slots, const int32_t *cu,
                         const int32_t *starts, int N, int rows, const Cache8 &c, void *k, void *v,
                         int sm_count, cudaStream_t stream) {
    // A warp's rows: up to 64 words of each pool at once, two a lane.
    const int per = c.Hkv * c.Dh / Codes<T>::kN, of_head = c.Dh / Codes<T>::kN;
    const int R = per >= 64 ? 1 : 64 / per < 32 ? 64 / per : 32;
    const uint32_t magic = (uint32_t)((1ull << 32) / of_head) + 1;  // words below 2^22, Dh <= 1024
    const int64_t blocks = row_groups(row_groups(rows, R), kReadThreads / 32);
    const int64_t most = 4ll * sm_count;
    return launch_pdl(k_read8<T>, dim3((unsigned)(blocks < 1 ? 1 : blocks < most ? blocks : most)),
                      dim3(kReadThreads), 0, stream, pt, slots, cu, starts, N, rows, R, magic, c,
                      (T *)k, (T *)v);
}

cudaError_t launch_read8(int dtype, const PageTable &pt, const int32_t *slots, const int32_t *cu,
                         const int32_t *starts, int N, int64_t rows, const Cache8 &c, void *k,
                         void *v, int sm_count, cudaStream_t stream) {
    return dtype == SC_BF16 ? read8<__nv_bfloat16>(pt, slots, cu, starts, N, (int)rows, c, k, v,
                                                   sm_count, stream)
                            : read8<float>(pt, slots, cu, starts, N, (int)rows, c, k, v, sm_count,
                                           stream);
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
