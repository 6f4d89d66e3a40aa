// attention_8bit.cuh -- what attention.cu's k_own does with tiles of an 8-bit cache, and the
// unpacking of a shared prefix.
//
// A key is ks k', a value vs v' (codes k', v' of e4m3, powers of two ks, vs of the block and
// head). The codes go to the tensor cores as f16, which holds them exactly, one conversion a pair;
// Q goes there as f16 too, times a power of two that takes its row's largest to 2^14
// (11 bits of f16 hold bf16's 8). The scales stay out of the products: with s_t a row's score in
// units of log2,
//   out = sum_t 2^(s_t + log2 vs_t - m) v'_t / sum_t 2^(s_t + log2 vs_t - m) / vs_t,
// so that the weights that meet v' are at most 1 (2^8 with the lazy maximum), whatever the
// sizes of the blocks' values, and are rounded to f16's 11 bits. m is the running
// maximum of s_t + log2 vs_t.
#pragma once

namespace sc {

// The scales of a tile's G groups of 8 keys, K's and V's: the aligned 16 bytes of the
// scale array that hold each, and which of the four it is.
template <int G>
struct TileScales8 {
    uint4 four[2][G];
    int at[2][G];
};

// The producer warp's part: lane k starts group k's copy. `id`: lane b's page of box b (of
// `box` keys, `boxes` of them there) of the tile that begins at key `key0` of the sequence. Copies
// go to L2 (.cg), as the other reads of a kernel that may start beside another.
template <int G>
__device__ __forceinline__ void copy_tile_scales(const AttnArgs &a, TileScales8<G> &s, int id,
                                                 int key0, int box, int boxes, int h) {
    const int lane = threadIdx.x & 31, which = lane / G & 1, g = lane % G;
    const int page = __shfl_sync(~0u, id, g * 8 / box);
    if (lane >= 2 * G) return;
    int at = 0;
    if (g * 8 / box < boxes) {
        const int bl = a.s8.block_log2, per_page = a.pt.page_size >> bl;
        const int64_t total = (int64_t)a.pt.n_pages * per_page * a.Hkv;
        const int64_t i =
            ((int64_t)page * per_page + (((key0 + g * 8) & (a.pt.page_size - 1)) >> bl)) * a.Hkv + h;
        const int64_t first = i & ~(int64_t)3;
        const uint32_t bytes = (uint32_t)min((int64_t)16, (total - first) * 4);
        const float *from = (which ? a.s8.v : a.s8.k) + first;
        at = (int)(i - first);
        if (SC_RD_OK(from, bytes))
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                             smem_addr(&s.four[which][g])),
                         "l"(from), "r"(bytes));
    }
    s.at[which][g] = at;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// d += a b for a 16 x 8 x 16 f16 product, fp32 accumulators.
__device__ __forceinline__ void mma16816_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                             uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t word_of(const uint4 &v, int e) {
    return e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w;
}

// A tile row of DH bytes has its 16-byte chunks swizzled as a TMA box of 64-byte (DH 64) or
// 128-byte rows lays them out.
template <int DH>
__device__ __forceinline__ uint32_t swz8(int row, int chunk) {
    return (uint32_t)(row * DH + ((chunk ^ (DH == 64 ? row >> 1 & 3 : row & 7)) << 4));
}

// The column order of the first product is free as long as Q and K agree: lane c of a row's four
// takes the columns 16 c .. 16 c + 15 (of each 64), four a step, which K's row holds as
// one 16-byte chunk. unit[p]: what a product of row p stands for, times scale_log2.
template <int DH>
__device__ __forceinline__ void load_queries8(uint32_t (&qf)[DH / 16][4], float (&unit)[2],
                                              const unsigned char *q, uint32_t block, int row0,
                                              float scale_log2) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        uint4 v[DH / 32];
        uint32_t most = 0;
#pragma unroll
        for (int b = 0; b < DH / 32; ++b) {
            v[b] = *reinterpret_cast<const uint4 *>(q + (b >> 1) * block +
                                                    swz(row0 + 8 * p + g, 2 * c + (b & 1)));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t w = word_of(v[b], e);
                most = max(most, max(w & 0x7FFFu, w >> 16 & 0x7FFFu));
            }
        }
        most = max(most, __shfl_xor_sync(~0u, most, 1));
        most = max(most, __shfl_xor_sync(~0u, most, 2));
        const uint32_t e = max(most >> 7, 32u);  // the largest's exponent, biased by 127
        const float to = __uint_as_float((268 - e) << 23);  // 2^(14 - (e - 127))
        unit[p] = __uint_as_float((e - 14) << 23) * scale_log2;
#pragma unroll
        for (int b = 0; b < DH / 32; ++b)
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const uint32_t two = word_of(v[b], w);
                qf[b * 2 + w / 2][w % 2 * 2 + p] = pack_f16(bf16_lo(two) * to, bf16_hi(two) * to);
            }
    }
}

// o += P V over a warp's 16 KB keys, of each row only the keys it sees; as tile8 lays P and o out.
template <int DH, int KB>
__device__ __forceinline__ void product_one_by_one8(float (&o)[DH / 8][4],
                                                    const uint32_t (&pf)[KB][4],
                                                    const unsigned char *v, int row0, int key0,
                                                    const int (&see)[2]) {
    const int lane = threadIdx.x & 31, c = lane & 3;
    constexpr int W = DH / 8;
#pragma unroll 1
    for (int k = 0; k < 16 * KB; ++k) {
        uint32_t w2[2] = {0, 0};
#pragma unroll
        for (int nt = 0; nt < 2 * KB; ++nt)
            if (nt == k >> 3) {
                w2[0] = pf[nt / 2][nt % 2 * 2];
                w2[1] = pf[nt / 2][nt % 2 * 2 + 1];
            }
        float w[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const uint32_t x = __shfl_sync(~0u, w2[p], (lane & ~3) | (k & 7) >> 1);
            w[p] = k & 1 ? f16_hi(x) : f16_lo(x);
        }
#pragma unroll
        for (int b = 0; b < 2 * W / 16; ++b) {  // this lane's 2 W columns
            const uint4 q = *reinterpret_cast<const uint4 *>(
                v + swz8<DH>(row0 + k, c * (2 * W / 16) + b));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t lo = e4m3x2_f16x2(word_of(q, e)), hi = e4m3x2_f16x2_hi(word_of(q, e));
                const float x[4] = {f16_lo(lo), f16_hi(lo), f16_lo(hi), f16_hi(hi)};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int col = b * 16 + e * 4 + u;
#pragma unroll
                    for (int p = 0; p < 2; ++p)
                        if (key0 + k < see[p]) {
                            float &to = o[col % W][2 * p + col / W];
                            to = fmaf(w[p], x[u], to);
                        }
                }
            }
        }
    }
}

// One tile's part of a warp: 16 rows by 16 KB keys from tile row 16 KB kw (key key0) on. The order
// of the output's columns is free too: lane g of the second product's eight takes the DH / 8
// columns from g DH / 8 on, which V's row holds together, step d the d-th of them; o[d][2p + e] is
// then row p's column (2 c + e) DH / 8 + d.
template <int DH, int KB, int G>
__device__ __forceinline__ void tile8(const unsigned char *k, uint32_t v_off,
                                      const TileScales8<G> &scales, int kw, int key0, int len,
                                      int least, const int (&see)[2],
                                      const uint32_t (&qf)[DH / 16][4], const float (&unit)[2],
                                      float (&m)[2], float (&limit)[2], f32x2 (&l2)[2],
                                      float (&o)[DH / 8][4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int row0 = kw * 16 * KB;
    const unsigned char *v = k + v_off;
    float s[2 * KB][4], inverse[2 * KB];
#pragma unroll
    for (int nt = 0; nt < 2 * KB; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = 0.0f;
#pragma unroll
        for (int b = 0; b < DH / 64; ++b) {
            const uint4 w = *reinterpret_cast<const uint4 *>(
                k + (row0 + nt * 8) * DH + swz8<DH>(g, c + 4 * b));
#pragma unroll
            for (int e = 0; e < 4; ++e)
                mma16816_f16(s[nt], qf[b * 4 + e], e4m3x2_f16x2(word_of(w, e)),
                             e4m3x2_f16x2_hi(word_of(w, e)));
        }
    }
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int nt = 0; nt < 2 * KB; ++nt) {
        const int group = 2 * KB * kw + nt;
        const uint32_t kb = scale_bits(
            reinterpret_cast<const uint32_t *>(&scales.four[0][group])[scales.at[0][group]]);
        const uint32_t vb = scale_bits(
            reinterpret_cast<const uint32_t *>(&scales.four[1][group])[scales.at[1][group]]);
        const float add = (float)((int)(vb >> 23) - 127);
        inverse[nt] = __uint_as_float(inverse_bits(vb));
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const float by = unit[p] * __uint_as_float(kb);
            f2_split(f2_fma(f2_make(s[nt][2 * p], s[nt][2 * p + 1]), f2_make(by, by),
                            f2_make(add, add)),
                     s[nt][2 * p], s[nt][2 * p + 1]);
            if (key0 + 16 * KB > least) {  // some row does not see some of these keys
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (key0 + nt * 8 + c * 2 + e >= see[p]) s[nt][2 * p + e] = -INFINITY;
            }
            top[p] = max3(top[p], s[nt][2 * p], s[nt][2 * p + 1]);
        }
    }
    // Only when some score passes its row's limit are the row maxima needed. A row that
    // has seen no key yet keeps m = -inf and sums of zero.
    if (__any_sync(~0u, top[0] > limit[0] || top[1] > limit[1])) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            top[p] = fmaxf(top[p], __shfl_xor_sync(~0u, top[p], 1));
            top[p] = fmaxf(top[p], __shfl_xor_sync(~0u, top[p], 2));
            if (!(top[p] > limit[p])) continue;
            const float f = ex2(m[p] - top[p]);
            m[p] = top[p];
            limit[p] = top[p] + kRescaleLog2;
            l2[p] = f2_mul(l2[p], f2_make(f, f));
#pragma unroll
            for (int d = 0; d < DH / 8; ++d) {
                o[d][2 * p] *= f;
                o[d][2 * p + 1] *= f;
            }
        }
    }
    uint32_t pf[KB][4];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const float off = m[p] == -INFINITY ? 0.0f : -m[p];
        const f32x2 off2 = f2_make(off, off);
#pragma unroll
        for (int nt = 0; nt < 2 * KB; ++nt) {
            float e0, e1;
            f2_split(f2_add(f2_make(s[nt][2 * p], s[nt][2 * p + 1]), off2), e0, e1);
            e0 = ex2(e0);
            e1 = ex2(e1);
            l2[p] = f2_fma(f2_make(e0, e1), f2_make(inverse[nt], inverse[nt]), l2[p]);
            pf[nt / 2][nt % 2 * 2 + p] = pack_f16(e0, e1);  // 2^-11 relative a term at most
        }
    }
    // A draft that some row does not see: were its V NaN, a weight of 0 would not keep it
    // from that row, so the block's product is made one by one.
    if (key0 + 16 * KB > least) {
        bool nan = false;
        const int lo = max(least - key0, 0), hi = min(len - key0, 16 * KB);
        for (int x = lane; x < (hi - lo) * (DH / 16); x += 32) {
            const uint4 w = *reinterpret_cast<const uint4 *>(
                v + (row0 + lo + x / (DH / 16)) * DH + x % (DH / 16) * 16);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                nan |= (((word_of(w, e) & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
        }
        if (__any_sync(~0u, nan)) {
            product_one_by_one8<DH, KB>(o, pf, v, row0, key0, see);
            return;
        }
    }
    constexpr int VW = DH / 32;  // words of DH / 8 codes
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
        uint32_t w[4][VW];  // of the keys 2 c, 2 c + 1, 2 c + 8, 2 c + 9
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int r = 2 * c + (x & 1) + (x & 2) * 4;
            if constexpr (DH == 64) {
                const uint2 u = *reinterpret_cast<const uint2 *>(
                    v + (row0 + kb * 16) * DH + swz8<DH>(r, g >> 1) + (g & 1) * 8);
                w[x][0] = u.x;
                w[x][1] = u.y;
            } else {
                const uint4 u = *reinterpret_cast<const uint4 *>(
                    v + (row0 + kb * 16) * DH + swz8<DH>(r, g));
#pragma unroll
                for (int e = 0; e < VW; ++e) w[x][e] = word_of(u, e);
            }
            // Codes past the sequence may be NaN, which a weight of 0 would not silence.
            if (key0 + 16 * KB > len && key0 + kb * 16 + r >= len)
#pragma unroll
                for (int e = 0; e < VW; ++e) w[x][e] = 0;
        }
#pragma unroll
        for (int e = 0; e < VW; ++e) {
            const uint32_t a0 = __byte_perm(w[0][e], w[1][e], 0x5140);
            const uint32_t a1 = __byte_perm(w[0][e], w[1][e], 0x7362);
            const uint32_t b0 = __byte_perm(w[2][e], w[3][e], 0x5140);
            const uint32_t b1 = __byte_perm(w[2][e], w[3][e], 0x7362);
            mma16816_f16(o[4 * e], pf[kb], e4m3x2_f16x2(a0), e4m3x2_f16x2(b0));
            mma16816_f16(o[4 * e + 1], pf[kb], e4m3x2_f16x2_hi(a0), e4m3x2_f16x2_hi(b0));
            mma16816_f16(o[4 * e + 2], pf[kb], e4m3x2_f16x2(a1), e4m3x2_f16x2(b1));
            mma16816_f16(o[4 * e + 3], pf[kb], e4m3x2_f16x2_hi(a1), e4m3x2_f16x2_hi(b1));
        }
    }
}

// The shared prefix as bf16 [keys, Hkv, Dh], for k_prefix: every key is read by many row tiles, so
// it is unpacked once, and stays in L2. Exact: a code has 4 bits, a scale none.
constexpr int kUnpackThreads = 256;
static __global__ void __launch_bounds__(kUnpackThreads)
    k_unpack(AttnArgs a, const unsigned char *__restrict__ k, const unsigned char *__restrict__ v,
             int Dh, bf16 *__restrict__ k16, bf16 *__restrict__ v16) {
    __shared__ int s_leader;
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    if (tid == 0) s_leader = a.N;
    __syncthreads();
    // The first listed sequence whose rows all see the whole prefix names its pages.
    for (int i = tid; i < a.N; i += kUnpackThreads) {
        int slot;
        if (prefix_keys(a, seq_len(a, i, &slot, false)) > 0) {
            atomicMin(&s_leader, i);
            break;
        }
    }
    __syncthreads();
    if (s_leader >= a.N) return;
    int slot;
    seq_len(a, s_leader, &slot, false);
    const int32_t *row = a.pt.table + (int64_t)slot * a.pt.max_pages;
    const int per = a.Hkv * Dh / 16, ps = a.pt.page_size, bl = a.s8.block_log2;
    const int64_t n = (int64_t)a.shared_keys * 2 * per;
    for (int64_t x = (int64_t)blockIdx.x * kUnpackThreads + tid; x < n;
         x += (int64_t)gridDim.x * kUnpackThreads) {
        const int t = (int)(x / (2 * per)), y = (int)(x - (int64_t)t * 2 * per);
        const bool is_v = y >= per;
        const int q = is_v ? y - per : y, at = t & (ps - 1);
        const int id = gld_l2(row + t / ps);
        if (id < 0 || id >= a.pt.n_pages) continue;  // k_prefix reports it
        const uint4 w = ld_plain((is_v ? v : k) + (((int64_t)id * ps + at) * per + q) * 16);
        const float *scales = is_v ? a.s8.v : a.s8.k;
        const float s = __uint_as_float(scale_bits(__float_as_uint(
            gld(scales + ((int64_t)id * (ps >> bl) + (at >> bl)) * a.Hkv + q * 16 / Dh))));
        bf16 *to = (is_v ? v16 : k16) + ((int64_t)t * per + q) * 16;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t out[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t four = word_of(w, 2 * half + e);
                const uint32_t lo = e4m3x2_f16x2(four), hi = e4m3x2_f16x2_hi(four);
                out[2 * e] = pack_bf16(f16_lo(lo) * s, f16_hi(lo) * s);
                out[2 * e + 1] = pack_bf16(f16_lo(hi) * s, f16_hi(hi) * s);
            }
            st_plain(to + 8 * half, make_uint4(out[0], out[1], out[2], out[3]));
        }
    }
}

// Bytes of the unpacked K, or V.
static size_t unpacked_bytes(const AttnShape &s, int page_size) {
    return (size_t)s.shared_pages * page_size * s.Hkv * s.Dh * 2;
}

static cudaError_t launch_unpack(const AttnArgs &a, const AttnShape &s, const void *k, const void *v,
                                 bf16 *k16, bf16 *v16, int sm_count, cudaStream_t stream) {
    const int64_t n = (int64_t)a.shared_keys * 2 * (s.Hkv * s.Dh / 16);
    const int64_t blocks = (n + kUnpackThreads - 1) / kUnpackThreads, most = 8ll * sm_count;
    return launch_pdl(k_unpack, dim3((unsigned)(blocks < most ? blocks : most)),
                      dim3(kUnpackThreads), 0, stream, a, (const unsigned char *)k,
                      (const unsigned char *)v, s.Dh, k16, v16);
}

}  // namespace sc
