// attention_prefix.cuh -- the shared prefix's part of attention.cu, on the
// tcgen05 tensor cores.
//
// For one kv head the rows of all sequences (N D G of them) are one query matrix against
// one K and V (rows that do not see all of the prefix are computed along; nothing reads them):
// tiles of 128 rows by 128 keys, S = Q K^T and O += P V with accumulators in
// TMEM, P written back to TMEM as the second product's bf16 operand.
//
// A CTA runs two streams of tiles, one warpgroup of softmax threads each
// (thread = row = TMEM lane), so that one stream's exponentials run while the
// tensor cores work for the other:
//   more than 128 rows a head: the streams are two row tiles that share every
//     K and V tile (halves the traffic from L2);
//   at most 128 rows: the same rows on alternate key tiles.
// The streams' tiles are numbered in turn (a0 b0 a1 b1 ..), tile n's S and P in
// TMEM buffer n % kBufs. One thread issues QK(n) once PV(n - kBufs), the buffer's
// last reader, is done; another issues PV(n) once P(n) is there (issuing and
// signalling a tile's two products takes one thread as long as the products).
// With three buffers (Dh = 64) a stream's next S is ready when its softmax ends; with
// Dh = 128 O leaves room for two. O is rescaled only when a row's maximum rose by more
// than 2^8 since the last time: weights then stay below 2^8, exact enough in
// the fp32 sums and bf16's exponent range.
//
// 1024 rows x 32 heads x 16384 keys of 64: 125 us (1.1 PFLOP/s), tensor cores and
// exponential unit 48 % busy each. A tile's softmax bounds it: its maxima take 470
// cycles and its exponentials 850 with both streams at it (1720 a tile and stream in
// all), the products 512 a tile. Measured slower or the same: exponentials computed while
// the maximum is still sought and S read again where it rose (141 us), S read twice
// instead of kept in registers (20 us more), turns at the exponentials (122-124),
// P in columns of its own so that QK waits for no PV (1 to 2 us more), two threads a row (35 more).
#pragma once

namespace sc {

constexpr int kPR = 128;                 // rows of a tile
constexpr int kPK = 128;                 // keys of a tile
constexpr int kPfxThreads = 384;         // 2 x 4 softmax warps; producer, QK, PV, an idle warp

struct PrefixArgs {
    AttnArgs a;
    int P;          // prefix keys
    int tpt;        // tokens of a row tile: 128 / G
    int n_tiles;    // row tiles of a kv head
    int split;      // 1: the two streams take alternate key tiles of one row tile
    int T;          // units of an item: key tiles, or pairs of them with split
    int64_t U;      // units of the call
    int n_cta;
    float *part;    // [2 (items + CTAs)] parts of 128 rows: O [128][Dh], m [128], l [128]
};

template <int DH>
struct PfxCfg {
    static constexpr int NB = DH / 64;
    static constexpr uint32_t kTile = kPK * 128 * NB;  // K, V or Q tile: 16 or 32 KB
    static constexpr uint32_t kBlk = kPK * 128;        // its 64-column block
    static constexpr int kSt = DH == 64 ? 5 : 2;       // tiles of the K and of the V ring
    static constexpr int kBufs = DH == 64 ? 3 : 2;     // S and P buffers of 128 columns
    static constexpr int kOCol = kBufs * kPK;          // O of the streams after them
    static_assert(kOCol + 2 * DH <= 512, "TMEM");
    static constexpr size_t kSmem = 1024 + (size_t)(2 + 2 * kSt) * kTile;
    static constexpr int kSlot = kPR * (DH + 2);
};

// tcgen05 pieces that only this kernel uses.

// True in one lane of the warp. Behind this branch, unlike behind a comparison of
// the lane number, the compiler keeps addresses and descriptors in the uniform
// registers that tcgen05.mma takes: 32 cycles a 128 x 64 x 16 step instead of 45.
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(e));
    return e != 0;
}

// D[tmem] (+)= A[tmem] * B[smem], one 128 x N x 16 step; issued by one thread.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Descriptor of an MN-major 128-byte-swizzled tile (rows = K, 64 contiguous
// MN values a row): 64-wide MN blocks lbo bytes apart, groups of 8 rows 1024.
__device__ __forceinline__ uint64_t sdesc_mn128(uint32_t saddr, uint32_t lbo) {
    uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(lbo >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// 32 columns of this thread's TMEM lane; valid after tmem_ld_wait().
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// After tmem_ld_wait(): no use of r moves above this point.
template <int N>
__device__ __forceinline__ void regs_ready(uint32_t (&r)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// Registers of the calling warpgroup's threads from here on. The launch has
// 384 x 168; 256 x 216 + 128 x 72 is as many. (The checked stores of the
// bounds-checked build call a function, which needs the launch's own split.)
template <int N>
__device__ __forceinline__ void more_regs() {
#ifndef SC_BOUNDS_CHECK
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
#endif
}
template <int N>
__device__ __forceinline__ void fewer_regs() {
#ifndef SC_BOUNDS_CHECK
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
#endif
}

struct RingPos {
    uint32_t i, phase;
    __device__ __forceinline__ void next(uint32_t n) {
        if (++i == n) {
            i = 0;
            phase ^= 1u;
        }
    }
};

struct PfxBars {
    uint64_t kfull[8], kempty[8], vfull[8], vempty[8];
    uint64_t qfull, qempty;
    uint64_t sfull[3], pready[3], pvdone[3];  // of the S and P buffers
    uint64_t odone[2];                        // a stream's last product of an item
    uint64_t done;                            // every MMA of the CTA
    uint32_t tmem;
    int leader;
    volatile int bad;
};

template <int DH>
__global__ void __launch_bounds__(kPfxThreads, 1)
    k_prefix(PrefixArgs x, const __grid_constant__ CUtensorMap mq,
             const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
    using C = PfxCfg<DH>;
    constexpr int ST = C::kSt;
    const AttnArgs &a = x.a;
    extern __shared__ unsigned char raw[];
    __shared__ PfxBars b;
    const uint32_t raw_a = smem_addr(raw);
    unsigned char *base = raw + (((raw_a + 1023u) & ~1023u) - raw_a);
    const uint32_t q_a = smem_addr(base), k_a = q_a + 2 * C::kTile, v_a = k_a + ST * C::kTile;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(&b.kfull[s], 1);
            mbar_init(&b.kempty[s], 1);
            mbar_init(&b.vfull[s], 1);
            mbar_init(&b.vempty[s], 1);
        }
        mbar_init(&b.qfull, 1);
        mbar_init(&b.qempty, 1);
        for (int s = 0; s < 3; ++s) {
            mbar_init(&b.sfull[s], 1);
            mbar_init(&b.pready[s], 4);
            mbar_init(&b.pvdone[s], 1);
        }
        for (int s = 0; s < 2; ++s) mbar_init(&b.odone[s], 1);
        mbar_init(&b.done, 2);
        b.leader = a.N;
        b.bad = 0;
        mbar_fence_init();
    }
    if (warp == 8 && lane == 0) {
        tma_prefetch_map(&mq);
        tma_prefetch_map(&mk);
        tma_prefetch_map(&mv);
    }
    if (warp == 9) tmem_alloc(&b.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = b.tmem;
    pdl_wait();
    pdl_launch_dependents();
    // The first listed sequence whose rows all see the whole prefix names its pages.
    for (int i = tid; i < a.N; i += kPfxThreads) {
        int slot;
        if (prefix_keys(a, seq_len(a, i, &slot, false)) > 0) {
            atomicMin(&b.leader, i);
            break;
        }
    }
    __syncthreads();
    const int leader = b.leader;
    const int64_t u0 = share_begin(blockIdx.x, x.U, x.n_cta);
    const int64_t u1 = leader < a.N ? share_begin(blockIdx.x + 1, x.U, x.n_cta) : u0;
    const int per = x.split ? 2 : 1;  // key tiles of a unit
    // f(head, first row tile, first unit, units, item) for each item piece of the CTA.
    auto walk = [&](auto &&f) {
        for (int64_t u = u0; u < u1;) {
            const int64_t w = u / x.T;
            const int t0 = (int)(u % x.T), n = (int)min((int64_t)(x.T - t0), u1 - u);
            if (!f((int)(w % a.Hkv), (int)(w / a.Hkv) * (x.split ? 1 : 2), t0, n, w)) return;
            u += n;
        }
    };

    if (warp == 11) {
        fewer_regs<72>();
    } else if (warp == 8) {  // --------------------------------------------- producer
        fewer_regs<72>();
        const int ps = a.pt.page_size;
        const int box = min(ps, kPK), nb = kPK / box;
        const int n_box = x.P / box;
        int slot = 0;
        if (u0 < u1) seq_len(a, leader, &slot, false);
        const int32_t *row = a.pt.table + (int64_t)slot * a.pt.max_pages;
        uint32_t gk = 0, gv = 0, items = 0;
        bool ok = true;
        // The prefix's next tile into the ring; the boxes past the prefix's end
        // are not read, and V's rows there are zeroed (their weights are 0).
        auto load = [&](const CUtensorMap *m, uint64_t *full, uint64_t *empty, uint32_t ring,
                        uint32_t &g, PageIds &ids, int h, bool is_v) {
            const uint32_t s = g % ST;
            if (g >= ST && !mbar_wait_bounded(&empty[s], (g / ST - 1) & 1u)) {
                raise_error(SC_DEV_TIMEOUT);
                return ok = false;
            }
            const int boxes = max(0, min(nb, n_box - ids.box()));
            const uint32_t dst = ring + s * C::kTile;
            if (is_v && boxes < nb) {
                unsigned char *at = base + (dst - q_a);
                for (int r = boxes * box * 8 + lane; r < kPK * 8; r += 32)
#pragma unroll
                    for (int c = 0; c < C::NB; ++c)
                        *reinterpret_cast<uint4 *>(at + c * C::kBlk + r * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
            }
            int id = ids.page();
            bool bad = lane < boxes && (id < 0 || id >= a.pt.n_pages);
            if (bad) id = 0;
            bad = __any_sync(~0u, bad);
            if (lane == 0) {
                if (bad) {
                    raise_error(SC_DEV_BAD_PAGE);
                    b.bad = 1;
                }
                mbar_arrive_expect_tx(&full[s], (uint32_t)boxes * box * DH * 2);
            }
            __syncwarp();
            if (lane < boxes) {
                const int key = id * ps + (ids.box() + lane) * box % ps;
#pragma unroll
                for (int c = 0; c < C::NB; ++c)
                    tma_load_3d(dst + c * C::kBlk + lane * box * 128, m, &full[s], c * 64, h, key);
            }
            ++g;
            ids.next(nb);
            return true;
        };
        PageIds kids, vids;
        walk([&](int h, int rt, int t0, int n, int64_t) {
            if (items > 0 && !mbar_wait_bounded(&b.qempty, (items - 1) & 1u)) {
                raise_error(SC_DEV_TIMEOUT);
                return ok = false;
            }
            ++items;
            if (lane == 0) {
                const int tiles = x.split || rt + 1 >= x.n_tiles ? 1 : 2;
                mbar_arrive_expect_tx(&b.qfull, (uint32_t)tiles * x.tpt * a.G * DH * 2);
                for (int s = 0; s < tiles; ++s)
                    for (int c = 0; c < C::NB; ++c)
                        tma_load_4d(q_a + s * C::kTile + c * C::kBlk, &mq, &b.qfull, c * 64, 0, h,
                                    (rt + s) * x.tpt);
            }
            // K runs ahead of V as far as QK runs ahead of PV.
            const int nt = n * per, lead = x.split ? C::kBufs - 1 : 1, b0 = t0 * per * nb;
            kids.start(row, ps / box, b0, n_box - 1);
            vids.start(row, ps / box, b0, n_box - 1);
            for (int t = -lead; t < nt; ++t) {
                if (t + lead < nt &&
                    !load(&mk, b.kfull, b.kempty, k_a, gk, kids, h, false))
                    return false;
                if (t >= 0 && !load(&mv, b.vfull, b.vempty, v_a, gv, vids, h, true))
                    return false;
            }
            return true;
        });
        // No copy and no MMA's arrival may be in flight when the CTA leaves.
        if (items > 0) mbar_wait_bounded(&b.qfull, (items - 1) & 1u);
        for (uint32_t c = gk > ST ? gk - ST : 0; c < gk; ++c)
            mbar_wait_bounded(&b.kfull[c % ST], (c / ST) & 1u);
        for (uint32_t c = gv > ST ? gv - ST : 0; c < gv; ++c)
            mbar_wait_bounded(&b.vfull[c % ST], (c / ST) & 1u);
    } else if (warp == 9 || warp == 10) {  // ------------------------------ MMA issue
        fewer_regs<72>();
        if (elect_one()) {
            constexpr uint32_t idq = idesc_bf16_f32(kPR, kPK);
            constexpr uint32_t idv = idesc_bf16_f32(kPR, DH) | (1u << 16);  // B is MN-major
            RingPos ring = {0, 0}, buf = {0, 0};  // of the K (V) tile and of the S and P buffer
            uint32_t items = 0;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                if (mbar_wait_bounded(bar, parity)) return true;
                raise_error(SC_DEV_TIMEOUT);
                return false;
            };
            if (warp == 9) {
                const uint64_t qd = sdesc_k128(q_a), kd = sdesc_k128(k_a);
                bool fresh = true;  // no buffer has been used yet: nothing to wait for
                walk([&](int h, int rt, int t0, int n, int64_t) {
                    const int streams = x.split || rt + 1 < x.n_tiles ? 2 : 1;
                    const int total = n * streams;
                    if (!wait(&b.qfull, items & 1u)) return false;
                    ++items;
                    for (int m = 0; m < total; ++m) {
                        const int s = m & (streams - 1);
                        if ((s == 0 || x.split) && !wait(&b.kfull[ring.i], ring.phase)) return false;
                        if (!fresh && !wait(&b.pvdone[buf.i], buf.phase ^ 1u)) return false;
                        tc_fence_after();
                        const uint64_t qt = qd + (s && !x.split ? C::kTile >> 4 : 0);
                        const uint64_t kt = kd + ring.i * (C::kTile >> 4);
                        const uint32_t d = tmem + buf.i * kPK;
#pragma unroll
                        for (int j = 0; j < DH / 16; ++j) {
                            const uint32_t off = (j / 4) * (C::kBlk >> 4) + 2 * (j % 4);
                            mma_bf16(d, qt + off, kt + off, idq, j != 0);
                        }
                        mma_commit(&b.sfull[buf.i]);
                        if (s == streams - 1 || x.split) {  // the K tile's last reader
                            mma_commit(&b.kempty[ring.i]);
                            ring.next(ST);
                        }
                        buf.next(C::kBufs);
                        if (buf.i == 0) fresh = false;
                    }
                    mma_commit(&b.qempty);
                    return true;
                });
            } else {
                const uint64_t vd = sdesc_mn128(v_a, C::kBlk);
                walk([&](int h, int rt, int t0, int n, int64_t) {
                    const int streams = x.split || rt + 1 < x.n_tiles ? 2 : 1;
                    const int total = n * streams;
                    for (int m = 0; m < total; ++m) {
                        const int s = m & (streams - 1);
                        if ((s == 0 || x.split) && !wait(&b.vfull[ring.i], ring.phase)) return false;
                        if (!wait(&b.pready[buf.i], buf.phase)) return false;
                        tc_fence_after();
                        const uint64_t vt = vd + ring.i * (C::kTile >> 4);
                        const uint32_t p = tmem + buf.i * kPK, o = tmem + C::kOCol + s * DH;
#pragma unroll
                        for (int j = 0; j < kPK / 16; ++j)
                            mma_bf16_ts(o, p + j * 8, vt + j * (2048 >> 4), idv,
                                        m >= streams || j > 0);
                        mma_commit(&b.pvdone[buf.i]);
                        if (m >= total - streams) mma_commit(&b.odone[s]);
                        if (s == streams - 1 || x.split) {
                            mma_commit(&b.vempty[ring.i]);
                            ring.next(ST);
                        }
                        buf.next(C::kBufs);
                    }
                    return true;
                });
            }
            mma_commit(&b.done);  // no MMA may still write TMEM when it is freed
            mbar_wait_bounded(&b.done, 0);
        }
        __syncwarp();
    } else {  // ------------------------------------------------------------- softmax
        const int s = warp >> 2, r = tid & 127;  // stream, row = TMEM lane
        const uint32_t lane_base = (uint32_t)(warp & 3) << 21;
        const uint32_t ot = tmem + lane_base + C::kOCol + s * DH;
        uint32_t seq = 0;   // tiles of earlier items, both streams
        uint32_t ends = 0;  // items of this stream that ended
        more_regs<216>();
        bool dead = false;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (!dead && !mbar_wait_bounded(bar, parity)) {
                raise_error(SC_DEV_TIMEOUT);
                dead = true;  // no more waits: the rest runs through on what is there
            }
            __syncwarp();
            tc_fence_after();
        };
        walk([&](int h, int rt, int t0, int n, int64_t w) {
            const int tile = x.split ? rt : rt + s;
            const int streams = x.split || rt + 1 < x.n_tiles ? 2 : 1;
            const uint32_t seq0 = seq;
            seq += (uint32_t)n * streams;
            if (tile >= x.n_tiles) return true;  // the second stream has no rows
            float m = -INFINITY, l = 0.0f;
            for (int t = 0; t < n; ++t) {
                const int key0 = ((t0 + t) * per + (x.split ? s : 0)) * kPK;
                const uint32_t at = seq0 + (uint32_t)t * streams + s, buf = at % C::kBufs;
                const uint32_t st = tmem + lane_base + buf * kPK;
                wait(&b.sfull[buf], at / C::kBufs & 1u);
                uint32_t v[kPK];
#pragma unroll
                for (int c = 0; c < kPK / 32; ++c) tmem_ld32(st + c * 32, v + c * 32);
                tmem_ld_wait();
                regs_ready(v);
                if (key0 + kPK > x.P) {
#pragma unroll
                    for (int c = 0; c < kPK; ++c)
                        if (key0 + c >= x.P) v[c] = 0xFF800000u;  // -inf
                }
                float top[4];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    top[c] = max3(__uint_as_float(v[c]), __uint_as_float(v[c + 4]),
                                  __uint_as_float(v[c + 8]));
#pragma unroll
                for (int c = 12; c < kPK; c += 2)
                    top[c / 2 & 3] = max3(top[c / 2 & 3], __uint_as_float(v[c]),
                                          __uint_as_float(v[c + 1]));
                const float now = fmaxf(max3(top[0], top[1], top[2]), top[3]) * a.scale_log2;
                const bool rise = now > m + kRescaleLog2 || m == -INFINITY;
                if (__any_sync(~0u, rise && now > m)) {
                    const float to = rise ? fmaxf(m, now) : m;
                    const float f = to == -INFINITY ? 1.0f : ex2(m - to);
                    m = to;
                    l *= f;
                    if (t > 0) {  // O is at rest after the stream's last product
                        wait(&b.pvdone[(at - streams) % C::kBufs], (at - streams) / C::kBufs & 1u);
#pragma unroll
                        for (int c = 0; c < DH / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(ot + c * 32, o);
                            tmem_ld_wait();
                            regs_ready(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st32(ot + c * 32, o);
                        }
                    }
                }
                const float off = m == -INFINITY ? 0.0f : -m;
                const f32x2 scale2 = f2_make(a.scale_log2, a.scale_log2), off2 = f2_make(off, off);
                f32x2 sum[2] = {0, 0};
#pragma unroll
                for (int c = 0; c < kPK / 2; ++c) {
                    float e0, e1;
                    f2_split(f2_fma(f2_make(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1])),
                                    scale2, off2),
                             e0, e1);
                    e0 = ex2(e0);
                    e1 = ex2(e1);
                    sum[c & 1] = f2_add(sum[c & 1], f2_make(e0, e1));
                    v[c] = pack_bf16(e0, e1);
                }
                float s0, s1;
                f2_split(f2_add(sum[0], sum[1]), s0, s1);
                l += s0 + s1;
                tmem_st32(st, v);
                tmem_st32(st + 32, v + 32);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.pready[buf]);
            }
            // A barrier of the stream's own, which its next item alone completes again. pvdone of the
            // last tile is not enough: when the next item has one stream, that one's tiles take all
            // buffers in turn, and pvdone could pass two phases before a late warp sees its parity.
            wait(&b.odone[s], ends++ & 1u);
            float *part = x.part + ((w + blockIdx.x) * 2 + s) * C::kSlot;
#pragma unroll
            for (int c = 0; c < DH / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(ot + c * 32, o);
                tmem_ld_wait();
                regs_ready(o);
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    gst(reinterpret_cast<uint4 *>(part + r * DH + c * 32 + e),
                        make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]));
            }
            // A NaN maximum marks a part with a bad page: k_merge leaves its rows alone.
            gst(part + kPR * DH + r, b.bad ? __int_as_float(0x7FC00000) : m);
            gst(part + kPR * DH + kPR + r, l);
            tc_fence_before();  // O was read before the next item's first P is announced
            return true;
        });
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace sc
