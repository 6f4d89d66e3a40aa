// attention.cu -- attention of a serving step over the paged cache (bf16).
//
// Row (i, j, hq) is new token j of D of sequence i under query head hq; it
// sees the sequence's first n = len - D + j + 1 keys of kv head hq / G:
//   out = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m),  s_t = scale q.k_t.
// The keys are walked once with a running maximum m and sum l in 32 bits
// (scores in units of log2, so that one exp2 a score is left); parts of a
// row's keys join by (m, l).
//
// k_own: the D G <= 32 rows of one sequence and kv head are too few for a
// full tensor-core tile and the call is bound by the keys' bytes, so the
// rows run on 16-row register MMAs and the work is what streams K and V:
// every CTA takes an equal share of all 64-key tiles of the call (a share may
// end inside a sequence). A producer warp alone reads lengths and tables, keeps a
// ring of tiles in flight, one TMA box a page, and copies each item's queries.
// The four consumer warps take a share of a tile's keys and, with 32 rows, of
// the rows each, and keep their own (m, l, O), joined once an item. Two
// sequences of 30-40 thousand tokens (143 MB): 26 us, 5.4 TB/s, 80 % of the measured copy
// rate. 128 x 8 drafts with 100-1200 own tokens (32 rows an item, 170 MB): 54 us,
// 3.1 TB/s; DRAM gives 245 MB for them and is busy 59 % of the time, issue slots 23 %.
// With D G > 32 the rows go in tiles of 32, and each walks all of the sequence's key tiles.
//
// k_merge joins the parts that CTAs left in the workspace, in a fixed order: 4
// to 6 us of dependent reads with few rows, 17 us for the 32768 rows of 128 x 8 x 32.
#include <cuda.h>
#include <cuda_bf16.h>

#include <limits.h>

#include <atomic>

#include "common.cuh"
#include "errors.cuh"
#include "kernels.h"
#include "launch.h"
#include "shortconv.h"
#include "tcgen05.cuh"
#include "tensor_map.h"
#include "tma.cuh"
#include "work_split.h"

namespace sc {

typedef __nv_bfloat16 bf16;

constexpr int kKT = 64;            // keys of a tile
constexpr int kMaxCtas = 456;      // three CTAs on each of 152 SMs
constexpr int kMaxPrefixCtas = 152;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleLog2 = 8.0f;  // a running maximum moves when a score passes it by 2^8

struct AttnArgs {
    const bf16 *q;
    int64_t q_stride;
    PageTable pt;
    const int32_t *slots;
    int N, D, G, Hkv;
    int shared_keys;   // keys whose part k_prefix computes (see prefix_keys)
    int beside;        // k_own runs beside k_prefix, on the SMs that it leaves
    float scale_log2;  // scale * log2(e)
    bf16 *out;
    int64_t *cum;      // [N + 1] first own tile of each sequence
    float *own_part;   // [items + CTAs] parts of MR rows: O [MR][Dh], m [MR], l [MR]
};

// Slots, lengths and tables are read in L2: k_own beside k_prefix starts without a wait of
// its own, which would also drop what its SM's L1 holds of them from before they changed.
__device__ __forceinline__ int gld_l2(const int32_t *p) {
    if (!SC_RD_OK(p, 4)) return 0;
    return __ldcg(p);
}

// Tokens of sequence i (its D new ones included), or -1 with a bad slot or length.
__device__ __forceinline__ int seq_len(const AttnArgs &a, int i, int *slot, bool report) {
    const int s = gld_l2(a.slots + i);
    *slot = s;
    if (s < 0 || s >= a.pt.n_slots) {
        if (report) raise_error(SC_DEV_BAD_SLOT);
        return -1;
    }
    const int len = gld_l2(a.pt.lens + s);
    if (len < 0 || len > (int64_t)a.pt.max_pages * a.pt.page_size) {
        if (report) raise_error(SC_DEV_BAD_LENGTH);
        return -1;
    }
    return len;
}

// Keys of a sequence of len tokens whose part k_prefix computes: the shared ones when every
// row sees them all, else none (that sequence's part is then its own from key 0 on, and k_prefix
// needs no mask: a weight of 0 would not silence a NaN in a V row that another row sees).
__device__ __forceinline__ int prefix_keys(const AttnArgs &a, int len) {
    return len - a.D + 1 >= a.shared_keys ? a.shared_keys : 0;
}
// Key tiles of a sequence's own part.
__device__ __forceinline__ int own_tiles(const AttnArgs &a, int len) {
    return len > 0 ? (len - prefix_keys(a, len) + kKT - 1) / kKT : 0;
}

// An item piece as the producer describes it to the consumers: tiles t0 .. t0 + n - 1
// of T of row tile rt and kv head h of sequence i (len tokens); w: the item's number.
// n = 0: no more.
struct OwnItem {
    int i, len, rt, h, w, t0, n, T;
};

// Start a 16-byte copy to shared memory; cp_async_arrive arrives on `bar` once, when
// all that this thread started have landed.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    if (!SC_RD_OK(src, 16)) {  // refused: zeros
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(0) : "memory");
        return;
    }
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// A producer warp's page ids: the table entries of `nb` boxes (of `box` tokens,
// nb a divisor of 32) a tile, tile after tile. Lane k holds the page of box b0 + k;
// the next 32 are in flight, so that a tile waits for no table entry.
struct PageIds {
    const int32_t *row;
    int shift, last, b0, at, cur, nxt;  // shift: log2 of the boxes of a page

    // From box b on; boxes past `last_box` repeat it.
    __device__ __forceinline__ void start(const int32_t *table_row, int boxes_of_page, int b,
                                          int last_box) {
        row = table_row;
        shift = 31 - __clz(boxes_of_page);
        last = last_box;
        begin(b, 0, 0, false);
    }
    // Again from box b; with `known`, c and n are what load(b) and load(b + 32) gave.
    __device__ __forceinline__ void begin(int b, int c, int n, bool known) {
        b0 = b;
        at = 0;
        cur = known ? c : load(b0);
        nxt = known ? n : load(b0 + 32);
    }
    __device__ __forceinline__ int load(int b) const {
        return gld_l2(row + (min(b + (int)(threadIdx.x & 31), last) >> shift));
    }
    // The tile's first box, and lane k's page of its k-th box.
    __device__ __forceinline__ int box() const { return b0 + at; }
    __device__ __forceinline__ int page() const {
        return __shfl_sync(~0u, cur, (at + threadIdx.x) & 31);
    }
    __device__ __forceinline__ void next(int nb) {
        at += nb;
        if (at < 32) return;
        at = 0;
        b0 += 32;
        cur = nxt;
        nxt = load(b0 + 32);
    }
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// d += a b for a 16 x 8 x 16 bf16 product, fp32 accumulators.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A tile row of 64 bf16 is 128 bytes with its 16-byte chunks XOR-swizzled by the
// row's low 3 bits, as a 128-byte-swizzled TMA box lays it out.
__device__ __forceinline__ uint32_t swz(int row, int chunk) {
    return (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4));
}

__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}
__device__ __forceinline__ f32x2 f2_add(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Whether some of eight bf16 values is an infinity or NaN.
__device__ __forceinline__ bool not_finite(const uint4 &v) {
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t w = e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w;
        bad |= (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
    }
    return bad;
}

// o += P V over a warp's 16 KB keys from key0 on (rows row0 .. of the swizzled V tile at vb),
// of each row only the keys it sees. P and o are laid out as mma16816's operands.
template <int DH, int KB>
__device__ __forceinline__ void product_one_by_one(float (&o)[DH / 8][4],
                                                   const uint32_t (&pf)[KB][4],
                                                   const unsigned char *vb, uint32_t block,
                                                   int row0, int key0, const int (&see)[2]) {
    const int lane = threadIdx.x & 31;
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
            w[p] = __uint_as_float(k & 1 ? x & 0xFFFF0000u : x << 16);
        }
#pragma unroll
        for (int d = 0; d < DH / 8; ++d) {
            const uint32_t v = *reinterpret_cast<const uint32_t *>(
                vb + (d >> 3) * block + swz(row0 + k, d & 7) + (lane & 3) * 4);
            const float v0 = __uint_as_float(v << 16), v1 = __uint_as_float(v & 0xFFFF0000u);
#pragma unroll
            for (int p = 0; p < 2; ++p)
                if (key0 + k < see[p]) {
                    o[d][2 * p] = fmaf(w[p], v0, o[d][2 * p]);
                    o[d][2 * p + 1] = fmaf(w[p], v1, o[d][2 * p + 1]);
                }
        }
    }
}

// RG groups of 16 rows times KG key groups: a consumer warp takes 16 rows by 64 / KG keys of
// a tile. 16 rows are bound by the tiles' bytes, and more, lighter warps start and
// end an item sooner; 32 rows of 64 columns are bound by the warps' own latency,
// and 32 keys a warp keep more of their work independent. CTAs of an SM and
// stages are what shared memory and registers allow.
template <int DH, int RG>
struct OwnCfg {
    static constexpr int MR = 16 * RG;
    static constexpr int KG = DH == 64 && RG == 2 ? 2 : 4;    // key groups
    static constexpr int KB = kKT / 16 / KG;                  // blocks of 16 keys of a warp
    static constexpr int kWarps = KG * RG;                    // consumer warps
    static constexpr int kThreads = 32 * (kWarps + 1);        // and the producer
    static constexpr int NB = DH / 64;                        // 64-wide column blocks
    static constexpr uint32_t kBlk = kKT * 128;               // one block of a tile, 8 KB
    static constexpr uint32_t kStage = 2 * NB * kBlk;         // K and V of a tile
    static constexpr int kCtas = DH == 64 ? 3 : (RG == 1 ? 2 : 1);
    static constexpr int kStages = DH == 64 ? 3 : (RG == 1 ? 2 : 4);
    static constexpr int kQBufs = DH == 64 && RG == 2 ? 1 : 2;  // items described ahead
    static constexpr uint32_t kQ = MR * 128 * NB;
    static constexpr int kOs = DH + 4;                        // floats of a row to join
    static constexpr uint32_t kJoin = KG * MR * (kOs + 2) * 4;  // O, m, l of each key group
    static constexpr size_t kSmem = 1024 + kStages * kStage + kQBufs * kQ + kJoin;
    static constexpr int kSlot = MR * (DH + 2);               // floats of a part
};

template <int DH, int RG>
__global__ void __launch_bounds__(OwnCfg<DH, RG>::kThreads, OwnCfg<DH, RG>::kCtas)
    k_own(AttnArgs a, const __grid_constant__ CUtensorMap mk,
          const __grid_constant__ CUtensorMap mv) {
    using C = OwnCfg<DH, RG>;
    constexpr int ST = C::kStages, kThreads = C::kThreads, KG = C::KG, KB = C::KB;
    constexpr int QB = C::kQBufs;
    extern __shared__ unsigned char raw[];
    __shared__ uint64_t s_full[ST], s_empty[ST];
    __shared__ uint64_t s_qfull[QB], s_qempty[QB];  // an item's queries and description
    __shared__ OwnItem s_item[QB];
    __shared__ int s_bad[ST];
    __shared__ int64_t s_scan[kThreads / 32];
    __shared__ int s_seq, s_slots[kThreads], s_lens[kThreads];  // of all sequences, if they fit
    __shared__ int64_t s_seq_unit;
    const uint32_t raw_a = smem_addr(raw);
    unsigned char *ring = raw + (((raw_a + 1023u) & ~1023u) - raw_a);
    const uint32_t ring_a = smem_addr(ring);
    unsigned char *qs = ring + ST * C::kStage;
    const uint32_t qs_a = smem_addr(qs);
    float *join = reinterpret_cast<float *>(qs + C::kQBufs * C::kQ);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(&s_full[s], 1);
            mbar_init(&s_empty[s], C::kWarps);
            s_bad[s] = 0;
        }
        for (int s = 0; s < QB; ++s) {
            mbar_init(&s_qfull[s], 33);  // every producer lane's copies, and the description
            mbar_init(&s_qempty[s], C::kWarps);
        }
        mbar_fence_init();
        tma_prefetch_map(&mk);
        tma_prefetch_map(&mv);
        s_seq = a.N;
    }
    __syncthreads();
    // Beside k_prefix: that kernel let this one start only after its own wait, so what this
    // one reads is there; it waits for k_prefix at its end, since k_merge, which waits
    // for this one alone, reads what both wrote.
    if (!a.beside) pdl_wait();
    pdl_launch_dependents();
    auto leave = [&]() {
        if (a.beside) pdl_wait();
    };

    // This thread's sequence of the first kThreads; all of them, mostly.
    int my_slot = 0;
    const int my_len = tid < a.N ? seq_len(a, tid, &my_slot, blockIdx.x == 0) : -1;

    // The units of the call and the sequence that holds this CTA's first one.
    const int rows = a.D * a.G;
    const int RT = (rows + C::MR - 1) / C::MR;
    const int per = RT * a.Hkv;  // items of a sequence
    int64_t U = 0, u0 = 0, u1 = 0;
    int n_cta = 1;
    // Units before this thread's sequence of i0 .. i0 + kThreads - 1, the units of that, and
    // the total with them.
    auto scan = [&](int i0, int64_t base, int64_t *begin, int64_t *mine, bool report) {
        const int i = i0 + tid;
        int slot = my_slot, len = my_len;
        if (i0 > 0) len = i < a.N ? seq_len(a, i, &slot, report) : -1;
        *mine = (int64_t)per * own_tiles(a, len);
        int64_t inc = *mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(~0u, inc, o);
            if (lane >= o) inc += up;
        }
        __syncthreads();  // s_scan of the scan before
        s_slots[tid] = slot;
        s_lens[tid] = len;
        if (lane == 31) s_scan[warp] = inc;
        __syncthreads();
        int64_t before = base, all = base;
#pragma unroll
        for (int k = 0; k < kThreads / 32; ++k) {
            if (k < warp) before += s_scan[k];
            all += s_scan[k];
        }
        *begin = before + inc - *mine;
        return all;
    };
    int64_t begin = 0, mine = 0;
    for (int i0 = 0; i0 < a.N; i0 += kThreads) U = scan(i0, U, &begin, &mine, blockIdx.x == 0);
    n_cta = (int)min((int64_t)gridDim.x, max(U, (int64_t)1));
    u0 = share_begin(blockIdx.x, U, n_cta);
    u1 = share_begin(blockIdx.x + 1, U, n_cta);
    if (blockIdx.x == 0 && tid == 0) gst(a.cum + a.N, U);
    if ((int)blockIdx.x >= n_cta && blockIdx.x > 0) return leave();
    for (int64_t i0 = 0, base = 0; i0 < a.N; i0 += kThreads) {
        if (a.N > kThreads) base = scan((int)i0, base, &begin, &mine, false);
        const int i = (int)i0 + tid;
        if (i >= a.N) continue;
        if (u0 >= begin && u0 < begin + mine) {
            s_seq = i;
            s_seq_unit = begin;
        }
        if (blockIdx.x == 0) gst(a.cum + i, begin);
    }
    __syncthreads();
    if (u0 >= u1 || s_seq >= a.N) return leave();

    if (warp == C::kWarps) {  // producer
        // It alone walks the CTA's units and reads lengths and tables, a sequence ahead,
        // and copies each item's queries: under the load of the tile copies a global read
        // takes thousands of cycles, which no consumer then waits for.
        const int ps = a.pt.page_size;
        const int box = min(ps, kKT), nb = kKT / box;  // keys of a box, boxes of a tile
        // Slots and lengths of 32 sequences from `known` on, one a lane.
        int known = s_seq, slot_l = 0, len_l = -1;
        auto fetch = [&](int from) {
            known = from;
            const int i = from + lane;
            if (a.N <= kThreads) {
                len_l = i < a.N ? s_lens[i] : -1;
                slot_l = i < a.N ? s_slots[i] : 0;
            } else {
                len_l = i < a.N ? seq_len(a, i, &slot_l, false) : -1;
            }
        };
        fetch(known);
        struct Seq {
            int i, len, T, first, c, n;  // first own box; c, n: this lane's first page ids, as
                                         // PageIds::begin takes them
            PageIds ids;
        };
        // The next sequence from i on with keys of its own (i = N: none).
        auto find = [&](int i, Seq &s) {
            s.T = 0;
            for (; i < a.N; ++i) {
                if (i - known >= 32) fetch(i);
                s.len = __shfl_sync(~0u, len_l, i - known);
                s.T = own_tiles(a, s.len);
                if (s.T > 0) break;
            }
            s.i = i;
            if (i >= a.N) return;
            const int slot = __shfl_sync(~0u, slot_l, i - known);
            s.first = prefix_keys(a, s.len) / box;
            s.ids.start(a.pt.table + (int64_t)slot * a.pt.max_pages, ps / box, s.first,
                        (s.len - 1) / box);
            s.c = s.ids.cur;
            s.n = s.ids.nxt;
        };
        uint32_t g = 0, items = 0;
        // Describe an item to the consumers and start its queries; false when a wait gave up.
        auto announce = [&](const OwnItem &it) {
            const uint32_t b = items % QB;
            if (items >= QB && !mbar_wait_bounded(&s_qempty[b], (items / QB - 1) & 1u)) {
                raise_error(SC_DEV_TIMEOUT);
                return false;
            }
            if (it.n > 0) {
                const bf16 *q = a.q + (int64_t)it.i * a.D * a.q_stride + it.h * a.G * DH;
                constexpr int kStep = 256 / DH;  // rows of 32 chunks
                int r = lane / (DH / 8), rr = it.rt * C::MR + r, j = rr / a.G, gq = rr - j * a.G;
                const int ch = lane % (DH / 8);
                const uint32_t col = b * C::kQ + (ch >> 3) * C::MR * 128;
                for (; r < C::MR; r += kStep, rr += kStep) {
                    const uint32_t off = col + swz(r, ch & 7);
                    if (rr < rows)
                        cp_async16(qs_a + off, q + j * a.q_stride + gq * DH + ch * 8);
                    else
                        *reinterpret_cast<uint4 *>(qs + off) = make_uint4(0u, 0u, 0u, 0u);
                    for (gq += kStep; gq >= a.G; gq -= a.G) ++j;
                }
            }
            cp_async_arrive(&s_qfull[b]);
            if (lane == 0) s_item[b] = it;
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_qfull[b]);
            ++items;
            return true;
        };
        auto produce = [&](Seq &s, const OwnItem &it) {
            if (!announce(it)) return false;
            s.ids.begin(s.first + it.t0 * nb, s.c, s.n, it.t0 == 0);
            for (int t = 0; t < it.n; ++t, ++g) {
                const uint32_t st = g % ST;
                if (g >= ST && !mbar_wait_bounded(&s_empty[st], (g / ST - 1) & 1u)) {
                    raise_error(SC_DEV_TIMEOUT);
                    return false;
                }
                const int boxes = min(nb, s.ids.last + 1 - s.ids.box());
                int id = s.ids.page();
                bool bad = lane < boxes && (id < 0 || id >= a.pt.n_pages);
                if (bad) id = 0;
                bad = __any_sync(~0u, bad);
                if (lane == 0) {
                    if (bad) raise_error(SC_DEV_BAD_PAGE);
                    s_bad[st] = bad;
                    mbar_arrive_expect_tx(&s_full[st], (uint32_t)boxes * box * DH * 4);
                }
                __syncwarp();
                if (lane < boxes) {
                    const int key = id * ps + (s.ids.box() + lane) * box % ps;
                    const uint32_t d = ring_a + st * C::kStage + lane * box * 128;
#pragma unroll
                    for (int c = 0; c < C::NB; ++c) {
                        tma_load_3d(d + c * C::kBlk, &mk, &s_full[st], c * 64, it.h, key);
                        tma_load_3d(d + (C::NB + c) * C::kBlk, &mv, &s_full[st], c * 64, it.h, key);
                    }
                }
                s.ids.next(nb);
            }
            return true;
        };
        Seq s, after;
        find(s_seq, s);
        after.i = -1;  // not looked for yet: the first tiles go first
        int64_t left = u1 - u0;
        int it = (int)((u0 - s_seq_unit) / s.T), t0 = (int)(u0 - s_seq_unit - (int64_t)it * s.T);
        int rt = it / a.Hkv, h = it - rt * a.Hkv;
        bool ok = true;
        while (ok && left > 0 && s.i < a.N) {
            const int n = (int)min((int64_t)(s.T - t0), left);
            ok = produce(s, OwnItem{s.i, s.len, rt, h, s.i * per + it, t0, n, s.T});
            left -= n;
            t0 = 0;
            if (left > 0 && after.i < 0) find(s.i + 1, after);
            if (++h == a.Hkv) {
                h = 0;
                ++rt;
            }
            if (++it == per) {
                it = rt = h = 0;
                s = after;
                after.i = -1;
            }
        }
        if (ok) announce(OwnItem{0, 0, 0, 0, 0, 0, 0, 0});
        // No copy may be in flight when the CTA leaves.
        asm volatile("cp.async.wait_all;" ::: "memory");
        for (uint32_t c = g > ST ? g - ST : 0; c < g; ++c)
            mbar_wait_bounded(&s_full[c % ST], (c / ST) & 1u);
        return;
    }

    uint32_t ring_at = 0, ring_phase = 0;
    bool dead = false;
    const int kw = warp % KG, rg = warp / KG;  // key and row group
    // This lane's ldmatrix address in a K and in a V block: a step of 16 columns flips bits 5, 6.
    const uint32_t k_lane = swz(kw * 16 * KB + (lane & 7) + ((lane >> 4) << 3), (lane >> 3) & 1);
    const uint32_t v_lane = swz(kw * 16 * KB + (lane & 15), lane >> 4);
    const f32x2 scale2 = f2_make(a.scale_log2, a.scale_log2);
    const float rescale = kRescaleLog2 / a.scale_log2;
    // What a thread does with the rows of row tile rt, the same for every item: the
    // tokens of the two rows it computes, the output rows it writes chunks of (counted from the
    // sequence's first row of the kv head, -1 past the item's rows; rows, since the D Hq Dh
    // elements of one sequence may pass 2^31).
    constexpr int kOn = 16 * DH / 4 / (32 * KG);
    const int gt = kw * 32 + lane;  // thread of the row group
    int rt_now = -1, row_j[2], o_row[kOn];
    auto set_rows = [&](int rt) {
        rt_now = rt;
        const int r0 = rt * C::MR;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int rr = r0 + rg * 16 + p * 8 + (lane >> 2);
            row_j[p] = rr < rows ? rr / a.G : INT_MIN / 2;
        }
#pragma unroll
        for (int k = 0; k < kOn; ++k) {
            const int rr = r0 + rg * 16 + (gt + k * 32 * KG) / (DH / 4);
            o_row[k] = rr < rows ? rr / a.G * a.Hkv * a.G + rr % a.G : -1;
        }
    };
    for (uint32_t items = 0;; ++items) {
        const uint32_t qb = items % QB;
        const bool ready = !dead && mbar_wait_bounded(&s_qfull[qb], (items / QB) & 1u);
        // The warps go on together or not at all: none waits at a barrier the others left.
        if (named_or(1, 32 * C::kWarps, !ready)) {
            if (!ready && !dead) raise_error(SC_DEV_TIMEOUT);
            return leave();
        }
        const OwnItem item = s_item[qb];
        const int i = item.i, len = item.len, h = item.h, t0 = item.t0, n = item.n;
        if (n == 0) return leave();
        if (item.rt != rt_now) set_rows(item.rt);
        uint32_t qf[DH / 16][4];
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk) {
            const int ch = kk * 2 + (lane >> 4);
            ldsm4(qf[kk], qs_a + qb * C::kQ + (ch >> 3) * C::MR * 128 +
                              swz(rg * 16 + (lane & 15), ch & 7));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_qempty[qb]);
        // A row's running maximum m (of the scores before scaling), the score that moves
        // it, and its offset -m scale; the sums of its weights in pairs.
        int see[2];
        float m[2], limit[2], off[2], o[DH / 8][4];
        f32x2 l2[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            see[p] = len - a.D + 1 + row_j[p];  // below zero for a row past the item's
            m[p] = limit[p] = -INFINITY;
            off[p] = 0.0f;
            l2[p] = f2_make(0.0f, 0.0f);
        }
        const int least = len - a.D + 1;  // keys that every row of the sequence sees
#pragma unroll
        for (int d = 0; d < DH / 8; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][e] = 0.0f;
        bool bad = false;
        const int from = prefix_keys(a, len);
        int key0 = from + t0 * kKT + kw * 16 * KB;
        for (int t = 0; t < n; ++t, key0 += kKT) {
            if (!dead && !mbar_wait_bounded(&s_full[ring_at], ring_phase)) {
                raise_error(SC_DEV_TIMEOUT);
                dead = true;  // no more waits: the rest runs through on what is there
            }
            bad |= s_bad[ring_at] != 0;
            const uint32_t stage = ring_a + ring_at * C::kStage;
            const uint32_t kt = stage + k_lane, vt = stage + C::NB * C::kBlk + v_lane;
            const bool tail = key0 + 16 * KB > len;
            if (tail) {  // V rows past the sequence hold anything: 0 x NaN must not reach the sum
                const int first = max(0, len - key0);
                for (int x = lane; x < (16 * KB - first) * C::NB * 8; x += 32) {
                    const int r = first + x / (C::NB * 8), ch = x % (C::NB * 8);
                    *reinterpret_cast<uint4 *>(ring + ring_at * C::kStage +
                                               (C::NB + (ch >> 3)) * C::kBlk +
                                               (kw * 16 * KB + r) * 128 +
                                               (ch & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                __syncwarp();
            }
            float sc[2 * KB][4];
#pragma unroll
            for (int nt = 0; nt < 2 * KB; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[nt][e] = 0.0f;
#pragma unroll
            for (int kk = 0; kk < DH / 16; ++kk)
#pragma unroll
                for (int kb = 0; kb < KB; ++kb) {
                    uint32_t b[4];
                    ldsm4(b, (kt ^ ((kk & 3) << 5)) + (kk >> 2) * C::kBlk + kb * 2048);
                    mma16816(sc[2 * kb], qf[kk], b[0], b[1]);
                    mma16816(sc[2 * kb + 1], qf[kk], b[2], b[3]);
                }
            if (key0 + 16 * KB > least) {  // some row does not see some of these keys
#pragma unroll
                for (int nt = 0; nt < 2 * KB; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (key0 + nt * 8 + (lane & 3) * 2 + (e & 1) >= see[e >> 1])
                            sc[nt][e] = -INFINITY;
            }
            float top[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                top[p] = fmaxf(sc[0][2 * p], sc[0][2 * p + 1]);
#pragma unroll
                for (int nt = 1; nt < 2 * KB; ++nt)
                    top[p] = max3(top[p], sc[nt][2 * p], sc[nt][2 * p + 1]);
            }
            // Only when some score passes its row's limit are the row maxima needed. A row that
            // has seen no key yet keeps m = -inf, offset 0 and sums of zero.
            if (__any_sync(~0u, top[0] > limit[0] || top[1] > limit[1])) {
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    top[p] = fmaxf(top[p], __shfl_xor_sync(~0u, top[p], 1));
                    top[p] = fmaxf(top[p], __shfl_xor_sync(~0u, top[p], 2));
                    if (!(top[p] > limit[p])) continue;
                    const float f = ex2((m[p] - top[p]) * a.scale_log2);
                    m[p] = top[p];
                    limit[p] = top[p] + rescale;
                    off[p] = -top[p] * a.scale_log2;
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
                const f32x2 off2 = f2_make(off[p], off[p]);
#pragma unroll
                for (int nt = 0; nt < 2 * KB; ++nt) {
                    float e0, e1;
                    f2_split(f2_fma(f2_make(sc[nt][2 * p], sc[nt][2 * p + 1]), scale2, off2), e0, e1);
                    e0 = ex2(e0);
                    e1 = ex2(e1);
                    l2[p] = f2_add(l2[p], f2_make(e0, e1));
                    // P enters the second product as bf16: 2^-8 relative a term at most.
                    pf[nt / 2][nt % 2 * 2 + p] = pack_bf16(e0, e1);
                }
            }
            // A draft that some row does not see: were its V not finite, a weight of 0 would
            // not keep it from that row, so the block's product is made one by one.
            bool plain = false;
            if (key0 + 16 * KB > least) {
                const unsigned char *vb = ring + ring_at * C::kStage + C::NB * C::kBlk;
                const int lo = max(least - key0, 0), hi = min(len - key0, 16 * KB);
                for (int x = lane; x < (hi - lo) * DH / 8; x += 32)
                    plain |= not_finite(*reinterpret_cast<const uint4 *>(
                        vb + (x % (DH / 8) >> 3) * C::kBlk +
                        swz(kw * 16 * KB + lo + x / (DH / 8), x & 7)));
                plain = __any_sync(~0u, plain);
                if (plain) product_one_by_one<DH, KB>(o, pf, vb, C::kBlk, kw * 16 * KB, key0, see);
            }
            if (!plain) {
#pragma unroll
                for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                    for (int dd = 0; dd < DH / 16; ++dd) {
                        uint32_t b[4];
                        ldsm4_t(b, (vt ^ ((dd & 3) << 5)) + (dd >> 2) * C::kBlk + kb * 2048);
                        mma16816(o[2 * dd], pf[kb], b[0], b[1]);
                        mma16816(o[2 * dd + 1], pf[kb], b[2], b[3]);
                    }
            }
            if (tail) fence_proxy_async_smem();  // the zeroed rows before the next copy there
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[ring_at]);
            if (++ring_at == ST) {
                ring_at = 0;
                ring_phase ^= 1u;
            }
        }
        // Join the key warps: each leaves its m, l and O, and a thread joins and writes
        // four columns of a row. (The next join comes after the next item's barrier.)
        float *jo = join + rg * KG * 16 * C::kOs;  // [key group][16][kOs]
        float *jm = join + KG * C::MR * C::kOs + rg * KG * 32;  // [key group][m 16, l 16]
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int r = p * 8 + (lane >> 2);
            float l, l1;
            f2_split(l2[p], l, l1);
            l += l1;
            l += __shfl_xor_sync(~0u, l, 1);
            l += __shfl_xor_sync(~0u, l, 2);
            if ((lane & 3) == 0) {
                jm[kw * 32 + r] = m[p] * a.scale_log2;
                jm[kw * 32 + 16 + r] = l;
            }
#pragma unroll
            for (int d = 0; d < DH / 8; ++d)
                *reinterpret_cast<float2 *>(jo + (kw * 16 + r) * C::kOs + d * 8 + (lane & 3) * 2) =
                    make_float2(o[d][2 * p], o[d][2 * p + 1]);
        }
        named_sync(1, 32 * C::kWarps);
        const bool whole = n == item.T && from == 0;  // nothing to join with
        float *part = a.own_part + (int64_t)(item.w + blockIdx.x) * C::kSlot;
        bf16 *out = a.out + ((int64_t)i * a.D * a.Hkv + h) * a.G * DH;
#pragma unroll
        for (int k = 0; k < kOn; ++k) {
            const int x = gt + k * 32 * KG, r = x / (DH / 4), c4 = x % (DH / 4);
            float top = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int q = 0; q < KG; ++q) top = fmaxf(top, jm[q * 32 + r]);
            const float off = top == -INFINITY ? 0.0f : top;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int q = 0; q < KG; ++q) {
                const float f = ex2(jm[q * 32 + r] - off);
                const float4 u =
                    *reinterpret_cast<float4 *>(jo + (q * 16 + r) * C::kOs + c4 * 4);
                sum = fmaf(f, jm[q * 32 + 16 + r], sum);
                v.x = fmaf(f, u.x, v.x);
                v.y = fmaf(f, u.y, v.y);
                v.z = fmaf(f, u.z, v.z);
                v.w = fmaf(f, u.w, v.w);
            }
            if (o_row[k] < 0) continue;
            if (whole) {
                if (bad) continue;
                const float inv = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;
                gst(reinterpret_cast<uint2 *>(out + (int64_t)o_row[k] * DH + c4 * 4),
                    make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv)));
            } else {
                const int row = rg * 16 + r;
                gst(reinterpret_cast<float4 *>(part + row * DH + c4 * 4), v);
                if (c4 == 0) {
                    // A NaN maximum marks a part with a bad page: k_merge leaves its rows alone.
                    gst(part + C::MR * DH + row, bad ? __int_as_float(0x7FC00000) : top);
                    gst(part + C::MR * DH + C::MR + row, sum);
                }
            }
        }
    }
}

}  // namespace sc

#include "attention_prefix.cuh"

namespace sc {

// A block joins rows of one token. Dh / 8 lanes hold eight columns of a row each; PG
// such groups share the row's parts (with few rows there are many parts and lanes
// to spare). Lane k of the row holds the maximum and sum of part k, then every group
// adds its parts, in a fixed order. No load waits for another part's.
constexpr int kMergeThreads = 256;
template <int DH, int PG>
__global__ void __launch_bounds__(kMergeThreads) k_merge(PrefixArgs x, int MR, int own_ctas) {
    AttnArgs &a = x.a;
    constexpr int L = DH / 8 * PG;
    const int rl = threadIdx.x % L, c8 = rl % (DH / 8), group = rl / (DH / 8);
    const int Hq = a.Hkv * a.G;
    const int token = blockIdx.x, i = token / a.D, j = token - i * a.D;
    const int at = blockIdx.y * (kMergeThreads / L) + threadIdx.x / L;
    const int hq = min(at, Hq - 1);  // lanes past the last row join it and write nothing
    const int h = hq / a.G, g = hq - h * a.G;
    // Slots and lengths need no wait: k_own let this kernel start when what wrote them was done.
    int slot;
    const int len = seq_len(a, i, &slot, false);
    const bool valid = len >= 0, prefix = prefix_keys(a, len) > 0;

    // The row's parts: prefix_n from prefix_at on, own_n from own_at on (its O; m and l
    // are at +m_off and +l_off).
    constexpr int kPSlot = kPR * (DH + 2);
    const float *prefix_at = nullptr, *own_at = nullptr;
    int prefix_n = 0, own_n = 0, prefix_m = 0, own_m = 0, step = 0;
    bool mine = valid && at < Hq;
    if (prefix) {
        const int tile = token / x.tpt, r = (token - tile * x.tpt) * a.G + g;
        const int64_t w = (int64_t)(x.split ? tile : tile >> 1) * a.Hkv + h;
        const int c0 = share_of(w * x.T, x.U, x.n_cta);
        const int c1 = share_of(w * x.T + x.T - 1, x.U, x.n_cta);
        prefix_at = x.part + ((w + c0) * 2 + (x.split ? 0 : tile & 1)) * kPSlot + r * DH;
        prefix_m = kPR * DH + r - r * DH;
        step = x.split ? kPSlot : 2 * kPSlot;
        prefix_n = (c1 - c0 + 1) * (x.split ? 2 : 1);
    }
    pdl_wait();
    pdl_launch_dependents();
    const int64_t U = gld(a.cum + a.N), u_i = gld(a.cum + i), u_n = gld(a.cum + i + 1);
    const int r = j * a.G + g, per = (a.D * a.G + MR - 1) / MR * a.Hkv;
    const int oslot = MR * (DH + 2), rt = r / MR, orow = r - rt * MR;
    if (u_n > u_i) {
        const int64_t d = u_n - u_i;
        const int64_t T = d <= UINT32_MAX ? (uint32_t)d / (uint32_t)per : d / per;
        const int n_cta = (int)min((int64_t)own_ctas, U);
        const int it = rt * a.Hkv + h;
        const int64_t u0 = u_i + it * T;
        const int c0 = share_of(u0, U, n_cta), c1 = share_of(u0 + T - 1, U, n_cta);
        own_at = a.own_part + ((int64_t)i * per + it + c0) * oslot + orow * DH;
        own_m = MR * DH + orow - orow * DH;
        own_n = c1 - c0 + 1;
        if (own_n == 1 && !prefix) {  // k_own wrote the row
            own_n = 0;
            mine = false;
        }
    }
    const int parts = prefix_n + own_n;
    const float *own_from = own_at - (int64_t)prefix_n * oslot;  // part p's, p >= prefix_n, at + p * oslot
    int most = parts;  // of the warp's rows: its lanes stay together
#pragma unroll
    for (int k = 16; k >= L; k >>= 1) most = max(most, __shfl_xor_sync(~0u, most, k));
    float top = -INFINITY, sum = 0.0f, o[8] = {};
    bool bad = false;
    for (int p0 = 0; p0 < most; p0 += L) {
        float m = -INFINITY, l = 0.0f;
        const int p = p0 + rl;
        if (p < parts) {
            const bool pre = p < prefix_n;
            const float *ml = pre ? prefix_at + (int64_t)p * step + prefix_m
                                  : own_from + (int64_t)p * oslot + own_m;
            m = gld(ml);
            l = gld(ml + (pre ? kPR : MR));
        }
        // Parts are loaded before the factors are known: with few rows, up to 32 (Dh 64) or 16 at
        // once, since the kernel is then a chain of dependent reads.
        const int here = min(L, parts - p0), rounds = min(L, most - p0);
        constexpr int kAhead = PG > 1 ? 8 : 4;
        float4 v[kAhead][2];
        auto fetch = [&](int q0) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int q = q0 + k * PG + group;
                if (q < here) {
                    const float4 *from = reinterpret_cast<const float4 *>(
                        p0 + q < prefix_n ? prefix_at + (int64_t)(p0 + q) * step
                                          : own_from + (int64_t)(p0 + q) * oslot);
                    v[k][0] = gld(from + c8 * 2);
                    v[k][1] = gld(from + c8 * 2 + 1);
                }
            }
        };
        fetch(0);
        float now = fmaxf(top, m);
        int nan = m != m;
#pragma unroll
        for (int k = L / 2; k; k >>= 1) {
            now = fmaxf(now, __shfl_xor_sync(~0u, now, k));
            nan |= __shfl_xor_sync(~0u, nan, k);
        }
        bad |= nan != 0;
        const float base = now == -INFINITY ? 0.0f : now;
        const float f = ex2(m - base), f0 = ex2(top - base);
        float s = l * f;
#pragma unroll
        for (int k = L / 2; k; k >>= 1) s += __shfl_xor_sync(~0u, s, k);
        sum = sum * f0 + s;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] *= f0;
        top = now;
        for (int q0 = 0; q0 < rounds; q0 += kAhead * PG) {
            if (q0 > 0) fetch(q0);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int q = q0 + k * PG + group;
                const float w = __shfl_sync(~0u, f, q, L);
                if (q >= here) continue;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    o[4 * e] = fmaf(w, v[k][e].x, o[4 * e]);
                    o[4 * e + 1] = fmaf(w, v[k][e].y, o[4 * e + 1]);
                    o[4 * e + 2] = fmaf(w, v[k][e].z, o[4 * e + 2]);
                    o[4 * e + 3] = fmaf(w, v[k][e].w, o[4 * e + 3]);
                }
            }
        }
    }
#pragma unroll
    for (int k = DH / 8; k < L; k <<= 1)
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] += __shfl_xor_sync(~0u, o[e], k);
    mine = mine && group == 0;
    if (bad || !mine) return;  // a bad page: the row is not written
    const float inv = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;
    gst(reinterpret_cast<uint4 *>(a.out + ((int64_t)token * Hq + hq) * DH + c8 * 8),
        make_uint4(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv),
                   pack_bf16(o[4] * inv, o[5] * inv), pack_bf16(o[6] * inv, o[7] * inv)));
}

// ------------------------------------------------------------ host side

// Pages [n_pages * page_size tokens, Hkv, Dh] in boxes of `keys` tokens of one
// head, 64 columns, 128-byte swizzle.
static cudaError_t map_pages(CUtensorMap *m, const void *ptr, const PageTable &pt, int Hkv, int Dh,
                             int keys) {
    EncodeTiledFn fn = encode_tiled();
    if (fn == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)Dh, (cuuint64_t)Hkv,
                                (cuuint64_t)pt.n_pages * pt.page_size};
    const cuuint64_t strides[2] = {(cuuint64_t)Dh * 2, (cuuint64_t)Hkv * Dh * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)keys};
    const cuuint32_t es[3] = {1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims,
                          strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Queries [N*D, Hkv, G, Dh] in boxes of the G heads of `tpt` tokens of one kv
// head, 64 columns, 128-byte swizzle; tokens past the last read as zeros.
static cudaError_t map_queries(CUtensorMap *m, const PrefixArgs &x, const AttnShape &s) {
    EncodeTiledFn fn = encode_tiled();
    if (fn == nullptr) return cudaErrorNotSupported;
    const int G = x.a.G;
    const cuuint64_t dims[4] = {(cuuint64_t)s.Dh, (cuuint64_t)G, (cuuint64_t)s.Hkv,
                                (cuuint64_t)s.N * s.D};
    const cuuint64_t strides[3] = {(cuuint64_t)s.Dh * 2, (cuuint64_t)G * s.Dh * 2,
                                   (cuuint64_t)x.a.q_stride * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)G, 1, (cuuint32_t)x.tpt};
    const cuuint32_t es[4] = {1, 1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<bf16 *>(x.a.q), dims,
                          strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Rows of an item: 16 hold up to 16 rows of a sequence and kv head, else 32.
static int own_rows(const AttnShape &s) { return s.D * (s.Hq / s.Hkv) <= 16 ? 16 : 32; }

static size_t own_part_floats(const AttnShape &s) {
    const int MR = own_rows(s);
    const size_t items =
        (size_t)s.N * s.Hkv * (((size_t)s.D * (s.Hq / s.Hkv) + MR - 1) / MR);
    return (items + kMaxCtas) * MR * (s.Dh + 2);
}
// [N + 1] first tiles.
static size_t cum_bytes(const AttnShape &s) { return ((size_t)s.N + 3) / 2 * 16; }

// The prefix's work: everything but the pointers.
static PrefixArgs prefix_plan(const AttnShape &s, int page_size, int sm_count) {
    PrefixArgs x = {};
    const int G = s.Hq / s.Hkv;
    x.P = s.shared_pages * page_size;
    x.tpt = kPR / G;
    x.n_tiles = (s.N * s.D + x.tpt - 1) / x.tpt;
    x.split = x.n_tiles == 1;
    const int keys = x.split ? 2 * kPK : kPK;
    x.T = (x.P + keys - 1) / keys;
    x.U = (int64_t)s.Hkv * (x.split ? 1 : (x.n_tiles + 1) / 2) * x.T;
    const int ctas = sm_count < kMaxPrefixCtas ? sm_count : kMaxPrefixCtas;
    x.n_cta = (int)(x.U < ctas ? x.U : ctas);
    // A small prefix costs fixed latencies more than work: it takes a CTA for every eight
    // units (four of 128-wide heads), up to half the SMs, and the own parts run on the
    // others meanwhile. 64 sequences of 64-1500 own tokens, us beside and one after the
    // other: 24.9 and 33.6 with 64 units, 31.7 and 40.2 with 384, 37.1 and 41.6 with 600 (the
    // rule ends at 608); of 1-30 own tokens 22.8 and 23.7 with 600, 25.5 and 25.4 with 768.
    // Heads of 128: 46.9 and 58.5 with 64, 58.9 and 66.0 with 256 (the rule ends at 304). Slower
    // beside: 16 sequences behind 1024 tokens (32 units), 25.9 and 20.3, behind 2048, 23.6 and 21.0.
    const int units = s.Dh == 64 ? 8 : 4;
    x.a.beside = x.U > 0 && x.U <= (int64_t)units * (ctas / 2);
    if (x.a.beside) x.n_cta = (int)((x.U + units - 1) / units);
    return x;
}
static size_t prefix_part_floats(const AttnShape &s) {
    if (s.shared_pages == 0) return 0;
    const PrefixArgs x = prefix_plan(s, 1, kMaxPrefixCtas);
    const size_t items = (size_t)s.Hkv * (x.split ? 1 : (x.n_tiles + 1) / 2);
    return 2 * (items + kMaxPrefixCtas) * kPR * (s.Dh + 2);
}

size_t attention_workspace_bytes(const AttnShape &s) {
    return cum_bytes(s) + (own_part_floats(s) + prefix_part_floats(s)) * 4;
}

template <typename F>
static cudaError_t smem_opt_in(F kern, size_t bytes, std::atomic<unsigned long long> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (done.load() & (1ull << dev))) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev);
    return e;
}

template <int DH, int RG>
static cudaError_t launch_own(const AttnArgs &a, const CUtensorMap &mk, const CUtensorMap &mv,
                              int sms, int *grid, cudaStream_t stream) {
    using C = OwnCfg<DH, RG>;
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = smem_opt_in(k_own<DH, RG>, C::kSmem, done);
    if (e != cudaSuccess) return e;
    *grid = C::kCtas * sms < kMaxCtas ? C::kCtas * sms : kMaxCtas;
    return launch_pdl(k_own<DH, RG>, dim3((unsigned)*grid), dim3(C::kThreads), C::kSmem, stream, a,
                      mk, mv);
}

template <int DH>
static cudaError_t launch_prefix(const PrefixArgs &x, const CUtensorMap &mq, const CUtensorMap &mk,
                                 const CUtensorMap &mv, cudaStream_t stream) {
    using C = PfxCfg<DH>;
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = smem_opt_in(k_prefix<DH>, C::kSmem, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(k_prefix<DH>, dim3((unsigned)x.n_cta), dim3(kPfxThreads), C::kSmem, stream, x,
                      mq, mk, mv);
}

cudaError_t launch_prefix_attention(const AttnShape &s, const void *q, int64_t q_stride,
                                    const void *k_pages, const void *v_pages, const PageTable &pt,
                                    const int32_t *slots, float scale, void *out,
                                    void *workspace, int sm_count, cudaStream_t stream) {
    PrefixArgs x = prefix_plan(s, pt.page_size, sm_count);
    AttnArgs &a = x.a;
    a.q = (const bf16 *)q;
    a.q_stride = q_stride;
    a.pt = pt;
    a.slots = slots;
    a.N = s.N;
    a.D = s.D;
    a.G = s.Hq / s.Hkv;
    a.Hkv = s.Hkv;
    a.shared_keys = x.P;
    a.scale_log2 = scale * kLog2e;
    a.out = (bf16 *)out;
    a.cum = (int64_t *)workspace;
    a.own_part = (float *)((char *)workspace + cum_bytes(s));
    x.part = a.own_part + own_part_floats(s);
    CUtensorMap mk, mv;
    const int own_box = pt.page_size < kKT ? pt.page_size : kKT;
    cudaError_t e = map_pages(&mk, k_pages, pt, s.Hkv, s.Dh, own_box);
    if (e != cudaSuccess) return e;
    e = map_pages(&mv, v_pages, pt, s.Hkv, s.Dh, own_box);
    if (e != cudaSuccess) return e;
    if (x.P > 0) {
        CUtensorMap mq, pk = mk, pv = mv;
        const int box = pt.page_size < kPK ? pt.page_size : kPK;
        if (box != own_box) {
            e = map_pages(&pk, k_pages, pt, s.Hkv, s.Dh, box);
            if (e != cudaSuccess) return e;
            e = map_pages(&pv, v_pages, pt, s.Hkv, s.Dh, box);
            if (e != cudaSuccess) return e;
        }
        e = map_queries(&mq, x, s);
        if (e != cudaSuccess) return e;
        e = s.Dh == 64 ? launch_prefix<64>(x, mq, pk, pv, stream)
                       : launch_prefix<128>(x, mq, pk, pv, stream);
        if (e != cudaSuccess) return e;
    }
    const int MR = own_rows(s);
    const int sms = a.beside ? sm_count - x.n_cta : sm_count;
    int grid = 0;
    if (s.Dh == 64)
        e = MR == 16 ? launch_own<64, 1>(a, mk, mv, sms, &grid, stream)
                     : launch_own<64, 2>(a, mk, mv, sms, &grid, stream);
    else
        e = MR == 16 ? launch_own<128, 1>(a, mk, mv, sms, &grid, stream)
                     : launch_own<128, 2>(a, mk, mv, sms, &grid, stream);
    if (e != cudaSuccess) return e;
    // With few rows all lanes of a warp share one: a whole step over two streams of 30-40
    // thousand tokens takes 39 us so, 45 with Dh / 8 lanes a row. With many there is work
    // enough: 128 x 8 drafts take 193 us with Dh / 8 lanes, 213 with whole warps. Between, one
    // token of sequences of 64-1500 tokens, us with whole warps and without: 1024 rows 14.9 and
    // 15.5, 2048 rows 23.3 both, 4096 rows 52.0 and 49.6, 16384 rows 210 and 201 (heads of 128:
    // 1024 rows 24.7 and 24.8, 4096 rows 77.9 and 75.2).
    const bool few = (int64_t)s.N * s.D * s.Hq <= 4096;
    const auto merge = s.Dh == 64 ? (few ? k_merge<64, 4> : k_merge<64, 1>)
                                  : (few ? k_merge<128, 2> : k_merge<128, 1>);
    const int block_rows = few ? kMergeThreads / 32 : kMergeThreads / (s.Dh / 8);  // of one token
    const dim3 blocks((unsigned)(s.N * s.D), (unsigned)((s.Hq + block_rows - 1) / block_rows));
    return launch_pdl(merge, blocks, dim3(kMergeThreads), 0, stream, x, MR, grid);
}

cudaError_t take_error_attention(cudaStream_t stream, unsigned int *sum) {
    return take_error_here(stream, sum);
}

#ifdef SC_BOUNDS_CHECK
cudaError_t bounds_install_attention(const BoundsRegion *r, int n, cudaStream_t stream) {
    return bounds_install_here(r, n, stream);
}
cudaError_t bounds_take_attention(cudaStream_t stream, unsigned long long *addr) {
    return bounds_take_first_bad_here(stream, addr);
}
#endif

}  // namespace sc
