// attention_8bit.cuh -- what attention.cu's k_own does with tiles of an 8-bit cache, and the
// unpacking of a shared prefix.
//
// A key is ks k', a value vs v' (codes k', v' of e4m3, powers of two ks, vs of the block and
// head). The codes go to the tensor cores as f16, which holds them exactly; Q goes there as f16 too,
// times a power of two that takes its row's largest to 2^14 (11 bits of f16 hold bf16's 8). The
// scales stay out of the products: with s_t a row's score in units of log2,
//   out = sum_t 2^(s_t + log2 vs_t - m) v'_t / sum_t 2^(s_t + log2 vs_t - m) / vs_t,
// so that the weights that meet v' lie below the row's largest, whatever the sizes of the
// blocks' values. m is the running maximum of s_t + log2 vs_t. Weights go to the second product as
// f16, at most 2^15: rounded by 2^-11 of themselves down to 2^-27 of the row's largest, by 2^-8, as bf16
// would be, down to 2^-30. Smaller ones lose what is too little to see, 2^-10 of a channel's
// sum w |v| in all, or, where the keys of much weight hold zeros in a channel, so that such weights are
// all it has, go into further products scaled up (small_weights8).
//
// (The register MMA of e4m3 itself is made of conversions of both operands and further MMAs on this
// GPU: 56 million warp instructions for 128 sequences of 200-6000 tokens, this takes 33.)
//
// What bounds it: the codes' bytes with up to 8 rows (128 sequences of 200-6000 tokens by 8 x 4
// heads: 404 MB from DRAM, the same that are needed, in 72 us; issue slots 42 %; 128 of 500-1500 by heads
// of 128: 259 MB in 50 us, 5.2 TB/s); with 16 and 32 rows the
// conversions and the softmax in the issue slots (128 of 500-1500 tokens: 34 us a call with 4 rows, 41
// with 16, 67 with 32, whose k_own issues in half of its cycles, waiting for its own results). Not better: four row tiles a warp instead of two row groups (k_own 46 to 80 us,
// spills); eight-row groups with heads of 128 (74 to 84); 256-byte L2 promotion with an item a head
// (920 MB read for 404).
#pragma once

namespace sc {

// A row's maximum moves when a score passes it by kRescale8 (in log2), and weighs 2^kTop8: weights
// are at most 2^15. Those below kLeast, which f16 rounds by more than 2^-8, are looked after in tile8: the
// less a maximum lags, the fewer they are. 128 sequences of 500-1500 tokens by 8 drafts of 8 x 4 heads, us
// with a lag of 2^8, 2^4 and 2^2: 67.8, 66.7, 67.2; with queries three times as large 101, 79, 76.
constexpr float kRescale8 = 2.0f, kTop8 = 15.0f - kRescale8;
constexpr float kLeastLog2 = -17.0f, kLeast = 0x1p-17f;
constexpr float kUnseen8 = 0x1p127f;  // the offset of a row without a key

// The scales of a tile's G groups of 8 keys, K's and V's: the aligned 16 bytes of the
// scale array that hold each, and which of the four it is.
template <int G>
struct TileScales8 {
    uint4 four[2][G];
    int at[2][G];
};

// The producer warp's part: lane k starts group k's copy. `id`: lane b's page of box b (of
// `box` keys, `boxes` of them there) of the tile that begins at key `key0` of the sequence. Copies
// go to L2 (.cg), as the other reads of a kernel that may start beside another. Arrays that do not
// start on 16 bytes (a layer's of stacked ones) are read word by word.
template <int HG, int G>
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
        const float *all = which ? a.s8.v : a.s8.k;
        const int64_t first = i & ~(int64_t)3;
        const uint32_t bytes = (uint32_t)min((int64_t)16, (total - first) * 4);
        const float *from = all + first;
        at = (int)(i - first);
        if ((reinterpret_cast<uintptr_t>(all) & 15) != 0) {
            at = 0;
#pragma unroll
            for (int e = 0; e < HG; ++e)
                reinterpret_cast<int *>(&s.four[which][g])[e] =
                    gld_l2(reinterpret_cast<const int32_t *>(all + i + e));
        } else if (SC_RD_OK(from, bytes))
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                             smem_addr(&s.four[which][g])),
                         "l"(from), "r"(bytes));
    }
    s.at[which][g] = at;
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
// Two 16 x 16 matrices of bytes, transposed: lane 4 g + c gets rows 4 c .. 4 c + 3 of column g
// (r[0]) and of column g + 8 (r[1]) of the first, and the same of the second.
__device__ __forceinline__ void ldsm2_t8(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t word_of(const uint4 &v, int e) {
    return e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// An 8 x 8 matrix of 16-bit values, transposed: lane 4 g + c holds row g's columns 2 c, 2 c + 1.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// An item is MR rows of a sequence for HG kv heads at once. A consumer warp takes WR rows of one
// head by 32 keys of a tile, or 16 with heads of 128: a row's sums are twice as many registers there,
// and tiles of half the bytes leave twice as many on their way (72 sequences of 5 drafts by 7 heads:
// 12.1 us, with 32 keys 13.8; 64 sequences of 8 by 7: 18.8 for 20.7; short single tokens even).
// Both products have the keys' matrix first (16 keys, or 16 columns of V, by 8 rows of queries), so
// that 8 rows fill a product and a code is converted once for all rows.
template <int DH, int MR_, int HG>
struct Own8Cfg {
    static constexpr int kDh = DH;
    static constexpr int MR = MR_;
    static constexpr int RG = MR == 32 ? 2 : 1;               // row groups
    static constexpr int WR = MR / RG;
    static constexpr int NT = WR / 8;                         // row tiles of a warp
    static constexpr int kHeads = HG;
    static constexpr int KG = 4 / (HG * RG);                  // key groups
    static constexpr int KH = DH == 64 ? 2 : 1;               // halves of 16 keys of a warp
    static constexpr int KT = 16 * KH * KG;                   // keys of a tile
    static constexpr int kWarps = 4;
    static constexpr int kThreads = 32 * (kWarps + 1);
    static constexpr int kRow = HG * DH == 64 ? 64 : 128;     // bytes of a key in a column block
    static constexpr int NC = HG * DH / kRow;                 // column blocks
    static constexpr uint32_t kBlk = KT * kRow;
    static constexpr uint32_t kV = NC * kBlk;                 // the tile's V behind its K
    static constexpr uint32_t kStage = 2 * kV;                // 16 KB, with 32 rows 8
    // By registers: 128 a thread, or 168. Heads of 64, us with 2, 3 and 4: 128 sequences of 200-6000
    // tokens 99, 81, 92; 8 drafts of 128 of 500-1500 72, 67, 106; 512 of 20-60 29.2, 30.8, 33.1.
    static constexpr int kCtas = DH == 64 || MR == 8 ? 3 : 2;
    static constexpr int kQBufs = 2;                          // items described ahead
    static constexpr uint32_t kQ = 0;                         // the consumers read their queries
    static constexpr int kOs = DH + 4;                        // floats of a row to join
    static constexpr uint32_t kJoin = KG > 1 ? kWarps * WR * (kOs + 2) * 4 : 0;
    // Tiles in flight: what the CTAs of an SM leave of its 228 KB beside 4.5 KB each of static and
    // reserved shared memory.
    static constexpr size_t kRest = 1024 + kJoin;
    static constexpr int kFit = (int)((228 * 1024 / kCtas - 4608 - kRest) / kStage);
    static constexpr int kStages = kFit < 8 ? kFit : 8;
    static_assert(kStages >= 2, "shared memory of an SM");
    static constexpr size_t kSmem = kRest + kStages * kStage;
    static constexpr int kSlot = MR * (DH + 2);               // floats of a part and head
    typedef TileScales8<KT / 8> Scales;
};
template <int DH, int MR>
struct OwnCfg<DH, MR, 1> : Own8Cfg<DH, MR, 1> {};
template <int DH, int MR>
struct OwnCfg<DH, MR, 2> : Own8Cfg<DH, MR, 2> {};
template <int DH, int MR>
struct OwnCfg<DH, MR, 4> : Own8Cfg<DH, MR, 4> {};

// Where this lane, 4 g + c, finds a tile's codes, as byte offsets from the tile's K (or V).
// Rows of 128 bytes have their 16-byte chunks XOR-swizzled by the row's low 3 bits, rows of 64 by its
// bits 1 and 2.
//
// The order of 16 keys in both products is free as long as they agree: key_of() gives the key
// of place i. Places g and g + 8, whose scores a lane holds, are then in one group of 8 keys,
// the four places 2 c, 2 c + 1, 2 c + 8, 2 c + 9 of a lane's second operand are one word of
// ldsm2_t8, and neither product's reads meet in a bank (in rows of 128 bytes).
template <typename C>
struct Lane8 {
    int g, c, half;      // half: of its column block, where that holds two heads
    uint32_t base;       // of this warp's head and its first key
    uint32_t k_at[2];    // chunk c of the keys at places g, g + 8; the next 64 columns: XOR 64
    uint32_t v_at;       // for ldsm2_t8: both halves' keys, or 32 columns of 16 keys; the next: XOR
    int key;             // at place g; at place g + 8: 2 more
    __device__ __forceinline__ Lane8(int hh, int row0) {
        const int lane = threadIdx.x & 31;
        g = lane >> 2;
        c = lane & 3;
        constexpr bool kTwo = C::kRow == 128 && C::kDh == 64;
        half = kTwo ? hh & 1 : 0;
        base = (kTwo ? hh >> 1 : C::kRow == 128 ? hh : 0) * C::kBlk + row0 * C::kRow;
        key = key_of(g);
        k_at[0] = at(key, c);
        k_at[1] = at(key + 2, c);
        const int i = lane & 15;  // word i / 4, byte i % 4
        const int i_key = key_of(2 * (i >> 2) + (i & 1) + 4 * (i & 2));
        v_at = C::KH == 2 ? at((lane & 16) + i_key, 0) : at(i_key, lane >> 4);
    }
    static __device__ __forceinline__ int key_of(int i) {
        return (i >> 2 & 1) * 8 + (i & 1) * 4 + (i >> 3) * 2 + (i >> 1 & 1);
    }
    // Chunk `chunk` of this warp's head at its key `row`.
    __device__ __forceinline__ uint32_t at(int row, int chunk) const {
        const int x = C::kRow == 64 ? row >> 1 & 3 : row & 7;
        return base + row * C::kRow + (uint32_t)((half * 4 + chunk) ^ x) * 16;
    }
};

// A warp's rows of an item: the lane's are rows 8 n + 2 c and the next, as pairs.
template <typename C>
struct Rows8 {
    // Row 8 n + g as the first product's second operand. The column order of that product is free
    // too: lane c takes the columns 16 c .. 16 c + 15 (of each 64), four a step, which K's row
    // holds as one chunk.
    uint32_t qf[C::NT][C::kDh / 16][2];
    f32x2 unit[C::NT];  // what a product stands for, times scale log2(e)
    f32x2 off[C::NT];   // o and l are in units of 2^-off: kTop8 - m, kUnseen8 before any key
    f32x2 l[C::NT];
    int row0;           // of the sequence's rows of a head
    int sees[2];        // of one row tile, the keys that its rows see
    float o[C::NT][C::kDh / 16][4];  // columns 16 j + g and 16 j + 8 + g, of both rows each

    // Keys that row 8 n + 2 c + p sees: `least` and one a token before its own; below zero for a row
    // past the item's. Two row tiles are short of registers, and few tiles of keys ask.
    __device__ __forceinline__ int see(const AttnArgs &a, int least, int n, int p) const {
        if (C::NT == 1) return sees[p];
        return find_see(a, least, n, p);
    }
    __device__ __forceinline__ int find_see(const AttnArgs &a, int least, int n, int p) const {
        const int rr = row0 + n * 8 + 2 * (threadIdx.x & 3) + p;
        return rr < a.D * a.G ? least + rr / a.G : INT_MIN / 2;
    }

    // The rows from row0 on of the `rows` of sequence i under kv head h.
    __device__ __forceinline__ void load(const AttnArgs &a, int i, int h, int row0, int rows) {
        const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
        constexpr int DH = C::kDh;
        this->row0 = row0;
        uint4 all[C::NT][DH / 32];
#pragma unroll
        for (int n = 0; n < C::NT; ++n) {
            const int rr = row0 + 8 * n + g, j = rr / a.G;
            const bf16 *q = a.q + ((int64_t)i * a.D + j) * a.q_stride +
                            (int64_t)(h * a.G + rr - j * a.G) * DH + 16 * c;
#pragma unroll
            for (int b = 0; b < DH / 32; ++b)
                all[n][b] = rr < rows ? gld_l2(reinterpret_cast<const uint4 *>(
                                            q + (b >> 1) * 64 + (b & 1) * 8))
                                      : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int n = 0; n < C::NT; ++n) {
            uint4(&v)[DH / 32] = all[n];
            uint32_t most = 0;
#pragma unroll
            for (int b = 0; b < DH / 32; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t w = word_of(v[b], e);
                    most = max(most, max(w & 0x7FFFu, w >> 16 & 0x7FFFu));
                }
            most = max(most, __shfl_xor_sync(~0u, most, 1));
            most = max(most, __shfl_xor_sync(~0u, most, 2));
            const uint32_t e = max(most >> 7, 32u);  // the largest's exponent, biased by 127
            const float to = __uint_as_float((268 - e) << 23);  // 2^(14 - (e - 127))
            const float u = __uint_as_float((e - 14) << 23) * a.scale_log2;
            unit[n] = f2_make(__shfl_sync(~0u, u, 8 * c), __shfl_sync(~0u, u, 8 * c + 4));
#pragma unroll
            for (int b = 0; b < DH / 32; ++b)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t two = word_of(v[b], w);
                    qf[n][b * 2 + w / 2][w % 2] = pack_f16(bf16_lo(two) * to, bf16_hi(two) * to);
                }
        }
    }
};

// o += P V over a warp's keys, of each row only the keys it sees; z[n][2 h + x]: the weights' logarithms
// of the key at place g + 8 x of 16, half h.
template <typename C>
__device__ __forceinline__ void product_one_by_one8(const AttnArgs &a, int least, Rows8<C> &r,
                                                    const f32x2 (&z)[C::NT][2 * C::KH], uint32_t v,
                                                    const Lane8<C> &at, int key0) {
    int see[C::NT][2];
#pragma unroll
    for (int n = 0; n < C::NT; ++n)
#pragma unroll
        for (int p = 0; p < 2; ++p) see[n][p] = r.see(a, least, n, p);
#pragma unroll 1
    for (int k = 0; k < 16 * C::KH; ++k) {
        const int g = (k >> 3 & 1) * 4 + (k & 1) * 2 + (k >> 2 & 1);  // of the lanes that hold key k
        const int x = (k >> 4) * 2 + (k >> 1 & 1);
        float w[C::NT][2];
#pragma unroll
        for (int n = 0; n < C::NT; ++n) {
            f32x2 mine = z[n][0];
#pragma unroll
            for (int i = 1; i < 2 * C::KH; ++i)
                if (i == x) mine = z[n][i];
            f2_split(mine, w[n][0], w[n][1]);
#pragma unroll
            for (int p = 0; p < 2; ++p) w[n][p] = ex2(__shfl_sync(~0u, w[n][p], 4 * g + at.c));
        }
#pragma unroll
        for (int j = 0; j < C::kDh / 16; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t code;
                asm volatile("ld.shared.u8 %0, [%1];"
                             : "=r"(code)
                             : "r"(v + at.at(k, j) + 8 * h + at.g)
                             : "memory");
                const float y = f16_lo(e4m3x2_f16x2(code));
#pragma unroll
                for (int n = 0; n < C::NT; ++n)
#pragma unroll
                    for (int p = 0; p < 2; ++p)
                        if (key0 + k < see[n][p])
                            r.o[n][j][2 * h + p] = fmaf(w[n][p], y, r.o[n][j][2 * h + p]);
            }
    }
}

// f(j, h, a) for the 16 x 16 blocks of a warp's V: columns 16 j of its 16 keys h, as a product's first
// operand. They come two at a time: both halves of 16 columns, or 32 columns. `live`: with some, the
// lane's keys inside the sequence, a byte each (codes past it may be NaN, which a weight of 0 would not
// silence).
template <typename C, typename F>
__device__ __forceinline__ void each_v_block8(uint32_t v_at, bool some, const uint32_t (&live)[C::KH],
                                              F &&f) {
    constexpr int KH = C::KH;
#pragma unroll
    for (int u = 0; u < KH * C::kDh / 32; ++u) {
        uint32_t w[4];
        ldsm2_t8(w, v_at ^ u * (KH == 2 ? 16 : 32));
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int h = KH == 2 ? x : 0, j = KH == 2 ? u : 2 * u + x;
            uint32_t w0 = w[2 * x], w1 = w[2 * x + 1];
            if (some) {
                w0 &= live[h];
                w1 &= live[h];
            }
            const uint32_t a[4] = {e4m3x2_f16x2(w0), e4m3x2_f16x2(w1), e4m3x2_f16x2_hi(w0),
                                   e4m3x2_f16x2_hi(w1)};
            f(j, h, a);
        }
    }
}

// What rounding to f16 took from the weights below kLeast, times V: each pass takes a row's largest rest
// and those within 2^-28 of it, times a power of two that takes it to 2^14, and the sums back. A row
// that has none, or none left, gets zeros, so that no row depends on another. Down to 2^-112, 2^-125
// of the row's largest weight. With two row tiles of 128 it is a call, which keeps the registers that it
// takes out of the tile's usual way: 72 sequences of 5 drafts by 2 x 7 heads 28.1 us, 29.7 without. Of 64
// it is not: 128 of 500-1500 tokens by 8 drafts 67 both, and 72.3 us for 75.5 where it has work (queries
// three times as large).
template <typename C>
struct Small8 {
    float o[C::NT][C::kDh / 16][4];
    f32x2 z[C::NT][2 * C::KH];  // the weights' logarithms, of the key at place g + 8 x of half h: 2 h + x
    uint32_t live[C::KH];
};
template <typename C>
__device__ __forceinline__ void small_weights8(Small8<C> &r, uint32_t v_at, bool some) {
    constexpr int KH = C::KH;
#pragma unroll
    for (int n = 0; n < C::NT; ++n) {  // one after the other, which takes fewer registers
        float rest[2 * KH][2];
#pragma unroll
        for (int x = 0; x < 2 * KH; ++x) {
            float e[2];
            f2_split(r.z[n][x], e[0], e[1]);
            e[0] = ex2(e[0]);
            e[1] = ex2(e[1]);
            const uint32_t two = pack_f16(e[0], e[1]);
            rest[x][0] = e[0] < kLeast ? e[0] - f16_lo(two) : 0.0f;
            rest[x][1] = e[1] < kLeast ? e[1] - f16_hi(two) : 0.0f;
        }
#pragma unroll 1
        for (int pass = 0; pass < 4; ++pass) {  // 4 x 28 powers of two
            float up[2], down[2];
            bool any = false;
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                float t = 0.0f;
#pragma unroll
                for (int x = 0; x < 2 * KH; ++x) t = fmaxf(t, fabsf(rest[x][p]));
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) t = fmaxf(t, __shfl_xor_sync(~0u, t, x));
                const uint32_t e = __float_as_uint(t) & 0x7F800000u;  // of 2^-112 .. 2^-17
                const bool has = t >= 0x1p-112f;
                any |= has;
                up[p] = has ? __uint_as_float((254u + 14u << 23) - e) : 0.0f;
                down[p] = has ? __uint_as_float(e - (14u << 23)) : 0.0f;
            }
            if (!__any_sync(~0u, any)) break;
            uint32_t pf[2 * KH];
#pragma unroll
            for (int x = 0; x < 2 * KH; ++x) {
                float e[2];
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const float w = rest[x][p] * up[p];
                    const bool take = fabsf(w) >= 0x1p-14f;
                    e[p] = take ? w : 0.0f;
                    if (take) rest[x][p] = 0.0f;
                }
                pf[x] = transposed(pack_f16(e[0], e[1]));
            }
            float d[4];
            each_v_block8<C>(v_at, some, r.live, [&](int j, int h, const uint32_t(&a)[4]) {
                if (h == 0) d[0] = d[1] = d[2] = d[3] = 0.0f;
                mma16816_f16(d, a, pf[2 * h], pf[2 * h + 1]);
                if (h < KH - 1) return;
#pragma unroll
                for (int e = 0; e < 4; ++e) r.o[n][j][e] = fmaf(d[e], down[e & 1], r.o[n][j][e]);
            });
        }
    }
}

template <typename C>
__device__ __noinline__ void small_weights8_call(Small8<C> &r, uint32_t v_at, bool some) {
    small_weights8<C>(r, v_at, some);
}

// One tile's part of a warp: its rows by its keys (from key key0 on), behind the `walked` that it has
// seen of the item.
template <typename C>
__device__ __forceinline__ void tile8(const AttnArgs &args, uint32_t k, uint32_t scales,
                                      const Lane8<C> &at, int hh, int group0, int key0, int len,
                                      int least, int walked, Rows8<C> &r) {
    constexpr int DH = C::kDh, NT = C::NT, KH = C::KH, kKeys = 16 * KH, kG = C::KT / 8;
    const int lane = threadIdx.x & 31;
    const uint32_t v = k + C::kV;
    f32x2 s[NT][2 * KH];  // s[n][2 h + x]: key at place g + 8 x of 16, half h
#pragma unroll
    for (int h = 0; h < KH; ++h) {
        float d[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) d[n][e] = 0.0f;
#pragma unroll
        for (int b = 0; b < DH / 64; ++b) {
            const uint4 w0 = lds16(k + (at.k_at[0] ^ b * 64) + h * 16 * C::kRow);
            const uint4 w1 = lds16(k + (at.k_at[1] ^ b * 64) + h * 16 * C::kRow);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t a[4] = {
                    e4m3x2_f16x2(word_of(w0, j)), e4m3x2_f16x2(word_of(w1, j)),
                    e4m3x2_f16x2_hi(word_of(w0, j)), e4m3x2_f16x2_hi(word_of(w1, j))};
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    mma16816_f16(d[n], a, r.qf[n][4 * b + j][0], r.qf[n][4 * b + j][1]);
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            s[n][2 * h] = f2_make(d[n][0], d[n][1]);
            s[n][2 * h + 1] = f2_make(d[n][2], d[n][3]);
        }
    }
    const bool some = key0 + kKeys > least;  // some row does not see some of these keys
    float top[NT][2], inverse[KH];
#pragma unroll
    for (int n = 0; n < NT; ++n) top[n][0] = top[n][1] = -INFINITY;
#pragma unroll
    for (int h = 0; h < KH; ++h) {  // the lane's keys of each 16 share their scales
        const int group = group0 + 2 * h + (at.g >> 2);
        uint32_t four = scales + group * 16 + hh * 4, four_v = four + 16 * kG;
        if constexpr (C::kHeads != 4) {  // TileScales8: four[2][kG], then at[2][kG]
            const uint32_t which = scales + 32 * kG + group * 4;
            four += lds4(which) * 4;
            four_v += lds4(which + 4 * kG) * 4;
        }
        const float kb = __uint_as_float(scale_bits(lds4(four)));
        const uint32_t vb = scale_bits(lds4(four_v));
        const float add = (float)((int)(vb >> 23) - 127);
        inverse[h] = __uint_as_float(inverse_bits(vb));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const f32x2 unit = f2_mul(r.unit[n], f2_make(kb, kb));
            float y[2][2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                s[n][2 * h + x] = f2_fma(s[n][2 * h + x], unit, f2_make(add, add));
                f2_split(s[n][2 * h + x], y[x][0], y[x][1]);
            }
#pragma unroll
            for (int p = 0; p < 2; ++p) top[n][p] = max3(top[n][p], y[0][p], y[1][p]);
        }
    }
    if (some) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int see[2] = {r.see(args, least, n, 0), r.see(args, least, n, 1)};
            top[n][0] = top[n][1] = -INFINITY;
#pragma unroll
            for (int x = 0; x < 2 * KH; ++x) {
                float y[2];
                f2_split(s[n][x], y[0], y[1]);
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    if (key0 + 16 * (x >> 1) + at.key + 2 * (x & 1) >= see[p]) y[p] = -INFINITY;
                    top[n][p] = fmaxf(top[n][p], y[p]);
                }
                s[n][x] = f2_make(y[0], y[1]);
            }
        }
    }
    // Only when some score passes its row's maximum by kRescale8 are the row maxima needed. A row that
    // has seen no key yet keeps its offset and sums of zero.
    bool rise = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float off[2];
        f2_split(r.off[n], off[0], off[1]);
#pragma unroll
        for (int p = 0; p < 2; ++p) rise |= top[n][p] + off[p] > kTop8 + kRescale8;
    }
    if (__any_sync(~0u, rise)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float f[2], h[2], off[2];
            f2_split(r.off[n], off[0], off[1]);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                float t = top[n][p];
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) t = fmaxf(t, __shfl_xor_sync(~0u, t, x));
                const float was = off[p];
                if (t + was > kTop8 + kRescale8) off[p] = kTop8 - t;
                f[p] = ex2(off[p] - was);
                h[p] = ex2(0.5f * (off[p] - was));  // f may be below fp32's numbers where l counts
            }
            r.off[n] = f2_make(off[0], off[1]);
            r.l[n] = f2_mul(f2_mul(r.l[n], f2_make(h[0], h[1])), f2_make(h[0], h[1]));
#pragma unroll
            for (int j = 0; j < DH / 16; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) r.o[n][j][e] *= f[e & 1];
        }
    }
    uint32_t pf[NT][2 * KH];  // the weights as the second product's second operand
    float low = INFINITY;     // the least weight's logarithm
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 2 * KH; ++x) {
            s[n][x] = f2_add(s[n][x], r.off[n]);
            float e0, e1;
            f2_split(s[n][x], e0, e1);
            low = min3(low, e0, e1);
            e0 = ex2(e0);
            e1 = ex2(e1);
            r.l[n] = f2_fma(f2_make(e0, e1), f2_make(inverse[x >> 1], inverse[x >> 1]), r.l[n]);
            pf[n][x] = transposed(pack_f16(e0, e1));
        }
    if (some) {  // of those that there are
        low = INFINITY;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < 2 * KH; ++x) {
                float z[2];
                f2_split(s[n][x], z[0], z[1]);
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    if (z[p] > -INFINITY) low = fminf(low, z[p]);
            }
    }
    const bool small = __any_sync(~0u, low < kLeastLog2);  // some weight is
    if (small && __any_sync(~0u, low < -126.0f)) {
        // A weight that 32 bits do not hold, beside a V scale so much larger, counts in the sum all the
        // same: 2^z / vs.
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float l[2];
            f2_split(r.l[n], l[0], l[1]);
#pragma unroll
            for (int x = 0; x < 2 * KH; ++x) {
                const float over_vs = (float)((int)(__float_as_uint(inverse[x >> 1]) >> 23) - 127);
                float z[2];
                f2_split(s[n][x], z[0], z[1]);
#pragma unroll
                for (int p = 0; p < 2; ++p)
                    if (ex2(z[p]) == 0.0f) l[p] = fmaf(ex2(z[p] + over_vs + 32.0f), 0x1p-32f, l[p]);
            }
            r.l[n] = f2_make(l[0], l[1]);
        }
    }
    uint32_t live[KH] = {};  // the lane's keys inside the sequence, a byte each
    if (some) {
        // A draft that some row does not see: were its V NaN, a weight of 0 would not keep it
        // from that row, so the product is made one by one.
        bool nan = false;
        const int from = max(least - key0, 0), to = min(len - key0, kKeys);
        for (int x = lane; x < (to - from) * (DH / 16); x += 32) {
            const uint4 w = lds16(v + at.at(from + x / (DH / 16), x % (DH / 16)));
#pragma unroll
            for (int e = 0; e < 4; ++e)
                nan |= (((word_of(w, e) & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
        }
        if (__any_sync(~0u, nan)) {
            product_one_by_one8<C>(args, least, r, s, v, at, key0);
            return;
        }
#pragma unroll
        for (int h = 0; h < KH; ++h) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (key0 + 16 * h + at.key_of(2 * at.c + (i & 1) + 4 * (i & 2)) < len)
                    live[h] |= 0xFFu << 8 * i;
        }
    }
    each_v_block8<C>(v + at.v_at, some, live, [&](int j, int h, const uint32_t(&a)[4]) {
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816_f16(r.o[n][j], a, pf[n][2 * h], pf[n][2 * h + 1]);
    });
    if (!small) return;
    // f16 takes 2^-25 of a small weight at most, and a code is 448 at most: a row in which every sum is
    // past that of all keys so far times 2^10 loses, in all, 2^-10 of sum w |v| at most, channel by
    // channel. The others take what was lost.
    const float enough = (float)(walked + kKeys) * 0x1p-6f;
    float least_o[NT][2], least_all = INFINITY;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            least_o[n][p] = INFINITY;
#pragma unroll
            for (int j = 0; j < DH / 16; ++j)
                least_o[n][p] = min3(least_o[n][p], fabsf(r.o[n][j][p]), fabsf(r.o[n][j][2 + p]));
        }
        least_all = min3(least_all, least_o[n][0], least_o[n][1]);
    }
    if (__any_sync(~0u, least_all < enough)) {
        Small8<C> x;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            bool take[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) {  // some lane's, of the row's
                float t = least_o[n][p];
#pragma unroll
                for (int y = 4; y < 32; y <<= 1) t = fminf(t, __shfl_xor_sync(~0u, t, y));
                take[p] = t < enough;
            }
#pragma unroll
            for (int j = 0; j < DH / 16; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) x.o[n][j][e] = r.o[n][j][e];
#pragma unroll
            for (int e = 0; e < 2 * KH; ++e) {
                float z[2];
                f2_split(s[n][e], z[0], z[1]);
                x.z[n][e] = f2_make(take[0] ? z[0] : 0.0f, take[1] ? z[1] : 0.0f);
            }
        }
#pragma unroll
        for (int h = 0; h < KH; ++h) x.live[h] = live[h];
        if constexpr (NT > 1 && DH == 128)
            small_weights8_call<C>(x, v + at.v_at, some);
        else
            small_weights8<C>(x, v + at.v_at, some);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < DH / 16; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) r.o[n][j][e] = x.o[n][j][e];
    }
}

// A consumer warp's part of k_own over an 8-bit cache.
template <typename C>
__device__ __forceinline__ void consume8(const AttnArgs &a, int rows, const OwnSmem<C> &s) {
    constexpr int DH = C::kDh, ST = C::kStages, QB = C::kQBufs, KG = C::KG, WR = C::WR, NT = C::NT;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kw = warp % KG, rg = warp / KG % C::RG, hh = warp / (KG * C::RG);
    const Lane8<C> at(hh, kw * 16 * C::KH);
    uint32_t ring_at = 0, ring_phase = 0;
    bool dead = false;
    for (uint32_t items = 0;; ++items) {
        const uint32_t qb = items % QB;
        const bool ready = !dead && mbar_wait_bounded(&s.qfull[qb], (items / QB) & 1u);
        // Where key groups join, the warps go on together or not at all: none waits at a
        // barrier the others left.
        if (KG > 1 ? named_or(1, 32 * C::kWarps, !ready) : !ready) {
            if (!ready && !dead) raise_error(SC_DEV_TIMEOUT);
            return;
        }
        const OwnItem item = s.item[qb];
        if (item.n == 0) return;
        const int len = item.len, least = len - a.D + 1;  // keys that every row sees
        const int row0 = item.rt * C::MR + rg * WR;       // of the sequence's rows of a head
        Rows8<C> r;
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.qempty[qb]);
        r.load(a, item.i, item.h + hh, row0, rows);
        if (NT == 1)
#pragma unroll
            for (int p = 0; p < 2; ++p) r.sees[p] = r.find_see(a, least, 0, p);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            r.l[n] = f2_make(0.0f, 0.0f);
            r.off[n] = f2_make(kUnseen8, kUnseen8);
#pragma unroll
            for (int j = 0; j < DH / 16; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) r.o[n][j][e] = 0.0f;
        }
        bool bad = false;
        const int from = prefix_keys(a, len);
        int key0 = from + item.t0 * C::KT + kw * 16 * C::KH;
        for (int t = 0; t < item.n; ++t, key0 += C::KT) {
            // A wait that gave up is the last one: no more tiles, since what describes one (its scales'
            // places are offsets) may be anything, and no rows written.
            if (!dead && !mbar_wait_bounded(&s.full[ring_at], ring_phase)) {
                raise_error(SC_DEV_TIMEOUT);
                dead = bad = true;
            }
            if (!dead) {
                bad |= s.bad[ring_at] != 0;
                tile8<C>(a, s.ring_a + ring_at * C::kStage, smem_addr(&s.scales[ring_at]), at, hh,
                         kw * 2 * C::KH, key0, len, least, t * 16 * C::KH, r);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.empty[ring_at]);
            if (++ring_at == ST) {
                ring_at = 0;
                ring_phase ^= 1u;
            }
        }
        const bool whole = item.n == item.T && from == 0;  // nothing to join with
        float *part = a.own_part + ((int64_t)(item.w + blockIdx.x) * C::kHeads + hh) * C::kSlot;
        bf16 *out = a.out + ((int64_t)item.i * a.D * a.Hkv + item.h + hh) * a.G * DH;
        auto out_row = [&](int rr) {
            return out + ((int64_t)(rr / a.G) * a.Hkv * a.G + rr % a.G) * DH;
        };
        // A NaN maximum marks a part with a bad page or a lost tile: k_merge leaves its rows alone.
        auto put_part = [&](int row, int col, float x) {
            gst(part + (rg * WR + row) * DH + col, x);
        };
        auto put_sums = [&](int row, float m, float l) {
            gst(part + C::MR * DH + rg * WR + row, bad ? __int_as_float(0x7FC00000) : m);
            gst(part + C::MR * DH + C::MR + rg * WR + row, l);
        };
        auto inverse_of = [](float l) { return l > 0.0f ? 1.0f / l : l == 0.0f ? 0.0f : l; };
        [[maybe_unused]] float *jm = s.join + C::kWarps * WR * C::kOs;  // [warp][m, l]
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float l[2], m[2], inv[2];
            f2_split(r.l[n], l[0], l[1]);
            f2_split(r.off[n], m[0], m[1]);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[p] += __shfl_xor_sync(~0u, l[p], x);
                inv[p] = inverse_of(l[p]);
                m[p] = m[p] == kUnseen8 ? -INFINITY : -m[p];
            }
            const int row = n * 8 + 2 * at.c;  // and the next
            if (KG > 1 || !whole) {
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    if (KG == 1 && row0 + row + p >= rows) continue;
#pragma unroll
                    for (int j = 0; j < DH / 16; ++j)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int col = 16 * j + 8 * h + at.g;
                            const float x = r.o[n][j][2 * h + p];
                            if constexpr (KG > 1)
                                s.join[(warp * WR + row + p) * C::kOs + col] = x;
                            else
                                put_part(row + p, col, x);
                        }
                    if (at.g != 0) continue;
                    if constexpr (KG > 1) {
                        jm[warp * 2 * WR + row + p] = m[p];
                        jm[(warp * 2 + 1) * WR + row + p] = l[p];
                    } else {
                        put_sums(row + p, m[p], l[p]);
                    }
                }
            } else {
                // Pairs of rows become pairs of columns: lane 4 g + c has row g's.
                const int rr = row0 + n * 8 + at.g;
                const bool mine = rr < rows && !bad;
                bf16 *to = out_row(min(rr, rows - 1)) + 2 * at.c;
#pragma unroll
                for (int j = 0; j < DH / 16; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t two =
                            transposed(pack_bf16(r.o[n][j][2 * h] * inv[0],
                                                 r.o[n][j][2 * h + 1] * inv[1]));
                        if (mine) gst(reinterpret_cast<uint32_t *>(to + 16 * j + 8 * h), two);
                    }
            }
        }
        if constexpr (KG > 1) {
            // The key groups of a head and row group join: a thread four columns of a row.
            // (The next join comes after the next item's barrier.)
            bad = named_or(1, 32 * C::kWarps, bad);
            const int w0 = warp - kw;
            for (int x = kw * 32 + lane; x < WR * DH / 4; x += 32 * KG) {
                const int row = x / (DH / 4), col = x % (DH / 4) * 4, rr = row0 + row;
                float top = -INFINITY, sum = 0.0f;
#pragma unroll
                for (int q = 0; q < KG; ++q) top = fmaxf(top, jm[(w0 + q) * 2 * WR + row]);
                const float off = top == -INFINITY ? 0.0f : top;
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int q = 0; q < KG; ++q) {
                    const float m = jm[(w0 + q) * 2 * WR + row] - off, f = ex2(m);
                    const float4 u = *reinterpret_cast<float4 *>(
                        s.join + ((w0 + q) * WR + row) * C::kOs + col);
                    sum = add_times_2_to(sum, jm[((w0 + q) * 2 + 1) * WR + row], m, f);
                    v.x = fmaf(f, u.x, v.x);
                    v.y = fmaf(f, u.y, v.y);
                    v.z = fmaf(f, u.z, v.z);
                    v.w = fmaf(f, u.w, v.w);
                }
                if (rr >= rows) continue;
                if (!whole) {
                    gst(reinterpret_cast<float4 *>(part + (rg * WR + row) * DH + col), v);
                    if (col == 0) put_sums(row, top, sum);
                } else if (!bad) {
                    const float inv = inverse_of(sum);
                    gst(reinterpret_cast<uint2 *>(out_row(rr) + col),
                        make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv)));
                }
            }
        }
    }
}

// The shared prefix as bf16 [keys, Hkv, Dh], for k_prefix: every key is read by many row tiles, so
// it is unpacked once, and stays in L2. Exact: a code has 4 bits, a scale none. 16384 tokens of 8 x 64
// (50 MB read and written): 12 us; 2976 of 2 x 128: 5.5, a chain of dependent reads. Converting in k_prefix
// instead, by four warps more between the copies and the products, took a step of 128 x 8 drafts behind
// 16384 tokens from 188 to 315 us, and 37 x 3 behind 2976 from 28.6 to 35: each row tile converts again.
constexpr int kUnpackThreads = 256;
constexpr int kUnpackWords = 2;  // of each pool, of a lane at once
static __global__ void __launch_bounds__(kUnpackThreads, 4)
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
    // A warp takes a key at a time, eight codes of K and of V a lane; the next key's are on their way.
    const int per = a.Hkv * Dh / 8, lp = __ffs(a.pt.page_size) - 1, bl = a.s8.block_log2;
    const int warps = gridDim.x * (kUnpackThreads / 32);
    for (int w0 = 0; w0 < per; w0 += 32 * kUnpackWords) {
        struct Batch {
            uint2 k[kUnpackWords], v[kUnpackWords];
            uint32_t ks[kUnpackWords], vs[kUnpackWords];
        };
        int head[kUnpackWords];
#pragma unroll
        for (int q = 0; q < kUnpackWords; ++q) head[q] = (w0 + 32 * q + (tid & 31)) * 8 / Dh;
        auto load = [&](Batch &b, int t) {
            const int id = gld_l2(row + (t >> lp));
            // A bad page is k_prefix's to report; its part counts for nothing.
            const int page = id < 0 || id >= a.pt.n_pages ? 0 : id;
            const int64_t at = ((int64_t)page << lp) + (t & (a.pt.page_size - 1));
#pragma unroll
            for (int q = 0; q < kUnpackWords; ++q) {
                const int x = w0 + 32 * q + (tid & 31);
                if (x >= per) continue;
                b.k[q] = gld(reinterpret_cast<const uint2 *>(k) + at * per + x);
                b.v[q] = gld(reinterpret_cast<const uint2 *>(v) + at * per + x);
                const int64_t s = (at >> bl) * a.Hkv + head[q];
                b.ks[q] = gld(reinterpret_cast<const uint32_t *>(a.s8.k) + s);
                b.vs[q] = gld(reinterpret_cast<const uint32_t *>(a.s8.v) + s);
            }
        };
        auto put = [&](const Batch &b, int t) {
#pragma unroll
            for (int q = 0; q < kUnpackWords; ++q) {
                const int x = w0 + 32 * q + (tid & 31);
                if (x >= per) continue;
                const int64_t to = ((int64_t)t * per + x) * 8;
                st_plain(k16 + to, e4m3_bf16x8(b.k[q], scale_bits(b.ks[q])));
                st_plain(v16 + to, e4m3_bf16x8(b.v[q], scale_bits(b.vs[q])));
            }
        };
        Batch even, odd;
        int t = blockIdx.x * (kUnpackThreads / 32) + (tid >> 5);
        if (t < a.shared_keys) load(even, t);
        while (t < a.shared_keys) {
            const int next = t + warps;
            if (next < a.shared_keys) load(odd, next);
            put(even, t);
            t = next;
            if (t >= a.shared_keys) break;
            if (t + warps < a.shared_keys) load(even, t + warps);
            put(odd, t);
            t += warps;
        }
    }
}

// Bytes of the unpacked K, or V.
static size_t unpacked_bytes(const AttnShape &s, int page_size) {
    return (size_t)s.shared_pages * page_size * s.Hkv * s.Dh * 2;
}

static cudaError_t launch_unpack(const AttnArgs &a, const AttnShape &s, const void *k, const void *v,
                                 bf16 *k16, bf16 *v16, int sm_count, cudaStream_t stream) {
    const int blocks = (a.shared_keys + kUnpackThreads / 32 - 1) / (kUnpackThreads / 32);
    const int most = 4 * sm_count;
    return launch_pdl(k_unpack, dim3((unsigned)(blocks < most ? blocks : most)),
                      dim3(kUnpackThreads), 0, stream, a, (const unsigned char *)k,
                      (const unsigned char *)v, s.Dh, k16, v16);
}

}  // namespace sc
