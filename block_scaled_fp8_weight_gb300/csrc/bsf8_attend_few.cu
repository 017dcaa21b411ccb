// bsf8_attend_few.cu -- attention over the paged block-scaled fp8 cache for up to 8 rows (a row is a
// (node, query head) of one request and cache head) at dim 128 and long contexts: single tokens.
//
// The formula, the cut of the work into items and the join are those of bsf8_attend.cu.  What differs
// is that keys and channels, not rows, fill the MMA's 128 lanes, and that the cached codes enter
// both products as they are:
//   S^T = K Q^T   A: a tile's 128 keys x 128 channels of codes, with their exponents as the scales
//                 of a block-scaled MMA.  B: each row of Q as the sum of two e4m3 parts, the parts as
//                 two columns with scales 2^eq and 2^(eq - 4); softmax adds them (fp32).
//   O^T += V^T P  A: the tile's codes again, 128 channels x 128 keys.  A value's exponent belongs to
//                 a key and 32 channels, so it goes into P: for each of the four channel blocks c a
//                 copy p 2^(e(key, c) - E), E the segment's largest exponent so far (0 where that power is
//                 below 2^-24, f16's smallest).  Lane quarter c of O^T is right in the columns of copy c
//                 only, and only those are read.  Each copy
//                 is the sum of four e4m3 parts (p = 2^(x - m), rounded to f16's 11 bits first, whole
//                 where it is above 2^-12, to 2^-35 below that), in columns of their own: 16 columns a row.
//                 (Three parts, to 2^-24 of p, lost what a channel holds where the key of the largest p has
//                 a zero; they took 182 us where four take 185.)
// So nothing is widened, and an SM's shared memory moves about 90 KB a tile (144 KB in bsf8_attend.cu)
// while HBM moves 33.
//
// Warps: a producer of keys (codes, both kinds of exponents), one of values (codes, and a segment's Q,
// which so comes tiles ahead); one for each product; three sets of four for the softmax, tile about,
// thread = key.  The rows' references m and the value exponent E are common
// to a tile's keys.  A set's warps exchange their largest exponents and whether any x passes the m that
// the set knows by more than 2.8; then the set takes the tile before's number of changes of m and E, and
// only where that is new, or an x did pass (a segment's first tiles, as a rule), forms new maxima and
// rescales O.  Sums stay with the thread, in fp32, to the segment's end.  O and Q are double-buffered
// by segment.
//
// Keys that do not exist or hold a NaN block: p is 0 there, and the key's thread clears their value
// codes first, as 0 times a NaN code is not 0.
//
// Bound: HBM at long contexts.  A tile of 128 keys takes an SM 1440 cycles at its share of the measured
// HBM rate, which is what it takes here; three sets (of the softmax's 3600 cycles a tile, latencies
// mostly) keep up with that, two did not.  64 requests of 70 to 16384 tokens (559097 keys), 4 rows, 8 heads: 183
// us in a graph with the join, 6.45 TB/s, 0.95 of the measured HBM rate.  At short contexts latency
// bounds: one request of 1000 tokens, a tile a block, takes 13 us -- prefix sums 2, table, codes and Q
// 2.5, products and softmax 2, output 1.5, the join 3, launches 2.
#include "bsf8_attend.cuh"

namespace bsf8 {

namespace {

constexpr int ROWS = kFewRows;
constexpr int kFewK = 0, kFewV = 1, kFewS = 2, kFewO = 3;  // then the sets
// Tiles whose value exponents and flags are kept: the keys' producer fills an entry again eight tiles
// later, once the S of the tile four later is done, which takes the place of this tile's or a later one's
// S, thus after the softmax has read that.
constexpr int kRing = 8;
constexpr float kFewBias = 13.0f;     // p = 2^(x - m + kFewBias); P holds p / 2^7
constexpr float kFewSlack = 2.8f;     // m lags the maximum by at most this: p / 2^7 <= 2^8.8 < 448, e4m3's largest
constexpr float kUnseen = 3.4028235e38f;  // bias - m of a row that has seen nothing: any x passes it

struct FewShape {
    static constexpr int DIM = 128, RT = ROWS, TN = 128, EB = 4, SLOT = TN * DIM, NSLOT = 4;
    static constexpr int SETS = 3, THREADS = (4 + 4 * SETS) * 32;
    static constexpr int START = kFewStart;
    static constexpr int NS = 4;                          // buffers of S
    static constexpr int NQ = 2 * ROWS, NP = 16 * ROWS;   // columns of S, of O
    static constexpr int PBUF = TN * NP;                  // a key's row of P: 128 bytes
    static_assert(NP == 128);
    // tensor memory columns: two O, S, scales of two tiles' keys and of two segments' rows
    static constexpr int CO = 0, CS = 2 * NP, CB = CS + NS * NQ, CA = CB + 8;
    static_assert(CA + 8 <= 512);
    static constexpr int oK = 0, oRing = NSLOT * SLOT, oP = 2 * NSLOT * SLOT, oQ = oP + SETS * PBUF;
    static constexpr int QBUF = 4096, oQs = oQ + 2 * QBUF;
    // a slot's key exponents, as tensor memory wants them and as they come; the values' as they come
    static constexpr int oExp = oQs + 2 * 512, oVex = oExp + NSLOT * 1024, oPrefix = oVex + kRing * 512;
};

struct FewShared : BlockShared {
    uint64_t k_full[4], k_free[4];    // ring slots of keys: codes and exponents landed; multiplied
    uint64_t c_full[4], c_free[4];    // of values
    uint64_t s_full[4], s_free[4];    // S written; read
    uint64_t p_full[3];               // a set's P written, O rescaled
    uint64_t pv_done[3];              // O updated, P and the values read
    uint64_t m_full[4];               // a tile (of four) has its references
    uint64_t vote[3];                 // a set's warps
    uint64_t q_full[2], q_free[2];    // a segment's Q written; multiplied
    uint64_t l_full[2], o_full[2];    // a segment's sums written; its last product done
    uint64_t o_free[2];               // its output read
    // The references: bias - m, by their number in the segment, and a tile's number and E.  Four of each: a
    // set that has not yet read a tile's keeps the third tile after that, its own next, from its vote.
    alignas(16) float off[4][ROWS];
    int2 ref[4];
    alignas(16) int grow[3][2][4];    // votes
    float most[3][4][ROWS];           // a warp's largest S
    float sum[2][12][ROWS], soff[2][3][ROWS];  // by the parity of the segment: sums, their bias - m
    // Rows that see a NaN of a channel block, by segment: while a set writes out a segment, the others pass
    // at most two more tiles, thus segments.
    int nan[4][4][ROWS];
    int valid[kRing];                 // a tile's 16-key groups that exist (bit i)
    int pages[2][2][32];              // the producers' block table entries: of a batch, of the next
};

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// A batch of tiles' boxes (box_rows keys, inside a page and a tile), one a lane: 32 / boxes tiles.
// The table's entries come by cp.async, a batch ahead.
struct Batch {
    int *ring;   // [2][32]
    int first;   // the lane's first 16-key group in the batch
    int phase;

    // exact: group * (magic * d - 2^32) < 2^32 for groups below 2^26 and d <= 64
    static __device__ __forceinline__ int in_page(const AttendParams &p, int grp) {
        return (int)(((unsigned long long)(unsigned)grp * p.page_magic) >> 32);
    }
    __device__ __forceinline__ void ask(const AttendParams &p, const Segment &g, int tile, int lane) {
        const int grp = 8 * tile + first;
        int *const at = ring + 32 * phase + lane;
        if (16 * grp < g.ctx + g.nodes)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(at)),
                         "l"(p.c.table + table_row(p, g) + in_page(p, grp))
                         : "memory");
        asm volatile("cp.async.commit_group;" ::: "memory");  // exponents asked for later are not waited for in rows()
        phase ^= 1;
    }
    // The cache rows (head h) of the batch asked for last, -1 where there are none.
    __device__ __forceinline__ int rows(const AttendParams &p, const Segment &g, int tile, int lane) {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        const int grp = 8 * tile + first, page = ring[32 * (phase ^ 1) + lane];
        if (16 * grp >= g.ctx + g.nodes) return -1;
        if ((unsigned)page >= (unsigned)p.c.pages) {
            report_index(p.status);
            return -1;
        }
        return (page * p.c.heads + g.h - in_page(p, grp)) * p.c.page_size + 16 * grp;
    }
};

// A segment's rows of Q, by a warp, eight lanes a row.  Each row scaled by a power of two 2^-eq so that
// its largest lies in [2^7, 2^8), as the sum of two e4m3 parts, the lower one times 2^4.  Exact for
// bf16 values within 2^14 of the row's largest, else off by at most 2^-22 of that.
__device__ __forceinline__ void put_q(const AttendParams &p, const Segment &g, uint8_t *qb, uint32_t *sc, int lane) {
#pragma unroll 1
    for (int r0 = 0; r0 < ROWS; r0 += 4) {
        const int row = r0 + (lane >> 3), u = lane & 7;
        uint4 v[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (row < g.nodes * p.g) {  // one row tile holds all rows
            const int t = row / p.g, hq = g.h * p.g + row - t * p.g;
            const uint4 *q =
                reinterpret_cast<const uint4 *>(p.q + ((size_t)g.b * p.T + t) * p.ldq + (size_t)hq * 128 + 16 * u);
            v[0] = q[0];
            v[1] = q[1];
        }
        const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
        uint32_t am = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) am = max(am, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
#pragma unroll
        for (int k = 1; k < 8; k <<= 1) am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, k));
        const int eq = max((int)(am >> 7) - 127 - 7, -100);  // at most 121
        // A row with an infinity or a NaN becomes NaN as a whole, as its scores are (the conversion to
        // e4m3 would make an infinity its largest value).
        const float qs = am >= 0x7F80u ? __uint_as_float(0x7FC00000u) : pow2i(-eq);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t x = pack_f16(__uint_as_float(w[j] << 16) * qs, __uint_as_float(w[j] & 0xFFFF0000u) * qs);
            const uint32_t h2 = f16_to_e4m3(x);
            const uint32_t l2 = f16_to_e4m3(f16x2_mul(f16x2_sub(x, e4m3_to_f16((uint16_t)h2)), 0x4C004C00u));
            hi[j >> 1] = j & 1 ? hi[j >> 1] | (h2 << 16) : h2;
            lo[j >> 1] = j & 1 ? lo[j >> 1] | (l2 << 16) : l2;
        }
        // rows of 128 bytes, 128-byte swizzle (ROWS is a multiple of 8)
        uint8_t *const d = qb + row * 128 + ((u ^ (row & 7)) << 4);
        *reinterpret_cast<uint4 *>(d) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4 *>(d + ROWS * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        if (u == 0) {  // the scales of columns row and ROWS + row, the same for every 32 channels
            sc[4 * row] = 0x01010101u * (uint32_t)(eq + 127);
            sc[4 * (ROWS + row)] = 0x01010101u * (uint32_t)(eq + 123);
        }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xFFFFFFFF;" : "=f"(y) : "f"(x));
    return y;
}

// The smaller one, NaN if either is.
__device__ __forceinline__ float min_nan(float a, float b) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

__device__ __forceinline__ uint32_t f16x2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// A pair of rows' p times the scale pair sc, 2^7 y, as four e4m3 pairs: y = a + b / 2^4 + c / 2^8 + d / 2^19.
// What a part leaves is exact in f16, and up to 2^8.8 at most 16 (half of its last place) of the next
// one's units, so nothing overflows; d saturates where y is large and takes what is left of a small one.
__device__ __forceinline__ void split4(uint32_t p2, uint32_t sc, uint32_t (&w)[4]) {
    uint32_t r = f16x2_mul(p2, sc);
    constexpr uint32_t down[4] = {0x20002000u, 0x30003000u, 0x40004000u, 0x6C006C00u};  // 2^-7, 2^-3, 2^1, 2^12
    constexpr uint32_t up[3] = {0xD800D800u, 0xC800C800u, 0xB800B800u};                 // -2^7, -2^3, -2^-1
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        w[k] = f16_to_e4m3(f16x2_mul(r, down[k]));
        if (k < 3) r = f16x2_fma(e4m3_to_f16((uint16_t)w[k]), up[k], r);
    }
}

}  // namespace

__global__ void __launch_bounds__(FewShape::THREADS, 1) attend_few_kernel(const __grid_constant__ AttendParams p) {
    using S = FewShape;
    constexpr int TN = S::TN, SETS = S::SETS;
    extern __shared__ uint8_t dyn_smem[];
    uint8_t *const base = dyn_smem + ((1024u - (smem_u32(dyn_smem) & 1023u)) & 1023u);
    __shared__ FewShared s;
    int *const prefix = reinterpret_cast<int *>(base + S::oPrefix);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&s.k_full[i], 33);  // the codes' byte count, the lanes' exponents
            mbar_init(&s.k_free[i], 1);
            mbar_init(&s.c_full[i], 1);
            mbar_init(&s.c_free[i], 1);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.s_free[i], 4);
            mbar_init(&s.m_full[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.q_full[i], 1);
            mbar_init(&s.q_free[i], 1);
            mbar_init(&s.l_full[i], 4 * SETS);
            mbar_init(&s.o_full[i], 1);
            mbar_init(&s.o_free[i], 4);
        }
        for (int i = 0; i < SETS; ++i) {
            mbar_init(&s.p_full[i], 4);
            mbar_init(&s.pv_done[i], 1);
            mbar_init(&s.vote[i], 4);
        }
        fence_mbar_init();
    }
    for (int i = threadIdx.x; i < 16 * ROWS; i += S::THREADS) (&s.nan[0][0][0])[i] = 0;
    hold_tmem(s, warp == kFewS);
    pdl_trigger();
    pdl_wait();
    sum_items<S>(p, s, prefix, warp, lane);
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, s.tmem, 0);
    const long long total = prefix[p.B];
    const int w0 = range_start(total, blockIdx.x), w1 = range_start(total, blockIdx.x + 1);
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool { return wait_warp(bar, parity, p.tries); };
    bool ok = true;  // no wait of this thread ran out
    const Segment first = segment_at<S>(p, prefix, w0, w1);

    if (warp == kFewK || warp == kFewV) {
        // ------------------------------------------------------------ producers
        const bool value = warp == kFewV;
        uint64_t *const full = value ? s.c_full : s.k_full, *const free = value ? s.c_free : s.k_free;
        const int nb = TN / p.box_rows, bt = 32 / nb, gpb = p.box_rows / 16;  // boxes a tile, tiles a batch, groups a box
        Batch batch{&s.pages[value][0][0], lane * gpb, 0};
        const uint32_t some = low_bits(nb), box_bytes = (uint32_t)p.box_rows * 128u;
        const int at = lane * p.box_rows * 128;  // of the lane's box
        // the exponents of keys 4 lane .. + 3: whose box, how far into it
        const int ex_box = (lane >> 2) / gpb, ex_off = 4 * lane - ex_box * p.box_rows;
        int tile = 0, seg = 0;
        Segment g = first;
        for (; live(g) && ok; ++seg) {
            const int tiles = g.kv1 - g.kv0, par = seg & 1;
            batch.ask(p, g, g.kv0, lane);
            if (value) {
                ok = seg < 2 || wait(&s.q_free[par], (uint32_t)((seg >> 1) & 1) ^ 1u);
                if (!ok) break;
                put_q(p, g, base + S::oQ + par * S::QBUF, reinterpret_cast<uint32_t *>(base + S::oQs + par * 512), lane);
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.q_full[par]);
            }
            int rows = -1, j = 0;
            uint32_t have = 0;  // the batch's boxes that exist
            for (int i = 0; i < tiles; ++i, ++tile) {
                if (j == 0) {
                    rows = batch.rows(p, g, g.kv0 + i, lane);
                    have = __ballot_sync(0xFFFFFFFFu, rows >= 0);
                    if (i + bt < tiles) batch.ask(p, g, g.kv0 + i + bt, lane);
                }
                const int slot = tile % S::NSLOT;
                ok = tile < S::NSLOT || wait(&free[slot], (uint32_t)((tile / S::NSLOT) & 1) ^ 1u);
                if (!ok) break;
                const int row = __shfl_sync(0xFFFFFFFFu, rows, (j * nb + lane) & 31);  // the box's first
                const uint32_t boxes = (have >> (j * nb)) & some;
                if (lane == 0) {
                    if (!value) {
                        uint32_t groups = low_bits((g.ctx + g.nodes - (g.kv0 + i) * TN + 15) >> 4) & 0xFFu;
                        if (boxes != some)
                            for (int k = 0; k < 8; ++k)
                                if (!((boxes >> (k / gpb)) & 1u)) groups &= ~(1u << k);
                        s.valid[tile % kRing] = (int)groups;
                    }
                    mbar_arrive_expect_tx(&full[slot], (uint32_t)__popc(boxes) * box_bytes);
                }
                __syncwarp();
                if (lane < nb && row >= 0 && !p.skip_loads)
                    tma_rows(base + (value ? S::oRing : S::oK) + slot * S::SLOT + at, value ? &p.vmap : &p.kmap, 0, row,
                             &full[slot]);
                if (!value) {  // 16 bytes a lane and kind: one instruction a kind, whatever the pages
                    const int ex_row = __shfl_sync(0xFFFFFFFFu, rows, (j * nb + ex_box) & 31);
                    if (ex_row >= 0 && !p.skip_loads) {
                        const size_t from = ((size_t)ex_row + ex_off) * S::EB;
                        cp_async16(base + S::oExp + slot * 1024 + 512 + lane * 16, p.c.kexp + from);
                        cp_async16(base + S::oVex + tile % kRing * 512 + lane * 16, p.c.vexp + from);
                    }
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(&full[slot])) : "memory");
                }
                j = j + 1 == bt ? 0 : j + 1;
            }
            next_segment<S>(p, g, w1);
        }
        // every copy must have landed before the block's memory goes away (bounded)
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (!p.skip_loads)
            for (int i = max(0, tile - S::NSLOT); i < tile; ++i)
                (void)mbar_wait_bounded(&full[i % S::NSLOT], (uint32_t)((i / S::NSLOT) & 1), ok ? p.timeout_ns : 100000000ull);
    } else if (warp == kFewS) {
        // ------------------------------------------------------------ S^T = K Q^T
        const bool one = elect_one();
        int tile = 0, seg = 0;
        Segment g = first;
        for (; live(g) && ok; ++seg) {
            const int tiles = __shfl_sync(0xFFFFFFFFu, g.kv1 - g.kv0, 0), par = seg & 1;
            ok = wait(&s.q_full[par], (uint32_t)((seg >> 1) & 1));
            if (!ok) break;
            fence_after();
            const uint32_t sfb = tmem + S::CA + 4 * par;
            if (one) copy_scales(sfb, desc_scales(smem_u32(base + S::oQs) + par * 512));  // in order with the MMAs
            __syncwarp();
            for (int i = 0; i < tiles; ++i, ++tile) {
                const int slot = tile % S::NSLOT, buf = tile % S::NS;
                ok = wait(&s.k_full[slot], (uint32_t)((tile / S::NSLOT) & 1)) &&
                     (tile < S::NS || wait(&s.s_free[buf], (uint32_t)((tile / S::NS) & 1) ^ 1u));
                if (!ok) break;
                fence_after();
                const uint32_t sfa = tmem + S::CB + 4 * (tile & 1), d = tmem + S::CS + buf * S::NQ;
                const uint64_t ad = desc_codes<128>(smem_u32(base + S::oK) + slot * S::SLOT);
                const uint64_t bd = desc_codes<128>(smem_u32(base + S::oQ) + par * S::QBUF);
                {   // the exponents as tensor memory wants them: 32 rows (lanes) of four words (columns), column
                    // c of row l being key 32 c + l's
                    uint32_t *const sc = reinterpret_cast<uint32_t *>(base + S::oExp + slot * 1024);
                    const uint4 w = *reinterpret_cast<const uint4 *>(sc + 128 + 4 * lane);  // keys 4 lane .. + 3
                    uint32_t *const d4 = sc + (4 * lane & 31) * 4 + (lane >> 3);
                    d4[0] = w.x, d4[4] = w.y, d4[8] = w.z, d4[12] = w.w;
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
                if (one) {
                    copy_scales(sfa, desc_scales(smem_u32(base + S::oExp) + slot * 1024));
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)  // 32 channels a step
                        umma_mx_ss(d, ad + 2 * ks, bd + 2 * ks, idesc_mx(S::NQ, ks, 0), sfa, sfb, ks > 0);
                    commit_a(&s.s_full[buf]);
                    commit_a(&s.k_free[slot]);
                    if (i + 1 == tiles) commit_a(&s.q_free[par]);
                }
                __syncwarp();
            }
            next_segment<S>(p, g, w1);
        }
        // the last products must be done before tensor memory goes back (bounded)
        if (tile > 0) (void)wait(&s.s_full[(tile - 1) % S::NS], (uint32_t)(((tile - 1) / S::NS) & 1));
    } else if (warp == kFewO) {
        // ------------------------------------------------------------ O^T += V^T P
        const bool one = elect_one();
        int tile = 0, seg = 0;
        Segment g = first;
        for (; live(g) && ok; ++seg) {
            const int tiles = __shfl_sync(0xFFFFFFFFu, g.kv1 - g.kv0, 0), par = seg & 1;
            ok = seg < 2 || wait(&s.o_free[par], (uint32_t)((seg >> 1) & 1) ^ 1u);
            for (int i = 0; i < tiles && ok; ++i, ++tile) {
                const int slot = tile % S::NSLOT, buf = tile % SETS;
                ok = wait(&s.c_full[slot], (uint32_t)((tile / S::NSLOT) & 1)) && wait(&s.p_full[buf], (uint32_t)((tile / SETS) & 1));
                if (!ok) break;
                fence_after();
                const uint32_t d = tmem + S::CO + par * S::NP;
                const uint64_t ad = desc_a(smem_u32(base + S::oRing) + slot * S::SLOT, TN * 128);
                const uint64_t bd = desc_a(smem_u32(base + S::oP) + buf * S::PBUF, TN * 128);
                if (one) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)  // 32 keys a step: four 8-key atoms
                        umma_8(d, ad + ks * (4096 >> 4), bd + ks * (4096 >> 4), idesc_8(S::NP), i > 0 || ks > 0);
                    commit_a(&s.pv_done[buf]);
                    commit_a(&s.c_free[slot]);
                    if (i + 1 == tiles) commit_a(&s.o_full[par]);
                }
                __syncwarp();
            }
            next_segment<S>(p, g, w1);
        }
        if (tile > 0) (void)wait(&s.pv_done[(tile - 1) % SETS], (uint32_t)(((tile - 1) / SETS) & 1));
    } else {
        // ------------------------------------------------------------ softmax and output
        const int set = (warp >> 2) - 1, quad = warp & 3, key = 32 * quad + lane;  // key of a tile, channel of O^T
        const uint32_t tl = tmem + ((uint32_t)(32 * quad) << 16);
        const float c = p.scale_log2;
        uint32_t vote_ph = 0;
        auto set_sync = [&]() -> bool {  // the set's four warps
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.vote[set]);
            vote_ph ^= 1u;
            return wait(&s.vote[set], vote_ph ^ 1u);
        };
        int it = 0, seg = 0;
        Segment g = first;
        for (; live(g) && ok; ++seg) {
            const int tiles = g.kv1 - g.kv0, par = seg & 1, rows = g.nodes * p.g;
            float l[ROWS], off[ROWS], last[ROWS];  // sums, in 2^(m - bias); bias - m now, and at the set's last tile
            int epoch = 0, E = 0;
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                l[r] = 0.0f;
                off[r] = last[r] = kUnseen;
            }
            for (int i = 0; i < tiles; ++i, ++it) {
                if (it % SETS != set) continue;
                const int buf = it % S::NS;
                ok = wait(&s.s_full[buf], (uint32_t)((it / S::NS) & 1));
                if (!ok) break;
                fence_after();
                uint32_t x[ROWS], xl[ROWS];
                ld_cols(tl + S::CS + buf * S::NQ, x);
                ld_cols(tl + S::CS + buf * S::NQ + ROWS, xl);
                const uint32_t valid = (uint32_t)s.valid[it % kRing];  // read before S is given back
                uint32_t ex = *reinterpret_cast<const uint32_t *>(base + S::oVex + it % kRing * 512 + 4 * key);
                const int slot = (g.kv0 + i) * TN + key;  // the thread's cache slot
                wait_ld();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.s_free[buf]);
                float sv[ROWS];
#pragma unroll
                for (int r = 0; r < ROWS; ++r) sv[r] = __uint_as_float(x[r]) + __uint_as_float(xl[r]);
                uint32_t vis = 0xFFFFFFFFu;  // rows that see the key
                uint32_t bad = 0;            // channel blocks (a byte each) whose values count as zeros
                if ((g.kv0 + i + 1) * TN > g.ctx || valid != 0xFFu) {
                    const int j = slot - g.ctx;
                    if (!((valid >> (key >> 4)) & 1u) || j >= g.nodes) {
                        vis = ex = 0;
                        bad = 0xFFFFFFFFu;
                    } else if (j >= 0) {
                        vis = 0;
                        for (int t = 0; t < g.nodes; ++t) {
                            const bool sees = p.mask ? (p.mask[((size_t)g.b * p.T + t) * p.W + (j >> 5)] >> (j & 31)) & 1 : j <= t;
                            if (sees) vis |= low_bits(p.g) << (t * p.g);
                        }
                    }
#pragma unroll
                    for (int r = 0; r < ROWS; ++r)
                        if (!((vis >> r) & 1u)) sv[r] = -INFINITY;
                }
                // does any x pass the references that the set knows?
                bool up = false;
#pragma unroll
                for (int r = 0; r < ROWS; ++r) up |= fmaf(sv[r], c, off[r]) > kFewBias + kFewSlack;
                const bool any = __any_sync(0xFFFFFFFFu, up);
                // the largest value exponent, NaN (255) left out
                const uint32_t nans = __vcmpeq4(ex, 0xFFFFFFFFu);
                ex &= ~nans;
                bad |= nans;
                uint32_t mx = __vmaxu4(ex, ex >> 16);
                mx = __reduce_max_sync(0xFFFFFFFFu, max(mx & 0xFFu, (mx >> 8) & 0xFFu));
                int *const votes = s.grow[set][(it / SETS) & 1];
                if (lane == 0) votes[quad] = (int)mx | (any ? 256 : 0);
                ok = set_sync();
                if (!ok) break;
                const int4 v4 = *reinterpret_cast<const int4 *>(votes);
                // the references of the tile before (at a segment's start too its tile is waited for: the last ones
                // have then been read)
                int now = 0, before = 0;
                if (it > 0) ok = wait(&s.m_full[(it - 1) & 3], (uint32_t)(((it - 1) >> 2) & 1));
                if (!ok) break;
                if (i > 0) {
                    const int2 v = s.ref[(it - 1) & 3];
                    now = v.x;
                    before = v.y;
                }
                E = max(max(before, max(v4.x & 255, v4.y & 255)), max(v4.z & 255, v4.w & 255));
                const int rise = E - before;
                bool grow = false;
                float f[ROWS];
                if (((v4.x | v4.y | v4.z | v4.w) & 256) || now != epoch) {
                    if (now != epoch) {
#pragma unroll
                        for (int r = 0; r < ROWS; r += 4) {
                            const float4 v = *reinterpret_cast<const float4 *>(&s.off[now & 3][r]);
                            off[r] = v.x, off[r + 1] = v.y, off[r + 2] = v.z, off[r + 3] = v.w;
                        }
                    }
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) {
                        const float w = warp_max(sv[r]);
                        if (lane == 0) s.most[set][quad][r] = w;
                    }
                    ok = set_sync();
                    if (!ok) break;
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) {
                        const float mt = fmaxf(fmaxf(s.most[set][0][r], s.most[set][1][r]),
                                               fmaxf(s.most[set][2][r], s.most[set][3][r]));
                        // m rounded down, and never falling: where its last place is no longer small against the slack an x
                        // below it may seem to pass it
                        const float next = fmaf(mt, c, off[r]) > kFewBias + kFewSlack ? fminf(off[r], __fmaf_ru(-mt, c, kFewBias)) : off[r];
                        f[r] = next == off[r] ? 1.0f : ex2(next - off[r]);
                        grow |= next != off[r];
                        off[r] = next;
                    }
                    now += grow;
                }
                if (quad == 0) {
                    if (lane == 0) {
                        if (grow) {
#pragma unroll
                            for (int r = 0; r < ROWS; r += 4)
                                *reinterpret_cast<float4 *>(&s.off[now & 3][r]) =
                                    make_float4(off[r], off[r + 1], off[r + 2], off[r + 3]);
                        }
                        s.ref[it & 3] = make_int2(now, E);
                        mbar_arrive(&s.m_full[it & 3]);
                    }
                    __syncwarp();
                }
                if (now != epoch) {
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) {
                        l[r] *= off[r] == last[r] ? 1.0f : ex2(off[r] - last[r]);
                        last[r] = off[r];
                    }
                    epoch = now;
                }
                uint32_t p2[ROWS / 2];
#pragma unroll
                for (int r = 0; r < ROWS; r += 2) {
                    // (cut off for such an m only: else no x passes it by more)
                    const float a = ex2(min_nan(fmaf(sv[r], c, off[r]), kFewBias + kFewSlack));
                    const float b = ex2(min_nan(fmaf(sv[r + 1], c, off[r + 1]), kFewBias + kFewSlack));
                    l[r] += a;
                    l[r + 1] += b;
                    p2[r / 2] = pack_f16(a, b);
                }
                // P's place is free once the set's last product is done.  Only then may the product of the tile before
                // be waited for: a phase's parity says which of two it is, not of three.
                ok = it < SETS || wait(&s.pv_done[set], (uint32_t)((it / SETS) & 1) ^ 1u);
                if (!ok) break;
                // ---- O in the units of the new references and value exponent
                if (i > 0 && (grow || rise)) {
                    ok = wait(&s.pv_done[(it - 1) % SETS], (uint32_t)(((it - 1) / SETS) & 1));
                    if (!ok) break;
                    fence_after();
                    const float fv = pow2i(max(-rise, -149));
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t at = tl + S::CO + par * S::NP + (4 * k + quad) * ROWS;
                        uint32_t o[ROWS];
                        ld_cols(at, o);
                        wait_ld();
#pragma unroll
                        for (int r = 0; r < ROWS; ++r)
                            o[r] = __float_as_uint(__uint_as_float(o[r]) * (grow ? f[r] * fv : fv));
                        st_cols(at, o);
                    }
                    wait_st();
                    fence_before();
                }
                // ---- P
                uint8_t *const pb = base + S::oP + set * S::PBUF + key * 128;
                // column 4 ROWS part + ROWS block + row of the key's 128-byte rows, swizzled
                constexpr int U = ROWS / 4;  // 16-byte units a part
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    uint32_t w[4][4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {  // four rows of a block a word
                        const int blk = 2 * u + (j >> 1), r = 4 * (j & 1);
                        const int e = (int)((ex >> (8 * blk)) & 0xFFu);
                        const uint32_t sc = f16_pow2(e - E);
                        uint32_t a[4], b[4];
                        split4(p2[r / 2], sc, a);
                        split4(p2[r / 2 + 1], sc, b);
#pragma unroll
                        for (int k = 0; k < 4; ++k) w[k][j] = a[k] | (b[k] << 16);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        *reinterpret_cast<uint4 *>(pb + (((k * U + u) ^ (key & 7)) << 4)) =
                            make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
                    }
                }
                if (__any_sync(0xFFFFFFFFu, bad)) {
                    ok = wait(&s.c_full[it % S::NSLOT], (uint32_t)((it / S::NSLOT) & 1));
                    if (!ok) break;
                    uint8_t *const v = base + S::oRing + (it % S::NSLOT) * S::SLOT + key * 128;
                    for (int u = 0; u < 8; ++u)
                        if ((bad >> (4 * (u & 6))) & 255u)
                            *reinterpret_cast<uint4 *>(v + ((u ^ (key & 7)) << 4)) = make_uint4(0, 0, 0, 0);
                    for (int r = 0; r < ROWS && r < rows; ++r)
                        if ((vis >> r) & 1u)
                            for (int k = 0; k < 4; ++k)
                                if ((nans >> (8 * k)) & 255u) s.nan[seg & 3][k][r] = 1;
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.p_full[set]);
            }
            if (!ok) break;
            // ---- the segment's sums
            ok = seg < 2 || wait(&s.o_free[par], (uint32_t)((seg >> 1) & 1) ^ 1u);
            if (!ok) break;
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                float a = l[r];
#pragma unroll
                for (int k = 16; k > 0; k >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, k);
                if (lane == 0) {
                    s.sum[par][warp - 4][r] = a;
                    if (quad == 0) s.soff[par][set][r] = last[r];
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.l_full[par]);
            if ((it - 1) % SETS == set) {
                // ---- the output, by the set of the last tile; thread = channel
                ok = wait(&s.l_full[par], (uint32_t)((seg >> 1) & 1)) && wait(&s.o_full[par], (uint32_t)((seg >> 1) & 1));
                if (!ok) break;
                fence_after();
                const bool whole = g.kv0 == 0 && g.kv1 == g.nt;
                const int slotw = 2 * blockIdx.x + (g.kv0 > 0 ? 0 : 1);
                const float fv = pow2i(E - 127);
                const bool tiny = E < 64;  // fv / L may be too small for fp32
                // lane r: row r's sum, in units of the last reference
                const int rl = lane % ROWS;
                const float end = s.soff[par][set][rl];
                float L = 0.0f;
#pragma unroll
                for (int w = 0; w < 4 * SETS; ++w) {
                    const float q = s.soff[par][w >> 2][rl], a = s.sum[par][w][rl];
                    L += a == 0.0f ? 0.0f : a * (q == end ? 1.0f : ex2(end - q));
                }
                const float inv = L == 0.0f ? 0.0f : (tiny ? 1.0f : fv) * 128.0f / L;
                const bool bad = s.nan[seg & 3][quad][rl];
                __syncwarp();
                if (lane < ROWS) s.nan[seg & 3][quad][lane] = 0;
                if (quad == 0 && lane < ROWS && lane < rows) {
                    const float Lt = L * 0x1p-13f;  // without the bias
                    const float M = end == kUnseen ? -INFINITY : kFewBias - end;
                    const int t = lane / p.g, hq = g.h * p.g + lane - t * p.g;
                    if (!whole)
                        p.stat[(size_t)slotw * ROWS + lane] = make_float2(M, Lt);
                    else if (p.lse)
                        p.lse[((size_t)g.b * p.T + t) * p.Hq + hq] =
                            L == 0.0f ? -INFINITY : (M + log2f(Lt)) * 0.69314718055994531f;
                }
                float y[ROWS];
#pragma unroll
                for (int k = 3; k >= 0; --k) {
                    uint32_t o[ROWS];
                    ld_cols(tl + S::CO + par * S::NP + (4 * k + quad) * ROWS, o);
                    wait_ld();
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) y[r] = (k == 3 ? 0.0f : y[r] * (k == 2 ? 0x1p-11f : 0x1p-4f)) + __uint_as_float(o[r]);
                }
                if (tiny)
#pragma unroll
                    for (int r = 0; r < ROWS; ++r) y[r] *= fv;
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.o_free[par]);
#pragma unroll
                for (int r = 0; r < ROWS; ++r) {
                    const float k = __shfl_sync(0xFFFFFFFFu, inv, r);
                    const bool nan = __shfl_sync(0xFFFFFFFFu, (int)bad, r);
                    const float z = nan ? __uint_as_float(0x7FC00000u) : k == 0.0f ? 0.0f : y[r] * k;
                    if (r < rows) {
                        if (whole) {
                            const int t = r / p.g, hq = g.h * p.g + r - t * p.g;
                            p.out[(((size_t)g.b * p.T + t) * p.Hq + hq) * S::DIM + key] = (uint16_t)pack_bf(z, 0.0f);
                        } else {
                            p.part[((size_t)slotw * ROWS + r) * S::DIM + key] = z;
                        }
                    }
                }
            }
            next_segment<S>(p, g, w1);
        }
    }

    if (!ok) report_timeout(p.status);
    free_tmem(tmem, warp == kFewS);
}

cudaError_t launch_attend_few(const AttendParams &prm, cudaStream_t stream) {
    return launch_attend_shape<FewShape>(attend_few_kernel, prm, stream);
}

}  // namespace bsf8
