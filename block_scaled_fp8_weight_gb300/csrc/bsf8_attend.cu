// bsf8_attend.cu -- attention of a token tree over the paged block-scaled fp8 cache (tcgen05).
//
//   out[row] = sum_l 2^(x_l - m) v_l / sum_l 2^(x_l - m),   x_l = scale log2(e) q[row].k_l,
// over the keys l that the row sees; a row is a (node, query head) of one request and cache
// head.  One pass over the cache with the running maximum m and sum of a softmax.  Up to 8 rows at
// dim 128 over long contexts run in bsf8_attend_few.cu, on the same cut of the work and the same join.
//
// Work.  An item is a tile of TN keys (128; 64 at dim 256) of one (request, head, tile of RT
// rows), a segment all items of one (request, head, row tile).  The segments of all requests, in that
// order, each as long as its items and START more for its start and end, are cut into one equal
// contiguous share per block (one block an SM), whatever the requests' lengths: every block computes the
// same prefix sums.  (Without the START places a block full of short requests held up the others: 64
// requests of 70 to 16384 tokens took 250 us, with them 184; 16 trees of 23 nodes 80 us, then 50.)
// A block that has a whole segment writes the output; else it writes a partial (its rows' normalised
// output, maximum and sum) to one of its two workspace slots -- only a block's first and last segment
// can be incomplete -- and a second kernel joins each row's partials in block order.  Nothing
// depends on timing: the same call gives the same bits.
//
// A block's warps, each with its own loop over the items:
//   producer  the codes, into rings of slots: keys by TMA boxes (swizzled for the MMA), values by
//             bulk copies (page runs of a head are contiguous);
//   scout     exponents and flags: the keys' exponents laid out for tensor memory, the largest value
//             exponent E of the segment so far, which groups of keys exist;
//   8 dequant a tile's values -> f16 in shared memory (128-byte swizzle), as code * 2^(e - E + 6): exact for
//             exponents within 2^21 of E, else off by at most 2^-31 of 448 * 2^E (from 2^31 below E on
//             they count as 0); e4m3 times a power of two needs no more than f16's 11 bits;
//   S         S = Q K^T on the cached codes (block-scaled MMA): the exponents go along as its scales.  Q is the
//             sum of two e4m3 parts (A, in tensor memory; at dim 256 in shared memory): 8 MMAs a tile;
//   O         O += P V (P in tensor memory as A, V as an N-major B): 8 MMAs of 16 keys;
//   8 softmax two sets of four, a set every other tile, thread = row: p = 2^(x - m + 9) (fp32, summed in
//             fp32), rounded to f16 for the second product: 11 bits of p at any p above 2^-23 of 2^m,
//             half of 2^-33 of it below.  (bf16 would round p to 8 bits: 1.4 times the error of the
//             output's own rounding.)  Where the keys' exponents allow |x| >= 2^21, x itself, rounded, takes
//             S's place first: x - m by one fma, with an m whose last place is large, would give the largest
//             p any value.  m, handed from set to set, only moves when the maximum has
//             grown by more than 2^6 over it: p stays below f16's largest, and rescaling O (a round
//             trip through registers) becomes rare; with 2^2 it took 4 us of 50 at 4096 tokens.
// RT rows of Q fill the MMA's 128 rows 128 / RT times; each copy handles its own part of the
// tile's key columns (its P is zero elsewhere), so that with few rows all four softmax warps
// still work; the copies' sums and outputs join at the segment's end.
// Masks are 32-bit words a row and 32 keys; tiles wholly inside the context skip them.  Keys
// past a request's end (a page's unused slots may hold anything) and keys on bad pages are
// masked, and their values are zeroed; a value block that holds NaN is zeroed too, and the rows
// that see it get their NaN at the end, so that it reaches no other row.
//
// Bound.  The cache is read once a row tile, 2 dim (1 + 1/32) bytes a key and head: 1440 cycles of an SM's
// share of HBM a tile of 128 keys at dim 128; the tensor cores need 1024 for it, the exponentials of
// 128 rows 512, shared memory (codes in and out, f16 in and out, the MMAs' reads: 144 KB) 1150.  It
// takes 2080: S of a tile waits for the product with the P two tiles before, whose place it takes
// (tensor memory has no room for more: two S, O and Q fill 460 of 512 columns, another S does not
// fit), so the latencies of softmax (2300 cycles) and of the products with their handoffs (1900) add
// up over two tiles.  P in columns of its own with Q in shared memory ran 20 percent slower, each tile
// halved between the sets 13 percent slower.
// Measured (in a graph): 2 requests of 131072 keys, 288 and 320 rows, thus 6 row tiles, x 4 heads at dim 128: 190 us
// (1.08 PFLOP/s of the tiles' products, 0.55 of the measured bf16 rate); 77 to 161 rows, 16 requests of 8192
// tokens at most, 4 heads: 45 us, of which a third is segments' starts and ends.
#include "bsf8_attend.cuh"

#include <mutex>

namespace bsf8 {

namespace {

template <int D, int ROWS>
struct Shape {
    static constexpr int DIM = D, RT = ROWS, THREADS = kThreadsA;
    static constexpr int START = kStart;
    static constexpr int TN = D == 256 ? 64 : 128;   // keys a tile
    static constexpr int EB = D / 32;                // exponent bytes a key
    static constexpr int SLOT = TN * D;              // bytes of a tile's codes
    static constexpr int NSLOT = D == 256 ? 2 : 4;   // ring slots of keys, and of values
    static constexpr int F16 = TN * D * 2;           // bytes of an f16 tile of values
    // tensor memory columns: two S (a tile's P, f16 pairs, takes its S's place), O, the scales of Q
    // and of two tiles' keys, and up to dim 128 Q (two e4m3 parts, four to a column)
    static constexpr int CS = 0, CO = 2 * TN, CA = CO + D, CB = CA + 4,
                         CQ = D == 256 ? 0 : CA + 32;
    static constexpr bool QS = D == 256;             // Q in shared memory
    static_assert(CQ + (QS ? 0 : D / 2) <= 512);
    static constexpr int oV = 0, oK = 2 * F16, oRing = oK + NSLOT * SLOT, oQ = oRing + NSLOT * SLOT;
    static constexpr int oExp = oQ + (QS ? 2 * 128 * D : 0), oStage = oExp + NSLOT * 1024;
    static constexpr int oPrefix = oStage + 2 * 128 * 17 * 4;
};

struct AttendShared : AttendPipes {
    uint64_t s_full[2];             // S written
    uint64_t p_full[2];             // P written, O rescaled
    uint64_t m_full[2][4];          // a softmax warp's rows have their maximum of the tile
    uint64_t q_full;                // a segment's Q is in place
    uint64_t soft, set[2];          // the softmax warps' own barriers (bounded, unlike bar.sync)
    float mrow[2][128];             // the rows' maxima, handed from set to set
    uint32_t amax[kSoftWarps][32];  // of the halves of Q's rows
    float2 stat[kSoftWarps][32];
    uint32_t nan[kSoftWarps][32];
};

}  // namespace

template <int D, int RT>
__global__ void __launch_bounds__(kThreadsA, 1) attend_kernel(const __grid_constant__ AttendParams p) {
    using S = Shape<D, RT>;
    constexpr int TN = S::TN, REP = 128 / RT, CPT = TN / REP;  // CPT: key columns a thread
    constexpr int CH = CPT <= 32 ? CPT : 16;  // taken CH at a time
    extern __shared__ uint8_t dyn_smem[];
    uint8_t *const base = dyn_smem + ((1024u - (smem_u32(dyn_smem) & 1023u)) & 1023u);
    __shared__ AttendShared s;
    int *const prefix = reinterpret_cast<int *>(base + S::oPrefix);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        init_pipes(s);
        for (int i = 0; i < 8; ++i) mbar_init(&s.m_full[i >> 2][i & 3], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_full[i], 4);
            mbar_init(&s.set[i], 4);
        }
        mbar_init(&s.q_full, kSoftWarps);
        mbar_init(&s.soft, kSoftWarps);
        fence_mbar_init();
    }
    hold_tmem(s, warp == kMmaWarp);
    pdl_trigger();
    pdl_wait();
    sum_items<S>(p, s, prefix, warp, lane);
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, s.tmem, 0);
    const long long total = prefix[p.B];
    const int w0 = range_start(total, blockIdx.x), w1 = range_start(total, blockIdx.x + 1);
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool { return wait_warp(bar, parity, p.tries); };
    bool ok = true;  // no wait of this thread ran out
    // The block's first segment; each role walks on from it.
    const Segment first = segment_at<S>(p, prefix, w0, w1);

    if (warp == kProducerWarp) {
        ok = produce<S>(p, s, base, first, w1, lane);
    } else if (warp == kScoutWarp) {
        ok = scout<S>(p, s, base, first, w1, lane);
    } else if (warp >= kMmaWarp) {
        // ------------------------------------------------------------ MMA issue: a thread a product
        // One thread issues an MMA about every 100 cycles whatever its size (to N = 128); two with
        // an accumulator each, one every 64.
        // The whole warp walks along, so that addresses and descriptors stay in uniform registers.
        const bool value = __shfl_sync(0xFFFFFFFFu, warp, 0) > kMmaWarp;
        const bool one = elect_one();
        int tile = 0;  // of the block so far
        uint32_t qph = 0;
        Segment g = first;
        for (; live(g) && ok; qph ^= 1u) {
            const int tiles = __shfl_sync(0xFFFFFFFFu, g.kv1 - g.kv0, 0);
            if (!value) ok = wait(&s.q_full, qph);
            for (int i = 0; i < tiles && ok; ++i, ++tile) {
                const int buf = tile & 1;
                const uint32_t bph = (uint32_t)((tile >> 1) & 1);
                const uint32_t sp = tmem + S::CS + buf * TN;
                if (value) {
                    ok = wait(&s.v_full[buf], bph) && wait(&s.p_full[buf], bph);
                    if (!ok) break;
                    fence_after();
                    const uint64_t bd = desc_a(smem_u32(base + S::oV) + buf * S::F16, TN * 128);
                    if (one) {
                        // At dim 128 as two accumulators of 64 channels in turn: 205 us where one of 128 takes 212 (long
                        // trees); at 64 and 256, and for S, no difference.
                        constexpr int OW = D == 128 ? 64 : D;
#pragma unroll
                        for (int ks = 0; ks < TN / 16; ++ks)  // 16 keys a step: two 8-key atoms
#pragma unroll
                            for (int k = 0; k < D; k += OW)
                                umma_a(tmem + S::CO + k, sp + 8 * ks, bd + ks * (2048 >> 4) + k / 64 * (TN * 128 >> 4),
                                       idesc_a(OW, true), i > 0 || ks > 0);
                        commit_a(&s.pv_done[buf]);
                    }
                } else {
                    const int slot = tile % S::NSLOT;
                    // S takes the place of the P of two tiles before
                    ok = wait(&s.k_full[slot], (uint32_t)((tile / S::NSLOT) & 1));
                    if (!ok) break;
                    fence_after();
                    const uint32_t sfb = tmem + S::CB + 4 * buf;  // in order with the MMAs of this thread
                    if (one) copy_scales(sfb, desc_scales(smem_u32(base + S::oExp) + slot * 1024));
                    __syncwarp();
                    ok = tile < 2 || wait(&s.pv_done[buf], bph ^ 1u);
                    if (!ok) break;
                    fence_after();
                    constexpr int RB = D < 128 ? 64 : 128;
                    const uint64_t bd = desc_codes<RB>(smem_u32(base + S::oK) + slot * S::SLOT);
                    const uint64_t ad = desc_codes<128>(smem_u32(base + S::oQ));
                    if (one) {
#pragma unroll
                        for (int part = 0; part < 2; ++part)  // Q's upper and lower parts
#pragma unroll
                            for (int ks = 0; ks < D / 32; ++ks) {  // 32 channels a step
                                const uint64_t bk = bd + (ks >> 2) * (TN * 128 >> 4) + 2 * (ks & 3);
                                const uint32_t id = idesc_mx(TN, part, ks & 3), fb = sfb + 2 * (ks >> 2);
                                if constexpr (S::QS)
                                    umma_mx_ss(sp, ad + part * (128 * D >> 4) + (ks >> 2) * (128 * 128 >> 4) + 2 * (ks & 3), bk,
                                               id, tmem + S::CA, fb, part + ks > 0);
                                else
                                    umma_mx_ts(sp, tmem + S::CQ + part * (D / 4) + 8 * ks, bk, id, tmem + S::CA, fb,
                                               part + ks > 0);
                            }
                        commit_a(&s.s_full[buf]);
                        commit_a(&s.k_free[slot]);
                    }
                }
                __syncwarp();
            }
            next_segment<S>(p, g, w1);
        }
        // the last products must be done before tensor memory goes back (bounded)
        if (tile > 0)
            (void)wait(value ? &s.pv_done[(tile - 1) & 1] : &s.s_full[(tile - 1) & 1], (uint32_t)(((tile - 1) >> 1) & 1));
    } else if (warp >= kSoftWarps) {
        ok = widen_values<S>(p, s, base, first, w1, warp, lane);
    } else {
        // ------------------------------------------------------------ softmax and output
        const int set = warp >> 2, quad = warp & 3;                // tiles of one parity; tensor memory lanes
        const uint32_t tl = tmem + ((uint32_t)(32 * quad) << 16);
        const int row = (32 * quad + lane) % RT;                   // row of the tile
        const int copy = 32 * quad / RT, col0 = copy * CPT;        // this copy's key columns
        int it = 0;
        uint32_t soft_ph = 0, set_ph = 0;
        auto soft_sync = [&]() -> bool {  // all softmax warps
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.soft);
            soft_ph ^= 1u;
            return wait(&s.soft, soft_ph ^ 1u);
        };
        auto set_sync = [&]() -> bool {   // the set's four
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.set[set]);
            set_ph ^= 1u;
            return wait(&s.set[set], set_ph ^ 1u);
        };
        // A segment's Q: each row scaled by a power of two 2^-eq so that its largest lies in
        // [2^7, 2^8), as the sum of two e4m3 parts, the lower one times 2^4 (its scale is 2^-4).  Exact
        // for bf16 values within 2^14 of the row's largest, else off by at most 2^-22 of that.  The
        // sets take half of the channels each: up to dim 128 from registers (asked for before the last
        // tile of the segment before is waited for), else 32 channels at a time.
        constexpr int HELD = D <= 128 ? D / 16 : 1;
        auto q_row = [&](const Segment &g, bool &real) -> const uint4 * {
            const int r = g.rt * RT + row;
            real = r < g.nodes * p.g;
            const int t = real ? r / p.g : 0, hq = g.h * p.g + (real ? r - t * p.g : 0);
            return reinterpret_cast<const uint4 *>(p.q + ((size_t)g.b * p.T + t) * p.ldq + (size_t)hq * D + set * (D / 2));
        };
        auto largest_of = [](uint32_t am, const uint4 &v) -> uint32_t {
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) am = max(am, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
            return am;
        };
        auto put_q = [&](const Segment &g, const uint4 (&held)[HELD], int &eq) -> bool {
            bool real;
            const uint4 *const qr = q_row(g, real);
            uint32_t am = 0;
            if constexpr (D <= 128) {
#pragma unroll
                for (int j = 0; j < HELD; ++j) am = largest_of(am, held[j]);
            } else if (real) {
#pragma unroll 8
                for (int j = 0; j < D / 16; ++j) am = largest_of(am, qr[j]);
            }
            s.amax[warp][lane] = am;
            if (!soft_sync()) return false;
            am = max(am, s.amax[warp ^ 4][lane]);
            // A row with an infinity or a NaN becomes NaN as a whole, as its scores are (the conversion to
            // e4m3 would make an infinity its largest value).
            const bool nan = am >= 0x7F80u;
            eq = nan ? -100 : max((int)(am >> 7) - 127 - 7, -100);  // at most 120
            const float qs = nan ? __uint_as_float(0x7FC00000u) : pow2i(-eq);
            constexpr int CHUNK = 32;
#pragma unroll(D <= 128 ? D / 64 : 1)
            for (int c0 = 0; c0 < D / 2; c0 += CHUNK) {
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if constexpr (D <= 128)
                        v = held[c0 / 8 + j];
                    else if (real)
                        v = qr[c0 / 8 + j];
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    uint32_t h2[4], l2[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t x = pack_f16(__uint_as_float(w[k] << 16) * qs, __uint_as_float(w[k] & 0xFFFF0000u) * qs);
                        h2[k] = f16_to_e4m3(x);
                        l2[k] = f16_to_e4m3(f16x2_mul(f16x2_sub(x, e4m3_to_f16((uint16_t)h2[k])), 0x4C004C00u));  // * 16
                    }
                    hi[2 * j] = h2[0] | (h2[1] << 16);
                    hi[2 * j + 1] = h2[2] | (h2[3] << 16);
                    lo[2 * j] = l2[0] | (l2[1] << 16);
                    lo[2 * j + 1] = l2[2] | (l2[3] << 16);
                }
                const int c = set * (D / 2) + c0;
                if constexpr (S::QS) {
                    const int lr = 32 * quad + lane;  // rows of 128 channels, 128-byte swizzle
                    uint8_t *d = base + S::oQ + (c >> 7) * (128 * 128) + lr * 128;
                    const int u = (c & 127) >> 4, x = lr & 7;
                    *reinterpret_cast<uint4 *>(d + ((u ^ x) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(d + (((u + 1) ^ x) << 4)) = make_uint4(hi[4], hi[5], hi[6], hi[7]);
                    *reinterpret_cast<uint4 *>(d + 128 * D + ((u ^ x) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    *reinterpret_cast<uint4 *>(d + 128 * D + (((u + 1) ^ x) << 4)) = make_uint4(lo[4], lo[5], lo[6], lo[7]);
                } else {
                    st_cols(tl + S::CQ + c / 4, hi);
                    st_cols(tl + S::CQ + D / 4 + c / 4, lo);
                }
            }
            if constexpr (S::QS)
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            else
                wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.q_full);
            return true;
        };
        {   // Q's scales: byte 0 (2^0) for the upper part, byte 1 (2^-4) for the lower
            const uint32_t f[4] = {0x7B7Fu, 0x7B7Fu, 0x7B7Fu, 0x7B7Fu};
            st_cols(tl + S::CA, f);  // both sets write the same
            wait_st();
        }
        // Per turn, once the last S of the segment before is there: the next segment's Q, then the output of
        // the one before, then the segment's tiles.
        Segment g = first;
        int r = 0, t = 0, hq = 0;          // row of the request and head; its node and query head
        bool real = false;
        float m = 0.0f, l = 0.0f;          // the rows' maximum at the set's last tile; its sum in 2^(m - bias)
        uint32_t nanblk = 0;
        while (ok) {
            Segment next = g;
            if (it > 0) next_segment<S>(p, next, w1);
            const bool more = live(next);
            int eq = 0;
            uint4 held[HELD] = {};
            if (D <= 128 && more) {
                bool there;
                const uint4 *const qr = q_row(next, there);
                if (there)
#pragma unroll
                    for (int j = 0; j < HELD; ++j) held[j] = qr[j];
            }
            // The last S is there, so its tile's value exponent is known and O has the product of two tiles before.  (Else
            // the set of the tile before it could take that product's phase, of the same parity, for the last one's
            // below, and read the exponent before it is written.)
            if (it > 0) ok = wait(&s.s_full[(it - 1) & 1], (uint32_t)(((it - 1) >> 1) & 1));
            if (!ok) break;
            fence_after();
            if (more) {
                ok = put_q(next, held, eq);
                if (!ok) break;
            }
            if (it > 0) {
                // ---- the segment's output; the sets take half of the channels each
                ok = wait(&s.pv_done[(it - 1) & 1], (uint32_t)(((it - 1) >> 1) & 1));
                if (!ok) break;
                fence_after();
                const int ev = s.info[(it - 1) % kInfo].ev;
                s.stat[warp][lane] = make_float2(m, l);
                s.nan[warp][lane] = nanblk;
                ok = soft_sync();
                if (!ok) break;
                // a copy's maximum is the later of its two sets'; copies and sets are added in order
                float M = -INFINITY, mc = -INFINITY, L = 0.0f;
#pragma unroll
                for (int q = 0; q < REP; ++q) {
                    const int w = q * (RT / 32) + quad % (RT / 32);
                    M = max3(M, s.stat[w][lane].x, s.stat[w + 4][lane].x);
                }
#pragma unroll
                for (int q = 0; q < 2 * REP; ++q) {
                    const float2 st = s.stat[(q >> 1) * (RT / 32) + quad % (RT / 32) + 4 * (q & 1)][lane];
                    L += st.y == 0.0f ? 0.0f : st.y * ex2(st.x == -INFINITY ? 0.0f : st.x - M);
                }
                mc = fmaxf(s.stat[quad][lane].x, s.stat[quad + 4][lane].x);
                nanblk = s.nan[quad][lane] | s.nan[quad + 4][lane];
                const bool any = s.stat[quad][lane].y != 0.0f || s.stat[quad + 4][lane].y != 0.0f;
                const bool whole = g.kv0 == 0 && g.kv1 == g.nt;
                const int slotw = 2 * blockIdx.x + (g.kv0 > 0 ? 0 : 1);
                // O (this copy) * f * fv = its share of the normalised output
                const float f = any ? ex2(mc == -INFINITY ? 0.0f : mc - M) / L : 0.0f;
                const float fv = pow2i(ev - 127 - kShift);
                auto share = [&](int k, float (&y)[16]) {  // of channels [k, k + 16)
                    uint32_t o[16];
                    ld_cols(tl + S::CO + k, o);
                    wait_ld();
                    const bool bad = (nanblk >> (k / 32)) & 1u;
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        y[j] = bad ? __uint_as_float(0x7FC00000u) : any ? __uint_as_float(o[j]) * f * fv : 0.0f;
                };
                const float Lt = L * pow2i(-(int)kBias);  // the sum in units of 2^M
                if (set == 0 && copy == 0 && real) {
                    if (!whole)
                        p.stat[(size_t)slotw * RT + row] = make_float2(M, Lt);
                    else if (p.lse)
                        p.lse[((size_t)g.b * p.T + t) * p.Hq + hq] =
                            L == 0.0f ? -INFINITY : (M + log2f(Lt)) * 0.69314718055994531f;
                }
                if constexpr (REP == 1) {
#pragma unroll 1
                    for (int k = set * (D / 2); k < (set + 1) * (D / 2); k += 16) {
                        float y[16];
                        share(k, y);
                        if (real) store_row<RT, D>(p, g, whole, slotw, row, t, hq, k, y);
                    }
                } else {
                    // through shared memory, W channels of the real rows of every copy at a time (padded to
                    // W + 1 floats a row); then a thread takes four channels of a row, the copies in order
                    float *const stage = reinterpret_cast<float *>(base + S::oStage) + set * (128 * 17);
                    const int rows = min(RT, g.nodes * p.g - g.rt * RT);
                    const int W = rows * REP <= 32 ? 64 : rows * REP <= 64 ? 32 : 16;
                    const int W1 = W + 1, W4 = W / 4, own = 32 * quad + lane;
                    const int c1 = (set + 1) * (D / 2);
                    for (int k0 = set * (D / 2); k0 < c1; k0 += W) {
                        const int wd = min(W, c1 - k0);
#pragma unroll 1
                        for (int k = 0; k < wd; k += 16) {
                            float y[16];
                            share(k0 + k, y);
                            if (row < rows)
#pragma unroll
                                for (int j = 0; j < 16; ++j) stage[(copy * rows + row) * W1 + k + j] = y[j];
                        }
                        ok = set_sync();
                        if (!ok) break;
                        for (int u = own; u < rows * W4; u += 128) {
                            const int rr = u / W4, j0 = 4 * (u - rr * W4);
                            if (j0 >= wd) continue;
                            float z[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                z[j] = stage[rr * W1 + j0 + j];
#pragma unroll
                                for (int q = 1; q < REP; ++q) z[j] += stage[(rr + q * rows) * W1 + j0 + j];
                            }
                            const int r2 = g.rt * RT + rr;
                            const int t2 = r2 / p.g, h2 = g.h * p.g + (r2 - t2 * p.g);
                            store_row<RT, D>(p, g, whole, slotw, rr, t2, h2, k0 + j0, z);
                        }
                        ok = set_sync();
                        if (!ok) break;
                    }
                }
                // the statistics are read, and O is, before the next tile's writes
                if (!ok) break;
                ok = soft_sync();
                if (!ok) break;
            }
            if (!more) break;
            g = next;
            const int tiles = g.kv1 - g.kv0;
            r = g.rt * RT + row;
            real = r < g.nodes * p.g;
            t = real ? r / p.g : 0;
            hq = g.h * p.g + (real ? r - t * p.g : 0);
            const float c = p.scale_log2 * pow2i(eq);  // S -> x
            // The largest key exponent byte e for which no |x| of the warp's rows can reach 2^kLarge:
            // |S| <= D 2^8 2^9 2^(e - 127), and S c = x with c < 2^above.
            const int above = (int)(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(c)) >> 23) - 126;
            const int narrow = kLarge - 17 - (D == 64 ? 6 : D == 128 ? 7 : 8) + 127 - above;

            m = -INFINITY;
            l = 0.0f;
            nanblk = 0;
            const int32_t *mrow = p.mask ? p.mask + ((size_t)g.b * p.T + t) * p.W : nullptr;
            for (int i = 0; i < tiles && ok; ++i, ++it) {
                if ((it & 1) != set) continue;
                const int info = it % kInfo, buf = set;
                const uint32_t tph = (uint32_t)((it >> 1) & 1);
                ok = wait(&s.s_full[buf], tph);
                if (!ok) break;
                fence_after();
                const TileInfo inf = load_info(&s.info[info]);
                const uint32_t tb = tl + S::CS + buf * TN, ts = tb + col0;
                const int slot0 = (g.kv0 + i) * TN + col0;  // cache slot of the thread's first column
                const uint32_t vb = (uint32_t)inf.valid;
                const bool masked = (g.kv0 + i + 1) * TN > g.ctx || vb != (1u << (TN / 16)) - 1u;
                // visible keys among columns [k, k + 32) of the thread
                auto seen = [&](int k) -> uint32_t {
                    const int s0 = slot0 + k, j0 = s0 - g.ctx;  // node of the first column (negative: context)
                    uint32_t w = low_bits(-j0);
                    if (j0 > -32 && j0 < g.nodes) {
                        uint32_t tree;
                        if (mrow) {
                            const int wi = j0 >> 5, sh = j0 & 31;  // floor division: wi = -1 before node 0
                            const uint32_t a = wi >= 0 ? (uint32_t)mrow[wi] : 0u;
                            const uint32_t b = wi + 1 < p.W ? (uint32_t)mrow[wi + 1] : 0u;
                            tree = __funnelshift_r(a, b, sh);
                        } else {
                            tree = low_bits(t + 1 - j0);
                        }
                        w |= tree & ~low_bits(-j0) & low_bits(g.nodes - j0);
                    }
                    const uint32_t gb = vb >> ((col0 + k) >> 4);
                    w &= ((gb & 1u) ? 0x0000FFFFu : 0u) | ((gb & 2u) ? 0xFFFF0000u : 0u);
                    return w;
                };
                // Scores that may be large become x, rounded, in place, and then have their maximum exactly.
                const bool wide = inf.flags >> 8 > narrow;
                const float ct = wide ? 1.0f : c, cm = wide ? c : 1.0f;
                if (masked || wide) {  // S of what a row does not see becomes -inf, in place
                    constexpr int MC = CPT < 32 ? CPT : 32;
#pragma unroll 1
                    for (int k = 0; k < CPT; k += MC) {
                        const uint32_t w = masked ? seen(k) : 0xFFFFFFFFu;
                        uint32_t y[MC];
                        ld_cols(ts + k, y);
                        wait_ld();
#pragma unroll
                        for (int j = 0; j < MC; ++j) y[j] = (w >> j) & 1u ? __float_as_uint(__uint_as_float(y[j]) * cm) : 0xFF800000u;
                        st_cols(ts + k, y);
                    }
                    wait_st();
                }
                const float ml = m;    // the rows' m at the set's last tile, and
                float mp = -INFINITY;  // at the tile before, the other set's
                auto receive = [&]() -> bool {
                    if (i == 0) return true;
                    if (!wait(&s.m_full[set ^ 1][quad], (uint32_t)(((it - 1) >> 1) & 1))) return false;
                    mp = s.mrow[set ^ 1][32 * quad + lane];
                    return true;
                };
                // from the thread's largest S: the rows' m at this tile, handed on to the other set
                auto settle = [&](float mt) {
                    const float me = mt == -INFINITY ? mt : mt * ct;
                    m = me - mp > kSlack ? me : mp;  // also out of -inf
                    s.mrow[set][32 * quad + lane] = m;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s.m_full[set][quad]);
                };
                // bias - m; of a large m less than that by up to its last place, so that p stays in range
                auto offset = [](float m) -> float {
                    return m == -INFINITY ? 0.0f : fabsf(m) < (float)(1 << kLarge) ? kBias - m : __fadd_rd(kBias, -m);
                };
                uint64_t sum;
                // p = 2^(x - m + bias) of a chunk, its sum and its f16 pairs
                auto powers = [&](const uint32_t (&y)[CH], uint64_t c2, uint64_t off2, uint32_t *out) {
#pragma unroll
                    for (int j = 0; j < CH; j += 2) {
                        float a, b;
                        fma2(a, b, y[j], y[j + 1], c2, off2);
                        a = ex2(a);
                        b = ex2(b);
                        sum = add2(sum, pair(a, b));
                        out[j / 2] = pack_f16(a, b);
                    }
                };
                auto largest = [&](const uint32_t (&y)[CH], float &m0, float &m1) {
#pragma unroll
                    for (int j = 0; j < CH; j += 4) {
                        m0 = max3(m0, __uint_as_float(y[j]), __uint_as_float(y[j + 1]));
                        m1 = max3(m1, __uint_as_float(y[j + 2]), __uint_as_float(y[j + 3]));
                    }
                };
                float m0 = -INFINITY, m1 = -INFINITY;
                if constexpr (CPT <= 64) {
                    // One pass, with the set's last m: after a segment's first tiles the maximum hardly
                    // ever passes it by more than the slack.  Else a second, with the m that the first
                    // found.  P waits in registers for that, as it takes S's place.
                    uint32_t pk[CPT / 2];
                    bool again = false;
#pragma unroll 1
                    while (true) {
                        const float off = offset(m);
                        const uint64_t c2 = pair(ct, ct), off2 = pair(off, off);
                        sum = pair(0.0f, 0.0f);
                        uint32_t x[CPT > CH ? 2 : 1][CH];
                        ld_cols(ts, x[0]);
                        if (!again) ok = receive();
                        wait_ld();
                        if (!ok) break;
#pragma unroll
                        for (int k = 0; k < CPT; k += CH) {
                            uint32_t(&y)[CH] = x[CPT > CH ? (k / CH) & 1 : 0];
                            if constexpr (CPT > CH)
                                if (k + CH < CPT) ld_cols(ts + k + CH, x[(k / CH + 1) & 1]);  // on its way meanwhile
                            largest(y, m0, m1);
                            powers(y, c2, off2, pk + k / 2);
                            if (CPT > CH) wait_ld();
                        }
                        if (again) break;
                        settle(fmaxf(m0, m1));
                        again = __any_sync(0xFFFFFFFFu, m != ml);
                        if (!again) break;
                    }
                    if (!ok) break;
                    st_cols(tb + col0 / 2, pk);
                    if constexpr (REP > 1) {  // P is zero at the other copies' keys
                        const uint32_t z[CPT / 2] = {};
#pragma unroll
                        for (int q = 0; q < REP; ++q)
                            if (q != copy) st_cols(tb + q * (CPT / 2), z);
                    }
                } else {
                    // Two passes: 64 registers of P on top of the rest would spill.  Both unrolled, 16 columns on their
                    // way while the 16 before are worked on (193 us long trees; 32 at a time in a loop: 205).
                    ok = receive();
                    if (!ok) break;
                    uint32_t x[2][CH], pk[CH / 2];
                    ld_cols(ts, x[0]);
#pragma unroll
                    for (int k = 0; k < CPT; k += CH) {
                        wait_ld();
                        ld_cols(ts + (k + CH) % CPT, x[(k / CH + 1) & 1]);  // the last: the first again
                        largest(x[(k / CH) & 1], m0, m1);
                    }
                    settle(fmaxf(m0, m1));
                    const float off = offset(m);
                    const uint64_t c2 = pair(ct, ct), off2 = pair(off, off);
                    sum = pair(0.0f, 0.0f);
                    static_assert(CPT / CH % 2 == 0 || CPT <= 64);
#pragma unroll
                    for (int k = 0; k < CPT; k += CH) {  // a chunk's P lands on columns already read
                        wait_ld();
                        if (k + CH < CPT) ld_cols(ts + k + CH, x[(k / CH + 1) & 1]);
                        powers(x[(k / CH) & 1], c2, off2, pk);
                        st_cols(tb + k / 2, pk);
                    }
                }
                const bool grow = m != mp;
                // ---- O in the units of the new maximum and value exponent
                if (i > 0) {
                    if (__any_sync(0xFFFFFFFFu, grow || inf.rise)) {
                        ok = wait(&s.pv_done[buf ^ 1], (uint32_t)(((it - 1) >> 1) & 1));
                        if (!ok) break;
                        fence_after();
                        const float f = (grow ? (mp == -INFINITY ? 0.0f : ex2(mp - m)) : 1.0f) * pow2i(max(-inf.rise, -149));
#pragma unroll 1
                        for (int k = 0; k < D; k += 32) {
                            uint32_t o[32];
                            ld_cols(tl + S::CO + k, o);
                            wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                            st_cols(tl + S::CO + k, o);
                        }
                    }
                }
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.p_full[buf]);
                l = l * (m == ml ? 1.0f : ml == -INFINITY ? 0.0f : ex2(ml - m)) + sum_pair(sum);
                if (inf.flags & 2) {
#pragma unroll 1
                    for (int k = 0; k < CPT; k += 32) {
                        const uint32_t w = real ? (masked ? seen(k) : 0xFFFFFFFFu) : 0u;
#pragma unroll 1
                        for (int j = 0; j < CPT - k && j < 32; ++j)
                            if ((w >> j) & 1u) nanblk |= s.nanblk[info][col0 + k + j];
                    }
                }
            }
            if (!ok) break;
        }
    }

    if (!ok) report_timeout(p.status);
    free_tmem(tmem, warp == kMmaWarp);
}

// ------------------------------------------------------------------ host side

namespace {

// Rows a tile: the smallest that holds all of a request's rows of a head, 128 past that; fewer would read
// the cache again.
int row_tile(int T, int g) { return T * g <= 32 ? 32 : T * g <= 64 ? 64 : 128; }

// Up to 8 rows at dim 128 the kernel with keys in the lanes, where requests may be longer than 2048
// tokens: 64 requests x 8 heads x 8 rows, contexts of all lengths up to 4000, 16000: 71, 186 us there, 78, 227
// in the one for 32 rows; up to 200, 2000: 28.6, 56.1 there, 28.3, 53.4 here; one request of 50, 16000: 11.5,
// 16.2 there, 10.2, 18.2 here.  (For 16 rows it took a third longer than the one for 32 at every length, at
// dim 64 as long.)
bool few_rows(int T, int g, int dim, int max_len) { return dim == 128 && T * g <= kFewRows && max_len > 2048; }

size_t round16(size_t n) { return (n + 15) / 16 * 16; }

using EncodeTiledFnA = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                    const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                    CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFnA encode_fn_a() {
    static EncodeTiledFnA fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFnA>(f);
    });
    return fn;
}

// Codes as [rows][dim] bytes; a box is box_rows rows (inside a page and a tile) of at most
// 128 bytes, swizzled by its width.
cudaError_t code_map(const CacheView &c, void *codes, int box_rows, CUtensorMap *out) {
    EncodeTiledFnA fn = encode_fn_a();
    if (!fn) return cudaErrorNotSupported;
    const cuuint32_t w = (cuuint32_t)std::min(c.dim, 128);
    const cuuint64_t dims[2] = {(cuuint64_t)c.dim, (cuuint64_t)c.pages * c.heads * c.page_size};
    const cuuint64_t strides[1] = {(cuuint64_t)c.dim};
    const cuuint32_t box[2] = {w, (cuuint32_t)box_rows}, es[2] = {1u, 1u};
    const CUresult r = fn(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, codes, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          w == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D>
cudaError_t launch_attend_dim(const AttendParams &prm, cudaStream_t stream) {
    switch (row_tile(prm.T, prm.g)) {
        case 32: return launch_attend_shape<Shape<D, 32>>(attend_kernel<D, 32>, prm, stream);
        case 64: return launch_attend_shape<Shape<D, 64>>(attend_kernel<D, 64>, prm, stream);
        default: return launch_attend_shape<Shape<D, 128>>(attend_kernel<D, 128>, prm, stream);
    }
}

}  // namespace

// Two partials a block, their statistics, and the prefix sums; 16 bytes to start on a whole sector.
size_t attend_workspace_bytes(int B, int T, int Hq, int heads, int dim) {
    const size_t rows = (size_t)kAttendBlocks * 2 * row_tile(T, Hq / heads);
    return 16 + rows * dim * 4 + rows * 8 + round16(((size_t)B + 1) * 4);
}

// Places of the largest call these arguments allow (work_of's sums); they are counted in 31 bits.
bool attend_fits(const CacheView &c, int B, int T, int Hq, int max_len) {
    const int g = Hq / c.heads, rt = row_tile(T, g), tn = c.dim == 256 ? 64 : 128;
    const int start = few_rows(T, g, c.dim, max_len) ? kFewStart : kStart;
    return (double)B * c.heads * (((long long)T * g + rt - 1) / rt) * (((long long)max_len + tn - 1) / tn + start) < 2147483648.0;
}

cudaError_t launch_attend(const CacheView &c, const AttendArgs &a, cudaStream_t stream) {
    AttendParams prm{};
    prm.c = c;
    const int tn = c.dim == 256 ? 64 : 128;
    prm.box_rows = 16;  // the largest power of two that divides a page, up to a tile
    while (prm.box_rows < tn && c.page_size % (2 * prm.box_rows) == 0) prm.box_rows *= 2;
    prm.page_magic = (1ull << 32) / (unsigned)(c.page_size / 16) + 1;
    cudaError_t e = code_map(c, c.k8, prm.box_rows, &prm.kmap);
    if (e == cudaSuccess) e = code_map(c, c.v8, prm.box_rows, &prm.vmap);
    if (e != cudaSuccess) return e;
    prm.q = a.q;
    prm.ldq = a.ldq;
    prm.ctx = a.ctx;
    prm.nodes = a.nodes;
    prm.mask = a.mask;
    prm.scale_log2 = a.scale * 1.4426950408889634f;
    prm.max_len = a.max_len;
    prm.out = a.out;
    prm.lse = a.lse;
    prm.B = a.B;
    prm.T = a.T;
    prm.Hq = a.Hq;
    prm.g = a.Hq / c.heads;
    prm.W = (a.T + 31) / 32;
    const int rt = row_tile(a.T, prm.g);  // the workspace holds 32 rows where 8 are used
    const size_t rows = (size_t)kAttendBlocks * 2 * rt;
    prm.part = reinterpret_cast<float *>((reinterpret_cast<uintptr_t>(a.workspace) + 31) / 32 * 32);
    prm.stat = reinterpret_cast<float2 *>(prm.part + rows * c.dim);
    prm.prefix = reinterpret_cast<int *>(prm.stat + rows);
    const Options opt = options();
    prm.timeout_ns = opt.timeout_ns;
    prm.tries = (uint32_t)std::min<unsigned long long>(std::max<unsigned long long>(opt.timeout_ns / kSuspendNs, 1), 0x7FFFFFFFu);
    prm.skip_loads = opt.skip_loads;
    prm.status = status_word();
    if (!prm.status) return cudaErrorInvalidSymbol;
    if (few_rows(a.T, prm.g, c.dim, a.max_len)) return launch_attend_few(prm, stream);
    switch (c.dim) {
        case 64: return launch_attend_dim<64>(prm, stream);
        case 128: return launch_attend_dim<128>(prm, stream);
        case 256: return launch_attend_dim<256>(prm, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace bsf8
