// bsf8_attend.cu -- attention of a token tree over the paged block-scaled fp8 cache (tcgen05).
//
//   out[row] = sum_l 2^(x_l - m) v_l / sum_l 2^(x_l - m),   x_l = scale log2(e) q[row].k_l,
// over the keys l that the row sees; a row is a (node, query head) of one request and cache
// head.  One pass over the cache with the running maximum m and sum of a softmax.
//
// Work.  An item is a tile of TN keys (128; 64 at dim 256) of one (request, head, tile of RT
// rows).  The items of all requests, in that order, are cut into one equal contiguous range per
// block (one block an SM), whatever the requests' lengths: every block computes the same prefix
// sums of the requests' items.  A block's range is a run of segments (consecutive keys of one
// row tile).  A segment that holds all keys of its rows writes the output; any other writes a
// partial (its rows' normalised output, maximum and sum) to one of the block's two workspace
// slots -- only a block's first and last segment can be incomplete -- and a second kernel
// joins the partials of each row in block order.  Nothing depends on timing: the same call
// gives the same bits.
//
// A block's warps, each with its own loop over the items:
//   producer  bulk copies of the codes (page runs of a head are contiguous) and cp.async of the
//             exponents into a ring of slots, K(0) K(1) V(0) K(2) V(1) ...;
//   8 dequant a slot's codes -> f16 tiles in shared memory (128-byte swizzle), as
//             code * 2^(e - E + 6), E the largest exponent of the tile (keys), or of the segment
//             so far (values): exact for exponents within 2^21 of E, else off by at most 2^-31
//             of 2^E; e4m3 times a power of two needs no more than f16's 11 bits;
//   MMA       one thread: S = Q K^T (Q in tensor memory as A, f16 scaled by a power of two a
//             row; exact products, fp32 sums), then O += P V (P in tensor memory as A, V as an
//             N-major B);  S(i + 1) is issued before O(i), so it runs under softmax(i);
//   4 softmax thread = row: maximum, p = 2^(x - m + 13) (fp32, summed in fp32), rounded to f16
//             for the second product: 11 bits of p at any p above 2^-27 of the largest, half of
//             2^-37 of it below.  (bf16 would round p to 8 bits: 1.4 times the error of the
//             output's own rounding.)  m only moves when the maximum has grown by more than
//             2^2 over it, which keeps p <= 2^15 and rescaling O (a round trip of O through
//             registers) rare.
// RT rows of Q fill the MMA's 128 rows 128 / RT times; each copy handles its own part of the
// tile's key columns (its P is zero elsewhere), so that with few rows all four softmax warps
// still work; the copies' maxima, sums and outputs join at the segment's end.
// Masks are 32-bit words a row and 32 keys; tiles wholly inside the context skip them.  Keys
// past a request's end (a page's unused slots may hold anything) and keys on bad pages are
// masked, and their values are zeroed; a value block that holds NaN is zeroed too, and the rows
// that see it get their NaN at the end, so that it reaches no other row.
//
// Bound: the cache is read once, 2 dim (1 + 1/32) bytes a key and head, from HBM; the shared
// memory of an SM (codes in, codes out, f16 in, the MMA's read of f16) is nearly as busy.
#include "bsf8_device.cuh"
#include "bsf8_internal.h"

#include <cuda.h>

#include <algorithm>
#include <mutex>

namespace bsf8 {

namespace {

constexpr int kAttendBlocks = 152;   // one an SM of a GB300 (no block waits for another)
constexpr int kMaxBatch = 1024;
constexpr int kSoftWarps = 8;        // two sets of four, a set every other tile
constexpr int kDeqWarps = 8;
constexpr int kProducerWarp = kSoftWarps + kDeqWarps, kScoutWarp = kProducerWarp + 1;
constexpr int kMmaWarp = kScoutWarp + 1;  // two: S, O
constexpr int kThreadsA = (kMmaWarp + 2) * 32;
constexpr int kInfo = 8;             // tiles whose exponents and flags are kept
constexpr float kBias = 13.0f;       // p = 2^(x - m + kBias)
constexpr float kSlack = 2.0f;       // m lags the maximum by at most this
constexpr int kShift = 6;            // f16 values are code * 2^(e - E + kShift)

template <int D>
struct Shape {
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
    static constexpr int oV = 0, oK = 2 * F16, oRing = oK + NSLOT * SLOT, oQ = oRing + NSLOT * SLOT;
    static constexpr int oExp = oQ + (QS ? 2 * 128 * D : 0), oStage = oExp + NSLOT * 1024;
    static constexpr int oPrefix = oStage + 2 * 128 * 17 * 4;
};

// At least 176 KB, so that no block of another kernel that holds tensor memory (84 KB of shared
// memory and more each) shares the SM: this block takes all 512 columns, and two blocks that
// each wait for the other's columns or for its grid would never end.
template <int D>
constexpr int attend_smem(int B) {
    return std::max(176 * 1024, 1024 + Shape<D>::oPrefix + (B + 1) * 4);
}

struct AttendParams {
    unsigned long long page_magic;  // floor(2^32 / (page_size / 16)) + 1: divides 16-key groups by a page's
    CUtensorMap kmap;  // the key codes as rows of D bytes, box min(D, 128) x box_rows, swizzled
    int box_rows;
    CacheView c;
    const uint16_t *q;
    long long ldq;
    const int32_t *ctx, *nodes, *mask;
    float scale_log2;  // scale * log2(e)
    int max_len;
    uint16_t *out;
    float *lse;
    int B, T, Hq, g, W;  // g: query heads a cache head, W: mask words a row
    float *part;         // [blocks][2][RT][D] normalised outputs
    float2 *stat;        // [blocks][2][RT] (m, sum)
    int *prefix;         // [B + 1] the requests' items, for the join
    uint32_t tries;      // suspensions of a wait
    unsigned long long timeout_ns;
    int skip_loads;
    int *status;
};

// A request's context and node counts, inside their bounds.
__device__ __forceinline__ bool lengths(const AttendParams &p, int b, int &ctx, int &nodes) {
    ctx = p.ctx[b];
    nodes = p.nodes ? p.nodes[b] : p.T;
    if (ctx >= 0 && nodes >= 0 && nodes <= p.T && (long long)ctx + nodes <= p.max_len) return true;
    ctx = max(0, min(ctx, p.max_len));
    nodes = max(0, min(nodes, min(p.T, p.max_len - ctx)));
    return false;
}

template <int D, int RT>
__device__ __forceinline__ int items_of(const AttendParams &p, int ctx, int nodes) {
    if (nodes == 0) return 0;
    const int nt = (ctx + nodes + Shape<D>::TN - 1) / Shape<D>::TN;
    return p.c.heads * ((nodes * p.g + RT - 1) / RT) * nt;
}

// The work of block w: items [w total / W, (w + 1) total / W).
__device__ __forceinline__ int range_start(long long total, int w) {
    return (int)(total * w / kAttendBlocks);
}

struct Segment {
    int b, h, rt, kv0, kv1, nt, ctx, nodes;
};

// The segment at item pos of a block whose range ends at end.
template <int D, int RT>
__device__ __forceinline__ Segment segment_at(const AttendParams &p, const int *prefix, int pos, int end) {
    Segment s{};
    if (pos >= end) return s;
    int lo = 0, hi = p.B;  // prefix[lo] <= pos < prefix[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= pos) lo = mid;
        else hi = mid;
    }
    s.b = lo;
    (void)lengths(p, lo, s.ctx, s.nodes);
    s.nt = (s.ctx + s.nodes + Shape<D>::TN - 1) / Shape<D>::TN;
    const int rts = (s.nodes * p.g + RT - 1) / RT;
    const int rem = pos - prefix[lo];
    const int seg = rem / s.nt;
    s.kv0 = rem - seg * s.nt;
    s.kv1 = min(s.nt, s.kv0 + (end - pos));
    s.h = seg / rts;
    s.rt = seg - s.h * rts;
    return s;
}

// The segment after s, at item pos < end.
template <int D, int RT>
__device__ __forceinline__ void next_segment(const AttendParams &p, Segment &s, int pos, int end) {
    if ((++s.rt) * RT >= s.nodes * p.g) {
        s.rt = 0;
        if (++s.h == p.c.heads) {
            s.h = 0;
            do {
                (void)lengths(p, ++s.b, s.ctx, s.nodes);
            } while (s.nodes == 0);  // ends: there are items left
            s.nt = (s.ctx + s.nodes + Shape<D>::TN - 1) / Shape<D>::TN;
        }
    }
    s.kv0 = 0;
    s.kv1 = min(s.nt, end - pos);
}

// ------------------------------------------------------------------ tcgen05 wrappers

// Shared-memory matrix descriptors, 128-byte swizzle: rows of 128 bytes, 8-row atoms of 1024
// bytes.  K-major (keys: a row is a key's 64 channels): stride 1024 between 8-key groups.
// N-major (values: a row is 64 channels of one key, the contraction): stride 1024 between
// 8-key groups, leading offset between 64-channel columns.
__device__ __forceinline__ uint64_t desc_a(uint32_t saddr, uint32_t lead) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lead >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// kind::f16, fp32 accumulator, f16 A and B, A K-major, M = 128.
__device__ __forceinline__ constexpr uint32_t idesc_a(int n, bool n_major) {
    return (1u << 4) | (n_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

__device__ __forceinline__ void umma_a(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// kind::mxf8f6f4, e4m3 A and B with a power-of-two scale (ue8m0) per row and 32 channels, fp32
// accumulator, M = 128; sa, sb: which byte of the scales' words.
__device__ __forceinline__ constexpr uint32_t idesc_mx(int n, int sa, int sb) {
    return ((uint32_t)sb << 4) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(128 >> 4) << 24) |
           ((uint32_t)sa << 29);
}

__device__ __forceinline__ void umma_mx_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                           uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], [%1], %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void umma_mx_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                           uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
}

// Codes of K (or Q): rows of RB = 128 or 64 bytes with the swizzle of that width, 8-row atoms.
template <int RB>
__device__ __forceinline__ uint64_t desc_codes(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)(8 * RB >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)(RB == 128 ? 2 : 4) << 61);
}

// 32 rows of 16 bytes, unswizzled (8-row groups of 128 bytes one after another) -> four tensor
// memory columns of 32 lanes, repeated in all four lane quarters.
__device__ __forceinline__ uint64_t desc_scales(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}

__device__ __forceinline__ void copy_scales(uint32_t t, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(t), "l"(desc) : "memory");
}

__device__ __forceinline__ void tma_rows(void *dst, const CUtensorMap *map, int col, int row, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(row), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void commit_a(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void ld_cols(uint32_t t, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(t)
                 : "memory");
}

__device__ __forceinline__ void ld_cols(uint32_t t, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t)
        : "memory");
}

__device__ __forceinline__ void ld_cols(uint32_t t, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(t)
        : "memory");
}

__device__ __forceinline__ void st_cols(uint32_t t, const uint32_t (&r)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(t), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3])
                 : "memory");
}

__device__ __forceinline__ void st_cols(uint32_t t, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

__device__ __forceinline__ void st_cols(uint32_t t, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void st_cols(uint32_t t, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(t),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
        "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
        "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// ------------------------------------------------------------------ small arithmetic

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));  // relative error about 2^-22
    return y;
}

// (x0, x1) * c + off and a + b, two fp32 at a time.
__device__ __forceinline__ void fma2(float &y0, float &y1, uint32_t x0, uint32_t x1, uint64_t c, uint64_t off) {
    uint64_t x, y;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "r"(x0), "r"(x1));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y) : "l"(x), "l"(c), "l"(off));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(y0), "=f"(y1) : "l"(y));
}

__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t x;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
    return x;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t y;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(a), "l"(b));
    return y;
}

__device__ __forceinline__ float sum_pair(uint64_t a) {
    float x, y;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a));
    return x + y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// f16 pair -> e4m3 pair, nearest even.
__device__ __forceinline__ uint32_t f16_to_e4m3(uint32_t two) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(d) : "r"(two));
    return d;
}

__device__ __forceinline__ uint32_t f16x2_sub(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t e4m3_to_f16(uint16_t two) {
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(two));
    return d;
}

__device__ __forceinline__ float pow2i(int k) {  // 2^k, k >= -149; 0 below
    return k >= -126 ? __uint_as_float((uint32_t)(k + 127) << 23)
                     : (k >= -149 ? __uint_as_float(1u << (k + 149)) : 0.0f);
}

// 2^k as an f16 pair, k clamped to [-30 (0), 40 (inf)].
__device__ __forceinline__ uint32_t f16_pow2(int k) {
    const float f = __uint_as_float((uint32_t)(min(max(k, -30), 40) + 127) << 23);
    return pack_f16(f, f);
}

// 16 codes times the scale pair sc -> 16 f16.
__device__ __forceinline__ void widen16(const uint4 &w, uint32_t sc, uint4 &lo, uint4 &hi) {
    lo.x = f16x2_mul(e4m3_to_f16((uint16_t)w.x), sc);
    lo.y = f16x2_mul(e4m3_to_f16((uint16_t)(w.x >> 16)), sc);
    lo.z = f16x2_mul(e4m3_to_f16((uint16_t)w.y), sc);
    lo.w = f16x2_mul(e4m3_to_f16((uint16_t)(w.y >> 16)), sc);
    hi.x = f16x2_mul(e4m3_to_f16((uint16_t)w.z), sc);
    hi.y = f16x2_mul(e4m3_to_f16((uint16_t)(w.z >> 16)), sc);
    hi.z = f16x2_mul(e4m3_to_f16((uint16_t)w.w), sc);
    hi.w = f16x2_mul(e4m3_to_f16((uint16_t)(w.w >> 16)), sc);
}

// Bits [0, n) set, n clamped to [0, 32].
__device__ __forceinline__ uint32_t low_bits(int n) {
    return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
}

__device__ __forceinline__ uint32_t pack_bf(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// N channels (from k) of a row's output: bf16 where the segment is the whole row, else a partial.
template <int RT, int D, int N>
__device__ __forceinline__ void store_row(const AttendParams &p, const Segment &g, bool whole, int slotw, int row,
                                          int t, int hq, int k, const float (&y)[N]) {
    if (whole) {
        uint16_t *dst = p.out + (((size_t)g.b * p.T + t) * p.Hq + hq) * D + k;
#pragma unroll
        for (int j = 0; j < N; j += 4)
            *reinterpret_cast<uint2 *>(dst + j) = make_uint2(pack_bf(y[j], y[j + 1]), pack_bf(y[j + 2], y[j + 3]));
    } else {
        float *dst = p.part + ((size_t)slotw * RT + row) * D + k;
#pragma unroll
        for (int j = 0; j < N; j += 4)
            *reinterpret_cast<float4 *>(dst + j) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
    }
}

// Waits for a phase of `bar`, at most `tries` suspensions of kSuspendNs each; false when they ran out.
// A few instructions: every role has several waits, and the block's roles share an SM's instruction
// caches.
constexpr uint32_t kSuspendNs = 20000;

__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity, uint32_t tries) {
    uint32_t left;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\tmov.u32 n, %3;\n"
        "AGAIN:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %4;\n\t"
        "@p bra DONE;\n\t"
        "sub.u32 n, n, 1;\n\t"
        "setp.ne.u32 q, n, 0;\n\t"
        "@q bra AGAIN;\n"
        "DONE:\n\t"
        "mov.u32 %0, n;\n\t}"
        : "=r"(left)
        : "r"(smem_u32(bar)), "r"(parity), "r"(tries), "r"(kSuspendNs)
        : "memory");
    return left != 0;
}

struct AttendShared {
    uint64_t k_full[4], k_free[4];  // ring slots of keys: codes landed and scales written; multiplied
    uint64_t c_full[4], c_free[4];  // of values: codes landed and exponents written; read by all dequant warps
    uint64_t v_full[2];             // the f16 values of a tile are written
    uint64_t s_full[2];             // S written
    uint64_t p_full[2];             // P written, O rescaled
    uint64_t pv_done[2];            // O updated, P and the f16 values read
    uint64_t m_full[2][4];          // a softmax warp's rows have their maximum of the tile
    uint64_t q_full;                // a segment's Q is in place
    uint64_t soft, set[2];          // the softmax warps' own barriers (bounded, unlike bar.sync)
    uint32_t tmem;
    int valid[kInfo];               // a tile's 16-key groups that exist (bit i)
    int ev[kInfo], vnan[kInfo];     // the segment's value exponent at the tile; a value block holds NaN
    int care[kInfo];                // the tile's values need care: missing keys, NaN
    uint8_t nanblk[kInfo][128];     // then: each key's NaN blocks
    float mrow[2][128];             // the rows' maxima, handed from set to set
    float2 stat[kSoftWarps][32];
    uint32_t nan[kSoftWarps][32];
    int scan[32];
};

}  // namespace

template <int D, int RT>
__global__ void __launch_bounds__(kThreadsA, 1) attend_kernel(const __grid_constant__ AttendParams p) {
    using S = Shape<D>;
    constexpr int TN = S::TN, REP = 128 / RT, CPT = TN / REP;  // CPT: key columns a thread
    constexpr int CH = CPT <= 32 ? CPT : CPT == 64 ? 16 : 32;  // taken CH at a time
    extern __shared__ uint8_t dyn_smem[];
    uint8_t *const base = dyn_smem + ((1024u - (smem_u32(dyn_smem) & 1023u)) & 1023u);
    __shared__ AttendShared s;
    int *const prefix = reinterpret_cast<int *>(base + S::oPrefix);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&s.k_full[i], 2);  // the producer's byte count, the scout
            mbar_init(&s.k_free[i], 1);
            mbar_init(&s.c_full[i], 2);
            mbar_init(&s.c_free[i], kDeqWarps);
            mbar_init(&s.m_full[0][i], 1);
            mbar_init(&s.m_full[1][i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.v_full[i], kDeqWarps);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_full[i], 4);
            mbar_init(&s.pv_done[i], 1);
            mbar_init(&s.set[i], 4);
        }
        mbar_init(&s.q_full, kSoftWarps);
        mbar_init(&s.soft, kSoftWarps);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();  // tensor memory is held before the next kernel's blocks may come
    fence_after();
    pdl_trigger();
    pdl_wait();

    // ------------------------------------------------ prefix sums of the requests' items
    const int per = (p.B + kThreadsA - 1) / kThreadsA;
    {
        const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
        int sum = 0;
        for (int b = b0; b < b1; ++b) {
            int ctx, nodes;
            if (!lengths(p, b, ctx, nodes) && blockIdx.x == 0) report_index(p.status);
            sum += items_of<D, RT>(p, ctx, nodes);
            prefix[b + 1] = sum;  // within the thread's requests; completed below
        }
        int up = sum;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int o = __shfl_up_sync(0xFFFFFFFFu, up, m);
            if (lane >= m) up += o;
        }
        if (lane == 31) s.scan[warp] = up;
        __syncthreads();
        int before = up - sum;
        for (int w = 0; w < warp; ++w) before += s.scan[w];
        for (int b = b0; b < b1; ++b) prefix[b + 1] += before;
        if (threadIdx.x == 0) prefix[0] = 0;
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b <= p.B; b += kThreadsA) p.prefix[b] = prefix[b];
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, s.tmem, 0);
    const long long total = prefix[p.B];
    const int w0 = range_start(total, blockIdx.x), w1 = range_start(total, blockIdx.x + 1);
    // A bounded wait of one thread, or of a warp; false when it ran out (the thread reports it at its
    // role's end).
    auto wait1 = [&](uint64_t *bar, uint32_t parity) -> bool { return wait_phase(bar, parity, p.tries); };
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        return __all_sync(0xFFFFFFFFu, wait_phase(bar, parity, p.tries));
    };
    bool ok = true;  // no wait of this thread ran out
    // The block's first segment; each role walks on from it.
    const Segment first = segment_at<D, RT>(p, prefix, w0, w1);

    // A batch of BT tiles' 16-key groups, one a lane: the page of the lane's group (a load that stays
    // in flight until the batch is used), then its cache row (head h), -1 if there is none.
    constexpr int NSB = TN / 16, BT = 32 / NSB;
    // exact: group * (magic * d - 2^32) < 2^32 for groups below 2^26 and d <= 64
    auto in_page = [&](int grp) -> int { return (int)(((unsigned long long)(unsigned)grp * p.page_magic) >> 32); };
    auto page_of = [&](const Segment &g, int tile) -> int {
        const int grp = (tile + lane / NSB) * NSB + lane % NSB;
        return 16 * grp < g.ctx + g.nodes ? p.c.table[(size_t)g.b * p.c.table_pages + in_page(grp)] : -1;
    };
    auto row_of = [&](const Segment &g, int tile, int page) -> int {
        const int grp = (tile + lane / NSB) * NSB + lane % NSB;
        if (16 * grp >= g.ctx + g.nodes) return -1;
        if ((unsigned)page >= (unsigned)p.c.pages) {
            report_index(p.status);
            return -1;
        }
        return (page * p.c.heads + g.h - in_page(grp)) * p.c.page_size + 16 * grp;
    };

    if (warp == kProducerWarp) {
        // ------------------------------------------------------------ producer: codes
        const int gpb = p.box_rows / 16;  // groups a box: boxes never cross a page's end
        const bool lead = lane < NSB && lane % gpb == 0;
        int tile = 0;
        Segment g = first;
        for (int pos = w0; pos < w1 && ok;) {
            const int tiles = g.kv1 - g.kv0;
            int page = page_of(g, g.kv0), rows = -1;
            for (int i = 0; i < tiles; ++i, ++tile) {
                const int j = i % BT;
                if (j == 0) {
                    rows = row_of(g, g.kv0 + i, page);
                    page = page_of(g, g.kv0 + i + BT);
                }
                const int row = __shfl_sync(0xFFFFFFFFu, rows, (j * NSB + lane) & 31);
                const bool go = lead && row >= 0;
                const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xFFFFFFFFu, go)) * (uint32_t)(p.box_rows * D);
                const int slot = tile % S::NSLOT;
                const uint32_t fph = (uint32_t)((tile / S::NSLOT) & 1) ^ 1u;
                ok = tile < S::NSLOT || wait(&s.k_free[slot], fph);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(&s.k_full[slot], bytes);
                __syncwarp();
                if (go && !p.skip_loads)
#pragma unroll
                    for (int c = 0; c < D; c += 128)  // 128-byte columns of the tile, one after another
                        tma_rows(base + S::oK + slot * S::SLOT + c * TN + lane * 16 * (D < 128 ? D : 128), &p.kmap, c, row,
                                 &s.k_full[slot]);
                ok = tile < S::NSLOT || wait(&s.c_free[slot], fph);
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(&s.c_full[slot], bytes);
                __syncwarp();
                if (go && !p.skip_loads)
                    bulk_g2s(base + S::oRing + slot * S::SLOT + lane * 16 * D, p.c.v8 + (size_t)row * D,
                             (uint32_t)(p.box_rows * D), &s.c_full[slot]);
            }
            pos += tiles;
            if (pos < w1) next_segment<D, RT>(p, g, pos, w1);
        }
        // every copy must have landed before the block's memory goes away (bounded)
        if (!p.skip_loads)
            for (int i = max(0, tile - S::NSLOT); i < tile + (ok ? 0 : 1); ++i) {
                const int slot = i % S::NSLOT;
                const uint32_t iph = (uint32_t)((i / S::NSLOT) & 1);
                (void)mbar_wait_bounded(&s.k_full[slot], iph, ok ? p.timeout_ns : 100000000ull);
                (void)mbar_wait_bounded(&s.c_full[slot], iph, ok ? p.timeout_ns : 100000000ull);
            }
    } else if (warp == kScoutWarp) {
        // ------------------------------------------------------------ scout: exponents and flags
        constexpr int KPL = 16 / S::EB;  // keys of a lane's 16 exponent bytes
        const int key0 = lane * KPL;
        int tile = 0;
        Segment g = first;
        for (int pos = w0; pos < w1 && ok;) {
            const int tiles = g.kv1 - g.kv0;
            int E = 0;  // the largest value exponent of the segment so far
            int page = page_of(g, g.kv0), rows = -1;
            uint4 kx = make_uint4(0, 0, 0, 0), vx = kx, kn = kx, vn = kx;
            uint32_t vb = 0, vbn = 0;
            // starts the loads of tile i's exponents
            auto load = [&](int i) {
                const int j = i % BT;
                if (j == 0) {
                    rows = row_of(g, g.kv0 + i, page);
                    page = page_of(g, g.kv0 + i + BT);
                }
                const int row = __shfl_sync(0xFFFFFFFFu, rows, (j * NSB + lane) & 31);
                vbn = __ballot_sync(0xFFFFFFFFu, lane < NSB && row >= 0);
                const int krow = __shfl_sync(0xFFFFFFFFu, rows, (j * NSB + (key0 >> 4)) & 31);
                kn = vn = make_uint4(0, 0, 0, 0);
                if (key0 < TN && krow >= 0) {
                    const size_t at = ((size_t)krow + (key0 & 15)) * S::EB;
                    kn = *reinterpret_cast<const uint4 *>(p.c.kexp + at);
                    vn = *reinterpret_cast<const uint4 *>(p.c.vexp + at);
                }
            };
            for (int i = -1; i < tiles; ++i) {
                kx = kn;
                vx = vn;
                vb = vbn;
                if (i + 1 < tiles) load(i + 1);
                if (i < 0) continue;
                const int slot = tile % S::NSLOT, info = tile % kInfo;
                const uint32_t fph = (uint32_t)((tile / S::NSLOT) & 1) ^ 1u;
                ok = tile < S::NSLOT || (wait(&s.k_free[slot], fph) && wait(&s.c_free[slot], fph));
                if (!ok) break;
                // the keys' as tensor memory wants them -- 32 rows (lanes) of four words (columns): column
                // c of row l is key 32 c + l's word (dim 256: key 32 (c % 2) + l's word c / 2) -- the
                // values' as they are
                uint8_t *const ex = base + S::oExp + slot * 1024;
                if (key0 < TN) {
                    uint32_t *const kw = reinterpret_cast<uint32_t *>(ex) + (key0 & 31) * 4 + (key0 >> 5);
                    const uint32_t w[4] = {kx.x, kx.y, kx.z, kx.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if constexpr (D == 64) {
                            kw[8 * j] = w[j] & 0xFFFFu;
                            kw[8 * j + 4] = w[j] >> 16;
                        } else if constexpr (D == 128) {
                            kw[4 * j] = w[j];
                        } else {
                            kw[4 * (j >> 1) + 2 * (j & 1)] = w[j];
                        }
                    }
                    *reinterpret_cast<uint4 *>(ex + 512 + lane * 16) = vx;
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the scales go by tcgen05.cp
                // the largest value exponent of the keys that exist, 255 (NaN) left out
                const int keys = min(TN, g.ctx + g.nodes - (g.kv0 + i) * TN);
                const bool part = keys < TN || vb != (1u << NSB) - 1u;
                uint4 v = vx;
                if (part) {
                    const int bytes = (vb >> (key0 >> 4)) & 1 ? (keys - key0) * S::EB : 0;
                    v.x &= low_bits(8 * bytes);
                    v.y &= low_bits(8 * bytes - 32);
                    v.z &= low_bits(8 * bytes - 64);
                    v.w &= low_bits(8 * bytes - 96);
                }
                uint32_t mx = __vmaxu4(__vmaxu4(v.x, v.y), __vmaxu4(v.z, v.w));
                const bool nan = __any_sync(0xFFFFFFFFu, __vcmpeq4(mx, 0xFFFFFFFFu) != 0);
                if (nan) {
                    auto drop = [](uint32_t x) { return x & ~__vcmpeq4(x, 0xFFFFFFFFu); };
                    mx = __vmaxu4(__vmaxu4(drop(v.x), drop(v.y)), __vmaxu4(drop(v.z), drop(v.w)));
                }
                mx = __vmaxu4(mx, mx >> 16);
                E = max(E, (int)__reduce_max_sync(0xFFFFFFFFu, max(mx & 0xFFu, (mx >> 8) & 0xFFu)));
                __syncwarp();
                if (nan)
                    for (int key = lane; key < TN; key += 32) {
                        uint32_t m = 0;
                        for (int j = 0; j < S::EB; ++j) m |= (ex[512 + key * S::EB + j] == 255 ? 1u : 0u) << j;
                        s.nanblk[info][key] = (uint8_t)m;
                    }
                if (lane == 0) {
                    s.valid[info] = (int)vb;
                    s.ev[info] = E;
                    s.vnan[info] = nan;
                    s.care[info] = nan || part;
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&s.k_full[slot]);
                    mbar_arrive(&s.c_full[slot]);
                }
                ++tile;
            }
            pos += tiles;
            if (pos < w1) next_segment<D, RT>(p, g, pos, w1);
        }
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
        for (int pos = w0; pos < w1 && ok; qph ^= 1u) {
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
#pragma unroll
                        for (int ks = 0; ks < TN / 16; ++ks)  // 16 keys a step: two 8-key atoms
                            umma_a(tmem + S::CO, sp + 8 * ks, bd + ks * (2048 >> 4), idesc_a(D, true), i > 0 || ks > 0);
                        commit_a(&s.pv_done[buf]);
                    }
                } else {
                    const int slot = tile % S::NSLOT;
                    // S takes the place of the P of two tiles before
                    ok = wait(&s.k_full[slot], (uint32_t)((tile / S::NSLOT) & 1)) &&
                         (tile < 2 || wait(&s.pv_done[buf], bph ^ 1u));
                    if (!ok) break;
                    fence_after();
                    constexpr int RB = D < 128 ? 64 : 128;
                    const uint64_t bd = desc_codes<RB>(smem_u32(base + S::oK) + slot * S::SLOT);
                    const uint64_t ad = desc_codes<128>(smem_u32(base + S::oQ));
                    const uint64_t xd = desc_scales(smem_u32(base + S::oExp) + slot * 1024);
                    const uint32_t sfb = tmem + S::CB + 4 * buf;
                    if (one) {
                        copy_scales(sfb, xd);  // in order with the MMAs of this thread
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
            pos += tiles;
            if (pos < w1) next_segment<D, RT>(p, g, pos, w1);
        }
        // the last products must be done before tensor memory goes back (bounded)
        if (tile > 0)
            (void)wait(value ? &s.pv_done[(tile - 1) & 1] : &s.s_full[(tile - 1) & 1], (uint32_t)(((tile - 1) >> 1) & 1));
    } else if (warp >= kSoftWarps) {
        // ------------------------------------------------------------ values to f16
        const int dw = warp - kSoftWarps;
        // A lane takes 32-channel blocks: two 16-byte loads of codes, one scale, four 16-byte stores.
        // Eight lanes of a quarter-warp: four rows (8-row atom rows 4 a .. 4 a + 3), two neighbouring
        // blocks of a 64-channel column: their stores hit all eight 16-byte units of the swizzled
        // f16 rows; their loads, of alternating columns, every bank twice.
        constexpr int NC = D / 64, RPW = TN / kDeqWarps, PASSES = RPW * NC * 2 / 32;
        const int b2 = lane & 1, rj = (lane >> 1) & 3, rg = lane >> 3;  // block of the column, row of four, group
        int tile = 0;
        Segment g = first;
        for (int pos = w0; pos < w1 && ok;) {
            const int tiles = g.kv1 - g.kv0;
            for (int i = 0; i < tiles; ++i, ++tile) {
                const int slot = tile % S::NSLOT, buf = tile & 1, info = tile % kInfo;
                ok = wait(&s.c_full[slot], (uint32_t)((tile / S::NSLOT) & 1)) &&
                     (tile < 2 || wait(&s.pv_done[buf], (uint32_t)((tile >> 1) & 1) ^ 1u));
                if (!ok) break;
                const uint8_t *src = base + S::oRing + slot * S::SLOT, *ex = base + S::oExp + slot * 1024 + 512;
                uint8_t *dst = base + S::oV + buf * S::F16;
                const int E = s.ev[info] - kShift;
                const bool care = s.care[info];  // missing keys and NaN blocks count as zeros
                uint4 w[PASSES][2];
                int e[PASSES];
#pragma unroll
                for (int ps = 0; ps < PASSES; ++ps) {  // every load before the first store
                    const int q = ps * 4 + rg;  // four-row group and column of the warp's part
                    const int row = dw * RPW + (q / NC) * 4 + rj, col = NC == 1 ? 0 : (q + rj) % NC;
                    const uint8_t *c = src + row * D + col * 64 + b2 * 32;
                    w[ps][0] = *reinterpret_cast<const uint4 *>(c);
                    w[ps][1] = *reinterpret_cast<const uint4 *>(c + 16);
                    e[ps] = ex[row * S::EB + 2 * col + b2];
                }
                if (care) {
                    const int keys = g.ctx + g.nodes - (g.kv0 + i) * TN;
                    const uint32_t vb = (uint32_t)s.valid[info];
#pragma unroll
                    for (int ps = 0; ps < PASSES; ++ps) {
                        const int row = dw * RPW + ((ps * 4 + rg) / NC) * 4 + rj;
                        if (row >= keys || !((vb >> (row >> 4)) & 1) || e[ps] == 255) {
                            w[ps][0] = w[ps][1] = make_uint4(0, 0, 0, 0);
                            e[ps] = 0;
                        }
                    }
                }
#pragma unroll
                for (int ps = 0; ps < PASSES; ++ps) {
                    const int q = ps * 4 + rg;
                    const int row = dw * RPW + (q / NC) * 4 + rj, col = NC == 1 ? 0 : (q + rj) % NC;
                    const uint32_t sc = f16_pow2(e[ps] - E);
                    uint8_t *d = dst + col * (TN * 128) + row * 128;
                    const int x = row & 7;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint4 lo, hi;
                        widen16(w[ps][h], sc, lo, hi);
                        const int u = 4 * b2 + 2 * h;
                        *reinterpret_cast<uint4 *>(d + ((u ^ x) << 4)) = lo;
                        *reinterpret_cast<uint4 *>(d + (((u + 1) ^ x) << 4)) = hi;
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // f16 for the MMA's reads
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&s.v_full[buf]);
                    mbar_arrive(&s.c_free[slot]);
                }
            }
            pos += tiles;
            if (pos < w1) next_segment<D, RT>(p, g, pos, w1);
        }
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
        // sets take half of the channels each.
        auto put_q = [&](const Segment &g) -> int {
            const int r = g.rt * RT + row;
            const bool real = r < g.nodes * p.g;
            const int t = real ? r / p.g : 0, hq = g.h * p.g + (real ? r - t * p.g : 0);
            const uint16_t *qr = p.q + ((size_t)g.b * p.T + t) * p.ldq + (size_t)hq * D;
            uint32_t am = 0;
            if (real)
#pragma unroll 8
                for (int c = 0; c < D; c += 8) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(qr + c);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) am = max(am, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
                }
            const int eq = max((int)(am >> 7) - 127 - 7, -100);
            const float qs = pow2i(-eq);  // eq <= 121
#pragma unroll 1
            for (int c = set * (D / 2); c < (set + 1) * (D / 2); c += 32) {
                uint32_t hi[8], lo[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (real) v = *reinterpret_cast<const uint4 *>(qr + c + 8 * j);
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
            return eq;
        };
        {   // Q's scales: byte 0 (2^0) for the upper part, byte 1 (2^-4) for the lower
            const uint32_t f[4] = {0x7B7Fu, 0x7B7Fu, 0x7B7Fu, 0x7B7Fu};
            st_cols(tl + S::CA, f);  // both sets write the same
            wait_st();
        }
        // Per turn: the next segment's Q (once the last S of the one before is there), then the output
        // of the one before, then the segment's tiles.
        Segment g = first;
        int r = 0, t = 0, hq = 0;          // row of the request and head; its node and query head
        bool real = false;
        float m = 0.0f, l = 0.0f;          // the rows' maximum at the set's last tile; its sum in 2^(m - bias)
        uint32_t nanblk = 0;
        for (int pos = w0; ok;) {
            const bool more = pos < w1;
            Segment next{};
            int eq = 0;
            if (more) {
                next = g;
                if (it > 0) next_segment<D, RT>(p, next, pos, w1);
                if (it > 0) ok = wait(&s.s_full[(it - 1) & 1], (uint32_t)(((it - 1) >> 1) & 1));
                if (!ok) break;
                fence_after();
                eq = put_q(next);
            }
            if (it > 0) {
                // ---- the segment's output; the sets take half of the channels each
                ok = wait(&s.pv_done[(it - 1) & 1], (uint32_t)(((it - 1) >> 1) & 1));
                if (!ok) break;
                fence_after();
                const int ev = s.ev[(it - 1) % kInfo];
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
            pos += tiles;

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
                const uint32_t tb = tl + S::CS + buf * TN, ts = tb + col0;
                const int slot0 = (g.kv0 + i) * TN + col0;  // cache slot of the thread's first column
                const uint32_t vb = (uint32_t)s.valid[info];
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
                if (masked) {  // S of what a row does not see becomes -inf, in place
                    constexpr int MC = CPT < 32 ? CPT : 32;
#pragma unroll 1
                    for (int k = 0; k < CPT; k += MC) {
                        const uint32_t w = seen(k);
                        uint32_t y[MC];
                        ld_cols(ts + k, y);
                        wait_ld();
#pragma unroll
                        for (int j = 0; j < MC; ++j) y[j] = (w >> j) & 1u ? y[j] : 0xFF800000u;
                        st_cols(ts + k, y);
                    }
                    wait_st();
                }
                const float ml = m;    // the rows' m at the set's last tile, and
                float mp = -INFINITY;  // at the tile before, the other set's
                // from the thread's largest S: the rows' m at this tile, handed on to the other set
                auto settle = [&](float mt) -> bool {
                    if (i > 0) {
                        if (!wait(&s.m_full[set ^ 1][quad], (uint32_t)(((it - 1) >> 1) & 1))) return false;
                        mp = s.mrow[set ^ 1][32 * quad + lane];
                    }
                    const float me = mt == -INFINITY ? mt : mt * c;
                    m = me > mp + kSlack ? me : mp;  // also out of -inf
                    s.mrow[set][32 * quad + lane] = m;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s.m_full[set][quad]);
                    return true;
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
                        const float off = m == -INFINITY ? 0.0f : kBias - m;
                        const uint64_t c2 = pair(c, c), off2 = pair(off, off);
                        sum = pair(0.0f, 0.0f);
                        uint32_t x[CPT > CH ? 2 : 1][CH];
                        ld_cols(ts, x[0]);
                        wait_ld();
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
                        ok = settle(fmaxf(m0, m1));
                        again = __any_sync(0xFFFFFFFFu, m != ml);
                        if (!ok || !again) break;
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
                    // Two passes: 64 registers of P on top of the rest would spill.
#pragma unroll 1
                    for (int k = 0; k < CPT; k += CH) {
                        uint32_t y[CH];
                        ld_cols(ts + k, y);
                        wait_ld();
                        largest(y, m0, m1);
                    }
                    ok = settle(fmaxf(m0, m1));
                    if (!ok) break;
                    const float off = m == -INFINITY ? 0.0f : kBias - m;
                    const uint64_t c2 = pair(c, c), off2 = pair(off, off);
                    sum = pair(0.0f, 0.0f);
#pragma unroll 1
                    for (int k = 0; k < CPT; k += CH) {  // a chunk's P lands on columns already read
                        uint32_t y[CH], pk[CH / 2];
                        ld_cols(ts + k, y);
                        wait_ld();
                        powers(y, c2, off2, pk);
                        st_cols(tb + k / 2, pk);
                    }
                }
                const bool grow = m != mp;
                // ---- O in the units of the new maximum and value exponent
                ok = wait(&s.v_full[buf], tph);
                if (!ok) break;
                if (i > 0) {
                    const int evp = s.ev[(it - 1) % kInfo], evn = s.ev[info];
                    if (__any_sync(0xFFFFFFFFu, grow || evn != evp)) {
                        ok = wait(&s.pv_done[buf ^ 1], (uint32_t)(((it - 1) >> 1) & 1));
                        if (!ok) break;
                        fence_after();
                        const float f = (grow ? (mp == -INFINITY ? 0.0f : ex2(mp - m)) : 1.0f) * pow2i(max(evp - evn, -149));
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
                l = l * (m == ml ? 1.0f : ml == -INFINITY ? 0.0f : ex2(ml - m)) + sum_pair(sum);
                if (s.vnan[info]) {
#pragma unroll 1
                    for (int k = 0; k < CPT; k += 32) {
                        const uint32_t w = real ? (masked ? seen(k) : 0xFFFFFFFFu) : 0u;
#pragma unroll 1
                        for (int j = 0; j < CPT - k && j < 32; ++j)
                            if ((w >> j) & 1u) nanblk |= s.nanblk[info][col0 + k + j];
                    }
                }
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.p_full[buf]);
            }
            if (!ok) break;
        }
    }

    if (!ok) report_timeout(p.status);
    __syncwarp();
    fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

// ------------------------------------------------------------------ the join
// A warp per row: rows past the request's nodes become zeros, rows that one block finished are
// left alone, the others are joined from their blocks' partials in block order:
//   out = sum w_i o_i / sum w_i,  w_i = 2^(m_i - max m) sum_i.
constexpr int kJoinWarps = 8;

template <int D, int RT>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ AttendParams p) {
    pdl_trigger();
    pdl_wait();
    constexpr int PC = D / 32;  // channels a lane
    const int lane = threadIdx.x & 31;
    const long long idx = (long long)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
    if (idx >= (long long)p.B * p.T * p.Hq) return;
    const int hq = (int)(idx % p.Hq), t = (int)(idx / p.Hq % p.T), b = (int)(idx / p.Hq / p.T);
    int ctx, nodes;
    (void)lengths(p, b, ctx, nodes);
    uint16_t *const dst = p.out + (size_t)idx * D + lane * PC;
    float y[PC] = {};
    float lse = -INFINITY;
    if (t < nodes) {
        const int h = hq / p.g, r = t * p.g + (hq - h * p.g), rt = r / RT, row = r - rt * RT;
        const int nt = (ctx + nodes + Shape<D>::TN - 1) / Shape<D>::TN;
        const long long total = p.prefix[p.B];
        const int first = p.prefix[b] + (h * ((nodes * p.g + RT - 1) / RT) + rt) * nt, last = first + nt - 1;
        auto block_of = [&](int item) {
            int w = (int)((long long)item * kAttendBlocks / total);
            while (range_start(total, w + 1) <= item) ++w;
            return w;
        };
        const int wa = block_of(first), wz = block_of(last);
        if (wa == wz) return;
        float M = -INFINITY;
        for (int w = wa + lane; w <= wz; w += 32) {
            const int s = range_start(total, w);
            if (range_start(total, w + 1) > s) M = fmaxf(M, p.stat[(size_t)(2 * w + (s > first ? 0 : 1)) * RT + row].x);
        }
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, k));
        float sum = 0.0f;
#pragma unroll 4
        for (int w = wa; w <= wz; ++w) {
            const int s = range_start(total, w);
            if (range_start(total, w + 1) <= s) continue;
            const size_t at = (size_t)(2 * w + (s > first ? 0 : 1)) * RT + row;
            const float2 st = p.stat[at];
            const float f = st.y == 0.0f ? 0.0f : ex2(st.x == -INFINITY ? 0.0f : st.x - M) * st.y;
            const float *o = p.part + at * D + lane * PC;
            sum += f;
#pragma unroll
            for (int j = 0; j < PC; ++j) y[j] = fmaf(f, o[j], y[j]);
        }
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
        for (int j = 0; j < PC; ++j) y[j] *= inv;
        if (sum != 0.0f) lse = (M + log2f(sum)) * 0.69314718055994531f;
    }
#pragma unroll
    for (int j = 0; j < PC; j += 2) *reinterpret_cast<uint32_t *>(dst + j) = pack_bf(y[j], y[j + 1]);
    if (p.lse && lane == 0) p.lse[idx] = lse;
}

// ------------------------------------------------------------------ host side

namespace {

// Rows a tile: the smallest that holds all of a request's rows of a head (more copies of a small
// tile mean less softmax work a thread), 128 past that.
int row_tile(int T, int g) { return T * g <= 32 ? 32 : T * g <= 64 ? 64 : 128; }

size_t round16(size_t n) { return (n + 15) / 16 * 16; }

template <typename F>
cudaError_t launch_attend_grid(F *fn, long long blocks, int threads, size_t smem, cudaStream_t stream,
                               const AttendParams &prm) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = options().pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, fn, prm);
}

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

// The key codes as [rows][dim] bytes; a box is box_rows rows (inside a page and a tile) of at most
// 128 bytes, swizzled by its width.
cudaError_t key_map(const CacheView &c, int box_rows, CUtensorMap *out) {
    EncodeTiledFnA fn = encode_fn_a();
    if (!fn) return cudaErrorNotSupported;
    const cuuint32_t w = (cuuint32_t)std::min(c.dim, 128);
    const cuuint64_t dims[2] = {(cuuint64_t)c.dim, (cuuint64_t)c.pages * c.heads * c.page_size};
    const cuuint64_t strides[1] = {(cuuint64_t)c.dim};
    const cuuint32_t box[2] = {w, (cuuint32_t)box_rows}, es[2] = {1u, 1u};
    const CUresult r = fn(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, c.k8, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          w == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, int RT>
cudaError_t launch_attend_as(const AttendParams &prm, cudaStream_t stream) {
    static int configured[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!__atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE)) {
        e = cudaFuncSetAttribute(attend_kernel<D, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 attend_smem<D>(kMaxBatch));
        if (e != cudaSuccess) return e;
        __atomic_store_n(&configured[dev], 1, __ATOMIC_RELEASE);
    }
    e = launch_attend_grid(attend_kernel<D, RT>, kAttendBlocks, kThreadsA, attend_smem<D>(prm.B), stream, prm);
    if (e != cudaSuccess) return e;
    const long long rows = (long long)prm.B * prm.T * prm.Hq;
    return launch_attend_grid(join_kernel<D, RT>, (rows + kJoinWarps - 1) / kJoinWarps, kJoinWarps * 32, 0, stream,
                              prm);
}

template <int D>
cudaError_t launch_attend_dim(const AttendParams &prm, cudaStream_t stream) {
    switch (row_tile(prm.T, prm.g)) {
        case 32: return launch_attend_as<D, 32>(prm, stream);
        case 64: return launch_attend_as<D, 64>(prm, stream);
        default: return launch_attend_as<D, 128>(prm, stream);
    }
}

}  // namespace

// Two partials a block, their statistics, and the prefix sums.
size_t attend_workspace_bytes(int B, int T, int Hq, int heads, int dim) {
    const size_t rows = (size_t)kAttendBlocks * 2 * row_tile(T, Hq / heads);
    return rows * dim * 4 + rows * 8 + round16(((size_t)B + 1) * 4);
}

// Items of the largest call these arguments allow; they are counted in 31 bits.
bool attend_fits(const CacheView &c, int B, int T, int Hq, int max_len) {
    const int g = Hq / c.heads, rt = row_tile(T, g), tn = c.dim == 256 ? 64 : 128;
    return (double)B * c.heads * (((long long)T * g + rt - 1) / rt) * (((long long)max_len + tn - 1) / tn) < 2147483648.0;
}

cudaError_t launch_attend(const CacheView &c, const AttendArgs &a, cudaStream_t stream) {
    AttendParams prm{};
    prm.c = c;
    const int tn = c.dim == 256 ? 64 : 128;
    prm.box_rows = 16;  // the largest power of two that divides a page, up to a tile
    while (prm.box_rows < tn && c.page_size % (2 * prm.box_rows) == 0) prm.box_rows *= 2;
    prm.page_magic = (1ull << 32) / (unsigned)(c.page_size / 16) + 1;
    const cudaError_t e = key_map(c, prm.box_rows, &prm.kmap);
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
    const size_t rows = (size_t)kAttendBlocks * 2 * row_tile(a.T, prm.g);
    prm.part = static_cast<float *>(a.workspace);
    prm.stat = reinterpret_cast<float2 *>(prm.part + rows * c.dim);
    prm.prefix = reinterpret_cast<int *>(prm.stat + rows);
    const Options opt = options();
    prm.timeout_ns = opt.timeout_ns;
    prm.tries = (uint32_t)std::min<unsigned long long>(std::max<unsigned long long>(opt.timeout_ns / kSuspendNs, 1), 0x7FFFFFFFu);
    prm.skip_loads = opt.skip_loads;
    prm.status = status_word();
    if (!prm.status) return cudaErrorInvalidSymbol;
    switch (c.dim) {
        case 64: return launch_attend_dim<64>(prm, stream);
        case 128: return launch_attend_dim<128>(prm, stream);
        case 256: return launch_attend_dim<256>(prm, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace bsf8
