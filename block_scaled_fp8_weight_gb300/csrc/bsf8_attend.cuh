// bsf8_attend.cuh -- what the attention kernels share: the cut of the work, the tcgen05 wrappers, the
// roles that do not depend on how rows and keys lie in tensor memory (producer, scout, values to
// f16), the join of partials.  bsf8_attend.cu says how the whole works.
#pragma once

#include "bsf8_device.cuh"
#include "bsf8_internal.h"

#include <cuda.h>

#include <algorithm>

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
constexpr float kBias = 9.0f;        // p = 2^(x - m + kBias)
constexpr float kSlack = 6.0f;       // m lags the maximum by at most this
constexpr int kLarge = 21;           // |x| from 2^21 on: its last place is no longer small against the slack
constexpr int kShift = 6;            // f16 values are code * 2^(e - E + kShift)

}  // namespace

struct AttendParams {
    unsigned long long page_magic;  // floor(2^32 / (page_size / 16)) + 1: divides 16-key groups by a page's
    CUtensorMap kmap;  // the key codes as rows of D bytes, box min(D, 128) x box_rows, swizzled
    CUtensorMap vmap;  // the value codes likewise
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
    float *part;         // [blocks][2][RT][D] normalised outputs (32-byte aligned)
    float2 *stat;        // [blocks][2][RT] (m, sum)
    int *prefix;         // [B + 1] the requests' work, for the join
    uint32_t tries;      // suspensions of a wait
    unsigned long long timeout_ns;
    int skip_loads;
    int *status;
};

// The kernel for up to 8 rows of a request and head at dim 128 (bsf8_attend_few.cu).
constexpr int kFewRows = 8;

// Tiles' worth of time that a segment takes besides its own, in that kernel (64 requests of 70 to 16384 tokens: 218 us
// with 2, 197 with 3, 187 with 4 and 5, 189 with 6) and in the other (trees of 23 nodes over up to 8192
// tokens: 58 us with 2, 53 with 3, 51 with 4 and 6).
constexpr int kFewStart = 4, kStart = 5;
cudaError_t launch_attend_few(const AttendParams &prm, cudaStream_t stream);

namespace {

// A request's context and node counts, inside their bounds.
__device__ __forceinline__ bool lengths(const AttendParams &p, int b, int &ctx, int &nodes) {
    ctx = p.ctx[b];
    nodes = p.nodes ? p.nodes[b] : p.T;
    if (ctx >= 0 && nodes >= 0 && nodes <= p.T && (long long)ctx + nodes <= p.max_len) return true;
    ctx = max(0, min(ctx, p.max_len));
    nodes = max(0, min(nodes, min(p.T, p.max_len - ctx)));
    return false;
}

// A request's work, in tiles: a segment (a row tile of a head over all keys) counts its tiles of keys
// and S::START for its start and end.
template <class S>
__device__ __forceinline__ int work_of(const AttendParams &p, int ctx, int nodes) {
    if (nodes == 0) return 0;
    const int nt = (ctx + nodes + S::TN - 1) / S::TN;
    return p.c.heads * ((nodes * p.g + S::RT - 1) / S::RT) * (nt + S::START);
}

// The share of block w: [w total / W, (w + 1) total / W).  The tiles whose places lie in it are the
// block's; a segment's places are START empty ones, then its tiles'.
__device__ __forceinline__ int range_start(long long total, int w) {
    return (int)(total * w / kAttendBlocks);
}

struct Segment {
    int b, h, rt, kv0, kv1, nt, ctx, nodes;
    int next;  // the place after its last
};

__device__ __forceinline__ bool live(const Segment &s) { return s.kv1 > s.kv0; }

// The segment at place pos of a block whose share ends at end; not live if none of its tiles are the
// block's (then none of a later segment's are).
template <class S>
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
    s.nt = (s.ctx + s.nodes + S::TN - 1) / S::TN;
    const int rts = (s.nodes * p.g + S::RT - 1) / S::RT;
    const int rem = pos - prefix[lo];
    const int seg = rem / (s.nt + S::START), in = rem - seg * (s.nt + S::START);
    s.kv0 = max(0, in - S::START);
    s.kv1 = min(s.nt, in + (end - pos) - S::START);
    s.next = pos - in + s.nt + S::START;
    s.h = seg / rts;
    s.rt = seg - s.h * rts;
    return s;
}

// The segment after s.
template <class S>
__device__ __forceinline__ void next_segment(const AttendParams &p, Segment &s, int end) {
    s.kv0 = s.kv1 = 0;
    if (s.next + S::START >= end) return;
    if ((++s.rt) * S::RT >= s.nodes * p.g) {
        s.rt = 0;
        if (++s.h == p.c.heads) {
            s.h = 0;
            do {
                (void)lengths(p, ++s.b, s.ctx, s.nodes);
            } while (s.nodes == 0);  // ends: there is work left
            s.nt = (s.ctx + s.nodes + S::TN - 1) / S::TN;
        }
    }
    s.kv1 = min(s.nt, end - s.next - S::START);
    s.next += s.nt + S::START;
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

// kind::f8f6f4, e4m3 A and B without scales, both given by columns (M- and N-major), M = 128.
__device__ __forceinline__ constexpr uint32_t idesc_8(int n) {
    return (1u << 4) | (1u << 15) | (1u << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

__device__ __forceinline__ void umma_8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
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

// 32 bytes, a whole sector, by a thread (32-byte aligned).
__device__ __forceinline__ void st_global8(void *dst, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// N channels (from k) of a row's output: bf16 where the segment is the whole row, else a partial.
template <int RT, int D, int N>
__device__ __forceinline__ void store_row(const AttendParams &p, const Segment &g, bool whole, int slotw, int row,
                                          int t, int hq, int k, const float (&y)[N]) {
    if (whole) {
        uint16_t *dst = p.out + (((size_t)g.b * p.T + t) * p.Hq + hq) * D + k;
        if constexpr (N == 16) {
#pragma unroll
            for (int j = 0; j < N; j += 8)
                *reinterpret_cast<uint4 *>(dst + j) = make_uint4(pack_bf(y[j], y[j + 1]), pack_bf(y[j + 2], y[j + 3]),
                                                                 pack_bf(y[j + 4], y[j + 5]), pack_bf(y[j + 6], y[j + 7]));
        } else {
#pragma unroll
            for (int j = 0; j < N; j += 4)
                *reinterpret_cast<uint2 *>(dst + j) = make_uint2(pack_bf(y[j], y[j + 1]), pack_bf(y[j + 2], y[j + 3]));
        }
    } else {
        float *dst = p.part + ((size_t)slotw * RT + row) * D + k;
        if constexpr (N == 16) {
#pragma unroll
            for (int k = 0; k < 16; k += 8) {
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(y[k + j]);
                st_global8(dst + k, w);
            }
        } else {
#pragma unroll
            for (int j = 0; j < N; j += 4)
                *reinterpret_cast<float4 *>(dst + j) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
        }
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

struct BlockShared {
    uint32_t tmem;
    int scan[32];
};

// What the scout says of a tile.  An entry is written again eight tiles later, once the dequant
// warps have read the slot of the tile four later, thus after the softmax of the tile two later.
struct __align__(16) TileInfo {
    int valid;   // the 16-key groups that exist (bit i)
    int ev;      // the segment's largest value exponent up to this tile,
    int rise;    // and by how much it passes the one up to the tile before
    int flags;   // 1: the values need care (missing keys, NaN); 2: a value block holds NaN; above 8 bits: the keys' largest exponent
};

__device__ __forceinline__ TileInfo load_info(const TileInfo *i) {
    const int4 v = *reinterpret_cast<const int4 *>(i);
    return TileInfo{v.x, v.y, v.z, v.w};
}

// What the roles of a block tell each other by, as far as the kernels share it.
struct AttendPipes : BlockShared {
    uint64_t k_full[4], k_free[4];  // ring slots of keys: codes landed and scales written; multiplied
    uint64_t c_full[4], c_free[4];  // of values: codes landed and exponents written; read by all dequant warps
    uint64_t v_full[2];             // the f16 values of a tile are written
    uint64_t pv_done[2];            // O updated, P and the f16 values read
    TileInfo info[kInfo];
    uint8_t nanblk[kInfo][128];     // where a value block holds NaN: each key's NaN blocks
};

__device__ __forceinline__ void init_pipes(AttendPipes &s) {
    for (int i = 0; i < 4; ++i) {
        mbar_init(&s.k_full[i], 2);  // the producer's byte count, the scout
        mbar_init(&s.k_free[i], 1);
        mbar_init(&s.c_full[i], 2);
        mbar_init(&s.c_free[i], kDeqWarps);
    }
    for (int i = 0; i < 2; ++i) {
        mbar_init(&s.v_full[i], kDeqWarps);
        mbar_init(&s.pv_done[i], 1);
    }
}

// Tensor memory, all of it: held before the next kernel's blocks may come.
__device__ __forceinline__ void hold_tmem(BlockShared &s, bool one) {
    if (one) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&s.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
}

__device__ __forceinline__ void free_tmem(uint32_t tmem, bool one) {
    __syncwarp();
    fence_before();
    __syncthreads();
    if (one) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
    }
}

__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, uint32_t tries) {
    return __all_sync(0xFFFFFFFFu, wait_phase(bar, parity, tries));
}

// Prefix sums of the requests' work, by the whole block (ends with a barrier).
template <class S>
__device__ __forceinline__ void sum_items(const AttendParams &p, BlockShared &s, int *prefix, int warp, int lane) {
    const int per = (p.B + S::THREADS - 1) / S::THREADS;
    {
        const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
        int sum = 0;
        for (int b = b0; b < b1; ++b) {
            int ctx, nodes;
            if (!lengths(p, b, ctx, nodes) && blockIdx.x == 0) report_index(p.status);
            sum += work_of<S>(p, ctx, nodes);
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
        for (int b = threadIdx.x; b <= p.B; b += S::THREADS) p.prefix[b] = prefix[b];
}

// A batch of BT tiles' 16-key groups, one a lane: the page of the lane's group (a load that stays
// in flight until the batch is used), then its cache row (head h), -1 if there is none.
template <class S>
struct Pages {
    static constexpr int TN = S::TN, NSB = TN / 16, BT = 32 / NSB;

    // exact: group * (magic * d - 2^32) < 2^32 for groups below 2^26 and d <= 64
    static __device__ __forceinline__ int in_page(const AttendParams &p, int grp) {
        return (int)(((unsigned long long)(unsigned)grp * p.page_magic) >> 32);
    }
    static __device__ __forceinline__ int page_of(const AttendParams &p, const Segment &g, int tile, int lane) {
        const int grp = (tile + lane / NSB) * NSB + lane % NSB;
        return 16 * grp < g.ctx + g.nodes ? p.c.table[(size_t)g.b * p.c.table_pages + in_page(p, grp)] : -1;
    }
    static __device__ __forceinline__ int row_of(const AttendParams &p, const Segment &g, int tile, int page, int lane) {
        const int grp = (tile + lane / NSB) * NSB + lane % NSB;
        if (16 * grp >= g.ctx + g.nodes) return -1;
        if ((unsigned)page >= (unsigned)p.c.pages) {
            report_index(p.status);
            return -1;
        }
        return (page * p.c.heads + g.h - in_page(p, grp)) * p.c.page_size + 16 * grp;
    }
};

// The producer warp: codes.  Keys by TMA boxes (swizzled, for the MMA), values as they are.
template <class S>
__device__ __forceinline__ bool produce(const AttendParams &p, AttendPipes &s, uint8_t *base, const Segment &first, int w1,
                                        int lane) {
    constexpr int TN = S::TN, D = S::DIM, NSB = TN / 16, BT = 32 / NSB;
    bool ok = true;  // no wait ran out
    const int gpb = p.box_rows / 16;  // groups a box: boxes never cross a page's end
    const bool lead = lane < NSB && lane % gpb == 0;
    int tile = 0;
    Segment g = first;
    while (live(g) && ok) {
        const int tiles = g.kv1 - g.kv0;
        int page = Pages<S>::page_of(p, g, g.kv0, lane), rows = -1;
        for (int i = 0; i < tiles; ++i, ++tile) {
            const int j = i % BT;
            if (j == 0) {
                rows = Pages<S>::row_of(p, g, g.kv0 + i, page, lane);
                page = Pages<S>::page_of(p, g, g.kv0 + i + BT, lane);
            }
            const int row = __shfl_sync(0xFFFFFFFFu, rows, (j * NSB + lane) & 31);
            const bool go = lead && row >= 0;
            const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xFFFFFFFFu, go)) * (uint32_t)(p.box_rows * D);
            const int slot = tile % S::NSLOT;
            const uint32_t fph = (uint32_t)((tile / S::NSLOT) & 1) ^ 1u;
            ok = tile < S::NSLOT || wait_warp(&s.k_free[slot], fph, p.tries);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&s.k_full[slot], bytes);
            __syncwarp();
            if (go && !p.skip_loads)
#pragma unroll
                for (int c = 0; c < D; c += 128)  // 128-byte columns of the tile, one after another
                    tma_rows(base + S::oK + slot * S::SLOT + c * TN + lane * 16 * (D < 128 ? D : 128), &p.kmap, c, row,
                             &s.k_full[slot]);
            ok = tile < S::NSLOT || wait_warp(&s.c_free[slot], fph, p.tries);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&s.c_full[slot], bytes);
            __syncwarp();
            if (go && !p.skip_loads)
                bulk_g2s(base + S::oRing + slot * S::SLOT + lane * 16 * D, p.c.v8 + (size_t)row * D,
                         (uint32_t)(p.box_rows * D), &s.c_full[slot]);
        }
        next_segment<S>(p, g, w1);
    }
    // every copy must have landed before the block's memory goes away (bounded)
    if (!p.skip_loads)
        for (int i = max(0, tile - S::NSLOT); i < tile + (ok ? 0 : 1); ++i) {
            const int slot = i % S::NSLOT;
            const uint32_t iph = (uint32_t)((i / S::NSLOT) & 1);
            (void)mbar_wait_bounded(&s.k_full[slot], iph, ok ? p.timeout_ns : 100000000ull);
            (void)mbar_wait_bounded(&s.c_full[slot], iph, ok ? p.timeout_ns : 100000000ull);
        }
    return ok;
}

// The scout warp: exponents and flags.
template <class S>
__device__ __forceinline__ bool scout(const AttendParams &p, AttendPipes &s, uint8_t *base, const Segment &first, int w1,
                                      int lane) {
    constexpr int TN = S::TN, D = S::DIM, NSB = TN / 16, BT = 32 / NSB;
    bool ok = true;  // no wait ran out
    constexpr int KPL = 16 / S::EB;  // keys of a lane's 16 exponent bytes
    const int key0 = lane * KPL;
    int tile = 0;
    Segment g = first;
    while (live(g) && ok) {
        const int tiles = g.kv1 - g.kv0;
        int E = 0;  // the largest value exponent of the segment so far
        int page = Pages<S>::page_of(p, g, g.kv0, lane), rows = -1;
        uint4 kx = make_uint4(0, 0, 0, 0), vx = kx, kn = kx, vn = kx;
        uint32_t vb = 0, vbn = 0;
        // starts the loads of tile i's exponents
        auto load = [&](int i) {
            const int j = i % BT;
            if (j == 0) {
                rows = Pages<S>::row_of(p, g, g.kv0 + i, page, lane);
                page = Pages<S>::page_of(p, g, g.kv0 + i + BT, lane);
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
            ok = tile < S::NSLOT || (wait_warp(&s.k_free[slot], fph, p.tries) && wait_warp(&s.c_free[slot], fph, p.tries));
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
            uint32_t mk = __vmaxu4(__vmaxu4(kx.x, kx.y), __vmaxu4(kx.z, kx.w));
            mk = __vmaxu4(mk, mk >> 16);
            const int kmax = (int)__reduce_max_sync(0xFFFFFFFFu, max(mk & 0xFFu, (mk >> 8) & 0xFFu));
            const int before = E;
            E = max(E, (int)__reduce_max_sync(0xFFFFFFFFu, max(mx & 0xFFu, (mx >> 8) & 0xFFu)));
            __syncwarp();
            if (nan)
                for (int key = lane; key < TN; key += 32) {
                    uint32_t m = 0;
                    for (int j = 0; j < S::EB; ++j) m |= (ex[512 + key * S::EB + j] == 255 ? 1u : 0u) << j;
                    s.nanblk[info][key] = (uint8_t)m;
                }
            if (lane == 0)
                *reinterpret_cast<int4 *>(&s.info[info]) =
                    make_int4((int)vb, E, i > 0 ? E - before : 0, (nan ? 2 : 0) | (nan || part ? 1 : 0) | kmax << 8);
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&s.k_full[slot]);
                mbar_arrive(&s.c_full[slot]);
            }
            ++tile;
        }
        next_segment<S>(p, g, w1);
    }
    return ok;
}

// The dequant warps: values to f16.
template <class S>
__device__ __forceinline__ bool widen_values(const AttendParams &p, AttendPipes &s, uint8_t *base, const Segment &first,
                                             int w1, int warp, int lane) {
    constexpr int TN = S::TN, D = S::DIM;
    bool ok = true;  // no wait ran out
    const int dw = warp - kSoftWarps;
    // A lane takes 32-channel blocks: two 16-byte loads of codes, one scale, four 16-byte stores.
    // Eight lanes of a quarter-warp: four rows (8-row atom rows 4 a .. 4 a + 3), two neighbouring
    // blocks of a 64-channel column: their stores hit all eight 16-byte units of the swizzled
    // f16 rows; their loads, of alternating columns, every bank twice.
    constexpr int NC = D / 64, RPW = TN / kDeqWarps, PASSES = RPW * NC * 2 / 32;
    const int b2 = lane & 1, rj = (lane >> 1) & 3, rg = lane >> 3;  // block of the column, row of four, group
    int tile = 0;
    Segment g = first;
    while (live(g) && ok) {
        const int tiles = g.kv1 - g.kv0;
        for (int i = 0; i < tiles; ++i, ++tile) {
            const int slot = tile % S::NSLOT, buf = tile & 1, info = tile % kInfo;
            ok = wait_warp(&s.c_full[slot], (uint32_t)((tile / S::NSLOT) & 1), p.tries) &&
                 (tile < 2 || wait_warp(&s.pv_done[buf], (uint32_t)((tile >> 1) & 1) ^ 1u, p.tries));
            if (!ok) break;
            const uint8_t *src = base + S::oRing + slot * S::SLOT, *ex = base + S::oExp + slot * 1024 + 512;
            uint8_t *dst = base + S::oV + buf * S::F16;
            const TileInfo inf = load_info(&s.info[info]);
            const int E = inf.ev - kShift;
            const bool care = inf.flags & 1;  // missing keys and NaN blocks count as zeros
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
                const uint32_t vb = (uint32_t)inf.valid;
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
        next_segment<S>(p, g, w1);
    }
    return ok;
}

}  // namespace

// ------------------------------------------------------------------ the join
// Rows past the request's nodes become zeros, rows that one block finished are left alone, the others
// are joined from their blocks' partials:
//   out = sum w_i o_i / sum w_i,  w_i = 2^(m_i - max m) sum_i.
// WPR warps a row: each takes every WPR-th partial, in order (a lane a partial's maximum and sum, then
// all lanes the channels, a group of partials in flight), and the warps' results are added in order.
// Bound by latency: three loads that depend on each other.  A row over 50 blocks: 20 us in a warp with a
// partial after another, 3 so.
namespace {

constexpr int kJoinWarps = 8;

template <int PC>
__device__ __forceinline__ void load_channels(const float *src, float (&o)[PC]) {
    if constexpr (PC == 2) {
        const float2 v = *reinterpret_cast<const float2 *>(src);
        o[0] = v.x, o[1] = v.y;
    } else {
#pragma unroll
        for (int j = 0; j < PC; j += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(src + j);
            o[j] = v.x, o[j + 1] = v.y, o[j + 2] = v.z, o[j + 3] = v.w;
        }
    }
}

}  // namespace

template <class S, int WPR>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ AttendParams p) {
    pdl_trigger();
    pdl_wait();
    constexpr int D = S::DIM, RT = S::RT;
    constexpr int PC = D / 32, GROUP = PC == 8 ? 4 : 8;  // channels a lane, partials in flight
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = WPR == 1 ? 0 : warp;
    const long long idx = WPR == 1 ? (long long)blockIdx.x * kJoinWarps + warp : blockIdx.x;
    if (idx >= (long long)p.B * p.T * p.Hq) return;
    const int hq = (int)(idx % p.Hq), t = (int)(idx / p.Hq % p.T), b = (int)(idx / p.Hq / p.T);
    const long long total = p.prefix[p.B];  // asked for with the lengths, not after them
    const int before = p.prefix[b];
    int ctx, nodes;
    (void)lengths(p, b, ctx, nodes);
    float y[PC] = {};
    float M = -INFINITY, sum = 0.0f;
    if (t < nodes) {
        const int h = hq / p.g, r = t * p.g + (hq - h * p.g), rt = r / RT, row = r - rt * RT;
        const int nt = (ctx + nodes + S::TN - 1) / S::TN;
        const int first = before + (h * ((nodes * p.g + RT - 1) / RT) + rt) * (nt + S::START) + S::START;
        const int last = first + nt - 1;  // the places of its tiles
        // the block of a place: an estimate that is at most one off, then the exact one
        const float per = (float)kAttendBlocks / (float)total;
        auto block_of = [&](int place) {
            int w = max(0, (int)((float)place * per) - 1);
            while (range_start(total, w + 1) <= place) ++w;
            return w;
        };
        const int wa = block_of(first), n = block_of(last) - wa + 1;
        if (n == 1) return;
        for (int base = part; base < n; base += 32 * WPR) {
            const int k = base + lane * WPR, w = wa + k;
            int at = -1;
            if (k < n) {
                const int s = range_start(total, w);
                if (range_start(total, w + 1) > s) at = (2 * w + (s > first ? 0 : 1)) * RT + row;
            }
            float2 st = make_float2(-INFINITY, 0.0f);
            if (at >= 0) st = p.stat[at];
            const int count = min(32, (n - base + WPR - 1) / WPR);
            float f = 0.0f;
            for (int j0 = 0; j0 < count; j0 += GROUP) {
                float o[GROUP][PC];
                bool in[GROUP];
#pragma unroll
                for (int j = 0; j < GROUP; ++j) {
                    const int a = __shfl_sync(0xFFFFFFFFu, at, (j0 + j) & 31);
                    in[j] = j0 + j < count && a >= 0;
                    if (in[j]) load_channels<PC>(p.part + (size_t)a * D + lane * PC, o[j]);
                }
                if (j0 == 0) {  // with the first group on its way
                    float m = st.x;
#pragma unroll
                    for (int q = 16; q > 0; q >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, q));
                    m = fmaxf(m, M);
                    const float g = M == -INFINITY ? 0.0f : ex2(M - m);
                    M = m;
                    sum *= g;
#pragma unroll
                    for (int c = 0; c < PC; ++c) y[c] *= g;
                    f = st.y == 0.0f ? 0.0f : ex2(st.x == -INFINITY ? 0.0f : st.x - M) * st.y;
                }
#pragma unroll
                for (int j = 0; j < GROUP; ++j) {
                    const float g = __shfl_sync(0xFFFFFFFFu, f, (j0 + j) & 31);
                    if (!in[j]) continue;
                    sum += g;
#pragma unroll
                    for (int c = 0; c < PC; ++c) y[c] = fmaf(g, o[j][c], y[c]);
                }
            }
        }
    }
    if constexpr (WPR > 1) {
        __shared__ float s_m[WPR], s_sum[WPR], s_y[WPR][D];
#pragma unroll
        for (int c = 0; c < PC; ++c) s_y[warp][lane * PC + c] = y[c];
        if (lane == 0) {
            s_m[warp] = M;
            s_sum[warp] = sum;
        }
        __syncthreads();
        if (warp > 0) return;
        M = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < WPR; ++w) M = fmaxf(M, s_m[w]);
#pragma unroll
        for (int c = 0; c < PC; ++c) y[c] = 0.0f;
        for (int w = 0; w < WPR; ++w) {
            const float g = s_m[w] == -INFINITY ? (M == -INFINITY ? 1.0f : 0.0f) : ex2(s_m[w] - M);
            sum = fmaf(g, s_sum[w], sum);
#pragma unroll
            for (int c = 0; c < PC; ++c) y[c] = fmaf(g, s_y[w][lane * PC + c], y[c]);
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint16_t *const dst = p.out + (size_t)idx * D + lane * PC;
#pragma unroll
    for (int c = 0; c < PC; c += 2) *reinterpret_cast<uint32_t *>(dst + c) = pack_bf(y[c] * inv, y[c + 1] * inv);
    if (p.lse && lane == 0) p.lse[idx] = sum == 0.0f ? -INFINITY : (M + log2f(sum)) * 0.69314718055994531f;
}

// Launches the join with the kernel's shape; the kernels' grids.
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

// At least 176 KB, so that no block of another kernel that holds tensor memory (84 KB of shared
// memory and more each) shares the SM: this block takes all 512 columns, and two blocks that
// each wait for the other's columns or for its grid would never end.
template <class S>
constexpr int attend_smem(int B) {
    return std::max(176 * 1024, 1024 + S::oPrefix + (B + 1) * 4);
}

// The kernel of shape S, then the join.
template <class S, typename F>
cudaError_t launch_attend_shape(F *kernel, const AttendParams &prm, cudaStream_t stream) {
    static int configured[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!__atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, attend_smem<S>(kMaxBatch));
        if (e != cudaSuccess) return e;
        __atomic_store_n(&configured[dev], 1, __ATOMIC_RELEASE);
    }
    e = launch_attend_grid(kernel, kAttendBlocks, S::THREADS, attend_smem<S>(prm.B), stream, prm);
    if (e != cudaSuccess) return e;
    // a block a row while all of them run at once, else a warp
    const long long rows = (long long)prm.B * prm.T * prm.Hq;
    if (rows <= 152 * 8) return launch_attend_grid(join_kernel<S, kJoinWarps>, rows, kJoinWarps * 32, 0, stream, prm);
    return launch_attend_grid(join_kernel<S, 1>, (rows + kJoinWarps - 1) / kJoinWarps, kJoinWarps * 32, 0, stream, prm);
}

}  // namespace bsf8
