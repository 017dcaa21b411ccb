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

#include <algorithm>

namespace bsf8 {

namespace {

constexpr int kAttendBlocks = 152;   // one an SM of a GB300 (no block waits for another)
constexpr int kMaxBatch = 4096;
constexpr int kSoftWarps = 4, kDeqWarps = 8;
constexpr int kProducerWarp = kSoftWarps + kDeqWarps, kMmaWarp = kProducerWarp + 1;
constexpr int kThreadsA = (kMmaWarp + 1) * 32;
constexpr int kInfo = 4;             // tiles whose exponents and flags are kept
constexpr float kBias = 13.0f;       // p = 2^(x - m + kBias)
constexpr float kSlack = 2.0f;       // m lags the maximum by at most this
constexpr int kShift = 6;            // f16 values are code * 2^(e - E + kShift)

template <int D>
struct Shape {
    static constexpr int TN = D == 256 ? 64 : 128;   // keys a tile
    static constexpr int NS = D == 256 ? 1 : 2;      // S buffers
    static constexpr int EB = D / 32;                // exponent bytes a key
    static constexpr int SLOT = TN * D;              // bytes of a tile's codes
    static constexpr int NSLOT = D == 64 ? 8 : 5;
    static constexpr int F16 = TN * D * 2;           // bytes of an f16 tile
    // tensor memory columns: Q (f16 pairs), P (f16 pairs), O, S
    static constexpr int CQ = 0, CP = D / 2, CO = D == 256 ? 256 : CP + TN / 2, CS = D == 256 ? 192 : CO + D;
    static constexpr int oK = 0, oV = F16, oRing = 3 * F16, oExp = oRing + NSLOT * SLOT;
    static constexpr int oStage = oExp + NSLOT * 512, oPrefix = oStage + 4 * 32 * 33 * 4;
};

// At least 176 KB, so that no block of another kernel that holds tensor memory (84 KB of shared
// memory and more each) shares the SM: this block takes all 512 columns, and two blocks that
// each wait for the other's columns or for its grid would never end.
template <int D>
constexpr int attend_smem(int B) {
    return std::max(176 * 1024, 1024 + Shape<D>::oPrefix + (B + 1) * 4);
}

struct AttendParams {
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
    Segment s;
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

__device__ __forceinline__ void commit_a(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

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
    asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));  // relative error at most 2^-22
    return y;
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

// N registers of P (f16 pairs) into columns [t, t + N) of the thread's lane.
template <int N>
__device__ __forceinline__ void st_part(uint32_t t, const uint32_t (&r)[N]) {
    constexpr int C = N < 32 ? N : 32;
#pragma unroll
    for (int k = 0; k < N; k += C) {
        uint32_t x[C];
#pragma unroll
        for (int j = 0; j < C; ++j) x[j] = r[k + j];
        st_cols(t + k, x);
    }
}

// 32 channels of a row's output: bf16 where the segment is the whole row, else a partial.
template <int RT, int D>
__device__ __forceinline__ void store_row(const AttendParams &p, const Segment &g, bool whole, int slotw, int row,
                                          int t, int hq, int k, const float (&y)[32]) {
    if (whole) {
        uint16_t *dst = p.out + (((size_t)g.b * p.T + t) * p.Hq + hq) * D + k;
#pragma unroll
        for (int j = 0; j < 32; j += 8)
            *reinterpret_cast<uint4 *>(dst + j) = make_uint4(pack_bf(y[j], y[j + 1]), pack_bf(y[j + 2], y[j + 3]),
                                                             pack_bf(y[j + 4], y[j + 5]), pack_bf(y[j + 6], y[j + 7]));
    } else {
        float *dst = p.part + ((size_t)slotw * RT + row) * D + k;
#pragma unroll
        for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4 *>(dst + j) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
    }
}

struct AttendShared {
    uint64_t full8[8], empty8[8];   // ring slots: codes and exponents landed; read by all dequant warps
    uint64_t k_full;                // the f16 keys of a tile are written
    uint64_t v_full[2];
    uint64_t s_full[2], s_empty[2]; // S written (and the f16 keys read); read by all softmax warps
    uint64_t p_full;                // P written, O rescaled
    uint64_t pv_done[2];            // O updated, P and the f16 values read
    uint64_t q_full;                // the segment's Q is in tensor memory
    uint64_t soft;                  // the softmax warps' own barrier (bounded, unlike bar.sync)
    uint32_t tmem;
    int err;
    int vbits[8];                   // a slot's 16-key groups that exist (bit i)
    int ek[kInfo], valid[kInfo];    // a tile's key exponent, its groups
    int ev[kInfo], vnan[kInfo];     // the segment's value exponent at the tile; a value block holds NaN
    uint8_t nanblk[kInfo][128];     // then: each key's NaN blocks
    float2 stat[4][32];
    int scan[16];
};

}  // namespace

template <int D, int RT>
__global__ void __launch_bounds__(kThreadsA, 1) attend_kernel(const __grid_constant__ AttendParams p) {
    using S = Shape<D>;
    constexpr int TN = S::TN, NS = S::NS, REP = 128 / RT, CPT = TN / REP;  // CPT: key columns a thread
    constexpr int CH = CPT < 32 ? CPT : 32;                                // taken CH at a time
    extern __shared__ uint8_t dyn_smem[];
    uint8_t *const base = dyn_smem + ((1024u - (smem_u32(dyn_smem) & 1023u)) & 1023u);
    __shared__ AttendShared s;
    int *const prefix = reinterpret_cast<int *>(base + S::oPrefix);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 8; ++i) {
            mbar_init(&s.full8[i], 33);  // 32 lanes' exponent copies and lane 0's byte count
            mbar_init(&s.empty8[i], kDeqWarps);
        }
        mbar_init(&s.k_full, kDeqWarps);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.v_full[i], kDeqWarps);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.s_empty[i], kSoftWarps);
            mbar_init(&s.pv_done[i], 1);
        }
        mbar_init(&s.p_full, kSoftWarps);
        mbar_init(&s.q_full, kSoftWarps);
        mbar_init(&s.soft, kSoftWarps);
        s.err = 0;
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
    const uint32_t tmem = s.tmem;
    const long long total = prefix[p.B];
    const int w0 = range_start(total, blockIdx.x), w1 = range_start(total, blockIdx.x + 1);
    volatile int *const err = &s.err;
    // A bounded wait by every lane; false when it ran out or another warp's did.
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        bool ok = mbar_try_wait(bar, parity);
        if (!ok) ok = mbar_wait_bounded(bar, parity, p.timeout_ns);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) {
            *err = 1;
            report_timeout(p.status);
        }
        return ok && !*err;
    };

    if (warp == kProducerWarp) {
        // ------------------------------------------------------------ producer
        constexpr int NSB = TN / 16;             // 16-key groups a tile
        constexpr int KPL = 16 / S::EB;          // keys of a lane's 16 exponent bytes
        int slot = 0, n = 0;
        uint32_t ph = 0;
        bool ok = true;
        // lane i < NSB: the cache row (head h) of the tile's 16-key group i, -1 if there is none
        auto group_row = [&](const Segment &g, int tile) -> long long {
            long long row = -1;
            const int tok = tile * TN + 16 * lane;
            if (lane < NSB && tok < g.ctx + g.nodes) {
                const int pi = tok / p.c.page_size;
                const int page = p.c.table[(size_t)g.b * p.c.table_pages + pi];
                if ((unsigned)page < (unsigned)p.c.pages)
                    row = ((long long)page * p.c.heads + g.h) * p.c.page_size + (tok - pi * p.c.page_size);
                else
                    report_index(p.status);
            }
            return row;
        };
        auto copy = [&](const uint8_t *codes, const uint8_t *exps, long long row) -> bool {
            if (n >= S::NSLOT && !wait(&s.empty8[slot], ph ^ 1u)) return false;
            const uint32_t there = __ballot_sync(0xFFFFFFFFu, row >= 0);
            const long long prev = __shfl_up_sync(0xFFFFFFFFu, row, 1);
            const bool follows = lane > 0 && row >= 0 && prev >= 0 && prev + 16 == row;
            const uint32_t fol = __ballot_sync(0xFFFFFFFFu, follows);
            uint64_t *const bar = &s.full8[slot];
            if (lane == 0) {
                s.vbits[slot] = (int)there;
                mbar_arrive_expect_tx(bar, (uint32_t)__popc(there) * 16u * D);
            }
            __syncwarp();
            if (!p.skip_loads && row >= 0 && !follows) {  // the first group of a contiguous run
                const int run = 1 + __ffs(~(fol >> (lane + 1))) - 1;
                bulk_g2s(base + S::oRing + slot * S::SLOT + lane * 16 * D, codes + (size_t)row * D,
                         (uint32_t)(run * 16 * D), bar);
            }
            const int key = lane * KPL;
            const long long erow = __shfl_sync(0xFFFFFFFFu, row, min(key / 16, 31));
            if (key < TN && erow >= 0) {
                const uint8_t *src = exps + ((size_t)erow + (key & 15)) * S::EB;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                 smem_u32(base + S::oExp + slot * 512 + lane * 16)),
                             "l"(src)
                             : "memory");
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
            ++n;
            if (++slot == S::NSLOT) {
                slot = 0;
                ph ^= 1u;
            }
            return true;
        };
        for (int pos = w0; pos < w1 && ok;) {
            const Segment g = segment_at<D, RT>(p, prefix, pos, w1);
            const int tiles = g.kv1 - g.kv0;
            long long row = group_row(g, g.kv0), next = -1;
            ok = copy(p.c.k8, p.c.kexp, row);
            for (int i = 0; i < tiles && ok; ++i) {
                if (i + 1 < tiles) {
                    next = group_row(g, g.kv0 + i + 1);
                    ok = copy(p.c.k8, p.c.kexp, next);
                }
                ok = ok && copy(p.c.v8, p.c.vexp, row);
                row = next;
            }
            pos += tiles;
        }
        // every copy must have landed before the block's memory goes away (bounded)
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (!p.skip_loads)
            for (int i = max(0, n - S::NSLOT); i < n; ++i)
                (void)mbar_wait_bounded(&s.full8[i % S::NSLOT], (uint32_t)((i / S::NSLOT) & 1), p.timeout_ns);
    } else if (warp == kMmaWarp) {
        // ------------------------------------------------------------ MMA issue
        constexpr uint32_t idS = idesc_a(TN, false), idO = idesc_a(D, true);
        const uint32_t sK = smem_u32(base + S::oK), sV = smem_u32(base + S::oV);
        int ik = 0, iv = 0, seg = 0;  // tiles of the block so far
        bool ok = true;
        auto issue_s = [&]() -> bool {
            if (!wait(&s.k_full, (uint32_t)(ik & 1))) return false;
            const int sb = ik % NS;
            if (ik >= NS && !wait(&s.s_empty[sb], (uint32_t)(((ik / NS) & 1) ^ 1))) return false;
            fence_after();
            if (lane == 0) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)  // channels: 64-channel column ks / 4, then 32 bytes a step
                    umma_a(tmem + S::CS + sb * TN, tmem + S::CQ + 8 * ks,
                           desc_a(sK + (ks >> 2) * (TN * 128), 16) + 2 * (ks & 3), idS, ks > 0);
                commit_a(&s.s_full[sb]);
            }
            __syncwarp();
            ++ik;
            return true;
        };
        for (int pos = w0; pos < w1 && ok; ++seg) {
            const Segment g = segment_at<D, RT>(p, prefix, pos, w1);
            const int tiles = g.kv1 - g.kv0;
            ok = wait(&s.q_full, (uint32_t)(seg & 1)) && issue_s();
            for (int i = 0; i < tiles && ok; ++i) {
                if (i + 1 < tiles) ok = issue_s();
                ok = ok && wait(&s.v_full[iv & 1], (uint32_t)((iv >> 1) & 1)) && wait(&s.p_full, (uint32_t)(iv & 1));
                if (!ok) break;
                fence_after();
                if (lane == 0) {
#pragma unroll
                    for (int ks = 0; ks < TN / 16; ++ks)  // 16 keys a step: two 8-key atoms
                        umma_a(tmem + S::CO, tmem + S::CP + 8 * ks,
                               desc_a(sV + (iv & 1) * S::F16 + ks * 2048, TN * 128), idO, i > 0 || ks > 0);
                    commit_a(&s.pv_done[iv & 1]);
                }
                __syncwarp();
                ++iv;
            }
            pos += tiles;
        }
        // the last products must be done before tensor memory goes back (bounded)
        if (iv > 0) (void)wait(&s.pv_done[(iv - 1) & 1], (uint32_t)(((iv - 1) >> 1) & 1));
        if (ik > 0) (void)wait(&s.s_full[(ik - 1) % NS], (uint32_t)(((ik - 1) / NS) & 1));
    } else if (warp >= kSoftWarps) {
        // ------------------------------------------------------------ dequant
        const int dw = warp - kSoftWarps;
        constexpr int NQ = D / 64, RPW = TN / kDeqWarps, PASSES = RPW / 8 * NQ;
        int slot = 0, ik = 0, iv = 0;
        uint32_t ph = 0;
        bool ok = true;
        // Conflict-free on both sides: in a quarter-warp, four 16-code chunks of an even row and
        // four of the next row from another 64-channel column (other banks in the codes; odd
        // against even 16-byte units in the swizzled f16 rows).
        const int ci = lane & 3, cj = (lane >> 2) & 1, cr = 2 * (lane >> 3) + cj;
        auto turn = [&](uint8_t *dst, int E, bool check, int keys, uint32_t vbits, bool value) {
            const uint8_t *src = base + S::oRing + slot * S::SLOT;
            const uint8_t *ex = base + S::oExp + slot * 512;
#pragma unroll
            for (int ps = 0; ps < PASSES; ++ps) {
                const int row = dw * RPW + (ps / NQ) * 8 + cr, ch = ci + 4 * ((cj + ps) % NQ);
                uint4 w = *reinterpret_cast<const uint4 *>(src + row * D + ch * 16);
                const int e = ex[row * S::EB + (ch >> 1)];
                if (check && value && (row >= keys || !((vbits >> (row >> 4)) & 1) || e == 255)) w = make_uint4(0, 0, 0, 0);
                const uint32_t sc = f16_pow2(e - E + kShift);
                uint4 lo, hi;
                widen16(w, check && value && w.x == 0 && w.y == 0 && w.z == 0 && w.w == 0 ? 0u : sc, lo, hi);
                uint8_t *d = dst + (ch >> 2) * (TN * 128) + row * 128;
                const int u = 2 * (ch & 3), x = row & 7;
                *reinterpret_cast<uint4 *>(d + ((u ^ x) << 4)) = lo;
                *reinterpret_cast<uint4 *>(d + (((u + 1) ^ x) << 4)) = hi;
            }
        };
        // The largest exponent byte of the tile's keys that exist, 255 (NaN) left out; bit 8: a 255
        // was among them.
        auto tile_exponent = [&](int keys, uint32_t vbits) -> int {
            constexpr int KPL = 16 / S::EB;
            const int key0 = lane * KPL;
            uint32_t mx = 0, nan = 0;
            if (key0 < TN) {
                const uint4 v = *reinterpret_cast<const uint4 *>(base + S::oExp + slot * 512 + lane * 16);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t x = w[j];
                    uint32_t keep = 0;  // byte mask of keys that exist
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = key0 + (4 * j + i) / S::EB;
                        if (key < keys && ((vbits >> (key >> 4)) & 1)) keep |= 0xFFu << (8 * i);
                    }
                    x &= keep;
                    const uint32_t is = __vcmpeq4(x, 0xFFFFFFFFu);
                    nan |= is;
                    mx = __vmaxu4(mx, x & ~is);
                }
            }
            mx = __vmaxu4(mx, mx >> 16);
            mx = max(mx & 0xFFu, (mx >> 8) & 0xFFu);
            mx = __reduce_max_sync(0xFFFFFFFFu, mx);
            return (int)mx | (__any_sync(0xFFFFFFFFu, nan != 0) ? 256 : 0);
        };
        auto release = [&]() {  // the slot is read; the f16 tile is on its way to the async proxy
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.empty8[slot]);
            if (++slot == S::NSLOT) {
                slot = 0;
                ph ^= 1u;
            }
        };
        auto keys_tile = [&](const Segment &g, int tile) -> bool {
            if (!wait(&s.full8[slot], ph)) return false;
            if (ik > 0 && !wait(&s.s_full[(ik - 1) % NS], (uint32_t)(((ik - 1) / NS) & 1))) return false;
            const int keys = min(TN, g.ctx + g.nodes - tile * TN);
            const uint32_t vb = (uint32_t)s.vbits[slot];
            const int E = tile_exponent(keys, vb) & 255;
            turn(base + S::oK, E, false, keys, vb, false);
            if (dw == 0 && lane == 0) {
                s.ek[ik % kInfo] = E;
                s.valid[ik % kInfo] = (int)vb;
            }
            release();
            if (lane == 0) mbar_arrive(&s.k_full);
            ++ik;
            return true;
        };
        for (int pos = w0; pos < w1 && ok;) {
            const Segment g = segment_at<D, RT>(p, prefix, pos, w1);
            const int tiles = g.kv1 - g.kv0;
            int EV = 0;  // the segment's running value exponent
            ok = keys_tile(g, g.kv0);
            for (int i = 0; i < tiles && ok; ++i) {
                if (i + 1 < tiles) ok = keys_tile(g, g.kv0 + i + 1);
                ok = ok && wait(&s.full8[slot], ph);
                if (ok && iv >= 2) ok = wait(&s.pv_done[iv & 1], (uint32_t)(((iv >> 1) & 1) ^ 1));
                if (!ok) break;
                const int keys = min(TN, g.ctx + g.nodes - (g.kv0 + i) * TN);
                const uint32_t vb = (uint32_t)s.vbits[slot];
                const int te = tile_exponent(keys, vb);
                const bool nan = te >= 256;
                EV = max(EV, te & 255);
                const bool check = nan || keys < TN || vb != (1u << (TN / 16)) - 1u;
                uint8_t *dst = base + S::oV + (iv & 1) * S::F16;
                if (check) turn(dst, EV, true, keys, vb, true);
                else turn(dst, EV, false, keys, vb, true);
                if (nan && dw == 0) {
                    const uint8_t *ex = base + S::oExp + slot * 512;
                    for (int key = lane; key < TN; key += 32) {
                        uint32_t m = 0;
                        for (int j = 0; j < S::EB; ++j) m |= (ex[key * S::EB + j] == 255 ? 1u : 0u) << j;
                        s.nanblk[iv % kInfo][key] = (uint8_t)m;
                    }
                    __syncwarp();
                }
                if (dw == 0 && lane == 0) {
                    s.ev[iv % kInfo] = EV;
                    s.vnan[iv % kInfo] = nan ? 1 : 0;
                }
                release();
                if (lane == 0) mbar_arrive(&s.v_full[iv & 1]);
                ++iv;
            }
            pos += tiles;
        }
    } else {
        // ------------------------------------------------------------ softmax and output
        const uint32_t tl = tmem + ((uint32_t)(32 * warp) << 16);  // this warp's tensor memory lanes
        const int row = (32 * warp + lane) % RT;                   // row of the tile
        const int col0 = (32 * warp / RT) * CPT;                   // this copy's key columns
        int it = 0;
        uint32_t soft_ph = 0;
        bool ok = true;
        auto soft_sync = [&]() -> bool {
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.soft);
            soft_ph ^= 1u;
            return wait(&s.soft, soft_ph ^ 1u);
        };
        {   // P is zero outside each copy's columns, once and for all
            const uint32_t z[16] = {};
            if (REP > 1) {
#pragma unroll
                for (int c = 0; c < TN / 2; c += 16) st_cols(tl + S::CP + c, z);
                wait_st();
            }
        }
        for (int pos = w0; pos < w1 && ok;) {
            const Segment g = segment_at<D, RT>(p, prefix, pos, w1);
            const int tiles = g.kv1 - g.kv0;
            const int r = g.rt * RT + row;         // row of the request and head
            const bool real = r < g.nodes * p.g;
            const int t = real ? r / p.g : 0, hq = g.h * p.g + (real ? r - t * p.g : 0);
            // ---- Q: the row scaled by a power of two so that its largest lies in [2^13, 2^14)
            const uint16_t *qr = p.q + ((size_t)g.b * p.T + t) * p.ldq + (size_t)hq * D;
            uint32_t am = 0;
            if (real)
                for (int c = 0; c < D; c += 8) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(qr + c);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) am = max(am, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
                }
            const int eq = max((int)(am >> 7) - 127 - 13, -100);
            const float qs = pow2i(-eq);  // eq <= 115
#pragma unroll 1
            for (int c = 0; c < D; c += 64) {
                uint32_t o[32];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (real) v = *reinterpret_cast<const uint4 *>(qr + c + 8 * j);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        o[4 * j + k] = pack_f16(__uint_as_float(w[k] << 16) * qs, __uint_as_float(w[k] & 0xFFFF0000u) * qs);
                }
                st_cols(tl + S::CQ + c / 2, o);
            }
            wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.q_full);
            const float crow = p.scale_log2 * pow2i(eq);

            float m = -INFINITY, l = 0.0f;
            int ev = 0;
            uint32_t nanblk = 0;
            const int32_t *mrow = p.mask ? p.mask + ((size_t)g.b * p.T + t) * p.W : nullptr;
            for (int i = 0; i < tiles && ok; ++i, ++it) {
                const int sb = it % NS, info = it % kInfo;
                ok = wait(&s.s_full[sb], (uint32_t)((it / NS) & 1));
                if (!ok) break;
                fence_after();
                const uint32_t ts = tl + S::CS + sb * TN + col0;
                const float c = crow * pow2i(s.ek[info] - 127 - kShift);  // S -> x
                const int slot0 = (g.kv0 + i) * TN + col0;                // cache slot of the thread's first column
                const uint32_t vb = (uint32_t)s.valid[info];
                const bool masked = (g.kv0 + i + 1) * TN > g.ctx || vb != (1u << (TN / 16)) - 1u;
                // visible keys among columns [k, k + CH) of the thread
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
                    return CH < 32 ? w & ((1u << (CH & 31)) - 1u) : w;
                };
                // ---- the maximum
                float mt = -INFINITY;
                uint32_t x[CH];
#pragma unroll
                for (int k = 0; k < CPT; k += CH) {
                    ld_cols(ts + k, x);
                    wait_ld();
                    if (masked) {
                        const uint32_t w = seen(k);
#pragma unroll
                        for (int j = 0; j < CH; ++j) x[j] = (w >> j) & 1u ? x[j] : 0xFF800000u;
                    }
#pragma unroll
                    for (int j = 0; j < CH; ++j) mt = fmaxf(mt, __uint_as_float(x[j]));
                }
                mt = mt == -INFINITY ? mt : mt * c;
                const bool grow = mt > m + kSlack;  // also out of m = -inf
                const float mn = grow ? mt : m;
                const float off = mn == -INFINITY ? 0.0f : kBias - mn;
                // ---- p, its sum, and P for the second product
                uint32_t pk[CPT / 2];
                float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
                for (int k = 0; k < CPT; k += CH) {
                    if (CPT > CH) {
                        ld_cols(ts + k, x);
                        wait_ld();
                        if (masked) {
                            const uint32_t w = seen(k);
#pragma unroll
                            for (int j = 0; j < CH; ++j) x[j] = (w >> j) & 1u ? x[j] : 0xFF800000u;
                        }
                    }
#pragma unroll
                    for (int j = 0; j < CH; j += 2) {
                        const float a = ex2(fmaf(__uint_as_float(x[j]), c, off));
                        const float b = ex2(fmaf(__uint_as_float(x[j + 1]), c, off));
                        sum0 += a;
                        sum1 += b;
                        pk[(k + j) / 2] = pack_f16(a, b);
                    }
                }
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.s_empty[sb]);
                // ---- the values' exponent; the product before this one must be done with P and O
                ok = wait(&s.v_full[it & 1], (uint32_t)((it >> 1) & 1));
                if (ok && it > 0) ok = wait(&s.pv_done[(it - 1) & 1], (uint32_t)(((it - 1) >> 1) & 1));
                if (!ok) break;
                fence_after();
                const int evn = s.ev[info];
                const float fm = grow ? (m == -INFINITY ? 0.0f : ex2(m - mn)) : 1.0f;
                if (i > 0 && __any_sync(0xFFFFFFFFu, grow || evn != ev)) {
                    const float f = fm * pow2i(max(ev - evn, -149));
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
                ev = evn;
                l = l * fm + (sum0 + sum1);
                m = mn;
                if (s.vnan[info]) {
#pragma unroll 1
                    for (int k = 0; k < CPT; k += CH) {
                        uint32_t w = real ? (masked ? seen(k) : 0xFFFFFFFFu) : 0u;
                        for (int j = 0; j < CH; ++j)
                            if ((w >> j) & 1u) nanblk |= s.nanblk[info][col0 + k + j];
                    }
                }
                st_part(tl + S::CP + col0 / 2, pk);
                wait_st();
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.p_full);
            }
            pos += tiles;
            if (!ok) break;
            // ---- the segment's output
            ok = wait(&s.pv_done[(it - 1) & 1], (uint32_t)(((it - 1) >> 1) & 1));
            if (!ok) break;
            fence_after();
            const bool whole = g.kv0 == 0 && g.kv1 == g.nt;
            const int slotw = 2 * blockIdx.x + (g.kv0 > 0 ? 0 : 1);
            float M = m, L = l;
            if (REP > 1) {  // the copies' maxima and sums
                s.stat[warp][lane] = make_float2(m, l);
                ok = soft_sync();
                if (!ok) break;
                M = -INFINITY;
#pragma unroll
                for (int q = 0; q < REP; ++q) M = fmaxf(M, s.stat[(warp + q * (RT / 32)) & 3][lane].x);
                L = 0.0f;
#pragma unroll
                for (int q = 0; q < REP; ++q) {  // in the order of the copies
                    const float2 st = s.stat[(q * (RT / 32) + warp % (RT / 32)) & 3][lane];
                    L += st.y == 0.0f ? 0.0f : st.y * ex2(st.x == -INFINITY ? 0.0f : st.x - M);
                }
            }
            // O (this copy) * f = its share of the normalised output
            const float f = L == 0.0f ? 0.0f : (l == 0.0f ? 0.0f : ex2(m == -INFINITY ? 0.0f : m - M)) / L;
            const float fv = pow2i(ev - 127 - kShift);
            const float Lt = L * pow2i(-(int)kBias);  // the sum in units of 2^M
            if (real && row < RT && 32 * warp < RT) {
                if (whole) {
                    if (p.lse)
                        p.lse[((size_t)g.b * p.T + t) * p.Hq + hq] =
                            L == 0.0f ? -INFINITY : (M + log2f(Lt)) * 0.69314718055994531f;
                } else {
                    p.stat[(size_t)slotw * RT + row] = make_float2(M, Lt);
                }
            }
            float *const stage = reinterpret_cast<float *>(base + S::oStage);
#pragma unroll 1
            for (int k = 0; k < D; k += 32) {
                uint32_t o[32];
                ld_cols(tl + S::CO + k, o);
                wait_ld();
                const bool bad = (nanblk >> (k / 32)) & 1u;
                float y[32];
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    y[j] = bad ? __uint_as_float(0x7FC00000u) : L == 0.0f ? 0.0f : __uint_as_float(o[j]) * f * fv;
                if (REP == 1) {
                    if (real) store_row<RT, D>(p, g, whole, slotw, row, t, hq, k, y);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) stage[(warp * 32 + lane) * 33 + j] = y[j];
                    ok = soft_sync();
                    if (!ok) break;
                    // thread -> a row's part of 32 / REP channels: the copies added in their order
                    constexpr int CW = 32 / REP;
                    const int rr = threadIdx.x / REP, j0 = (threadIdx.x % REP) * CW;
                    float z[CW];
#pragma unroll
                    for (int j = 0; j < CW; ++j) {
                        z[j] = stage[rr * 33 + j0 + j];
#pragma unroll
                        for (int q = 1; q < REP; ++q) z[j] += stage[(rr + q * RT) * 33 + j0 + j];
                    }
                    const int r2 = g.rt * RT + rr;
                    if (r2 < g.nodes * p.g) {
                        const int t2 = r2 / p.g, h2 = g.h * p.g + (r2 - t2 * p.g);
                        if (whole) {
                            uint16_t *dst = p.out + (((size_t)g.b * p.T + t2) * p.Hq + h2) * D + k + j0;
#pragma unroll
                            for (int j = 0; j < CW; j += 8)
                                *reinterpret_cast<uint4 *>(dst + j) =
                                    make_uint4(pack_bf(z[j], z[j + 1]), pack_bf(z[j + 2], z[j + 3]),
                                               pack_bf(z[j + 4], z[j + 5]), pack_bf(z[j + 6], z[j + 7]));
                        } else {
                            float *dst = p.part + ((size_t)slotw * RT + rr) * D + k + j0;
#pragma unroll
                            for (int j = 0; j < CW; j += 4)
                                *reinterpret_cast<float4 *>(dst + j) = make_float4(z[j], z[j + 1], z[j + 2], z[j + 3]);
                        }
                    }
                    ok = soft_sync();
                    if (!ok) break;
                }
            }
        }
    }

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
