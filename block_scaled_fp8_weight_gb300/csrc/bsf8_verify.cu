// bsf8_verify.cu -- verification of drafted token trees against the target's probabilities.
//
// Recursive rejection (bsf8.h states it in full): with P, Q the fixed-point probabilities at
// the walk's node and Z the mass left, child x is kept iff floor(U Q'(x) / 2^24) < R(x) with
// Q' = floor(Q Z / 2^40); otherwise R = max(R - Q', 0) and Z = sum R.  As every Q' >= 0,
//   R after the rejections with masses Z_1 .. Z_k  =  max(P - sum_j floor(Q Z_j / 2^40), 0),
// so R is never stored: a pass recomputes it from the rows of p and q.  All sums are integer
// sums, so neither the split of a row over threads and blocks nor their order changes a bit.
//
// A cluster of blocks per request.  What the walk may ask of single elements -- p and q of each
// node's token at its parent -- is loaded up front by one thread a node, which also settles the
// node's test for the case that no sibling was asked before it.  Warp 0 of every block then walks
// the tree in shared memory (the same steps in each), and the vocabulary is read only where a sum of
// R is needed: once a rejection, and for the last draw unless the last step was a rejection (its sum
// is the draw's).  A pass gives each block a contiguous slice of the row and each warp a contiguous
// part of it, so the draw's element is found by adding up slices, then warps, then one warp's part,
// which its block reads again (from L2).
// HBM bound at large batches (a row of p and q a rejection, and one for the last draw), latency bound at
// small ones: the chain nodes, their probabilities, a pass, the cluster's barrier, the draw.  64 requests
// of 16 nodes over 131072 tokens: 43 to 48 us in a graph, by the walks (110 with each node tested on the way and
// 64-bit products for every element); one of 6 nodes over 50257: 8.6 to 10.3 us.
#include "bsf8_device.cuh"
#include "bsf8_internal.h"

#include <algorithm>

namespace bsf8 {

namespace {

constexpr int kVThreads = 256;
constexpr int kVWarps = kVThreads / 32;
constexpr int kNodes = 256;        // BSF8_MAX_NODES
static_assert(kNodes <= kVThreads, "a thread a node");
constexpr int kMaxVCluster = 8;    // the portable cluster size
constexpr int kBatch = 4;          // 16-byte loads of a row a thread has in flight
typedef unsigned long long u64;
constexpr u64 kOne = 1ull << 40;

// floor(p * 2^40), p clamped to [0, 1], NaN as 0, in two steps of 20 bits: adding 2^23 towards zero
// leaves floor(x) in the low bits of the sum (0 <= x < 2^23), and the rest is exact in fp32.  The
// conversion instruction to 64 bits runs at a small part of the rate of these.
__device__ __forceinline__ u64 fix(float p) {
    const float x = fminf(fmaxf(p, 0.0f), 1.0f) * 1048576.0f;
    const float t = __fadd_rz(x, 8388608.0f);
    const float r = (x - (t - 8388608.0f)) * 1048576.0f;
    const uint32_t hi = __float_as_uint(t) & 0x7FFFFFu;
    const uint32_t lo = __float_as_uint(__fadd_rz(r, 8388608.0f)) & 0x7FFFFFu;
    return (u64)hi * 1048576u + lo;
}

__device__ __forceinline__ u64 times(u64 q, u64 z) {  // floor(q z / 2^40)
    return (__umul64hi(q, z) << 24) | ((q * z) >> 40);
}

__device__ __forceinline__ u64 part(u64 u, u64 z) {  // floor(u z / 2^24)
    return (__umul64hi(u, z) << 40) | ((u * z) >> 24);
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
    return v;
}

__device__ __forceinline__ u64 ld_cluster_u64(uint32_t addr) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}

}  // namespace

struct VerifyShared {
    u64 P[kNodes], Q[kNodes];  // of node i's token, at node i's parent
    uint32_t U[kNodes];
    int parent[kNodes], tok[kNodes], path[kNodes];
    uint8_t first[kNodes];     // kept if asked before its siblings
    u64 Z[kNodes];             // the mass before each rejection at the walk's node
    int gone[kNodes];          // the token of each rejection there
    u64 wsum[kVWarps];         // a pass: each warp's sum of R
    u64 bsum[2];               // this block's, read by the cluster (slots taken in turn)
    u64 rsum[kMaxVCluster];    // every block's
    int cur, rej;              // the walk's node, rejections there
    int small;                 // every Z here is below 2^42
    int stop;                  // the draw is next: no child is left to ask and R is summed
    u64 at;                    // the draw's threshold inside a warp's part
    int warp;                  // that warp, or -1
};

// floor(q z / 2^40) for q <= 2^40 and z < 2^42, from parts of 20 bits.
__device__ __forceinline__ u64 times20(u64 q, uint32_t zh, uint32_t zl) {
    const uint32_t qh = (uint32_t)(q >> 20), ql = (uint32_t)q & 0xFFFFFu;
    return (u64)qh * zh + (((u64)qh * zl + (u64)ql * zh + (((u64)ql * zl) >> 20)) >> 20);
}

// R of element x, whose fixed-point probabilities at the walk's node are P and Q.
__device__ __noinline__ u64 left_of(u64 P, u64 Q, int x, const VerifyShared &s, bool drawn) {
    if (drawn) {
        u64 off = s.rej > 0 ? Q : 0;  // the first rejection's mass is 2^40
        // (as soon as it reaches P nothing is left: the sum of all need not fit 64 bits)
        for (int j = 1; j < s.rej && off < P; ++j)
            off += s.small ? times20(Q, (uint32_t)(s.Z[j] >> 20), (uint32_t)s.Z[j] & 0xFFFFFu) : times(Q, s.Z[j]);
        return P > off ? P - off : 0;
    }
    for (int j = 0; j < s.rej; ++j)
        if (s.gone[j] == x) return 0;
    return P;
}

// Elements x .. x + 3 of a row; those outside [0, V) count as 0 and are not read.  row + x is
// 16-byte aligned.
__device__ __forceinline__ void load4(const float *row, int x, int V, float (&v)[4]) {
    if (x >= 0 && x + 4 <= V) {
        const float4 f = *reinterpret_cast<const float4 *>(row + x);
        v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (unsigned)(x + i) < (unsigned)V ? row[x + i] : 0.0f;
    }
}

// The walk's own state, the same in every lane of warp 0.
struct Walk {
    u64 total;                    // the mass Z of R
    int cur, rej, next, count;    // node, rejections there, next child to ask, nodes kept
    bool done, summed;            // no child is left to ask; the sums are those of the present R
};

// The next thing after a sum (or the start), by warp 0: on along the walk until a rejection (whose
// sum of R is wanted) or the last child; or, when R was all 0 after that, a sum of P instead.
__device__ __forceinline__ void step(VerifyShared &s, Walk &w, int n, bool drawn, int lane) {
    if (w.done) w.rej = 0;
    while (!w.done) {
        // the next child of w.cur
        int i = n;
        for (int base = w.next & ~31; base < n; base += 32) {
            const int c = base + lane;
            const uint32_t m = __ballot_sync(0xFFFFFFFFu, c >= w.next && c < n && s.parent[c] == w.cur);
            if (m) {
                i = base + __ffs(m) - 1;
                break;
            }
        }
        w.next = min(n, i + 1);
        if (i == n) {
            w.done = true;
            break;
        }
        bool kept = s.first[i];
        if (w.rej > 0) kept = part(s.U[i], times(s.Q[i], w.total)) < left_of(s.P[i], s.Q[i], s.tok[i], s, drawn);
        w.summed = false;
        if (!kept) {
            __syncwarp();
            if (lane == 0) {
                s.Z[w.rej] = w.total;
                s.gone[w.rej] = s.tok[i];
                if (w.total >= 1ull << 42) s.small = 0;
                s.rej = w.rej + 1;
            }
            __syncwarp();
            ++w.rej;
            break;
        }
        w.cur = i;
        w.rej = 0;
        w.total = kOne;
        __syncwarp();
        if (lane == 0) {
            s.path[w.count] = i;
            s.cur = i;
            s.rej = 0;
            s.small = 1;
        }
        __syncwarp();
        ++w.count;
    }
    __syncwarp();
    if (lane == 0) {
        s.rej = w.rej;
        s.stop = w.done && w.summed;
    }
}

__global__ void __launch_bounds__(kVThreads, 4) verify_kernel(const VerifyArgs a, int cluster, int *status) {
    __shared__ VerifyShared s;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = blockIdx.x / cluster, rank = blockIdx.x % cluster;
    const int T = a.T, V = a.V;
    // every node's words at once with the node count
    const size_t nb = (size_t)b * T + tid;
    const bool mine = tid < T;
    const float u0 = mine ? a.u[nb] : 0.0f;
    const int par0 = mine ? a.parent[nb] : -1, x0 = mine ? a.tokens[nb] : 0;
    int n = a.nodes ? a.nodes[b] : T;
    if (n < 1 || n > T) {
        if (tid == 0) report_index(status);
        n = max(1, min(n, T));
    }
    const bool drawn = a.q != nullptr;
    const float *const pb = a.p + (size_t)b * T * a.ld;
    const float *const qb = drawn ? a.q + (size_t)b * T * a.ld : nullptr;
    if (tid < n) {  // T <= kVThreads
        const int i = tid;
        s.U[i] = (uint32_t)(fminf(fmaxf(u0, 0.0f), 0.99999994f) * 16777216.0f);
        int par = -1, x = 0;
        u64 P = 0, Q = 0;
        if (i > 0) {
            par = par0;
            x = x0;
            if ((unsigned)par >= (unsigned)i || (unsigned)x >= (unsigned)V) {
                report_index(status);
                par = -1;
                x = 0;
            } else {
                P = fix(pb[(size_t)par * a.ld + x]);
                Q = drawn ? fix(qb[(size_t)par * a.ld + x]) : kOne;
            }
        }
        s.parent[i] = par;
        s.tok[i] = x;
        s.P[i] = P;
        s.Q[i] = Q;
        s.first[i] = part(s.U[i], Q) < P;
    }
    if (tid == 0) {
        s.cur = s.rej = s.path[0] = 0;
        s.small = 1;
    }
    Walk w{kOne, 0, 0, 1, 1, false, false};
    __syncthreads();
    if (warp == 0) step(s, w, n, drawn, lane);
    __syncthreads();

    int per_warp = 0, mis = 0, groups = 0;  // of the last pass's row
    // Warp 0 changes the walk's state only between the last two barriers of a turn, so that every
    // thread reads the same state at its top.
    for (uint32_t pass = 0; !s.stop; ++pass) {
        // -------------------------------------------------------------- a pass: the sums of R
        const float *prow = pb + (size_t)s.cur * a.ld;
        const float *qrow = drawn ? qb + (size_t)s.cur * a.ld : nullptr;
        // p and q are 16-byte aligned and share ld, so their rows share the misalignment
        mis = (int)((size_t)(prow - a.p) & 3);
        groups = (V + mis + 3) / 4;
        per_warp = ((groups + cluster * kVWarps - 1) / (cluster * kVWarps) + 31) / 32 * 32;
        const int g0 = (rank * kVWarps + warp) * per_warp, g1 = min(groups, g0 + per_warp);
        const int rej = s.rej;
        const bool useq = drawn && rej > 0;
        u64 sum = 0;
        const uint32_t zh1 = rej > 1 ? (uint32_t)(s.Z[1] >> 20) : 0, zl1 = rej > 1 ? (uint32_t)s.Z[1] & 0xFFFFFu : 0;
        // r less floor(Q z / 2^40), at least 0 (Q < 2^31, z < 2^42 in parts of 22 and 20 bits; the
        // quotient is below 2^33, and at or above 2^32 it exceeds r)
        auto less = [](uint32_t r, uint32_t Q, uint32_t zh, uint32_t zl) -> uint32_t {
            const u64 t = (u64)Q * zh + (u64)__umulhi(Q, zl << 12);
            const uint32_t off = (uint32_t)(t >> 20);
            return (uint32_t)(t >> 52) ? 0u : max(r, off) - off;
        };
        // Almost all probabilities of a large vocabulary are small: below 2^-9 the fixed point fits 31
        // bits, one conversion (negative and NaN give 0) and 32-bit differences do.
        auto add = [&](const float4 &pf, const float4 &qf, int x) {
            const float top = fmaxf(fmaxf(fmaxf(pf.x, pf.y), fmaxf(pf.z, pf.w)),
                                    useq ? fmaxf(fmaxf(qf.x, qf.y), fmaxf(qf.z, qf.w)) : 0.0f);
            const float pv[4] = {pf.x, pf.y, pf.z, pf.w}, qv[4] = {qf.x, qf.y, qf.z, qf.w};
            if (top < 0.001953125f && (rej == 0 || (useq && s.small))) {
                uint32_t r[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) r[i] = __float2uint_rz(pv[i] * 1099511627776.0f);
                if (useq) {
                    uint32_t Q[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        Q[i] = __float2uint_rz(qv[i] * 1099511627776.0f);
                        r[i] = max(r[i], Q[i]) - Q[i];
                    }
                    uint32_t zh = zh1, zl = zl1;
#pragma unroll 1
                    for (int j = 1; j < rej; ++j) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) r[i] = less(r[i], Q[i], zh, zl);
                        zh = (uint32_t)(s.Z[j + 1 < rej ? j + 1 : j] >> 20);
                        zl = (uint32_t)s.Z[j + 1 < rej ? j + 1 : j] & 0xFFFFFu;
                    }
                }
                sum += (u64)(r[0] + r[1]) + (r[2] + r[3]);  // each below 2^31
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    sum += left_of(fix(pv[i]), useq ? fix(qv[i]) : 0, x + i, s, drawn);
            }
        };
        // whole groups of four, kBatch loads of each row in flight; then the ragged ones
        const int gi = max(g0, mis > 0 ? 1 : 0), ge = min(g1, (V + mis) / 4);
        int g = gi + lane;
        for (; g + 32 * (kBatch - 1) < ge; g += 32 * kBatch) {
            float4 pf[kBatch], qf[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) pf[j] = *reinterpret_cast<const float4 *>(prow + 4 * (g + 32 * j) - mis);
#pragma unroll
            for (int j = 0; j < kBatch; ++j)
                qf[j] = useq ? *reinterpret_cast<const float4 *>(qrow + 4 * (g + 32 * j) - mis) : make_float4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < kBatch; ++j) add(pf[j], qf[j], 4 * (g + 32 * j) - mis);
        }
        auto ragged = [&](int k) {
            float pv[4], qv[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            load4(prow, 4 * k - mis, V, pv);
            if (useq) load4(qrow, 4 * k - mis, V, qv);
            add(make_float4(pv[0], pv[1], pv[2], pv[3]), make_float4(qv[0], qv[1], qv[2], qv[3]), 4 * k - mis);
        };
        for (; g < g1; g += 32) ragged(g);
        if (gi > g0 && g0 == 0 && g1 > 0 && lane == 0) ragged(0);  // the row's first, partial group
        sum = warp_sum(sum);
        if (lane == 0) s.wsum[warp] = sum;
        __syncthreads();
        if (warp == 0) {
            const u64 t = warp_sum(lane < kVWarps ? s.wsum[lane] : 0);
            if (lane == 0) {
                s.bsum[pass & 1] = t;
                s.rsum[0] = t;
            }
        }
        // A slot of bsum is written again two passes on: by then its readers have passed the
        // barrier of the pass between.
        if (cluster > 1) cluster_barrier();
        if (warp == 0) {
            u64 t = 0;
            __syncwarp();
            if (cluster > 1) {
                if (lane < cluster) s.rsum[lane] = t = ld_cluster_u64(map_to_rank(&s.bsum[pass & 1], lane));
            } else if (lane == 0) {
                t = s.rsum[0];
            }
            w.total = warp_sum(t);
            w.summed = w.total > 0 || w.rej == 0;  // nothing left after rejections: once more, from P
            if (w.done && w.summed) {
                if (lane == 0) s.stop = 1;
            } else {
                step(s, w, n, drawn, lane);
            }
        }
        __syncthreads();
    }

    // ------------------------------------------------------------------ the draw
    if (warp == 0) {
        const u64 thr = part(s.U[0], w.total);
        const u64 mine = lane < kVWarps ? s.wsum[lane] : 0;
        u64 upto = mine;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const u64 o = __shfl_up_sync(0xFFFFFFFFu, upto, m);
            if (lane >= m) upto += o;
        }
        const u64 before = warp_sum(lane < rank ? s.rsum[lane] : 0) + upto - mine;
        const uint32_t here = __ballot_sync(0xFFFFFFFFu, thr >= before && thr < before + mine);
        if (lane == 0) s.warp = here ? __ffs(here) - 1 : -1;
        if (thr >= before && thr < before + mine) s.at = thr - before;
        if (rank == 0) {
            if (lane == 0) {
                a.count[b] = w.count;
                if (w.total == 0) a.token[b] = V - 1;
            }
            for (int i = lane; i < T; i += 32) a.path[(size_t)b * T + i] = i < w.count ? s.path[i] : -1;
        }
    }
    __syncthreads();
    if (s.warp >= 0) {  // one block of the cluster: its warp's part again, in order over the threads
        const float *prow = pb + (size_t)s.cur * a.ld;
        const float *qrow = drawn ? qb + (size_t)s.cur * a.ld : nullptr;
        const int w0 = (rank * kVWarps + s.warp) * per_warp, w1 = min(groups, w0 + per_warp);
        const int each = (per_warp + kVThreads - 1) / kVThreads;
        const int g0 = min(w1, w0 + tid * each), g1 = min(w1, g0 + each);
        const bool useq = drawn && s.rej > 0;
        u64 sum = 0;
        for (int g = g0; g < g1; ++g) {
            float pv[4], qv[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            load4(prow, 4 * g - mis, V, pv);
            if (useq) load4(qrow, 4 * g - mis, V, qv);
#pragma unroll
            for (int i = 0; i < 4; ++i) sum += left_of(fix(pv[i]), fix(qv[i]), 4 * g - mis + i, s, drawn);
        }
        u64 upto = sum;  // inclusive sums over the warp's lanes
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const u64 o = __shfl_up_sync(0xFFFFFFFFu, upto, m);
            if (lane >= m) upto += o;
        }
        __syncthreads();  // s.wsum was read by warp 0, before the barrier above
        if (lane == 31) s.wsum[warp] = upto;
        __syncthreads();
        u64 before = upto - sum;
        for (int w = 0; w < warp; ++w) before += s.wsum[w];
        if (s.at >= before && s.at < before + sum) {
            u64 left = s.at - before;
            int found = -1;
            for (int g = g0; g < g1 && found < 0; ++g) {
                float pv[4], qv[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                load4(prow, 4 * g - mis, V, pv);
                if (useq) load4(qrow, 4 * g - mis, V, qv);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const u64 r = left_of(fix(pv[i]), fix(qv[i]), 4 * g - mis + i, s, drawn);
                    if (found < 0 && left < r) found = 4 * g - mis + i;
                    left -= found < 0 ? r : 0;
                }
            }
            a.token[b] = found;
        }
    }
    if (cluster > 1) cluster_barrier();  // no block leaves while another may read its sums
}

cudaError_t launch_verify(const VerifyArgs &a, cudaStream_t stream) {
    int *status = status_word();
    if (!status) return cudaErrorInvalidSymbol;
    // Blocks a request: 8 unless fewer give each at most 4096 elements.  Also with many requests: the
    // walks differ in length, and the longest one's passes are the faster the more SMs share them.
    int cluster = 1;
    while (cluster < kMaxVCluster && a.V > 4096 * cluster) cluster *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.B * cluster), 1, 1);
    cfg.blockDim = dim3(kVThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attrs[2];
    int na = 0;
    if (options().pdl) {
        attrs[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attrs[na].val.programmaticStreamSerializationAllowed = 1;
        ++na;
    }
    if (cluster > 1) {
        attrs[na].id = cudaLaunchAttributeClusterDimension;
        attrs[na].val.clusterDim.x = (unsigned)cluster;
        attrs[na].val.clusterDim.y = 1;
        attrs[na].val.clusterDim.z = 1;
        ++na;
    }
    cfg.attrs = attrs;
    cfg.numAttrs = na;
    return cudaLaunchKernelEx(&cfg, verify_kernel, a, cluster, status);
}

}  // namespace bsf8
