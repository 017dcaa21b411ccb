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
// node's token at its parent -- is loaded up front by one thread a node; thread 0 of every
// block then walks the tree in shared memory (the same steps in each), and the vocabulary is
// read only where a sum of R is needed: once a rejection, and for the last draw unless the
// last step was a rejection (its sum is the draw's).  A pass gives each block a contiguous
// slice of the row and each warp a contiguous part of it, so the draw's element is found by
// adding up slices, then warps, then one warp's part, which its block reads again (from L2).
// HBM bound at large batches (one row of p and q a request), latency bound at small ones.
#include "bsf8_device.cuh"
#include "bsf8_internal.h"

#include <algorithm>

namespace bsf8 {

namespace {

constexpr int kVThreads = 512;
constexpr int kVWarps = kVThreads / 32;
constexpr int kNodes = 256;        // BSF8_MAX_NODES
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
    u64 Z[kNodes];             // the mass before each rejection at the walk's node
    int gone[kNodes];          // the token of each rejection there
    u64 wsum[kVWarps];         // a pass: each warp's sum of R
    u64 bsum[2];               // this block's, read by the cluster (slots taken in turn)
    u64 rsum[kMaxVCluster];    // every block's
    u64 total;                 // the mass Z of R
    int cur, rej, next, count; // the walk's node, rejections there, next child, nodes kept
    int done, summed;          // no child is left to ask; the sums are those of the present R
    int small;                 // every Z here is below 2^42
    int stop;                  // both: the draw is next
    u64 at;                    // the draw's threshold inside a warp's part
    int warp;                  // that warp, or -1
};

// floor(q z / 2^40) for q <= 2^40 and z < 2^42, from parts of 20 bits.
__device__ __forceinline__ u64 times20(u64 q, uint32_t zh, uint32_t zl) {
    const uint32_t qh = (uint32_t)(q >> 20), ql = (uint32_t)q & 0xFFFFFu;
    return (u64)qh * zh + (((u64)qh * zl + (u64)ql * zh + (((u64)ql * zl) >> 20)) >> 20);
}

// R of element x, whose fixed-point probabilities at the walk's node are P and Q.
__device__ __forceinline__ u64 left_of(u64 P, u64 Q, int x, const VerifyShared &s, bool drawn) {
    if (drawn) {
        u64 off = s.rej > 0 ? Q : 0;  // the first rejection's mass is 2^40
        for (int j = 1; j < s.rej; ++j)
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

// The walk from where it stands until a rejection (whose sum of R is wanted) or the last child.
__device__ __forceinline__ void walk(VerifyShared &s, int n, bool drawn) {
    int i = s.next;
    s.done = 1;
    for (; i < n && s.done; ++i) {
        if (s.parent[i] != s.cur) continue;
        const u64 z = s.total;
        const u64 q = times(s.Q[i], z);
        if (part(s.U[i], q) < left_of(s.P[i], s.Q[i], s.tok[i], s, drawn)) {  // kept
            s.cur = i;
            s.path[s.count++] = i;
            s.rej = 0;
            s.small = 1;
            s.total = kOne;
        } else {
            s.Z[s.rej] = z;
            if (z >= 1ull << 42) s.small = 0;
            s.gone[s.rej] = s.tok[i];
            ++s.rej;
            s.done = 0;
        }
        s.summed = 0;
    }
    s.next = i;
}

// The next thing after a sum (or the start), by thread 0: on along the walk, or, when R was all 0
// after the last child, a sum of P instead.
__device__ __forceinline__ void step(VerifyShared &s, int n, bool drawn) {
    if (s.done) s.rej = 0;
    else walk(s, n, drawn);
    s.stop = s.done && s.summed;
}

// Cluster barrier whose lanes need not arrive together.
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__global__ void __launch_bounds__(kVThreads) verify_kernel(const VerifyArgs a, int cluster, int *status) {
    __shared__ VerifyShared s;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = blockIdx.x / cluster, rank = blockIdx.x % cluster;
    const int T = a.T, V = a.V;
    int n = a.nodes ? a.nodes[b] : T;
    if (n < 1 || n > T) {
        if (tid == 0) report_index(status);
        n = max(1, min(n, T));
    }
    const bool drawn = a.q != nullptr;
    const float *const pb = a.p + (size_t)b * T * a.ld;
    const float *const qb = drawn ? a.q + (size_t)b * T * a.ld : nullptr;
    for (int i = tid; i < n; i += kVThreads) {
        s.U[i] = (uint32_t)(fminf(fmaxf(a.u[(size_t)b * T + i], 0.0f), 0.99999994f) * 16777216.0f);
        int par = -1, x = 0;
        u64 P = 0, Q = 0;
        if (i > 0) {
            par = a.parent[(size_t)b * T + i];
            x = a.tokens[(size_t)b * T + i];
            if ((unsigned)par >= (unsigned)i || (unsigned)x >= (unsigned)V) {
                report_index(status);
                par = -1;
            } else {
                P = fix(pb[(size_t)par * a.ld + x]);
                Q = drawn ? fix(qb[(size_t)par * a.ld + x]) : kOne;
            }
        }
        s.parent[i] = par;
        s.tok[i] = x;
        s.P[i] = P;
        s.Q[i] = Q;
    }
    if (tid == 0) {
        s.cur = s.rej = s.summed = s.done = 0;
        s.small = 1;
        s.next = s.count = 1;
        s.path[0] = 0;
        s.total = kOne;
    }
    __syncthreads();
    if (tid == 0) step(s, n, drawn);
    __syncthreads();

    int per_warp = 0, mis = 0, groups = 0;  // of the last pass's row
    // Thread 0 changes the walk's state only between the last two barriers of a turn, so that every
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
        auto add = [&](const float (&pv)[4], const float (&qv)[4], int x) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const u64 P = fix(pv[i]);
                if (rej == 0) {
                    sum += P;
                } else if (rej == 1 && drawn) {
                    const u64 Q = fix(qv[i]);
                    sum += P > Q ? P - Q : 0;
                } else {
                    sum += left_of(P, drawn ? fix(qv[i]) : 0, x + i, s, drawn);
                }
            }
        };
        // whole groups of four, kBatch loads of each row in flight; then the ragged ones
        const int gi = max(g0, mis > 0 ? 1 : 0), ge = min(g1, (V + mis) / 4);
        int g = gi + lane;
        for (; g + 32 * (kBatch - 1) < ge; g += 32 * kBatch) {
            float4 pf[kBatch], qf[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) pf[j] = *reinterpret_cast<const float4 *>(prow + 4 * (g + 32 * j) - mis);
            if (useq)
#pragma unroll
                for (int j = 0; j < kBatch; ++j) qf[j] = *reinterpret_cast<const float4 *>(qrow + 4 * (g + 32 * j) - mis);
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const float pv[4] = {pf[j].x, pf[j].y, pf[j].z, pf[j].w};
                const float qv[4] = {qf[j].x, qf[j].y, qf[j].z, qf[j].w};
                add(pv, qv, 4 * (g + 32 * j) - mis);
            }
        }
        for (; g < g1; g += 32) {
            float pv[4], qv[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            load4(prow, 4 * g - mis, V, pv);
            if (useq) load4(qrow, 4 * g - mis, V, qv);
            add(pv, qv, 4 * g - mis);
        }
        if (gi > g0 && g0 == 0 && g1 > 0 && lane == 0) {  // the row's first, partial group
            float pv[4], qv[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            load4(prow, -mis, V, pv);
            if (useq) load4(qrow, -mis, V, qv);
            add(pv, qv, -mis);
        }
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
        if (cluster > 1) {
            cluster_barrier();
            if (tid < cluster) s.rsum[tid] = ld_cluster_u64(map_to_rank(&s.bsum[pass & 1], tid));
        }
        __syncthreads();
        if (tid == 0) {
            u64 t = 0;
            for (int r = 0; r < cluster; ++r) t += s.rsum[r];
            s.total = t;
            s.summed = t > 0 || s.rej == 0;  // nothing left after rejections: once more, from P
            s.stop = s.done && s.summed;
            if (!s.stop) step(s, n, drawn);
        }
        __syncthreads();
    }

    // ------------------------------------------------------------------ the draw
    if (tid == 0) {
        const u64 thr = part(s.U[0], s.total);
        u64 before = 0;
        for (int r = 0; r < rank; ++r) before += s.rsum[r];
        s.warp = -1;
        for (int w = 0; w < kVWarps; ++w) {
            if (thr >= before && thr < before + s.wsum[w]) {
                s.warp = w;
                s.at = thr - before;
            }
            before += s.wsum[w];
        }
        if (s.total == 0 && rank == 0) a.token[b] = V - 1;
    }
    if (rank == 0) {
        for (int i = tid; i < T; i += kVThreads) a.path[(size_t)b * T + i] = i < s.count ? s.path[i] : -1;
        if (tid == 0) a.count[b] = s.count;
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
        __syncthreads();  // s.wsum is read above by thread 0 only, before its barrier
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
