// bsf8_plan.cu -- the pages and slots of a step: pages of requests that are done go back to the free
// stack, the others get what their new tokens need, and each new token its request and slot.
//
// One cluster does it all: its blocks each take the same sums over the requests (a thread a request, two
// scans), so that nothing but the pages themselves goes from one to the other -- what the first half gives
// back the second may hand out, with the cluster's barrier between them -- and share the pages and tokens
// evenly.  Few requests, tokens and pages take one small block: what it costs is the chain of loads, scans and
// barriers.  (1024 requests, half of them leaving, 198000 tokens: 9.2 us in a graph, 13.7 with eight blocks, 30 with
// those of 512 threads, three scans and a search a token; seven requests of a few tokens 2.6.)
#include "bsf8_device.cuh"
#include "bsf8_internal.h"

#include <algorithm>

namespace bsf8 {

namespace {

constexpr int kPlanCluster = 16;  // 8 where the device does not schedule those

template <int NT>
struct PlanShared {
    // sums over the requests before each, and over all: pages that come back, pages handed out, tokens
    int back[NT + 1], need[NT + 1], start[NT + 1];
    int lens[NT], held[NT];  // held: after what comes back
    int wsum[2][3][NT / 32];
};

// The sums of K numbers over the threads before this one (v), and over all (all); one barrier.  The last number's sums
// stop at `most`, at most 2^30 + 1 (a sum that is cut off there is still one: in any order; two of them fit 32 bits without a
// sign).  `set`: slots in turn.
template <int NT, int K>
__device__ __forceinline__ void before_me(PlanShared<NT> &s, int set, int (&v)[K], int (&all)[K], int most) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto add = [&](int k, int a, int b) { return k == K - 1 ? (int)min((uint32_t)a + (uint32_t)b, (uint32_t)most) : a + b; };
    int up[K], w[K];
#pragma unroll
    for (int k = 0; k < K; ++k) up[k] = v[k];
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int o = __shfl_up_sync(0xFFFFFFFFu, up[k], m);
            if (lane >= m) up[k] = add(k, up[k], o);
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (lane == 31) s.wsum[set][k][warp] = up[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) w[k] = lane < NT / 32 ? s.wsum[set][k][lane] : 0;
#pragma unroll
    for (int m = 1; m < NT / 32; m <<= 1) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int o = __shfl_up_sync(0xFFFFFFFFu, w[k], m);
            if (lane >= m) w[k] = add(k, w[k], o);
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        all[k] = __shfl_sync(0xFFFFFFFFu, w[k], NT / 32 - 1);
        const int p = __shfl_sync(0xFFFFFFFFu, w[k], max(warp - 1, 0));
        const int o = __shfl_up_sync(0xFFFFFFFFu, up[k], 1);
        v[k] = add(k, lane > 0 ? o : 0, warp > 0 ? p : 0);
    }
}

// The request of item i: sum[b] <= i < sum[b + 1].
__device__ __forceinline__ int owner(const int *sum, int B, int i) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sum[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <int NT>
__global__ void __launch_bounds__(NT) plan_kernel(const PlanArgs a, int cluster, int *status) {
    __shared__ PlanShared<NT> s;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, rank = blockIdx.x, B = a.B;
    const int P = a.page_size;
    const long long capacity = (long long)a.table_pages * P;
    bool bad = false;
    int count = *a.count;
    // a thread's request
    int held = 0, len = 0, add = 0, back = 0, need = 0;
    if (tid < B) {
        held = a.held[tid], len = a.lens[tid], add = a.add[tid];
        const bool done = a.done && a.done[tid] != 0;
        if (held < 0 || held > a.table_pages) {
            bad = true;
            held = max(0, min(held, a.table_pages));
        }
        if (len < 0 || add < 0 || (long long)len + add > capacity) {
            bad = true;
            len = add = 0;
        }
        if (done) {
            back = held;
            held = 0;
        }
        if (add > 0) need = max(0, (len + add - 1) / P + 1 - held);
        s.lens[tid] = len;
        s.held[tid] = held;
    }
    if (count < 0 || count > a.pool) {
        bad = true;
        count = max(0, min(count, a.pool));
    }
    // pages that come back and pages asked for (each below 2^31 in all), and tokens asked for, as far as they count
    int v[3] = {back, need, min(add, a.N + 1)}, all[3];
    before_me(s, 0, v, all, a.N + 1);
    int returned = all[0];
    if (returned > a.pool - count) {
        bad = true;  // more than the stack can hold: the rest is lost
        returned = a.pool - count;
    }
    const int top = count + returned;
    if (tid < B) s.back[tid] = v[0];
    // what does not fit, pages or tokens, by a request and those before it, gets nothing
    if ((need > 0 && need > top - v[1]) || add > a.N - v[2]) need = add = 0;
    int at[2] = {need, add}, granted[2];
    before_me(s, 1, at, granted, a.N);
    if (tid < B) s.need[tid] = at[0], s.start[tid] = at[1];
    if (tid == 0) s.back[B] = all[0], s.need[B] = granted[0], s.start[B] = granted[1];
    if (bad && rank == 0) report_index(status);
    __syncthreads();

    const int threads = cluster * NT, me = rank * NT + tid;
    // the pages that come back, onto the stack, four a thread on their way
    for (int i0 = me; i0 < returned; i0 += 4 * threads) {
        int page[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + j * threads;
            if (i < returned) {
                const int b = owner(s.back, B, i);
                page[j] = a.table[(size_t)b * a.table_pages + (i - s.back[b])];
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i0 + j * threads < returned) a.free[count + i0 + j * threads] = page[j];
    }
    if (cluster > 1) cluster_arrive();
    // the tokens, four a thread one after another
    const int last = s.start[B];
    const bool aligned = ((reinterpret_cast<uintptr_t>(a.req) | reinterpret_cast<uintptr_t>(a.slot)) & 15) == 0;
    for (long long r0 = 4LL * me; r0 < a.N; r0 += 4LL * threads) {
        const int i0 = (int)r0;
        int req[4], slot[4], b = i0 < last ? owner(s.start, B, i0) : 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + j;
            req[j] = 0, slot[j] = -1;
            if (i < last) {
                while (s.start[b + 1] <= i) ++b;
                req[j] = b;
                slot[j] = s.lens[b] + (i - s.start[b]);
            }
        }
        if (aligned && i0 + 4 <= a.N) {
            *reinterpret_cast<int4 *>(a.req + i0) = make_int4(req[0], req[1], req[2], req[3]);
            *reinterpret_cast<int4 *>(a.slot + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i0 + j < a.N) a.req[i0 + j] = req[j], a.slot[i0 + j] = slot[j];
        }
    }
    // (every block has read the books by then, and its pages are back)
    if (cluster > 1) cluster_wait();
    else __syncthreads();
    // the pages handed out, from its top
    const int used = s.need[B];
    for (int i0 = me; i0 < used; i0 += 4 * threads) {
        int page[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i0 + j * threads < used) page[j] = __ldcg(a.free + (top - 1 - (i0 + j * threads)));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + j * threads;
            if (i < used) {
                const int b = owner(s.need, B, i);
                a.table[(size_t)b * a.table_pages + s.held[b] + (i - s.need[b])] = page[j];
            }
        }
    }
    if (rank == 0) {
        if (tid < B) {
            a.start[tid] = s.start[tid];
            a.granted[tid] = add;
            a.held[tid] = held + need;
        }
        if (tid == 0) {
            a.start[B] = last;
            *a.count = top - used;
        }
    }
}

template <int NT>
cudaError_t plan_threads(const PlanArgs &a, int cluster, cudaStream_t stream, int *status) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)cluster, 1, 1);
    cfg.blockDim = dim3(NT, 1, 1);
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
    return cudaLaunchKernelEx(&cfg, plan_kernel<NT>, a, cluster, status);
}

}  // namespace

cudaError_t launch_plan(const PlanArgs &a, cudaStream_t stream) {
    int *status = status_word();
    if (!status) return cudaErrorInvalidSymbol;
    // One block where tokens are few, and pages that may come back (those handed out are no more than tokens and requests).
    // One block / the cluster: 64 requests, 576 tokens 3.7 us / 4.9; 128, 1152 tokens 4.7 / 5.05; 64, 4096 tokens 5.95 / 5.0.
    // 64 requests of one token, tables of 64 pages, none leaves 2.7 / 4.1, one 3.9 / 4.9, all 14.7 / 5.2; of 512 pages 3.0 /
    // 3.8, 4.4 / 4.9, 88 / 5.9; of 2048 2.3 / 3.6, 8.4 / 5.4, 340 / 8.5: how many leave only the device knows.
    if (a.B <= 128 && a.N <= 1536 && (!a.done || (long long)a.B * a.table_pages <= 4096)) return plan_threads<128>(a, 1, stream, status);
    // clusters of 16 blocks: asked for once per device
    static int known[64] = {0};  // 0 unknown, else the cluster
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int cluster = __atomic_load_n(&known[dev], __ATOMIC_ACQUIRE);
    if (cluster == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kPlanCluster, 1, 1);
        cfg.blockDim = dim3(1024, 1, 1);
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = kPlanCluster;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int n = 0;
        const bool fits = cudaFuncSetAttribute(plan_kernel<1024>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                          cudaOccupancyMaxActiveClusters(&n, plan_kernel<1024>, &cfg) == cudaSuccess && n > 0;
        if (!fits) (void)cudaGetLastError();
        cluster = fits ? kPlanCluster : kPlanCluster / 2;
        __atomic_store_n(&known[dev], cluster, __ATOMIC_RELEASE);
    }
    return plan_threads<1024>(a, cluster, stream, status);
}

}  // namespace bsf8
