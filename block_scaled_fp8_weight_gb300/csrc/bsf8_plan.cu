// bsf8_plan.cu -- the pages and slots of a step: pages of requests that are done go back to the free
// stack, the others get what their new tokens need, and each new token its request and slot.
//
// One cluster does it all: its blocks each take the same sums over the requests (at most 1024, two
// integers a request), so that nothing but the pages themselves goes from one to the other -- what the
// first half gives back the second may hand out, with the cluster's barrier between them -- and share
// the pages and tokens evenly.  Bound by latency: the requests' words, three sums over a block, the
// barrier, a page, its entry.
#include "bsf8_device.cuh"
#include "bsf8_internal.h"

#include <algorithm>

namespace bsf8 {

namespace {

constexpr int kPThreads = 512, kPWarps = kPThreads / 32, kPer = 2;  // 1024 requests
constexpr int kMaxRequests = kPThreads * kPer;
constexpr int kPlanCluster = 8;

struct PlanShared {
    // sums over the requests before each, and over all: pages that come back, pages handed out, tokens
    int back[kMaxRequests + 1], need[kMaxRequests + 1], start[kMaxRequests + 1];
    int lens[kMaxRequests], held[kMaxRequests];  // held: after what comes back
    long long wsum[2][kPWarps];
};

// The sums over the threads before this one, and over all in `total`; barriers inside.
__device__ __forceinline__ long long before_me(long long v, long long *wsum, long long &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long up = v;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const long long o = __shfl_up_sync(0xFFFFFFFFu, up, m);
        if (lane >= m) up += o;
    }
    if (lane == 31) wsum[warp] = up;
    __syncthreads();
    long long before = up - v;
    total = 0;
#pragma unroll
    for (int w = 0; w < kPWarps; ++w) {
        if (w < warp) before += wsum[w];
        total += wsum[w];
    }
    return before;
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

__global__ void __launch_bounds__(kPThreads) plan_kernel(const PlanArgs a, int cluster, int *status) {
    __shared__ PlanShared s;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, rank = blockIdx.x;
    const int P = a.page_size;
    const long long capacity = (long long)a.table_pages * P;
    bool bad = false;
    int count = *a.count;
    if (count < 0 || count > a.pool) {
        bad = true;
        count = max(0, min(count, a.pool));
    }
    // a thread's requests
    long long back = 0, need = 0, ask = 0;
    int nb[kPer], nn[kPer], na[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int b = tid * kPer + j;
        nb[j] = nn[j] = na[j] = 0;
        if (b < a.B) {
            int held = a.held[b], len = a.lens[b], add = a.add[b];
            const bool done = a.done && a.done[b] != 0;
            if (held < 0 || held > a.table_pages) {
                bad = true;
                held = max(0, min(held, a.table_pages));
            }
            if (len < 0 || add < 0 || (long long)len + add > capacity) {
                bad = true;
                len = add = 0;
            }
            if (done) {
                nb[j] = held;
                held = 0;
            }
            if (add > 0) nn[j] = max(0, (len + add - 1) / P + 1 - held);
            na[j] = add;
            s.lens[b] = len;
            s.held[b] = held;
        }
        back += nb[j];
        need += nn[j];
        ask += na[j];
    }
    long long total, tokens;
    long long back0 = before_me(back, s.wsum[0], total);  // at most B table_pages: fits 31 bits
    if (count + total > a.pool) {
        bad = true;  // more than the stack can hold: the rest is lost
        total = a.pool - count;
    }
    const int top = count + (int)total;
    // pages and tokens asked for by a request and those before it: what does not fit gets nothing
    const long long need0 = before_me(need, s.wsum[1], total);
    __syncthreads();
    const long long ask0 = before_me(ask, s.wsum[0], tokens);
    need = ask = 0;
    long long upn = need0, upa = ask0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int b = tid * kPer + j;
        upn += nn[j];
        upa += na[j];
        if ((nn[j] > 0 && upn > top) || upa > a.N) nn[j] = na[j] = 0;
        need += nn[j];
        ask += na[j];
        if (b < a.B) s.back[b] = (int)back0;
        back0 += nb[j];
    }
    __syncthreads();
    // both sums of what is granted, in one: pages and tokens are below 2^31
    long long both;
    long long at = before_me(need << 32 | ask, s.wsum[1], both);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int b = tid * kPer + j;
        if (b < a.B) {
            s.need[b] = (int)(at >> 32);
            s.start[b] = (int)(at & 0x7FFFFFFF);
        }
        at += (long long)nn[j] << 32 | na[j];
    }
    if (tid * kPer < a.B && (tid + 1) * kPer >= a.B) s.back[a.B] = (int)back0;  // the last request's thread
    if (tid == 0) {
        s.need[a.B] = (int)(both >> 32);
        s.start[a.B] = (int)(both & 0x7FFFFFFF);
    }
    if (bad && rank == 0) report_index(status);
    __syncthreads();

    // the pages that come back, onto the stack
    const int threads = cluster * kPThreads, me = rank * kPThreads + tid;
    for (int i = me; i < top - count; i += threads) {
        const int b = owner(s.back, a.B, i);
        a.free[count + i] = a.table[(size_t)b * a.table_pages + (i - s.back[b])];
    }
    // (every block has read the books by then)
    if (cluster > 1) cluster_barrier();
    else __syncthreads();
    // the pages handed out, from its top
    const int used = s.need[a.B];
    for (int i = me; i < used; i += threads) {
        const int b = owner(s.need, a.B, i);
        a.table[(size_t)b * a.table_pages + s.held[b] + (i - s.need[b])] = __ldcg(a.free + (top - 1 - i));
    }
    const int last = s.start[a.B];
    for (int i = me; i < a.N; i += threads) {
        int b = 0, slot = -1;
        if (i < last) {
            b = owner(s.start, a.B, i);
            slot = s.lens[b] + (i - s.start[b]);
        }
        a.req[i] = b;
        a.slot[i] = slot;
    }
    if (rank == 0) {
        for (int b = tid; b <= a.B; b += kPThreads) {
            a.start[b] = s.start[b];
            if (b < a.B) {
                a.granted[b] = s.start[b + 1] - s.start[b];
                a.held[b] = s.held[b] + s.need[b + 1] - s.need[b];
            }
        }
        if (tid == 0) *a.count = top - used;
    }
}

}  // namespace

cudaError_t launch_plan(const PlanArgs &a, cudaStream_t stream) {
    int *status = status_word();
    if (!status) return cudaErrorInvalidSymbol;
    const int cluster = a.B > 64 || a.N > 2048 ? kPlanCluster : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)cluster, 1, 1);
    cfg.blockDim = dim3(kPThreads, 1, 1);
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
    return cudaLaunchKernelEx(&cfg, plan_kernel, a, cluster, status);
}

}  // namespace bsf8
