// bsf8_sample.cu -- a token, or the whole processed distribution, from rows of logits: temperature,
// top-k, min-p, top-p, and a draw by a number that the caller gives.
//
// Each logit has a weight in whole numbers (bsf8.h states it), w = floor(2^40 2^-y), y = (max - x)
// log2(e) / t, and every sum is of these: which tokens stay and which one is drawn depends on no order of
// threads and on no split of the row.
//
// A cluster of blocks a row; a block takes a contiguous slice of it, a warp a contiguous part of that.
// The order that top-k and top-p go by (larger logits first, then the lower index) is that of the bits of
// d = max - x >= 0, whose digits a histogram at a time narrows down: counts for top-k, weights for top-p.
#include "bsf8_device.cuh"
#include "bsf8_internal.h"

#include <algorithm>

namespace bsf8 {

namespace {

typedef unsigned long long u64;
constexpr int kTThreads = 512, kTWarps = kTThreads / 32;
constexpr int kMaxTCluster = 8;
constexpr u64 kWhole = 1ull << 40;
constexpr int kBins = 1024;
constexpr uint32_t kInfBits = 0x7F800000u;
static_assert(kBins == 2 * kTThreads, "two bins a thread");

struct TokenShared {
    float wmax[kTWarps], bmax;      // bmax, bsum, bmin: read by the cluster
    int wmin[kTWarps], bmin;
    u64 wsum[kTWarps], bsum;
    int wcount[kTWarps], bcount;
    uint32_t count[kBins];          // a histogram: elements, their weights' low 12 bits and the rest
    uint32_t low[kBins];
    u64 high[kBins];
    u64 tsum[kTWarps];
    int tcount[kTWarps];
    int bin;                        // the bin in which the wanted rank or weight lies,
    int before;                     // and what is before it
    u64 mass;
    u64 at;                         // the draw, inside a warp's part
    int warp;
    int cut;
};

// 2^-f on [0, 1): a polynomial fitted to it (least squares, weighted towards the largest relative error,
// 2^-22), every step rounded by itself so that any machine gets the same bits.
__device__ __forceinline__ float exp2_of(float f) {
    float p = -0.0009449035860598087f;
    p = __fadd_rn(__fmul_rn(p, f), 0.00920579768717289f);
    p = __fadd_rn(__fmul_rn(p, f), -0.0552973598241806f);
    p = __fadd_rn(__fmul_rn(p, f), 0.2401801496744156f);
    p = __fadd_rn(__fmul_rn(p, f), -0.6931437253952026f);
    return __fadd_rn(__fmul_rn(p, f), 1.0f);
}

// The weight at distance d = max - x >= 0; `rate` is log2(e) / t, infinite for the largest alone.
__device__ __forceinline__ u64 weight(float d, float rate) {
    const float y = d == 0.0f ? 0.0f : __fmul_rn(d, rate);
    if (!(y <= 40.0f)) return 0;
    const float n = floorf(y);
    const uint32_t m = (uint32_t)(exp2_of(__fsub_rn(y, n)) * 16777216.0f);  // 2^23 .. 2^24
    return ((u64)m << 16) >> (int)n;
}

__device__ __forceinline__ u64 part_of(u64 u, u64 z) {  // floor(u z / 2^24)
    return (__umul64hi(u, z) << 40) | ((u * z) >> 24);
}

__device__ __forceinline__ u64 ld_cluster64(uint32_t addr) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t ld_cluster32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

template <typename T>
struct Logit;
template <>
struct Logit<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(const uint4 &w, float (&y)[4]) {
        y[0] = __uint_as_float(w.x), y[1] = __uint_as_float(w.y), y[2] = __uint_as_float(w.z), y[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ float one(const float *p) { return *p; }
};
template <>
struct Logit<uint16_t> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(const uint4 &w, float (&y)[8]) {
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[2 * i] = __uint_as_float(a[i] << 16);
            y[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ float one(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }
};

}  // namespace

template <typename T, bool PROBS>
__global__ void __launch_bounds__(kTThreads) sample_kernel(const SampleArgs a, int cluster) {
    __shared__ TokenShared s;
    pdl_trigger();
    pdl_wait();
    using L = Logit<T>;
    constexpr int VEC = L::N;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = blockIdx.x / cluster, rank = blockIdx.x % cluster, V = a.V;
    const T *const x = static_cast<const T *>(a.logits) + (size_t)row * a.ld;
    // groups of VEC elements that start on 16 bytes; the first and last may be partly outside the row
    const int mis = (int)(((size_t)row * a.ld) % VEC), groups = (V + mis + VEC - 1) / VEC;
    const int per_warp = ((groups + cluster * kTWarps - 1) / (cluster * kTWarps) + 31) / 32 * 32;
    const int g0 = min(groups, (rank * kTWarps + warp) * per_warp), g1 = min(groups, g0 + per_warp);
    const float tp = a.temperature ? a.temperature[row] : 1.0f;
    const bool greedy = !(tp > 0.0f);
    const float rate = greedy ? INFINITY : __fdiv_rn(1.4426950408889634f, tp);
    int k = a.top_k ? a.top_k[row] : 0;
    if (k <= 0 || k > V) k = V;
    if (greedy) k = 1;
    const float mp = a.min_p ? fminf(fmaxf(a.min_p[row], 0.0f), 1.0f) : 0.0f;
    const u64 least = max((u64)1, (u64)ceilf(mp * 1099511627776.0f));
    const float pp = a.top_p ? a.top_p[row] : 1.0f;
    const bool nucleus = pp < 1.0f;
    const u64 pfix = nucleus ? (u64)(fmaxf(pp, 0.0f) * 16777216.0f) : 0;

    // elements of group g: outside the row, and NaN, as -inf
    auto load = [&](int g, float (&y)[VEC]) {
        const int e = g * VEC - mis;
        if (e >= 0 && e + VEC <= V) {
            L::unpack(*reinterpret_cast<const uint4 *>(x + e), y);
#pragma unroll
            for (int i = 0; i < VEC; ++i) y[i] = fmaxf(y[i], -INFINITY);  // NaN becomes -inf
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                y[i] = (unsigned)(e + i) < (unsigned)V ? fmaxf(L::one(x + e + i), -INFINITY) : -INFINITY;
        }
    };
    auto barrier = [&]() {
        if (cluster > 1) cluster_barrier();
        else __syncthreads();
    };

    // ---------------------------------------------------------------- the largest
    float top = -INFINITY;
    for (int g = g0 + lane; g < g1; g += 32) {
        float y[VEC];
        load(g, y);
#pragma unroll
        for (int i = 0; i < VEC; ++i) top = fmaxf(top, y[i]);
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
    if (lane == 0) s.wmax[warp] = top;
    __syncthreads();
    if (tid == 0) {
        float v = -INFINITY;
        for (int w = 0; w < kTWarps; ++w) v = fmaxf(v, s.wmax[w]);
        s.bmax = v;
    }
    barrier();
    top = -INFINITY;
    for (int c = 0; c < cluster; ++c)
        top = fmaxf(top, cluster > 1 ? __uint_as_float(ld_cluster32(map_to_rank(&s.bmax, c))) : s.bmax);

    const bool none = top == -INFINITY;
    // the distance of an element, as bits that order as it does; infinite where it has no part
    auto distance = [&](float v) { return v == top ? (none ? INFINITY : 0.0f) : __fsub_rn(top, v); };

    // What stays: elements below `cut` in the order of (bits of d, index), with weight `least` at least.
    uint32_t cut_bits = kInfBits;    // those below it,
    int cut_index = -1;              // and of those that equal it the ones up to this index

    // Narrows the cut down to the element in which the running count (or weight) reaches `want`: of those inside
    // the present cut.  Returns how many stay of those that equal the new cut's bits.
    auto narrow = [&](bool by_weight, u64 want_in, bool fraction) {
        const uint32_t limit = cut_bits;
        const int limit_index = cut_index;
        uint32_t base = 0, most = kInfBits;
        u64 want = want_in;
        int level = 0, shift = 18;
        while (true) {
            for (int i = tid; i < kBins; i += kTThreads) s.count[i] = s.low[i] = 0, s.high[i] = 0;
            __syncthreads();
            for (int g = g0 + lane; g < g1; g += 32) {
                float y[VEC];
                load(g, y);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float d = distance(y[i]);
                    const uint32_t bits = __float_as_uint(d);
                    if (bits - base > most || bits >= kInfBits) continue;
                    if (bits > limit || (bits == limit && g * VEC - mis + i > limit_index)) continue;
                    int bin;
                    if (level == 0) {  // 16 octaves of 32 bins, what is below and above them in one each
                        const int b = (int)(bits >> 18) - (119 << 5);
                        bin = b < 0 ? 0 : min(b + 1, 513);
                    } else {
                        bin = (int)((bits - base) >> shift);
                    }
                    if (by_weight) {
                        const u64 w = weight(d, rate);
                        if (w < least) continue;
                        atomicAdd(&s.low[bin], (uint32_t)w & 0xFFFu);
                        atomicAdd(reinterpret_cast<unsigned long long *>(&s.high[bin]), (unsigned long long)(w >> 12));
                    }
                    atomicAdd(&s.count[bin], 1u);
                }
            }
            barrier();
            // the cluster's histogram, two bins a thread, and the sums before each
            u64 w2[2] = {0, 0};
            int c2[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int bin = 2 * tid + j;
                for (int c = 0; c < cluster; ++c) {
                    if (cluster > 1) {
                        c2[j] += (int)ld_cluster32(map_to_rank(&s.count[bin], c));
                        if (by_weight)
                            w2[j] += (u64)ld_cluster32(map_to_rank(&s.low[bin], c)) + (ld_cluster64(map_to_rank(&s.high[bin], c)) << 12);
                    } else {
                        c2[j] += (int)s.count[bin];
                        if (by_weight) w2[j] += (u64)s.low[bin] + (s.high[bin] << 12);
                    }
                }
            }
            u64 upw = w2[0] + w2[1];
            int upc = c2[0] + c2[1];
            const u64 myw = upw;
            const int myc = upc;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const u64 ow = __shfl_up_sync(0xFFFFFFFFu, upw, m);
                const int oc = __shfl_up_sync(0xFFFFFFFFu, upc, m);
                if (lane >= m) upw += ow, upc += oc;
            }
            if (lane == 31) s.tsum[warp] = upw, s.tcount[warp] = upc;
            if (tid == 0) s.bin = -1;
            __syncthreads();
            u64 all = 0;
            upw -= myw;
            upc -= myc;
            for (int w = 0; w < kTWarps; ++w) {
                if (w < warp) upw += s.tsum[w], upc += s.tcount[w];
                all += by_weight ? s.tsum[w] : (u64)s.tcount[w];
            }
            if (level == 0 && fraction) want = max((u64)1, part_of(want, all));
            // the bin in which the running sum reaches it
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const u64 before = by_weight ? upw : (u64)upc, mine = by_weight ? w2[j] : (u64)c2[j];
                if (before < want && before + mine >= want) {
                    s.bin = 2 * tid + j;
                    s.mass = before;
                    s.before = upc;
                }
                upw += w2[j];
                upc += c2[j];
            }
            barrier();
            const int bin = s.bin;
            if (bin < 0) return;  // less than that in all: everything stays
            want -= s.mass;
            if (level == 0) {
                if (bin == 0) {
                    most = (119u << 23) - 1;
                    shift = 20;
                } else if (bin == 513) {
                    base = (uint32_t)(119 * 32 + 512) << 18;
                    most = kInfBits - base;
                    shift = 20;
                } else {
                    base = (uint32_t)(119 * 32 + bin - 1) << 18;
                    most = (1u << 18) - 1;
                    shift = 8;
                }
            } else {
                base += (uint32_t)bin << shift;
                if (shift == 0) break;
                most = (1u << shift) - 1;
                shift = shift == 20 ? 10 : 0;
            }
            ++level;
        }
        // elements of these bits have one weight: as many of them, by index, as it takes
        const u64 each = by_weight ? weight(__uint_as_float(base), rate) : 1;
        const u64 keep = (want + each - 1) / each;
        // the index of the keep-th of them
        int mine = 0;
        for (int g = g0 + lane; g < g1; g += 32) {
            float y[VEC];
            load(g, y);
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                mine += __float_as_uint(distance(y[i])) == base && (base != limit || g * VEC - mis + i <= limit_index) ? 1 : 0;
        }
        mine = __reduce_add_sync(0xFFFFFFFFu, mine);
        if (lane == 0) s.wcount[warp] = mine;
        __syncthreads();
        if (tid == 0) {
            int v = 0;
            for (int w = 0; w < kTWarps; ++w) v += s.wcount[w];
            s.bcount = v;
            s.cut = -1;
        }
        barrier();
        u64 before = 0;
        for (int c = 0; c < rank; ++c) before += ld_cluster32(map_to_rank(&s.bcount, c));
        for (int w = 0; w < warp; ++w) before += s.wcount[w];
        if (before < keep && before + mine >= keep) {  // this warp's part has it
            for (int gb = g0; gb < g1; gb += 32) {
                const int g = gb + lane;
                float y[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) y[i] = -INFINITY;
                if (g < g1) load(g, y);
                int n = 0;
                bool is[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    is[i] = __float_as_uint(distance(y[i])) == base && (base != limit || g * VEC - mis + i <= limit_index);
                    n += is[i] ? 1 : 0;
                }
                int upto = n;
#pragma unroll
                for (int m = 1; m < 32; m <<= 1) {
                    const int o = __shfl_up_sync(0xFFFFFFFFu, upto, m);
                    if (lane >= m) upto += o;
                }
                u64 r = before + upto - n;
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (is[i] && ++r == keep) s.cut = g * VEC - mis + i;
                before += __shfl_sync(0xFFFFFFFFu, upto, 31);
                if (before >= keep) break;
            }
        }
        barrier();
        int found = -1;
        for (int c = 0; c < cluster; ++c) found = max(found, cluster > 1 ? (int)ld_cluster32(map_to_rank(&s.cut, c)) : s.cut);
        cut_bits = base;
        cut_index = found;
        barrier();  // s.cut is written again
    };

    if (!none) {
        if (k < V) narrow(false, (u64)k, false);
        if (nucleus && !greedy) narrow(true, pfix, true);
    }

    // ---------------------------------------------------------------- what stays, in order of index
    auto kept = [&](float v, int index) -> u64 {
        const float d = distance(v);
        const uint32_t bits = __float_as_uint(d);
        if (bits >= kInfBits || bits > cut_bits || (bits == cut_bits && index > cut_index)) return 0;
        const u64 w = weight(d, rate);
        return w >= least ? w : 0;
    };
    u64 sum = 0;
    for (int g = g0 + lane; g < g1; g += 32) {
        float y[VEC];
        load(g, y);
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum += kept(y[i], g * VEC - mis + i);
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, m);
    if (lane == 0) s.wsum[warp] = sum;
    __syncthreads();
    if (tid == 0) {
        u64 v = 0;
        for (int w = 0; w < kTWarps; ++w) v += s.wsum[w];
        s.bsum = v;
    }
    barrier();
    u64 total = 0, first = 0;
    for (int c = 0; c < cluster; ++c) {
        const u64 v = cluster > 1 ? ld_cluster64(map_to_rank(&s.bsum, c)) : s.bsum;
        if (c < rank) first += v;
        total += v;
    }
    const float inv = total ? 1.0f / (float)total : 0.0f;
    auto share = [&](u64 w) { return fmaf((float)(uint32_t)(w >> 20), 1048576.0f, (float)(uint32_t)(w & 0xFFFFFu)) * inv; };

    if constexpr (PROBS) {
        float *const out = a.p + (size_t)row * V;
        for (int g = g0 + lane; g < g1; g += 32) {
            float y[VEC];
            load(g, y);
            const int e = g * VEC - mis;
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if ((unsigned)(e + i) < (unsigned)V) out[e + i] = share(kept(y[i], e + i));
        }
    } else {
        if (total == 0) {
            if (rank == 0 && tid == 0) {
                a.token[row] = -1;
                a.p[row] = 0.0f;
            }
        } else {
            const float u = a.u[row];
            const u64 at = part_of((u64)(fminf(fmaxf(u, 0.0f), 0.99999994f) * 16777216.0f), total);
            u64 before = first;
            for (int w = 0; w < warp; ++w) before += s.wsum[w];
            if (at >= before && at < before + sum) {  // this warp's part has it
                for (int gb = g0; gb < g1; gb += 32) {
                    const int g = gb + lane;
                    float y[VEC];
#pragma unroll
                    for (int i = 0; i < VEC; ++i) y[i] = -INFINITY;
                    if (g < g1) load(g, y);
                    u64 w[VEC], mine = 0;
#pragma unroll
                    for (int i = 0; i < VEC; ++i) mine += w[i] = kept(y[i], g * VEC - mis + i);
                    u64 upto = mine;
#pragma unroll
                    for (int m = 1; m < 32; m <<= 1) {
                        const u64 o = __shfl_up_sync(0xFFFFFFFFu, upto, m);
                        if (lane >= m) upto += o;
                    }
                    u64 r = before + upto - mine;
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        if (at >= r && at < r + w[i]) {
                            a.token[row] = g * VEC - mis + i;
                            a.p[row] = share(w[i]);
                        }
                        r += w[i];
                    }
                    before += __shfl_sync(0xFFFFFFFFu, upto, 31);
                    if (before > at) break;
                }
            }
        }
    }
    if (cluster > 1) cluster_barrier();  // no block leaves while another may read its sums
}

template <typename T, bool PROBS>
cudaError_t sample_typed(const SampleArgs &a, cudaStream_t stream) {
    int cluster = 1;
    while (cluster < kMaxTCluster && a.V > 4096 * cluster) cluster *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.N * cluster), 1, 1);
    cfg.blockDim = dim3(kTThreads, 1, 1);
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
    return cudaLaunchKernelEx(&cfg, sample_kernel<T, PROBS>, a, cluster);
}

cudaError_t launch_sample(const SampleArgs &a, bool probs, cudaStream_t stream) {
    if (a.bf16) return probs ? sample_typed<uint16_t, true>(a, stream) : sample_typed<uint16_t, false>(a, stream);
    return probs ? sample_typed<float, true>(a, stream) : sample_typed<float, false>(a, stream);
}

}  // namespace bsf8
