// bsf8_sample.cu -- a token, or the whole processed distribution, from rows of logits: temperature,
// top-k, min-p, top-p, and a draw by a number that the caller gives.
//
// Each logit has a weight in whole numbers (bsf8.h states it), w = floor(2^40 2^-y), y = (max - x)
// log2(e) / t, and every sum is of these: which tokens stay and which one is drawn depends on no order of
// threads and on no split of the row.
//
// A cluster of blocks a row; a block takes a contiguous slice of it, a warp a contiguous part of that.  The
// slice is read once, for the row's largest logit, and kept in shared memory for what follows (rows too
// long for that are read again, from L2).  Then, by what the row asks for:
//   - the best one: the lowest index that has the largest logit;
//   - top-k: the k-th largest of the threads' own largest logits is at most the k-th largest of all, so that
//     little more than k elements reach it; the first block sorts those, and all that follows (min-p,
//     top-p, the draw) is done on them;
//   - top-p alone: a histogram of y tells about where the weights reach the share; the few elements there are
//     narrowed down to the one by bins of their exact weights, those before them added up;
//   - neither: the weights are added up as they lie.
// Where more elements than the sort takes are alike (or k is larger than that), the digits of
// d = max - x >= 0 are narrowed down by one histogram after another instead, then those of x among elements whose rounded d
// is one.
#include "bsf8_device.cuh"
#include "bsf8_internal.h"

#include <algorithm>
#include <cfloat>

namespace bsf8 {

namespace {

typedef unsigned long long u64;
constexpr int kTThreads = 256, kTWarps = kTThreads / 32;
constexpr int kMaxTCluster = 8;
constexpr int kBins = 1024;      // of the digits' histograms, and of the sort
constexpr int kOctaves = 41, kParts = 64;  // the histogram by y: y <= 40 in 64ths
constexpr int kSteps = kOctaves * kParts;
constexpr int kList = 2048;      // elements that the first block takes up,
constexpr int kOwn = 704;        // and that a block of a cluster finds
// Blocks an SM: their latencies hide each other (192 rows of 131072 bf16, k = 50: 30 us, 53 by two of 512 threads).  At the
// 64 registers that leaves, each of the four kernels spills 12 to 68 bytes a thread, the functions out of line 32 to 56.
constexpr int kTBlocks = 4;
constexpr uint32_t kInfBits = 0x7F800000u;
constexpr int kMaxShared = 228 * 1024;  // an SM's, of which each block takes 1 KB more than it asks for
constexpr int kEach = kList / kTThreads, kBinsEach = kBins / kTThreads;

struct TokenShared {
    float wmax[kTWarps], wlow[kTWarps], bmax;      // bmax, bsum, bmin ..: read by the cluster
    int bmin;
    u64 wsum[kTWarps], bsum, wevery[kTWarps], bevery;
    int wcount[kTWarps], bcount;
    uint32_t wfirst[kTWarps], wlast[kTWarps], bfirst, blast;
    u64 tsum[kTWarps];
    int tcount[kTWarps];
    float max8[kTThreads / 8];      // largest logits of eight threads
    float blow;                     // the smallest of the threads' largest ones, -inf left out
    int bin;                        // the bin in which the wanted rank or weight lies,
    int before;                     // and what is before it
    u64 mass;
    float wstep[2][kParts];         // about the weights by step of two octaves
    int cut;
    int listed;                     // elements in list
    u64 cut_key, total;             // of the first block: what stays, its sum
    float octave[kOctaves], all8[kOctaves];  // about the weights of this block by octave, and of all
    u64 list[kOwn];                 // this block's elements, as keys
    union {
        u64 sort[kList];
        int tally[kList];           // counts of the search for the k-th
        uint32_t steps[kSteps];     // elements by y
        struct {
            uint32_t count[kBins], low[kBins];
            u64 high[kBins];
        };
    };
};

// 2^-f on [0, 1): a polynomial fitted to it (least squares, weighted towards the largest relative error, 2^-21.92 with its
// roundings over all multiples of 2^-24), every step rounded by itself so that any machine gets the same bits.  It stays
// in [1/2, 1].
__device__ __forceinline__ float exp2_of(float f) {
    float p = -0.0009449035860598087f;
    p = __fadd_rn(__fmul_rn(p, f), 0.00920579768717289f);
    p = __fadd_rn(__fmul_rn(p, f), -0.0552973598241806f);
    p = __fadd_rn(__fmul_rn(p, f), 0.2401801496744156f);
    p = __fadd_rn(__fmul_rn(p, f), -0.6931437253952026f);
    return __fadd_rn(__fmul_rn(p, f), 1.0f);
}

// The weight at distance d = max - x >= 0; `rate` is log2(e) / t.
__device__ __forceinline__ u64 weight(float d, float rate) {
    const float y = __fmul_rn(d, rate);
    if (!(y <= 40.0f)) return 0;
    // without conversions: adding 2^23 towards zero leaves floor(y) in the low bits, and a p in [1/2, 1] is its own
    // bits less those of 1/4 (in units of 2^-24)
    const float t = __fadd_rz(y, 8388608.0f);
    const uint32_t m = __float_as_uint(exp2_of(__fsub_rn(y, __fsub_rn(t, 8388608.0f)))) - 0x3E800000u;  // 2^23 .. 2^24
    return ((u64)m << 16) >> (__float_as_uint(t) & 63u);
}

// The same for two elements at a time.
struct Two {
    float y[2];
    uint32_t n[2], m[2];  // w = (m << 16) >> n where y <= 40
};

__device__ __forceinline__ u64 two(float a, float b) {
    u64 x;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a), "f"(b));
    return x;
}
__device__ __forceinline__ void apart(u64 x, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
// a * b; `zero` is a pair of -0 that comes to the kernel as an argument: the assembler turns a product and
// a sum of pairs into one fma, .rn or not, unless it cannot know that this is a product.
__device__ __forceinline__ u64 mul2(u64 a, u64 b, u64 zero) {
    u64 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(zero));
    return d;
}
__device__ __forceinline__ u64 sum2(u64 a, u64 b) {
    u64 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ u64 sum2_rz(u64 a, u64 b) {
    u64 d;
    asm("add.rz.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ u64 less2(u64 a, u64 b) {  // a - b, rounded once
    u64 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(b), "l"(two(-1.0f, -1.0f)), "l"(a));
    return d;
}

__device__ __forceinline__ Two weights2(float a, float b, u64 top, u64 rate, u64 zero) {
    Two r;
    const u64 y = mul2(less2(top, two(a, b)), rate, zero);
    const u64 big = two(8388608.0f, 8388608.0f);
    const u64 t = sum2_rz(y, big);
    const u64 f = less2(y, sum2(t, two(-8388608.0f, -8388608.0f)));
    u64 p = two(-0.0009449035860598087f, -0.0009449035860598087f);
    p = sum2(mul2(p, f, zero), two(0.00920579768717289f, 0.00920579768717289f));
    p = sum2(mul2(p, f, zero), two(-0.0552973598241806f, -0.0552973598241806f));
    p = sum2(mul2(p, f, zero), two(0.2401801496744156f, 0.2401801496744156f));
    p = sum2(mul2(p, f, zero), two(-0.6931437253952026f, -0.6931437253952026f));
    p = sum2(mul2(p, f, zero), two(1.0f, 1.0f));
    float p0, p1, t0, t1;
    apart(y, r.y[0], r.y[1]);
    apart(p, p0, p1);
    apart(t, t0, t1);
    r.n[0] = __float_as_uint(t0) & 63u;
    r.n[1] = __float_as_uint(t1) & 63u;
    r.m[0] = __float_as_uint(p0) - 0x3E800000u;
    r.m[1] = __float_as_uint(p1) - 0x3E800000u;
    return r;
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

struct Yes {
    static constexpr bool value = true;
};
struct No {
    static constexpr bool value = false;
};

// Larger for larger values.
__device__ __forceinline__ uint32_t order_of(float f) {
    const uint32_t b = __float_as_uint(f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }

// An element's place in the order that top-k and top-p go by, smaller for larger logits, then for lower indices; 0 and -0
// are one.  Of the logit itself: max - x is rounded, and many x far below a large maximum have one distance.
__device__ __forceinline__ u64 key_at(float v, int index) { return (u64)~order_of(v + 0.0f) << 20 | (u64)index; }
__device__ __forceinline__ float logit_of(u64 key) { return value_of(~(uint32_t)(key >> 20)); }

// max - x, 0 for the largest itself (inf - inf)
__device__ __forceinline__ float distance_to(float top, float v) { return v == top ? 0.0f : __fsub_rn(top, v); }

// A group of 16 bytes: its elements, NaN as -inf.
template <typename T>
struct Logit;
template <>
struct Logit<float> {
    static constexpr int N = 4;
    static constexpr uint32_t kNone = 0xFF800000u;  // -inf, as a word of elements
    static __device__ __forceinline__ void unpack(const uint4 &w, float (&y)[4]) {
        y[0] = __uint_as_float(w.x), y[1] = __uint_as_float(w.y), y[2] = __uint_as_float(w.z), y[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ float one(const float *p) { return *p; }
    static __device__ __forceinline__ uint32_t clean(uint32_t w) { return __float_as_uint(fmaxf(__uint_as_float(w), -INFINITY)); }
    static __device__ __forceinline__ void set(uint4 &w, int i, const float *p) {
        (i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w) = __float_as_uint(*p);
    }
};
template <>
struct Logit<uint16_t> {
    static constexpr int N = 8;
    static constexpr uint32_t kNone = 0xFF80FF80u;
    static __device__ __forceinline__ void unpack(const uint4 &w, float (&y)[8]) {
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[2 * i] = __uint_as_float(a[i] << 16);
            y[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ float one(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }
    static __device__ __forceinline__ uint32_t clean(uint32_t w) {
        uint32_t d;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(w), "r"(kNone));
        return d;
    }
    static __device__ __forceinline__ void set(uint4 &w, int i, const uint16_t *p) {
        uint32_t &a = i < 2 ? w.x : i < 4 ? w.y : i < 6 ? w.z : w.w;
        a = i & 1 ? (a & 0xFFFFu) | (uint32_t)*p << 16 : (a & 0xFFFF0000u) | *p;
    }
};

// The sums over the threads before this one, and over all; a barrier inside (and one before the next call).
__device__ __forceinline__ u64 sum_before(u64 v, TokenShared &s, u64 &all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    u64 up = v;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const u64 o = __shfl_up_sync(0xFFFFFFFFu, up, m);
        if (lane >= m) up += o;
    }
    if (lane == 31) s.tsum[warp] = up;
    __syncthreads();
    u64 before = up - v;
    all = 0;
#pragma unroll
    for (int w = 0; w < kTWarps; ++w) {
        if (w < warp) before += s.tsum[w];
        all += s.tsum[w];
    }
    return before;
}

// Sorts s.sort[0 .. n), all different, by the whole block: by counting how many are smaller up to 256 of them (a
// thread or more each), else into bins of even width in the logits first.  `bins`: kBins words of scratch.  Ends with a
// barrier.
__device__ __noinline__ void sort_list(TokenShared &s, int *bins, int n) {
    const int tid = threadIdx.x;
    int size = 32;
    while (size < n) size *= 2;
    if (size <= kTThreads) {
        const int each = kTThreads / size, i = tid / each, part = tid % each;  // threads an element: 1 .. 8
        const u64 mine = i < n ? s.sort[i] : ~0ull;
        int rank = 0;
        for (int j = part; j < n; j += each) rank += s.sort[j] < mine ? 1 : 0;
        for (int m = 1; m < each; m <<= 1) rank += __shfl_xor_sync(0xFFFFFFFFu, rank, m);
        __syncthreads();
        if (i < n && part == 0) s.sort[rank] = mine;
        __syncthreads();
        return;
    }
    u64 v[kEach];
    uint32_t lo = 0xFFFFFFFFu, hi = 0;
#pragma unroll
    for (int r = 0; r < kEach; ++r) {
        v[r] = tid + r * kTThreads < n ? s.sort[tid + r * kTThreads] : ~0ull;
        if (tid + r * kTThreads < n) {
            lo = min(lo, (uint32_t)(v[r] >> 20));
            hi = max(hi, (uint32_t)(v[r] >> 20));
        }
    }
    lo = __reduce_min_sync(0xFFFFFFFFu, lo);
    hi = __reduce_max_sync(0xFFFFFFFFu, hi);
    if ((tid & 31) == 0) s.tcount[tid >> 5] = (int)lo, s.wcount[tid >> 5] = (int)hi;
    for (int i = tid; i < kBins; i += kTThreads) bins[i] = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kTWarps; ++w) lo = min(lo, (uint32_t)s.tcount[w]), hi = max(hi, (uint32_t)s.wcount[w]);
    const float first = value_of(~lo), per = fminf((float)(kBins - 1) / (first - value_of(~hi)), 1e38f);
    auto bin_of = [&](u64 key) { return min((int)((first - logit_of(key)) * per), kBins - 1); };
#pragma unroll
    for (int r = 0; r < kEach; ++r)
        if (tid + r * kTThreads < n) atomicAdd(&bins[bin_of(v[r])], 1);
    __syncthreads();
    int c[kBinsEach], sum = 0;
#pragma unroll
    for (int r = 0; r < kBinsEach; ++r) sum += c[r] = bins[kBinsEach * tid + r];
    u64 all;
    int at = (int)sum_before((u64)sum, s, all);
#pragma unroll
    for (int r = 0; r < kBinsEach; ++r) {
        bins[kBinsEach * tid + r] = at;
        at += c[r];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kEach; ++r)
        if (tid + r * kTThreads < n) s.sort[atomicAdd(&bins[bin_of(v[r])], 1)] = v[r];
    __syncthreads();
    int rank[kEach];
#pragma unroll
    for (int r = 0; r < kEach; ++r) {
        rank[r] = 0;
        if (tid + r * kTThreads >= n) continue;
        v[r] = s.sort[tid + r * kTThreads];
        const int bin = bin_of(v[r]), from = bin > 0 ? bins[bin - 1] : 0, to = bins[bin];
        rank[r] = from;
        for (int j = from; j < to; ++j) rank[r] += s.sort[j] < v[r] ? 1 : 0;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kEach; ++r)
        if (tid + r * kTThreads < n) s.sort[rank[r]] = v[r];
    __syncthreads();
}

// Of s.sort[0 .. n) in order, all different, the element in which the weights, from `run` on, reach `cut`: its key and the
// sum up to it in s.cut_key and s.total, which stay if there is none.  By bins over the logits in question, or
// over the indices of those of one logit, whose weights are added up; the few of the last bin are compared.  Loses s.sort.
__device__ __noinline__ void find_cut(TokenShared &s, int n, float top, float rate, u64 run, u64 cut, int V) {
    constexpr int kFew = 32;
    const int tid = threadIdx.x, warp = tid >> 5;
    // how many a bin has, and their weights by 20 bits (2048 of at most 2^40): atomics of 64 bits try again and again
    uint32_t *const counts = reinterpret_cast<uint32_t *>(s.sort), *const low = counts + kBins, *const high = low + kBins;
    u64 *const few = s.sort + 3 * kBins / 2;
    u64 v[kEach];
    uint32_t in = 0;  // elements in question
#pragma unroll
    for (int r = 0; r < kEach; ++r) {
        const int at = tid + r * kTThreads;
        v[r] = at < n ? s.sort[at] : 0;
        in |= at < n ? 1u << r : 0u;
    }
    auto weight_of = [&](u64 key) { return weight(distance_to(top, logit_of(key)), rate); };
    int count = n, index0 = 0, bits = 32 - __clz(V - 1);  // the indices in question, 2^bits of them
    while (count > kFew) {
        uint32_t lo = 0xFFFFFFFFu, hi = 0;
#pragma unroll
        for (int r = 0; r < kEach; ++r) {
            if (!(in >> r & 1)) continue;
            lo = min(lo, (uint32_t)(v[r] >> 20));
            hi = max(hi, (uint32_t)(v[r] >> 20));
        }
        lo = __reduce_min_sync(0xFFFFFFFFu, lo);
        hi = __reduce_max_sync(0xFFFFFFFFu, hi);
        if ((tid & 31) == 0) s.tcount[warp] = (int)lo, s.wcount[warp] = (int)hi;
        __syncthreads();
        for (int i = tid; i < 3 * kBins; i += kTThreads) counts[i] = 0;
        if (tid == 0) s.bin = -1;
#pragma unroll
        for (int i = 0; i < kTWarps; ++i) lo = min(lo, (uint32_t)s.tcount[i]), hi = max(hi, (uint32_t)s.wcount[i]);
        const bool by_index = lo == hi;
        const int shift = max(0, (by_index ? bits : 32 - __clz(hi - lo)) - 10);
        auto bin_of = [&](u64 key) {
            return (by_index ? (uint32_t)(key & 0xFFFFFu) - (uint32_t)index0 : (uint32_t)(key >> 20) - lo) >> shift;
        };
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kEach; ++r) {
            if (!(in >> r & 1)) continue;
            const uint32_t bin = bin_of(v[r]);
            const u64 w = weight_of(v[r]);
            atomicAdd(&counts[bin], 1u);
            atomicAdd(&low[bin], (uint32_t)w & 0xFFFFFu);
            atomicAdd(&high[bin], (uint32_t)(w >> 20));
        }
        __syncthreads();
        u64 m[kBinsEach], sum = 0, all;
#pragma unroll
        for (int i = 0; i < kBinsEach; ++i) sum += m[i] = ((u64)high[kBinsEach * tid + i] << 20) + low[kBinsEach * tid + i];
        u64 before = run + sum_before(sum, s, all);
#pragma unroll
        for (int i = 0; i < kBinsEach; ++i) {
            if (before < cut && before + m[i] >= cut) s.bin = kBinsEach * tid + i, s.mass = before;
            before += m[i];
        }
        __syncthreads();
        const int bin = s.bin;
        if (bin < 0) return;
        run = s.mass;
        count = (int)counts[bin];  // (one index has one element)
#pragma unroll
        for (int r = 0; r < kEach; ++r)
            if ((in >> r & 1) && bin_of(v[r]) != (uint32_t)bin) in &= ~(1u << r);
        if (by_index) index0 += bin << shift, bits = shift;
    }
    if (tid == 0) s.cut = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kEach; ++r) {
        if (!(in >> r & 1)) continue;
        const int at = 2 * atomicAdd(&s.cut, 1);
        few[at] = v[r], few[at + 1] = weight_of(v[r]);
    }
    __syncthreads();
    if (tid < count) {
        const u64 me = few[2 * tid], mine = few[2 * tid + 1];
        for (int j = 0; j < count; ++j)
            if (few[2 * j] < me) run += few[2 * j + 1];
        if (run < cut && run + mine >= cut) s.cut_key = me, s.total = run + mine;
    }
}

}  // namespace

template <typename T, bool PROBS>
__global__ void __launch_bounds__(kTThreads, kTBlocks) sample_kernel(const SampleArgs a, int cluster, int staged, float minus_zero) {
    extern __shared__ __align__(16) uint8_t memory[];
    TokenShared &s = *reinterpret_cast<TokenShared *>(memory);
    // one of a few blocks may find as many elements as are sorted: its list lies behind
    const bool long_list = cluster < 8;
    u64 *const list = long_list ? reinterpret_cast<u64 *>(memory + (sizeof(TokenShared) + 15) / 16 * 16) : s.list;
    const int own = long_list ? kList : kOwn;
    // the threads' largest logits, kept apart by fourths of their groups (halves of four blocks, none of eight)
    const int subs = cluster >= 8 ? 1 : cluster == 4 ? 2 : 4;
    float *const tmax = reinterpret_cast<float *>(memory + (sizeof(TokenShared) + 15) / 16 * 16 + (long_list ? kList * 8 : 0));
    uint4 *const stage = reinterpret_cast<uint4 *>(tmax + subs * kTThreads);
    pdl_trigger();
    pdl_wait();
    using L = Logit<T>;
    constexpr int VEC = L::N;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = blockIdx.x / cluster, rank = blockIdx.x % cluster, V = a.V;
    const T *const x = static_cast<const T *>(a.logits) + (size_t)row * a.ld;
    // groups of VEC elements that start on 16 bytes; the first and last may be partly outside the row
    const int mis = (int)(((size_t)row * a.ld) % VEC), groups = (V + mis + VEC - 1) / VEC;
    const int per_warp = ((groups + cluster * kTWarps - 1) / (cluster * kTWarps) + 7) / 8 * 8;
    const int b0 = rank * kTWarps * per_warp;  // the block's first group
    const int g0 = min(groups, b0 + warp * per_warp), g1 = min(groups, g0 + per_warp);
    const float tp = a.temperature ? a.temperature[row] : 1.0f;
    const bool greedy = !(tp >= 1.17549435e-38f);  // a temperature below fp32's normal numbers counts as 0
    const float rate = greedy ? 1.0f : __fdiv_rn(1.4426950408889634f, tp);
    int k = a.top_k ? a.top_k[row] : 0;
    if (k <= 0 || k > V) k = V;
    const float mp = a.min_p ? fminf(fmaxf(a.min_p[row], 0.0f), 1.0f) : 0.0f;
    const u64 least = max((u64)1, (u64)ceilf(mp * 1099511627776.0f));
    const float pp = a.top_p ? a.top_p[row] : 1.0f;
    const bool nucleus = pp < 1.0f;
    const u64 pfix = nucleus ? (u64)(fmaxf(pp, 0.0f) * 16777216.0f) : 0;
    const float u = PROBS ? 0.0f : a.u[row];
    float *const out = PROBS ? a.p + (size_t)row * V : nullptr;

    // group g from the caller's memory: elements outside the row, and NaN, as -inf
    auto fetch = [&](int g) -> uint4 {
        const int e = g * VEC - mis;
        uint4 w;
        if (e >= 0 && e + VEC <= V) {
            w = *reinterpret_cast<const uint4 *>(x + e);
        } else {
            w = make_uint4(L::kNone, L::kNone, L::kNone, L::kNone);
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if ((unsigned)(e + i) < (unsigned)V) L::set(w, i, x + e + i);
        }
        return make_uint4(L::clean(w.x), L::clean(w.y), L::clean(w.z), L::clean(w.w));
    };
    auto load = [&](int g, float (&y)[VEC]) { L::unpack(staged ? stage[g - b0] : fetch(g), y); };
    // f(elements, first one's index) of the warp's part, a lane's groups 32 apart, four on their way
    auto each = [&](auto f) {
        int g = g0 + lane;
        for (; g + 96 < g1; g += 128) {
            uint4 w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = staged ? stage[g + 32 * j - b0] : fetch(g + 32 * j);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float y[VEC];
                L::unpack(w[j], y);
                f(y, (g + 32 * j) * VEC - mis);
            }
        }
        for (; g < g1; g += 32) {
            float y[VEC];
            load(g, y);
            f(y, g * VEC - mis);
        }
    };
    auto barrier = [&]() {
        if (cluster > 1) cluster_barrier();
        else __syncthreads();
    };
    auto of32 = [&](const void *p, int c) { return cluster > 1 ? ld_cluster32(map_to_rank(p, c)) : *static_cast<const uint32_t *>(p); };
    auto of64 = [&](const void *p, int c) { return cluster > 1 ? ld_cluster64(map_to_rank(p, c)) : *static_cast<const u64 *>(p); };

    // ---------------------------------------------------------------- the largest
    float top;
    {
        constexpr int U = 4;  // loads in flight
        float m[U] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        int g = g0 + lane;
        for (; g + 32 * (U - 1) < g1; g += 32 * U) {
            uint4 w[U];
#pragma unroll
            for (int j = 0; j < U; ++j) w[j] = fetch(g + 32 * j);
#pragma unroll
            for (int j = 0; j < U; ++j) {
                if (staged) stage[g + 32 * j - b0] = w[j];
                float y[VEC];
                L::unpack(w[j], y);
#pragma unroll
                for (int i = 0; i < VEC; ++i) m[j] = fmaxf(m[j], y[i]);
            }
        }
#pragma unroll
        for (int j = 0; j < U - 1; ++j, g += 32) {
            if (g >= g1) break;
            const uint4 w = fetch(g);
            if (staged) stage[g - b0] = w;
            float y[VEC];
            L::unpack(w, y);
#pragma unroll
            for (int i = 0; i < VEC; ++i) m[j] = fmaxf(m[j], y[i]);
        }
        if (subs == 4) {
#pragma unroll
            for (int j = 0; j < U; ++j) tmax[j * kTThreads + tid] = m[j];
        }
        m[0] = fmaxf(m[0], m[2]);
        m[1] = fmaxf(m[1], m[3]);
        if (subs == 2) tmax[tid] = m[0], tmax[kTThreads + tid] = m[1];
        top = fmaxf(m[0], m[1]);
        if (subs == 1) tmax[tid] = top;
    }
    float wtop = top, wlow = top > -INFINITY ? top : INFINITY;  // (of the threads that have any)
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        wtop = fmaxf(wtop, __shfl_xor_sync(0xFFFFFFFFu, wtop, m));
        wlow = fminf(wlow, __shfl_xor_sync(0xFFFFFFFFu, wlow, m));
        if (m == 4 && (lane & 7) == 0) s.max8[tid >> 3] = wtop;
    }
    if (lane == 0) s.wmax[warp] = wtop, s.wlow[warp] = wlow;
    if (tid == 0) s.listed = 0, s.bmin = 0x7FFFFFFF;
    for (int i = tid; i < kList; i += kTThreads) s.tally[i] = 0;
    __syncthreads();
    if (warp == 0) {
        wtop = s.wmax[lane & (kTWarps - 1)];
        wlow = s.wlow[lane & (kTWarps - 1)];
#pragma unroll
        for (int m = 8; m > 0; m >>= 1) {
            wtop = fmaxf(wtop, __shfl_xor_sync(0xFFFFFFFFu, wtop, m));
            wlow = fminf(wlow, __shfl_xor_sync(0xFFFFFFFFu, wlow, m));
        }
        if (lane == 0) s.bmax = wtop, s.blow = wlow;
    }
    barrier();
    const float mine = top;  // this thread's own
    top = lane < cluster ? __uint_as_float(of32(&s.bmax, lane)) : -INFINITY;
    float low = lane < cluster ? __uint_as_float(of32(&s.blow, lane)) : INFINITY;
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
        low = fminf(low, __shfl_xor_sync(0xFFFFFFFFu, low, m));
    }
    const bool none = top == -INFINITY;

    // p of the row's elements from their weights; 0 where nothing stays
    float inv = 0.0f;
    auto share = [&](u64 w) { return fmaf((float)(uint32_t)(w >> 20), 1048576.0f, (float)(uint32_t)(w & 0xFFFFFu)) * inv; };
    auto draw_at = [&](u64 sum) { return part_of((u64)(fminf(fmaxf(u, 0.0f), 0.99999994f) * 16777216.0f), sum); };
    auto zeros = [&]() {  // of this block's slice of the distribution
        const int from = max(0, b0 * VEC - mis), to = min(V, (b0 + kTWarps * per_warp) * VEC - mis);
        float *const o = out + from;
        const int n = to - from, head = min(max(n, 0), (int)((16 - (reinterpret_cast<uintptr_t>(o) & 15)) & 15) / 4);
        if (tid < head) o[tid] = 0.0f;
        for (int i = head + 4 * tid; i + 4 <= n; i += 4 * kTThreads) *reinterpret_cast<float4 *>(o + i) = make_float4(0, 0, 0, 0);
        const int tail = head + max(n - head, 0) / 4 * 4;
        if (tail + tid < n) o[tail + tid] = 0.0f;
    };

    if (none || greedy) {
        // ------------------------------------------------------------ the best one, or none
        if (!none && mine == top) {
            int at = 0x7FFFFFFF;
            for (int g = g0 + lane; g < g1 && at == 0x7FFFFFFF; g += 32) {
                float y[VEC];
                load(g, y);
#pragma unroll
                for (int i = VEC - 1; i >= 0; --i)
                    if (y[i] == top) at = g * VEC - mis + i;
            }
            atomicMin(&s.bmin, at);
        }
        if (PROBS) zeros();
        barrier();
        if (rank == 0 && warp == 0) {
            int at = lane < cluster ? (int)of32(&s.bmin, lane) : 0x7FFFFFFF;
            at = __reduce_min_sync(0xFFFFFFFFu, at);
            if (lane == 0) {
                if (PROBS) {
                    if (!none) out[at] = 1.0f;
                } else {
                    a.token[row] = none ? -1 : at;
                    a.p[row] = none ? 0.0f : 1.0f;
                }
            }
        }
        if (cluster > 1) cluster_barrier();  // no block leaves while another may read its memory
        return;
    }

    // the distance of an element, infinite where it has no part
    auto distance = [&](float v) { return distance_to(top, v); };
    auto weight_of = [&](u64 key) { return weight(distance(logit_of(key)), rate); };
    auto keep_in_list = [&](float v, int index) {
        if (distance(v) == INFINITY) return;
        const int at = atomicAdd(&s.listed, 1);
        if (at < own) list[at] = key_at(v, index);
    };
    // the blocks' lists, in the first one's `sort`; how many elements (none are moved where they are too many)
    auto collect = [&]() {
        int upto = lane < cluster ? (int)of32(&s.listed, lane) : 0;
#pragma unroll
        for (int m = 1; m < kMaxTCluster; m <<= 1) {
            const int o = __shfl_up_sync(0xFFFFFFFFu, upto, m);
            if (lane >= m) upto += o;
        }
        const int n = __shfl_sync(0xFFFFFFFFu, upto, kMaxTCluster - 1);
        if (__any_sync(0xFFFFFFFFu, lane < cluster && (int)of32(&s.listed, lane) > own)) return kList + 1;
        if (n > kList || rank > 0) return n;
        int end[kMaxTCluster];
#pragma unroll
        for (int c = 0; c < kMaxTCluster; ++c) end[c] = __shfl_sync(0xFFFFFFFFu, upto, c);
        for (int i = tid; i < n; i += kTThreads) {
            int c = 0, from = 0;
#pragma unroll
            for (int j = 0; j < kMaxTCluster - 1; ++j)
                if (i >= end[j]) c = j + 1, from = end[j];
            s.sort[i] = of64(&list[i - from], c);
        }
        return n;
    };
    const u64 top2 = two(top, top), rate2 = two(rate, rate), zero2 = two(minus_zero, minus_zero);
    // what is found to stay: elements of logits above cut_x, and of those that equal it the ones up to cut_index (all: -inf)
    float cut_x = -INFINITY;
    int cut_index = 0x7FFFFFFF;
    auto stays = [&](float v, int index) { return v > cut_x || (v == cut_x && index <= cut_index); };
    bool summed = false;  // the cut is found, and the sums of what stays in each warp's part

    // ---------------------------------------------------------------- top-k by a few candidates
    const bool few = V <= kList && (k < V || nucleus);
    constexpr int kMax8 = kTThreads / 8;
    const int g8 = kMax8 * cluster, gt = kTThreads * cluster * subs;  // maxima of eight threads, of (a part of) one
    // with k of so many maxima to reach, some -real ln(1 - k / real) elements do; where that is far above k and the block has
    // the whole row, all elements take the maxima's place (18 rows of 4435, k = 1000 and top-p: 41 us by the digits below, 21)
    const int real = min(gt, groups);
    const bool one = cluster == 1 && 2 * k > real;
    const int most_k = one ? kList - 96 : (int)((float)real * fminf(0.95f, 1.0f - expf(-1800.0f / (float)real)));
    if (top < INFINITY && (few || (k < V && k <= most_k))) {
        float least_value = -INFINITY;
        if (!few) {
            // (a little below) the k-th largest of the maxima
            uint32_t v[kMaxTCluster];
            const int nv = 2 * k <= g8 ? 1 : cluster * subs;  // at most eight
            if (one) {
                v[0] = 0;
            } else if (nv == 1) {
                v[0] = tid < g8 ? order_of(__uint_as_float(of32(&s.max8[tid % kMax8], tid / kMax8))) : 0u;
            } else {
#pragma unroll
                for (int c = 0; c < kMaxTCluster; ++c)
                    v[c] = c < nv ? order_of(__uint_as_float(of32(&tmax[c / cluster * kTThreads + tid], c % cluster))) : 0u;
            }
            // a histogram between the least and the largest of them, finer again where those are far apart; what
            // lies above the bins counts in the first one
            uint32_t from = order_of(one ? -FLT_MAX : low), range = order_of(top) - from;
            for (int turn = 0; turn < 3 && (turn == 0 || range >= 65536); ++turn) {
                const int shift = max(0, 32 - __clz(range) - 11);
                if (turn > 0) {
                    __syncthreads();
                    for (int i = tid; i < kList; i += kTThreads) s.tally[i] = 0;
                    __syncthreads();
                }
                auto add = [&](uint32_t x) {
                    if (x >= from) atomicAdd(&s.tally[kList - 1 - min((x - from) >> shift, (uint32_t)(kList - 1))], 1);
                };
                if (one) {
                    each([&](const float (&y)[VEC], int) {
#pragma unroll
                        for (int i = 0; i < VEC; ++i) add(order_of(y[i]));
                    });
                } else {
                    add(v[0]);
                }
                if (!one && nv > 1) {
#pragma unroll
                    for (int c = 1; c < kMaxTCluster; ++c)
                        if (c < nv) add(v[c]);
                }
                if (tid == 0) s.bin = -1;
                __syncthreads();
                int n[kEach], sum = 0;
#pragma unroll
                for (int i = 0; i < kEach; ++i) sum += n[i] = s.tally[kEach * tid + i];
                u64 all;
                int before = (int)sum_before((u64)sum, s, all);
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    if (before < k && before + n[i] >= k) s.bin = kList - 1 - (kEach * tid + i);
                    before += n[i];
                }
                __syncthreads();
                if (s.bin < 0) {  // fewer than k threads (or elements) have any
                    from = 0;
                    break;
                }
                from += (uint32_t)s.bin << shift;
                range = (1u << shift) - 1;
            }
            least_value = value_of(from);
            if (!(least_value >= -INFINITY)) least_value = -INFINITY;  // (no such number)
        }
        each([&](const float (&y)[VEC], int at) {
            float m = y[0];
#pragma unroll
            for (int i = 1; i < VEC; ++i) m = fmaxf(m, y[i]);
            if (m >= least_value) {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (y[i] >= least_value) keep_in_list(y[i], at + i);
            }
        });
        if (PROBS) zeros();
        barrier();
        const int n = collect();
        if (n <= kList) {
            barrier();  // the lists are read: the other blocks leave
            if (rank == 0) {
                sort_list(s, reinterpret_cast<int *>(list), n);
                // some a thread, in order: weights, what min-p and top-p leave of the first k
                u64 w[kEach], key[kEach], sum = 0;
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    const int at = kEach * tid + i;
                    key[i] = at < min(n, k) ? s.sort[at] : ~0ull;
                    w[i] = at < min(n, k) ? weight_of(key[i]) : 0;
                    if (w[i] < least) w[i] = 0;
                    sum += w[i];
                }
                u64 all, before;
                if (nucleus) {
                    before = sum_before(sum, s, all);
                    const u64 cut = max((u64)1, part_of(pfix, all));
#pragma unroll
                    for (int i = 0; i < kEach; ++i) {
                        const u64 wi = w[i];
                        if (before >= cut) w[i] = 0;
                        before += wi;
                    }
                }
                __syncthreads();
                if (PROBS) {
                    sum = 0;
#pragma unroll
                    for (int i = 0; i < kEach; ++i) sum += w[i];
                    (void)sum_before(sum, s, all);
                    inv = 1.0f / (float)all;
#pragma unroll
                    for (int i = 0; i < kEach; ++i)
                        if (w[i]) out[(int)(key[i] & 0xFFFFFu)] = share(w[i]);
                } else {
                    // the draw goes by index: sums over 2048 equal parts of the row, then inside one of them
                    uint32_t *const low = reinterpret_cast<uint32_t *>(s.sort), *const high = low + kList;  // by 20 bits
                    for (int i = tid; i < kList; i += kTThreads) s.sort[i] = 0;
                    if (tid == 0) s.listed = 0;
                    __syncthreads();
                    const int shift = max(0, 32 - __clz(V - 1) - 11);
#pragma unroll
                    for (int i = 0; i < kEach; ++i) {
                        if (w[i] == 0) continue;
                        const uint32_t at = (uint32_t)(key[i] & 0xFFFFFu) >> shift;
                        atomicAdd(&low[at], (uint32_t)w[i] & 0xFFFFFu);
                        atomicAdd(&high[at], (uint32_t)(w[i] >> 20));
                    }
                    __syncthreads();
                    u64 part[kEach];
                    sum = 0;
#pragma unroll
                    for (int i = 0; i < kEach; ++i) sum += part[i] = ((u64)high[kEach * tid + i] << 20) + low[kEach * tid + i];
                    before = sum_before(sum, s, all);
                    inv = 1.0f / (float)all;
                    const u64 at = draw_at(all);
#pragma unroll
                    for (int i = 0; i < kEach; ++i) {
                        if (at >= before && at < before + part[i]) s.bin = kEach * tid + i, s.mass = before;
                        before += part[i];
                    }
                    __syncthreads();
                    const int bin = s.bin;
#pragma unroll
                    for (int i = 0; i < kEach; ++i)
                        if (w[i] && (int)((uint32_t)(key[i] & 0xFFFFFu) >> shift) == bin)
                            list[atomicAdd(&s.listed, 1)] = (key[i] & 0xFFFFFu) << 41 | w[i];
                    __syncthreads();
                    const int listed = s.listed;  // at most 512 indices a part
                    for (int i = tid; i < listed; i += kTThreads) {
                        const u64 me = list[i], one = (1ull << 41) - 1;
                        before = s.mass;
                        for (int j = 0; j < listed; ++j)
                            if (list[j] < me) before += list[j] & one;
                        if (at >= before && at < before + (me & one)) {
                            a.token[row] = (int)(me >> 41);
                            a.p[row] = share(me & one);
                        }
                    }
                }
            }
            return;
        }
        barrier();  // the lists are begun again
        if (tid == 0) s.listed = 0;
        __syncthreads();
    }

    // ---------------------------------------------------------------- top-p by a histogram of y
    // Weights of 11 bits in each 64th of an octave tell to a thousandth (of the smaller side) where they reach the
    // share.  Of the elements there the one is looked for, everything else is added up exactly, and if the cut is not among
    // them after all the digits below find it.  (p = 0.9, rows of 131072 bf16: 38 rows 34 us, 76 55, 114 68, 152 87, 192 93:
    // blocks that share an SM slow each other.  Of the 53 us of a row among as many as run at once the largest takes 6, the
    // histogram 10, its edges 4.5, the exact weights 17, the cut 8, the draw 6.)
    if (nucleus && k == V && top < INFINITY) {
        for (int i = tid; i < kSteps; i += kTThreads) s.steps[i] = 0;
        __syncthreads();
        const float farthest = least > 1 ? fminf(40.0f, 40.001f - log2f((float)least)) : 40.0f;
        const u64 eighths = two(8.0f * kParts, 8.0f * kParts), big = two(8388608.0f, 8388608.0f);
        each([&](const float (&y)[VEC], int) {
#pragma unroll
            for (int i = 0; i < VEC; i += 2) {
                const u64 z = mul2(less2(top2, two(y[i], y[i + 1])), rate2, zero2);
                u64 t;
                asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(t) : "l"(z), "l"(eighths), "l"(big));
                float y0, y1, t0, t1;
                apart(z, y0, y1);
                apart(t, t0, t1);
                const uint32_t q0 = __float_as_uint(t0) & 0x7FFFu, q1 = __float_as_uint(t1) & 0x7FFFu;
                // 2048 less what an eighth of a step takes off: at most 2^20 elements
                if (y0 <= farthest) atomicAdd(&s.steps[q0 >> 3], (16373u - 22u * (q0 & 7)) >> 3);
                if (y1 <= farthest) atomicAdd(&s.steps[q1 >> 3], (16373u - 22u * (q1 & 7)) >> 3);
            }
        });
        __syncthreads();
        // the weight of a step, in units of its octave's largest
        auto step_mass = [&](uint32_t v, int step) { return (float)v * exp2f(-11.0f - (float)step / kParts); };
        const int o = tid / 4, c0 = tid % 4;  // four threads an octave
        static_assert(kTThreads / 4 >= kOctaves && kTThreads == 4 * kParts, "threads an octave, and a step");
        {
            float v = 0.0f;
            if (o < kOctaves)
#pragma unroll 4
                for (int j = c0; j < kParts; j += 4) v += step_mass(s.steps[o * kParts + j], j);
            v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
            v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
            if (c0 == 0 && o < kOctaves) s.octave[o] = v * exp2f(-(float)o);
        }
        barrier();
        // two octaves, then the steps in them: where the share less and more a thousandth lies (every block for itself)
        int edge[2];
        {
            float v = 0.0f;
            if (o < kOctaves) {
                if (c0 < cluster) v = __uint_as_float(of32(&s.octave[o], c0));
                if (c0 + 4 < cluster) v += __uint_as_float(of32(&s.octave[o], c0 + 4));
            }
            v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
            v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
            if (c0 == 0 && o < kOctaves) s.all8[o] = v;
            __syncthreads();
            // two of them a lane, in every warp: the sums before each
            auto sums = [&](const float *m, int n, float &m0, float &m1, float &all_) {
                m0 = 2 * lane < n ? m[2 * lane] : 0.0f;
                m1 = 2 * lane + 1 < n ? m[2 * lane + 1] : 0.0f;
                float up = m0 + m1;
#pragma unroll
                for (int i = 1; i < 32; i <<= 1) {
                    const float x = __shfl_up_sync(0xFFFFFFFFu, up, i);
                    if (lane >= i) up += x;
                }
                all_ = __shfl_sync(0xFFFFFFFFu, up, 31);
                m1 = up;        // up to the second,
                m0 = up - (2 * lane + 1 < n ? m[2 * lane + 1] : 0.0f);  // and up to the first
            };
            // the first that passes `want` (the last of n if none does)
            auto first = [&](float m0, float m1, float want, int n) {
                const uint32_t f = __ballot_sync(0xFFFFFFFFu, m0 > want), g = __ballot_sync(0xFFFFFFFFu, m1 > want);
                const int i = f ? 2 * (__ffs(f) - 1) : 64, j = g ? 2 * (__ffs(g) - 1) + 1 : 64;
                return min(min(i, j), n - 1);
            };
            const float p0 = fmaxf(pp, 0.0f), slack = 0.003f * p0 * (1.0f - p0) + 1e-6f;
            float m0, m1, whole, before[2];
            sums(s.all8, kOctaves, m0, m1, whole);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float want = (e ? p0 + slack : p0 - slack) * whole;
                edge[e] = first(m0, m1, want, kOctaves);
                // what the octaves before it hold
                const int at = edge[e] - 1;
                const float a0 = __shfl_sync(0xFFFFFFFFu, m0, max(at, 0) / 2), a1 = __shfl_sync(0xFFFFFFFFu, m1, max(at, 0) / 2);
                before[e] = want - (at < 0 ? 0.0f : at & 1 ? a1 : a0);
            }
            // four threads a step, two blocks' counts each
            const int step = tid / 4;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float m = 0.0f;
                if (c0 < cluster) m = step_mass(of32(&s.steps[edge[e] * kParts + step], c0), step);
                if (c0 + 4 < cluster) m += step_mass(of32(&s.steps[edge[e] * kParts + step], c0 + 4), step);
                m += __shfl_xor_sync(0xFFFFFFFFu, m, 1);
                m += __shfl_xor_sync(0xFFFFFFFFu, m, 2);
                if (c0 == 0) s.wstep[e][step] = m * exp2f(-(float)edge[e]);
            }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sums(s.wstep[e], kParts, m0, m1, whole);
                edge[e] = edge[e] * kParts + first(m0, m1, before[e], kParts);
            }
        }
        barrier();  // (the histograms are read)
        u64 sum = 0, every = 0;
        const float from = (float)edge[0] * (1.0f / kParts), to = (float)(edge[1] + 1) * (1.0f / kParts);
        auto part_by = [&](auto all_stay) {  // all_stay: no weight is too small to stay
            each([&](const float (&y)[VEC], int at) {
                uint32_t here = 0;  // those of the steps in question
#pragma unroll
                for (int i = 0; i < VEC; i += 2) {
                    const Two w = weights2(y[i], y[i + 1], top2, rate2, zero2);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const u64 wj = ((u64)w.m[j] << 16) >> w.n[j];
                        const bool real = w.y[j] <= 40.0f && (decltype(all_stay)::value || wj >= least);
                        if (real) every += wj;
                        if (real && w.y[j] < from) sum += wj;
                        here |= real && w.y[j] >= from && w.y[j] < to ? 1u << (i + j) : 0u;
                    }
                }
                while (here) {
                    const int i = __ffs(here) - 1;
                    here &= here - 1;
                    float v = y[0];
#pragma unroll
                    for (int j = 1; j < VEC; ++j) v = i == j ? y[j] : v;
                    keep_in_list(v, at + i);
                }
            });
        };
        if (least <= 1) part_by(Yes{});
        else part_by(No{});
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) {
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, m);
            every += __shfl_xor_sync(0xFFFFFFFFu, every, m);
        }
        if (lane == 0) s.wsum[warp] = sum, s.wevery[warp] = every;
        __syncthreads();
        if (warp == 0) {
            u64 v = s.wsum[lane % kTWarps], w = s.wevery[lane % kTWarps];
#pragma unroll
            for (int m = kTWarps / 2; m > 0; m >>= 1) {
                v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
                w += __shfl_xor_sync(0xFFFFFFFFu, w, m);
            }
            if (lane == 0) s.bsum = v, s.bevery = w;
        }
        barrier();
        const int n = collect();
        bool found = n <= kList;
        if (found) {
            if (rank == 0) {
                u64 below = lane < cluster ? of64(&s.bsum, lane) : 0, all = lane < cluster ? of64(&s.bevery, lane) : 0;
#pragma unroll
                for (int m = kMaxTCluster / 2; m > 0; m >>= 1) {
                    below += __shfl_xor_sync(0xFFFFFFFFu, below, m);
                    all += __shfl_xor_sync(0xFFFFFFFFu, all, m);
                }
                below = __shfl_sync(0xFFFFFFFFu, below, 0);
                const u64 cut = max((u64)1, part_of(pfix, __shfl_sync(0xFFFFFFFFu, all, 0)));
                if (tid == 0) s.total = 0;
                __syncthreads();
                find_cut(s, n, top, rate, below, cut, V);
            }
            barrier();
            const u64 kept_all = of64(&s.total, 0);
            found = kept_all != 0;  // else the cut is elsewhere
            if (found) {
                summed = true;
                const u64 key = of64(&s.cut_key, 0);
                cut_x = logit_of(key);
                cut_index = (int)(key & 0xFFFFFu);
                inv = 1.0f / (float)kept_all;
            }
        }
        if (!found) {
            barrier();  // the lists are read
        } else if (!PROBS) {
            // this block's share of them, into the sums of the warps whose part they lie in (by 20 bits)
            if (tid < kTWarps) s.tcount[tid] = s.wcount[tid] = 0;
            __syncthreads();
            for (int i = tid; i < s.listed; i += kTThreads) {
                const u64 key = list[i];
                const int part = (((int)(key & 0xFFFFFu) + mis) / VEC - b0) / per_warp;
                if (part >= kTWarps || !stays(logit_of(key), (int)(key & 0xFFFFFu))) continue;
                const u64 w = weight_of(key);
                atomicAdd(&s.tcount[part], (int)((uint32_t)w & 0xFFFFFu));
                atomicAdd(&s.wcount[part], (int)(w >> 20));
            }
            __syncthreads();
            if (tid < kTWarps) s.wsum[tid] += ((u64)(uint32_t)s.wcount[tid] << 20) + (uint32_t)s.tcount[tid];
            __syncthreads();
        }
    }

    // ---------------------------------------------------------------- by digits, where there are too many alike
    // Narrows the cut down to the element in which the running count (or weight) reaches `want`: of those inside
    // the present cut.
    auto narrow = [&](bool by_weight, u64 want_in, bool fraction) {
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
                    if (bits - base > most || bits >= kInfBits || !stays(y[i], g * VEC - mis + i)) continue;
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
            // the cluster's histogram, some bins a thread, and the sums before each
            u64 w2[kBinsEach] = {}, upw = 0;
            int c2[kBinsEach] = {}, upc = 0;
#pragma unroll
            for (int j = 0; j < kBinsEach; ++j) {
                const int bin = kBinsEach * tid + j;
                for (int c = 0; c < cluster; ++c) {
                    c2[j] += (int)of32(&s.count[bin], c);
                    if (by_weight) w2[j] += (u64)of32(&s.low[bin], c) + (of64(&s.high[bin], c) << 12);
                }
                upw += w2[j];
                upc += c2[j];
            }
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
            for (int j = 0; j < kBinsEach; ++j) {
                const u64 before = by_weight ? upw : (u64)upc, mine = by_weight ? w2[j] : (u64)c2[j];
                if (before < want && before + mine >= want) {
                    s.bin = kBinsEach * tid + j;
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
        // elements at this distance have one weight: as many of them as it takes, by their logits where those differ (far below
        // a large maximum), then by index
        const u64 each = by_weight ? weight(__uint_as_float(base), rate) : 1;
        u64 keep = (want + each - 1) / each;
        float least_x = -INFINITY, most_x = INFINITY;  // the logits in question
        auto is_one = [&](float v, int index) {
            return __float_as_uint(distance(v)) == base && v >= least_x && v <= most_x && stays(v, index);
        };
        int mine;
        while (true) {
            mine = 0;
            float least_of = INFINITY, most_of = -INFINITY;
            for (int g = g0 + lane; g < g1; g += 32) {
                float y[VEC];
                load(g, y);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const bool in = is_one(y[i], g * VEC - mis + i);
                    mine += in ? 1 : 0;
                    least_of = in ? fminf(least_of, y[i]) : least_of;
                    most_of = in ? fmaxf(most_of, y[i]) : most_of;
                }
            }
            mine = __reduce_add_sync(0xFFFFFFFFu, mine);
            uint32_t lo = __reduce_min_sync(0xFFFFFFFFu, order_of(least_of + 0.0f)), hi = __reduce_max_sync(0xFFFFFFFFu, order_of(most_of + 0.0f));
            if (lane == 0) s.wcount[warp] = mine, s.wfirst[warp] = lo, s.wlast[warp] = hi;
            __syncthreads();
            if (tid == 0) {
                int v = 0;
#pragma unroll
                for (int w = 0; w < kTWarps; ++w) {
                    v += s.wcount[w];
                    lo = min(lo, s.wfirst[w]);
                    hi = max(hi, s.wlast[w]);
                }
                s.bcount = v, s.bfirst = lo, s.blast = hi;
                s.cut = -1;
            }
            barrier();
            lo = __reduce_min_sync(0xFFFFFFFFu, lane < cluster ? of32(&s.bfirst, lane) : ~0u);
            hi = __reduce_max_sync(0xFFFFFFFFu, lane < cluster ? of32(&s.blast, lane) : 0u);
            least_x = value_of(lo);
            most_x = value_of(hi);
            if (lo == hi) break;
            // which of the logits, from the largest: 10 bits of them a turn
            for (int i = tid; i < kBins; i += kTThreads) s.count[i] = 0;
            __syncthreads();
            const int narrower = max(0, 32 - __clz(hi - lo) - 10);
            for (int g = g0 + lane; g < g1; g += 32) {
                float y[VEC];
                load(g, y);
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if (is_one(y[i], g * VEC - mis + i)) atomicAdd(&s.count[(hi - order_of(y[i] + 0.0f)) >> narrower], 1u);
            }
            barrier();
            int n[kBinsEach], sum = 0;
#pragma unroll
            for (int j = 0; j < kBinsEach; ++j) {
                n[j] = 0;
                for (int c = 0; c < cluster; ++c) n[j] += (int)of32(&s.count[kBinsEach * tid + j], c);
                sum += n[j];
            }
            u64 all;
            u64 before = sum_before((u64)sum, s, all);
#pragma unroll
            for (int j = 0; j < kBinsEach; ++j) {
                if (before < keep && before + n[j] >= keep) s.bin = kBinsEach * tid + j, s.mass = before;
                before += n[j];
            }
            barrier();
            keep -= s.mass;
            hi -= (uint32_t)s.bin << narrower;
            lo = max(lo, hi - min(hi, (1u << narrower) - 1u));
            least_x = value_of(lo);
            most_x = value_of(hi);
        }
        // the index of the keep-th of them
        u64 before = __reduce_add_sync(0xFFFFFFFFu, lane < rank ? of32(&s.bcount, lane) : 0u);
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
                    is[i] = y[i] == most_x && stays(y[i], g * VEC - mis + i);
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
        cut_index = __reduce_max_sync(0xFFFFFFFFu, lane < cluster ? (int)of32(&s.cut, lane) : -1);
        cut_x = most_x;
        barrier();  // s.cut is written again
    };

    if (!summed) {
        if (k < V) narrow(false, (u64)k, false);
        if (nucleus) narrow(true, pfix, true);
    }

    // ---------------------------------------------------------------- what stays, in order of index
    auto kept = [&](float v, int index) -> u64 {
        const float d = distance(v);
        if (d == INFINITY || !stays(v, index)) return 0;
        const u64 w = weight(d, rate);
        return w >= least ? w : 0;
    };
    if (!summed) {
        u64 sum = 0;
        if (cut_x == -INFINITY && top < INFINITY) {  // nothing is cut off
            auto add = [&](auto all) {  // all: no weight is too small to stay
                each([&](const float (&y)[VEC], int) {
#pragma unroll
                    for (int i = 0; i < VEC; i += 2) {
                        const Two w = weights2(y[i], y[i + 1], top2, rate2, zero2);
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const u64 wj = ((u64)w.m[j] << 16) >> w.n[j];
                            if (w.y[j] <= 40.0f && (decltype(all)::value || wj >= least)) sum += wj;
                        }
                    }
                });
            };
            if (least <= 1) add(Yes{});
            else add(No{});
        } else {
            each([&](const float (&y)[VEC], int at) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) sum += kept(y[i], at + i);
            });
        }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, m);
        if (lane == 0) s.wsum[warp] = sum;
        __syncthreads();
    }
    u64 total = 0, first = 0;
    if (!(PROBS && summed)) {
        if (warp == 0) {
            u64 v = lane < kTWarps ? s.wsum[lane] : 0;
#pragma unroll
            for (int m = 8; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
            if (lane == 0) s.bsum = v;
        }
        barrier();
        const u64 v = lane < cluster ? of64(&s.bsum, lane) : 0;
        first = lane < rank ? v : 0;
        total = v;
#pragma unroll
        for (int m = kMaxTCluster / 2; m > 0; m >>= 1) {
            first += __shfl_xor_sync(0xFFFFFFFFu, first, m);
            total += __shfl_xor_sync(0xFFFFFFFFu, total, m);
        }
        first = __shfl_sync(0xFFFFFFFFu, first, 0);
        total = __shfl_sync(0xFFFFFFFFu, total, 0);
        inv = 1.0f / (float)total;
    }

    if constexpr (PROBS) {
        each([&](const float (&y)[VEC], int e) {
            float p[VEC];
            if (top < INFINITY && (cut_x == -INFINITY || summed)) {
#pragma unroll
                for (int i = 0; i < VEC; i += 2) {
                    const Two w = weights2(y[i], y[i + 1], top2, rate2, zero2);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const u64 wj = ((u64)w.m[j] << 16) >> w.n[j];
                        const bool in = w.y[j] <= 40.0f && wj >= least && (!summed || stays(y[i + j], e + i + j));
                        p[i + j] = in ? share(wj) : 0.0f;
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) p[i] = share(kept(y[i], e + i));
            }
            if (e >= 0 && e + VEC <= V && (reinterpret_cast<uintptr_t>(out + e) & 15) == 0) {
#pragma unroll
                for (int i = 0; i < VEC; i += 4)
                    *reinterpret_cast<float4 *>(out + e + i) = make_float4(p[i], p[i + 1], p[i + 2], p[i + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    if ((unsigned)(e + i) < (unsigned)V) out[e + i] = p[i];
            }
        });
    } else {
        const u64 at = draw_at(total);
        if (at >= first && at < first + s.bsum) {  // this block's slice has it: which warp's part
            u64 before = first;
            int w = 0;
            while (at >= before + s.wsum[w]) before += s.wsum[w++];
            // the whole block over that part, a thread some groups one after another; then a warp over those of one
            const int p0 = b0 + w * per_warp, p1 = min(groups, p0 + per_warp), some = (per_warp + kTThreads - 1) / kTThreads;
            const int mine0 = p0 + tid * some;
            u64 own = 0, all;
            for (int g = mine0; g < min(p1, mine0 + some); ++g) {
                float y[VEC];
                load(g, y);
#pragma unroll
                for (int i = 0; i < VEC; ++i) own += kept(y[i], g * VEC - mis + i);
            }
            before += sum_before(own, s, all);
            if (at >= before && at < before + own) s.bin = mine0, s.mass = before;
            __syncthreads();
            if (warp == 0) {
                before = s.mass;
                const int e0 = s.bin * VEC, e1 = min(e0 + some * VEC, p1 * VEC);
                for (int e = e0; e < e1 && before <= at; e += 32) {
                    float v = -INFINITY;
                    const int index = e + lane - mis;
                    if (e + lane < e1)
                        v = staged ? L::one(reinterpret_cast<const T *>(stage) + (e + lane - b0 * VEC))
                                   : (unsigned)index < (unsigned)V ? fmaxf(L::one(x + index), -INFINITY) : -INFINITY;
                    const u64 wi = kept(v, index);
                    u64 upto = wi;
#pragma unroll
                    for (int m = 1; m < 32; m <<= 1) {
                        const u64 q = __shfl_up_sync(0xFFFFFFFFu, upto, m);
                        if (lane >= m) upto += q;
                    }
                    const u64 r = before + upto - wi;
                    if (at >= r && at < r + wi) {
                        a.token[row] = index;
                        a.p[row] = share(wi);
                    }
                    before += __shfl_sync(0xFFFFFFFFu, upto, 31);
                }
            }
        }
    }
    if (cluster > 1) cluster_barrier();  // no block leaves while another may read its sums
}

// Clusters that run at once with so many blocks an SM: fewer than the SMs in all would take, as a cluster stays within
// one part of them (by an even share of the SMs 16 rows of 131072 bf16 took a block an SM, two turns and 18 us; now 12;
// 38 rows 19, now 15).  Not for more than that: 48 fp32 rows by four blocks an SM where three do 19 us, 16 by three.
template <typename T, bool PROBS>
cudaError_t clusters_at_once(const cudaLaunchConfig_t &cfg, int dev, int cluster, int blocks, int *n) {
    static int known[64][kMaxTCluster + 1][kTBlocks];  // and one more; 0: not asked yet
    int *const at = &known[dev][cluster][blocks];
    int v = __atomic_load_n(at, __ATOMIC_RELAXED);
    if (v == 0) {
        if (cluster == 1) {
            v = 152 * blocks;
        } else {
            const cudaError_t e = cudaOccupancyMaxActiveClusters(&v, sample_kernel<T, PROBS>, &cfg);
            if (e != cudaSuccess) return e;
        }
        __atomic_store_n(at, ++v, __ATOMIC_RELAXED);
    }
    *n = v - 1;
    return cudaSuccess;
}

template <typename T, bool PROBS>
cudaError_t sample_typed(const SampleArgs &a, cudaStream_t stream) {
    // Blocks a row: eight unless fewer give each at most 4096 elements (one alone 8192: 190 rows of that 7.9 us, by two 8.7), or
    // unless that is more than eight blocks an SM in all, two turns of four (192 rows of 131072 that ask for different
    // things: 62 us by eight blocks, 61 by four, 71 by two; for top-k alone 37, 30, 25; 48 rows 41, 58, 89).
    int cluster = 1;
    while (cluster < kMaxTCluster && a.V > (cluster == 1 ? 8192 : 4096 * cluster)) cluster *= 2;
    while (cluster > 2 && (long long)a.N * cluster > 1216) cluster /= 2;
    // a block's slice, as the kernel cuts it (rows that do not start on 16 bytes may take a group more)
    constexpr int VEC = 16 / sizeof(T);
    const long long groups = (a.V + (a.ld % VEC ? VEC - 1 : 0) + VEC - 1) / VEC;
    const long long per_warp = ((groups + cluster * kTWarps - 1) / (cluster * kTWarps) + 7) / 8 * 8;
    const long long slice = per_warp * kTWarps * 16;
    const int subs = cluster >= 8 ? 1 : cluster == 4 ? 2 : 4;
    const size_t fixed = (sizeof(TokenShared) + 15) / 16 * 16 + (cluster < 8 ? kList * 8 : 0) + subs * kTThreads * sizeof(float);
    static int configured[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!__atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE)) {
        e = cudaFuncSetAttribute(sample_kernel<T, PROBS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kMaxShared - 1024);
        if (e != cudaSuccess) return e;
        __atomic_store_n(&configured[dev], 1, __ATOMIC_RELEASE);
    }
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
    // No more blocks an SM than the call needs to run at once (the first are placed while the kernel before still holds
    // some of the SMs: four on one and one on the next took twice as long): all that these leave free is asked for,
    // and slices are kept that fit in it (one row of 131072 fp32 10.8 -> 9.5 us).
    auto room = [](int blocks) { return (size_t)(kMaxShared / blocks / 128 * 128 - 1024); };
    int blocks = 1;
    for (; blocks < kTBlocks; ++blocks) {
        int n = 0;
        cfg.dynamicSmemBytes = room(blocks);
        e = clusters_at_once<T, PROBS>(cfg, dev, cluster, blocks, &n);
        if (e != cudaSuccess) return e;
        if (n >= a.N) break;
    }
    cfg.dynamicSmemBytes = room(blocks);
    const int staged = slice <= (long long)(room(blocks) - fixed);
    return cudaLaunchKernelEx(&cfg, sample_kernel<T, PROBS>, a, cluster, staged, -0.0f);
}

cudaError_t launch_sample(const SampleArgs &a, bool probs, cudaStream_t stream) {
    if (a.bf16) return probs ? sample_typed<uint16_t, true>(a, stream) : sample_typed<uint16_t, false>(a, stream);
    return probs ? sample_typed<float, true>(a, stream) : sample_typed<float, false>(a, stream);
}

}  // namespace bsf8
