// bsf8_select.cu -- bounds of the cached pages' keys, and the pages of each request and cache head that
// a query's products with those bounds put first.
//
// A page's bounds are its keys' largest and smallest value in each channel, as 8-bit integers under a
// power of two per 32 channels (scoring a page by such bounds is a published idea), so that for any query q
//     q . k  <=  sum_d max(q_d, 0) hi_d + min(q_d, 0) lo_d     for every key k of the page.
// The score is that sum over all rows that share the cache head (heads of the group, nodes of the
// tree): with the rows' positive and negative parts added up first, one product of 2 dim terms a page
// whatever the rows.  Queries and bounds are integers in it and only a page's few block sums are added
// in fp32, in a fixed order: which pages come first depends on no order of threads.
#include "bsf8_device.cuh"
#include "bsf8_internal.h"

#include <algorithm>
#include <type_traits>

namespace bsf8 {

namespace {

constexpr int kBThreads = 256;
constexpr int kBMax = 1024;  // requests
constexpr int kBBlocks = 4;  // an SM
constexpr int kBAhead = 4;   // a lane's keys on their way (8 and 16 need registers that a fourth block has more of)

__device__ __forceinline__ uint32_t bmax2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t bmin2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// 2^(byte - 127), byte 0 .. 254.
__device__ __forceinline__ float pow2_byte(uint32_t byte) { return __uint_as_float(byte ? byte << 23 : 0x400000u); }

// Requests' page sums: items[b] pages before request b.
__device__ __forceinline__ int sum_pages(int v, int *wsum, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int up = v;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, up, m);
        if (lane >= m) up += o;
    }
    if (lane == 31) wsum[warp] = up;
    __syncthreads();
    int before = up - v;
    total = 0;
#pragma unroll
    for (int w = 0; w < kBThreads / 32; ++w) {
        if (w < warp) before += wsum[w];
        total += wsum[w];
    }
    return before;
}

}  // namespace

// ------------------------------------------------------------------------------------ bounds
// D / 16 lanes a key, 16 channels a lane (one 16-byte load), the keys' values rebuilt to bf16 -- exactly, they have four
// bits -- and their maxima and minima kept in pairs.  A warp's groups of lanes share the keys of one page where pages are
// few, and take a page each where all warps have enough of them and pages are short: then nothing goes from lane to lane.
// Bound by the ALU pipe: 13 instructions rebuild and compare four codes.  Three requests of 21843 tokens in all, 8 heads, dim
// 128, 36 MB: 11.1 us, 3.3 TB/s, 2 us of them prefix sums before the first load; 64 requests of 5000 tokens in pages of 16:
// 51 us, 3.7 TB/s (95 by a warp a page), of 4000 at dim 64 22 (67); 16 of 60000 in pages of 128: 90, 5.7 TB/s.
template <int D>
__global__ void __launch_bounds__(kBThreads, kBBlocks) bounds_kernel(const CacheView c, const BoundsView v, const int32_t *start,
                                                           const int32_t *end, int B, int *status) {
    __shared__ int s_first[kBMax], s_sum[kBMax + 1], s_w[kBThreads / 32];
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31;
    constexpr int PER = kBMax / kBThreads;
    {
        int n[PER], sum = 0;
        const long long capacity = (long long)v.table_pages * c.page_size;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int b = tid * PER + j;
            n[j] = 0;
            if (b < B) {
                const int from = start ? start[b] : 0, to = end[b];
                if (from < 0 || to < from || to > capacity) {
                    if (blockIdx.x == 0) report_index(status);
                } else {
                    s_first[b] = from / c.page_size;
                    n[j] = to / c.page_size - from / c.page_size;
                }
            }
            sum += n[j];
        }
        int total;
        int at = sum_pages(sum, s_w, total);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int b = tid * PER + j;
            if (b < B) s_sum[b] = at;
            at += n[j];
        }
        if (tid == 0) s_sum[B] = total;
    }
    __syncthreads();
    constexpr int LPR = D / 16, RP = 32 / LPR, EB = D / 32;  // lanes a key, keys a pass
    const int items = s_sum[B];
    const long long warps = (long long)gridDim.x * (kBThreads / 32), all = (long long)items * c.heads;
    int split = RP;  // groups of lanes that share a page's keys
    while (split > 1 && c.page_size < 16 * split && all * (split / 2) >= warps * RP) split /= 2;
    const int u = lane % LPR, part = lane / LPR % split, together = RP / split;
    for (long long it0 = ((long long)blockIdx.x * (kBThreads / 32) + (tid >> 5)) * together; it0 < all; it0 += warps * together) {
        const long long it = it0 + lane / LPR / split;
        const int pi = all < (1LL << 31) ? (int)it / c.heads : (int)(it / c.heads), h = (int)(it - (long long)pi * c.heads);
        int page = -1;
        if (it < all) {
            int lo = 0, hi = B;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_sum[mid] <= pi) lo = mid;
                else hi = mid;
            }
            page = v.table[(size_t)lo * v.table_pages + s_first[lo] + (pi - s_sum[lo])];
            if ((unsigned)page >= (unsigned)c.pages) {
                if (u == 0 && part == 0) report_index(status);
                page = -1;
            }
        }
        const size_t row0 = ((size_t)max(page, 0) * c.heads + h) * c.page_size;
        const uint8_t *const codes = c.k8 + row0 * D + 16 * u;
        const uint8_t *const exps = c.kexp + row0 * EB + u / 2;
        uint32_t mx[8], mn[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) mx[i] = 0xFF80FF80u, mn[i] = 0x7F807F80u;  // -inf, +inf
        uint32_t nan = 0;
        // keys k, k + split, ..: their loads together on their way
        auto keys = [&](int k, auto count) {
            constexpr int K = decltype(count)::value;
            uint4 w[K];
            uint32_t e[K];
#pragma unroll
            for (int j = 0; j < K; ++j) {
                w[j] = *reinterpret_cast<const uint4 *>(codes + (size_t)(k + j * split) * D);
                e[j] = exps[(size_t)(k + j * split) * EB];
            }
#pragma unroll
            for (int j = 0; j < K; ++j) {
                nan |= e[j] == 255 ? 1u : 0u;
                const Scale sc = make_scale(e[j]);
                const uint32_t ws[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t a, b;
                    rebuild4(ws[i], sc, a, b);
                    mx[2 * i] = bmax2(mx[2 * i], a);
                    mn[2 * i] = bmin2(mn[2 * i], a);
                    mx[2 * i + 1] = bmax2(mx[2 * i + 1], b);
                    mn[2 * i + 1] = bmin2(mn[2 * i + 1], b);
                }
            }
        };
        if (page >= 0) {
            int k = part, left = c.page_size / split;  // even: a page is a multiple of 16 keys, split at most 8
            for (; left >= kBAhead; left -= kBAhead, k += kBAhead * split) keys(k, std::integral_constant<int, kBAhead>());
            if (left & 2) keys(k, std::integral_constant<int, 2>());
        }
        __syncwarp();
        for (int m = LPR; m < LPR * split; m <<= 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                mx[i] = bmax2(mx[i], __shfl_xor_sync(0xFFFFFFFFu, mx[i], m));
                mn[i] = bmin2(mn[i], __shfl_xor_sync(0xFFFFFFFFu, mn[i], m));
            }
            nan |= __shfl_xor_sync(0xFFFFFFFFu, nan, m);
        }
        // the largest magnitude of the block's 32 channels, and whether any of its keys is marked NaN: this lane's and
        // its neighbour's
        uint32_t am = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            am = max(am, max((mx[i] << 16) & 0x7FFFFFFFu, mx[i] & 0x7FFF0000u));
            am = max(am, max((mn[i] << 16) & 0x7FFFFFFFu, mn[i] & 0x7FFF0000u));
        }
        am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
        nan |= __shfl_xor_sync(0xFFFFFFFFu, nan, 1);
        if (page < 0) continue;
        // 127 = 1.984375 * 2^6: adding 0x1FFFF carries into the exponent past that mantissa
        uint32_t e = (uint32_t)max(0, (int)((am + 0x1FFFFu) >> 23) - 6);
        const bool none = nan != 0 || am >= 0x7F800000u;
        if (none) e = 255;
        const float inv = none ? 0.0f : __uint_as_float((254u - e) << 23);  // 2^(127 - e)
        const size_t at = (size_t)page * v.heads + h;
#pragma unroll
        for (int which = 0; which < 2; ++which) {  // maxima, minima: by the page's first two groups of lanes, or its one
            if (split > 1 && part != which) continue;
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                o[i] = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t w = which == 0 ? mx[2 * i + j / 2] : mn[2 * i + j / 2];
                    const float x = j & 1 ? hi16(w) : lo16(w);
                    float y = x * inv;
                    if (y == 0.0f) y = x;  // too small a part for fp32: as far from 0 as its sign says
                    const int q = none ? 0 : (int)(which == 0 ? ceilf(y) : floorf(y));
                    o[i] |= (uint32_t)(q & 255) << (8 * j);
                }
            }
            *reinterpret_cast<uint4 *>(v.codes + (at * 2 + which) * D + 16 * u) = make_uint4(o[0], o[1], o[2], o[3]);
            if (which == 0 && (u & 1) == 0) v.exps[at * EB + u / 2] = (uint8_t)e;
        }
    }
}

cudaError_t launch_bounds(const CacheView &c, const BoundsView &v, const int32_t *start, const int32_t *end, int B,
                          cudaStream_t stream) {
    int *status = status_word();
    if (!status) return cudaErrorInvalidSymbol;
    cudaLaunchConfig_t cfg = {};
    const long long most = (long long)B * v.table_pages * v.heads;
    cfg.gridDim = dim3((unsigned)std::min<long long>((most + 7) / 8, 152 * kBBlocks), 1, 1);
    cfg.blockDim = dim3(kBThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = options().pdl ? 1 : 0;
    switch (c.dim) {
        case 64: return cudaLaunchKernelEx(&cfg, bounds_kernel<64>, c, v, start, end, B, status);
        case 128: return cudaLaunchKernelEx(&cfg, bounds_kernel<128>, c, v, start, end, B, status);
        case 256: return cudaLaunchKernelEx(&cfg, bounds_kernel<256>, c, v, start, end, B, status);
        default: return cudaErrorInvalidValue;
    }
}

// ------------------------------------------------------------------------------------ selection
// A cluster of blocks a request and cache head.  Every block adds up the rows' queries (integers: any
// order), scores its share of the pages and puts their keys -- the scores' bits, ordered as integers --
// into the first block's shared memory, which then finds the key of rank `keep` by digits of what the
// keys differ in, and writes the pages before it, ties by their index, in ascending order.
// Bounds come by asynchronous copies, 8 KB a warp on their way: two blocks an SM at 128 registers keep what a lane's
// two chains of products need (three at 80 spilled: 32 requests 21.7 us for 16).  32 requests of up to 65536 tokens, 8
// heads: 16 us with the bounds (34 MB) in L2, 23 without, of which DRAM is 5; one of 131072: 10, the chain of loads (lengths,
// table, bounds), the queries' four barriers, a turn of products (1.5), the cluster's barrier, the digits (2) and the list (1.5).
// Rows of queries cost each block of the cluster the same: 512 of them at dim 128 9 us (16 by conversions and a division a row).
namespace {

constexpr int kSThreads = 256, kSWarps = kSThreads / 32;
constexpr int kMaxSCluster = 8;
constexpr int kSBins = 2048, kSBinsEach = kSBins / kSThreads;
constexpr uint32_t kTopKey = 0xFF800000u;  // of +inf

struct SelectShared {
    alignas(16) int q[2][256];  // sums of the rows' positive and negative parts; then their bytes
    int red[kSWarps], wsum[kSWarps];
    uint32_t lo, hi;            // smallest and largest key below the top one
    int top;                    // keys that are the top one
    int want, digit, count;
};

__device__ __forceinline__ int dp4a_ss(uint32_t a, uint32_t b, int c) {
    int d;
    asm("dp4a.s32.s32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

__device__ __forceinline__ int dp4a_su(uint32_t a, uint32_t b, int c) {
    int d;
    asm("dp4a.s32.u32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// 16 bytes, or zeros where `bytes` is 0 (then nothing is read).
__device__ __forceinline__ void async16(void *dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}

// A page's exponent bytes of a head, held by one lane; byte(word, lane, i): byte i of what `lane` holds.
template <int EB>
struct ExpWord {
    typedef typename std::conditional<EB == 2, uint16_t, uint32_t>::type T;
    static __device__ __forceinline__ uint32_t byte(T w, int lane, int i) { return __shfl_sync(0xFFFFFFFFu, (uint32_t)w, lane) >> 8 * i & 255u; }
};
template <>
struct ExpWord<8> {
    typedef uint2 T;
    static __device__ __forceinline__ uint32_t byte(uint2 w, int lane, int i) {
        const uint32_t x = __shfl_sync(0xFFFFFFFFu, w.x, lane), y = __shfl_sync(0xFFFFFFFFu, w.y, lane);
        return (i < 4 ? x : y) >> 8 * (i & 3) & 255u;
    }
};

// Larger keys for larger scores; equal ones for 0 and -0.  None above kTopKey: a NaN (infinities of both signs added up,
// which exponents that kv_bounds does not write can give) has that of +inf, or more pages than `keep` would be listed.
__device__ __forceinline__ uint32_t key_of(float f) {
    if (!(f < INFINITY)) return kTopKey;
    const uint32_t b = __float_as_uint(f + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

}  // namespace

// How a warp goes through its pages: PAGES a turn, in BATCHES of 2 KB.  Four copies of 16 bytes a lane bring a batch to
// shared memory, whole sectors at a time; there a lane takes all of 32 channels, LPP lanes a page.
template <int D>
struct Turn {
    static constexpr int LPP = D / 32, PPB = 32 / LPP;  // lanes a page, pages a batch
    static constexpr int PAGES = D == 256 ? 16 : 32, BATCHES = PAGES / PPB;
    static constexpr int CHUNKS = D / 8;                // of 16 bytes a page
    static constexpr int BLOCK = kSWarps * 2048;
    // where chunk c of a batch's page lies: eight lanes that read theirs at once touch all banks
    static __device__ __forceinline__ int at(int page, int c) {
        return page * CHUNKS + (D == 64 ? c ^ ((page & 1) | (page & 2) << 1) : D == 128 ? c ^ (page & 1) : c ^ (c >> 3 & 1));
    }
};

// `depth` batches of a warp (2 or 4, no more than a turn's) are on their way at a time.
template <int D>
__global__ void __launch_bounds__(kSThreads, 2) select_kernel(const BoundsView v, const SelectArgs a, int cluster, int depth, int *status) {
    using W = Turn<D>;
    __shared__ SelectShared s;
    extern __shared__ __align__(16) uint8_t select_memory[];
    static_assert(W::BLOCK >= kSBins * 4, "the histogram lies there after the scores");
    uint8_t *const batches = select_memory;
    int *const hist = reinterpret_cast<int *>(select_memory);  // counts of the keys; then the chosen pages, where that many suffice
    uint32_t *const keys = reinterpret_cast<uint32_t *>(select_memory + depth * W::BLOCK);
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = blockIdx.x % cluster, pair = blockIdx.x / cluster;
    const int b = pair / v.heads, h = pair - b * v.heads, g = a.Hq / v.heads;
    const int P = v.page_size;
    int ctx = a.ctx[b], nodes = a.nodes ? a.nodes[b] : a.T;
    if (ctx < 0 || nodes < 0 || nodes > a.T || (long long)ctx + nodes > a.max_len) {
        if (tid == 0 && rank == 0) report_index(status);
        ctx = max(0, min(ctx, a.max_len));
        nodes = max(0, min(nodes, min(a.T, a.max_len - ctx)));
    }
    const int full = ctx / P, n = min(a.keep, full);
    const int32_t *const table = v.table + (size_t)b * v.table_pages;
    int32_t *const out = a.pages + (size_t)pair * a.width;
    const bool choose = full > a.keep;  // else all of them stay
    if (cluster > 1) cluster_arrive();  // the first block's memory may be written once it runs

    if (choose) {
        // a lane each asks for a page's entry and exponents, then its bounds come, batches on their way while earlier ones are
        // multiplied; the first before the queries are looked at
        constexpr int LPP = W::LPP, PPB = W::PPB, PAGES = W::PAGES, EB = D / 32;
        using Word = typename ExpWord<EB>::T;
        const int blk = lane % LPP;
        const int first = (rank * kSWarps + warp) * PAGES, stride = cluster * kSWarps * PAGES;
        uint8_t *const mine = batches + warp * depth * 2048;
        auto entry = [&](int p) { return lane < PAGES && p + lane < full ? table[p + lane] : -1; };
        auto row_of = [&](int page) { return (unsigned)page < (unsigned)v.pages ? page * v.heads + h : -1; };
        auto word_of = [&](int row) { return row >= 0 ? reinterpret_cast<const Word *>(v.exps)[row] : Word{}; };
        // two batches of a turn's rows, `sub` the first
        auto ask = [&](int row, int sub) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int in = (lane + 32 * (j & 3)) / W::CHUNKS, c = (lane + 32 * (j & 3)) % W::CHUNKS;
                const int from = __shfl_sync(0xFFFFFFFFu, row, PPB * (sub + j / 4) + in);
                async16(mine + ((sub + j / 4) & (depth - 1)) * 2048 + 16 * W::at(in, c), v.codes + (size_t)max(from, 0) * 2 * D + 16 * c,
                        from >= 0 ? 16u : 0u);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        int row = row_of(entry(first));
        // ---------------------------------------------------------- the rows' queries
        constexpr int LPQ = D / 8;  // 16-byte pieces a row
        const int rows = nodes * g, u = tid % LPQ;
        const float inv_g = 1.0f / (float)g;
        auto piece = [&](int r) {
            const int t = (int)(((float)r + 0.5f) * inv_g);  // r / g: both below 2^13
            return *reinterpret_cast<const uint4 *>(a.q + ((size_t)b * a.T + t) * a.ldq + (size_t)(h * g + r - t * g) * D + 8 * u);
        };
        for (int i = tid; i < 2 * D; i += kSThreads) s.q[i / D][i % D] = 0;
        // f(piece) of this thread's rows, four on their way; the first ones stay for the second turn
        constexpr int RPP = kSThreads / LPQ;  // rows at a time
        const int r0 = tid / LPQ;
        constexpr int KEPT = 4;
        uint4 kept[KEPT];
#pragma unroll
        for (int j = 0; j < KEPT; ++j)
            if (r0 + j * RPP < rows) kept[j] = piece(r0 + j * RPP);
        Word word = word_of(row);
        for (int i = 0; i < depth; i += 2) ask(row, i);
        int next = entry(first + stride);
        auto each = [&](auto f) {
#pragma unroll
            for (int j = 0; j < KEPT; ++j)
                if (r0 + j * RPP < rows) f(kept[j]);
            for (int r = r0 + KEPT * RPP; r < rows; r += 4 * RPP) {
                uint4 w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (r + j * RPP < rows) w[j] = piece(r + j * RPP);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (r + j * RPP < rows) f(w[j]);
            }
        };
        auto block_max = [&](uint32_t v) {
            v = __reduce_max_sync(0xFFFFFFFFu, v);
            if (lane == 0) s.red[warp] = (int)v;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kSWarps; ++w) v = max(v, (uint32_t)s.red[w]);
            return v;
        };
        uint32_t am = 0;  // two magnitudes at a time
        each([&](const uint4 &w) {
            am = __vmaxu2(__vmaxu2(am, w.x & 0x7FFF7FFFu), w.y & 0x7FFF7FFFu);
            am = __vmaxu2(__vmaxu2(am, w.z & 0x7FFF7FFFu), w.w & 0x7FFF7FFFu);
        });
        am = block_max(max(am & 0xFFFFu, am >> 16));
        const bool finite = am < 0x7F80u;
        if (!finite) {  // again without what is infinite or NaN
            am = 0;
            each([&](const uint4 &w) {
                const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t lo = x[i] & 0x7FFFu, hi = (x[i] >> 16) & 0x7FFFu;
                    am = max(am, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
                }
            });
            __syncthreads();
            am = block_max(am);
        }
        // the largest to [2^17, 2^18); it counts as 2^-100 at least
        const int k = max((int)(am >> 7) - 127, -100);
        const float scale = __uint_as_float((uint32_t)(127 + 17 - k) << 23);
        // The integers by adding 1.5 * 2^23, which rounds as rint does and leaves them in the low bits; what that adds to
        // the sums (modulo 2^32) goes off at the end.  up: of the positive ones, dn: of all, then of the rest.
        constexpr float kRound = 12582912.0f;
        const uint32_t zero = __float_as_uint(kRound);
        uint32_t up[8] = {}, dn[8] = {}, count = 0;
        each([&](const uint4 &w) {
            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
            ++count;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t bits = i & 1 ? x[i / 2] & 0xFFFF0000u : x[i / 2] << 16;
                if (!finite && (bits & 0x7F800000u) == 0x7F800000u) bits = 0;
                const uint32_t z = __float_as_uint(__fmaf_rn(__uint_as_float(bits), scale, kRound));
                up[i] += max(z, zero);
                dn[i] += z;
            }
        });
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            up[i] -= count * zero;
            dn[i] -= count * zero + up[i];
        }
#pragma unroll
        for (int m = LPQ; m < 32; m <<= 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                up[i] += __shfl_xor_sync(0xFFFFFFFFu, up[i], m);
                dn[i] += __shfl_xor_sync(0xFFFFFFFFu, dn[i], m);
            }
        }
        if (lane < LPQ && warp * 32 / LPQ < rows) {  // warps that had rows
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (up[i]) atomicAdd(&s.q[0][8 * u + i], (int)up[i]);
                if (dn[i]) atomicAdd(&s.q[1][8 * u + i], (int)dn[i]);
            }
        }
        __syncthreads();
        uint32_t big = 0;  // (every warp for itself)
#pragma unroll
        for (int i = 0; i < 2 * D; i += 32) big = max(big, (uint32_t)abs(s.q[(i + lane) / D][(i + lane) % D]));
        big = __reduce_max_sync(0xFFFFFFFFu, big);
        const int sh = max(0, 32 - __clz(big) - 14), half = (1 << sh) >> 1;
        // ---------------------------------------------------------- scores
        // the sums in two bytes, high and low, four channels a word, where the sums were
        uint32_t high = 0, low = 0;
        if (tid < 2 * D / 4) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int z = (s.q[4 * tid / D][4 * tid % D + j] + half) >> sh;  // |z| <= 2^14
                high |= (uint32_t)((z >> 8) & 255) << (8 * j);
                low |= (uint32_t)(z & 255) << (8 * j);
            }
        }
        __syncthreads();
        if (tid < 2 * D / 4) {
            s.q[0][tid] = (int)high;
            s.q[1][tid] = (int)low;
        }
        __syncthreads();
        uint4 qh[4], ql[4];  // of this lane's 32 channels: against the maxima, then against the minima
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = (i / 2 * D + 32 * blk + 16 * (i & 1)) / 4;
            qh[i] = *reinterpret_cast<const uint4 *>(&s.q[0][at]);
            ql[i] = *reinterpret_cast<const uint4 *>(&s.q[1][at]);
        }
        if (cluster > 1) cluster_wait();
        const uint32_t keys0 = cluster > 1 ? map_to_rank(keys, 0) : 0;
        for (int p0 = first; p0 < full; p0 += stride) {
            const int ahead = row_of(next), after = entry(p0 + 2 * stride);
            const Word later = word_of(ahead);
            if (row < 0 && lane < PAGES && p0 + lane < full) report_index(status);  // no such page
#pragma unroll 1
            for (int sub = 0; sub < W::BATCHES; sub += 2) {
                if (depth == 4) asm volatile("cp.async.wait_group 1;" ::: "memory");
                else asm volatile("cp.async.wait_group 0;" ::: "memory");
                __syncwarp();
                // two batches side by side: what their chains take adds up otherwise
                int S[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint8_t *const batch = mine + ((sub + k) & (depth - 1)) * 2048;
                    int high[2] = {}, low[2] = {};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 w = *reinterpret_cast<const uint4 *>(batch + 16 * W::at(lane / LPP, i / 2 * (D / 16) + 2 * blk + (i & 1)));
                        int &H = high[i & 1], &L = low[i & 1];
                        H = dp4a_ss(w.x, qh[i].x, H), L = dp4a_su(w.x, ql[i].x, L);
                        H = dp4a_ss(w.y, qh[i].y, H), L = dp4a_su(w.y, ql[i].y, L);
                        H = dp4a_ss(w.z, qh[i].z, H), L = dp4a_su(w.z, ql[i].z, L);
                        H = dp4a_ss(w.w, qh[i].w, H), L = dp4a_su(w.w, ql[i].w, L);
                    }
                    S[k] = (high[0] + high[1]) * 256 + low[0] + low[1];  // |S| < 2^27
                }
                __syncwarp();
                ask(sub + depth < W::BATCHES ? row : ahead, (sub + depth) & (W::BATCHES - 1));
                float f[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t byte = ExpWord<EB>::byte(word, PPB * (sub + k) + lane / LPP, blk);
                    f[k] = byte == 255 ? INFINITY : __fmul_rn(__fmul_rn((float)S[k], 7.450580596923828e-9f), pow2_byte(byte));
                }
#pragma unroll
                for (int m = 1; m < LPP; m <<= 1) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) f[k] = __fadd_rn(f[k], __shfl_xor_sync(0xFFFFFFFFu, f[k], m));
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int i = PPB * (sub + k) + lane / LPP, p = p0 + i;
                    uint32_t key = __shfl_sync(0xFFFFFFFFu, row, i) < 0 ? 0 : key_of(f[k]);
                    if (p < a.sink || p >= full - a.recent) key = kTopKey;
                    if (blk != 0 || p >= full) continue;
                    if (cluster > 1) st_cluster_u32(keys0 + 4 * p, key);
                    else keys[p] = key;
                }
            }
            row = ahead;
            next = after;
            word = later;
        }
        // what was asked for past the last page writes zeros, and that memory is the histogram's next
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (cluster > 1) {
        cluster_wait();
    }
    if (cluster > 1) cluster_barrier();
    else __syncthreads();
    if (rank != 0) return;

    // -------------------------------------------------------------- the pages
    if (!choose) {
        for (int p = tid; p < n; p += kSThreads) out[p] = table[p];
    } else {
        uint32_t lo = 0xFFFFFFFFu, hi = 0;
        int top = 0;
        for (int p = tid; p < full; p += kSThreads) {
            const uint32_t x = keys[p];
            if (x >= kTopKey) {
                ++top;
            } else {
                lo = min(lo, x);
                hi = max(hi, x);
            }
        }
        if (tid == 0) s.lo = 0xFFFFFFFFu, s.hi = 0, s.top = 0;
        for (int i = tid; i < kSBins; i += kSThreads) hist[i] = 0;
        __syncthreads();
        lo = __reduce_min_sync(0xFFFFFFFFu, lo);
        hi = __reduce_max_sync(0xFFFFFFFFu, hi);
        top = __reduce_add_sync(0xFFFFFFFFu, top);
        if (lane == 0) {
            atomicMin(&s.lo, lo);
            atomicMax(&s.hi, hi);
            if (top) atomicAdd(&s.top, top);
        }
        __syncthreads();
        // keys above `key` stay, and the first `equal` of those that have it
        uint32_t key;
        int equal;
        if (s.top >= n) {
            key = kTopKey;
            equal = n;
        } else {
            lo = s.lo;
            uint32_t base = 0, most = s.hi - lo;  // keys - lo of [base, base + most] are in question
            int want = n - s.top;
            while (true) {  // 11 bits of them a turn, until a bin's keys are all wanted
                const int shift = max(0, 32 - __clz(most) - 11);
                for (int p = tid; p < full; p += kSThreads) {
                    const uint32_t x = keys[p];
                    if (x < kTopKey && x - lo >= base && x - lo - base <= most) atomicAdd(&hist[kSBins - 1 - ((x - lo - base) >> shift)], 1);
                }
                __syncthreads();
                // bins from the top, some a thread
                int c[kSBinsEach], sum = 0;
#pragma unroll
                for (int i = 0; i < kSBinsEach; ++i) sum += c[i] = hist[kSBinsEach * tid + i];
                int upto = sum;
#pragma unroll
                for (int m = 1; m < 32; m <<= 1) {
                    const int o = __shfl_up_sync(0xFFFFFFFFu, upto, m);
                    if (lane >= m) upto += o;
                }
                if (lane == 31) s.wsum[warp] = upto;
                __syncthreads();
                int before = upto - sum;
#pragma unroll
                for (int w = 0; w < kSWarps; ++w) before += w < warp ? s.wsum[w] : 0;
#pragma unroll
                for (int i = 0; i < kSBinsEach; ++i) {
                    if (before < want && before + c[i] >= want) {
                        s.digit = kSBins - 1 - (kSBinsEach * tid + i);
                        s.want = want - before;
                        s.count = c[i];
                    }
                    before += c[i];
                    hist[kSBinsEach * tid + i] = 0;  // for the next turn
                }
                __syncthreads();
                base += (uint32_t)s.digit << shift;
                want = s.want;
                if (shift == 0 || want == s.count) break;
                most = (1u << shift) - 1u;
                __syncthreads();
            }
            // all of the bin's keys: those from its start on (which is not 0: then all pages would stay)
            const bool all = want == s.count;
            key = all ? lo + base - 1 : lo + base;
            equal = all ? 0 : want;
        }
        // in ascending order: a thread takes a run of pages
        const int run = ((full + kSThreads - 1) / kSThreads) | 1;  // odd: no two lanes on a bank
        const int p0 = min(full, tid * run), p1 = min(full, p0 + run);
        uint32_t c = 0;  // above, equal: 16 bits each
        for (int p = p0; p < p1; ++p) c += keys[p] > key ? 0x10000u : keys[p] == key ? 1u : 0u;
        uint32_t upto = c;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, upto, m);
            if (lane >= m) upto += o;
        }
        if (lane == 31) s.red[warp] = (int)upto;
        __syncthreads();
        upto -= c;
#pragma unroll
        for (int w = 0; w < kSWarps; ++w) upto += w < warp ? (uint32_t)s.red[w] : 0u;
        int above = (int)(upto >> 16), same = (int)(upto & 0xFFFFu);
        const bool listed = n <= kSBins;  // then their entries are asked for at once
        auto put = [&](int at, int p) {
            if (listed) hist[at] = p;
            else out[at] = table[p];
        };
        if (c)
            for (int p = p0; p < p1; ++p) {
                if (keys[p] > key) {
                    put(above++ + min(same, equal), p);
                } else if (keys[p] == key) {
                    if (same < equal) put(above + same, p);
                    ++same;
                }
            }
        if (listed) {
            __syncthreads();
            for (int i = tid; i < n; i += kSThreads) out[i] = table[hist[i]];
        }
    }
    // the pages of the tail and of the nodes, then none
    const int last = (int)(((long long)ctx + nodes + P - 1) / P);
    for (int i = n + tid; i < a.width; i += kSThreads) {
        const int p = full + (i - n);
        out[i] = p < last && p < v.table_pages ? table[p] : -1;
    }
    if (h == 0 && tid == 0) a.kept[b] = n * P + (ctx - full * P);
}

template <int D>
cudaError_t select_dim(const BoundsView &v, const SelectArgs &a, cudaStream_t stream, int *status) {
    constexpr int kMost = 224 * 1024;  // dynamic shared memory
    static_assert(kMaxSelectPages * 4 + 2 * Turn<D>::BLOCK <= kMost && kMost + sizeof(SelectShared) <= 227 * 1024, "two batches fit with the most keys");
    const int most = std::min(v.table_pages, a.max_len / v.page_size);
    int depth = Turn<D>::BATCHES;
    while (depth > 2 && most * 4 + depth * Turn<D>::BLOCK > kMost) depth /= 2;
    const size_t smem = (size_t)most * 4 + depth * Turn<D>::BLOCK;
    static int configured[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!__atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE)) {
        e = cudaFuncSetAttribute(select_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
        if (e != cudaSuccess) return e;
        __atomic_store_n(&configured[dev], 1, __ATOMIC_RELEASE);
    }
    // blocks a pair: as many as run at once, with 128 pages each at least where the request is longest
    const long long pairs = (long long)a.B * v.heads;
    const long long resident = 152LL * std::max<size_t>(1, std::min<size_t>(2, 228 * 1024 / (smem + sizeof(SelectShared) + 1024)));
    int cluster = 1;
    while (cluster < kMaxSCluster && 2 * cluster * pairs <= resident && most > 128 * cluster) cluster *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(pairs * cluster), 1, 1);
    cfg.blockDim = dim3(kSThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
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
    return cudaLaunchKernelEx(&cfg, select_kernel<D>, v, a, cluster, depth, status);
}

cudaError_t launch_select(const BoundsView &v, const SelectArgs &a, cudaStream_t stream) {
    int *status = status_word();
    if (!status) return cudaErrorInvalidSymbol;
    switch (v.dim) {
        case 64: return select_dim<64>(v, a, stream, status);
        case 128: return select_dim<128>(v, a, stream, status);
        case 256: return select_dim<256>(v, a, stream, status);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace bsf8
