// bsf8_cache.cu -- the paged key/value cache: append (with the per-head norm and the
// rotation in the same pass), read back, and the commit of a token tree's kept nodes.
//
// A cached row (token, head) is dim e4m3 codes and dim / 32 exponent bytes, one per 32
// channels, chosen as make_twin_rows chooses them.  All three move each byte once and are
// bound by HBM at prompt sizes (the append by instruction issue too), by launch and load latency at
// decode sizes.
#include "bsf8_device.cuh"
#include "bsf8_internal.h"

#include <algorithm>

namespace bsf8 {

// Loads here are plain ones, not the read-only path (__ldg, __restrict__): the compiler may
// move those above the dependency wait, and everything these kernels read may have been
// written by the kernel before.

namespace {

template <typename... Params, typename... Args>
cudaError_t launch_cache(void (*kernel)(Params...), long long blocks, int threads, cudaStream_t stream,
                         Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min(blocks, 1LL << 30), 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = options().pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

// Row (page, head, offset) of a token in the cache's arrays, for head 0; negative where an
// index leaves its table.  Heads are page_size rows apart.
__device__ __forceinline__ long long cache_row(const CacheView &c, int req, int slot) {
    if ((unsigned)req >= (unsigned)c.requests || slot < 0) return -1;
    const int pi = slot / c.page_size;
    if (pi >= c.table_pages) return -1;
    const int page = *(c.table + (size_t)req * c.table_pages + pi);
    if ((unsigned)page >= (unsigned)c.pages) return -1;
    return ((long long)page * c.heads) * c.page_size + (slot - pi * c.page_size);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

__device__ __forceinline__ void unpack8(const uint4 &w, float (&y)[8]) {
    y[0] = bf16_lo(w.x); y[1] = bf16_hi(w.x);
    y[2] = bf16_lo(w.y); y[3] = bf16_hi(w.y);
    y[4] = bf16_lo(w.z); y[5] = bf16_hi(w.z);
    y[6] = bf16_lo(w.w); y[7] = bf16_hi(w.w);
}

}  // namespace

// -------------------------------------------------------------------- append
//
// D / 8 lanes hold a row, 8 channels a lane (one 16-byte load): the norm's sum is a shuffle
// tree over them, a rotation partner of the split form sits rot / 16 lanes away, and the
// four lanes of a 32-channel block share its exponent.  A row is (token, q | k | v, head); a
// token's rows are numbered q heads, k heads, v heads.

// A block takes up to kTokens consecutive tokens and, by blockIdx.y, 256 / LPR rows of each: a lane
// group has one row number throughout, so that from token to token only addresses move on.  The
// tokens' places and positions are looked up once, by a thread a token, while the first rows are on
// their way; kAhead rows a lane group stay in flight.  (Looking them up in every lane group cost more
// instructions than the norm, the rotation and the rounding together.)  What hides latency best is warps:
// five blocks an SM with a row ahead 41 us, four with one 45, with two 45, six with one 43.
// In a graph, 8191 tokens of 32 + 8 + 8 heads of 128: 41 us, 4.5 TB/s of the 185 MB that it must move (0.66 of the
// measured HBM rate; some 150 instructions for two rows a warp); 63 tokens: 3 us.
constexpr int kTokens = 64, kAhead = 1, kAppendBlocks = 5;

template <int D>
__global__ void __launch_bounds__(256, kAppendBlocks) append_kernel(const CacheView c, const AppendArgs a, int tokens, int *status) {
    __shared__ long long s_row[kTokens];  // cache row of head 0; -1: not kept
    __shared__ int s_pos[kTokens];        // -1: the token is left out
    pdl_trigger();
    pdl_wait();
    constexpr int LPR = D / 8;
    const int sub = threadIdx.x % LPR, lane = threadIdx.x & 31;
    const uint32_t gmask = LPR == 32 ? 0xFFFFFFFFu : ((1u << LPR) - 1u) << (lane - sub);
    const int c0 = sub * 8;  // this lane's first channel
    const int n0 = (int)blockIdx.x * tokens, count = min(tokens, a.N - n0);
    // the row: query, key or value head
    int r = (int)blockIdx.y * (256 / LPR) + threadIdx.x / LPR;
    const bool real = r < a.Hq + 2 * c.heads;
    const int kind = !real ? 3 : r < a.Hq ? 0 : r < a.Hq + c.heads ? 1 : 2;
    r -= kind == 0 ? 0 : kind == 1 ? a.Hq : a.Hq + c.heads;
    const long long ld = kind == 0 ? a.ldq : kind == 1 ? a.ldk : a.ldv;
    const uint16_t *src = (kind == 0 ? a.q : kind == 1 ? a.k : a.v) + (size_t)r * D + c0 + n0 * ld;
    uint4 w[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
        if (real && j < count) w[j] = *reinterpret_cast<const uint4 *>(src + j * ld);
    if (threadIdx.x < count) {
        const int n = n0 + threadIdx.x;
        const int slot = a.slot[n], req = a.req[n], pos = a.rot > 0 ? a.pos[n] : 0;
        const bool good = a.rot == 0 || (unsigned)pos < (unsigned)a.positions;
        const long long row = slot < 0 ? -1 : cache_row(c, req, slot);
        if (!good || (row < 0 && slot >= 0)) report_index(status);
        s_row[threadIdx.x] = row;
        s_pos[threadIdx.x] = good ? pos : -1;
    }
    __syncthreads();
    if (!real) return;
    src += kAhead * ld;
    uint16_t *out = a.q_out + ((size_t)n0 * a.Hq + r) * D + c0;
    uint8_t *const codes_at = (kind == 1 ? c.k8 : c.v8) + (size_t)r * c.page_size * D + c0;
    uint8_t *const exps_at = (kind == 1 ? c.kexp : c.vexp) + (size_t)r * c.page_size * (D / 32) + c0 / 32;
    const uint16_t *const nw = kind == 0 ? a.q_norm : kind == 1 ? a.k_norm : nullptr;
    float g[8];
    if (nw) unpack8(*reinterpret_cast<const uint4 *>(nw + c0), g);
    const int half = a.rot / 2;
    const bool turns = kind < 2 && a.rot > 0, turned = turns && c0 < a.rot;
    const float *const angles = a.cos_sin + (a.interleaved ? c0 / 2 : (c0 < half ? c0 : c0 - half));
    const int from = !turned ? lane : c0 < half ? lane + half / 8 : lane - half / 8;  // split form's partner

    for (int t0 = 0; t0 < count; t0 += kAhead) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int t = t0 + j;
            if (t >= count) break;  // uniform over the block
            float y[8];
            unpack8(w[j], y);
            if (t + kAhead < count) w[j] = *reinterpret_cast<const uint4 *>(src);
            src += ld;
            const int pos = s_pos[t];
            if (pos >= 0) {
                if (nw) {
                    float ss = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
                    for (int k = LPR / 2; k > 0; k >>= 1) ss += __shfl_xor_sync(gmask, ss, k);
                    const float s = rsqrtf(fmaf(ss, 1.0f / D, a.eps));
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = y[i] * s * g[i];
                }
                if (turns) {
                    const float *const at = angles + (size_t)pos * a.rot;
                    if (a.interleaved) {
                        if (turned) {
                            const float4 x = *reinterpret_cast<const float4 *>(at);
                            const float4 z = *reinterpret_cast<const float4 *>(at + half);
                            const float cs[4] = {x.x, x.y, x.z, x.w}, sn[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float u = y[2 * i], v = y[2 * i + 1];
                                y[2 * i] = u * cs[i] - v * sn[i];
                                y[2 * i + 1] = v * cs[i] + u * sn[i];
                            }
                        }
                    } else {  // the partner channel is rot / 2 away; its sine counts negative below it
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float4 x = make_float4(1, 1, 1, 1), z = make_float4(0, 0, 0, 0);
                            if (turned) {
                                x = *reinterpret_cast<const float4 *>(at + 4 * k);
                                z = *reinterpret_cast<const float4 *>(at + half + 4 * k);
                            }
                            const float cs[4] = {x.x, x.y, x.z, x.w}, sn[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float o = __shfl_sync(gmask, y[4 * k + i], from);
                                const float u = fmaf(y[4 * k + i], cs[i], c0 < half ? -o * sn[i] : o * sn[i]);
                                if (turned) y[4 * k + i] = u;  // else as it is: an infinity times 0 is none
                            }
                        }
                    }
                }
                if (kind == 0) {
                    *reinterpret_cast<uint4 *>(out) = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]),
                                                                 pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
                } else {
                    uint32_t am = 0;  // magnitude bits order as magnitudes do, NaN above infinity
#pragma unroll
                    for (int i = 0; i < 8; ++i) am = max(am, __float_as_uint(y[i]) & 0x7FFFFFFFu);
                    am = max(am, __shfl_xor_sync(gmask, am, 1));
                    am = max(am, __shfl_xor_sync(gmask, am, 2));
                    // 448 = 1.75 * 2^8: adding 0x1FFFFF carries into the exponent past mantissa 0.75
                    int e = max(0, (int)((am + 0x1FFFFFu) >> 23) - 8);
                    uint2 codes;
                    if (am >= 0x7F800000u) {
                        e = 255;
                        codes = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
                    } else {
                        const float inv = __uint_as_float((uint32_t)(254 - e) << 23);  // 2^(127 - e), exact products
                        codes = make_uint2(pack_e4m3(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                                           pack_e4m3(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
                    }
                    const long long row = s_row[t];
                    if (row >= 0) {
                        *reinterpret_cast<uint2 *>(codes_at + row * D) = codes;
                        if ((sub & 3) == 0) exps_at[row * (D / 32)] = (uint8_t)e;
                    }
                }
            }
            out += (size_t)a.Hq * D;
        }
    }
}

template <int D>
cudaError_t append_dim(const CacheView &c, const AppendArgs &a, cudaStream_t stream, int *status) {
    constexpr int G = 256 / (D / 8);
    const int chunks = (a.Hq + 2 * c.heads + G - 1) / G;
    // tokens a block: the work in whole waves of resident blocks, as few as kTokens allow (with four blocks
    // an SM, 8191 tokens in three waves of 16: 50 us, in one of 41: 45 us; in a full one and a quarter: 64 us)
    const long long resident = 152 * kAppendBlocks, work = (long long)a.N * chunks;
    const long long waves = (work + resident * kTokens - 1) / (resident * kTokens);
    const int tokens = (int)((work + resident * waves - 1) / (resident * waves));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.N + tokens - 1) / tokens), (unsigned)chunks, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = options().pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, append_kernel<D>, c, a, tokens, status);
}

cudaError_t launch_append(const CacheView &c, const AppendArgs &a, cudaStream_t stream) {
    int *status = status_word();
    if (!status) return cudaErrorInvalidSymbol;
    switch (c.dim) {
        case 64: return append_dim<64>(c, a, stream, status);
        case 128: return append_dim<128>(c, a, stream, status);
        case 256: return append_dim<256>(c, a, stream, status);
        default: return cudaErrorInvalidValue;
    }
}

// ---------------------------------------------------------------------- read
// A token's pieces are its rows' runs of 16 codes (one 16-byte load, two 16-byte stores), keys then
// values; a thread takes kReadPieces of a token's, equally far apart, all of their loads in flight:
// the chain slot, page, codes is walked once for them.  The rebuild is bsf8_dequant's.
// In a graph, 65536 tokens of 8 heads of 128: 70 us, 5.8 TB/s (0.86 of the measured HBM rate; one piece a thread:
// 88 us); 257 tokens: 3 us.
constexpr int kReadPieces = 4;

__global__ void __launch_bounds__(256) kv_read_kernel(const CacheView c, const int32_t *req, const int32_t *slot,
                                                      uint16_t *k_out, uint16_t *v_out, int side, long long threads,
                                                      int per, int *status) {
    pdl_trigger();
    pdl_wait();
    const int cpr = c.dim / 16;  // pieces a row; side: a side's; per: threads a token
    const long long step = (long long)gridDim.x * blockDim.x;
    for (long long it = (long long)blockIdx.x * blockDim.x + threadIdx.x; it < threads; it += step) {
        const int n = (int)(it / per), t = (int)(it - (long long)n * per);
        const int sl = slot[n];
        const long long row0 = cache_row(c, req[n], sl);
        if (row0 < 0 && sl >= 0) report_index(status);
        uint4 q[kReadPieces];
        uint32_t e[kReadPieces];
#pragma unroll
        for (int j = 0; j < kReadPieces; ++j) {
            const int pc = t + j * per;
            const bool key = k_out && pc < side;
            const int x = key || !k_out ? pc : pc - side;  // piece of its side
            q[j] = make_uint4(0, 0, 0, 0);
            e[j] = 127;
            if (x < side && row0 >= 0) {
                const int h = x / cpr, p = x - h * cpr;
                const size_t r = (size_t)row0 + (size_t)h * c.page_size;
                q[j] = *reinterpret_cast<const uint4 *>((key ? c.k8 : c.v8) + r * c.dim + 16 * p);
                e[j] = (key ? c.kexp : c.vexp)[r * (c.dim / 32) + p / 2];
            }
        }
#pragma unroll
        for (int j = 0; j < kReadPieces; ++j) {
            const int pc = t + j * per;
            const bool key = k_out && pc < side;
            const int x = key || !k_out ? pc : pc - side;
            if (x >= side || (!key && !v_out)) continue;
            const Scale sc = make_scale(e[j]);
            const uint32_t qw[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
            uint32_t o[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                rebuild4(qw[i], sc, o[2 * i], o[2 * i + 1]);
                if (nan_code_mask(qw[i])) patch_nan_codes(qw[i], o[2 * i], o[2 * i + 1]);
            }
            uint4 *dst = reinterpret_cast<uint4 *>((key ? k_out : v_out) + ((size_t)n * side + x) * 16);
            dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
            dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
    }
}

cudaError_t launch_kv_read(const CacheView &c, const int32_t *req, const int32_t *slot, void *k_out,
                           void *v_out, int N, cudaStream_t stream) {
    int *status = status_word();
    if (!status) return cudaErrorInvalidSymbol;
    const int side = c.heads * (c.dim / 16), both = side * (k_out && v_out ? 2 : 1);
    const int per = (both + kReadPieces - 1) / kReadPieces;
    const long long threads = (long long)N * per;
    return launch_cache(kv_read_kernel, (threads + 255) / 256, 256, stream, c, req, slot,
                        static_cast<uint16_t *>(k_out), static_cast<uint16_t *>(v_out), side, threads, per, status);
}

// -------------------------------------------------------------------- commit
// A block per request; a thread owns a 16-byte column of a head's rows (or a head's exponent
// bytes) and moves the kept nodes in order, eight loads before their eight stores.  In place
// without a hazard: an entry is moved only where path[i] >= i (a strictly increasing path has no
// other), and a store to slot i can only hit a source path[j] with j <= i, which its thread has read
// already.  Bound by latency: path and table, then batches of loads; 192 requests: 3.1 us in a graph.
constexpr int kCommitBatch = 8;

template <typename U>
__device__ __forceinline__ void commit_column(uint8_t *base, size_t row_bytes, const long long *rows, int count,
                                              size_t col, size_t head_off) {
    for (int i = rows[0] < 0 ? 1 : 0; i < count; i += kCommitBatch) {  // (node 0 is in its place already)
        U v[kCommitBatch];
#pragma unroll
        for (int j = 0; j < kCommitBatch; ++j)
            if (i + j < count && rows[2 * (i + j)] >= 0)
                v[j] = *reinterpret_cast<const U *>(base + ((size_t)rows[2 * (i + j)] + head_off) * row_bytes + col);
#pragma unroll
        for (int j = 0; j < kCommitBatch; ++j)
            if (i + j < count && rows[2 * (i + j)] >= 0)
                *reinterpret_cast<U *>(base + ((size_t)rows[2 * (i + j) + 1] + head_off) * row_bytes + col) = v[j];
    }
}

__global__ void __launch_bounds__(256) kv_commit_kernel(const CacheView c, const int32_t *ctx,
                                                        const int32_t *path,
                                                        const int32_t *count, int T, int *status) {
    __shared__ long long rows[2 * 256];  // source and target row of each kept node (head 0)
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.x;
    const int told = *(count + b), n = max(0, min(told, T)), at = *(ctx + b);
    if (told != n && threadIdx.x == 0) report_index(status);
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int32_t *const entry = path + (size_t)b * T + i;
        const int from = *entry, last = i > 0 ? *(entry - 1) : -1;
        long long src = -1, dst = -1;
        if (from >= i && from > last && at >= 0 && from <= 0x7FFFFFFF - at) {
            src = cache_row(c, b, at + from);
            dst = cache_row(c, b, at + i);
        }
        if (src < 0 || dst < 0) report_index(status);
        // nothing to move: not there, or there already
        rows[2 * i] = dst < 0 || from == i ? -1 : src;
        rows[2 * i + 1] = dst;
    }
    __syncthreads();
    const int cpr = c.dim / 16, cols = c.heads * cpr;
    for (int t = threadIdx.x; t < 2 * cols + 2 * c.heads; t += blockDim.x) {
        if (t < 2 * cols) {
            const int k = t % cols, h = k / cpr;
            commit_column<uint4>(t < cols ? c.k8 : c.v8, c.dim, rows, n, 16 * (size_t)(k - h * cpr),
                                 (size_t)h * c.page_size);
        } else {
            const int k = t - 2 * cols, h = k % c.heads;
            uint8_t *base = k < c.heads ? c.kexp : c.vexp;
            const size_t off = (size_t)h * c.page_size;
            if (c.dim == 64) commit_column<uint16_t>(base, 2, rows, n, 0, off);
            else if (c.dim == 128) commit_column<uint32_t>(base, 4, rows, n, 0, off);
            else commit_column<uint2>(base, 8, rows, n, 0, off);
        }
    }
}

cudaError_t launch_kv_commit(const CacheView &c, const int32_t *ctx, const int32_t *path, const int32_t *count,
                             int B, int T, cudaStream_t stream) {
    int *status = status_word();
    if (!status) return cudaErrorInvalidSymbol;
    const int cols = 2 * c.heads * (c.dim / 16 + 1);
    const int threads = std::min(256, (cols + 31) / 32 * 32);
    return launch_cache(kv_commit_kernel, B, threads, stream, c, ctx, path, count, T, status);
}

}  // namespace bsf8
