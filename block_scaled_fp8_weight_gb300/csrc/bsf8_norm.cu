// bsf8_norm.cu -- what lies between two linear layers: the block's output normed, gated, scaled and
// added to the residual, and the sum normed for the next block, in one pass.
//
//   z = x rsqrt(mean x^2 + eps) post,   r = residual + scale gate z,   h = r rsqrt(mean r^2 + eps) w
//
// A row stays in its threads' registers, 8 channels a piece, from its loads to its stores; the two means
// are the only exchange.  All arithmetic is fp32; h is taken from r before r's rounding to its type, so
// that each output is rounded once.
#include "bsf8_device.cuh"
#include "bsf8_internal.h"

#include <algorithm>

namespace bsf8 {

namespace {

constexpr int kMaxWarps = 32;
constexpr int kRowsWarps = 20;  // a block of the kernel for many rows: 96 registers a thread (at 64 it spilled, to L2: no L1 is left)
constexpr int kMaxRows = 225 * 1024;
constexpr int kMaxRow = 4 * 3 * 1024 * 16;  // bytes of the longest row's pieces: 192 KB

__device__ __forceinline__ void widen8(const uint4 &w, float (&y)[8]) {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[2 * i] = __uint_as_float(a[i] << 16);
        y[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint4 narrow8(const float (&y)[8]) {
    return make_uint4(bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3]), bf16_pair(y[4], y[5]), bf16_pair(y[6], y[7]));
}

__device__ __forceinline__ void async16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Eight channels of the residual.
template <bool F32>
__device__ __forceinline__ const uint4 *residual_at(const NormArgs &a, long long row, int c) {
    return reinterpret_cast<const uint4 *>(static_cast<const char *>(a.residual) + (row * a.ldr + c) * (F32 ? 4 : 2));
}

template <bool F32>
__device__ __forceinline__ void residual_of(const uint4 &r, const uint4 &r2, float (&y)[8]) {
    if constexpr (F32) {
        y[0] = __uint_as_float(r.x), y[1] = __uint_as_float(r.y), y[2] = __uint_as_float(r.z), y[3] = __uint_as_float(r.w);
        y[4] = __uint_as_float(r2.x), y[5] = __uint_as_float(r2.y), y[6] = __uint_as_float(r2.z), y[7] = __uint_as_float(r2.w);
    } else {
        widen8(r, y);
    }
}

// A row's squares are added up in one order whatever the kernel, so that a row's bits do not depend on how many come with
// it: channels in fours, one after another; the fours of 256 channels (64) by a tree, neighbours first; then those sums,
// c, c + 32, .. one after another and the 32 of them by a tree, far ones first.
template <int N>
__device__ __forceinline__ float squares(const float (&z)[N]) {
    float sum[N / 4];
#pragma unroll
    for (int k = 0; k < N / 4; ++k) {
        sum[k] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[k] = fmaf(z[4 * k + i], z[4 * k + i], sum[k]);
    }
    return N == 4 ? sum[0] : sum[0] + sum[N / 4 - 1];
}

// J trees over a warp's lanes side by side: lane l gets the sum of all lanes' v[l % J], every shuffle carrying what
// the other lane needs.
template <int J>
__device__ __forceinline__ float lane_sums(float (&v)[J]) {
    const uint32_t lane = threadIdx.x & 31;
    int n = J;
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
        if (n == 1) {
            v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], m);
            continue;
        }
        n /= 2;
#pragma unroll
        for (int q = 0; q < J / 2; ++q) {
            if (q >= n) continue;
            const bool odd = lane & m;
            const float keep = odd ? v[2 * q + 1] : v[2 * q], send = odd ? v[2 * q] : v[2 * q + 1];
            v[q] = keep + __shfl_xor_sync(0xFFFFFFFFu, send, m);
        }
    }
    return v[0];
}

__device__ __forceinline__ float far_first(float v) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
    return v;
}

}  // namespace

// P pieces of 8 channels a thread; `warps` warps a row, blockDim / (32 warps) rows a block.  Few rows: one piece a
// thread, its loads straight to registers (P = 1).  Many: four pieces a thread, which go to shared memory by the
// thread's own asynchronous copies (nothing is handed from thread to thread there) and wait there for the row's first
// sum; with few threads a row six blocks and more share an SM, so that the loads, sums and stores of one run under
// those of the others.  (Four pieces at 64 registers spill 4 or 12 bytes a thread.)
template <int P, bool F32>
__global__ void __launch_bounds__(1024) norm_kernel(const NormArgs a, int warps) {
    constexpr int WORDS = F32 ? 3 : 2;  // of 16 bytes a piece: x, the residual
    __shared__ float s_sum[2][P * kMaxWarps];
    extern __shared__ uint4 ring[];
    pdl_trigger();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = warp / warps, w0 = sub * warps;             // the block's row, its first warp
    const int t = (int)threadIdx.x - 32 * w0, threads = 32 * warps;
    const int rows = (int)(blockDim.x >> 5) / warps;
    const int step = (int)blockDim.x;
    const float inv = 1.0f / (float)a.H;
    const long long row = (long long)blockIdx.x * rows + sub;
    const bool real = row < a.M, full = a.gate_kind == kGateFull;
    auto slot = [&](int p) { return ring + (size_t)p * WORDS * step + threadIdx.x; };
    uint4 x0, r0, r1;  // P = 1
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int c = 8 * (t + p * threads);
        if (!real || c >= a.H) continue;
        if constexpr (P == 1) {
            x0 = *reinterpret_cast<const uint4 *>(a.x + row * a.ldx + c);
            if (a.residual) {
                r0 = residual_at<F32>(a, row, c)[0];
                if (F32) r1 = residual_at<F32>(a, row, c)[1];
            }
        } else {
            async16(slot(p), a.x + row * a.ldx + c);
            if (a.residual) {
                async16(slot(p) + step, residual_at<F32>(a, row, c));
                if (F32) async16(slot(p) + 2 * step, residual_at<F32>(a, row, c) + 1);
            }
        }
    }
    if constexpr (P > 1) asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
    auto vec = [&](const uint16_t *v, int p) { return *reinterpret_cast<const uint4 *>(v + 8 * (t + p * threads)); };
    // the sum over the row of the pieces' sums
    auto row_sum = [&](float (&v)[P], int which) {
        float sum = lane_sums(v);
        if (warps == 1) {
            if (P > 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2), sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
            return sum;
        }
        float *const at = s_sum[which] + P * w0;  // by 256 channels
        if (lane < P) at[lane * warps + warp - w0] = sum;
        __syncthreads();
        sum = lane < P * warps ? at[lane] : 0.0f;
        if (P > 1 && P * warps > 32) {
            float more[P];
#pragma unroll
            for (int k = 1; k < P; ++k) more[k] = lane + 32 * k < P * warps ? at[lane + 32 * k] : 0.0f;
#pragma unroll
            for (int k = 1; k < P; ++k) sum += more[k];
        }
        return far_first(sum);
    };
    float f = a.scale;
    if (a.gate_kind == kGateToken && real) f *= __uint_as_float((uint32_t)a.gate[row * a.ldg] << 16);
    float z[P][8], ss[P];
    if (a.post) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            ss[p] = 0.0f;
            if (!real || 8 * (t + p * threads) >= a.H) continue;
            widen8(P == 1 ? x0 : *slot(p), z[p]);
            ss[p] = squares(z[p]);
        }
    }
    const float n = a.post ? rsqrtf(fmaf(row_sum(ss, 0), inv, a.eps)) : 1.0f;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int c = 8 * (t + p * threads);
        ss[p] = 0.0f;
        if (!real || c >= a.H) continue;
        const uint4 *const at = slot(p);
        float g[8];
        widen8(P == 1 ? x0 : at[0], z[p]);
        if (a.post) {
            widen8(vec(a.post, p), g);
#pragma unroll
            for (int i = 0; i < 8; ++i) z[p][i] = z[p][i] * n * g[i];
        }
        if (full || a.gate_kind == kGateChannel) {
            widen8(vec(full ? a.gate + row * a.ldg : a.gate, p), g);
#pragma unroll
            for (int i = 0; i < 8; ++i) z[p][i] *= g[i];
        }
        float r[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (a.residual) residual_of<F32>(P == 1 ? r0 : at[step], P == 1 ? r1 : at[F32 ? 2 * step : 0], r);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[p][i] = fmaf(f, z[p][i], r[i]);
        ss[p] = squares(z[p]);
        if (a.r_out) {
            if constexpr (F32) {
                float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.r_out) + row * a.H + c);
                o[0] = make_float4(z[p][0], z[p][1], z[p][2], z[p][3]);
                o[1] = make_float4(z[p][4], z[p][5], z[p][6], z[p][7]);
            } else {
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.r_out) + row * a.H + c) = narrow8(z[p]);
            }
        }
    }
    if (!a.h) return;
    const float k = rsqrtf(fmaf(row_sum(ss, 1), inv, a.eps));
    if (!real) return;
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int c = 8 * (t + p * threads);
        if (c >= a.H) continue;
        float g[8];
        widen8(vec(a.weight, p), g);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] *= z[p][i] * k;
        *reinterpret_cast<uint4 *>(a.h + row * a.H + c) = narrow8(g);
    }
}

// Channels that a thread takes at a time in the kernel for many rows: a residual of 16 bytes, next to its
// neighbours' (eight channels a thread were two of 16 bytes, each half a sector from the next lane's).
template <bool F32>
struct Unit;
template <>
struct Unit<false> {
    static constexpr int N = 8;
    typedef uint4 Half;  // bf16 values
    static __device__ __forceinline__ void widen(const uint4 &w, float (&y)[8]) { widen8(w, y); }
    static __device__ __forceinline__ uint4 narrow(const float (&y)[8]) { return narrow8(y); }
    static __device__ __forceinline__ void residual(const uint4 &w, float (&y)[8]) { widen8(w, y); }
    static __device__ __forceinline__ uint4 store(const float (&y)[8]) { return narrow8(y); }
};
template <>
struct Unit<true> {
    static constexpr int N = 4;
    typedef uint2 Half;
    static __device__ __forceinline__ void widen(const uint2 &w, float (&y)[4]) {
        y[0] = __uint_as_float(w.x << 16), y[1] = __uint_as_float(w.x & 0xFFFF0000u);
        y[2] = __uint_as_float(w.y << 16), y[3] = __uint_as_float(w.y & 0xFFFF0000u);
    }
    static __device__ __forceinline__ uint2 narrow(const float (&y)[4]) { return make_uint2(bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3])); }
    static __device__ __forceinline__ void residual(const uint4 &w, float (&y)[4]) {
        y[0] = __uint_as_float(w.x), y[1] = __uint_as_float(w.y), y[2] = __uint_as_float(w.z), y[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ uint4 store(const float (&y)[4]) {
        return make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3]));
    }
};

// Many rows: one block an SM in groups of `warps` warps, a group a row at a time, 32 channels a thread.  The weights
// lie in shared memory for good; a row comes there by bulk copies of one thread, the next row's (or the one after) asked
// for as soon as this one's are used up, under its last stores.
// 8191 rows of 5120 (fp32 residual, both norms, channel gate): 85 us, 5.9 TB/s of what must move (0.87 of the measured
// rate); waits for the loads are two thirds of a row's time in its group.  Six groups at 64 registers: 135 us, their
// spills go to L2; a block a row (the kernel above): 110; the same with 640 threads a row: 97.
template <bool F32>
__global__ void __launch_bounds__(kRowsWarps * 32, 1) norm_rows_kernel(const NormArgs a, int warps, int groups, int depth,
                                                                       unsigned long long timeout_ns, int skip_loads, int *status) {
    using U = Unit<F32>;
    using Half = typename U::Half;
    constexpr int N = U::N, J = 32 / N;
    static_assert(4 * kRowsWarps <= 96, "three sums of 256 channels a lane");
    __shared__ __align__(8) float s_sum[2][J * kRowsWarps];
    __shared__ uint64_t s_full[2 * kRowsWarps];
    extern __shared__ uint4 memory[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = warp / warps, w0 = group * warps;
    const int t = (int)threadIdx.x - 32 * w0, threads = 32 * warps, step = (int)blockDim.x, units = a.H / N;
    const int first = group * depth, buffers = groups * depth;  // its first buffer
    if (t == 0) {
        for (int d = 0; d < depth; ++d) mbar_init(&s_full[first + d], 1);
    }
    fence_mbar_init();
    __syncthreads();
    pdl_trigger();
    pdl_wait();
    const float inv = 1.0f / (float)a.H;
    const bool full = a.gate_kind == kGateFull, channel = a.gate_kind == kGateChannel;
    // the buffers' rows of the residual, of x and of a full gate; then weight, post_weight and a channel gate
    Half *const x_rows = reinterpret_cast<Half *>(memory + buffers * units);
    Half *const vec = x_rows + (full ? 2 : 1) * buffers * units;
    const uint32_t row_bytes = (uint32_t)a.H * 2;
    auto ask = [&](long long row, int b) {
        if (t != 0 || row >= a.M) return;
        mbar_arrive_expect_tx(&s_full[b], row_bytes * (full ? 2u : 1u) + (a.residual ? row_bytes * (F32 ? 2u : 1u) : 0u));
        if (skip_loads) return;
        bulk_g2s(x_rows + b * units, a.x + row * a.ldx, row_bytes, &s_full[b]);
        if (full) bulk_g2s(x_rows + (buffers + b) * units, a.gate + row * a.ldg, row_bytes, &s_full[b]);
        if (a.residual)
            bulk_g2s(memory + b * units, static_cast<const char *>(a.residual) + row * a.ldr * (F32 ? 4 : 2), row_bytes * (F32 ? 2 : 1), &s_full[b]);
    };
    const long long stride = (long long)gridDim.x * groups;
    long long row = (long long)blockIdx.x * groups + group;
    for (int d = 0; d < depth; ++d) ask(row + d * stride, first + d);
    for (int i = threadIdx.x; i < units; i += step) {
        if (a.h) vec[i] = reinterpret_cast<const Half *>(a.weight)[i];
        if (a.post) vec[units + i] = reinterpret_cast<const Half *>(a.post)[i];
        if (channel) vec[2 * units + i] = reinterpret_cast<const Half *>(a.gate)[i];
    }
    __syncthreads();
    // the sum over the row of the units' sums
    uint32_t sums = 0;  // two sets of slots in turn: one is written again after the barrier of the other
    auto group_sum = [&](float (&v)[J]) {
        float sum = lane_sums(v);
        if (warps == 1) {
            if (J == 8) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, J / 2);
            return sum + __shfl_xor_sync(0xFFFFFFFFu, sum, J / 4);
        }
        float *const at = s_sum[sums++ & 1] + J * w0;  // by 32 N channels
        if (lane < J) at[lane * warps + warp - w0] = sum;
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
        auto piece = [&](int c) {
            if (c >= 4 * warps) return 0.0f;
            if constexpr (J == 4) return at[c];
            const float2 two = reinterpret_cast<const float2 *>(at)[c];
            return two.x + two.y;
        };
        sum = piece(lane);
        if (4 * warps > 32) {
            const float more = piece(lane + 32), last = piece(lane + 64);
            sum = sum + more + last;
        }
        return far_first(sum);
    };
    // whether v holds for the whole group, which so goes on or leaves as one
    auto group_all = [&](bool v) {
        if (warps == 1) return __all_sync(0xFFFFFFFFu, v) != 0;
        uint32_t all;
        asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                     : "=r"(all)
                     : "r"((uint32_t)v), "r"(group + 1), "r"(threads)
                     : "memory");
        return all != 0;
    };
    uint32_t phase = 0;
    int d = 0;
    for (; row < a.M; row += stride) {
        const int b = first + d;
        float f = a.scale;
        if (a.gate_kind == kGateToken) f *= __uint_as_float((uint32_t)a.gate[row * a.ldg] << 16);
        if (!group_all(mbar_wait_bounded(&s_full[b], phase, timeout_ns))) {
            // the wait ran out: what was asked for may still land, and the block's memory is not left before
            report_timeout(status);
            if (!skip_loads) {
                (void)mbar_wait_bounded(&s_full[b], phase, timeout_ns);
                if (depth > 1 && row + stride < a.M) (void)mbar_wait_bounded(&s_full[first + (d ^ 1)], phase ^ d, timeout_ns);
            }
            return;
        }
        if (++d == depth) d = 0, phase ^= 1;
        const uint4 *const r_at = memory + b * units;
        const Half *const x_at = x_rows + b * units, *const g_at = x_rows + (buffers + b) * units;
        float z[J][N], ss[J], n = 1.0f;
        if (a.post) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                ss[j] = 0.0f;
                if (t + j * threads >= units) continue;
                U::widen(x_at[t + j * threads], z[j]);
                ss[j] = squares(z[j]);
            }
            n = rsqrtf(fmaf(group_sum(ss), inv, a.eps));
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int u = t + j * threads;
            ss[j] = 0.0f;
            if (u >= units) continue;
            float g[N];
            U::widen(x_at[t + j * threads], z[j]);
            if (a.post) {
                U::widen(vec[units + u], g);
#pragma unroll
                for (int i = 0; i < N; ++i) z[j][i] = z[j][i] * n * g[i];
            }
            if (channel || full) {
                U::widen(full ? g_at[u] : vec[2 * units + u], g);
#pragma unroll
                for (int i = 0; i < N; ++i) z[j][i] *= g[i];
            }
            float r[N] = {};
            if (a.residual) U::residual(r_at[u], r);
#pragma unroll
            for (int i = 0; i < N; ++i) z[j][i] = fmaf(f, z[j][i], r[i]);
            ss[j] = squares(z[j]);
            if (a.r_out) static_cast<uint4 *>(a.r_out)[row * units + u] = U::store(z[j]);
        }
        const float k = rsqrtf(fmaf(group_sum(ss), inv, a.eps));
        if (warps == 1) __syncwarp();
        ask(row + depth * stride, b);  // the whole group has read this row
        if (!a.h) continue;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int u = t + j * threads;
            if (u >= units) continue;
            float g[N];
            U::widen(vec[u], g);
#pragma unroll
            for (int i = 0; i < N; ++i) g[i] *= z[j][i] * k;
            reinterpret_cast<Half *>(a.h)[row * units + u] = U::narrow(g);
        }
    }
}

// Groups of a block: as many as its threads, named barriers (15) and shared memory allow; with two rows each where that
// takes no group away (8191 rows, fp32 residual, both norms, channel gate: of 7168 two groups 127 -> 119 us, of 12288 one
// group 257 -> 195; of 5120 three groups for four 87 -> 90).
template <bool F32>
int row_groups(int H, bool full, int *depth, size_t *bytes) {
    const int warps = (H / 8 + 127) / 128;
    const size_t row = (size_t)H * (2 + (F32 ? 4 : 2) + (full ? 2 : 0)), weights = (size_t)3 * H * 2;
    const int most = std::min(warps == 1 ? kRowsWarps : 15, kRowsWarps / warps);
    if (weights + row > (size_t)kMaxRows) return 0;
    const int one = std::min(most, (int)((kMaxRows - weights) / row)), two = std::min(most, (int)((kMaxRows - weights) / (2 * row)));
    *depth = two == one ? 2 : 1;
    *bytes = weights + one * *depth * row;
    return one;
}

template <bool F32>
cudaError_t launch_rows(const NormArgs &a, int groups, int depth, size_t smem, cudaStream_t stream) {
    static int configured[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!__atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE)) {
        e = cudaFuncSetAttribute(norm_rows_kernel<F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxRows);
        if (e != cudaSuccess) return e;
        __atomic_store_n(&configured[dev], 1, __ATOMIC_RELEASE);
    }
    int *status = status_word();
    if (!status) return cudaErrorInvalidSymbol;
    const int warps = (a.H / 8 + 127) / 128;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min<long long>(((long long)a.M + groups - 1) / groups, 152), 1, 1);
    cfg.blockDim = dim3((unsigned)(groups * warps * 32), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = options().pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, norm_rows_kernel<F32>, a, warps, groups, depth, options().timeout_ns, options().skip_loads, status);
}

template <int P, bool F32>
cudaError_t norm_pieces(const NormArgs &a, cudaStream_t stream) {
    const int warps = (a.H / 8 + 32 * P - 1) / (32 * P);
    const int rows = warps >= 5 ? 1 : 8 / warps, threads = rows * warps * 32;
    const size_t smem = P == 1 ? 0 : (size_t)P * (F32 ? 3 : 2) * threads * sizeof(uint4);
    if (P > 1) {
        static int configured[64] = {0};
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        if (!__atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE)) {
            e = cudaFuncSetAttribute(norm_kernel<P, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxRow);
            if (e != cudaSuccess) return e;
            __atomic_store_n(&configured[dev], 1, __ATOMIC_RELEASE);
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((long long)a.M + rows - 1) / rows), 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = options().pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, norm_kernel<P, F32>, a, warps);
}

template <bool F32>
cudaError_t norm_typed(const NormArgs &a, cudaStream_t stream) {
    // One piece a thread while the SMs hold all rows in a turn or two, and for an fp32 residual without a first norm where
    // rows are short.  Else the rows' kernel if more than two bytes a channel come beside x (its copies make whole sectors
    // of them), four pieces a thread if not.  One piece / four / the rows' kernel, us (gate: a post norm and an fp32
    // residual too): 304 rows of 5120 bf16 3.3 / 3.9 / 4.8, gate 4.8 / 7.4 / 6.9; 500 of 4096 bf16 4.6 / 5.6 / 5.2, gate
    // 7.2 / 11.7 / 7.4; 304 of 7168 bf16 4.7 / 4.3 / 4.6; 8191 of 5120 bf16 66 / 51 / 57, with a full gate 89 / 76 / 69, gate
    // 100 / 120 / 85, fp32 without a first norm 80 / 98 / 88; of 5632 (one piece a thread takes more than 20 warps a row, and
    // an SM holds fewer rows) bf16 111 / 55 / 65, full gate 144 / 87 / 74, gate 165 / 129 / 97, fp32 121 / 108 / 90; of 6144,
    // 6656 and 7168 the same order (7168: bf16 124 / 70 / 83, fp32 138 / 135 / 119).  From 300 to 1000 rows it is within 5 %
    // of the best at most of these sizes, but 304 rows of 5632 and 6144 are 15 % faster by one piece (5.0 for 4.3), and 500
    // rows with a full gate from 5632 on, 1000 at 4096, 10 to 25 % by four pieces (8.1 for 6.1).  Six rows of 12288, gate
    // - / 7.1 / 6.1.
    const bool full = a.gate_kind == kGateFull;
    const long long few = 152LL * (F32 || full || a.H > 5120 ? 10240 : 16384);  // channels
    if (a.H <= 8192 && (a.M * (long long)a.H <= few || (F32 && !a.post && !full && a.H <= 5120))) return norm_pieces<1, F32>(a, stream);
    int depth;
    size_t smem;
    const int groups = F32 || full ? row_groups<F32>(a.H, full, &depth, &smem) : 0;
    return groups > 0 ? launch_rows<F32>(a, groups, depth, smem, stream) : norm_pieces<4, F32>(a, stream);
}

cudaError_t launch_norm(const NormArgs &a, cudaStream_t stream) {
    return a.fp32 ? norm_typed<true>(a, stream) : norm_typed<false>(a, stream);
}

}  // namespace bsf8
