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

// Eight channels of a row of x, and of the residual.
template <bool F32>
struct Piece {
    uint4 x, r, r2;

    __device__ __forceinline__ void load(const NormArgs &a, long long row, int c) {
        x = *reinterpret_cast<const uint4 *>(a.x + row * a.ldx + c);
        if (!a.residual) return;
        if constexpr (F32) {
            const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(a.residual) + row * a.ldr + c);
            r = p[0];
            r2 = p[1];
        } else {
            r = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.residual) + row * a.ldr + c);
        }
    }
    __device__ __forceinline__ void residual(float (&y)[8]) const {
        if constexpr (F32) {
            y[0] = __uint_as_float(r.x), y[1] = __uint_as_float(r.y), y[2] = __uint_as_float(r.z), y[3] = __uint_as_float(r.w);
            y[4] = __uint_as_float(r2.x), y[5] = __uint_as_float(r2.y), y[6] = __uint_as_float(r2.z), y[7] = __uint_as_float(r2.w);
        } else {
            widen8(r, y);
        }
    }
};

}  // namespace

// P pieces of 8 channels a thread; `warps` warps a row, blockDim / (32 warps) rows a block at a time.
template <int P, bool F32>
__global__ void __launch_bounds__(1024) norm_kernel(const NormArgs a, int warps) {
    __shared__ float s_sum[2][kMaxWarps];
    pdl_trigger();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = warp / warps, w0 = sub * warps;             // the block's row, its first warp
    const int t = (int)threadIdx.x - 32 * w0, threads = 32 * warps;
    const int rows = (int)(blockDim.x >> 5) / warps;
    const int pieces = a.H / 8;
    const float inv = 1.0f / (float)a.H;
    uint4 wv[P], pv[P], gv[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int c = 8 * (t + p * threads);
        wv[p] = pv[p] = gv[p] = make_uint4(0, 0, 0, 0);
        if (c < a.H) {
            if (a.weight) wv[p] = *reinterpret_cast<const uint4 *>(a.weight + c);
            if (a.post) pv[p] = *reinterpret_cast<const uint4 *>(a.post + c);
            if (a.gate_kind == kGateChannel) gv[p] = *reinterpret_cast<const uint4 *>(a.gate + c);
        }
    }
    // the sum of v over the row's threads
    uint32_t sums = 0;  // two sets of slots in turn: one is written again after the barrier of the other
    auto row_sum = [&](float v) {
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
        if (warps == 1) return v;
        float *const at = s_sum[sums++ & 1];
        if (lane == 0) at[warp] = v;
        __syncthreads();
        v = 0.0f;
        for (int w = 0; w < warps; ++w) v += at[w0 + w];
        return v;
    };
    const long long step = (long long)gridDim.x * rows;
    Piece<F32> next[P];
    const long long first = (long long)blockIdx.x * rows;
    auto load = [&](long long row) {
        if (row >= a.M) return;
#pragma unroll
        for (int p = 0; p < P; ++p)
            if (t + p * threads < pieces) next[p].load(a, row, 8 * (t + p * threads));
    };
    load(first + sub);
    for (long long base = first; base < a.M; base += step) {  // the same turns for every thread: barriers
        const long long row = base + sub;
        const bool real = row < a.M;
        float z[P][8];
        float ss = 0.0f;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            if (!real || t + p * threads >= pieces) {
#pragma unroll
                for (int i = 0; i < 8; ++i) z[p][i] = 0.0f;
                continue;
            }
            widen8(next[p].x, z[p]);
            if (a.post) {
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(z[p][i], z[p][i], ss);
            }
        }
        float f = a.scale;
        if (a.gate_kind == kGateToken && real) f *= __uint_as_float((uint32_t)a.gate[row * a.ldg] << 16);
        const float n = a.post ? rsqrtf(fmaf(row_sum(ss), inv, a.eps)) : 1.0f;
        ss = 0.0f;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int c = 8 * (t + p * threads);
            if (!real || c >= a.H) continue;
            float g[8];
            if (a.post) {
                widen8(pv[p], g);
#pragma unroll
                for (int i = 0; i < 8; ++i) z[p][i] = z[p][i] * n * g[i];
            }
            if (a.gate_kind == kGateChannel || a.gate_kind == kGateFull) {
                if (a.gate_kind == kGateFull) gv[p] = *reinterpret_cast<const uint4 *>(a.gate + row * a.ldg + c);
                widen8(gv[p], g);
#pragma unroll
                for (int i = 0; i < 8; ++i) z[p][i] *= g[i];
            }
            float r[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (a.residual) next[p].residual(r);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                z[p][i] = fmaf(f, z[p][i], r[i]);
                ss = fmaf(z[p][i], z[p][i], ss);
            }
        }
        load(row + step);  // the next row's, while this one's sum goes round
        if (a.r_out && real) {
#pragma unroll
            for (int p = 0; p < P; ++p) {
                const int c = 8 * (t + p * threads);
                if (c >= a.H) continue;
                if constexpr (F32) {
                    float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.r_out) + row * a.H + c);
                    o[0] = make_float4(z[p][0], z[p][1], z[p][2], z[p][3]);
                    o[1] = make_float4(z[p][4], z[p][5], z[p][6], z[p][7]);
                } else {
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.r_out) + row * a.H + c) = narrow8(z[p]);
                }
            }
        }
        if (!a.h) continue;
        const float k = rsqrtf(fmaf(row_sum(ss), inv, a.eps));
        if (!real) continue;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int c = 8 * (t + p * threads);
            if (c >= a.H) continue;
            float g[8];
            widen8(wv[p], g);
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] *= z[p][i] * k;
            *reinterpret_cast<uint4 *>(a.h + row * a.H + c) = narrow8(g);
        }
    }
}

template <int P, bool F32>
cudaError_t norm_pieces(const NormArgs &a, cudaStream_t stream) {
    const int warps = (a.H / 8 + 32 * P - 1) / (32 * P);
    const int rows = warps >= 8 ? 1 : 8 / warps;
    cudaLaunchConfig_t cfg = {};
    const int per_sm = std::max(1, 2048 / (rows * warps * 32));
    cfg.gridDim = dim3((unsigned)std::min<long long>(((long long)a.M + rows - 1) / rows, 152LL * per_sm), 1, 1);
    cfg.blockDim = dim3((unsigned)(rows * warps * 32), 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = options().pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, norm_kernel<P, F32>, a, warps);
}

cudaError_t launch_norm(const NormArgs &a, cudaStream_t stream) {
    if (a.H <= 8192) return a.fp32 ? norm_pieces<1, true>(a, stream) : norm_pieces<1, false>(a, stream);
    if (a.H <= 16384) return a.fp32 ? norm_pieces<2, true>(a, stream) : norm_pieces<2, false>(a, stream);
    return a.fp32 ? norm_pieces<4, true>(a, stream) : norm_pieces<4, false>(a, stream);
}

}  // namespace bsf8
