// bsf8_attend.cu -- attention of a token tree over the paged cache.
#include "bsf8_device.cuh"
#include "bsf8_internal.h"

#include <algorithm>

namespace bsf8 {

namespace {

__device__ __forceinline__ float value(uint32_t code, uint32_t e) {
    const Scale sc = make_scale(e);
    uint32_t lo, hi;
    rebuild4(code, sc, lo, hi);
    if (nan_code_mask(code & 0xFFu)) return __uint_as_float(0x7FC00000u);
    return __uint_as_float(lo << 16);
}

}  // namespace

// A warp per query row, a channel piece of D / 32 a lane, one key after another.
template <int D>
__global__ void __launch_bounds__(32) attend_row_kernel(const CacheView c, const AttendArgs a, int *status) {
    pdl_trigger();
    pdl_wait();
    constexpr int P = D / 32;
    const int lane = threadIdx.x;
    const int h = blockIdx.x % a.Hq, t = (blockIdx.x / a.Hq) % a.T, b = blockIdx.x / (a.Hq * a.T);
    const int g = a.Hq / c.heads, W = (a.T + 31) / 32;
    int ctx = a.ctx[b], nodes = a.nodes ? a.nodes[b] : a.T;
    if (ctx < 0 || nodes < 0 || nodes > a.T || (long long)ctx + nodes > a.max_len) {
        if (lane == 0) report_index(status);
        ctx = max(0, min(ctx, a.max_len));
        nodes = max(0, min(nodes, min(a.T, a.max_len - ctx)));
    }
    float q[P], o[P], m = -INFINITY, l = 0.0f;
    const uint16_t *qr = a.q + ((size_t)b * a.T + t) * a.ldq + (size_t)h * D;
    for (int i = 0; i < P; ++i) {
        q[i] = __uint_as_float((uint32_t)qr[lane * P + i] << 16);
        o[i] = 0.0f;
    }
    const int len = t < nodes ? ctx + nodes : 0;
    for (int s = 0; s < len; ++s) {
        const int j = s - ctx;
        if (j >= 0) {
            const bool see = a.mask ? (a.mask[((size_t)b * a.T + t) * W + j / 32] >> (j % 32)) & 1 : j <= t;
            if (!see) continue;
        }
        const int page = c.table[(size_t)b * c.table_pages + s / c.page_size];
        if ((unsigned)page >= (unsigned)c.pages) {
            if (lane == 0) report_index(status);
            continue;
        }
        const size_t r = ((size_t)page * c.heads + h / g) * c.page_size + s % c.page_size;
        float x = 0.0f;
        for (int i = 0; i < P; ++i)
            x += q[i] * value(c.k8[r * D + lane * P + i], c.kexp[r * (D / 32) + (lane * P + i) / 32]);
        for (int k = 16; k > 0; k >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, k);
        x *= a.scale;
        const float mn = fmaxf(m, x);
        const float f = m == -INFINITY ? 0.0f : expf(m - mn), p = expf(x - mn);
        l = l * f + p;
        for (int i = 0; i < P; ++i)
            o[i] = o[i] * f + p * value(c.v8[r * D + lane * P + i], c.vexp[r * (D / 32) + (lane * P + i) / 32]);
        m = mn;
    }
    for (int i = 0; i < P; ++i)
        a.out[(((size_t)b * a.T + t) * a.Hq + h) * D + lane * P + i] = f32_to_bf16_rn(l != 0.0f ? o[i] / l : 0.0f);
    if (a.lse && lane == 0) a.lse[((size_t)b * a.T + t) * a.Hq + h] = l != 0.0f ? m + logf(l) : -INFINITY;
}

size_t attend_workspace_bytes(int, int, int, int, int) { return 0; }

cudaError_t launch_attend(const CacheView &c, const AttendArgs &a, cudaStream_t stream) {
    int *status = status_word();
    if (!status) return cudaErrorInvalidSymbol;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.B * a.T * a.Hq), 1, 1);
    cfg.blockDim = dim3(32, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = options().pdl ? 1 : 0;
    switch (c.dim) {
        case 64: return cudaLaunchKernelEx(&cfg, attend_row_kernel<64>, c, a, status);
        case 128: return cudaLaunchKernelEx(&cfg, attend_row_kernel<128>, c, a, status);
        default: return cudaLaunchKernelEx(&cfg, attend_row_kernel<256>, c, a, status);
    }
}

}  // namespace bsf8
