/*
 * bsf8.h -- C ABI of libbsf8, a block-scaled FP8 weight library for GB300 (sm_103a).
 *
 * The method (pages "recipes/docker-images/mia-tp4/adapter/wo_a_w8.py" and
 * "recipes/docker-images/mia-tp4/adapter/shared_pad_k.py"):
 *   A bf16 weight W[G][N][K] is kept as an fp8 "twin": one e4m3 code per element plus
 *   one exponent byte (ue8m0, byte = e + 127) per 32x32 block.  The small-batch linear
 *   y[m][g][n] = sum_k x[m][g*K + k] * W[g][n][k] reads the twin, rebuilds each bf16
 *   weight exactly as bf16(e4m3 * 2^(byte-127)) in registers and accumulates in fp32;
 *   split-K partials are summed in a fixed order, so results are deterministic.
 *
 * Conventions for every entry point:
 *   - Pointers are DEVICE pointers owned by the caller, except where a parameter says
 *     "host".  The library never allocates, and every buffer a call touches is named in its
 *     argument list -- with one exception: bsf8_gemm_static_scratch keeps its partials in a
 *     buffer compiled into the library (BSF8_STATIC_SCRATCH_BYTES, 8 MiB on every GPU that
 *     loads it), which calls that can overlap on the GPU must not use at the same time.
 *   - bf16 tensors are passed as void* holding IEEE bfloat16 bit patterns.
 *   - Row-major layouts:  w8[G][N][K] (uint8 e4m3fn codes),  exp[G][N/32][K/32]
 *     (uint8, byte = e + 127),  x[M][ldx] (bf16; group g uses columns [g*K, (g+1)*K)),
 *     y[M][G][N] (bf16),  partials[S][M][G][N] (fp32).
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = the legacy default
 *     stream), do not synchronise the host, and allocate nothing.
 *   - Every call validates its arguments on the host first and returns a status code
 *     without launching anything when they are invalid; on success it returns BSF8_OK
 *     once the work is enqueued.  Faults found by the kernels themselves (a bounded
 *     wait that ran out) are recorded in a device status word read by
 *     bsf8_device_status().
 *   - Shapes: N and K are multiples of 32 (one exponent per 32x32 block); G >= 1.
 *
 * This library needs an sm_103a GPU (GB300); it has no CPU fallback.
 */
#ifndef BSF8_H
#define BSF8_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A cudaStream_t without pulling in the CUDA headers. */
typedef struct CUstream_st *bsf8_stream_t;

/* Status codes. */
enum {
    BSF8_OK = 0,
    BSF8_ERR_SHAPE = 1,     /* N or K not a multiple of 32, a size < 1, M out of range  */
    BSF8_ERR_ALIGN = 2,     /* a pointer or stride breaks the 16-byte rule of the call  */
    BSF8_ERR_STRIDE = 3,    /* ldx < G*K                                                */
    BSF8_ERR_WORKSPACE = 4, /* workspace missing or smaller than the call needs         */
    BSF8_ERR_NULL = 5,      /* a required pointer is NULL                               */
    BSF8_ERR_CUDA = 6,      /* a CUDA runtime call failed (launch, attribute, copy)     */
    BSF8_ERR_TIMEOUT = 7,   /* a kernel gave up a bounded wait (device status only)     */
    BSF8_ERR_DEVICE = 8,    /* the current device is not sm_103 / cannot run the kernels */
    BSF8_ERR_VALUE = 9,     /* an option or scalar argument is out of range             */
    BSF8_ERR_INDEX = 10     /* a kernel met an index outside its table and skipped it   */
                            /* (device status only)                                     */
};

/* Largest row count a single bsf8_gemm call accepts.  The pages serve 2..8 and 9..192
 * decode / verify / draft rows from the twin and prefill through a rebuilt bf16 copy (the
 * drop mode); here prefill-sized calls run from the twin too: past 192 rows the
 * tensor-core kernel takes the tokens in tiles of 192. */
#define BSF8_MAX_M 16384

/* Returns a static, human-readable name for a status code. */
const char *bsf8_strerror(int status);

/* Library version as major*10000 + minor*100 + patch. */
int bsf8_version(void);

/* The CUDA runtime error code (a cudaError_t value) behind the most recent
 * BSF8_ERR_CUDA or BSF8_ERR_DEVICE returned by any call of this process, 0 if none
 * has occurred.  Kept process-wide (not per thread); for diagnostics only. */
int bsf8_last_cuda_error(void);

/* --------------------------------------------------------------------- make_twin
 * "wo_a_w8.py", make_twin(): per 32x32 block of the bf16 weight w[G][N][K]
 *   amax = max |w| (raised to at least 2^-126),  e = ceil(log2(amax/448)) in [-127,127],
 *   w8   = e4m3 round-to-nearest-even of w / 2^e,  exp = e + 127,
 *   block_ok = 1 iff bf16(e4m3 * 2^e) == w for all 1024 elements (value equality),
 * and *accepted = 1 iff every block is ok (the pages keep the twin only then).
 * Blocks holding NaN or Inf get block_ok = 0, exp = 0xFF and codes 0x7F (the pages
 * leave them undefined; the tensor is rejected either way).
 *   w        device, bf16 [G][N][K], 16-byte aligned
 *   w8       device, out, uint8 [G][N][K], 16-byte aligned
 *   exp      device, out, uint8 [G][N/32][K/32]
 *   block_ok device, out, uint8 [G][N/32][K/32], or NULL
 *   accepted device, out, one int32 (written 1 or 0 on the stream)
 * Errors: BSF8_ERR_NULL, BSF8_ERR_SHAPE, BSF8_ERR_ALIGN, BSF8_ERR_CUDA. */
int bsf8_make_twin(const void *w, uint8_t *w8, uint8_t *exp, uint8_t *block_ok,
                   int32_t *accepted, int G, int N, int K, bsf8_stream_t stream);

/* ----------------------------------------------------------------------- dequant
 * "wo_a_w8.py", _dequant_kernel(): out[g][n][k] = bf16( e4m3(w8[g][n][k]) *
 * 2^(exp[g][n/32][k/32] - 127) ), rounded to nearest even; exact for every code and
 * exponent byte (byte 255 is a +inf scale: 0 -> NaN, others -> +-inf; e4m3 NaN codes
 * give NaN).  The page's drop mode serves prefill from such a per-call copy.
 *   w8  device, uint8 [G][N][K], 16-byte aligned
 *   exp device, uint8 [G][N/32][K/32]
 *   out device, out, bf16 [G][N][K], 16-byte aligned
 * Errors: BSF8_ERR_NULL, BSF8_ERR_SHAPE, BSF8_ERR_ALIGN, BSF8_ERR_CUDA. */
int bsf8_dequant(const uint8_t *w8, const uint8_t *exp, void *out, int G, int N, int K,
                 bsf8_stream_t stream);

/* -------------------------------------------------------------------------- GEMM
 * "wo_a_w8.py", _wo_a_partial_w8() / _wo_a_mid_kernel() and their fixed-order
 * reduction (module docstring: "Split-K partials are summed in a fixed order"):
 *   y[m][g][n] = bf16( sum_{s=0..S-1} P[s][m][g][n] ),  summed s = 0, 1, ... in fp32,
 *   P[s][m][g][n] = sum over split s's columns of x[m][g*K+k] * bf16(W8[g][n][k]*2^e),
 * with the products accumulated in fp32 on the tensor cores.  Split s covers columns
 * [s*c*32, min(K, (s+1)*c*32)) with c = ceil((K/32)/S) (it may be empty).
 *   x         device, bf16 [M][ldx], 16-byte aligned, ldx a multiple of 8, ldx >= G*K
 *   w8, exp   the twin (layouts above); w8 16-byte aligned
 *   y         device, out, bf16 [M][G][N]
 *   M         1 .. BSF8_MAX_M
 *   split_k   0 = the library chooses (bsf8_gemm_auto_split), else 1 .. K/32
 *   workspace device scratch of at least bsf8_gemm_workspace_bytes(...) bytes, or
 *             NULL when that is 0: fp32 partials between the two passes, which the call
 *             runs when its kernel writes partials (the tensor-core kernel, M > 16, with
 *             more than 8 splits, or 2..8 splits whose blocks take more than one wave of
 *             the device's SMs -- past 192 rows at least ceil(K/2048) splits, as a token
 *             tile's accumulators must fit tensor memory; the other kernels when a slab of
 *             16 rows needs more than 64 column tasks, e.g. split_k > 64).  No zeroing is
 *             needed; it must not be shared by calls that can overlap.
 * The splits are summed inside one thread block, across a cluster of up to 8 blocks (16
 * for the decode-ahead tensor-core kernel, where the device schedules such clusters)
 * through distributed shared memory, or by the fixed-order reduce of a second pass, always
 * in the same fixed order as bsf8_gemm_partials followed by bsf8_splitk_reduce, which run
 * the same kernel (bsf8_gemm_kernel) and give the same bits.
 * The twin is treated as a static parameter: with programmatic dependent launch
 * (BSF8_OPT_PDL) the kernel starts reading w8 and exp while the kernel before it on the
 * stream may still run, if that kernel allows it (the library's kernels that write a
 * twin -- make_twin, pad_k -- never do; a caller's kernel that writes w8 or exp must not
 * trigger its dependents early).  x is read and y written only after that kernel ends
 * (before, x's rows may be prefetched into L2, which reads nothing into the call).
 * Errors: BSF8_ERR_NULL, BSF8_ERR_SHAPE, BSF8_ERR_ALIGN, BSF8_ERR_STRIDE,
 *         BSF8_ERR_WORKSPACE, BSF8_ERR_CUDA; BSF8_ERR_VALUE when BSF8_OPT_GEMM_PATH forces a
 *         kernel that cannot run the call. */
int bsf8_gemm(const void *x, const uint8_t *w8, const uint8_t *exp, void *y,
              int M, int N, int K, int G, int split_k, int64_t ldx,
              void *workspace, size_t workspace_bytes, bsf8_stream_t stream);

/* Workspace bsf8_gemm needs for these sizes (0 for most shapes; see bsf8_gemm). */
size_t bsf8_gemm_workspace_bytes(int M, int N, int K, int G, int split_k);

/* The split count bsf8_gemm uses for split_k = 0.  Returns a value in 1 .. K/32, or a
 * negative status for invalid sizes.  1 up to 8 rows, and for 9..32 rows where the
 * decode-ahead tensor-core kernel takes the call in one split (its one-split grid fits the
 * device's SMs); otherwise 1 up to 16 rows, and past 16 (the tensor-core kernel) as many
 * splits as keep its blocks in one wave of the current device's SMs, then enough that a
 * split's accumulators fit tensor memory.  With no device, past 16 rows a size-only rule
 * (at most 8) applies. */
int bsf8_gemm_auto_split(int M, int N, int K, int G);

/* Kernels of bsf8_gemm, as bsf8_gemm_kernel reports them and BSF8_OPT_GEMM_PATH forces them. */
enum {
    BSF8_KERNEL_STREAM = 2,          /* cp.async weight streaming, mma.sync (any M)          */
    BSF8_KERNEL_DECODE_AHEAD = 4,    /* weights rebuilt into tensor memory before the        */
                                     /* dependency wait, mma.sync (M <= 8)                   */
    BSF8_KERNEL_TENSOR_CORE = 5,     /* tcgen05 MMAs on 128-row blocks (any M, token tiles   */
                                     /* of 192)                                              */
    BSF8_KERNEL_WIDE = 6,            /* wide weights, codes widened to f16 (M <= 8)          */
    BSF8_KERNEL_DECODE_AHEAD_TC = 7  /* weights rebuilt into tensor memory as the tcgen05 A  */
                                     /* operand before the dependency wait (M <= 32)         */
};

/* The kernel bsf8_gemm -- and bsf8_gemm_partials, bsf8_gemm_static_scratch -- runs for these
 * sizes and split count (0 = the library's choice) under the current options and device: a
 * BSF8_KERNEL_* value.  Negative: -BSF8_ERR_SHAPE for invalid sizes, -BSF8_ERR_VALUE when
 * BSF8_OPT_GEMM_PATH forces a kernel that cannot run the call.  The choice never depends on
 * whether the caller asks for y or for the fp32 partials. */
int bsf8_gemm_kernel(int M, int N, int K, int G, int split_k);

/* First pass alone: writes the fp32 partials P[S][M][G][N] (S = split_k >= 1, every
 * split written, empty splits as +0) with the kernel bsf8_gemm runs for the same sizes and
 * split count.  Same arguments as bsf8_gemm.
 *   partials device, out, fp32 [S][M][G][N], 16-byte aligned
 * Errors: as bsf8_gemm. */
int bsf8_gemm_partials(const void *x, const uint8_t *w8, const uint8_t *exp,
                       float *partials, int M, int N, int K, int G, int split_k,
                       int64_t ldx, bsf8_stream_t stream);

/* Second pass alone ("wo_a_w8.py", the reduce after _partial_w8): for i < count,
 *   y[i] = bf16_rne( ((P[0][i] + P[1][i]) + P[2][i]) + ... + P[S-1][i] )
 * in fp32, left to right.
 *   partials device, fp32 [S][count]
 *   y        device, out, bf16 [count]
 * While the device status word holds BSF8_ERR_TIMEOUT (a first pass gave up a wait and
 * left incomplete partials) the kernel writes nothing; bsf8_device_status reads and
 * clears the word.
 * Errors: BSF8_ERR_NULL, BSF8_ERR_SHAPE, BSF8_ERR_CUDA. */
int bsf8_splitk_reduce(const float *partials, void *y, int S, int64_t count,
                       bsf8_stream_t stream);

/* The same fixed-order sum kept in fp32: y[i] = ((P[0][i] + P[1][i]) + ...) + P[S-1][i],
 * y a device float array of `count` values.  With bsf8_gemm_partials it gives the GEMM's
 * fp32 output -- the head variant of "docs/tp4-adapters.md" (draft_head_fp8: the block
 * logits of up to 64..128 rows as fp32, the head streamed once per call); with one split
 * the partials are that output already.  Errors and the timeout rule as bsf8_splitk_reduce. */
int bsf8_splitk_reduce_f32(const float *partials, float *y, int S, int64_t count,
                           bsf8_stream_t stream);

/* ------------------------------------- per-(row, 32-column) scales (1 x 32 blocks)
 * The adapter table of "docs/tp4-adapters.md" (draft_main_proj): e4m3 codes with one
 * power-of-two scale per (weight row, 32 columns), checked to reproduce the bf16 weight
 * exactly, for the draft's projection of up to 16 rows.  The pages give no formula for it;
 * these entry points take make_twin's rule with the block narrowed to 1 x 32.  Layouts as
 * above except the exponents (and make_twin_rows' flags): exp[G][N][K/32], byte e + 127.
 *   bsf8_make_twin_rows: as bsf8_make_twin, per 1 x 32 segment.
 *   bsf8_dequant_rows:   as bsf8_dequant with the per-row exponents.
 *   bsf8_gemm_rows:      as bsf8_gemm (same x, y, split rule and fixed-order sum) with the
 *                        per-row exponents, on the decode-ahead kernel for M <= 8 and on the
 *                        decode-ahead tensor-core kernel for 9..32 rows where bsf8_gemm uses
 *                        them, else on the cp.async streaming kernel (every M
 *                        up to BSF8_MAX_M; meant for the pages' <= 16 rows); split_k 0 means
 *                        1 up to 8 rows and where the decode-ahead tensor-core kernel takes
 *                        the call in one split, else the streaming kernel's choice; workspace per
 *                        bsf8_gemm_rows_workspace_bytes (0 unless a slab needs more than
 *                        64 column tasks).
 * Errors as the block-scale counterparts. */
int bsf8_make_twin_rows(const void *w, uint8_t *w8, uint8_t *exp, uint8_t *block_ok,
                        int32_t *accepted, int G, int N, int K, bsf8_stream_t stream);
int bsf8_dequant_rows(const uint8_t *w8, const uint8_t *exp, void *out, int G, int N, int K,
                      bsf8_stream_t stream);
size_t bsf8_gemm_rows_workspace_bytes(int M, int N, int K, int G, int split_k);
int bsf8_gemm_rows(const void *x, const uint8_t *w8, const uint8_t *exp, void *y, int M,
                   int N, int K, int G, int split_k, int64_t ldx, void *workspace,
                   size_t workspace_bytes, bsf8_stream_t stream);

/* --------------------------------------------------- GEMM without a workspace
 * The pages have no counterpart for this entry point; it serves callers that cannot
 * allocate device memory for a workspace -- e.g. a serving engine that has reserved all of
 * the GPU's memory for its own arena, or a plugin running inside one that may not call
 * the allocator.  With the split count bsf8_gemm uses (split_k 0: bsf8_gemm_auto_split):
 * where bsf8_gemm needs no workspace for the call (bsf8_gemm_workspace_bytes = 0: most
 * shapes, whose kernels sum their splits on chip) it is bsf8_gemm; otherwise it runs
 * bsf8_gemm_partials and then bsf8_splitk_reduce -- the same kernel and the same fixed-order
 * sum -- so its result equals bsf8_gemm's bit for bit, with the partials held in a buffer
 * compiled into the library:
 *   - the buffer is BSF8_STATIC_SCRATCH_BYTES (8 MiB) of device memory that every GPU
 *     which loads the library holds until the process exits;
 *   - a call that needs partials whose S*M*G*N*4 bytes (S = the split count used) exceed
 *     it returns BSF8_ERR_WORKSPACE without launching anything;
 *   - nothing is allocated and nothing needs clearing: every split writes all of its
 *     partials before the reduce reads them;
 *   - every call on a device shares that one buffer, so calls that can overlap on the GPU
 *     (on different streams, or on several host threads) race and must be serialised by
 *     the caller;
 *   - the first call on a device looks up the buffer's device address (a host call,
 *     cudaGetSymbolAddress), so make that first call before any stream capture.
 * Errors: as bsf8_gemm (BSF8_ERR_WORKSPACE as described: a call at exactly the limit runs). */
#define BSF8_STATIC_SCRATCH_BYTES (8u * 1024u * 1024u)

int bsf8_gemm_static_scratch(const void *x, const uint8_t *w8, const uint8_t *exp, void *y,
                             int M, int N, int K, int G, int split_k, int64_t ldx,
                             bsf8_stream_t stream);

/* --------------------------------------------------------------- L2 prefetch
 * "docs/tp4-adapters.md", adapter table, l2_prefetch row: pull a twin -- the codes
 * w8[G][N][K] and the exponents exp[G][N/32][K/32] -- into L2 ahead of the GEMM that reads
 * it, typically on a side stream while other work runs (collectives, kernels that do not
 * let the GEMM start early).  A hint: it reads nothing into the program and writes
 * nothing, so results are the same with or without it; the lines may be evicted again
 * before the GEMM runs if other traffic passes through L2 meanwhile.
 *   w8, exp  device, 16-byte aligned (exp's last partial 16 bytes are not prefetched)
 * Errors: BSF8_ERR_NULL, BSF8_ERR_SHAPE, BSF8_ERR_ALIGN, BSF8_ERR_CUDA. */
int bsf8_prefetch_l2(const uint8_t *w8, const uint8_t *exp, int G, int N, int K,
                     bsf8_stream_t stream);

/* ------------------------------------------------------------------------- pad-K
 * "shared_pad_k.py", _pad_weight(): the twin [G][N][K] becomes [G][N][Kp] with code 0
 * (+0) in the new columns and its exponents [G][N/32][K/32] become [G][N/32][Kp/32]
 * with pad_exp in the new block columns (127 = scale 1.0, the page's choice; any byte
 * but 255 leaves every output unchanged, since 0 * 2^e = 0).
 *   w8, exp           device, the input twin; w8 16-byte aligned
 *   w8_out, exp_out   device, out; w8_out 16-byte aligned
 *   Kp                a multiple of 32, >= K;  pad_exp  0 .. 255
 * Errors: BSF8_ERR_NULL, BSF8_ERR_SHAPE, BSF8_ERR_ALIGN, BSF8_ERR_VALUE, BSF8_ERR_CUDA. */
int bsf8_pad_k(const uint8_t *w8, const uint8_t *exp, uint8_t *w8_out, uint8_t *exp_out,
               int G, int N, int K, int Kp, int pad_exp, bsf8_stream_t stream);

/* "shared_pad_k.py", _pad_input(): x[M][ldx] (group g in columns [g*K, (g+1)*K))
 * becomes x_out[M][G*Kp] with +0 in the new columns of every group.
 *   x      device, bf16, 16-byte aligned, ldx a multiple of 8, ldx >= G*K
 *   x_out  device, out, bf16 [M][G*Kp], 16-byte aligned
 * Errors: BSF8_ERR_NULL, BSF8_ERR_SHAPE, BSF8_ERR_ALIGN, BSF8_ERR_STRIDE, BSF8_ERR_CUDA. */
int bsf8_pad_x(const void *x, int64_t ldx, void *x_out, int M, int G, int K, int Kp,
               bsf8_stream_t stream);

/* ================================================================ decode operators
 * What a decode, verify or draft pass runs beside its linear layers: queries and keys are
 * normed and rotated, keys and values go into a paged cache in the twin's number format with
 * one exponent per (row, 32 channels), a tree of drafted tokens attends to that cache, the
 * drafts are verified against the target's probabilities, and the kept ones move together.
 * The pages serve these passes (decode, verify, draft rows) but show none of these operators;
 * the format is bsf8_make_twin_rows' (e4m3 codes, exponent byte e + 127, the smallest
 * e >= -127 with 448 * 2^e >= amax; a block with an infinity or a NaN gets byte 255 and codes
 * 0x7F, and reads back as NaN).
 *
 * The cache: token `slot` of request b lies in page table[b][slot / page_size], row
 * slot % page_size.  A page holds [heads][page_size][dim] codes and
 * [heads][page_size][dim / 32] exponent bytes, for keys and for values.
 *   k8, v8      device, uint8 [pages][heads][page_size][dim], 16-byte aligned
 *   kexp, vexp  device, uint8 [pages][heads][page_size][dim / 32], 16-byte aligned
 *   page_size   a multiple of 16, 16 .. 1024;  dim  64, 128 or 256
 *   pages * heads * page_size < 2^31
 * The struct itself is host memory, read before the call returns.  table is a device array
 * int32 [requests][table_pages]; only entries of slots that a call touches are read.
 *
 * Indices that live on the device (table entries, slots, requests, positions, lengths)
 * cannot be checked on the host.  The kernels check them: an index outside its table makes
 * the kernel skip that row and record BSF8_ERR_INDEX in the device status word
 * (bsf8_device_status), and nothing outside the given buffers is read or written. */
typedef struct {
    uint8_t *k8, *kexp, *v8, *vexp;
    int pages, page_size, heads, dim;
} bsf8_kv_cache;

/* Most nodes of a token tree (its root, the last kept token, counts), and most cached tokens of a
 * request that attention reaches (slots and 16-token groups are counted in 31 and 26 bits there). */
#define BSF8_MAX_NODES 256
#define BSF8_MAX_LEN (1 << 30)

/* Norms, rotates and appends the projections of N tokens in one pass.  Per head row x of
 * dim channels, in fp32:
 *   y = x * w / sqrt(mean(x^2) + eps)            where the norm's weight w is given
 *   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin) for the first `rot` channels, the
 *   pairs (a, b) = (i, i + rot/2), or (2i, 2i + 1) when `interleaved`, with
 *   cos = cos_sin[pos][i] and sin = cos_sin[pos][rot/2 + i], i < rot/2
 * for queries and keys; queries are rounded once to bf16, keys and values (values neither
 * normed nor rotated) once to cache codes.
 *   q, k, v    device, bf16; head h of token n at q[n * ldq + h * dim] (ldk, ldv likewise);
 *              q may be NULL with Hq = 0: only keys and values are appended
 *   q_out      device, out, bf16 [N][Hq][dim]
 *   req, slot  device, int32 [N]: where token n goes; slot < 0: its k and v are not kept
 *              (a padded row), its q is written all the same
 *   pos        device, int32 [N] (0 .. positions - 1), needed where rot > 0; may differ from
 *              the slot: the siblings of a token tree share a position
 *   cos_sin    device, fp32 [positions][rot], 16-byte aligned
 *   rot        0 (no rotation) .. dim, a multiple of 16
 *   q_norm, k_norm  device, bf16 [dim], or NULL (no norm);  eps >= 0, finite
 * Pointers of bf16 rows 16-byte aligned, ld* multiples of 8.  Two tokens of a call must not
 * name the same (req, slot).  A token with a bad position is skipped whole (its q rows are
 * not written), one with a bad req, slot or page keeps its q rows.
 * Errors: BSF8_ERR_NULL, BSF8_ERR_SHAPE, BSF8_ERR_ALIGN, BSF8_ERR_STRIDE, BSF8_ERR_VALUE,
 *         BSF8_ERR_CUDA. */
int bsf8_qkv_append(const void *q, const void *k, const void *v, int64_t ldq, int64_t ldk,
                    int64_t ldv, void *q_out, const bsf8_kv_cache *cache, const int32_t *table,
                    int requests, int table_pages, const int32_t *req, const int32_t *slot,
                    const int32_t *pos, const float *cos_sin, int positions, int rot,
                    int interleaved, const void *q_norm, const void *k_norm, float eps, int N,
                    int Hq, bsf8_stream_t stream);

/* Reads N cached tokens back: k_out and v_out (device, out, bf16 [N][heads][dim], 16-byte
 * aligned; either may be NULL) get bf16(e4m3(code) * 2^(byte - 127)) of token slot[n] of
 * request req[n]; rows with slot < 0 become zeros, and so do rows with a bad index.
 * Errors: BSF8_ERR_NULL, BSF8_ERR_SHAPE, BSF8_ERR_ALIGN, BSF8_ERR_CUDA. */
int bsf8_kv_read(const bsf8_kv_cache *cache, const int32_t *table, int requests, int table_pages,
                 const int32_t *req, const int32_t *slot, void *k_out, void *v_out, int N,
                 bsf8_stream_t stream);

/* Attention of a token tree over the cache.  Request b has ctx[b] cached tokens (slots 0 ..
 * ctx[b] - 1) that every node sees, and nodes[b] tree nodes, already appended at slots
 * ctx[b] + j; query row t of the request is node t:
 *   out[b][t][h] = sum_l p_l v_l / sum_l p_l,   p_l = exp(scale * q[b][t][h] . k_l),
 * over the ctx[b] tokens and the nodes j < nodes[b] with bit j of mask[b][t] set (mask NULL:
 * j <= t, a chain; T = 1 is the single-token step).  Query head h reads cache head
 * h / (Hq / heads).  A row that sees nothing, and rows t >= nodes[b], give zeros and an lse of
 * -inf.  A key or a value block that holds NaN (exponent byte 255, as bsf8_qkv_append marks it; the
 * code 0x7F under another byte is not looked for) reaches exactly the rows that see it; a query head
 * with an infinity or a NaN gives NaN (its lse too) where it sees anything, and no other does.
 * Scores, sums and softmax statistics are fp32.  What goes into the products has fewer bits:
 *   - a query head: exact for channels within 2^14 of its largest, else off by at most 2^-22 of that;
 *   - p: rounded to 11 bits, and to 2^-33 of the row's largest below 2^-23 of it;
 *   - a value: exact within 2^20 of the largest one cached for its request and cache head (seen by
 *     the row or not), else off by at most 2^-24 of that; with up to 8 rows a head at dim 128 its
 *     product with p is held to 2^-35 of it.
 * The output's own rounding to bf16 (2^-9) is what shows unless values differ by more than these.
 *   q      device, bf16, 16-byte aligned; node t of request b at q + (b * T + t) * ldq, its
 *          heads one after another; ldq >= Hq * dim, a multiple of 8
 *   ctx    device, int32 [B];  nodes  device, int32 [B], or NULL (all T)
 *   mask   device, int32 [B][T][ceil(T / 32)], bit j % 32 of word j / 32, or NULL
 *   max_len  host: no request has more than max_len cached tokens, its nodes included
 *          (1 .. table_pages * page_size, at most BSF8_MAX_LEN); it sizes the launch, and
 *          longer requests count as BSF8_ERR_INDEX and are cut there
 *   out    device, out, bf16 [B][T][Hq][dim], 16-byte aligned
 *   lse    device, out, fp32 [B][T][Hq]: log of the sum of p_l, or NULL
 *   workspace  device, 16-byte aligned, of at least bsf8_tree_attention_workspace_bytes(...);
 *          no zeroing needed; not to be shared by calls that can overlap
 *   T      1 .. BSF8_MAX_NODES;  B  1 .. 1024;  Hq a multiple of heads;  scale finite, > 0
 * Errors: BSF8_ERR_NULL, BSF8_ERR_SHAPE, BSF8_ERR_ALIGN, BSF8_ERR_STRIDE, BSF8_ERR_VALUE,
 *         BSF8_ERR_WORKSPACE, BSF8_ERR_CUDA. */
int bsf8_tree_attention(const void *q, int64_t ldq, const bsf8_kv_cache *cache,
                        const int32_t *table, int table_pages, const int32_t *ctx,
                        const int32_t *nodes, const int32_t *mask, float scale, int max_len,
                        void *out, float *lse, int B, int T, int Hq, void *workspace,
                        size_t workspace_bytes, bsf8_stream_t stream);

/* Workspace bsf8_tree_attention needs (0 for invalid sizes). */
size_t bsf8_tree_attention_workspace_bytes(int B, int T, int Hq, int heads, int dim);

/* Verifies drafted token trees against the target's probabilities by recursive rejection, so
 * that the kept tokens and the next one are distributed as the target's own.  Request b's
 * tree has nodes[b] nodes; node 0 is the last token kept before, parent[b][i] < i.  p[b][i] is
 * the target's distribution after node i, q[b][i] the draft's, from which the children of i
 * were drawn independently; q NULL: the children were not drawn at random (a draft's top
 * tokens), each then counts as drawn from a distribution that has only its token.
 * The walk starts at node 0.  At node c, with R = P(c) and Z = 2^40, its children are asked in
 * order of their index; child i with token x and number u = u[b][i]:
 *   Q' = floor(Q(c) * Z / 2^40);   kept if floor(floor(u * 2^24) * Q'(x) / 2^24) < R(x):
 *   the walk goes on at node i; else R = max(R - Q', 0), Z = sum of R, next child,
 * where P(x) = floor(p(x) * 2^40), Q likewise (p and q clamped to [0, 1], a NaN counts as 0).
 * When no child is kept, the next token is drawn from R (from P(c) where R is all 0): the
 * lowest x with  R(0) + .. + R(x) > floor(floor(u[b][0] * 2^24) * sum of R / 2^24),  V - 1
 * where there is none.  All of it in integers: the result does not depend on any order.
 *   p, q    device, fp32, node i of request b at p + (b * T + i) * ld, 16-byte aligned
 *   tokens  device, int32 [B][T] (0 .. V - 1; [b][0] is not read)
 *   parent  device, int32 [B][T] ([b][0] is not read)
 *   u       device, fp32 [B][T], uniform in [0, 1), multiples of 2^-24 used whole
 *   nodes   device, int32 [B], or NULL (all T)
 *   path    device, out, int32 [B][T]: the kept nodes in order, node 0 first, then -1
 *   count   device, out, int32 [B]: how many are kept (node 0 counts)
 *   token   device, out, int32 [B]: the next token
 *   T  1 .. BSF8_MAX_NODES;  V  1 .. 2^20;  ld >= V
 * A child with a bad token or parent is never kept (BSF8_ERR_INDEX).
 * Errors: BSF8_ERR_NULL, BSF8_ERR_SHAPE, BSF8_ERR_ALIGN, BSF8_ERR_STRIDE, BSF8_ERR_CUDA. */
int bsf8_verify_tree(const float *p, const float *q, int64_t ld, const int32_t *tokens,
                     const int32_t *parent, const float *u, const int32_t *nodes, int32_t *path,
                     int32_t *count, int32_t *token, int B, int T, int V, bsf8_stream_t stream);

/* Moves the kept nodes of each request's tree together: for i < count[b], slot
 * ctx[b] + path[b][i] -> ctx[b] + i, keys and values, codes and exponents, bit for bit.
 * path[b] is strictly increasing over the first count[b] (as bsf8_verify_tree gives it); the
 * slots behind keep what they held.  An entry below 0 or its own place, or not above the one
 * before it, is left out, and a count outside 0 .. T is cut to that (BSF8_ERR_INDEX).
 *   ctx, count  device, int32 [B];  path  device, int32 [B][T];  T  1 .. BSF8_MAX_NODES
 * Errors: BSF8_ERR_NULL, BSF8_ERR_SHAPE, BSF8_ERR_ALIGN, BSF8_ERR_CUDA. */
int bsf8_kv_commit(const bsf8_kv_cache *cache, const int32_t *table, int table_pages,
                   const int32_t *ctx, const int32_t *path, const int32_t *count, int B, int T,
                   bsf8_stream_t stream);

/* Plans a step: whose pages come back, which pages the new tokens get, where each token goes.  The books
 * of the pages live on the device, and the call keeps them:
 *   table       int32 [B][table_pages]: row b's first held[b] entries are its pages
 *   held        int32 [B]
 *   free_pages  int32 [pool]: a stack of free pages, the first *free_count of them
 *   free_count  int32 [1]
 * A page is one row's alone, or lies on the stack once: a row that leaves gives all of its pages back, so that one which
 * another row holds too would be handed out while it is read, and twice (nothing here looks for that).  Requests that share
 * pages need tables and counts of users of the caller's own; the calls that read a table take such rows.
 * In this order, the requests from the first to the last each time:
 *   - where done[b] is not 0 (done NULL: nowhere) the row's pages go back onto the stack, entry by entry, and
 *     held[b] becomes 0;
 *   - a request with lens[b] tokens and add[b] > 0 new ones needs max(0, ceil((lens + add) / page_size) - held)
 *     pages.  It is granted its tokens where that is 0 or where the pages needed by it and all requests
 *     before it are on the stack, and where the tokens asked for by it and those before it are at most N.
 *     What is granted pages takes them from the top of the stack, one after another.
 * Then the granted tokens lie one after another, request by request:
 *   req, slot   int32 [N], out: token i's request and its slot, lens[b] onwards; behind the last one 0 and -1
 *               (rows that bsf8_qkv_append does not keep)
 *   start       int32 [B + 1], out: where each request's tokens begin; start[B] is how many there are
 *   granted     int32 [B], out: add[b] or 0
 * lens, add and done are int32 [B] and stay as they are (lens grows by what is kept of the step: the
 * caller's).  Table entries past a row's pages and the stack above its count keep what they held.
 * A row with lens or add below 0, or past table_pages * page_size together, counts as add 0; held outside
 * 0 .. table_pages, a count outside 0 .. pool and pages that the stack has no room for are cut off
 * (BSF8_ERR_INDEX in the device status, each).
 *   B  1 .. 1024;  N  0 .. 2^30;  pool  1 .. 2^30;  page_size as in the cache;  table_pages * page_size and
 *   table_pages * B below 2^31;  none of the arrays may overlap.
 * Errors: BSF8_ERR_NULL, BSF8_ERR_SHAPE, BSF8_ERR_ALIGN, BSF8_ERR_CUDA. */
int bsf8_kv_plan(int32_t *table, int table_pages, int page_size, int32_t *held, int32_t *free_pages,
                 int32_t *free_count, int pool, const int32_t *lens, const int32_t *add, const int32_t *done,
                 int32_t *req, int32_t *slot, int32_t *start, int32_t *granted, int B, int N,
                 bsf8_stream_t stream);

/* Bounds of the pages' keys, for bsf8_select_pages: per page, head and channel the largest (hi) and
 * smallest (lo) key as 8-bit integers under one power of two per 32 channels, byte e + 127:
 * the smallest e >= -127 with 127 * 2^e >= every |hi|, |lo| of the 32, codes ceil(hi / 2^e) and
 * floor(lo / 2^e).  Byte 255 and codes 0 where a key's 32 channels are marked NaN (byte 255) or infinite.
 *   codes  device, int8 [pages][heads][2][dim] (hi, lo), 16-byte aligned
 *   exps   device, uint8 [pages][heads][dim / 32], on dim / 32 bytes
 * The sizes are the cache's. */
typedef struct {
    int8_t *codes;
    uint8_t *exps;
    int pages, page_size, heads, dim;
} bsf8_page_bounds;

/* Writes the bounds of the pages that became full: of request b the pages with their last slot in
 * [start[b], end[b]), that is pages start / page_size .. end / page_size - 1 (int32 [B], start NULL: 0).  After a
 * prompt or a commit: its requests' lengths before and after.  Values are taken as bf16, which they are
 * exactly (below 2^-126 rounded to its grid).  A start below 0, an end below it or past the table: none of that
 * request's; a bad page: not that one (BSF8_ERR_INDEX).  The same page may be given twice.
 *   table  device, int32 [B][table_pages];  B  1 .. 1024;  B * table_pages below 2^31
 * Errors: BSF8_ERR_NULL, BSF8_ERR_SHAPE (bounds of other sizes than the cache's among it), BSF8_ERR_ALIGN,
 *         BSF8_ERR_CUDA. */
int bsf8_kv_bounds(const bsf8_kv_cache *cache, const bsf8_page_bounds *bounds, const int32_t *table,
                   int table_pages, const int32_t *start, const int32_t *end, int B, bsf8_stream_t stream);

/* The pages that attention of a step reads, for each request and cache head: of the request's
 * ctx / page_size full pages the `keep` with the highest scores (all where there are fewer), equal ones by
 * their index, in ascending order; then the pages that hold the rest of the context and the nodes.
 * The score is an upper bound of the sum of q . k over the query rows that share the cache head (its
 * nodes[b] nodes, Hq / heads heads each), but for the roundings of q:
 *   a    = the rows' largest |q| (elements that are infinite or NaN count as 0), 2^k <= a < 2^(k+1), k >= -100
 *   Q+_d = sum over the rows of max(n, 0),  Q-_d = sum of min(n, 0),  n = rint(q_d * 2^(17 - k))
 *   both (Q + 2^(s-1)) >> s, s >= 0 the smallest that leaves the largest |Q| 14 bits (s = 0: as they are)
 *   score = sum over 32-channel blocks, added in pairs (fp32), of fp32(sum_d Q+_d hi_d + Q-_d lo_d) 2^(e - 27)
 * and +inf for a page with a byte 255, for the first `sink` pages and the last `recent` full ones, and where the sum
 * is NaN (bytes above 249, which bsf8_kv_bounds does not write, can add up to infinities of both signs).
 *   q       as in bsf8_tree_attention;  ctx, nodes, max_len too
 *   bounds  of every full page of the requests
 *   pages   device, out, int32 [B][heads][width], width = bsf8_select_width(T, page_size, keep): page numbers
 *           (the table's entries), -1 behind the last one
 *   kept    device, out, int32 [B]: tokens of the context in them, keep * page_size + ctx % page_size at most
 * With these, bsf8_sparse_attention finds context and nodes as bsf8_tree_attention does.
 *   keep  1 .. BSF8_MAX_SELECT_PAGES;  sink, recent >= 0, together at most keep;  max_len / page_size at most
 *   BSF8_MAX_SELECT_PAGES;  T * Hq / heads at most 4096;  B  1 .. 1024
 * A page number outside the bounds scores lowest of all (BSF8_ERR_INDEX); lengths as in bsf8_tree_attention.
 * Errors: BSF8_ERR_NULL, BSF8_ERR_SHAPE, BSF8_ERR_ALIGN, BSF8_ERR_STRIDE, BSF8_ERR_VALUE, BSF8_ERR_CUDA. */
#define BSF8_MAX_SELECT_PAGES 49152
int bsf8_select_pages(const void *q, int64_t ldq, const bsf8_page_bounds *bounds, const int32_t *table,
                      int table_pages, const int32_t *ctx, const int32_t *nodes, int max_len, int keep,
                      int sink, int recent, int32_t *pages, int32_t *kept, int B, int T, int Hq,
                      bsf8_stream_t stream);

/* keep plus the most pages that the rest of a context and T nodes take; 0 for invalid arguments. */
int bsf8_select_width(int T, int page_size, int keep);

/* bsf8_tree_attention over a block table for each request and cache head, as bsf8_select_pages gives it:
 * pages int32 [B][heads][width] in table's place, kept [B] in ctx's, the rest as there (its workspace
 * too; max_len at most width * page_size, at least kept + nodes of every request).
 * Errors: as bsf8_tree_attention. */
int bsf8_sparse_attention(const void *q, int64_t ldq, const bsf8_kv_cache *cache, const int32_t *pages,
                          int width, const int32_t *kept, const int32_t *nodes, const int32_t *mask,
                          float scale, int max_len, void *out, float *lse, int B, int T, int Hq,
                          void *workspace, size_t workspace_bytes, bsf8_stream_t stream);

/* A token from each row of logits.  With m the row's largest logit and t its temperature, a logit x weighs
 *   w = 2^40 for x = m, else floor(2^40 * 2^-y) for y = (m - x) * (log2(e) / t) <= 40, 0 beyond
 * (fp32 steps, each rounded; 2^-y by a polynomial to 2^-21.9 of itself; -inf and NaN weigh 0).  t below 2^-126 or
 * NaN counts as 0: only the lowest index of x = m weighs.  Of these stay, in this order,
 *   top_k   the first k by (larger x, then lower index);  k <= 0 or >= V: all
 *   min_p   those with w >= ceil(min_p * 2^40);  NaN counts as 0, above 1 as 1
 *   top_p   in the same order, those before which less than max(1, floor(floor(p * 2^24) * W / 2^24)) has been
 *           given, W the sum of w by then;  p >= 1 or NaN: all;  p < 0 counts as 0
 * and the token is the lowest x with  w(0) + .. + w(x) > floor(floor(u * 2^24) * W / 2^24) over those that
 * stay, W their sum.  All sums are of integers: the result depends on no order.
 *   logits  device, bf16 (bf16 != 0) or fp32, row n at element n * ld, 16-byte aligned, ld >= V
 *   u       device, fp32 [N], uniform in [0, 1)
 *   temperature, top_p, min_p  device, fp32 [N], top_k int32 [N]; NULL: 1, all, none, all
 *   token   device, out, int32 [N]; -1 for a row of nothing but -inf and NaN
 *   p       device, out, fp32 [N]: the token's share w / W (0 for token -1), off by at most 2^-22 of itself
 *   N  0 .. 2^20;  V  1 .. 2^20
 * Errors: BSF8_ERR_NULL, BSF8_ERR_SHAPE, BSF8_ERR_ALIGN, BSF8_ERR_STRIDE, BSF8_ERR_CUDA. */
int bsf8_sample_tokens(const void *logits, int bf16, int64_t ld, const float *u, const float *temperature,
                       const int32_t *top_k, const float *top_p, const float *min_p, int32_t *token, float *p,
                       int N, int V, bsf8_stream_t stream);

/* The distributions that bsf8_sample_tokens draws from: p[n][x] = w / W of those that stay, 0 of the others
 * (as bsf8_verify_tree takes p and q).  p device, out, fp32 [N][V], 16-byte aligned.  Else as there. */
int bsf8_token_probs(const void *logits, int bf16, int64_t ld, const float *temperature, const int32_t *top_k,
                     const float *top_p, const float *min_p, float *p, int N, int V, bsf8_stream_t stream);

/* From one block to the next: per row of H channels, in fp32,
 *   z = x * rsqrt(mean(x^2) + eps) * post_weight     (post_weight NULL: z = x)
 *   r = residual + scale * gate * z                  (residual NULL: 0;  no gate: 1)
 *   h = r * rsqrt(mean(r^2) + eps) * weight          (of r before its rounding)
 * A row's bits depend on the row, H, fp32 and what is applied alone, not on how many rows come with it.
 *   x            device, bf16 [M][ldx];  post_weight, weight  device, bf16 [H]
 *   residual     device, [M][ldr], fp32 where fp32 != 0, else bf16
 *   gate         device, bf16: BSF8_GATE_CHANNEL [H], BSF8_GATE_TOKEN one of each row at gate[m * ldg],
 *                BSF8_GATE_FULL [M][ldg]
 *   r_out        device, out, [M][H] of the residual's type, or NULL; may be the residual itself (ldr = H)
 *   h_out        device, out, bf16 [M][H], or NULL (then weight is not read); may be x itself (ldx = H)
 * Pointers 16-byte aligned (a token gate's: 2), ldx, ldg (full) and ldr multiples of 16 bytes.
 *   H  8 .. BSF8_MAX_HIDDEN, a multiple of 8;  eps >= 0, scale finite
 * Errors: BSF8_ERR_NULL, BSF8_ERR_SHAPE, BSF8_ERR_ALIGN, BSF8_ERR_STRIDE, BSF8_ERR_VALUE, BSF8_ERR_CUDA. */
#define BSF8_MAX_HIDDEN 32768
enum { BSF8_GATE_NONE = 0, BSF8_GATE_CHANNEL = 1, BSF8_GATE_TOKEN = 2, BSF8_GATE_FULL = 3 };
int bsf8_residual_norm(const void *x, int64_t ldx, const void *residual, int64_t ldr, int fp32,
                       const void *post_weight, const void *gate, int gate_kind, int64_t ldg, float scale,
                       const void *weight, float eps, void *r_out, void *h_out, int M, int H,
                       bsf8_stream_t stream);

/* ------------------------------------------------------------------ diagnostics
 * Not part of the method: a measurement aid.  Launches 2*nsm one-warp blocks on `stream`;
 * the block on SM i writes out[2i] = the global nanosecond timer and out[2i+1] = SM i's
 * cycle counter (slots of SMs no block reached keep their contents).  Two samples around
 * a timed region give each SM's average clock over it.
 *   out  device, uint64 [nsm][2];  nsm  1 .. 4096 (the device's SM count)
 * Errors: BSF8_ERR_NULL, BSF8_ERR_SHAPE, BSF8_ERR_CUDA, BSF8_ERR_DEVICE. */
int bsf8_sm_clock_sample(uint64_t *out, int nsm, bsf8_stream_t stream);

/* --------------------------------------------------------------- status, options
 * Synchronises `stream`, then reads into *status (host) and clears the device status
 * word of the current device: BSF8_OK, or BSF8_ERR_TIMEOUT if a kernel gave up a
 * bounded wait since the last read (its outputs are then undefined).
 * Errors: BSF8_ERR_NULL, BSF8_ERR_CUDA. */
int bsf8_device_status(int *status, bsf8_stream_t stream);

/* Process-wide options (host state, read at each launch). */
enum {
    BSF8_OPT_PDL = 1,              /* 1 (default): programmatic dependent launch on    */
    BSF8_OPT_WAIT_TIMEOUT_NS = 2,  /* bound of every in-kernel wait (default 2e9 ns)   */
    BSF8_OPT_DEBUG_SKIP_LOADS = 3, /* test only: the GEMM kernels that wait on         */
                                   /* mbarriers (decode-ahead, decode-ahead tensor-    */
                                   /* core, tensor-core, wide-weight) issue no weight  */
                                   /* loads, the attention kernels none of the cache,  */
                                   /* the norms of many rows none at all, so their     */
                                   /* bounded waits run out and the call ends with     */
                                   /* BSF8_ERR_TIMEOUT in the status                   */
    BSF8_OPT_GEMM_PATH = 4         /* 0 (default): the kernel chosen by shape:         */
                                   /*  - up to 8 token rows: the decode-ahead kernel   */
                                   /*    when its grid fits two blocks an SM, else the */
                                   /*    wide-weight kernel at split_k 1, else the     */
                                   /*    cp.async streaming kernel;                    */
                                   /*  - 9..32 rows: the decode-ahead tensor-core      */
                                   /*    kernel when its plan holds (S x tasks of at   */
                                   /*    most 512 columns <= 16, past 8 where the      */
                                   /*    device schedules such clusters) and its grid  */
                                   /*    fits one block an SM;                         */
                                   /*  - else 9..16 rows: the tensor-core kernel at    */
                                   /*    split_k 1 over at least one 128-row block per */
                                   /*    SM, the streaming kernel otherwise;           */
                                   /*  - beyond 16 rows: the tensor-core kernel.       */
                                   /* Else a BSF8_KERNEL_* value forces that kernel:   */
                                   /* 2 streaming (any call); 4 decode-ahead (M <= 8); */
                                   /* 5 tensor-core; 6 wide-weight (M <= 8; K and the  */
                                   /* split's columns multiples of 128, at most 6144   */
                                   /* columns a split); 7 decode-ahead tensor-core     */
                                   /* (M <= 32, S x ceil(split columns / 512) <= 16).  */
                                   /* A call the forced kernel cannot run returns      */
                                   /* BSF8_ERR_VALUE (see bsf8_gemm_kernel).           */
};
/* Errors: BSF8_ERR_VALUE for an unknown option or a negative value. */
int bsf8_set_option(int option, int64_t value);
int64_t bsf8_get_option(int option);

#ifdef __cplusplus
}
#endif

#endif /* BSF8_H */
