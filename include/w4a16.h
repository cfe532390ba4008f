/*
 * w4a16.h — C ABI of libw4a16.so: weight-only INT4 x FP16 matmul on GB300 (sm_103a).
 *
 *   Y[M][N] = X[M][K] (FP16) x dequant(Wq)[K][N],   dequant(Wq)[k][n] = (q[k][n] - 8) * s[k/G][n]
 *
 * accumulated in FP32 and stored as FP16 (round to nearest even).
 *
 * The operation is the one the pages on the Marlin kernel describe:
 *  - "quant_marlin_kernel" (aicassindra.com), "The architecture: every piece
 *    explained": INT4 codes packed eight to a 32-bit word in a kernel-specific
 *    permuted order, one FP16 scale per group of weights along the reduction
 *    dimension (commonly 128), unpack to FP16 and multiply by the group scale,
 *    tensor-core MMA against FP16 activations, split-K with a global reduction
 *    of partial sums; activations stay FP16 and the output is FP16.
 *  - same page, "End-to-end flow": activations (tokens x in-features) times
 *    weights (in-features x out-features); repacking is done once, offline.
 *  - "Low-Precision Quantization Kernels in Production" (llms.blog), section 1
 *    (Marlin, "Pre-Permuted Weight Layouts"): the packed layout is a contract
 *    between the repacking step and the kernel; section 3 (FlashInfer): split-K
 *    with a deterministic reduction in global memory, CUDA Graph capture.
 * The zero-point 8 is the symmetric reading (the pages print no zero-point).
 * w4a16_gemm_zp takes one integer zero-point z[g][n] in 0..15 per group and
 * column instead: dequant(Wq)[k][n] = (q[k][n] - z[k/G][n]) * s[k/G][n], the
 * 4-bit format of AWQ checkpoints, which "Low-Precision Quantization Kernels in
 * Production" (llms.blog), section 1, lists among those the Marlin family serves.
 *
 * Conventions for every entry point:
 *  - Pointers named "device" are CUDA device pointers of the current device,
 *    owned by the caller, and must be 16-byte aligned. Arrays are row-major and
 *    contiguous. FP16 values are passed as IEEE binary16 bit patterns (uint16_t).
 *  - Work is enqueued on `stream` (NULL = the legacy default stream) and the
 *    call returns without synchronising. Results are ready when the stream is.
 *  - A call that returns anything but W4A16_OK has launched nothing, except
 *    W4A16_ERR_CUDA from a failed launch (see w4a16_last_cuda_error()).
 *  - Group size G must be 32, 64 or 128, or equal to K (one scale per column);
 *    G = -1 is accepted as "equal to K". K must be a multiple of 8 (16-byte X
 *    rows) and N a multiple of 8 (16-byte Y rows). A shape whose tensor-core
 *    schedule would exceed 2^31 pipeline stages (about 2^31 * 16384 multiply-adds,
 *    far beyond device memory) is rejected with W4A16_ERR_INVALID_ARG.
 *  - The GEMM kernels are launched with programmatic dependent launch: a GEMM
 *    may start, and start streaming its packed weights, scales and zero-points,
 *    before the kernel enqueued just ahead of it on the stream has finished; it
 *    waits for that kernel before it reads x, bias or residual and before it
 *    writes y. So the kernel enqueued immediately before a GEMM on the same
 *    stream must not write that GEMM's packed weights, scales or zero-points.
 *    The repack calls (w4a16_pack, w4a16_pack_zeros, w4a16_sp_pack,
 *    w4a16_w8_pack) end with a kernel that writes nothing for this reason, so a
 *    GEMM may follow them directly. After writing packed buffers with a kernel
 *    of your own, enqueue another ordinary kernel (one launched without
 *    programmatic serialization) or synchronise before the GEMM.
 */
#ifndef W4A16_H
#define W4A16_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; declared here so the header needs no CUDA headers. */
struct CUstream_st;
typedef struct CUstream_st* w4a16_stream_t;

typedef enum {
    W4A16_OK = 0,
    W4A16_ERR_INVALID_ARG = 1,  /* a size, pointer, alignment or group size is invalid */
    W4A16_ERR_UNSUPPORTED = 2,  /* the device is not compute capability 10.3 (sm_103)  */
    W4A16_ERR_CUDA = 3,         /* a CUDA runtime call failed; code in w4a16_last_cuda_error() */
    W4A16_ERR_TIMEOUT = 4,      /* a kernel gave up waiting on one of its own pipeline barriers */
    W4A16_ERR_WORKSPACE = 5     /* the caller's workspace is smaller than w4a16_workspace_bytes() */
} w4a16_status;

/* Version of the packed layout written by w4a16_pack and read by the GEMM. Packed
 * buffers are a contract with this library: repack when the version changes. */
int w4a16_layout_version(void);

/* Static text for a status code. */
const char* w4a16_status_string(int status);

/* The cudaError_t of the last W4A16_ERR_CUDA returned on this host thread (0 if none). */
int w4a16_last_cuda_error(void);

/* Number of uint32 words of the packed weights: ceil(N/128) * KC * 1024, with
 * KC = ceil(K/64) rounded up to a multiple of 4 (K padded to a multiple of 256).
 * Returns 0 for invalid sizes. */
size_t w4a16_packed_words(int K, int N, int group_size);

/* Number of FP16 elements of the packed scales: ceil(N/128) * ceil(K/G) * 128.
 * Returns 0 for invalid sizes. */
size_t w4a16_scales_elems(int K, int N, int group_size);

/*
 * Repack codes and scales once, offline ("End-to-end flow": the layout is
 * computed once and exploited on every forward pass).
 *   codes          device, uint8 [K][N], values 0..15 (only the low nibble is read)
 *   scales         device, binary16 [ceil(K/G)][N] (or bfloat16 for w4a16_bf16_gemm:
 *                  the scales are copied as 16-bit patterns)
 *   packed         device out, uint32 [w4a16_packed_words(K, N, G)]
 *   scales_packed  device out, binary16 [w4a16_scales_elems(K, N, G)]
 * Packed layout (version 2): column tiles of 128 output features, reduction
 * chunks of 64. For tile nt, chunk kc, half j (32 values of k), feature n_in
 * and word w: word index (((nt*KC + kc)*2 + j)*128 + n_in)*4 + w with
 * KC = ceil(K/64) rounded up to a multiple of 4; the word holds
 * k0 = kc*64 + j*32 + w*8 .. k0+7 of column n = nt*128 + n_in, nibble i (bits 4i..4i+3) holding k = k0 + 2*(i%4) + i/4.
 * Positions outside K x N hold code 8 (weight 0). Scales: element
 * (nt*ceil(K/G) + g)*128 + n_in holds s[g][nt*128 + n_in] (0 outside N).
 */
w4a16_status w4a16_pack(const uint8_t* codes, const uint16_t* scales,
                        uint32_t* packed, uint16_t* scales_packed,
                        int K, int N, int group_size, w4a16_stream_t stream);

/*
 * Y = X x dequant(W), FP32 accumulation, FP16 output.
 *   x              device, binary16 [M][K]
 *   packed         device, output of w4a16_pack for (K, N, G)
 *   scales_packed  device, output of w4a16_pack for (K, N, G)
 *   y              device out, binary16 [M][N]; must not overlap the inputs
 * M = 0 is a no-op. Uses a per-device workspace that the library allocates on
 * the first call on each device (about 40 MB); make that first call outside
 * CUDA Graph capture. Calls on one device that run concurrently on different
 * streams share that workspace and must not overlap in time; use
 * w4a16_gemm_ws with separate workspaces for that. Repeated calls with equal
 * inputs give bit-identical outputs.
 */
w4a16_status w4a16_gemm(const uint16_t* x, const uint32_t* packed, const uint16_t* scales_packed,
                        uint16_t* y, int M, int N, int K, int group_size, w4a16_stream_t stream);

/* Bytes of caller workspace w4a16_gemm_ws needs for this shape, in any weight
 * format of this library (0 for invalid sizes). */
size_t w4a16_workspace_bytes(int M, int N, int K, int group_size);

/*
 * As w4a16_gemm, with a caller-owned device workspace of at least
 * w4a16_workspace_bytes(M, N, K, G) bytes, 256-byte aligned, ZEROED ONCE by the
 * caller before its first use; the kernels leave it ready for the next call.
 * This variant never allocates, so it can be captured into a CUDA Graph on
 * its first call. Returns W4A16_ERR_WORKSPACE if ws_bytes is too small.
 */
w4a16_status w4a16_gemm_ws(const uint16_t* x, const uint32_t* packed,
                           const uint16_t* scales_packed, uint16_t* y,
                           int M, int N, int K, int group_size,
                           void* workspace, size_t ws_bytes, w4a16_stream_t stream);

/* Activation of w4a16_gemm_fused, applied after the bias add. */
typedef enum {
    W4A16_ACT_NONE = 0,
    W4A16_ACT_SILU = 1, /* z / (1 + e^-z) */
    W4A16_ACT_RELU = 2  /* max(z, 0) */
} w4a16_activation;

/*
 * Y = act(X x dequant(W) + bias) + residual: the GEMM with the operations that
 * follow it in a layer fused into its epilogue ("quant_marlin_kernel", "End-to-end
 * flow": the output tile flows straight into a bias add and an activation), so Y
 * is written once instead of being re-read by separate kernels. The bias add, the
 * activation and the residual add run in FP32 on the accumulator; the result is
 * rounded once to FP16.
 *   bias       device, binary16 [N], or NULL for none
 *   residual   device, binary16 [M][N] row-major, or NULL for none; it may be the
 *              same buffer as y (an in-place y += ...) but must not otherwise
 *              overlap y
 *   activation a w4a16_activation
 *   workspace  as for w4a16_gemm_ws (ws_bytes bytes, zeroed once), or NULL to use
 *              the library's own workspace as w4a16_gemm does
 * Every other argument, layout and error is that of w4a16_gemm / w4a16_gemm_ws.
 * Returns W4A16_ERR_INVALID_ARG for an unknown activation or an odd bias or
 * residual address.
 */
w4a16_status w4a16_gemm_fused(const uint16_t* x, const uint32_t* packed,
                              const uint16_t* scales_packed, uint16_t* y,
                              int M, int N, int K, int group_size,
                              const uint16_t* bias, const uint16_t* residual, int activation,
                              void* workspace, size_t ws_bytes, w4a16_stream_t stream);

/*
 * w4a16_gemm_fused on row-strided activations, outputs and residual: X row m
 * starts at x + m * ldx, Y row m at y + m * ldy, residual row m at residual +
 * m * ldr (elements). A layer can read the leading K columns of a wider output
 * (the first 4096 of a fused QKV projection, the first 11008 of a gate/up
 * projection) and write into a slice of a wider buffer without a copy; the pages
 * have no counterpart (their kernels read contiguous activations).
 *   ldx  >= K, a multiple of 8 (rows start on 16-byte boundaries)
 *   ldy  >= N;   ldr >= N when residual is given (ignored otherwise)
 * Every other argument, layout and error is that of w4a16_gemm_fused; the rows of
 * Y must not overlap X or the residual (other than residual == y, same stride).
 * Returns W4A16_ERR_INVALID_ARG for strides outside these bounds.
 */
w4a16_status w4a16_gemm_strided(const uint16_t* x, int ldx, const uint32_t* packed,
                                const uint16_t* scales_packed, uint16_t* y, int ldy,
                                int M, int N, int K, int group_size,
                                const uint16_t* bias, const uint16_t* residual, int ldr, int activation,
                                void* workspace, size_t ws_bytes, w4a16_stream_t stream);

/* Bytes of the packed zero-points: ceil(N/128) * ceil(K/G) * 64 (two 4-bit
 * zero-points a byte). Returns 0 for invalid sizes. */
size_t w4a16_zeros_bytes(int K, int N, int group_size);

/*
 * Repack per-group zero-points once, offline, into the tile order the
 * zero-point GEMM streams beside the scales.
 *   zeros         device, uint8 [ceil(K/G)][N], values 0..15 (only the low nibble is read)
 *   zeros_packed  device out, uint8 [w4a16_zeros_bytes(K, N, G)], 16-byte aligned
 * Layout: byte (nt*ceil(K/G) + g)*64 + b holds z[g][nt*128 + 2b] in bits 0..3 and
 * z[g][nt*128 + 2b + 1] in bits 4..7; columns past N hold 8.
 * The codes and scales are packed by w4a16_pack as for the symmetric format.
 */
w4a16_status w4a16_pack_zeros(const uint8_t* zeros, uint8_t* zeros_packed, int K, int N, int group_size,
                              w4a16_stream_t stream);

/*
 * Y = act(X x dequant(W) + bias) + residual with per-group zero-points:
 * dequant(W)[k][n] = (q[k][n] - z[k/G][n]) * s[k/G][n]. (1024 + q) - (1024 + z)
 * is formed exactly in FP16, so the dequantised weight is rounded once, at the
 * product with the scale, as in the symmetric format.
 *   zeros_packed   device, output of w4a16_pack_zeros for (K, N, G); must not be NULL
 * Every other argument (bias, residual and activation may be NULL / 0 for a plain
 * GEMM; workspace NULL for the library's own), layout and error is that of
 * w4a16_gemm_fused. Zero-points all equal to 8 give bit-identical results to
 * w4a16_gemm_fused.
 */
w4a16_status w4a16_gemm_zp(const uint16_t* x, const uint32_t* packed, const uint16_t* scales_packed,
                           const uint8_t* zeros_packed, uint16_t* y, int M, int N, int K, int group_size,
                           const uint16_t* bias, const uint16_t* residual, int activation,
                           void* workspace, size_t ws_bytes, w4a16_stream_t stream);

/* ---------------------------------------------------------------- BF16 activations
 * The 4-bit GEMM (zero-point 8, layout of w4a16_pack) with every 16-bit tensor in
 * bfloat16 instead of binary16: X, the scales, bias, residual and Y, passed as
 * bfloat16 bit patterns (uint16_t). Both tensor-core operands are BF16: the weights
 * are dequantised to BF16, (128 + q) - 136 = q - 8 exactly, then one rounding at
 * the product with the scale (BF16 keeps 8 significant bits, so each weight
 * carries up to 2^-8 relative error against 2^-11 in the FP16 form).
 * ("Low-Precision Quantization Kernels in Production" (llms.blog), introduction:
 * FP16 and BF16 are the 16-bit types the weights are quantised from and the
 * tensor cores run.)
 *   scales_packed  w4a16_pack's scales output for BF16 scales (the repack copies
 *                  16-bit patterns, so the same call serves both types)
 * Every other argument, layout and error is that of w4a16_gemm_fused.
 */
w4a16_status w4a16_bf16_gemm(const uint16_t* x, const uint32_t* packed, const uint16_t* scales_packed,
                             uint16_t* y, int M, int N, int K, int group_size,
                             const uint16_t* bias, const uint16_t* residual, int activation,
                             void* workspace, size_t ws_bytes, w4a16_stream_t stream);

/* ---------------------------------------------------------------- 2:4 sparse 4-bit codes
 * Sparse-MARLIN ("MARLIN: Mixed-Precision Auto-Regressive Parallel Inference on
 * Large Language Models" note, key results: INT4 weights with 2:4 sparsity): the
 * 4-bit GEMM (zero-point 8, FP16) on codes that are 2:4 sparse along k, i.e. at
 * most two codes other than 8 (weight 0) in every aligned group of four k of a
 * column. Only two codes per group are stored, with their 2-bit positions, and
 * the sparse tensor-core MMA skips the other two: half the MMAs and 3/4 of the
 * weight bytes of the dense format. The result is that of w4a16_gemm_fused on the
 * same codes (exactly the same products, in another order of summation). */

/* Bytes of the sparse packed weights: ceil(N/128) * (KC/2) * 6144, KC as for
 * w4a16_packed_words. Returns 0 for invalid sizes. */
size_t w4a16_sp_packed_bytes(int K, int N, int group_size);

/*
 * Repack 2:4 sparse codes and scales once, offline.
 *   codes          device, uint8 [K][N], values 0..15, at most two codes other than 8
 *                  in every aligned group of four k of a column
 *   scales         device, binary16 [ceil(K/G)][N]
 *   packed         device out, uint8 [w4a16_sp_packed_bytes(K, N, G)], 16-byte aligned
 *   scales_packed  device out, binary16 [w4a16_scales_elems(K, N, G)] (as w4a16_pack)
 *   violations     device, 8-byte aligned counter, or NULL: the kernel adds the number
 *                  of groups that hold more than two codes other than 8 (those keep
 *                  their first two, so their results differ from the dense GEMM)
 * Sparse layout (version 1): chunks of 128 values of k (KC/2 per column), 6144
 * bytes per (column tile nt, chunk sc) at (nt*(KC/2) + sc)*6144:
 *   4096 bytes of stored codes: word ((b*128 + n_in)*4 + wd) holds stored values
 *     j0 = b*32 + wd*8 .. j0+7 of column nt*128 + n_in, nibble i holding stored
 *     value j0 + 2*(i%4) + i/4; stored value j is the code at k = 128*sc + 4*(j/2) +
 *     (position j%2 of group j/2);
 *   2048 bytes of position words, in the order the sparse MMA reads them from
 *     tensor memory: word (L*4 + mm), nibble u describes group t = 4*((L%16)/8) +
 *     u%4 of k = 128*sc + 32*mm + 4t .. +3 of column nt*128 + 16*(L/16) + 8*(u/4) +
 *     L%8: bits 0..1 the position (0..3) of the group's first stored code, bits
 *     2..3 that of its second (first < second).
 * A group stores the positions of its codes other than 8 in increasing order,
 * filled up to two with the smallest free positions (code 8). Padding (k >= K,
 * n >= N): code 8 at positions 0 and 1.
 */
w4a16_status w4a16_sp_pack(const uint8_t* codes, const uint16_t* scales, uint8_t* packed,
                           uint16_t* scales_packed, int K, int N, int group_size,
                           unsigned long long* violations, w4a16_stream_t stream);

/*
 * Y = act(X x dequant(W) + bias) + residual for 2:4 sparse codes packed by
 * w4a16_sp_pack. Arguments, epilogue and workspace as for w4a16_gemm_fused.
 */
w4a16_status w4a16_sp_gemm(const uint16_t* x, const uint8_t* packed, const uint16_t* scales_packed,
                           uint16_t* y, int M, int N, int K, int group_size,
                           const uint16_t* bias, const uint16_t* residual, int activation,
                           void* workspace, size_t ws_bytes, w4a16_stream_t stream);

/* ---------------------------------------------------------------- W8A16: 8-bit codes
 * The same GEMM for 8-bit weights: dequant(Wq)[k][n] = (q[k][n] - 128) * s[k/G][n],
 * q in 0..255, one FP16 scale per group ("Low-Precision Quantization Kernels in
 * Production" (llms.blog), section 1: the Marlin family serves 8-bit checkpoints
 * as well as 4-bit ones; 128 is the symmetric zero-point of unsigned 8-bit codes,
 * the pages print none). */

/* Bytes of the 8-bit packed codes: ceil(N/128) * KC * 8192, KC as for
 * w4a16_packed_words. Returns 0 for invalid sizes. */
size_t w4a16_w8_packed_bytes(int K, int N, int group_size);

/*
 * Repack 8-bit codes and scales once, offline.
 *   codes          device, uint8 [K][N], values 0..255
 *   scales         device, binary16 [ceil(K/G)][N]
 *   packed         device out, uint8 [w4a16_w8_packed_bytes(K, N, G)], 16-byte aligned
 *   scales_packed  device out, binary16 [w4a16_scales_elems(K, N, G)] (as w4a16_pack)
 * Packed layout (8-bit, version 1): column tiles of 128 output features, chunks of
 * 64 values of k, each in four quarters of 16. Byte
 * (((nt*KC + kc)*4 + j4)*128 + n_in)*16 + b belongs to word b/4, which holds
 * k0 = kc*64 + j4*16 + 4*(b/4) .. k0+3 of column nt*128 + n_in; bytes 0, 1, 2, 3 of
 * the word hold k0, k0+2, k0+1, k0+3. Positions outside K x N hold 128 (weight 0).
 */
w4a16_status w4a16_w8_pack(const uint8_t* codes, const uint16_t* scales, uint8_t* packed,
                           uint16_t* scales_packed, int K, int N, int group_size,
                           w4a16_stream_t stream);

/*
 * Y = act(X x dequant(W) + bias) + residual for 8-bit codes. (1024 + q) - 1152 is
 * q - 128 exactly in FP16; the dequantised weight is rounded once, at the product
 * with the scale.
 *   packed         device, output of w4a16_w8_pack for (K, N, G)
 * bias, residual, activation and workspace as for w4a16_gemm_fused (NULL / 0 for a
 * plain GEMM); w4a16_workspace_bytes covers this format too.
 */
w4a16_status w4a16_w8_gemm(const uint16_t* x, const uint8_t* packed, const uint16_t* scales_packed,
                           uint16_t* y, int M, int N, int K, int group_size,
                           const uint16_t* bias, const uint16_t* residual, int activation,
                           void* workspace, size_t ws_bytes, w4a16_stream_t stream);

/*
 * Synchronises `stream`, then reads and clears the error word that the kernels
 * set when one of their bounded waits gave up (W4A16_ERR_TIMEOUT), for the
 * given workspace. NULL covers the library's own workspace of the current device,
 * the error word of the kernels that run without a workspace (the decode and the
 * CUDA-core kernel) and, once a w4a16_gemm_noalloc call has run on that device,
 * the fixed array that call uses. After a timeout the split-K counters of the workspace (or
 * array) are reset as well.
 */
w4a16_status w4a16_check_device_status(void* workspace, w4a16_stream_t stream);

/*
 * Self-test of failure detection (no counterpart in the pages): launches one warp
 * that waits, with the kernels' own bounded wait, on a barrier that nothing ever
 * completes. After limit_ns (1 .. 10^10) the wait gives up, sets the error word of
 * `workspace` (NULL = the library's own workspace of the current device) and the
 * kernel returns; w4a16_check_device_status then reports W4A16_ERR_TIMEOUT and
 * clears it. The context stays usable. Nothing faults, traps or hangs.
 */
w4a16_status w4a16_selftest_wait_timeout(void* workspace, long long limit_ns, w4a16_stream_t stream);

/*
 * Sets the limit of every bounded wait in the kernels launched after this call
 * (default 1 s, or W4A16_WAIT_LIMIT_NS read at the first call on a device), for
 * tests of failure detection; no counterpart in the pages. A wait that runs out
 * makes its CTA give up: it stops issuing, waits (with a fixed 1 s bound) for the
 * copies and MMAs it already issued, frees its tensor memory and returns, and the
 * error word reports W4A16_ERR_TIMEOUT (w4a16_check_device_status); the results of
 * that launch are not valid. limit_ns <= 0 changes nothing. Returns the previous
 * limit. Applies to every device and host thread of the process.
 */
long long w4a16_set_wait_limit_ns(long long limit_ns);

/* Which kernel the dispatcher picks for a shape of the 4-bit FP16 format
 * (w4a16_gemm, w4a16_gemm_ws, w4a16_gemm_fused) on the current device. It picks
 * path 3 by itself for up to eight rows of X when K is a multiple of 32, and for up to
 * sixteen on layers of at most 4096 x 4096 with N >= 16 x the SM count (where it
 * measured faster on GB300), path 2 otherwise; path 1 only when forced:
 *   *path = 1: the CUDA-core kernel for one to four rows of X ("Low-Precision
 *              Quantization Kernels in Production" (llms.blog), section 2: the
 *              activation vector held on chip, weights streamed, unpacked in
 *              registers, group-scaled and reduced across a warp; section 5: at
 *              batch 1 the matmul is a memory-bound GEMV). *tile_m = the rows of X
 *              it is built for (1, 2 or 4); *grid = CTAs, one per block of 16 or
 *              32 output columns, each over the whole of K (no workspace is used).
 *   *path = 2: the tensor-core kernel (dequantised weights in tensor memory,
 *              tcgen05 MMA); *tile_m = rows of X per tile; *grid = CTAs.
 *   *path = 3: the decode kernel for one to sixteen rows of X ("quant_marlin_kernel",
 *              "The architecture": register-level unpack feeding the tensor-core
 *              MMA from registers; here warp-level MMAs). *tile_m = the rows of X
 *              it is built for (8 or 16); *grid = CTAs, one per block of 16 to 128
 *              output columns, each over the whole of K (no workspace is used).
 * The other weight formats always run path 2. */
w4a16_status w4a16_plan(int M, int N, int K, int group_size, int* path, int* tile_m, int* grid);

/* Forces the dispatcher's choice for the 4-bit FP16 format, for tests and
 * ablations (no counterpart in the pages): 0 = automatic (the default), 1 = the
 * CUDA-core kernel for every shape it serves (M <= 4), 2 = the tensor-core kernel
 * for every M, 3 = the decode kernel for every shape it serves (M <= 16, K a
 * multiple of 32). Shapes a forced path does not serve run path 2. Applies to every
 * later call in the process, on every device and host thread. Returns the previous
 * setting, or -1 (nothing changed) for another value. */
int w4a16_force_path(int path);

/*
 * w4a16_gemm without any device allocation by the library or the caller. The
 * pages have no counterpart; this entry point exists for callers that may not
 * allocate GPU memory at all: plug-ins whose host framework owns every byte of
 * device memory, and latency-critical loops that cannot afford cudaMalloc's
 * implicit device-wide synchronisation.
 *   Arguments, layouts and results are those of w4a16_gemm; the caller still
 *   passes x, packed, scales_packed and y.
 *   The split-K scratch of the tensor-core kernel (error word, tile counters,
 *   FP32 partials) lives in one fixed device array of W4A16_NOALLOC_MAX_BYTES
 *   inside the library, held by every GPU that loads the library until the
 *   process exits. A shape whose scratch would exceed it returns
 *   W4A16_ERR_WORKSPACE with nothing launched (on a 152-SM GB300 this admits
 *   every shape with M <= 32; at larger M only shapes the dispatcher gives few
 *   split tiles, such as 4096x12288 at M = 64; 4096x4096 at M = 64 needs
 *   8 MiB + 4352 bytes and is rejected). Shapes the decode kernel takes
 *   (M <= 8, K a multiple of 32) use no scratch at all, only its error word.
 *   The first call on each device looks the array's device address up; make
 *   that first call before any stream capture.
 *   A call that uses the scratch enqueues a clear of its tile counters, then the
 *   GEMM; the error word is left for w4a16_check_device_status(NULL, ...), which
 *   reads and clears it. Arguments are checked before anything is enqueued: a
 *   refused call touches nothing. Every call on a device shares the one array:
 *   calls whose work overlaps on the GPU (different streams, no ordering between
 *   them) race and give wrong results; order them on one stream or with events.
 *   Allocates nothing: no cudaMalloc, no cudaFree, no allocating library call.
 */
#define W4A16_NOALLOC_MAX_BYTES ((size_t)8 << 20)
w4a16_status w4a16_gemm_noalloc(const uint16_t* x, const uint32_t* packed,
                                const uint16_t* scales_packed, uint16_t* y,
                                int M, int N, int K, int group_size, w4a16_stream_t stream);

/* ---------------------------------------------------------------- the serving step
 * What a decoder runs beside its 4-bit matmuls: norms of queries and keys and their
 * rotation by position, a paged key-value cache held in 4 or 8 bits (block tables, new
 * keys and values, attention) and the sampling of the next token. The pages have no counterpart. All calls enqueue on `stream` without
 * synchronising and can be captured into a CUDA Graph (the first call on a device
 * outside capture); lengths, tables and settings are device arrays that are read
 * when the kernels run. Results are the same on every call with equal inputs.
 * The kernels are launched with programmatic dependent launch too: one may take its
 * place on the GPU early, but reads and writes nothing in memory before the kernel
 * enqueued ahead of it has finished, and lets the next one start only after that.
 * So any kernel may precede them, and a GEMM that follows one of them directly
 * reads its weights early only from what was complete before that call's kernel.
 *
 * The cache: uint8 [pages][kv_heads][page_size / 16][16 * (D + 6)], 16-byte aligned,
 * w4a16_kv4_page_bytes() a page; D = head_dim is 64 or 128, page_size 16, 32, 64, 128
 * or 256. Slot s is token s mod page_size of page s / page_size. A tile of 16 tokens:
 *   K codes   [16][D/2]: byte j of a token holds d = 2j in bits 0..3, 2j + 1 in bits 4..7
 *   V codes   [2][8][4][D/32][2] 16-bit words: word (h, n, c, w, e) holds, in bits
 *             4i..4i+3, d = n*D/8 + 4w + i of token 8h + 2c + e
 *   K scales  binary16 [16];  V scales  binary16 [16]
 *   K zero-points  uint8 [16];  V zero-points  uint8 [16]
 * A stored value is (code - zero) * scale, one scale and zero-point for a token's row
 * of D values. A row x is stored, in FP32 with IEEE operations, as
 *   lo = min(x, 0), hi = max(x, 0), s = binary16(min((hi - lo) / 15, 65504)), r = 1 / s,
 *   zero = clamp(rint(-lo * r), 0, 15), code = clamp(rint(x * r) + zero, 0, 15)
 * (s = 0: codes and zero-point 0). A row that holds an infinity or a NaN gets scale
 * NaN, which shows in whatever reads it. Memory of the cache that no slot was written
 * to may hold anything. */
typedef enum { W4A16_FP16 = 0, W4A16_BF16 = 1, W4A16_FP32 = 2 } w4a16_dtype;

/* Bytes of one page of the cache (0 for sizes it does not have). */
size_t w4a16_kv4_page_bytes(int kv_heads, int head_dim, int page_size);

/*
 * Block tables and slot maps of a batch, from its lengths, in one launch.
 *   seq_lens     device, int32 [batch]: tokens of each request with this step's new ones
 *   new_lens     device, int32 [batch]: this step's new tokens (negative counts as 0)
 *   free_pages   device, int32 [n_free]: pages nobody holds, taken in order
 *   taken_in     device, int32 [1]: how many of them are taken already; NULL: none
 *   taken_out    device out, int32 [1]: how many are taken after this call; more than
 *                n_free means that pages were short. Must not be taken_in. Nothing puts pages
 *                back: a new free list, with those of requests that have ended, is the caller's
 *   block_table  device in/out, int32 [batch][max_pages]: columns below
 *                ceil((seq - new) / page_size) are kept; those below ceil(seq / page_size)
 *                get pages from the free list, requests in order (-1 where it is short);
 *                the others get -1
 *   slots        device out, int64 [max_tokens]: the new tokens' slots, request by
 *                request; -1 for a token without a page, at a negative position or
 *                past max_pages, and for places past the batch's new tokens
 *   positions    device out, int32 [max_tokens]: their positions, seq - new + i; -1 past them
 *   starts       device out, int32 [batch + 1]: each request's first new token, and their
 *                sum. Tokens past max_tokens are counted but get no slot.
 */
w4a16_status w4a16_kv4_tables(const int32_t* seq_lens, const int32_t* new_lens, int batch,
                              const int32_t* free_pages, int n_free, const int32_t* taken_in,
                              int32_t* taken_out, int32_t* block_table, int max_pages, int page_size,
                              int64_t* slots, int32_t* positions, int max_tokens, int32_t* starts,
                              w4a16_stream_t stream);

/*
 * Quantises new keys and values into their slots.
 *   k, v     device, binary16 or bfloat16, token t's head h at t * token_stride +
 *            h * head_stride elements (slices of a fused projection's output work);
 *            16-byte aligned, strides multiples of 8 and at least head_dim
 *   slots    device, int64 [tokens]; slots outside the cache (such as -1) are skipped.
 *            A slot given twice ends with one of its rows, K and V each whole or mixed.
 *   cache    device in/out, of `pages` pages
 *   dtype    W4A16_FP16 or W4A16_BF16
 */
w4a16_status w4a16_kv4_append(const void* k, int64_t k_token_stride, int64_t k_head_stride,
                              const void* v, int64_t v_token_stride, int64_t v_head_stride,
                              const int64_t* slots, uint8_t* cache, int pages, int tokens,
                              int kv_heads, int head_dim, int page_size, int dtype,
                              w4a16_stream_t stream);

/* The values that slots stand for, rounded once to dtype (any w4a16_dtype): k and v are
 * device out, [tokens][kv_heads][head_dim], 16-byte aligned; slots outside the cache read 0. */
w4a16_status w4a16_kv4_read(const uint8_t* cache, int pages, const int64_t* slots, void* k, void* v,
                            int tokens, int kv_heads, int head_dim, int page_size, int dtype,
                            w4a16_stream_t stream);

/* Bytes of caller workspace w4a16_kv4_attention needs on the current device (0 if the
 * device cannot be used). */
size_t w4a16_kv4_workspace_bytes(void);

/*
 * Causal attention of new query tokens over the cache, which holds their own keys and
 * values already: query i of a request with n queries and s cached tokens has position
 * s - n + i and sees the cached tokens at positions up to its own and, if window > 0,
 * above its own minus window. out = softmax(scale * q K^T) V; a query that sees nothing
 * gets zeros (and lse -infinity). Query heads h * g .. h * g + g - 1 share KV head h
 * (g = q_heads / kv_heads).
 *   q, out       device, binary16 or bfloat16 [tokens][q_heads][head_dim] at token and
 *                head strides in elements (multiples of 8, at least head_dim), 16-byte
 *                aligned; out must not overlap an input
 *   block_table  device, int32 rows of table_cols pages, table_stride apart (at least
 *                table_cols, or 0: one row for every request); an entry outside the cache
 *                hides its tokens, as do tokens past the last column (positions count them)
 *   seq_lens     device, int32 [batch]; starts: device, int32 [batch + 1], request b's
 *                queries are tokens starts[b] .. starts[b + 1] - 1 (as w4a16_kv4_tables
 *                writes them). Tokens of no request are not written.
 *   lse          device out, float [tokens][q_heads]: log of the softmax's sum, or NULL
 *   max_q        the largest number of queries of a request, or more: it chooses the
 *                kernel; results hold for any value
 *   scale        the softmax scale, usually 1 / sqrt(head_dim)
 *   workspace    w4a16_kv4_workspace_bytes() bytes, 256-byte aligned, zeroed once; or
 *                NULL for the library's own (shared with the GEMMs: calls that use it
 *                must not overlap in time on different streams)
 */
w4a16_status w4a16_kv4_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                 const uint8_t* cache, int pages, const int32_t* block_table,
                                 int64_t table_stride, int table_cols, const int32_t* seq_lens,
                                 const int32_t* starts, void* out, int64_t out_token_stride,
                                 int64_t out_head_stride, float* lse, int batch, int tokens,
                                 int q_heads, int kv_heads, int head_dim, int page_size, int max_q,
                                 float scale, int window, int dtype, void* workspace,
                                 size_t ws_bytes, w4a16_stream_t stream);

/* Forces the kernel of w4a16_kv4_attention, for tests and ablations: 0 = automatic (the
 * default), 1 = the stream-K kernel for every request, 2 = the tcgen05 kernel for every
 * request of more than 32 rows (query token, head of a group) of a call whose max_q says
 * that there may be one. Applies to every later call in the process. Returns the previous
 * setting, or -1 (nothing changed) for another value. */
int w4a16_kv4_force_path(int path);

/* Positions.
 *
 * A rotation turns the first `rot` values of a head's row (rot a multiple of 8, at most head_dim) by angles of the row's
 * position: pair i, of angle i, is (x[i], x[i + rot / 2]), or (x[2i], x[2i + 1]) if `interleaved` is 1 (0 otherwise):
 *   (a, b) -> (a cos - b sin, b cos + a sin)       in FP32
 * w4a16_kv8_append rounds each product and sum of it; w4a16_qk_norm_rope puts its factors together first and sums by fused
 * operations, so the two may differ in an FP32 number's last bits. The angles' cosines and sines come from a table, device
 * float [rope_rows][rot], 16-byte aligned: of each position rot / 2 cosines, then rot / 2 sines. Scaled or learned angles
 * are a matter of the table.
 *
 * w4a16_rope_table fills one with the angles p * base^(-2i / rot) of positions p = 0 .. rows - 1, computed in 64 bits. */
w4a16_status w4a16_rope_table(float* table, int rows, int rot, double base, w4a16_stream_t stream);

/*
 * Norms of queries and keys for each head, then the rotation, in one pass; rounded once:
 *   y = x / sqrt(mean(x^2) + eps) * weight, over a row of head_dim values, mean and factors in FP32
 * Before that rounding a result is within 2^-20 of |y| (rotated: of |a cos| + |b sin|) of its value, where no square or
 * sum of squares passes FP32's range (the mean of bfloat16 values above 2^63 is infinite).
 *   q, k       device, binary16 or bfloat16 [tokens][heads][head_dim] at token and head strides in elements (multiples of
 *              8, at least head_dim), 16-byte aligned. q_heads or kv_heads 0: without queries or keys, whose
 *              pointers and strides are then not looked at
 *   q_out, k_out  device out, likewise; the input itself at its own strides (in place), or memory that overlaps no input
 *   q_weight, k_weight  device, [head_dim] of the inputs' type, 16-byte aligned; NULL: no norm
 *   positions  device, int32 [tokens]; NULL, with rope: no rotation. Rows of a negative position are not written, those of
 *              a position past the table's rows become NaN
 */
w4a16_status w4a16_qk_norm_rope(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                void* q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                                const void* k, int64_t k_token_stride, int64_t k_head_stride,
                                void* k_out, int64_t k_out_token_stride, int64_t k_out_head_stride,
                                const void* q_weight, const void* k_weight, float eps,
                                const int32_t* positions, const float* rope, int rope_rows, int rot,
                                int interleaved, int tokens, int q_heads, int kv_heads, int head_dim,
                                int dtype, w4a16_stream_t stream);

/* The cache in 8 bits: as the 4-bit one, with codes of 8 bits and one scale for a tile of 16 tokens and head, where the 4-bit
 * one has a scale and a zero-point for each token: uint8 [pages][kv_heads][page_size / 16][32 * D + 16], 16-byte aligned,
 * w4a16_kv8_page_bytes() a page. Tables and slots are the same (w4a16_kv4_tables). A tile:
 *   K codes   [D/64][16][64]: byte i of token t in slab p is d = 64p + i
 *   V codes   [D/64][2][8][4][4][2][2]: byte (p, h, n, c, j, e, i) is d = 64p + 8n + 2j + i of token 8h + 2c + e
 *   K scale, V scale  float, of all 16 tokens;  8 bytes unused
 * A stored value is (code - 128) * scale. Memory of the cache that no slot was written to may hold anything. */

/* Bytes of one page of the cache (0 for sizes it does not have). */
size_t w4a16_kv8_page_bytes(int kv_heads, int head_dim, int page_size);

/*
 * Quantises new keys, rotated on the way, and values into their slots. Tokens that are neighbours in the list and
 * whose slots are neighbours in one tile (s, s + 1, ...) are a run and are stored together, K and V alike, in FP32
 * with IEEE operations: with a = max |x| * (1 / 127) over the run's rows of a head (0 below 2^-40, at most 2^40) and old the tile's
 * scale, or 0 if the run begins at the tile's first token,
 *   s = max(old, a), r = 1 / s, code = clamp(rint(x * r), -127, 127) + 128      (s = 0: 128)
 * and where s > old the codes of the tile's tokens before the run become clamp(rint((code - 128) * (old * r)), -127, 127) + 128.
 * So a tile's tokens are to be written in their order, from its first one on, as a request's are, and each tile by one run of a
 * call; two runs of one call in a tile leave any values in it, and one that begins within a tile that was not begun takes
 * whatever is in memory for its scale. Tokens written again (drafts that were not accepted) are written again in order; the scale stays
 * as large as it was. A row with an infinity or a NaN, or a key at a position that the table does not have, makes the
 * scale NaN, which shows in whatever reads a token of that tile and head until the tile is begun again.
 * Tokens stored earlier thus change with their tile's later ones, by up to half a step of the new scale: where the 4-bit cache's partly
 * filled pages may be shared by requests that go on apart, or read on another stream while their tails are written, this one's
 * may not (its full tiles may). Each such request wants a copy of the tile, and a reader of it to wait.
 *   k, v, slots, cache, dtype  as w4a16_kv4_append
 *   positions, rope, rope_rows, rot, interleaved  the keys' rotation; positions and rope NULL: none
 */
w4a16_status w4a16_kv8_append(const void* k, int64_t k_token_stride, int64_t k_head_stride,
                              const void* v, int64_t v_token_stride, int64_t v_head_stride,
                              const int64_t* slots, const int32_t* positions, const float* rope,
                              int rope_rows, int rot, int interleaved, uint8_t* cache, int pages,
                              int tokens, int kv_heads, int head_dim, int page_size, int dtype,
                              w4a16_stream_t stream);

/* The values that slots stand for, as w4a16_kv4_read. */
w4a16_status w4a16_kv8_read(const uint8_t* cache, int pages, const int64_t* slots, void* k, void* v,
                            int tokens, int kv_heads, int head_dim, int page_size, int dtype,
                            w4a16_stream_t stream);

/* Bytes of caller workspace w4a16_kv8_attention needs on the current device (0 if the
 * device cannot be used). */
size_t w4a16_kv8_workspace_bytes(void);

/* Causal attention of new query tokens over the 8-bit cache: arguments, masks and results as
 * w4a16_kv4_attention, its workspace w4a16_kv8_workspace_bytes() bytes. Requests of many rows (the tcgen05
 * kernel's) have their probabilities times V's scale fed as binary16 numbers, relative to the largest
 * scale of the request so far: tiles whose scale is more than 2^20 times smaller lose bits. For bfloat16
 * outputs it is one such number, 11 bits, an eighth of an output's rounding; for binary16 outputs, and for
 * few rows whatever the output, 22 bits. Which requests have many rows (more than 32 of a KV head, in batches with
 * a request of more than 60, or 96 of head_dim 64, and 2400 rows of all heads) is a choice by speed alone. */
w4a16_status w4a16_kv8_attention(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                 const uint8_t* cache, int pages, const int32_t* block_table,
                                 int64_t table_stride, int table_cols, const int32_t* seq_lens,
                                 const int32_t* starts, void* out, int64_t out_token_stride,
                                 int64_t out_head_stride, float* lse, int batch, int tokens,
                                 int q_heads, int kv_heads, int head_dim, int page_size, int max_q,
                                 float scale, int window, int dtype, void* workspace,
                                 size_t ws_bytes, w4a16_stream_t stream);

/* Forces the kernel of w4a16_kv8_attention, as w4a16_kv4_force_path. */
int w4a16_kv8_force_path(int path);

/*
 * Samples one token per row. With m the row's maximum and e(x) = exp((x - m) / T) in
 * FP32, a token weighs rint(2^31 e(x)), a whole number, so that sums are exact and do not
 * depend on their order. Tokens are ranked by logit, equal ones by index. In turn, top-k
 * keeps ranks below k; top-p keeps a token if the weight ranked before it is below p times
 * the weight of what top-k kept; min-p keeps e(x) >= min_p; the first rank is always
 * kept. The result is the first token, in index order, at which the running kept weight
 * exceeds floor(u * kept weight). NaN logits count as -infinity; a row without a
 * logit above -infinity gives token -1 and probability 0.
 *   logits       device, [batch] rows row_stride elements apart (at least vocab, or 0: one
 *                row, drawn from batch times), vocab (at most 262144) valid; W4A16_FP16, W4A16_BF16 or W4A16_FP32, any element alignment
 *   u            device, float [batch], uniform in [0, 1)
 *   temperature  device, float [batch], or NULL for 1; not above 0: the largest logit
 *   top_k        device, int32 [batch], or NULL; 0 or less: no limit
 *   top_p, min_p device, float [batch], or NULL for 1 and 0
 *   token        device out, int32 [batch];  prob: device out, float [batch], the token's
 *                share of the kept weight, or NULL
 */
w4a16_status w4a16_sample(const void* logits, int64_t row_stride, const float* u,
                          const float* temperature, const int32_t* top_k, const float* top_p,
                          const float* min_p, int32_t* token, float* prob, int batch, int vocab,
                          int dtype, w4a16_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* W4A16_H */
