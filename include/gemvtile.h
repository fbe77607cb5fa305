/*
 * gemvtile.h -- C ABI of the MI355X (gfx950) FP16 / BF16 GEMM and GEMV library,
 * with block-scaled 8-bit products, products grouped by expert, products with
 * 4-bit weights, and the norm and routing around them.
 *
 * Every entry point takes plain pointers and sizes; no C++ or framework type
 * crosses this boundary.  All matrices are dense and row-major.  "fp16" means
 * IEEE 754 binary16; "bf16" means bfloat16 (1 sign bit, 8 exponent bits with
 * bias 127, 7 fraction bits: the upper half of a binary32).  Device pointers are HIP device (or managed) pointers on
 * the device that is current for the calling host thread.
 *
 * Ownership: the caller allocates and frees every buffer.  The library keeps
 * no pointer after a call returns and allocates no device memory on these
 * paths (no hidden workspace).
 *
 * Streams: every compute call is stream-ordered and asynchronous.  It
 * enqueues its kernel on `stream` (a hipStream_t; NULL is the default stream)
 * and returns at once; the result is ready when that stream reaches the
 * point of the call.  Errors found before the launch are returned without any
 * HIP call being made, so they are reported identically on a machine with no
 * GPU.
 *
 * Aliasing: D (or y) must not overlap A, B (or x, W); doing so is undefined.
 * Thread safety: calls from several host threads are safe; the library's only
 * mutable state is a per-device cache of the compute-unit count.
 */
#ifndef GEMVTILE_H
#define GEMVTILE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes returned by every entry point. */
enum gemvtile_status {
    GEMVTILE_OK = 0,
    GEMVTILE_ERR_INVALID_ARG = 1, /* NULL pointer with a nonzero extent, negative size */
    GEMVTILE_ERR_UNSUPPORTED = 2, /* K % 8 != 0 (16 in 8 bits), misaligned pointer, size beyond the limits below */
    GEMVTILE_ERR_LAUNCH = 3,      /* the HIP launch failed (no gfx950 device, bad stream, ...) */
    GEMVTILE_ERR_DEVICE = 4,      /* a HIP runtime query failed */
    GEMVTILE_ERR_SCRATCH = 5      /* gemm_splitk_f16_noalloc: partial sums beyond its static scratch */
};

/*
 * gemm_f16 -- D = A · Bᵀ with FP32 accumulation and one final rounding of each
 * output to fp16, round-to-nearest, ties to even.
 *
 *   D[m,n] = fp16_rne( sum_{k<K} A[m,k] * B[n,k] )   for m < M, n < N
 *
 * Defined by "使用 TMA 为 GEMM 建立 Pipeline" (TVM TIRx GEMM chapter), step 4
 * full kernel: A is (M,K), B is (N,K), D is (M,N), fp16 in and out with the
 * accumulator in FP32; the same layout is the Croqtile tutorial's ch. 7
 * pipelined matmul (lhs [M,K], rhs [N,K]) and the SM120 walk-through
 * "TensorCore_GEMM_with_TMA" §2.2 entrance, whose epilogue rounds with `_rn`.
 *
 *   A  device pointer, [M,K] fp16, row-major (leading dimension K), 16-byte aligned
 *   B  device pointer, [N,K] fp16, row-major (leading dimension K), 16-byte aligned
 *   D  device pointer, [M,N] fp16, row-major (leading dimension N), 2-byte aligned;
 *      only the M·N elements are written
 *   M, N, K  sizes; 0 <= M, N <= 2^31 - 512; 0 <= K <= 4,194,296 and K % 8 == 0
 *   stream   hipStream_t or NULL
 *
 * M == 0 or N == 0: returns GEMVTILE_OK and touches nothing (pointers may be NULL).
 * K == 0: D is filled with +0 (the empty sum); A and B may be NULL.
 * M, N need not be multiples of any tile size: edge tiles read zeros beyond
 * the matrix and write only inside it.  The summation order within FP32 is
 * unspecified (several results are correct up to rounding).
 * Otherwise the tiled kernel runs with 256x256 output tiles, or with
 * 256x128, 128x256, 128x128 or 128x64 ones when the output has too few 256x256
 * tiles to keep every compute unit busy (gemvtile_gemm_tile gives the choice);
 * it writes D with non-temporal stores, so D is not left in the caches.
 * When the smaller side has at most 64 rows -- a decode batch against a
 * weight matrix --, the call runs a bandwidth-bound kernel that streams the
 * larger operand once instead of the tiled one (32, 48 or 64 rows of it per
 * workgroup when it gives every compute unit 32, else 16, 8, 4, 2 or 1;
 * with 17..64 rows on the smaller side and few on the larger, the smaller
 * side is split into 16-row blocks over the workgroups instead), and when
 * M == 1 or N == 1 the GEMV kernel of gemv_f16; results are deterministic
 * either way.
 * Returns a gemvtile_status.
 */
int gemm_f16(const void *A, const void *B, void *D, int64_t M, int64_t N, int64_t K, void *stream);

/*
 * gemv_f16 -- y = x · Wᵀ (the batch-1 decode product), FP32 accumulation,
 * one fp16 rounding (nearest, ties to even) per output.
 *
 *   y[n] = fp16_rne( sum_{k<K} x[k] * W[n,k] )   for n < N
 *
 * Defined by "Learning TileLang with GEMV", §01 GEMV: the matrix is (N,K)
 * row-major as nn.Linear stores its weight, all kernels accumulate in FP32.
 *
 *   x  device pointer, [K] fp16, 16-byte aligned
 *   W  device pointer, [N,K] fp16, row-major (leading dimension K), 16-byte aligned
 *   y  device pointer, [N] fp16, 2-byte aligned
 *   N, K  sizes; 0 <= N <= 2^31 - 1; 0 <= K <= 2^31 - 8 and K % 8 == 0
 *   stream hipStream_t or NULL
 *
 * N == 0: returns GEMVTILE_OK and touches nothing.  K == 0: y is filled with +0.
 * When N is too small to give every compute unit a workgroup of 16 rows, or
 * when K >= 8192, the waves of a workgroup also split K (§5.2
 * block_split_k's reason: enough blocks in flight); the slices' FP32 partial
 * sums are added in LDS in a fixed order (gemvtile_gemv_grid gives the
 * workgroup count).  The row sums
 * are deterministic: no atomics, no split across workgroups, no workspace.
 * Returns a gemvtile_status.
 */
int gemv_f16(const void *x, const void *W, void *y, int64_t N, int64_t K, void *stream);

/*
 * gemm_bf16 / gemv_bf16 -- gemm_f16 and gemv_f16 with bf16 operands and
 * results: the same contract (layouts, sizes and their limits, alignment,
 * degenerate shapes, streams, errors, determinism), FP32 accumulation, and
 * one rounding of each output to bf16, round-to-nearest, ties to even.
 *
 *   D[m,n] = bf16_rne( sum_k A[m,k] * B[n,k] )     y[n] = bf16_rne( sum_k x[k] * W[n,k] )
 *
 * bf16 in and out with FP32 accumulators is the element type of the SM120
 * walk-through "TensorCore_GEMM_with_TMA" (§2.2 entrance: nv_bfloat16 A, B,
 * C; §2.3 kernel: FP32 accumulators rounded with __float22bfloat162_rn).
 * Shapes route as for fp16 (M or N == 1: the GEMV kernel; M or N <= 16, or
 * 17..64 rows on the smaller side as gemm_f16 describes: the skinny kernel;
 * otherwise the tiled
 * kernel), each in its default launch shape.
 */
int gemm_bf16(const void *A, const void *B, void *D, int64_t M, int64_t N, int64_t K, void *stream);
int gemv_bf16(const void *x, const void *W, void *y, int64_t N, int64_t K, void *stream);

/* Activation codes of the fused epilogue. */
enum gemvtile_act {
    GEMVTILE_ACT_NONE = 0, /* identity */
    GEMVTILE_ACT_RELU = 1  /* v < 0 -> +0, else v (a NaN stays NaN) */
};

/*
 * gemm_bias_f16 / gemm_bias_bf16 -- the GEMM with a fused epilogue: a bias
 * added to every row and an activation, before the one rounding.
 *
 *   D[m,n] = rne( act( sum_{k<K} A[m,k] * B[n,k] + bias[n] ) )
 *
 * The pages' kernels end their epilogue at the rounded store and define no
 * bias or activation; this is the plain definition of the usual fused
 * epilogue, in the same element format as gemm_f16 (fp16) or gemm_bf16
 * (bf16).  The sum is accumulated in FP32, bias[n] is added in FP32, the
 * activation is applied, and the result is rounded once (nearest, ties to
 * even).
 *
 *   A, B, D, M, N, K, stream  as for gemm_f16 / gemm_bf16 (same layouts,
 *            limits, alignment and degenerate shapes)
 *   bias   device pointer to N elements of the operand format, 2-byte
 *          aligned, or NULL for no bias
 *   act    GEMVTILE_ACT_NONE or GEMVTILE_ACT_RELU
 *
 * K == 0: D[m,n] = act(bias[n]) (+0 with no bias).  Every shape runs the
 * tiled kernel with the tile gemvtile_gemm_tile gives (the skinny and GEMV
 * kernels have no fused epilogue), so outputs with 16 rows or fewer on a
 * side are slower here than through gemm_f16.  An unknown act returns
 * GEMVTILE_ERR_INVALID_ARG, a misaligned bias GEMVTILE_ERR_UNSUPPORTED, both
 * before any HIP call.  Returns a gemvtile_status.
 */
int gemm_bias_f16(const void *A, const void *B, const void *bias, void *D, int64_t M, int64_t N, int64_t K, int act,
                  void *stream);
int gemm_bias_bf16(const void *A, const void *B, const void *bias, void *D, int64_t M, int64_t N, int64_t K, int act,
                   void *stream);

/*
 * gemm_splitk_f16 / gemm_splitk_bf16 -- gemm_f16 / gemm_bf16 with K split
 * across workgroups, for outputs too small to keep every compute unit busy
 * even with 128x128 tiles (a 1024x1024 output has 64 of them), and for
 * decode-batch shapes with 2..16 rows on one side whose other side has too
 * few blocks of 16 rows (8 x 1024 has 64).  Same contract and result
 * definition as gemm_f16 / gemm_bf16.
 *
 * The pages split K over blocks for the GEMV ("Learning TileLang with GEMV",
 * §5.2 block_split_k) and add the partial sums with FP32 atomics into a
 * zeroed output.  Here each (tile, K slice) workgroup unit stores its FP32
 * partial sums to `workspace`, [splits][M][N] floats, and a second kernel
 * adds the slices in slice order and rounds once: no atomics, no zeroing,
 * and every output is deterministic (the summation order depends only on
 * the shape and the device's compute-unit count).
 *
 *   workspace        device memory, 16-byte aligned, owned by the caller; its
 *                    contents on entry do not matter and are overwritten
 *   workspace_bytes  its size; at least gemvtile_gemm_splitk_workspace(M, N,
 *                    K, #CUs) for the current device
 *
 * Shapes that do not split (their tiles or row blocks already fill the CUs,
 * K too short for the split to pay, or one row on a side) run exactly as
 * gemm_f16 / gemm_bf16 and do not touch the workspace, which may then be
 * NULL.  A workspace that is too small
 * or NULL when needed returns GEMVTILE_ERR_INVALID_ARG, a misaligned one
 * GEMVTILE_ERR_UNSUPPORTED; these checks follow the (cached) compute-unit
 * query and precede any launch.  Calls that share a workspace must be
 * ordered on one stream.  Returns a gemvtile_status.
 */
int gemm_splitk_f16(const void *A, const void *B, void *D, int64_t M, int64_t N, int64_t K, void *workspace,
                    int64_t workspace_bytes, void *stream);
int gemm_splitk_bf16(const void *A, const void *B, void *D, int64_t M, int64_t N, int64_t K, void *workspace,
                     int64_t workspace_bytes, void *stream);

/*
 * gemm_splitk_f16_noalloc -- gemm_splitk_f16 for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation): no workspace argument, and no
 * allocation of any kind on the call path.  Same result, rounding and
 * determinism as gemm_splitk_f16 (the same kernels, in the same order).
 *
 * The FP32 partial sums go to a static device array of 16 MiB
 * (splits * M * N * 4 bytes are needed, see gemvtile_gemm_splitk_workspace)
 * that the library holds on each device it runs on until the process ends.
 * Shapes split only while their tiles (128x128 whenever they split) leave
 * compute units idle, and tiles * splits <= #CUs, so on parts with up to
 * 256 compute units every shape fits; a shape that needs more (on a larger
 * part) returns GEMVTILE_ERR_SCRATCH before any launch (use
 * gemm_splitk_f16 with a workspace then).  Shapes that do not split run
 * exactly as gemm_f16 and need none.  Every partial sum the reduction reads
 * is written by the same call, so the array needs no clearing; it keeps the
 * last call's contents.  All calls on one device share its one array:
 * calls that overlap on one GPU (on different streams, or from different
 * host threads without ordering) race and give undefined results; order
 * them on one stream.  Returns a gemvtile_status.
 */
int gemm_splitk_f16_noalloc(const void *A, const void *B, void *D, int64_t M, int64_t N, int64_t K, void *stream);

/*
 * gemvtile_gemm_splitk_splits / gemvtile_gemm_splitk_workspace -- the number
 * of K slices gemm_splitk_* uses for an M x N x K product on `num_cus`
 * compute units, and the workspace bytes it needs (splits * M * N * 4, or 0
 * when it does not split).  With T tiles of the tile gemvtile_gemm_tile
 * picks and KT = ceil(K / 64) K tiles: no split when T >= num_cus or
 * KT < 20; otherwise
 * splits = min(floor(num_cus / T), floor(KT / 10)), each slice ceil(KT /
 * splits) K tiles, minus slices left empty; 1 (0 bytes) below 2, and 1 unless
 * the K loop gets shorter by KT (splits - 1) / splits >= 12 + splits M N /
 * 2^18 K tiles (evaluated in double precision): a fixed cost, and one for
 * the partial sums' traffic.  With 2..16 rows on one side (the skinny
 * kernel), with B = ceil(R / 16) blocks of the other side's R rows and KT =
 * ceil(K / 512): no split when B >= num_cus, KT < 4 or KT num_cus < 8
 * num_cus + 64 B; otherwise splits = min(floor(num_cus / B), floor(KT / 2)),
 * each slice ceil(KT / splits) K tiles, minus slices left empty.  One row
 * on a side (the GEMV) never splits.  Host-only arithmetic; 1 and 0 for
 * sizes <= 0 or num_cus out of (0, 2^20].
 */
int gemvtile_gemm_splitk_splits(int64_t M, int64_t N, int64_t K, int64_t num_cus);
int64_t gemvtile_gemm_splitk_workspace(int64_t M, int64_t N, int64_t K, int64_t num_cus);

/* A static, human-readable name for a status code (never NULL). */
const char *gemvtile_status_string(int status);

/*
 * gemvtile_tile_coord -- the grouped tile order the persistent GEMM walks
 * (host-callable, no GPU needed).  Tile index t in [0, tiles_m*tiles_n) maps
 * to the output tile (*tm, *tn); consecutive t run down `group_m` tile rows of
 * one tile column, then move to the next column; the last group may be
 * shorter.  This is the threadblock swizzle of "TensorCore_GEMM_with_TMA"
 * §2.3 kernel (GROUP_M = 8), which the TVM chapter's step 6 persistent
 * scheduler (l2_group_size = 8) also uses for L2 locality.
 * Returns GEMVTILE_ERR_INVALID_ARG for t out of range, non-positive sizes or
 * NULL outputs.
 */
int gemvtile_tile_coord(int64_t t, int64_t tiles_m, int64_t tiles_n, int64_t group_m, int64_t *tm, int64_t *tn);

/*
 * gemvtile_gemm_config -- the compile-time shape of the 256x256 tiled GEMM
 * kernel that gemm_f16 launches on large outputs: output tile BM x BN, K
 * tile BK, LDS ring depth, threads per workgroup and the grouped-order
 * height.  Any output pointer may be NULL.
 */
void gemvtile_gemm_config(int *bm, int *bn, int *bk, int *stages, int *threads, int *group_m);

/*
 * gemvtile_gemm_tile -- the output tile (bm x bn) and LDS ring depth the
 * tiled GEMM takes for an M x N output on `num_cus` compute units (gemm_f16
 * and gemm_bf16 when they take the tiled kernel).  Of 256x256 (2
 * stages), 256x128 and 128x256 (3 stages), 128x128 and 128x64 (4 stages),
 * it is the one with the least ceil(#tiles / num_cus) * bm * bn / rate,
 * where rate is the tile's measured work rate relative to 256x256 with
 * tiles to spare (1, 0.9, 0.9, 0.76, 0.55); ties go to the larger tile.
 * The split-K entry points choose the same way among the first four.  Smaller tiles fill the CUs
 * when large ones would leave some idle (an 8192 x 1024 output has 128 tiles
 * of 256x256, 256 of 256x128); their deeper rings cover the load latency
 * over their shorter K tiles.  Any output pointer may be NULL.  Host-only
 * arithmetic; returns GEMVTILE_ERR_INVALID_ARG for M, N or num_cus <= 0 or
 * num_cus > 2^20.
 */
int gemvtile_gemm_tile(int64_t M, int64_t N, int64_t num_cus, int *bm, int *bn, int *stages);

/*
 * gemvtile_device_caps -- the current device's compute-unit count, peak
 * engine clock (kHz), peak memory clock (kHz) and memory bus width (bits),
 * for recomputing the roofline peaks from the part itself.  Any output
 * pointer may be NULL.  Returns GEMVTILE_ERR_DEVICE if a HIP query fails.
 */
int gemvtile_device_caps(int *num_cus, int *clock_khz, int *mem_clock_khz, int *mem_bus_bits);

/*
 * gemvtile_gemv_grid -- the number of workgroups gemv_f16 (and gemv_bf16)
 * launches for an N x K matrix on a device with `num_cus` compute units:
 * ceil(N/R) with R = 2 rows per workgroup (K split 8 ways over the
 * workgroup's 8 waves) when K >= 8192 and N >= 2*num_cus; otherwise R = 16
 * rows per workgroup when N >= 16*num_cus, else 8, 4 or 2 rows (K split 2,
 * 4 or 8 ways) while N >= 8, 4 or 2 times num_cus; else 1 row (K split 8
 * ways).  Host-only arithmetic; returns 0 for N <= 0, K < 0 or num_cus
 * outside [1, 2^20].
 */
int64_t gemvtile_gemv_grid(int64_t N, int64_t K, int64_t num_cus);

/*
 * gemvtile_gemm_grid -- the number of workgroups gemm_f16 launches for an
 * M x N x K product on a device with `num_cus` compute units: the GEMV grid
 * of the other side's rows when M or N is 1; when the smaller side has at
 * most 64 rows (the skinny kernel), ceil(R/p) with R = N if M <= 16, else M
 * if N <= 16, else the larger side, and p rows per workgroup: when
 * R >= 32*num_cus, the one of 32, 48, 64 with the least
 * ceil(ceil(R/p)/num_cus)*p (ties to the larger), else the largest of 16,
 * 8, 4, 2 such that R >= p*num_cus, else 1; except that,
 * when the smaller side S has 17..64 rows and that p is below 8 (or 8 with
 * S <= 32), ceil(S/16)*ceil(R/q) with q the largest of 16, 8, 4, 2 such
 * that ceil(S/16)*ceil(R/q) >= num_cus, else q = 1 (the smaller side split
 * into 16-row blocks); otherwise the persistent grid min(#tiles, num_cus)
 * over the tiles gemvtile_gemm_tile picks.  Host-only arithmetic; returns 0
 * for empty outputs.
 */
int64_t gemvtile_gemm_grid(int64_t M, int64_t N, int64_t K, int64_t num_cus);

/*
 * gemvtile_gemm_f16_variant -- gemm_f16 with an internal kernel variant, for
 * ablation measurements only (same contract and results as gemm_f16).
 *   0  what gemm_f16 runs: on tiled shapes the tile of gemvtile_gemm_tile;
 *      with 256x256 tiles, 4 waves of 128x128, 16x16x32 MFMA blocks, K tiles
 *      of 64 in a 2-stage LDS ring, the next K step's operand reads one every
 *      2 MFMA slots, a refill load every 4 slots, swizzled LDS, persistent
 *      grouped XCD-aware schedule, and the early-free K loop (a second
 *      barrier per K tile, at MFMA slot 48 of K step 0, after which the
 *      wave's stage is refilled, half a K tile sooner than with one barrier);
 *      each K step's MFMAs in serpentine order over the wave's 16x16 blocks
 *   1  as 20 without the LDS swizzle
 *   2  as 10 with single-stage LDS (load, wait, compute: no overlap)
 *   3  as 20 with one workgroup per tile (no persistent loop, no XCD remap)
 *   10 as 30 with 32x32x16 MFMA blocks, one operand read per slot, a refill
 *      load every 2 of its 64 slots per K tile
 *   20 the 256x256 tiled kernel of variant 0, whatever the shape
 *   21, 22, 23 the same schedule on 256x128, 128x256 (3-stage rings) and
 *      128x128 (4-stage ring) output tiles (4 waves of 128x64, 64x128,
 *      64x64): the smaller tiles of variant 0, whatever the shape
 *   24, 25, 26 as 21, 22, 23 with 2-stage rings   27 as 23 with 5 stages
 *   32 the 128x64 tile of variant 0 (4-stage ring, 4 waves of 32x64),
 *      whatever the shape
 *   28 as 20 with D written by ordinary (cached) stores instead of
 *      non-temporal ones
 *   30 as 20 with one barrier per K tile (the ring without the early free)
 *   31 as 20 with the MFMAs of a K step in row-major order over the blocks
 * Variants 1..32 always run the tiled kernel, whatever the shape; variant
 * 0 routes shapes as gemm_f16 does (M or N == 1: the GEMV kernel; M or N
 * <= 16, and some shapes with 17..64 rows on the smaller side: the skinny
 * kernel).  The skinny kernel (only for M <= 16 or N <= 16, and 160 also
 * for 17..64 rows on the smaller side, else GEMVTILE_ERR_UNSUPPORTED):
 *   100 the gemm_f16 choice (32, 48, 64, 16, 8, 4, 2 or 1 rows of the
 *       large side per workgroup, see gemvtile_gemm_grid)
 *   104 operands loaded straight into registers (8 waves, 4 K steps of 32
 *       in flight per wave), 16 large-side rows per workgroup
 *   112 operands staged through a 4-stage LDS ring of 1 KiB row segments,
 *       16 waves, 16 large-side rows per workgroup
 *   130 as 112 with workgroup b starting its K walk at K tile b (mod the
 *       number of K tiles)
 *   147 as 130 with the large side loaded non-temporally
 *   152 as 147 with every workgroup starting its K walk at K tile 0
 *   160 the small side split into blocks of 16 rows along the grid's y
 *       dimension, each workgroup staging one block against 16, 8, 4, 2 or
 *       1 rows of the large side (the most that still give every compute
 *       unit a workgroup); also for 17..64 rows on the smaller side
 * (gemm_f16's choice at 16 rows per workgroup starts workgroup b at K tile
 * b / 8, its index within its XCD, and loads the large side non-temporally
 * from K = 8192 up.)
 * The wave-specialised kernel, whatever the shape:
 *   200, 201 256x128 output tiles, 4 consumer waves (MFMA only, 128x64
 *       each) and 4 loader waves (tile loads only) handing K tiles over at
 *       one barrier per K tile, with a 3-stage (200) or 2-stage (201) ring
 * Other numbers (ablations measured and not kept) return
 * GEMVTILE_ERR_INVALID_ARG.
 */
int gemvtile_gemm_f16_variant(const void *A, const void *B, void *D, int64_t M, int64_t N, int64_t K,
                              void *stream, int variant);

/*
 * gemvtile_gemm_f16_timed -- measurement only: the 256x256 tiled kernel of
 * gemm_f16 (variant 20) on an M x N x K product (M, N > 16, K > 0; same
 * result as gemm_f16), with one record of 8 uint64 per workgroup written to
 * `stamps` (host-visible or device memory of `stamps_len` uint64, at least
 * 8 * min(#256x256 tiles, #CUs), 8-byte aligned) by its first thread:
 *   [0], [1]  the constant 100 MHz real-time counter and the shader-cycle
 *             counter when the workgroup started
 *   [2], [3]  the same when the K loop of its first output tile ended
 *   [4], [5]  the same when it finished, after every store of every wave
 *             completed
 *   [6], [7]  the HW_ID and XCC_ID hardware registers (XCD in bits 0..3 of
 *             the latter)
 * Cycle deltas over real-time deltas give the clock each workgroup ran at.
 * Returns GEMVTILE_ERR_UNSUPPORTED for shapes gemm_f16 would not run on the
 * tiled kernel, GEMVTILE_ERR_INVALID_ARG for too small a buffer.
 */
int gemvtile_gemm_f16_timed(const void *A, const void *B, void *D, int64_t M, int64_t N, int64_t K, void *stream,
                            uint64_t *stamps, int64_t stamps_len);

/*
 * gemvtile_gemv_f16_variant -- gemv_f16 with an internal launch shape, for
 * measurements only (same contract and results as gemv_f16):
 *   0  the gemv_f16 default (picks one of 8..12 from N, K and the
 *      compute-unit count, see gemvtile_gemv_grid, or its cached twin
 *      37..41 when W holds fewer than 2^25 elements)
 *   6  2 rows per wave, 8 waves, 4 chunk steps in flight, ordinary (cached)
 *      loads of W, each wave starting its walk along K at a different group
 *   7  as 6 with non-temporal loads of W and every wave starting at the
 *      row's first column
 *   8..11  2 rows per wave, 8 waves, 4 steps, non-temporal W, rotated start,
 *      K split over 1, 2, 4, 8 waves per row group (16, 8, 4, 2 rows per
 *      workgroup)
 *   12 1 row per workgroup, K split 8 ways
 *   20 as 8 with grid-strided rows: local row r (0..15) of workgroup b is
 *      row r*G + b (G = the grid size), so workgroups running side by side
 *      read adjacent rows, instead of 16 consecutive rows per workgroup
 *   21 as 8 with x staged in LDS once per workgroup (K <= 16384, else
 *      GEMVTILE_ERR_INVALID_ARG) instead of loaded by every wave
 *   28 as 7 with 8 chunk steps in flight
 *   29 as 7 with 4 rows per wave and 4 waves
 *   37..41 as 8..12 with cached (not non-temporal) loads of W
 * Other numbers return GEMVTILE_ERR_INVALID_ARG.
 */
int gemvtile_gemv_f16_variant(const void *x, const void *W, void *y, int64_t N, int64_t K, void *stream,
                              int variant);

/*
 * gemvtile_ring_trace -- the K-loop schedule of the tiled GEMM kernel, for
 * checking on the CPU (host-only; no GPU needed).  The kernel's K loop is a
 * walker over K tiles that issues tile loads, operand reads, MFMAs, waits
 * and barriers; this runs the same walker on the host for the kernel of
 * tiled variant `variant` (a gemvtile_gemm_f16_variant number: 0 = 20, the
 * 256x256 default; 1 and 3 share its ring; 10, 20..27, 30 and 31) over `ktu`
 * K tiles (of 64 elements), recording each event instead of issuing it.
 * The ring follows "使用 TMA 为 GEMM 建立 Pipeline" (TVM TIRx GEMM chapter),
 * step 5 (Pipeline 机制): K tile k in stage k % stages, refilled with tile
 * k + stages once consumed; completion is tracked by in-order vmcnt waits
 * instead of the chapter's per-stage mbarrier phases.
 *
 *   ktu     K tiles the loop walks (1 .. 2^20): ceil(K / 64), or one K slice
 *           of a split-K unit
 *   events  host memory for `cap` events of five int32 {code, a, b, c, d}:
 *             1 load      a = K tile, b = load index, c = ring stage
 *             2 wait      a = vmcnt (vector-memory operations allowed to
 *                         stay in flight)
 *             3 LDS wait  (the wave's LDS reads are complete)
 *             4 barrier   (workgroup barrier)
 *             5 read      a = K tile, b = K step, c = read index, d = stage;
 *                         with nA x nB MFMA blocks per wave, read index 0
 *                         fetches A block 0, 1..nB the B blocks 0..nB-1,
 *                         and nB+1.. the A blocks 1..nA-1
 *             6 MFMA      a = fragment buffer, b = MFMA index in the K step,
 *                         c = its block row (A block), d = its block
 *                         column (B block)
 *             7 prep      a = K tile, b = part: part b of working out the
 *                         addresses of that K tile's refill loads (the
 *                         early-free schedule), ahead of those loads
 *             8 init      the accumulators are zeroed (once, after the
 *                         prologue's loads are issued)
 *           events beyond `cap` are counted but not written; may be NULL
 *           when cap == 0
 *   info    if not NULL, 10 ints: loads per wave per K tile, operand reads
 *           per wave per K step, K steps per K tile, MFMAs per wave per K
 *           step, ring stages, output tile rows and columns, 1 for the
 *           early-free schedule (two barriers per K tile) or 0, and the
 *           waves along the tile's rows and along its columns
 * Each wave of the workgroup runs this same sequence.  Returns the number
 * of events, or -1 for a variant without a multi-stage ring or arguments
 * out of range.
 */
int64_t gemvtile_ring_trace(int variant, int64_t ktu, int32_t *events, int64_t cap, int *info);

/*
 * Block-scaled 8-bit operands.  "e4m3" is the 8-bit format with 4 exponent
 * bits (bias 7) and 3 fraction bits, whose largest number is 448, whose 0x7f
 * and 0xff are NaN and which has no infinities (torch.float8_e4m3fn).  An
 * operand [R,K] of them comes with FP32 scales [ceil(R/r), ceil(K/128)], one
 * for each block of r rows and 128 columns: element (i,k) stands for
 * value[i,k] * scale[i/r, k/128].  r is 1 for activations and gradients and
 * 128 for weights.
 *
 * quantize_fp8_rows_f16, _bf16 -- x [M,K] to q [M,K] e4m3 and scale
 * [M, ceil(K/128)], r = 1.
 * quantize_fp8_tiles_f16, _bf16 -- each of the E matrices of x [E,N,K] to q
 * [E,N,K] and scale [E, ceil(N/128), ceil(K/128)], r = 128 (E = 1 for one
 * weight matrix, or the experts of a layer).
 *
 *   scale = max(fp32(amax / 448), 2^-80),  amax the block's largest |x|
 *   q     = the e4m3 number nearest to x / scale (the real quotient), ties to even
 *
 * A block of zeros has scale 2^-80 and q = 0.  A block with an infinity has an
 * infinite scale (q = 0 for its finite numbers, NaN for the infinite) and one
 * with a NaN a NaN scale (q = NaN), so whatever is multiplied with it comes out
 * NaN.
 *
 *   x, q      device pointers, row-major, 16-byte aligned
 *   scale     device pointer, FP32, 4-byte aligned
 *   sizes     >= 0; K % 16 == 0; M * ceil(K/128) <= 2^29 - 32 row blocks, E *
 *             ceil(N/128) * ceil(K/128) < 2^23 tiles, each of M, N, K < 2^31
 * A size of 0 returns GEMVTILE_OK and touches nothing.
 */
int quantize_fp8_rows_f16(const void *x, void *q, float *scale, int64_t M, int64_t K, void *stream);
int quantize_fp8_rows_bf16(const void *x, void *q, float *scale, int64_t M, int64_t K, void *stream);
int quantize_fp8_tiles_f16(const void *x, void *q, float *scale, int64_t E, int64_t N, int64_t K, void *stream);
int quantize_fp8_tiles_bf16(const void *x, void *q, float *scale, int64_t E, int64_t N, int64_t K, void *stream);

/*
 * gemm_fp8_f16, gemm_fp8_bf16 -- D = A · Bᵀ of block-scaled e4m3 operands,
 * rounded once to fp16 / bf16 (nearest, ties to even):
 *
 *   D[m,n] = sum_b scale_A[m,b] * scale_B[n/r,b] * sum_{k in block b} A[m,k] * B[n,k]
 *
 *   A        device pointer, [M,K] e4m3, row-major, 16-byte aligned
 *   scale_A  device pointer, [M, ceil(K/128)] FP32, 4-byte aligned
 *   B        device pointer, [N,K] e4m3, row-major, 16-byte aligned
 *   scale_B  device pointer, [ceil(N/r), ceil(K/128)] FP32, 4-byte aligned
 *   scale_B_rows  r: 128 (a weight quantised in tiles) or 1 (an operand
 *            quantised by rows, as both are in the gradient of a weight:
 *            dB = dDᵀ · A takes A = dDᵀ [N,M], B = Aᵀ [K,M]); other values
 *            return GEMVTILE_ERR_INVALID_ARG
 *   D        device pointer, [M,N] fp16 / bf16, row-major, 2-byte aligned
 *   M, N, K  sizes; 0 <= M, N <= 2^25; 0 <= K <= 4,194,288 and K % 16 == 0
 *
 * The products within a block of 128 are exact.  With up to 4 rows of A they
 * are added in FP32; larger products use the 8-bit matrix instructions, which
 * add them in a window aligned to the largest (within 2^-11 of it).  (Grouped:
 * in FP32 where gemvtile_grouped_plan returns 1.)  Blocks are scaled and added in
 * FP32.  scale_A * scale_B is formed in FP32 first: it has to be finite there
 * for the result to be, and 2^-126 or more for full accuracy (below that it
 * loses bits, and below 2^-149 it is 0, even where a block's sum of up to 2.5e7
 * would bring the result into range; scales of the quantisers are 2^-80 or
 * more).  M == 0 or N == 0 touches nothing; K == 0
 * fills D with +0.  Results are deterministic.
 */
int gemm_fp8_f16(const void *A, const float *scale_A, const void *B, const float *scale_B, void *D, int64_t M, int64_t N,
                 int64_t K, int64_t scale_B_rows, void *stream);
int gemm_fp8_bf16(const void *A, const float *scale_A, const void *B, const float *scale_B, void *D, int64_t M,
                  int64_t N, int64_t K, int64_t scale_B_rows, void *stream);

/*
 * Products grouped by expert.  X (or dY) holds T rows sorted by group;
 * group e of E owns rows offsets[e] .. offsets[e+1] - 1, any number of them,
 * none included.  offsets [E+1] is int32 in device memory and is read by the
 * kernels only, so a router's result can be used without a synchronisation:
 * offsets[0] >= 0, non-decreasing, offsets[E] <= T.  Rows before offsets[0]
 * and from offsets[E] on belong to no group: nothing of them is read, and
 * their rows of the output stay as they were.  Offsets that break these rules
 * give wrong results but no access outside the buffers.
 *
 * gemm_grouped_f16, _bf16        D[t,n]  = sum_k X[t,k] * W[e,n,k]    t in group e
 * gemm_grouped_dgrad_f16, _bf16  dX[t,k] = sum_n dY[t,n] * W[e,n,k]   t in group e
 * gemm_grouped_wgrad_f16, _bf16  dW[e,n,k] = sum_{t in group e} dY[t,n] * X[t,k]
 *                                (zeros for a group without rows)
 * gemm_grouped_fp8_f16, _bf16    gemm_grouped on e4m3 X with scale_X
 *                                [T, ceil(K/128)] (r = 1) and W with scale_W
 *                                [E, ceil(N/128), ceil(K/128)] (r = 128)
 *
 * FP32 accumulation and one rounding (nearest, ties to even) of each output;
 * results are deterministic.  X and D [T,K] and [T,N], dY and dX [T,N] and
 * [T,K], W and dW [E,N,K], all row-major; inputs, dX and dW 16-byte aligned,
 * D 2-byte, offsets and scales 4-byte aligned.
 *   T, N, K, E  sizes >= 0; T <= 2^31 - 512, N, K <= 2^20, E <= 1024;
 *               K % 8 == 0 (16 for 8-bit operands), for the two gradients
 *               N % 8 == 0 as well; dW of fewer than 2^24 blocks of 128 x 128;
 *               otherwise GEMVTILE_ERR_UNSUPPORTED
 * E == 0, T == 0 (but for dW, which is then zeros) or an output without
 * elements touches nothing.  A sum over no elements (K == 0, or N == 0 for
 * dX) is +0.
 */
int gemm_grouped_f16(const void *X, const void *W, const int32_t *offsets, void *D, int64_t T, int64_t N, int64_t K,
                     int64_t E, void *stream);
int gemm_grouped_bf16(const void *X, const void *W, const int32_t *offsets, void *D, int64_t T, int64_t N, int64_t K,
                      int64_t E, void *stream);
int gemm_grouped_dgrad_f16(const void *dY, const void *W, const int32_t *offsets, void *dX, int64_t T, int64_t N,
                           int64_t K, int64_t E, void *stream);
int gemm_grouped_dgrad_bf16(const void *dY, const void *W, const int32_t *offsets, void *dX, int64_t T, int64_t N,
                            int64_t K, int64_t E, void *stream);
int gemm_grouped_wgrad_f16(const void *dY, const void *X, const int32_t *offsets, void *dW, int64_t T, int64_t N,
                           int64_t K, int64_t E, void *stream);
int gemm_grouped_wgrad_bf16(const void *dY, const void *X, const int32_t *offsets, void *dW, int64_t T, int64_t N,
                            int64_t K, int64_t E, void *stream);
int gemm_grouped_fp8_f16(const void *X, const float *scale_X, const void *W, const float *scale_W,
                         const int32_t *offsets, void *D, int64_t T, int64_t N, int64_t K, int64_t E, void *stream);
int gemm_grouped_fp8_bf16(const void *X, const float *scale_X, const void *W, const float *scale_W,
                          const int32_t *offsets, void *D, int64_t T, int64_t N, int64_t K, int64_t E, void *stream);

/*
 * gemvtile_grouped_plan -- how gemm_grouped_* (op 0), _dgrad_ (1), _wgrad_ (2)
 * and _fp8_ (3) run on `num_cus` compute units: *rows is the number of a
 * group's rows that one workgroup takes at a time, *cols the columns of the
 * output, and the return value 2 for the kernel of small tiles (no more of them
 * than compute units are expected), 1 for the one that streams W once (few rows
 * for each group; *cols is then one block of columns, of which a workgroup takes
 * as many as gemvtile_grouped_stream_blocks says), 0 for the tiled one (a last
 * round of 256x256 16-bit tiles that would keep at most half of the compute
 * units busy is cut into 128x128 ones).  Host-only; returns -1 for arguments out
 * of range.
 */
int gemvtile_grouped_plan(int op, int64_t T, int64_t N, int64_t K, int64_t E, int64_t num_cus, int *rows, int *cols);

/*
 * gemvtile_grouped_stream_blocks -- for a grouped product that is streamed, the
 * blocks of 16 columns of the output that a workgroup takes: 1, or 2 where there
 * are then two workgroups for each compute unit.  Arguments as for
 * gemvtile_grouped_plan.  Host-only; returns -1 for a product that is not
 * streamed and for arguments out of range.
 */
int gemvtile_grouped_stream_blocks(int op, int64_t T, int64_t N, int64_t K, int64_t E, int64_t num_cus);

/*
 * gemvtile_grouped_ring_trace -- the K loop of the tiled 16-bit grouped kernels
 * for a `rows` x `cols` output tile (256x256, 256x128 or 128x128), as
 * gemvtile_ring_trace records that of the tiled GEMM: K tiles first .. ktu - 1
 * (of 64 elements of the sum; ktu <= 2^25 - 8, at most 4096 of them) as the loop
 * walks them, after the loads of the first info[2] of them have been issued.
 * Its loop has no drain: the loads past the last K tile fetch nothing.
 * `events` as there; info, 3 ints: loads per wave and K tile, ring stages, K
 * tiles loaded ahead.  Host-only; returns the number of events, or -1 for
 * arguments out of range.
 */
int64_t gemvtile_grouped_ring_trace(int rows, int cols, int64_t first, int64_t ktu, int32_t *events, int64_t cap,
                                    int *info);

/*
 * gemvtile_group_unit -- the rows that unit `unit` of a grouped product covers
 * when every group's rows are cut into units of `rows`, as the kernels work it
 * out from the offsets (here in host memory).  Writes the group, its unit's
 * first row and one past its last; returns the most units that a launch allows
 * for, -1 for a unit past the last one, -2 for arguments out of range.
 */
int64_t gemvtile_group_unit(const int32_t *offsets, int64_t E, int64_t T, int64_t rows, int64_t unit, int64_t *group,
                            int64_t *first, int64_t *past);

/*
 * Operators around the products: weights in 4 bits, the norm before a product,
 * the router before the products by expert, and the rows' way there and back.
 * All of them are asynchronous, keep nothing between calls, allocate nothing,
 * use no atomics that decide an order (results are deterministic) and can be
 * captured.  Outputs overlap neither inputs nor one another, but for a norm's h.
 *
 * "e2m1" is the 4-bit format with 2 exponent bits (bias 1) and 1 fraction bit:
 * 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives.  An operand [N,K] of them is
 * held as bytes [N,K/2], column 2i in the low half of byte i, and scale bytes
 * [N,K/32]: byte s of 32 columns of a row stands for 2^(s - 127), 255 for NaN (the
 * OCP microscaling format MXFP4).
 *
 * quantize_fp4_f16, _bf16 -- x [N,K] to such numbers q and scales:
 *   s = the least with amax <= 6 * 2^(s - 127) (at least 0), amax the block's
 *       largest |x|: no number is beyond the format's largest
 *   q = the e2m1 number nearest to x / 2^(s - 127), ties to even; the sign of
 *       zero is kept
 * A block with an infinity or a NaN has s = 255 and q = 0.
 *   x, q      16-byte aligned; sizes >= 0, K % 32 == 0, N * K <= 2^36 - 4096
 * (E matrices of [N,K] are one of [E N, K].)
 *
 * gemv_fp4_f16, _bf16 -- a matrix-vector product with such weights for each of M
 * rows, rounded once (nearest, ties to even):
 *
 *   y[m,n] = sum_b 2^(scale_W[n,b] - 127) * sum_{k in block b} x[m,k] * W[n,k]
 *
 * Products are exact and added in FP32: scaled before they are added, or, where the
 * scaled numbers are none of the 16-bit format's (scales outside 2^-125 .. 2^125 in bf16,
 * 2^-23 .. 2^13 in fp16) and at a ragged end of K, a block's first and then scaled.  Four
 * blocks of K and up to 64 rows of W go one way together, so the last bits of an output
 * may depend on the scales of rows beside its own; the same call gives the same bits.
 * Where the magnitudes |x W|, scaled or not, add up to 2^128, y may be infinite or NaN.
 * Meant for decode batches: up to 48 rows share what a workgroup reads of W, fewer
 * where more workgroups make up for reading it again; more rows read it again.
 *   x        [M,K] fp16 / bf16, 16-byte aligned
 *   W        [N,K/2] bytes, 16-byte aligned;  scale_W  [N,K/32] bytes
 *   y        [M,N] fp16 / bf16, 2-byte aligned
 *   M, N, K  >= 0; M <= 2^19, N <= 2^25, K <= 4,194,272 and K % 32 == 0
 * M == 0 or N == 0 touches nothing; K == 0 fills y with +0.
 */
int quantize_fp4_f16(const void *x, void *q, void *scale, int64_t N, int64_t K, void *stream);
int quantize_fp4_bf16(const void *x, void *q, void *scale, int64_t N, int64_t K, void *stream);
int gemv_fp4_f16(const void *x, const void *W, const void *scale_W, void *y, int64_t M, int64_t N, int64_t K,
                 void *stream);
int gemv_fp4_bf16(const void *x, const void *W, const void *scale_W, void *y, int64_t M, int64_t N, int64_t K,
                  void *stream);

/*
 * rmsnorm_f16, _bf16, rmsnorm_fp8_f16, _bf16 -- root-mean-square norm of T rows of
 * C, with the residual's addition before it:
 *
 *   h = x + residual, rounded once     (residual and h both NULL: h is x)
 *   r = 1 / sqrt(sum_c h^2 / C + eps)
 *   y = h * r * weight
 *
 * rmsnorm_* rounds y to 16 bits.  rmsnorm_fp8_* gives q [T,C] e4m3 and scale
 * [T, ceil(C/128)] FP32 with one scale for each 128 columns of a row, as
 * quantize_fp8_rows_* does, of y before any rounding: scale = max(amax / 448,
 * 2^-80), q = e4m3(y / scale); y itself in 16 bits too if it is not NULL.  What a
 * block with an infinity or a NaN becomes is as there.
 *   x, residual, weight [C], h, y, q  16-byte aligned; h may be x or residual
 *            (the stream is then updated in place), other outputs overlap nothing
 *   scale, rstd                       4-byte aligned; rstd [T] takes r for the
 *            gradient, or NULL
 *   T, C     >= 0; T <= 2^31 - 512, C <= 32768, C % 8 == 0 (16 for rmsnorm_fp8_*)
 *   eps      >= 0, in FP64, as the sum of squares and r are; rstd is r rounded to FP32.
 *            y in 16 bits is rounded from an FP32 number, made of r and h * r in FP32;
 *            q is the number nearest to y / scale, whatever the sizes of h, weight and
 *            r (a row of zeros over an eps of 0 is NaN)
 * T == 0 or C == 0 touches nothing.
 *
 * rmsnorm_grad_f16, _bf16 -- the gradients, given dy, h, weight and rstd, and dh, the
 * gradient that reaches h elsewhere (along the residual; NULL: none):
 *
 *   dx[t,c]    = r weight dy - h r^3 (sum_c weight dy h) / C + dh     one rounding;
 *                the gradient of x and of residual alike
 *   dweight[c] = sum_t dy h r                                        FP32
 *
 * Products and sums are in FP32 (weight * dy, h * r and their product have to be in its
 * range); the rows' shares of dweight are added in an order that T and C alone decide.
 *   dy, dh, h, weight, dx  16-byte aligned; rstd, dweight 4-byte aligned; dx
 *            overlaps nothing
 *   workspace  gemvtile_rmsnorm_grad_workspace(T, C) bytes of device memory, owned
 *            by the caller, 16-byte aligned; its contents do not matter.  Too small
 *            or NULL: GEMVTILE_ERR_INVALID_ARG, also where few rows make no use of it.
 *            Calls that share one have to be ordered, captured ones included
 *   T, C     as above, C % 8 == 0.  T == 0 fills dweight with zeros.
 */
int rmsnorm_f16(const void *x, const void *residual, const void *weight, void *h, void *y, float *rstd, int64_t T,
                int64_t C, double eps, void *stream);
int rmsnorm_bf16(const void *x, const void *residual, const void *weight, void *h, void *y, float *rstd, int64_t T,
                 int64_t C, double eps, void *stream);
int rmsnorm_fp8_f16(const void *x, const void *residual, const void *weight, void *h, void *y, void *q, float *scale,
                    float *rstd, int64_t T, int64_t C, double eps, void *stream);
int rmsnorm_fp8_bf16(const void *x, const void *residual, const void *weight, void *h, void *y, void *q, float *scale,
                     float *rstd, int64_t T, int64_t C, double eps, void *stream);
int rmsnorm_grad_f16(const void *dy, const void *dh, const void *h, const void *weight, const float *rstd, void *dx,
                     float *dweight, int64_t T, int64_t C, void *workspace, int64_t workspace_bytes, void *stream);
int rmsnorm_grad_bf16(const void *dy, const void *dh, const void *h, const void *weight, const float *rstd, void *dx,
                      float *dweight, int64_t T, int64_t C, void *workspace, int64_t workspace_bytes, void *stream);
int64_t gemvtile_rmsnorm_grad_workspace(int64_t T, int64_t C);

/* Scores of a router. */
enum gemvtile_score {
    GEMVTILE_SCORE_SOFTMAX = 0, /* exp(logit) / sum over the token's experts */
    GEMVTILE_SCORE_SIGMOID = 1  /* 1 / (1 + exp(-logit)) */
};

/*
 * route_topk_f16, _bf16, _f32 -- the k experts of each of T tokens, and their weights.
 *
 *   choice[e]  = score[e] + bias[e], or, with bias NULL, logit[e]
 *   The E experts are `groups` groups of E / groups that follow one another.  A
 *   group counts by its best choice (group_best 1) or by the sum of its two best
 *   (2; with bias NULL the sum of its two best scores), and the top_groups best
 *   groups are kept, ties to the lowest.
 *   ids [T,k] int32  the k largest choices of the kept groups, largest first, ties
 *                    to the lowest expert
 *   weights [T,k]    FP32: scale * score[id] (no bias), divided by the sum of the k
 *                    scores if norm is 1; worked out in FP32 (the ids are not), so a
 *                    few units in the last place off, and in proportion to the logits
 *                    where those are large
 *
 * Ids are those of choices computed in 64 bits, whatever the logits' type.  A logit
 * of -inf is an expert with score 0, chosen after all others unless a bias lifts it (a
 * bias of -inf does not); where every score that is divided by is 0 (all logits -inf)
 * the weights are 0.  A NaN choice (of the logit or the bias) ranks below all others.
 * With softmax a NaN or +inf among a token's logits makes its weights NaN, and with a
 * bias every choice (ids are the lowest then), with sums of two and no bias those sums
 * (the lowest groups are kept, and in them the largest logits); with a sigmoid a NaN
 * logit makes the weights NaN where it is chosen.  Ids are always k different numbers of 0 .. E - 1.
 *
 *   logits   [T,E] fp16 / bf16 / FP32, 16-byte aligned
 *   bias     [E] FP32 or NULL; ids, weights 4-byte aligned
 *   T >= 0, T <= 2^26 - 64; 1 <= k <= 32, E <= 1024, groups <= 64 dividing E,
 *   1 <= top_groups <= groups, k <= top_groups * E / groups
 *
 * route_topk_grad_f16, _bf16, _f32 -- dlogits [T,E] (16-byte aligned, the logits'
 * type, written whole, one rounding) for dweights [T,k], with the ids held fixed as
 * the choice among them is not differentiated.  The ids of a token are different (of
 * one that is not, one of its places counts); one outside 0 .. E - 1 is left out.
 */
int route_topk_f16(const void *logits, const float *bias, int32_t *ids, float *weights, int64_t T, int64_t E, int64_t k,
                   int64_t groups, int64_t top_groups, int group_best, int score, int norm, float scale, void *stream);
int route_topk_bf16(const void *logits, const float *bias, int32_t *ids, float *weights, int64_t T, int64_t E, int64_t k,
                    int64_t groups, int64_t top_groups, int group_best, int score, int norm, float scale, void *stream);
int route_topk_f32(const void *logits, const float *bias, int32_t *ids, float *weights, int64_t T, int64_t E, int64_t k,
                   int64_t groups, int64_t top_groups, int group_best, int score, int norm, float scale, void *stream);
int route_topk_grad_f16(const void *logits, const int32_t *ids, const float *dweights, void *dlogits, int64_t T,
                        int64_t E, int64_t k, int score, int norm, float scale, void *stream);
int route_topk_grad_bf16(const void *logits, const int32_t *ids, const float *dweights, void *dlogits, int64_t T,
                         int64_t E, int64_t k, int score, int norm, float scale, void *stream);
int route_topk_grad_f32(const void *logits, const int32_t *ids, const float *dweights, void *dlogits, int64_t T,
                        int64_t E, int64_t k, int score, int norm, float scale, void *stream);

/*
 * route_sort -- the T * k slots (t, j) sorted by expert, those of an expert in their
 * order: offsets [E+1] int32 as gemm_grouped_* take them (expert e has rows
 * offsets[e] .. offsets[e+1] - 1), and pos [T,k] int32, the row of each slot.  A slot
 * whose id is outside 0 .. E - 1 has no row (pos -1; so a card that holds some of the
 * experts sorts the slots of those).
 *   ids, offsets, pos  4-byte aligned, not overlapping
 *   workspace  gemvtile_route_sort_workspace(T, k, E) bytes (0 for up to 2048 slots;
 *            it may then be NULL), 16-byte aligned, owned by the caller; as for
 *            rmsnorm_grad_*
 *   T >= 0, k >= 1, 1 <= E <= 1024, T * k <= 2^31 - 512.  T == 0: offsets are zeros.
 */
int route_sort(const int32_t *ids, int32_t *offsets, int32_t *pos, int64_t T, int64_t k, int64_t E, void *workspace,
               int64_t workspace_bytes, void *stream);
int64_t gemvtile_route_sort_workspace(int64_t T, int64_t k, int64_t E);

/*
 * The rows of T tokens and the R rows sorted by expert.  pos [T,k] is the row of each
 * slot; a slot whose pos is outside 0 .. R - 1 is left out, and no row may stand in
 * pos twice (what is written there is then one of the two).  Rows that no slot has
 * stay as they were.
 *
 * route_gather_f16, _bf16, _fp8        Xs[pos[t,j]] = X[t]; _fp8 moves e4m3 rows with
 *                                      their scales [.., ceil(K/128)]
 * route_combine_f16, _bf16             Y[t] = sum_j weights[t,j] * D[pos[t,j]]
 *                                      (weights NULL: ones, the gradient of a gather)
 * route_combine_grad_f16, _bf16        dD[pos[t,j]] = weights[t,j] * dY[t]
 *                                      dweights[t,j] = sum_c dY[t,c] * D[pos[t,j],c]
 *                                      (0 for a slot that is left out)
 *
 * Sums in FP32, one rounding of each 16-bit output.
 *   X, Y, dY [T,K]; Xs, D, dD [R,K]  16-byte aligned; pos, scales and weights 4-byte
 *   T < 2^24, 1 <= k <= 32, R <= 2^31 - 512, K <= 2^20, K % 8 == 0 (16 for _fp8)
 * T == 0 or K == 0 touches nothing, but for dweights, which are then zeros where T > 0.
 */
int route_gather_f16(const void *X, const int32_t *pos, void *Xs, int64_t T, int64_t k, int64_t R, int64_t K,
                     void *stream);
int route_gather_bf16(const void *X, const int32_t *pos, void *Xs, int64_t T, int64_t k, int64_t R, int64_t K,
                      void *stream);
int route_gather_fp8(const void *X, const float *scale, const int32_t *pos, void *Xs, float *scales, int64_t T, int64_t k,
                     int64_t R, int64_t K, void *stream);
int route_combine_f16(const void *D, const int32_t *pos, const float *weights, void *Y, int64_t T, int64_t k, int64_t R,
                      int64_t K, void *stream);
int route_combine_bf16(const void *D, const int32_t *pos, const float *weights, void *Y, int64_t T, int64_t k, int64_t R,
                       int64_t K, void *stream);
int route_combine_grad_f16(const void *dY, const void *D, const int32_t *pos, const float *weights, void *dD,
                           float *dweights, int64_t T, int64_t k, int64_t R, int64_t K, void *stream);
int route_combine_grad_bf16(const void *dY, const void *D, const int32_t *pos, const float *weights, void *dD,
                            float *dweights, int64_t T, int64_t k, int64_t R, int64_t K, void *stream);

/*
 * gemvtile_xcd_logical_id -- the logical workgroup id the persistent GEMM
 * gives hardware workgroup `w` of a `grid`-wide launch.  Workgroups are
 * dispatched to the 8 XCDs round-robin; when grid % 8 == 0 the renumbering
 * gives each XCD one contiguous range of ids (so neighbouring tiles in the
 * grouped order share an L2), otherwise it is the identity.  Host-only;
 * returns -1 for w outside [0, grid) or grid <= 0.
 */
int64_t gemvtile_xcd_logical_id(int64_t w, int64_t grid);

#ifdef __cplusplus
}
#endif

#endif /* GEMVTILE_H */
