/*
 * lbv.h -- few-row low-bit verify matmul for GB300 (sm_103a).
 *
 *   Y[M,N] = X[M,K] . dequant(Wp)[K,N],   1 <= M <= 8 drafted rows.
 *
 * Wp is a packed low-bit weight matrix that is consumed directly: every
 * weight is decoded once, in registers, and used against every row; it is
 * never expanded in memory.  (Ishizuki README, "Kernels written for the
 * verify": the verify kernel decodes each weight once into a matrix fragment
 * and multiplies it against every drafted row; Bonsai-27B-mlx-1bit model card:
 * packed weights are consumed directly, never expanded back to FP16.)
 *
 * Conventions for every entry point:
 *   - Plain C ABI: pointers and sizes only.  "dev" pointers are CUDA device
 *     memory of the current device, "host" pointers are host memory.
 *   - The caller owns every buffer.  The library never allocates in
 *     lbv_verify_gemm, lbv_verify_fused, lbv_verify_grouped, lbv_fwht128 or
 *     lbv_dequant_fp16.  Plans are created and
 *     destroyed by the caller and are immutable in between (safe to share
 *     between host threads).
 *   - Device work is asynchronous on the given stream; a status of LBV_OK
 *     means the work was enqueued.  Errors are returned, never aborted on; no
 *     kernel traps.  lbv_last_error() gives a thread-local message for the
 *     last failing call of the calling thread.
 *   - X rows are fp16 or bf16 (the plan's xdtype), row-major with leading
 *     dimension ldx (elements); Y is fp32 row-major with leading dimension ldy.
 *     Rows >= M of Y are never written.
 */
#ifndef LBV_H
#define LBV_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define LBV_API __attribute__((visibility("default")))
#else
#define LBV_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* A CUDA stream (binary-compatible with cudaStream_t); NULL = legacy stream. */
typedef struct CUstream_st* lbv_stream;

typedef enum {
    LBV_OK = 0,
    LBV_ERR_INVALID_ARG = 1,   /* bad pointer, size, M, dtype or leading dimension */
    LBV_ERR_UNSUPPORTED = 2,   /* valid request this build does not implement     */
    LBV_ERR_CUDA = 3,          /* a CUDA runtime call failed (message has details) */
    LBV_ERR_WORKSPACE = 4,     /* caller buffer too small                           */
    LBV_ERR_TIMEOUT = 5,       /* a bounded device wait gave up                     */
    LBV_ERR_BOUNDS = 6         /* a kernel's own range check failed (an internal
                                  error: the access was skipped, the output is wrong) */
} lbv_status;

typedef enum {
    /* 1-bit sign, one fp16 scale per 128 K-weights of a column: bit 0 -> -s,
     * bit 1 -> +s, 1.125 bits/weight.  Bonsai-27B-mlx-1bit model card,
     * format description. */
    LBV_FMT_SIGN1_G128 = 0,
    /* 2-bit affine groups, w = s*q + b, q in {0..3}, fp16 (s, b) per group of
     * 32, 64 or 128 K-weights: 2 + 32/g bits/weight.  Ishizuki README ("plain
     * MLX affine packs"); dflash-mlx-bonsai2 README ("Why"). */
    LBV_FMT_AFFINE2 = 1,
    /* GGUF Q4_0 blocks of 32: fp16 d and 16 bytes of nibbles, w = d*(q-8),
     * 4.5 bits/weight.  Ishizuki README, "Credits" (GGUF blocks read as they
     * are). */
    LBV_FMT_Q4_0 = 2
} lbv_format;

/* LBV_F32: only where an entry point says so (rows of lbv_rope_append, logits of
 * lbv_sample); plans, groups and caches take the two 16-bit types. */
typedef enum { LBV_F16 = 0, LBV_BF16 = 1, LBV_F32 = 2 } lbv_dtype;

/* Plan flags. */
#define LBV_PLAN_MEASURE     0x1u  /* time the candidate launch shapes (as
                                      back-to-back launches over copies of
                                      scratch weights, >= 2x L2, after an L2
                                      flush) and the 1-row path at plan
                                      creation and keep the fastest per row
                                      count (allocates and synchronises
                                      inside lbv_plan_create) */
#define LBV_PLAN_FORCE_FEWROW 0x2u /* always use the few-row kernel           */
#define LBV_PLAN_FORCE_GEMV   0x4u /* always use the 1-row path (run per row) */
#define LBV_PLAN_PDL          0x8u /* launch with programmatic dependent launch:
                                      the kernel starts streaming Wp before the
                                      previous kernel on the stream has finished
                                      (X is read and Y written only after it has).
                                      Only valid if the kernel launched just
                                      before on the stream never writes Wp. */
#define LBV_PLAN_TCGEN05     0x10u /* use the tcgen05 few-row kernel (A operand
                                      in tensor memory, 128-column tiles) for
                                      every M.  Such a plan reads its own device
                                      layout: pack with lbv_plan_pack and size
                                      buffers with lbv_plan_packed_bytes.  Not
                                      combinable with LBV_PLAN_FORCE_GEMV. */
#define LBV_PLAN_TC_E4M3      0x40u /* use the e4m3 tensor-memory kernel for every M
                                      (1-bit sign g128 and 2-bit affine g128
                                      only, K % 128 == 0; LBV_ERR_UNSUPPORTED
                                      otherwise): weights decoded to e4m3 bytes
                                      in tensor memory, the activations split
                                      exactly into three e4m3 terms per row,
                                      tcgen05.mma kind::f8f6f4, fp32
                                      accumulation.  Such a plan reads its own
                                      device layout: pack with lbv_plan_pack and
                                      size buffers with lbv_plan_packed_bytes.
                                      Not combinable with LBV_PLAN_TCGEN05,
                                      LBV_PLAN_FORCE_GEMV or
                                      LBV_PLAN_TEST_WAIT_LIMIT. */
#define LBV_PLAN_TEST_WAIT_LIMIT 0x20u /* test only: the few-row kernel's waits
                                      on its weight stages give up after 256
                                      tries, and the first warp of the first
                                      CTA leaves its second stage's copy out,
                                      so that wait runs out on purpose: the
                                      warp stops, waits (with the normal
                                      limit) for the copies it did issue and
                                      the kernel ends; the plan's device status
                                      then reports LBV_ERR_TIMEOUT and the
                                      output is incomplete.  Not combinable with
                                      LBV_PLAN_TCGEN05, LBV_PLAN_FORCE_GEMV or
                                      LBV_PLAN_MEASURE. */

/* Kernel ids reported by lbv_plan_query. */
#define LBV_KERNEL_FEWROW    1     /* mma.sync few-row kernel (default)       */
#define LBV_KERNEL_GEMV      2     /* 1-row path, run once per row           */
#define LBV_KERNEL_FEWROW_TC 3     /* tcgen05 few-row kernel (LBV_PLAN_TCGEN05) */
#define LBV_KERNEL_FEWROW_TC8 4    /* e4m3 tensor-memory kernel (LBV_PLAN_TC_E4M3) */

typedef struct lbv_plan lbv_plan;   /* opaque, library-owned */

/* ------------------------------------------------------------------------ */
/* Packing (host): canonical file layout -> the library's device layout.     */

/*
 * Size in bytes of the default device layout (the one the mma.sync few-row
 * kernel and the 1-row path read) of a K x N matrix, or 0 for an invalid
 * shape.  One record per (16-column tile, K chunk), tile-major.  For
 * N % 16 == 0 and K a multiple of the format's chunk (256 for sign1, 128 for
 * affine2, 64 for Q4_0) it equals the canonical size exactly
 * (1.125, 2 + 32/g and 4.5 bits per weight); otherwise the last column tile
 * and K chunk are padded with zero codes and zero scales, which contribute
 * exactly 0.  `group` is ignored except for LBV_FMT_AFFINE2.
 */
LBV_API size_t lbv_packed_bytes(lbv_format fmt, int K, int N, int group);

/*
 * bits: host uint32 [N][K/32], bit k%32 of word k/32 = sign bit of weight
 * (k, n) (little end first); scales: host fp16 bit patterns [N][K/128].
 * K % 128 == 0.  out: host buffer of lbv_packed_bytes() bytes.
 * Bonsai-27B-mlx-1bit model card, format description.
 */
LBV_API lbv_status lbv_pack_sign_g128(const uint32_t* bits, const uint16_t* scales, int K, int N,
                              void* out, size_t out_bytes);

/*
 * codes: host uint32 [N][K/16], code of weight (k, n) in bits 2*(k%16)..+1 of
 * word k/16 ("16 per uint32, little end first"); scales, biases: host fp16
 * bit patterns [N][K/group], group in {32, 64, 128}, K % group == 0.
 */
LBV_API lbv_status lbv_pack_affine2(const uint32_t* codes, const uint16_t* scales,
                            const uint16_t* biases, int K, int N, int group, void* out,
                            size_t out_bytes);

/*
 * blocks: host bytes [N][K/32][18] in GGUF order: d (fp16, little-endian),
 * then qs[16]; element j < 16 = qs[j] & 15, element j + 16 = qs[j] >> 4.
 * K % 32 == 0.
 */
LBV_API lbv_status lbv_pack_q4_0(const uint8_t* blocks, int K, int N, void* out, size_t out_bytes);

/* ------------------------------------------------------------------------ */
/* Plans: all kernel and launch-shape selection happens here, once per shape
 * (Ishizuki releases v0.6.1: each weight shape's kernel is set up once when
 * the model loads; the verify kernel starts at the row count where it is
 * faster, per matrix).  The activation dtype is part of the key (Ishizuki
 * releases v0.6.1, "Verify kernels no longer mix up precisions"). */

/* Creates a plan for the current device.  Returns LBV_ERR_INVALID_ARG for
 * K, N <= 0 or a K the format cannot hold, LBV_ERR_UNSUPPORTED for a group
 * other than 32/64/128 (affine2) or a K so large that no K split (at most 8
 * CTAs) leaves each CTA's slice of X room in shared memory beside its weight
 * ring: on GB300 about 44-53 thousand, by format and activation dtype.  *out
 * is NULL on failure. */
LBV_API lbv_status lbv_plan_create(lbv_format fmt, int K, int N, int group, lbv_dtype xdtype,
                           unsigned flags, lbv_plan** out);
LBV_API lbv_status lbv_plan_destroy(lbv_plan* plan);

/* Size in bytes of the device layout the plan's kernels read: equal to
 * lbv_packed_bytes() of the plan's shape, except for LBV_PLAN_TCGEN05 plans,
 * whose layout is one record per (128-column tile, K chunk) (128 K for sign1
 * and affine2 g128, 64 K otherwise), padded with zero codes and scales, and
 * LBV_PLAN_TC_E4M3 plans, whose layout is one record per (128-column tile,
 * 32-column quarter, 128-K group), padded the same way.  0 for a NULL plan. */
LBV_API size_t lbv_plan_packed_bytes(const lbv_plan* plan);

/* Packs canonical host arrays into the plan's device layout (host buffer of
 * lbv_plan_packed_bytes() bytes).  part0..part2 are the arrays of
 * lbv_pack_sign_g128 (bits, scales, unused), lbv_pack_affine2 (codes, scales,
 * biases) or lbv_pack_q4_0 (blocks, unused, unused), laid out as documented
 * there.  LBV_ERR_WORKSPACE if out_bytes is too small. */
LBV_API lbv_status lbv_plan_pack(const lbv_plan* plan, const void* part0, const void* part1,
                                 const void* part2, void* out, size_t out_bytes);

/* For a row count M (1..8): the kernel that lbv_verify_gemm will launch
 * (LBV_KERNEL_FEWROW, LBV_KERNEL_GEMV, LBV_KERNEL_FEWROW_TC or LBV_KERNEL_FEWROW_TC8), its K
 * split (cluster size) and the
 * workspace it needs (always 0 in this build).  Any output may be NULL. */
LBV_API lbv_status lbv_plan_query(const lbv_plan* plan, int M, int* kernel_id, int* splits,
                          size_t* workspace_bytes);

/* The plan's launch shape for the few-row kernel: warps per CTA, column tiles
 * (16 columns each) per warp, K split and CTAs along N.  For tests and
 * benchmarks; any output may be NULL. */
LBV_API lbv_status lbv_plan_shape(const lbv_plan* plan, int* warps, int* tiles_per_warp, int* splits,
                          int* ctas_n);

/* Overrides the few-row launch shape ((warps, tiles_per_warp) in {(8, 2),
 * (8, 4), (16, 1), (16, 2)}, splits in 1..8, ctas_n = clusters along N >= 1, or 0 for as many
 * as can be resident).  Returns
 * LBV_ERR_UNSUPPORTED if the shape does not fit the device (shared memory).
 * For tuning sweeps; not thread-safe against concurrent verify calls.
 * LBV_PLAN_TCGEN05 plans report warps = tiles_per_warp = 0 and ignore both
 * on input (their kernel has a fixed CTA: three decode warpgroups and one
 * MMA warp each); so do LBV_PLAN_TC_E4M3 plans (four warpgroups of four
 * decode warps and one MMA warp each), whose splits must be 1, 2, 4 or 8. */
LBV_API lbv_status lbv_plan_set_shape(lbv_plan* plan, int warps, int tiles_per_warp, int splits,
                              int ctas_n);

/* With LBV_PLAN_MEASURE: the measured cold-L2 time (us) of the few-row kernel
 * and of the 1-row path run M times at row count M, and the crossover (the
 * smallest M that uses the few-row kernel; 9 if none).  Zero times without
 * LBV_PLAN_MEASURE.  Any output may be NULL. */
LBV_API lbv_status lbv_plan_measured(const lbv_plan* plan, int M, float* fewrow_us, float* gemv_us,
                             int* crossover);

/* Reads (and clears) the plan's device status word: LBV_ERR_TIMEOUT if a
 * verify kernel of this plan gave up a bounded wait for its weight copies
 * since the last check (its output is then incomplete), LBV_ERR_BOUNDS if a
 * kernel found one of its copy or buffer ranges outside its bounds and skipped
 * the access (the checked build's range checks, and the e4m3 kernel's
 * shared-memory carve-up check in every build), else LBV_OK.  Synchronises
 * with the device. */
LBV_API lbv_status lbv_plan_device_status(const lbv_plan* plan);

/*
 * Rows-per-call statistics ("dflash-mlx-bonsai2" README, Commands: the fork
 * keeps a histogram of how many drafted rows each verify call carried and
 * prints it at exit on request).  counts: host array of 8; counts[m - 1] =
 * the calls of this plan with M = m (lbv_verify_gemm, lbv_verify_fused,
 * lbv_verify_fused_noalloc) that returned LBV_OK since the plan was created
 * or last reset.  Failed calls and the plan's own launch measurement are not
 * counted.  A call counts when it is enqueued: one captured into a CUDA graph
 * counts once, at capture, since the graph's replays do not pass through the
 * library.  Counting is atomic: plans stay safe to share between threads.
 * LBV_ERR_INVALID_ARG for a NULL plan or counts.
 */
LBV_API lbv_status lbv_plan_rows_histogram(const lbv_plan* plan, uint64_t* counts);
LBV_API lbv_status lbv_plan_rows_reset(lbv_plan* plan);

/* ------------------------------------------------------------------------ */
/* The verify matmul.                                                         */

/*
 * Y[m][n] = sum_k X[m][k] * w[k][n] for m < M, n < N, fp32 accumulation.
 * X: dev [M][ldx] (plan xdtype), ldx >= K; Wp: dev, the device layout from
 * lbv_pack_* (lbv_packed_bytes bytes, 16-byte aligned); Y: dev fp32 [M][ldy],
 * ldy >= N.  1 <= M <= 8, else LBV_ERR_INVALID_ARG.  workspace may be NULL
 * with workspace_bytes 0 (no plan in this build needs one).  Rows >= M cost
 * the same as a full block of 8 and are never read or written (Ishizuki
 * releases v0.6.1; dflash-mlx-bonsai2 README: 2-8-row calls are padded to 8).
 * The result of row m depends only on row m of X (bitwise).
 */
LBV_API lbv_status lbv_verify_gemm(const lbv_plan* plan, const void* X, int M, int ldx,
                           const void* Wp, float* Y, int ldy, void* workspace,
                           size_t workspace_bytes, lbv_stream stream);

/*
 * Blockwise normalized Walsh-Hadamard rotation of activation rows:
 * Xr[m][b*128 + i] = RNE( sum_j H[i][j] * sx_j / sqrt(128) ), where
 * H[i][j] = (-1)^popcount(i & j) (Sylvester, natural order), x_j = X[m][b*128+j]
 * and sx_j = -x_j where bit (b*128+j) of `signs` is set (signs: dev uint32
 * [K/32], NULL for none).  The sum is exact and the one rounding is to the
 * dtype, so the result is the correctly rounded rotation.  X, Xr: dev [M][K]
 * contiguous, K % 128 == 0, 1 <= M <= 8; in place (X == Xr) allowed.
 * dflash-mlx-bonsai2 README, "What this fork adds" (fused sign, Hadamard
 * prep); Ishizuki README (2-bit Hadamard-rotated weights).
 */
LBV_API lbv_status lbv_fwht128(const void* X, void* Xr, int M, int K, lbv_dtype dtype,
                       const uint32_t* signs, lbv_stream stream);

/* ------------------------------------------------------------------------ */
/* Fused head: the rotation as the verify's prologue and a greedy argmax as  */
/* its epilogue, in one launch of the few-row kernel.                        */

#define LBV_FUSED_ROTATE 0x1u  /* rotate X blockwise before the product        */
#define LBV_FUSED_ARGMAX 0x2u  /* per-row argmax over the N logits              */

/* Bytes of the workspace an argmax call needs (128). */
LBV_API size_t lbv_fused_workspace_bytes(void);

/*
 * Y[m][:] = X'[m][:] . dequant(Wp) for rows m < M, with in the same kernel:
 *   LBV_FUSED_ROTATE: X' is the blockwise rotation of lbv_fwht128 (signs
 *     optional, dev uint32 [K/32] or NULL), computed per CTA from the staged
 *     X tile and kept in shared memory.  Its arithmetic differs from
 *     lbv_fwht128's: fp32 sums (the 16-point stages on the tensor cores), one
 *     fp32 multiplication by 1/sqrt(128), one rounding to the dtype; a
 *     rotated element can differ from the correctly rounded one by a unit in
 *     the last place.  Without it X' = X.  Needs K % 128 == 0.
 *   LBV_FUSED_ARGMAX: argmax_idx[m] (dev int32 [M]) = the column of the
 *     largest fp32 logit of row m, the smallest such column on ties, -0 equal
 *     to +0, the first NaN if any; argmax_val[m] (dev fp32 [M], or NULL) =
 *     that logit, bit for bit the value Y would hold.  The logits need not be
 *     written: Y may then be NULL (ldy ignored).
 * dflash-mlx-bonsai2 README, "What this fork adds" (the verify GEMM with a
 * fused sign, Hadamard and row-sum prep) and "What it does to the numbers"
 * (greedy decoding; acceptance decided by the argmax, up to fp16 ties).
 *
 * The other arguments and rules are those of lbv_verify_gemm, except that
 * the few-row kernel is used at every M (never the 1-row path).
 * workspace: dev, 16-byte aligned, >= lbv_fused_workspace_bytes(), needed
 * with LBV_FUSED_ARGMAX (else ignored; LBV_ERR_WORKSPACE when missing or
 * short).  The caller zeroes it once before its first use; every call leaves
 * it zeroed when its kernel completes.  Calls that may run at the same time
 * (other streams) need distinct workspaces; calls in one stream can share one.
 * Errors: LBV_ERR_INVALID_ARG as lbv_verify_gemm, for unknown ops bits, for
 * no output (Y NULL without LBV_FUSED_ARGMAX), for argmax_idx NULL with
 * LBV_FUSED_ARGMAX and for misaligned signs, argmax_idx or argmax_val;
 * LBV_ERR_UNSUPPORTED for LBV_PLAN_TCGEN05 plans (LBV_PLAN_TC_E4M3 plans
 * support every op), for the rotation with
 * K % 128 != 0 or with K slices of the plan's launch shape that are not
 * whole 128-element blocks.  If a bounded wait in the kernel gives up, the
 * plan's device status records it (lbv_plan_device_status) and argmax_idx
 * may be -1.
 */
LBV_API lbv_status lbv_verify_fused(const lbv_plan* plan, const void* X, int M, int ldx,
                                    const void* Wp, unsigned ops, const uint32_t* signs,
                                    float* Y, int ldy, int32_t* argmax_idx, float* argmax_val,
                                    void* workspace, size_t workspace_bytes, lbv_stream stream);

/*
 * lbv_verify_fused without a caller workspace, for callers that cannot
 * allocate device memory: an engine whose memory is one arena sized at start-up
 * (nothing may call cudaMalloc after that), or host code that must not make a
 * blocking allocation on its decode path.  The argmax scratch (the 128-byte
 * workspace layout; 256 bytes reserved) is a device array of the library
 * module itself, one per device, held by every device that loads the library
 * until the process exits.  Set-up: the first call on a device looks up the
 * array's device address (cudaGetSymbolAddress) and clears it on that call's
 * stream, so make the first call on each device before any stream capture; a
 * cudaDeviceReset invalidates the looked-up address for the rest of the
 * process.  Every call leaves the scratch zero.  The library allocates
 * nothing.  M > 8 is rejected (the scratch holds 8 rows).  Other arguments,
 * rules and errors as lbv_verify_fused.  Races: the scratch is shared by every
 * call on a device, so calls that could overlap in time (other streams, other
 * host threads without ordering) must not be made; calls in one stream are
 * ordered and safe.  The pages have no counterpart of this entry point.
 */
LBV_API lbv_status lbv_verify_fused_noalloc(const lbv_plan* plan, const void* X, int M, int ldx,
                                            const void* Wp, unsigned ops,
                                            const uint32_t* signs, float* Y, int ldy,
                                            int32_t* argmax_idx, float* argmax_val,
                                            lbv_stream stream);

/* ------------------------------------------------------------------------ */
/* Grouped verify: independent problems of one format and dtype in one       */
/* launch -- a model's matrices (the Q4_0 layer stack) or routed experts,    */
/* each with its own rows.                                                   */

typedef struct lbv_group lbv_group;     /* opaque, library-owned */

/* One problem of a grouped call (the i-th shape of the group). */
typedef struct lbv_problem {
    const void* X;      /* dev [M][ldx], the group's dtype                      */
    int M;              /* rows, 0..8; 0 skips the problem (nothing is written)  */
    int ldx;            /* >= K_i                                               */
    const void* Wp;     /* dev, the default device layout of K_i x N_i
                           (lbv_pack_*, lbv_packed_bytes), 16-byte aligned      */
    float* Y;           /* dev [M][ldy] fp32, rows >= M untouched               */
    int ldy;            /* >= N_i                                               */
} lbv_problem;

/*
 * Creates a group plan for `count` (1..256) problems of shapes K[i] x N[i]
 * (host arrays, each valid for the format as in lbv_plan_create).  The
 * problems of a launch class share one launch shape: 16 warps, two tiles per
 * unit, a K split (cluster size) that suits each of them, and cluster rows
 * (at least two waves of resident clusters) divided among them in proportion
 * to their packed bytes.  There is one class when some split of 1..8 suits
 * every problem (the split needing the fewest CTAs); otherwise each problem
 * joins the class of the smallest split at which its X slice fits in shared
 * memory.  flags: LBV_PLAN_PDL and/or LBV_PLAN_MEASURE, which times, per
 * class, the default shape and one to six waves of every split from the
 * class's own up to 8 on scratch buffers (allocated and freed here, cold L2,
 * M = 8) and keeps the fastest.  LBV_ERR_UNSUPPORTED if a problem fits no
 * split of 1..8.
 * Ijah README, "What's new (v0.2)": grouped routed-expert verify, each
 * expert's weights read once per verify cycle for all the rows routed to it,
 * bit-identical output.  Ishizuki README, acknowledgements: a megakernel over
 * a model's matrices needs a grid-wide barrier; these problems are
 * independent, so their launches need none.
 */
LBV_API lbv_status lbv_group_create(lbv_format fmt, int group, lbv_dtype xdtype, int count,
                                    const int* K, const int* N, unsigned flags, lbv_group** out);
LBV_API lbv_status lbv_group_destroy(lbv_group* group);

/* Launch classes of the plan (0 for NULL), and the class of a problem (-1 if
 * out of range). */
LBV_API int lbv_group_launches(const lbv_group* group);
LBV_API int lbv_group_problem_launch(const lbv_group* group, int problem);

/* Launch shape of class `launch`: tiles per warp unit (1 or 2), K split,
 * cluster rows with every problem of the class active.  set_shape puts every
 * problem in one class with the given shape; LBV_ERR_UNSUPPORTED if the split
 * does not suit every problem or the shape does not fit. */
LBV_API lbv_status lbv_group_shape(const lbv_group* group, int launch, int* tpw, int* splits,
                                   int* rows);
LBV_API lbv_status lbv_group_set_shape(lbv_group* group, int tpw, int splits, int rows);

/*
 * Y_i[m][:] = X_i[m][:] . dequant(Wp_i) for every problem i (problems: host
 * array of `count`, read during the call), one launch per class with an
 * active problem, in order on `stream`.  Row m of problem i is bit for bit
 * what lbv_verify_gemm gives with a plan of the same shape and the K split of
 * the problem's class (lbv_plan_set_shape(plan, 16, tpw, splits, 0)).
 * Problems with M = 0 get no clusters; a call with every M = 0 launches
 * nothing.  Errors: LBV_ERR_INVALID_ARG for M outside 0..8, null or
 * misaligned pointers of an active problem, ldx < K_i or ldy < N_i.  The
 * library allocates nothing.
 */
LBV_API lbv_status lbv_verify_grouped(const lbv_group* group, const lbv_problem* problems,
                                      lbv_stream stream);

/* As lbv_plan_device_status, for the group's kernels. */
LBV_API lbv_status lbv_group_device_status(const lbv_group* group);

/* As lbv_plan_rows_histogram, per active problem of each lbv_verify_grouped
 * call that returned LBV_OK: counts[m - 1] = problems run with M = m. */
LBV_API lbv_status lbv_group_rows_histogram(const lbv_group* group, uint64_t* counts);
LBV_API lbv_status lbv_group_rows_reset(lbv_group* group);

/*
 * The same counts over every plan and group of the process since the library
 * was loaded (not reset by the calls above).  With the environment variable
 * LBV_VERIFY_STATS set (and not "0"), the library prints them to stderr when
 * the process exits: one line, "lbv: verify rows per call: 1:n1 ... 8:n8
 * (calls C, mean rows R)".
 */
LBV_API lbv_status lbv_rows_histogram(uint64_t* counts);

/* ------------------------------------------------------------------------ */
/* The verify step around the matmul: the new tokens' keys and values enter a */
/* paged cache with their positions rotated in, the new tokens attend over    */
/* that cache, and tokens are drawn from the head's logits.                   */

/* The new tokens of one step.  Request r has the rows q_start[r] ..
 * q_start[r + 1] - 1 of the token-major tensors (n_r >= 0 of them) and a
 * context of kv_len[r] tokens, the new ones included: its new token i has the
 * cache position kv_len[r] - n_r + i.  Position p of request r lives in slot
 * p % page_size of page block_table[r][p / page_size].  All arrays are dev
 * int32, read by the kernels when they run.  Rows at or past
 * q_start[requests] belong to no request: nothing is written for them, and what
 * they hold does not matter (the append may load it). */
typedef struct lbv_batch {
    const int32_t* q_start;      /* [requests + 1], ascending, q_start[0] >= 0    */
    const int32_t* kv_len;       /* [requests]                                    */
    const int32_t* block_table;  /* [requests][table_stride], rows do not overlap */
    int requests;                /* 1..4096                                       */
    int tokens;                  /* rows of the token-major tensors, >= 0         */
    int table_stride;            /* >= table_pages                                */
    int table_pages;             /* entries per request                           */
} lbv_batch;

/* A token-major tensor [tokens][heads][head_dim]; strides in elements, the
 * last dimension contiguous. */
typedef struct lbv_rows {
    void* data;                  /* dev                                           */
    int heads;
    int dtype;                   /* lbv_dtype                                     */
    int64_t token_stride;
    int64_t head_stride;
} lbv_rows;

typedef struct lbv_kv_cache lbv_kv_cache;   /* opaque, library-owned, host memory only */

/* Describes a caller-owned paged cache: k and v (dev, 16-byte aligned, dtype
 * fp16 or bf16) hold pages x page_size x heads x head_dim elements at
 * page * page_stride + slot * token_stride + head * head_stride (elements,
 * any order of the dimensions, each a multiple of 8; one set of strides for
 * both).  page_size: a power of two, 8..1024; head_dim: 64 or 128.  Offsets
 * are 64-bit throughout.  Allocates host memory only; the handle is immutable.
 * LBV_ERR_UNSUPPORTED for other head dims and page sizes. */
LBV_API lbv_status lbv_kv_cache_create(void* k, void* v, int pages, int page_size, int heads,
                                       int head_dim, int64_t page_stride, int64_t token_stride,
                                       int64_t head_stride, lbv_dtype dtype, lbv_kv_cache** out);
LBV_API lbv_status lbv_kv_cache_destroy(lbv_kv_cache* cache);

/*
 * A paged cache held in 4 bits.  An element is round(code * scale + bias), rounded once
 * to the cache's dtype (fp16 or bf16), for a code of 0..15 and the scale and bias
 * (of that dtype) of its 64 elements of a head: 4.5 bits an element.  A page is
 * lbv_kv_cache4_page_bytes() bytes (0 for sizes that lbv_kv_cache4_create refuses),
 *     [heads][page_size / C][chunk of C = min(page_size, 64) slots]
 * and a chunk of keys (K) and values (V)
 *     codes  [K, V][head_dim / 64][C][32] bytes: word w (32 bits, little-endian) has element
 *            8 w + i in the bits from 4 (i / 2) + 16 (i % 2) on,
 *     scales [K, V][head_dim / 64][C] pairs of (scale, bias).
 * data: dev, 32-byte aligned, `pages` pages one after the other.  The handle is one
 * of lbv_kv_cache: lbv_rope_append (which rounds to the nearest code),
 * lbv_attend, lbv_kv_read, lbv_kv_keep and lbv_kv_copy_pages take it as they take a
 * cache of 16 bits.  Sizes and errors as lbv_kv_cache_create.
 */
LBV_API size_t lbv_kv_cache4_page_bytes(int page_size, int heads, int head_dim);
LBV_API lbv_status lbv_kv_cache4_create(void* data, int pages, int page_size, int heads,
                                        int head_dim, lbv_dtype dtype, lbv_kv_cache** out);

typedef enum {
    LBV_ROPE_HALF = 0,         /* pair j of a head: elements j and j + rot_dim/2   */
    LBV_ROPE_INTERLEAVED = 1   /* pair j of a head: elements 2j and 2j + 1          */
} lbv_rope_layout;

typedef enum {
    LBV_ROPE_NONE = 0,         /* f_j = base^(-2j/rot_dim)                          */
    LBV_ROPE_LINEAR = 1,       /* f_j / factor                                      */
    LBV_ROPE_BY_PARTS = 2      /* f_j * ((1 - g) / factor + g), g = clamp((r - low) /
                                  (high - low), 0, 1) with r = trained * f_j / 2 pi the
                                  turns of pair j in the trained length (Peng et al.
                                  2023, "YaRN", section 3.2).  Engines also ramp over
                                  the pair's index j between two bounds (rounded to
                                  whole pairs or not); a checkpoint that runs with those
                                  frequencies needs them given to lbv_rope_create as
                                  they are.                                         */
} lbv_rope_scaling;

/* Host helper: radians per position of the rot_dim/2 pairs.  rot_dim even,
 * base > 0; factor > 0 unless LBV_ROPE_NONE; trained > 0 and low < high for
 * LBV_ROPE_BY_PARTS. */
LBV_API lbv_status lbv_rope_frequencies(int rot_dim, double base, lbv_rope_scaling scaling,
                                        double factor, double trained, double low, double high,
                                        double* freqs);

typedef struct lbv_rope lbv_rope;           /* opaque, library-owned, host memory only */

/* A rotation of the first rot_dim elements of a head (a multiple of 8, 8..128)
 * by position * freqs[j] radians (host [rot_dim/2], finite; copied), cos and
 * sin multiplied by `factor` (1 for plain rotary positions).  The angle is
 * reduced exactly: frequencies are kept as 64-bit fractions of a turn and the
 * product with the position wraps by itself. */
LBV_API lbv_status lbv_rope_create(const double* freqs, int rot_dim, lbv_rope_layout layout,
                                   float factor, lbv_rope** out);
LBV_API lbv_status lbv_rope_destroy(lbv_rope* rope);

/*
 * For every new token: rotates its query heads into q_out and its key heads
 * into the cache, and copies its value heads into the cache.
 *   q, k, v: rows of one dtype (fp32 as the verify matmul writes them, fp16 or
 *     bf16); k and v have the cache's heads.  q_out: the cache's dtype, the
 *     heads of q; may be q itself when the dtypes agree.  q and q_out may both be
 *     NULL (keys and values only).
 *   positions: dev int32 [tokens] rotary positions, or NULL for the cache
 *     positions (a tree of drafted tokens has siblings at one position).
 * Sums are fp32, rounded once.  A token whose slot does not exist (a negative
 * position, one past the block table, a page outside the cache) has its key
 * and value left out; its query is rotated all the same.
 * A cache of 4 bits gets, for each 64 elements x of a rotated key or a value (fp32):
 * bias = min x and scale = (max x - min x) * (1 / 15), each rounded to the cache's
 * dtype, and the codes (x - bias) * (1 / scale), rounded to the nearest whole number in
 * 0..15 (all 0 where the scale is 0 or below 2^-126).  So that equal inputs give equal
 * codes wherever the definition is followed, every operation is rounded by itself
 * there: the angle's fraction of a turn is cut to 2^-40 and taken to fp32 radians, whose
 * cos and sin are fp32, and so are products and sums.  A group with a NaN or a
 * magnitude above 2^15 (fp16, whose 16-bit cache holds up to 65504) or 2^126 (bf16)
 * cannot be held and reads as NaN, all 64 of it: to lbv_attend it is a key or a value
 * that is not finite.
 * Errors: LBV_ERR_INVALID_ARG for null or misaligned pointers, sizes that do
 * not agree and dtypes that cannot be; LBV_ERR_UNSUPPORTED if rot_dim exceeds
 * the head.  The library allocates nothing.
 */
LBV_API lbv_status lbv_rope_append(const lbv_rope* rope, const lbv_batch* batch,
                                   const lbv_kv_cache* cache, const lbv_rows* q,
                                   const lbv_rows* k, const lbv_rows* v, const lbv_rows* q_out,
                                   const int32_t* positions, lbv_stream stream);

/* Bytes of the workspace lbv_attend needs for this cache, a batch (its counts
 * alone are read) and so many query heads; 0 for NULL.  They hold the parts of
 * the larger kernel for every SM (41 MB for heads of 128, 21 MB for 64, on 152
 * SMs), so one workspace serves batches of every size over caches of its head_dim. */
LBV_API size_t lbv_attend_workspace_bytes(const lbv_kv_cache* cache, const lbv_batch* batch,
                                          int heads);

/*
 * Attention of every new token of the batch over its request's context:
 *   out[t][h] = sum_j softmax_j(scale q[t][h] . k_j) v_j,   k, v of cache head
 *   h / (q->heads / cache heads),
 * over the keys j that token i of request r (cache position P = kv_len - n + i)
 * sees: those below kv_len that the block table maps, and
 *   without tree: j <= P;
 *   with tree (dev uint64 [tokens]): every key before the request's new tokens,
 *     and new token b < 64 where bit b of the token's word is set (a token sees
 *     itself only by its own bit; new tokens past the 64th are seen by none);
 *   with window > 0, also j > P - window (0: no window).
 * lse (dev fp32 [tokens][heads], or NULL) = the natural log of the sum of
 * exp(scale q . k_j).  A row that sees nothing gets out 0 and lse -inf.
 *   q, out: rows of the cache's dtype; q->heads a multiple of the cache's
 * heads.  Sums and softmax are fp32, the probabilities enter the second
 * product in the cache's dtype, out is rounded once.  What the product is divided
 * by adds the rounded probabilities in the few-row kernel (up to 16 rows, new
 * tokens times query heads of a group, a request on average); in the
 * tensor-memory kernel (more rows) those of blocks where one key is half of a row's
 * sum so far, and the unrounded ones of the others.  Over a cache of 4 bits the
 * few-row kernel serves up to 24 rows and divides by the sum of the unrounded
 * probabilities (an error of half a step of the type, where 4 bits hold a value to 2^-5
 * of its group's range).  So the same request may
 * differ by the rounding of the probabilities between batches of either kind.
 * lse adds the unrounded ones in both.  Scores are fp32 sums, of any size below
 * 2^127 (times scale and log2 e): the largest weighs most however large it is, and from
 * 2^24 on those that agree to fp32's rounding errors may share its weight.  Cache slots
 * at or past kv_len may hold anything; keys and values below it are taken to be finite
 * (one that is not makes NaN of rows that share a block with it, also of those that
 * the mask hides it from).
 * Contexts are shorter than 2^30.  A mapped page outside the cache reads as zeros.
 *   workspace: dev, 256-byte aligned, lbv_attend_workspace_bytes(); zeroed once
 * by the caller, left ready for the next call by every call; calls that may
 * run at the same time need distinct ones.  The result does not depend on
 * timing.  Errors: LBV_ERR_INVALID_ARG, LBV_ERR_WORKSPACE.  The library
 * allocates nothing.
 */
LBV_API lbv_status lbv_attend(const lbv_kv_cache* cache, const lbv_batch* batch, const lbv_rows* q,
                              const lbv_rows* out, float scale, int window, const uint64_t* tree,
                              float* lse, void* workspace, size_t workspace_bytes,
                              lbv_stream stream);

/* lbv_attend whose first `sinks` (>= 0) positions of a request stay visible behind a
 * window: with window > 0, key j is seen if j > P - window or j < sinks, beside the
 * other conditions.  Only the pages of those positions and of the windows are read.
 * lbv_attend is this call with sinks 0; without a window sinks change nothing. */
LBV_API lbv_status lbv_attend_sinks(const lbv_kv_cache* cache, const lbv_batch* batch,
                                    const lbv_rows* q, const lbv_rows* out, float scale, int window,
                                    int sinks, const uint64_t* tree, float* lse, void* workspace,
                                    size_t workspace_bytes, lbv_stream stream);

/* LBV_ERR_TIMEOUT if an attention kernel that used the workspace gave up a
 * bounded wait since the last check (its output is then incomplete), else
 * LBV_OK; clears the record.  Synchronises with the device. */
LBV_API lbv_status lbv_attend_status(void* workspace);

/*
 * Test export: lbv_attend whose waits give up after about half a millisecond
 * (in place of a second) and whose first CTA stops copying after `copies` (>= 0)
 * copies (a block of keys and values in the few-row kernel, one of either in
 * the tensor-memory kernel), so that what waits for the next one gives up.  The
 * call ends, lbv_attend_status reports LBV_ERR_TIMEOUT, and what other CTAs
 * computed is right.
 */
LBV_API lbv_status lbv_attend_test_wait(const lbv_kv_cache* cache, const lbv_batch* batch,
                                        const lbv_rows* q, const lbv_rows* out, float scale,
                                        int window, const uint64_t* tree, float* lse,
                                        void* workspace, size_t workspace_bytes, int copies,
                                        lbv_stream stream);

/*
 * The keys and values of the batch's new tokens as they are held: k[t][h] and v[t][h]
 * (rows of the cache's dtype with the cache's heads; one of them may be NULL) for every
 * row t of a request.  With q_start over whole contexts it reads those.  A token whose slot
 * does not exist reads as zeros.  Errors: LBV_ERR_INVALID_ARG.
 */
LBV_API lbv_status lbv_kv_read(const lbv_batch* batch, const lbv_kv_cache* cache, const lbv_rows* k,
                               const lbv_rows* v, lbv_stream stream);

/*
 * Keeps some of the batch's new tokens and closes up the cache behind the context they
 * follow: of request r the new tokens b < 64 whose bit b of kept[r] (dev uint64
 * [requests]) is set move, in order, to the cache positions kv_len - n, kv_len - n + 1, ...;
 * left[r] (dev int32 [requests], or NULL) = kv_len - n + their number.  Bits at or
 * past n do not count; new tokens past the 64th are dropped, unless all 64 bits are set:
 * then all n new tokens stay, however many (a prompt in a batch beside drafts).  What the
 * slots from left[r] to kv_len hold afterwards does not matter.  Keys keep the rotary
 * positions that they were appended with.  A move from or to a slot that does not exist
 * is left out.
 * The slots of the new tokens belong to one request each; left is apart from the batch's
 * arrays and from kept.  Errors: LBV_ERR_INVALID_ARG.
 */
LBV_API lbv_status lbv_kv_keep(const lbv_batch* batch, const lbv_kv_cache* cache, const uint64_t* kept,
                               int32_t* left, lbv_stream stream);

/*
 * Copies page src[i] to page dst[i], keys and values of every slot, for i < count (dev
 * int32 arrays; at most the cache's pages): for requests that share pages and write to
 * one of them, or to close up a cache.
 * A pair with a page outside the cache is left out.  No page is dst of one pair and
 * src or dst of another (the page would hold a mixture).  Errors:
 * LBV_ERR_INVALID_ARG.
 */
LBV_API lbv_status lbv_kv_copy_pages(const lbv_kv_cache* cache, const int32_t* src, const int32_t* dst,
                                     int count, lbv_stream stream);

/* How lbv_sample draws: dev arrays with one entry per row, each may be NULL. */
typedef struct lbv_sample_rules {
    const float* temperature;    /* NULL: 1; a row with T <= 0 (or NaN) takes its
                                    largest logit                                */
    const int32_t* top_k;        /* keep the k largest; <= 0: off                */
    const float* top_p;          /* keep the largest tokens until their weights
                                    reach this share (of what top-k kept); >= 1:
                                    off                                          */
    const float* min_p;          /* keep tokens of at least this share of the
                                    largest token's weight; <= 0: off            */
    const uint32_t* mask;        /* [M][mask_ld]: token i is allowed if bit i % 32
                                    of word i / 32 is set; NULL: all             */
    int64_t mask_ld;             /* words per row                                */
    int temperature_last;        /* 0: the filters see the weights after the
                                    temperature; 1: before it (Ishizuki README,
                                    sampler chain: top-k, top-p, min-p,
                                    temperature)                                 */
} lbv_sample_rules;

/*
 * token[m] = a token of row m < M drawn by u[m] (dev fp32, in [0, 1), taken to
 * 24 bits), prob[m] (or NULL) = its probability among the kept tokens.
 * logits: dev [M][ld], fp32 as the verify matmul writes them, fp16 or bf16.
 *   Weights are whole numbers, W = floor(2^40 exp((l - max) / T)) with fp32
 * arithmetic inside the exponential, so their sums do not depend on an order
 * and equal inputs give equal tokens at any batch.  Rank is by logit, the
 * lower index first among equals (-0 equals +0).  top-p keeps a token while the
 * weights ranked before it are less than floor(floor(top_p 2^24) total / 2^24);
 * the first token is always kept.  The token is the lowest index at which the
 * running sum of kept weights in index order exceeds floor(floor(u 2^24) kept
 * / 2^24).  NaN and -inf logits are never drawn; +inf ones share all weight.  A
 * row with nothing left to draw gives token -1 and prob 0.
 *   N at most 2^23 (LBV_ERR_UNSUPPORTED).  The library allocates nothing.
 */
LBV_API lbv_status lbv_sample(const void* logits, int M, int N, int64_t ld, lbv_dtype dtype,
                              const lbv_sample_rules* rules, const float* u, int32_t* token,
                              float* prob, lbv_stream stream);

/*
 * Test export: X' exactly as lbv_verify_fused with LBV_FUSED_ROTATE computes
 * it inside the verify kernel (the same device code, run on its own), for
 * element-by-element checks.  Arguments as lbv_fwht128 (in place allowed).
 */
LBV_API lbv_status lbv_fused_rotation(const void* X, void* Xr, int M, int K, lbv_dtype dtype,
                                      const uint32_t* signs, lbv_stream stream);

/*
 * Test export: the dense fp16 dequantized matrix, W[k][n] (dev, [K][N]
 * row-major, ldw = N) rounded once to nearest even from the exact weight.
 * Not part of the verify path (the verify never expands weights).
 */
LBV_API lbv_status lbv_dequant_fp16(const lbv_plan* plan, const void* Wp, uint16_t* W,
                            lbv_stream stream);

/* Thread-local message of the calling thread's last failing call ("" if none). */
LBV_API const char* lbv_last_error(void);

/* Library version string. */
LBV_API const char* lbv_version(void);

/*
 * 1 in the checked build (liblbv_checked.so, compiled with LBV_CHECKED), 0 in
 * the release library.  The checked build's kernels test, before each access
 * they cannot prove in range by construction, that it lies inside its buffer:
 * the shared-memory carve-up against the launch's dynamic shared memory, every
 * weight copy against the packed matrix and its ring slot, the X slice against
 * K and its row buffer, a stage's chunks against the staged slice, the K split's
 * partial slots against their buffer.  A failed test sets the status word's
 * bounds bit (LBV_ERR_BOUNDS from lbv_plan_device_status) and skips the access;
 * the kernel still ends, and its output is then wrong.  It stands in for a
 * memory checker where none can run.  The kernels around the matmul (append,
 * attention, sampling) have no such tests: they are the same in both builds.
 */
LBV_API int lbv_checked_build(void);

#ifdef __cplusplus
}
#endif
#endif /* LBV_H */
