/*
 * qg.h -- C ABI of the MI355X (gfx950) quantized GEMM library (libqg.so).
 *
 * The library computes Y = X * dequant(W)^T for low-bit weights with the
 * dequantization done inside the GEMM kernels, for dense layers and for
 * token-sorted MoE grouped layers.  The operations follow the problem
 * statement of the Humming announcement (vLLM / Ant Group, "Announcing
 * Humming", spke.com Japanese translation):
 *   - section "Unified quantization representation": a weight format is
 *     described by its bit width / number format, scale granularity, scale
 *     type and an optional zero point; activations have their own format.
 *   - section "Per-workload tuning and JIT compilation": preprocessing
 *     validates parameters, pads dimensions and repacks the tensors into the
 *     layout of the target kernel; at inference the chosen kernel runs on the
 *     preprocessed weights and the runtime activations; configurations are
 *     prepared per input-size (M) range and dispatched at run time.
 *   - section "Shared CUDA components": dequantization and scaling happen
 *     inside the kernel; dense and MoE GEMMs have their own task mapping.
 * and the AIREITER benchmark page ("vLLM Humming performance benchmark"),
 * sections "H100 group-32 W4A8" (MXFP4 weights x MXFP8 activations, one scale
 * per 32) and "SM80 single-request decode" (INT3 weights, M = 1).
 *
 * Conventions for every entry point:
 *   - Plain C, no exceptions cross the boundary, no abort/assert on caller
 *     input.  Every call validates all arguments before it launches anything;
 *     a failed validation has no side effects and returns a status.
 *   - "device" pointers are HIP device memory on the current device, "host"
 *     pointers are ordinary process memory.  The caller owns every buffer,
 *     including packed weights and workspaces; the library allocates nothing
 *     that outlives a call and has no destroy call.
 *   - Device work is enqueued on the caller's stream and is asynchronous;
 *     only qg_preprocess synchronizes (its stream) before returning.
 *   - Calls are thread-safe; two calls that share a workspace must be ordered
 *     on one stream.
 *
 * Standard (input) format handed to qg_preprocess, per expert:
 *   codes  : [N][K] row-major, each row an LSB-first bitstream of b-bit codes
 *            (code k sits in bits [b*k, b*k+b) of the row; rows are K*b/8
 *            bytes).  INT-b codes are two's complement, UINT-b codes are plain,
 *            e2m1 uses bit 3 as its sign, e0m codes bit b-1, e4m3 bit 7.
 *   scales : [N][K/g]: bf16 bit patterns (A16 formats) or e8m0 bytes (MXFP4);
 *            W8A8: fp32 [ceil(N/128)][K/128]; INT8 x INT8: fp32 [N].
 *   zeros  : [N][K/g] uint8 in 0..2^b-1 for UINT-b formats, NULL otherwise.
 * Activations: x is [rows][ldx] row-major: bf16, e4m3 bytes (MXFP8), or e2m1
 * codes two per byte (MXFP4: element k in the low nibble of byte k/2 when k is
 * even, the high nibble when odd; ldx counts elements), the MX types with
 * x_scales [rows][K/32] e8m0 bytes (row stride K/32), per desc.atype; e4m3
 * bytes with fp32 x_scales [rows] (FP8_TOKEN) or [rows][K/128] (FP8_BLOCK);
 * int8 with fp32 x_scales [rows] (INT8_TOKEN).
 * y is [rows][ldy] row-major, bf16 or fp32.
 *
 * Numerics (the contract the CPU oracle checks):
 *   - A16 formats: the dequantized weight is the exact real (q - z) * s, with
 *     q the decoded code, z the group's zero point (0 for signed formats) and
 *     s the group's bf16 scale.  Kernels form sum_k x*(q - z) per K-group with
 *     bf16 MFMA (codes are exact in bf16) and apply s per group in fp32.
 *   - Per-token FP8: y[r] = s_r * sum_k e4m3(a[r,k]) * Wdq[n,k] (MXFP4 Wdq).
 *   - W8A8: sum over 128-K blocks kb of sa[r][kb] * sw[n/128][kb] * the
 *     block's sum of e4m3 products, each block's partial scaled in fp32.
 *   - INT8 x INT8: the sum of products is an exact int32; y = its fp32 value
 *     times the row's scale times the column's scale, two fp32 roundings.
 *   - MXFP4 x MXFP8: e2m1 * 2^(e-127) times e4m3 * 2^(ea-127), exact operands
 *     into gfx950 scaled MFMA; MXFP4 x MXFP4 likewise with e2m1 activations.
 *   - fp32 accumulation; QG_O_BF16 output is the fp32 result rounded to
 *     nearest-even; QG_O_F32 exposes the fp32 accumulators.
 */
#ifndef QG_H_
#define QG_H_

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define QG_ABI_VERSION 1
#define QG_LAYOUT_VERSION 2

typedef enum {
  QG_OK = 0,
  QG_ERR_INVALID_ARGUMENT = 1, /* null pointer, bad enum, negative size */
  QG_ERR_SHAPE = 2,            /* K % group != 0, K % 32 != 0, ld too small, ... */
  QG_ERR_ALIGNMENT = 3,        /* a device pointer or leading dimension misaligned */
  QG_ERR_UNSUPPORTED = 4,      /* valid request with no kernel: caller may fall back */
  QG_ERR_BUFFER_TOO_SMALL = 5, /* packed buffer or workspace below the required size */
  QG_ERR_HIP = 6               /* a HIP call failed; see qg_last_hip_error() */
} qg_status;

typedef enum {
  QG_W_INT4 = 0,   /* signed two's complement [-8, 7], no zero point */
  QG_W_UINT4 = 1,  /* unsigned [0, 15] with a uint4 zero point per group */
  QG_W_INT3 = 2,   /* signed two's complement [-4, 3], no zero point */
  QG_W_UINT3 = 3,  /* unsigned [0, 7] with a zero point per group */
  QG_W_MXFP4 = 4,  /* OCP e2m1 with one e8m0 scale per 32 along K */
  QG_W_INT8 = 5,   /* signed two's complement [-128, 127], no zero point */
  QG_W_UINT8 = 6,  /* unsigned [0, 255] with a uint8 zero point per group */
  QG_W_INT2 = 7,   /* signed two's complement [-2, 1], no zero point */
  QG_W_UINT2 = 8,  /* unsigned [0, 3] with a zero point per group */
  QG_W_INT1 = 9,   /* signed two's complement 1-bit: code 0 = 0, code 1 = -1 */
  QG_W_UINT1 = 10, /* unsigned [0, 1] with a zero point per group */
  QG_W_E0M3 = 11,  /* zero-exponent float: sign bit 3, magnitude bits 0..2 (-7..7) */
  QG_W_E0M7 = 12,  /* zero-exponent float: sign bit 7, magnitude bits 0..6 (-127..127) */
  QG_W_FP8 = 13    /* OCP e4m3 (one byte per weight) */
} qg_wtype;

typedef enum { QG_S_BF16 = 0, QG_S_E8M0 = 1, QG_S_F32 = 2 } qg_stype;
/* FP8_TOKEN: e4m3 bytes with one fp32 scale per row (x_scales [rows]).
 * FP8_BLOCK: e4m3 bytes with one fp32 scale per row and 128 K (x_scales
 * [rows][K/128], row stride K/128). */
typedef enum {
  QG_A_BF16 = 0,
  QG_A_MXFP8 = 1,
  QG_A_MXFP4 = 2,
  QG_A_FP8_TOKEN = 3,
  QG_A_FP8_BLOCK = 4,
  QG_A_INT8_TOKEN = 6 /* int8 with one fp32 scale per row (x_scales [rows]); 5 is not assigned and refused */
} qg_atype;
typedef enum { QG_O_BF16 = 0, QG_O_F32 = 1 } qg_otype;
/* Activation of a gated feed-forward block: v / (1 + e^-v), or
 * v (1 + tanh(sqrt(2 / pi) (v + 0.044715 v^3))) / 2. */
typedef enum { QG_ACT_SILU = 0, QG_ACT_GELU_TANH = 1 } qg_act;

/* How MoE rows are addressed.  A pair p = t*topk + j is token t's j-th expert
 * choice.  BY_TOKEN: row t of the operand (gate/up input).  BY_PAIR: row p
 * (down input, and the usual output).  SORTED: row i of the expert-sorted
 * order, i.e. the row of pair sorted_pair_ids[i]. */
typedef enum { QG_ROWS_BY_TOKEN = 0, QG_ROWS_BY_PAIR = 1, QG_ROWS_SORTED = 2 } qg_rowmode;

/* Layer + compute description ("Layer Config" / "Compute Config" of the
 * announcement's tuning section).  Supported (wtype, stype, atype, group):
 *   INT4/UINT4/INT3/UINT3, BF16 scales, BF16 activations, group 32, 64 or 128;
 *   INT8/UINT8/INT2/UINT2/INT1/UINT1, E0M3/E0M7 and FP8 (e4m3), BF16 scales,
 *   BF16 activations, group 32, 64 or 128 (the announcement's "WnA16"
 *   section: integer and floating-point weights of 1 to 8 bits on the shared
 *   dequantize-and-compute path; e0m codes, section "Quantization support",
 *   hold the values of INT4 without -8 / INT8 without -128 and are stored as
 *   those integers; the LDS-tiled large-M kernels serve the 4- and 3-bit
 *   formats and E0M3; the others run the decode kernels up to 16 rows when
 *   K % 512 == 0 and the 16-row skinny kernel otherwise);
 *   MXFP4, E8M0 scales, FP8_TOKEN activations, group 32 (W4A8 with per-token
 *   FP8 activations, section "End to end": the scaled MFMA with unit
 *   activation block scales, each output row times its row's fp32 scale;
 *   skinny kernel below 128 rows (dense) or for experts with few rows (MoE),
 *   the LDS-tiled scaled-MFMA kernel otherwise);
 *   FP8 (e4m3), F32 scales, FP8_BLOCK activations, group 128 (W8A8 with
 *   block-wise scaling, section "W8A8 / W4A8 / W4A4": one fp32 scale per
 *   128 x 128 block of W, scales [N/128 rounded up][K/128]; K % 128 == 0;
 *   skinny kernel below 128 rows (dense) or for experts with few rows (MoE),
 *   the LDS-tiled e4m3 x e4m3 scaled-MFMA kernel otherwise);
 *   MXFP4, E8M0 scales, MXFP8 activations, group 32 (W4A8 on the scaled MFMA);
 *   MXFP4, E8M0 scales, BF16 activations, group 32 (each code dequantized in
 *   the kernel to the exact bf16 e2m1 * 2^(e-127); the announcement's
 *   "Choosing the activation type": MXFP4 checkpoints on a bf16 compute path);
 *   MXFP4, E8M0 scales, MXFP4 activations, group 32, K % 128 == 0 (W4A4, the
 *   announcement's "W8A8 / W4A8 / W4A4" section: dense calls from 128 rows
 *   put both e2m1 operands into the scaled MFMA, and so do qg_moe_gemm's
 *   tiled kernels; the skinny kernel (dense below 128 rows, MoE experts with
 *   few rows) widens each activation fragment to e4m3 in registers -- every
 *   e2m1 value is an e4m3 value under the same scale).
 *   INT8, F32 scales, INT8_TOKEN activations, group = K, K < 2^17, one expert
 *   (integer products with one scale per output channel and per token; dense
 *   calls without autotune, and qg_gated_gemm).
 * Other valid combinations return QG_ERR_UNSUPPORTED. */
typedef struct {
  int32_t abi_version; /* must be QG_ABI_VERSION */
  int32_t wtype;       /* qg_wtype */
  int32_t stype;       /* qg_stype */
  int32_t group_size;  /* K elements per scale */
  int32_t atype;       /* qg_atype the weights will be multiplied with */
  int32_t num_experts; /* 1 for a dense layer */
  int64_t n;           /* output features (rows of W) */
  int64_t k;           /* input features; must be a multiple of 32 and of group_size */
} qg_layer_desc;

/* A preprocessed weight: plain data, owned by the caller, safe to copy.
 * Filled by qg_preprocess (or qg_weight_bind for a blob packed earlier). */
typedef struct {
  qg_layer_desc desc;
  void *data;              /* device buffer holding the packed layout */
  uint64_t bytes;          /* size of data in bytes */
  int32_t layout_version;  /* QG_LAYOUT_VERSION */
  int32_t n_tiles;         /* ceil(N / 16) */
  int32_t k_blocks;        /* K / 128 rounded up */
  int32_t groups_padded;   /* K / group rounded up to a multiple of 32 */
  uint64_t expert_stride;  /* bytes from one expert's section to the next */
  uint64_t scales_offset;  /* byte offset of the scales inside an expert section */
  uint64_t zeros_offset;   /* byte offset of the zero points (0 if none) */
} qg_weight;

/* Bytes of device memory the packed layout of `desc` needs (all experts). */
qg_status qg_packed_size(const qg_layer_desc *desc, uint64_t *bytes);

/* Host-only repack of experts [expert_begin, expert_begin + expert_count) from
 * the standard format into the packed layout.  codes/scales/zeros point at the
 * first of those experts (host memory, standard format).  dst is a host buffer
 * of qg_packed_size bytes laid out for all experts; only the given experts'
 * sections are written.  Runs on the CPU; needs no GPU. */
qg_status qg_repack_host(const qg_layer_desc *desc, const void *codes, const void *scales,
                         const void *zeros, int32_t expert_begin, int32_t expert_count,
                         void *dst, uint64_t dst_bytes);

/* Validate, pad and repack host standard-format tensors for experts
 * [expert_begin, expert_begin + expert_count) and copy them into the device
 * buffer dst_dev (qg_packed_size bytes, 256-byte aligned).  Fills *out (which
 * is valid once every expert has been preprocessed).  Synchronizes `stream`
 * before returning. */
qg_status qg_preprocess(const qg_layer_desc *desc, const void *codes, const void *scales,
                        const void *zeros, int32_t expert_begin, int32_t expert_count,
                        void *dst_dev, uint64_t dst_bytes, hipStream_t stream, qg_weight *out);

/* Describe an already packed device blob (e.g. one restored from storage that
 * qg_repack_host produced) without touching it. */
qg_status qg_weight_bind(const qg_layer_desc *desc, void *dst_dev, uint64_t dst_bytes,
                         qg_weight *out);

/* Workspace bytes qg_gemm needs for `m` rows (0 when none is needed).
 * Layout of a dense workspace: the first 64 KiB hold the arrival counters of
 * split-K launches (one per output tile; a launch that splits K counts its
 * workgroups in and leaves the counters at zero again), and the bytes after
 * them are scratch (fp32 partial tiles, the large-M kernels' pre-pass
 * results) whose contents never matter.  So a workspace must be zero-filled
 * once before its first use (its first 64 KiB suffice) and then serves any
 * sequence of qg_gemm / qg_gemm_ex calls -- any layer, any m -- ordered on one
 * stream, provided it holds the size each call asks for. */
qg_status qg_gemm_workspace_size(const qg_weight *w, int64_t m, uint64_t *bytes);

/* Dense GEMM: y[m][n] = x[m][:K] * dequant(W)^T.
 *   x        device, [m][ldx] bf16, e4m3 bytes or e2m1 nibble pairs (per
 *            desc.atype), 16-B aligned, ldx >= K and the row pitch (ldx
 *            elements) a multiple of 16 bytes (ldx % 32 == 0 for MXFP4).
 *   x_scales device, [m][K/32] e8m0 (MX activations), fp32 [m] (FP8_TOKEN)
 *            or fp32 [m][K/128] (FP8_BLOCK), 4-B aligned for fp32; ignored /
 *            may be NULL for bf16 activations.
 * The MX large-M kernel addresses X with 32-bit offsets: an MX call whose
 * activation rows span 4 GiB or more (m * row pitch) returns
 * QG_ERR_UNSUPPORTED.
 *   y        device, [m][ldy] of otype, 16-B aligned, ldy >= N.
 *   ws       device workspace of at least qg_gemm_workspace_size bytes
 *            (may be NULL when that size is 0).
 * m == 0 is a no-op returning QG_OK.  Asynchronous on `stream`. */
qg_status qg_gemm(const qg_weight *w, const void *x, const void *x_scales, int64_t m,
                  int64_t ldx, void *y, int32_t otype, int64_t ldy, void *ws, uint64_t ws_bytes,
                  hipStream_t stream);
/* (ws, when needed, must hold zeros on entry; see qg_gemm_workspace_size.) */

/* qg_gemm for callers that cannot allocate memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the same
 * kernels, with the workspace replaced by a static device array of
 * QG_NOALLOC_SCRATCH_BYTES that each GPU the library runs on holds until the
 * process ends.  The call allocates nothing (no hipMalloc / hipFree, no
 * allocating library call); on its first use on a device it looks the
 * array's address up and clears its split-K counter prefix with a kernel on
 * `stream`.  Every call on one GPU shares that GPU's array and the array
 * keeps the last call's contents: calls that may overlap on one GPU (other
 * streams, other threads) race and must be ordered by the caller.  A call
 * whose kernels would need more scratch than the array holds returns
 * QG_ERR_BUFFER_TOO_SMALL before launching anything (qg_gemm with a caller
 * workspace serves it).  Arguments and all other errors as in qg_gemm. */
#define QG_NOALLOC_SCRATCH_BYTES (8u << 20)
qg_status qg_gemm_noalloc(const qg_weight *w, const void *x, const void *x_scales, int64_t m, int64_t ldx,
                          void *y, int32_t otype, int64_t ldy, hipStream_t stream);

/* Compute options of qg_gemm_ex (the announcement's "Compute Config" names
 * batch invariance among the compute options of a GEMM, section "Per-workload
 * tuning and JIT compilation").
 *   QG_GEMM_BATCH_INVARIANT: every output row is bit-identical whatever m is
 *   (and whatever the other rows hold): the kernel and its reduction order
 *   are chosen from (N, K) only, never from m.  Slower than the default at
 *   small m (the large-M kernel serves every m when K % 128 == 0).  An
 *   integer-format layer with m * K * 2 >= 2^31 returns QG_ERR_UNSUPPORTED
 *   rather than switching kernels.  (INT8_TOKEN layers are batch-invariant
 *   with and without it: their sums are exact.)
 *   QG_GEMM_QUANTIZE_X (INT8_TOKEN layers; an invalid argument for others): x
 *   is bf16 [m][ldx] (ldx % 8 == 0) and the call quantizes its rows as
 *   qg_quantize_int8 does, into ws; x_scales is ignored. */
#define QG_GEMM_BATCH_INVARIANT 1u
#define QG_GEMM_QUANTIZE_X 2u

/* qg_gemm_workspace_size for the compute options `flags` (0 = qg_gemm's). */
qg_status qg_gemm_workspace_size_ex(const qg_weight *w, int64_t m, uint32_t flags, uint64_t *bytes);

/* qg_gemm with compute options `flags` (a combination of QG_GEMM_* bits;
 * unknown bits: QG_ERR_INVALID_ARGUMENT).  flags == 0 is exactly qg_gemm.
 * ws must hold qg_gemm_workspace_size_ex(w, m, flags) bytes, zero-filled once
 * as for qg_gemm. */
qg_status qg_gemm_ex(const qg_weight *w, const void *x, const void *x_scales, int64_t m,
                     int64_t ldx, void *y, int32_t otype, int64_t ldy, void *ws, uint64_t ws_bytes,
                     uint32_t flags, hipStream_t stream);

/* Autotune of the dense tuning table (announcement, "Future plans": candidate
 * configurations are benchmarked on the target device to find better
 * execution parameters per workload, complementing the heuristics).
 * qg_gemm_autotune runs the dense GEMM of this call once per candidate kernel
 * variant (the heuristic's choice, the decode / skinny / tiled kernels' other
 * compiled shapes that can serve m rows), times each with HIP events over
 * `reps` launches (1..64) after one warm-up launch, and records the fastest in
 * a process-wide table keyed by (wtype, group, N, K) and the M bucket of m
 * (1, 2-4, 5-8, 9-16, 17-64, 65-256, 257-1024, > 1024).  From then on qg_gemm,
 * qg_gemm_workspace_size and qg_describe_dispatch use that variant for every
 * m of the bucket it can serve (otherwise the heuristics); batch-invariant
 * calls ignore the table.  Query qg_gemm_workspace_size again after tuning:
 * the tuned variant may need a different workspace.
 *   x, x_scales, ldx, y, otype, ldy  as in qg_gemm; y is overwritten (the
 *            result of the last candidate run).
 *   ws       device, 256-B aligned, qg_gemm_autotune_workspace_size bytes;
 *            contents on entry do not matter (the call clears what must
 *            start at zero).  Not a qg_gemm workspace: it leaves scratch.
 *   flush    optional device buffer (16-B aligned, flush_bytes a multiple of
 *            16) read in full before every timed launch so that each launch
 *            starts from cold caches (pass more than the 256 MB MALL), or NULL.
 *   chosen   optional host buffer receiving the chosen variant's description;
 *   chosen_us optional host float receiving its mean time per launch (us).
 * Synchronizes `stream`.  Thread-safe (the table is guarded by a mutex). */
qg_status qg_gemm_autotune_workspace_size(const qg_weight *w, int64_t m, uint64_t *bytes);
qg_status qg_gemm_autotune(const qg_weight *w, const void *x, const void *x_scales, int64_t m,
                           int64_t ldx, void *y, int32_t otype, int64_t ldy, void *ws, uint64_t ws_bytes,
                           const void *flush, uint64_t flush_bytes, int32_t reps, hipStream_t stream,
                           char *chosen, uint64_t chosen_bytes, float *chosen_us);
/* MoE autotune (announcement, section "Future plans": benchmark candidate
 * configurations on the target device, complementing the heuristics).
 * qg_moe_autotune runs this grouped GEMM (the arguments of qg_moe_gemm, with
 * num_tokens >= 1 and the pairs already sorted by qg_moe_sort) once per
 * candidate dispatch plan -- every expert on the skinny kernel, or experts
 * with >= 16, 32, 64 or 128 rows on the tiled kernels' 128-row tiles and the
 * rest on the 64-row small tiles or the skinny kernel, MX tiles 128 or 256
 * columns wide -- times each with HIP events over `reps` calls (1..64) after
 * one warm-up call, and records the fastest plan in a process-wide table keyed
 * by (wtype, atype, group, N, K, experts) and the bucket of num_tokens * topk
 * (1-8, 9-64, 65-512, 513-4096, 4097-32768, more).  From then on qg_moe_gemm,
 * qg_moe_workspace_size and qg_describe_moe_dispatch use that plan for the
 * bucket (unless an experiment override of the MoE dispatch is set); query
 * qg_moe_workspace_size again after tuning.  y is overwritten (the last
 * candidate's result).
 *   ws     device, 256-B aligned, qg_moe_autotune_workspace_size bytes;
 *          contents on entry do not matter.  Not a qg_moe_gemm workspace.
 *   flush, flush_bytes, reps, chosen, chosen_bytes, chosen_us  as in
 *          qg_gemm_autotune (chosen: the plan's description).
 * Synchronizes `stream`.  Thread-safe (the table is guarded by a mutex). */
qg_status qg_moe_autotune_workspace_size(const qg_weight *w, int64_t num_tokens, int32_t topk, uint64_t *bytes);
qg_status qg_moe_autotune(const qg_weight *w, const void *x, const void *x_scales, int32_t x_rows,
                          const int32_t *sorted_pair_ids, const int32_t *expert_offsets, int64_t num_tokens,
                          int32_t topk, void *y, int32_t otype, int32_t y_rows, void *ws, uint64_t ws_bytes,
                          const void *flush, uint64_t flush_bytes, int32_t reps, hipStream_t stream, char *chosen,
                          uint64_t chosen_bytes, float *chosen_us);
/* Forget every autotuned entry, dense and MoE (back to the heuristics). */
void qg_autotune_reset(void);

/* Experiment overrides of the tuning table, for tests and parameter sweeps
 * (production code sets none).  At the first dispatch of the process the
 * library reads the environment variables of these names once; after that
 * only these calls change them.  name is one of QG_TUNE ("T,KR,W,splits": the
 * skinny kernel with these parameters), QG_DECODE ("0" disables the decode
 * kernel, "T,KR[,splits]" picks an instance), QG_TILED ("0" disables the
 * large-M kernels), QG_TILED_BM, QG_MX_BN, QG_MX_WAVES, QG_A16_WAVES,
 * QG_A16_BN, QG_MOE_TILED_MIN, QG_MOE_GROUP_M, QG_MOE_SMALL_BM, QG_MOE_SMALL,
 * QG_MOE_MX_BN, QG_DECODE_WIDE, QG_GROUP_M; value NULL or "" clears the override.  An unknown name returns
 * QG_ERR_INVALID_ARGUMENT.  A value outside an override's range is ignored
 * (the heuristic applies).  Thread-safe; a dispatch sees the overrides before
 * or after a concurrent change, never a mix.  qg_clear_overrides clears all
 * (the environment is not read again). */
qg_status qg_set_override(const char *name, const char *value);
void qg_clear_overrides(void);

/* Workspace bytes for qg_moe_sort and qg_moe_gemm with this many tokens (one
 * buffer of this size serves both; its contents on entry do not matter). */
qg_status qg_moe_workspace_size(const qg_weight *w, int64_t num_tokens, int32_t topk,
                                uint64_t *bytes);

/* Route-sort the pairs of a top-k router by expert (counting sort on the GPU).
 *   topk_ids        device int32 [num_tokens][topk], values in 0..num_experts-1
 *                   (out-of-range ids are skipped and counted nowhere).
 *   sorted_pair_ids device int32 [num_tokens*topk]: pair ids grouped by expert;
 *                   the order inside an expert's segment is unspecified.
 *   expert_offsets  device int32 [num_experts+1]: segment e is
 *                   [offsets[e], offsets[e+1]).
 *   ws              device workspace of qg_moe_workspace_size bytes.
 * Asynchronous on `stream`.  num_tokens == 0 writes zero offsets. */
qg_status qg_moe_sort(const int32_t *topk_ids, int64_t num_tokens, int32_t topk,
                      int32_t num_experts, int32_t *sorted_pair_ids, int32_t *expert_offsets,
                      void *ws, uint64_t ws_bytes, hipStream_t stream);

/* Grouped GEMM over the sorted pairs: for every pair p routed to expert e,
 * (any K that is a multiple of 32 and of the group; long K loops inside the
 * kernels' workgroups)
 *   y[row_y(p)] = x[row_x(p)] * dequant(W[e])^T
 * with row_x given by x_rows (BY_TOKEN: p / topk; BY_PAIR: p; SORTED: the
 * pair's position in sorted_pair_ids) and row_y by y_rows (BY_PAIR or SORTED).
 * x, x_scales, y as in qg_gemm with ldx = K and ldy = N (dense rows).
 * ws: device, 256-B aligned, at least qg_moe_workspace_size bytes (holds the
 * tile list of the large-expert kernel and, for integer formats, the group
 * row sums of x; overwritten by every call, so calls sharing one ws must be
 * ordered on one stream).
 * More than 1024 experts: QG_ERR_UNSUPPORTED (here and in qg_moe_sort).
 * Asynchronous on `stream`. */
qg_status qg_moe_gemm(const qg_weight *w, const void *x, const void *x_scales, int32_t x_rows,
                      const int32_t *sorted_pair_ids, const int32_t *expert_offsets,
                      int64_t num_tokens, int32_t topk, void *y, int32_t otype, int32_t y_rows,
                      void *ws, uint64_t ws_bytes, hipStream_t stream);

/* Activation quantization bf16 -> MXFP8 (announcement, section "Choosing the
 * activation type": a deployment may run a layer with MXFP8 activations on a
 * bf16 model, e.g. the MoE layers, so activations are quantized at run time
 * before the W4A8 GEMM).  Per row, per block of 32 values along K, following
 * the OCP Microscaling Formats v1.0 conversion: scale X = 2^(floor(log2
 * max|v|) - 8) clamped to 2^-127 .. 2^127 (X = 1 for an all-zero block), stored
 * as the e8m0 code log2(X) + 127; element = v / X rounded to the nearest e4m3
 * value, ties to the even code, magnitudes beyond 448 saturated to 448, sign
 * kept (a negative value that rounds to zero gives 0x80).  The result is
 * exact (no fp32 rounding is involved for bf16 inputs).
 *   x        device, bf16 [rows][ldx], 16-B aligned, ldx >= k, ldx % 8 == 0.
 *   q        device, e4m3 bytes [rows][ldq], 8-B aligned, ldq >= k, ldq % 8 == 0.
 *   q_scales device, e8m0 bytes [rows][k/32] (row stride k/32, the x_scales
 *            layout of qg_gemm / qg_moe_gemm), any alignment.
 * k % 32 != 0 or ld too small: QG_ERR_SHAPE.  rows == 0 or k == 0: no-op.
 * NaN / Inf inputs give unspecified codes.  Asynchronous on `stream`. */
qg_status qg_quantize_mxfp8(const void *x, int64_t rows, int64_t k, int64_t ldx, void *q,
                            int64_t ldq, void *q_scales, hipStream_t stream);

/* bf16 activations -> MXFP4 (e2m1 codes + e8m0 scales), the input of a W4A4
 * GEMM (announcement, section "W8A8 / W4A8 / W4A4": MXFP4 on both operands).
 * Per row, per block of 32 values along K, the OCP Microscaling Formats v1.0
 * conversion with e2m1's largest power of two, 2^2: scale X = 2^(floor(log2
 * max|v|) - 2) clamped to 2^-127 .. 2^127 (X = 1 for an all-zero block),
 * stored as the e8m0 code log2(X) + 127; element = v / X rounded to the
 * nearest e2m1 value (0, 0.5, 1, 1.5, 2, 3, 4, 6), ties to the even code,
 * magnitudes beyond 6 saturated to 6, sign kept (a negative value that rounds
 * to zero gives code 0x8).  Exact for bf16 inputs (no fp32 rounding).
 *   x        device, bf16 [rows][ldx], 16-B aligned, ldx >= k, ldx % 8 == 0.
 *   q        device, e2m1 nibble pairs [rows][ldq elements] (element j in the
 *            low nibble of byte j/2 when j is even), 4-B aligned, ldq >= k,
 *            ldq % 8 == 0.
 *   q_scales device, e8m0 bytes [rows][k/32] (row stride k/32), any alignment.
 * k % 32 != 0 or ld too small: QG_ERR_SHAPE.  rows == 0 or k == 0: no-op.
 * NaN / Inf inputs give unspecified codes.  Asynchronous on `stream`. */
qg_status qg_quantize_mxfp4(const void *x, int64_t rows, int64_t k, int64_t ldx, void *q,
                            int64_t ldq, void *q_scales, hipStream_t stream);

/* bf16 activations -> e4m3 with fp32 scales: per token (block == 0, one scale
 * per row; the announcement's section "End to end" serves W4A8 with per-token
 * FP8 activations) or per 128 values of a row (block == 128, the W8A8 input;
 * section "W8A8 / W4A8 / W4A4").  Per block with largest magnitude a (a
 * bf16 value, exact in fp32): scale s = a / 448 in IEEE fp32 (nearest-even;
 * s = 1 for an all-zero block); code = e4m3 of the fp32 quotient v / s
 * (IEEE division), nearest with ties to the even code, saturated at 448, sign
 * kept (a negative value that rounds to zero gives 0x80).
 *   x        device, bf16 [rows][ldx], 16-B aligned, ldx >= k, ldx % 8 == 0.
 *   q        device, e4m3 bytes [rows][ldq], 16-B aligned, ldq >= k, ldq % 16 == 0.
 *   q_scales device, fp32 [rows] (block 0) or [rows][ceil(k/128)] (block 128,
 *            row stride ceil(k/128)), 4-B aligned.
 * k % 8 != 0 or ld too small: QG_ERR_SHAPE; block not 0 or 128:
 * QG_ERR_INVALID_ARGUMENT.  rows == 0 or k == 0: no-op.  NaN / Inf inputs give
 * unspecified codes.  Asynchronous on `stream`. */
qg_status qg_quantize_fp8(const void *x, int64_t rows, int64_t k, int64_t ldx, int32_t block, void *q,
                          int64_t ldq, float *q_scales, hipStream_t stream);

/* SiLU-gated product of a fused gate/up projection (MoE output stage between
 * gate_up and down; announcement, section "Shared CUDA components": scaling
 * and bias work belongs to the output stage):
 *   h[r][j] = silu(gu[r][j]) * gu[r][inter + j],  silu(v) = v / (1 + e^-v),
 * for j < inter, computed in fp32 and rounded to bf16 (nearest-even).  With
 * h_type QG_A_MXFP8 those bf16 values are then quantized exactly as
 * qg_quantize_mxfp8 does, ready for an MXFP8 down projection.
 *   gu       device, [rows][ldgu] of gu_type (QG_O_BF16 or QG_O_F32, i.e. the
 *            gate_up GEMM's output type), 16-B aligned, ldgu >= 2*inter,
 *            rows 16-B aligned (ldgu % 8 for bf16, % 4 for fp32).
 *   h        device, [rows][ldh]: bf16 (16-B aligned, ldh % 8 == 0) or e4m3
 *            bytes (8-B aligned, ldh % 8 == 0), ldh >= inter.
 *   h_scales device, e8m0 [rows][inter/32] (QG_A_MXFP8 only, else ignored).
 * inter % 8 (bf16 output) or % 32 (MXFP8 output) != 0: QG_ERR_SHAPE.
 * rows == 0 is a no-op.  Asynchronous on `stream`. */
qg_status qg_silu_mul(const void *gu, int32_t gu_type, int64_t rows, int64_t inter, int64_t ldgu,
                      void *h, int32_t h_type, int64_t ldh, void *h_scales, hipStream_t stream);

/* Weighted combine of each token's top-k expert rows (MoE output stage):
 *   out[t][c] = sum_j topk_weights[t][j] * y[t*topk + j][c]  (+ bias[c])
 * summed in fp32 over j = 0 .. topk-1 in order, then stored as out_type
 * (bf16 nearest-even, or fp32).  y holds one row per pair p = t*topk + j, i.e.
 * the QG_ROWS_BY_PAIR output of qg_moe_gemm.
 *   y            device, [num_tokens*topk][ldy] of y_type (QG_O_BF16 / QG_O_F32),
 *                16-B aligned rows.
 *   topk_weights device, fp32 [num_tokens][topk], 4-B aligned.
 *   bias         device, bf16 [n] (16-B aligned) or NULL.
 *   out          device, [num_tokens][ldout] of out_type, 16-B aligned rows.
 * n % 8 != 0 or ld too small: QG_ERR_SHAPE; topk < 1: QG_ERR_INVALID_ARGUMENT.
 * num_tokens == 0 is a no-op.  out must not overlap y.  Asynchronous. */
qg_status qg_moe_combine(const void *y, int32_t y_type, int64_t ldy, const float *topk_weights,
                         int64_t num_tokens, int32_t topk, int64_t n, const void *bias, void *out,
                         int32_t out_type, int64_t ldout, hipStream_t stream);

/* bf16 activations -> int8 with one fp32 scale per row, the input of an
 * INT8_TOKEN layer: scale s = a / 127 in IEEE fp32 with a the row's largest
 * magnitude (s = 1 for a row of zeros); code = the integer nearest the fp32
 * quotient v / s (IEEE division), ties to even, in -127 .. 127.
 *   x        device, bf16 [rows][ldx], 16-B aligned, ldx >= k, ldx % 8 == 0.
 *   q        device, int8 [rows][ldq], 8-B aligned, ldq >= k, ldq % 8 == 0
 *            (qg_gemm wants 16-B aligned rows).
 *   q_scales device, fp32 [rows], 4-B aligned.
 * k % 8 != 0 or ld too small: QG_ERR_SHAPE.  rows == 0 or k == 0: no-op.  NaN /
 * Inf inputs give unspecified codes.  Asynchronous on `stream`. */
qg_status qg_quantize_int8(const void *x, int64_t rows, int64_t k, int64_t ldx, void *q, int64_t ldq,
                           float *q_scales, hipStream_t stream);

/* The gate / up half of a feed-forward block on an INT8_TOKEN layer in one
 * kernel: with w the fused layer of n = 2 * inter output channels (gate
 * 0 .. inter - 1, then up, as in qg_silu_mul),
 *   h[r][j] = act(y[r][j]) * y[r][inter + j],  y as qg_gemm gives it in fp32,
 * rounded once to otype.  x, x_scales, ldx, flags, stream as in qg_gemm_ex; h
 * device [m][ldh], 16-B aligned, ldh >= inter, 4-B aligned rows; ws
 * qg_gated_gemm_workspace_size bytes, zero-filled once as for qg_gemm.  An odd
 * n: QG_ERR_SHAPE; layers of other formats: QG_ERR_UNSUPPORTED (qg_gemm and
 * qg_silu_mul serve them).  m == 0 is a no-op. */
qg_status qg_gated_gemm_workspace_size(const qg_weight *w, int64_t m, uint32_t flags, uint64_t *bytes);
qg_status qg_gated_gemm(const qg_weight *w, const void *x, const void *x_scales, int64_t m, int64_t ldx, void *h,
                        int32_t otype, int64_t ldh, int32_t act, void *ws, uint64_t ws_bytes, uint32_t flags,
                        hipStream_t stream);

/* The same half of the block in bf16, for models before they are quantized
 * and for training, in one kernel:
 *   g = x Wg^T, u = x Wu^T, h = act(g) u   (fp32, rounded once to bf16).
 *   x   device, bf16 [m][ldx]; w device, bf16 [2 * inter][ldw], the gate rows
 *       first; both 16-B aligned, ld >= k, ld % 8 == 0, ld <= 2^22, k % 8 == 0;
 *       inter <= 2^24.
 *   h   device, bf16 [m][ldh], 16-B aligned, ldh >= inter.
 *   gu  device, [m][ldgu] of gu_type, 16-B aligned, ldgu >= 2 * inter, or NULL:
 *       g in columns 0 .. inter - 1 and u behind it, for the backward pass
 *       (QG_O_F32 keeps them as computed, QG_O_BF16 takes half the memory and
 *       rounds them).
 *   ws  qg_ffn_gated_workspace_size bytes, 256-B aligned, zero-filled once (its
 *       first 64 KiB suffice); NULL when that size is 0.
 * No rows, columns or strides beyond these are read or written.  m == 0 is a
 * no-op.  Asynchronous on `stream`. */
qg_status qg_ffn_gated_workspace_size(int64_t m, int64_t k, int64_t inter, uint64_t *bytes);
qg_status qg_ffn_gated(const void *x, int64_t ldx, const void *w, int64_t ldw, int64_t m, int64_t k, int64_t inter,
                       int32_t act, void *h, int64_t ldh, void *gu, int32_t gu_type, int64_t ldgu, void *ws,
                       uint64_t ws_bytes, hipStream_t stream);

/* Backward pass of qg_ffn_gated: with dh the gradient of h,
 *   du = dh act(g), dg = dh u act'(g)      (fp32, rounded once to bf16; kept
 *       in two bf16 parts for dx up to 16 and for dw up to 32 tokens.  With more
 *       tokens that rounding is in dx and dw, 1.7e-3 of their norm, whatever
 *       dw_type is)
 *   dx = dg Wg + du Wu,  dw = [dg du]^T x  (summed in fp32, rounded once).
 *   x, w  as in the forward pass.  dh device, bf16 [m][lddh], lddh >= inter.
 *   dx    device, bf16 [m][lddx], 16-B aligned, lddx >= k, or NULL.
 *   dw    device, [2 * inter][lddw] of dw_type (QG_O_BF16 or QG_O_F32), 16-B
 *         aligned, lddw >= k, or NULL.  It is overwritten; m == 0 fills it with
 *         zeros.
 *   gu    what the forward pass left, or NULL: g and u are computed again.
 *   ws    qg_ffn_gated_backward_workspace_size bytes (recompute: gu is NULL),
 *         256-B aligned, zero-filled once as above.
 * Asynchronous on `stream`. */
qg_status qg_ffn_gated_backward_workspace_size(int64_t m, int64_t k, int64_t inter, int32_t recompute,
                                               uint64_t *bytes);
qg_status qg_ffn_gated_backward(const void *x, int64_t ldx, const void *w, int64_t ldw, const void *dh, int64_t lddh,
                                int64_t m, int64_t k, int64_t inter, int32_t act, void *dx, int64_t lddx, void *dw,
                                int32_t dw_type, int64_t lddw, const void *gu, int32_t gu_type, int64_t ldgu,
                                void *ws, uint64_t ws_bytes, hipStream_t stream);

/* Log probabilities of given tokens, with entropy, rank and the top
 * alternatives of every row, from logits as a head layer's GEMM writes them:
 * with z = scale * logits (scale = 1 / temperature),
 *   logp[r] = z[t_r] - log sum_v exp(z[v]),  entropy[r] = -sum_v p_v log p_v,
 *   rank[r] = the number of logits greater than the token's,
 *   top_ids / top_logp [r][top] = the largest logits' ids and log
 *   probabilities, equal logits in the order of their ids.
 *   logits  device, [rows][ldl] of ltype (QG_O_BF16 / QG_O_F32), ldl >= vocab;
 *           any element alignment (rows on 16 bytes are faster).
 *   tokens  device int32 [rows], or NULL (then logp and rank are NULL).  A
 *           token outside 0 .. vocab - 1 has logp NaN and rank -1.
 *   stats   device fp32 [rows][2]: the largest logit and
 *           log sum_v exp(z[v] - max z), for the backward pass; logp, entropy, stats, rank, top_ids and top_logp
 *           may each be NULL (top > 0: not both of the last two).
 *   top     0 .. QG_MAX_ALTERNATIVES.
 *   ws      qg_token_logprobs_workspace_size bytes, 256-B aligned, zero-filled
 *           once (its first 64 KiB suffice) and left so; NULL when that is 0.
 * A logit of -inf is a masked token: probability 0 and never an alternative;
 * alternatives that do not exist have id -1 and log probability -inf.  A row
 * with every token masked: logp -inf, entropy 0, rank 0, stats (0, -inf).  NaN
 * or +inf logits make logp, entropy and top_logp of their row NaN; a NaN is
 * never an alternative.  vocab <= 2^24.  rows == 0 is a no-op.  Asynchronous. */
#define QG_MAX_ALTERNATIVES 32
qg_status qg_token_logprobs_workspace_size(int64_t rows, int64_t vocab, int32_t top, uint64_t *bytes);
qg_status qg_token_logprobs(const void *logits, int32_t ltype, int64_t rows, int64_t vocab, int64_t ldl,
                            const int32_t *tokens, float scale, int32_t top, float *logp, float *entropy,
                            float *stats, int32_t *rank, int32_t *top_ids, float *top_logp, void *ws,
                            uint64_t ws_bytes, hipStream_t stream);

/* Gradient of the logits from those of logp (dlogp, fp32 [rows] or NULL) and of
 * the entropy (dentropy, fp32 [rows] or NULL; entropy as the forward pass gave
 * it), with stats of the forward pass on the same logits and scale:
 *   dlogits[r][v] = scale * (dlogp (1{v = t_r} - p_v) - dentropy p_v (log p_v + entropy)).
 *   dlogits device, [rows][lddl] of ltype, lddl >= vocab; it may be the logits'
 *   own buffer (same pointer and stride).
 * Masked tokens and wholly masked rows get 0 (the token itself its dlogp); a
 * token outside the vocabulary contributes nothing.  Asynchronous. */
qg_status qg_token_logprobs_backward(const void *logits, int32_t ltype, int64_t rows, int64_t vocab, int64_t ldl,
                                     const int32_t *tokens, float scale, const float *stats, const float *entropy,
                                     const float *dlogp, const float *dentropy, void *dlogits, int64_t lddl,
                                     hipStream_t stream);

/* Root-mean-square norm of rows with the residual's addition, to bf16 and / or
 * to 8 bits with scales for the layer behind it:
 *   s = x + residual, rounded to res_type (without residual and sum: s = x),
 *   y[j] = s[j] w[j] / sqrt(mean_j(s[j]^2) + eps),
 * in fp32, y and the codes each rounded once from there.
 *   x        device, [rows][ldx] of x_type (QG_O_BF16 / QG_O_F32, a GEMM's output).
 *   residual device, [rows][ldr] of res_type, or NULL.
 *   sum      device, [rows][lds] of res_type, or NULL: s, for the next residual
 *            and for the backward pass.  It may be x's or the residual's own
 *            buffer (same pointer, stride and type).
 *   weight   device, bf16 [k].  eps > 0.
 *   y        device, bf16 [rows][ldy], or NULL.
 *   q, q_scales, q_type  the codes of y and their scales, or NULL, NULL and
 *            QG_A_BF16 (one of y and q is wanted): QG_A_INT8_TOKEN, QG_A_FP8_TOKEN,
 *            QG_A_FP8_BLOCK or QG_A_MXFP8, layouts and scales as qg_quantize_int8,
 *            qg_quantize_fp8 and qg_quantize_mxfp8 (fp32 scales are at least
 *            2^-126), of the fp32 y: the codes nearest to y times the fp32
 *            reciprocal of the scale, ties to even; [rows][ldq] bytes.
 * k % 8 == 0 (MXFP8: % 32), k <= 2^24; 16-B aligned rows (q: 8-B; a product that
 * reads it wants 16).  Outputs other than sum overlap no input.  rows == 0 is a
 * no-op.  A row with NaN, Inf or a mean square beyond fp32 gives unspecified
 * values in that row.  Asynchronous on `stream`. */
qg_status qg_rmsnorm(const void *x, int32_t x_type, int64_t ldx, const void *residual, int32_t res_type, int64_t ldr,
                     void *sum, int64_t lds, const void *weight, float eps, int64_t rows, int64_t k, void *y,
                     int64_t ldy, int32_t q_type, void *q, int64_t ldq, void *q_scales, hipStream_t stream);

/* Backward pass of qg_rmsnorm: with s as the forward pass normed it (its sum, or x
 * where there was none), r = 1 / sqrt(mean(s^2) + eps), g = dy w,
 *   dx = r (g - s r^2 mean_j(g s)) + dsum,  dw = sum over the rows of dy s r
 * (fp32, each rounded once).  dx is the gradient of x and of the residual alike.
 *   s    device, [rows][lds] of s_type.  dy device, bf16 [rows][lddy].
 *   dsum device, [rows][ldds] of s_type: the gradient that reaches s past the
 *        norm, or NULL.
 *   dx   device, [rows][lddx] of s_type, or NULL; it may be dsum's own buffer.
 *   dw   device, [k] of dw_type, 16-B aligned, or NULL; overwritten (rows == 0:
 *        zeros).
 *   ws   qg_rmsnorm_backward_workspace_size bytes (enough for fewer rows too), 256-B
 *        aligned, any contents (the first 64 KiB are left alone: it may be a product's
 *        workspace); NULL without dw.
 * Sums over the rows are in a fixed order.  Alignments and limits as above. */
qg_status qg_rmsnorm_backward_workspace_size(int64_t rows, int64_t k, uint64_t *bytes);
qg_status qg_rmsnorm_backward(const void *s, int32_t s_type, int64_t lds, const void *weight, float eps, int64_t rows,
                              int64_t k, const void *dy, int64_t lddy, const void *dsum, int64_t ldds, void *dx,
                              int64_t lddx, void *dw, int32_t dw_type, void *ws, uint64_t ws_bytes,
                              hipStream_t stream);

/* Low-rank adapters of many requests added in place to the output of a projection
 * that they share: for every row r of adapter a
 *   y[r] += scales[a] (x[r] A_a^T) B_a^T
 * (fp32 sums; the low-rank row enters the second product as two bf16 parts for a
 * bf16 y, three for an fp32 one; y is rounded once).  Rows of no adapter keep
 * their bits.
 *   x       device, bf16 [m][ldx]: the projection's input before any quantization.
 *   a, b    device, bf16 [num_adapters][rank][lda] and [num_adapters][n][ldb], lda
 *           >= k, ldb >= rank; adapters of a lower rank are padded with zeros.  x,
 *           a and b 16-B aligned, their strides multiples of 8, lda and ldb <=
 *           2^22, k % 8 == 0, rank % 8 == 0, rank <= QG_LORA_MAX_RANK, num_adapters
 *           <= 1024, m <= 2^21, n <= 2^24.
 *   scales  device, fp32 [num_adapters], or NULL: 1.
 *   sorted_rows, offsets  device, the rows grouped by adapter, as qg_moe_sort
 *           gives them for the rows' adapter ids (topk 1, num_experts =
 *           num_adapters; ids outside, such as -1, are rows of no adapter): one
 *           call serves every projection of a batch.  A row is listed once at most;
 *           entries that name no row are skipped.
 *   y       device, [m][ldy] of y_type (QG_O_BF16 / QG_O_F32), ldy >= n, any element
 *           alignment (rows on 16 bytes are faster); some columns of a fused
 *           projection are y + their first column.  It overlaps no input.
 *   ws      qg_lora_workspace_size bytes (enough for every smaller m too), 256-B
 *           aligned, any contents (the first 64 KiB are left alone: it may be a
 *           product's workspace); NULL when that size is 0.
 * m == 0 is a no-op.  A row's result does not depend on the other rows' values.
 * Asynchronous on `stream`. */
#define QG_LORA_MAX_RANK 256
qg_status qg_lora_workspace_size(int64_t m, int64_t k, int64_t n, int32_t num_adapters, int32_t rank,
                                 uint64_t *bytes);
qg_status qg_lora(const void *x, int64_t ldx, const void *a, int64_t lda, const void *b, int64_t ldb,
                  const float *scales, int32_t num_adapters, int32_t rank, const int32_t *sorted_rows,
                  const int32_t *offsets, int64_t m, int64_t k, int64_t n, void *y, int32_t y_type, int64_t ldy,
                  void *ws, uint64_t ws_bytes, hipStream_t stream);

/* Softmax cross entropy of hidden states against a head's weights, for large
 * vocabularies: the logits exist tile by tile and are never in memory.  With
 * z = scale x W^T (fp32 sums of bf16 products),
 *   lse[r] = log sum_v exp(z[r][v]),  loss[r] = lse[r] - z[r][t_r].
 *   x       device, bf16 [m][ldx]; w device, bf16 [vocab][ldw]; 16-B aligned, ld
 *           >= k, ld % 8 == 0, ld <= 2^22, k % 8 == 0; vocab <= 2^24.
 *   targets device int32 [m]; a target outside 0 .. vocab - 1 is ignored: loss 0
 *           and no gradient (its lse is that of its logits).  NULL without loss.
 *   scale   > 0: 1, or one over the temperature.
 *   loss, lse  device fp32 [m], one of them may be NULL; lse is for the backward
 *           pass.
 *   ws      qg_linear_xent_workspace_size bytes (enough for every smaller m too),
 *           256-B aligned, zero-filled once (its first 64 KiB suffice).
 * A logit of -inf is a token of probability 0 (loss +inf where it is the target).  NaN
 * in a row of x or a logit of +inf gives NaN in that row alone, nothing but -inf an lse
 * of -inf and a loss of NaN.  m == 0 is a no-op.  Sums are in a fixed order.
 * Asynchronous on `stream`. */
qg_status qg_linear_xent_workspace_size(int64_t m, int64_t k, int64_t vocab, uint64_t *bytes);
qg_status qg_linear_xent(const void *x, int64_t ldx, const void *w, int64_t ldw, int64_t m, int64_t k, int64_t vocab,
                         const int32_t *targets, float scale, float *loss, float *lse, void *ws, uint64_t ws_bytes,
                         hipStream_t stream);

/* Gradients of qg_linear_xent from that of the losses (dloss, fp32 [m]), with lse
 * of the forward pass on the same x, w and scale:
 *   d[r][v] = dloss[r] (exp(z[r][v] - lse[r]) - 1{v = t_r}),
 *   dx = scale d W,  dw = scale d^T x.
 * The vocabulary goes in pieces: d exists for one piece, in bf16 (two bf16 parts
 * for dx up to 16 and for dw up to 32 tokens; with more that rounding, 1.7e-3 of
 * the norm, is in dx and dw whatever dw_type is), relative to the largest |dloss|.
 *   dx   device, bf16 [m][lddx], 16-B aligned, lddx >= k, or NULL.
 *   dw   device, [vocab][lddw] of dw_type, 16-B aligned, lddw >= k, or NULL; it is
 *        overwritten; m == 0 fills it with zeros.
 *   ws   qg_linear_xent_backward_workspace_size bytes (enough for every smaller m
 *        too; whatever the vocabulary at most 128 MB or 16384 m for d, 80 MB or 4 m k
 *        for parts of dx, and 48 MB), 256-B aligned, zero-filled once.
 * An ignored row's dx is 0, and it adds nothing to dw as long as its x is finite.
 * Asynchronous on `stream`. */
qg_status qg_linear_xent_backward_workspace_size(int64_t m, int64_t k, int64_t vocab, uint64_t *bytes);
qg_status qg_linear_xent_backward(const void *x, int64_t ldx, const void *w, int64_t ldw, int64_t m, int64_t k,
                                  int64_t vocab, const int32_t *targets, float scale, const float *lse,
                                  const float *dloss, void *dx, int64_t lddx, void *dw, int32_t dw_type, int64_t lddw,
                                  void *ws, uint64_t ws_bytes, hipStream_t stream);

/* Measurement utilities, used for roofline calibration and cold-cache timing.
 * qg_stream_read reads `bytes` (a multiple of 16; src 16-B aligned, device)
 * with 128-bit loads and folds them into `sink` (device, at least 16 KiB, any
 * contents); nothing else is written.  Reading a buffer larger than the 256 MB
 * MALL evicts earlier data from the caches.  qg_stream_copy copies `bytes`
 * (a multiple of 16, both pointers 16-B aligned, device, non-overlapping).
 * Both are asynchronous on `stream`. */
qg_status qg_stream_read(const void *src, uint64_t bytes, void *sink, hipStream_t stream);
qg_status qg_stream_copy(void *dst, const void *src, uint64_t bytes, hipStream_t stream);

/* Name of the kernel variant the tuning table selects for `m` rows (dense) or
 * `m` pairs (MoE: the skinny kernel's variant for experts with few rows) and
 * the tile parameters, written as a NUL-terminated string into buf.
 * qg_describe_dispatch_ex does the same for the compute options `flags` of
 * qg_gemm_ex (dense layers only). */
qg_status qg_describe_dispatch(const qg_weight *w, int64_t m, char *buf, uint64_t buf_bytes);
qg_status qg_describe_dispatch_ex(const qg_weight *w, int64_t m, uint32_t flags, char *buf, uint64_t buf_bytes);

/* The MoE dispatch of qg_moe_gemm for num_tokens * topk pairs, as text:
 * which kernel serves experts by row count (the tiled kernels' row threshold,
 * the small-tile form or the skinny kernel's variant below it).  Which
 * experts fall on which side depends on the routing (device data). */
qg_status qg_describe_moe_dispatch(const qg_weight *w, int64_t num_tokens, int32_t topk, char *buf,
                                   uint64_t buf_bytes);

/* The kernels that qg_lora takes for these sizes, as text: one launch, or the two
 * with their blocks of the rank, parts of k, 16-row blocks, steps of the rank and
 * column chunks. */
qg_status qg_describe_lora(int64_t m, int64_t k, int64_t n, int32_t num_adapters, int32_t rank, int32_t y_type, char *buf,
                           uint64_t buf_bytes);

/* The shapes of the products that qg_linear_xent (the first) and
 * qg_linear_xent_backward (the others, for the pieces of the vocabulary) take, as
 * text: tile, stages in LDS and parts of the contraction. */
qg_status qg_describe_linear_xent(int64_t m, int64_t k, int64_t vocab, char *buf, uint64_t buf_bytes);

/* Static description of a status code (never NULL). */
const char *qg_status_string(qg_status status);

/* The hipError_t behind the calling thread's last QG_ERR_HIP (0 if none). */
int32_t qg_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* QG_H_ */
