/*
 * bsgg.h -- C ABI of the GB300 grouped block-scaled GEMM with fused epilogue.
 *
 * The operation (cuDNN-frontend documentation, "Grouped GEMM + Quant (SM100)",
 * Equations, Steps 1-3; "Grouped GEMM + SwiGLU (SM100)", Step 2; "Grouped GEMM
 * + sReLU (SM100)", Equations and Tanh soft clamp):
 *
 *   for every expert group g and every row m in [padded_offsets[g-1], padded_offsets[g]):
 *     C[m, n] = alpha[g] * sum_k dequant(A[m, k], SFA) * dequant(B[n, k, g], SFB)
 *             (+ bias_g[n] when a bias is given; C itself can be stored, before any
 *              clamp or activation: "Grouped GEMM + GLU + Hadamard + Quant (SM100)",
 *              Equations)
 *     D[m, j] = prob[m] * C[m, j]                                   (GATE)
 *             = gamma * prob[m] * X_b * swish(G_b)  over paired 32-col blocks (SWIGLU,
 *               N/2 outputs)
 *             = gamma * prob[m] * (X_b + 1) * G_b * sigmoid(1.702 G_b)  (GEGLU, N/2 outputs)
 *               with X_b, G_b first clamped to [-glu_limit, glu_limit] when a limit is set
 *             = prob[m] * relu(C)^2, or (s * min(tanh(relu(C)/s), 1))^2  (SRELU)
 *   and, for FP8/FP4 outputs, per block of v values of D along a row (SFD_row)
 *   and along a column (SFD_col, blocks of v rows):
 *     SFD = norm_const * max|D| / q_max  (rounded up to a power of two for UE8M0,
 *                                         to nearest for E4M3 scales)
 *     Dq  = convert_rne_satfinite(D * (norm_const / SFD))
 *   For 16/32-bit outputs, amax[g] = max |D| over the rows of group g.
 *
 * Everything runs in hand-written CUDA kernels for sm_103a (tcgen05 block-scaled
 * MMAs accumulating in tensor memory, TMA operand pipelines).  There is no CPU
 * path: every entry point that computes needs a CUDA device.
 *
 * Conventions shared by all entry points
 *  - Pointers in bsgg_args are DEVICE pointers (except in bsgg_run_host), owned
 *    by the caller, and must stay valid until the stream work completes.
 *  - All tensors are dense and C-contiguous, 16-byte aligned:
 *      A        (m_pad, K)      K-major, 1 byte per FP8 value, FP4 packed 2 per
 *                               byte (element 2i in the low nibble)
 *      B        (L, N, K)       K-major, same element encoding as A
 *      SFA      swizzled SF(m_pad, K)          (bsgg_sf_bytes(m_pad, K, v, 1) bytes)
 *      SFB      swizzled SF(N, K) per expert   (bsgg_sf_bytes(N, K, v, L) bytes)
 *      padded_offsets int32 (L), alpha float (L), prob float (m_pad),
 *      norm_const float (1)
 *      D, D_col (m_pad, N_out)  N-major; N_out = N/2 for SWIGLU/GEGLU, 2N for
 *                               the backward epilogues, else N;
 *                               bf16/f16/f32, or 1-byte FP8 codes, or packed FP4
 *      C        (m_pad, N)      N-major, bf16/f16, with MXFP8 inputs also f32 or
 *                               unscaled FP8/FP4 codes (optional pre-activation output)
 *      bias     (L, N)          N contiguous, bf16/f16/f32 (optional)
 *      SFD_row  swizzled SF(m_pad, N_out); SFD_col swizzled SF(N_out, m_pad)
 *      amax     float (L), 2L for the backward epilogues
 *    where SF(rows, cols) is the pages' (32, 4, ceil(rows/128), 4,
 *    ceil(ceil(cols/v)/4), L) layout in physical order (L, ceil(rows/128),
 *    ceil(ceil(cols/v)/4), 32, 4, 4) ("Grouped GEMM + SwiGLU (SM100)",
 *    Canonical layouts) and v is the scale-factor vector size (32 for MXFP8
 *    with UE8M0 scales, 16 for NVFP4 with E4M3 scales).  Output scale factors
 *    use the input's scale format and v ("Grouped GEMM + Quant (SM100)",
 *    Additional Type Constraints: SFA, SFB, SFD_row, SFD_col share a dtype).
 *  - Streams are passed as `void*` holding a cudaStream_t (NULL = legacy
 *    default stream).  bsgg_run and bsgg_pack_sf are asynchronous.
 *  - Errors are returned as bsgg_status; no entry point throws or aborts.
 *    Host-side validation mirrors the pages' "Support Surface and Constraints".
 *    Device-side values (padded_offsets) are checked by the kernel itself; a
 *    violation is reported through bsgg_query_device_status, and the kernel
 *    then writes no output.
 */
#ifndef BSGG_H
#define BSGG_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Every entry point below is exported with default visibility; the library is
 * compiled with hidden visibility otherwise, so that two builds of it (the
 * release and the range-checking one) can live in one process without sharing
 * any internal symbol. */
#if defined(__GNUC__)
#define BSGG_API __attribute__((visibility("default")))
#else
#define BSGG_API
#endif

typedef enum {
  BSGG_OK = 0,
  BSGG_ERR_INVALID_ARG = 1,     /* null/misaligned pointer, bad shape or enum */
  BSGG_ERR_UNSUPPORTED = 2,     /* valid on the pages but not built here */
  BSGG_ERR_CUDA = 3,            /* a CUDA runtime call failed */
  BSGG_ERR_DEVICE_TIMEOUT = 4,  /* a kernel wait ran out; the kernel returned early */
  BSGG_ERR_BAD_OFFSETS = 5,     /* padded_offsets not non-decreasing multiples of 128
                                   ending at m_pad; the kernel wrote nothing */
  BSGG_ERR_BAD_POINTERS = 6,    /* discrete weight mode: a b_ptrs / sfb_ptrs entry of a
                                   non-empty group is null or not 16-byte aligned; the
                                   kernel wrote nothing */
  BSGG_ERR_DEVICE_BOUNDS = 7    /* range-checking build only (libbsgg_debug.so): an index
                                   failed its range check; that access was skipped (see
                                   bsgg_debug_bounds_violation) */
} bsgg_status;

/* Input formats ("Grouped GEMM + Quant (SM100)", Data Types table). */
typedef enum {
  BSGG_IN_MXFP8_E4M3 = 0,  /* float8_e4m3fn data, float8_e8m0fnu scales, v = 32 */
  BSGG_IN_MXFP8_E5M2 = 1,  /* float8_e5m2 data,   float8_e8m0fnu scales, v = 32 */
  BSGG_IN_NVFP4 = 2,       /* float4_e2m1fn_x2 data, float8_e4m3fn scales, v = 16 */
  BSGG_IN_FP4_UE8M0_16 = 3,/* float4_e2m1fn_x2 data, float8_e8m0fnu scales, v = 16 */
  BSGG_IN_MXFP4 = 4,       /* float4_e2m1fn_x2 data, float8_e8m0fnu scales, v = 32 */
  BSGG_IN_BF16 = 5         /* bfloat16 A and B, no scale factors: the BF16 backend of
                              "Grouped GEMM + dGLU (SM100)" (Backend dispatch, BF16
                              contract).  Backward DSWIGLU / DGEGLU only (dGeGLU with
                              its fixed constants: dgeglu_custom = 0), BF16/F16/F32 D,
                              no D_col; K % 8 == 0; single CTAs and CTA pairs.  The
                              dGeGLU saved C is scaled by beta as well (X = beta C). */
} bsgg_in_format;

/* Output formats of D (and D_col). */
typedef enum {
  BSGG_OUT_BF16 = 0, BSGG_OUT_F16 = 1, BSGG_OUT_F32 = 2,
  BSGG_OUT_E4M3 = 3, BSGG_OUT_E5M2 = 4, BSGG_OUT_E2M1 = 5
} bsgg_out_format;

/* Epilogues: gating ("Grouped GEMM + Quant (SM100)", Step 2), SwiGLU ("Grouped GEMM +
 * SwiGLU (SM100)", Step 2), squared ReLU with optional tanh soft clamp ("Grouped GEMM +
 * sReLU (SM100)"), GeGLU ("Grouped GEMM + GLU + Hadamard + Quant (SM100)", Equations),
 * and the dSwiGLU backward ("Grouped GEMM + dGLU (SM100)", Block-scaled contract):
 *   ref = alpha_g^2 * sum_k A B;  X, G = beta_g * the saved forward C's input and gate
 *   32-column blocks;  D = [ref*prob*swish(G) | ref*prob*X*sigmoid(G)*(1 + G*(1 - sigmoid(G)))]
 *   in C's block order (width 2N);  dprob[m] += sum_n X*swish(G)*ref. */
typedef enum {
  BSGG_EPI_GATE = 0, BSGG_EPI_SWIGLU = 1, BSGG_EPI_SRELU = 2, BSGG_EPI_GEGLU = 3, BSGG_EPI_DSWIGLU = 4,
  BSGG_EPI_DGEGLU = 5,  /* dGeGLU backward (same page): the saved C unscaled (beta not read),
                           gate G clamped above at clamp_max, up U clamped to [clamp_min,
                           clamp_max]; s = sigmoid(a * Gc);
                           d gate = ref*prob*(Uc + offset)*s*(1 + a*Gc*(1 - s)) if G <= clamp_max,
                           d up = ref*prob*Gc*s if clamp_min <= U <= clamp_max, else 0;
                           dprob[m] += sum_n ref*Gc*s*(Uc + offset) */
  BSGG_EPI_DSITUGLU = 6 /* dSiTU-GLU backward (same page, Equations): the saved C unscaled;
                           T_g = b1*tanh(G/b1)*sigmoid(G), T_u = b2*tanh(U/b2);
                           d gate = ref*prob*T_u*dT_g/dG, d up = ref*prob*T_g*dT_u/dU;
                           dprob[m] += sum_n ref*T_g*T_u */
} bsgg_epilogue;

/* Problem description, fixed at plan creation (the pages' constructor +
 * check_support + compile, "Grouped GEMM + Quant (SM100)", Class API). */
typedef struct {
  int64_t m_pad;          /* rows of A/D/prob = padded_offsets[L-1]; a positive multiple
                             of 128 (a batch whose groups are all empty, m_pad = 0, is
                             refused with BSGG_ERR_INVALID_ARG: the caller skips the call,
                             and every amax of such a batch is 0) */
  int64_t n;              /* GEMM N (rows of each expert's B); multiple of 32 (64 for SWIGLU
                             and GEGLU); for DSWIGLU the compact gradient width (D is 2N wide) */
  int64_t k;              /* reduction length in elements; multiple of 16 (FP8) / 32 (FP4) */
  int32_t num_groups;     /* L, 1..1024 */
  int32_t in_format;      /* bsgg_in_format */
  int32_t out_format;     /* bsgg_out_format */
  int32_t epilogue;       /* bsgg_epilogue */
  int32_t want_col;       /* 1: also write D_col and SFD_col (quantized outputs only) */
  int32_t gate_first;     /* SWIGLU/GEGLU block order: 0 = [X_b | G_b] ("Grouped GEMM +
                             SwiGLU (SM100)", Step 2), 1 = [G_b | U_b] ("Grouped GEMM + GLU +
                             Hadamard + Quant (SM100)", Equations) */
  float tanh_clamp_s;     /* SRELU soft clamp s > 0, or 0 for none */
  int32_t tile_m;         /* rows per MMA tile: 128 (one CTA) or 256 (a pair of CTAs with
                             2-CTA instructions); 0 = library choice.  The pages' mma_tiler_mn[0]
                             ("Grouped GEMM + Quant (SM100)", Common Parameters) */
  int32_t tile_n;         /* columns per MMA tile: 128 or 256 (256 when tile_m = 256); 0 = library
                             choice.  The pages' mma_tiler_mn[1] */
  /* Thread-block cluster shape (cluster_m, cluster_n): the pages' cluster_shape_mn
     ("Grouped GEMM + Quant (SM100)", Common Parameters; Support Surface and Constraints,
     Tiling and Cluster).  Built: (1, 1) with tile_m = 128; (2, 1) with tile 256 x 256 (the
     CTA pair; tile (0, 0) with cluster (2, 1) selects it).  (0, 0) = the library's choice.
     A (2, 1) cluster of 128-row or 128-column tiles would share an operand tile between two
     CTAs by TMA multicast, which this library never issues: it returns
     BSGG_ERR_UNSUPPORTED, as do the other powers of two up to 4 that the pages allow; any
     other value returns BSGG_ERR_INVALID_ARG. */
  int32_t cluster_m;
  int32_t cluster_n;
  /* Forward epilogue options of "Grouped GEMM + GLU + Hadamard + Quant (SM100)"
     (Equations; Configuration).  All zero = none of them. */
  float glu_limit;        /* SWIGLU/GEGLU: both halves clamped to [-glu_limit, glu_limit]
                             before the activation; 0 = no clamp; must be finite, >= 0 */
  float glu_alpha;        /* SWIGLU/GEGLU: output scale gamma; 0 (unset) or 1 = none; finite */
  int32_t want_c;         /* 1: also store C = alpha_g * acc (+ bias), before any clamp or
                             activation, (m_pad, N) N-major, in c_format */
  int32_t c_format;       /* BSGG_OUT_BF16 or BSGG_OUT_F16 (when want_c); with MXFP8 inputs
                             also BSGG_OUT_F32, or BSGG_OUT_E4M3 / E5M2 / E2M1: C converted
                             with round-to-nearest-even and saturation, no scale factor */
  int32_t want_bias;      /* 1: add bias_g[n] to C; bias is (L, N), N contiguous per expert
                             (the pages' (N, L) tensor with stride (1, N)) */
  int32_t bias_format;    /* BSGG_OUT_BF16, BSGG_OUT_F16 or BSGG_OUT_F32 (when want_bias) */
  /* Discrete weight mode ("Grouped GEMM + GLU + Hadamard + Quant (SM100)", Discrete weight
     mode): 1 = each expert's B and SFB are separate allocations named by the device
     pointer arrays b_ptrs / sfb_ptrs instead of the dense b / sfb tensors (the two
     modes are mutually exclusive).  B_g is (N, K) K-major, SFB_g is SF(N, K) with one
     slice (bsgg_sf_bytes(N, K, v, 1) bytes).  The plan then owns 256 * L + 256 bytes
     of device memory for one TMA descriptor pair per expert, written by a small
     kernel on the stream before every launch. */
  int32_t discrete_b;
  /* DSWIGLU: storage type of the saved forward C, BSGG_OUT_BF16, BSGG_OUT_F16 or
     BSGG_OUT_F32 ("Grouped GEMM + dGLU (SM100)", BF16 contract: C in BF16/FP16/FP32). */
  int32_t saved_c_format;
  /* Hadamard output ("Grouped GEMM + GLU + Hadamard + Quant (SM100)", Outputs and
     Equations), forward epilogues only; H16 is the 16 x 16 Sylvester Hadamard matrix.
     1 = rowwise: RHT = (H16 / 4) x for every 16-column block x of bf16-rounded D;
         (m_pad, N_out) N-major in rht_format: BSGG_OUT_BF16, or BSGG_OUT_E2M1 (packed
         NVFP4 with E4M3 scales per 16 in SFRHT = swizzled SF(m_pad, N_out) under
         rht_norm_const, whatever the input's scale type).
     2 = colwise (rht_format BSGG_OUT_E2M1, N_out % 128 == 0): (H16 / 4) x for every
         column and every block x of 16 consecutive tokens of an expert (rows of its
         padded range, counted from its start), NVFP4 with one E4M3 scale per block;
         expert g (padded rows [start_g, end_g), expert_m = end_g - start_g) is the
         logical (N_out, expert_m) matrix, tokens contiguous, from flat element
         N_out * start_g of RHT (m_pad * N_out / 2 bytes in all), its scales the
         swizzled SF(N_out, expert_m) from byte N_out * start_g / 16 of SFRHT
         (m_pad * N_out / 16 bytes in all). */
  int32_t want_rht;
  int32_t rht_format;
  /* DGEGLU: 0 = the page's defaults (geglu_alpha 1.702, clamp [-7, 7], linear_offset 1),
     1 = the four values below (finite, clamp_min <= clamp_max). */
  int32_t dgeglu_custom;
  float dgeglu_alpha;
  float dgeglu_clamp_min;
  float dgeglu_clamp_max;
  float dgeglu_linear_offset;
  /* DSITUGLU: the tanh scales b1 (gate) and b2 (up), finite and > 0; 0 = 1. */
  float situ_beta1;
  float situ_beta2;
} bsgg_desc;

/* Tensors of one call.  Unused outputs may be NULL: d_col/sfd_col unless
 * want_col; sfd_row/sfd_col/norm_const for 16/32-bit outputs; amax for
 * quantized outputs; bias unless want_bias; c unless want_c.  amax is
 * required for BF16/F16 outputs and optional for F32 ("Grouped GEMM + Quant
 * (SM100)", Scale Factor Output Requirements); with BSGG_IN_BF16 inputs it is
 * optional, and sfa, sfb and sfb_ptrs are not read (NULL). */
typedef struct {
  const void* a;
  const void* sfa;
  const void* b;
  const void* sfb;
  const int32_t* padded_offsets;
  const float* alpha;
  const float* prob;         /* required: pass ones for no gating */
  const float* norm_const;   /* required for quantized outputs */
  void* d;
  void* d_col;
  void* sfd_row;
  void* sfd_col;
  float* amax;               /* zeroed by bsgg_run on the stream before the kernel */
  const void* bias;          /* (L, N) in bias_format; required iff want_bias */
  void* c;                   /* (m_pad, N) in c_format; required iff want_c */
  /* discrete_b only (b and sfb then NULL): device arrays of L int64 device
     addresses.  Entries of empty groups are not read by the GEMM and may be 0;
     the others must be 16-byte aligned (checked on the device: a violation is
     BSGG_ERR_BAD_POINTERS from bsgg_query_device_status, and nothing is written). */
  const int64_t* b_ptrs;
  const int64_t* sfb_ptrs;
  /* DSWIGLU, DGEGLU and DSITUGLU: the saved forward C (m_pad, 2N) N-major in saved_c_format,
     its per-group scale beta (L; DSWIGLU, and DGEGLU with BSGG_IN_BF16), and dprob
     (m_pad), which the kernel
     ACCUMULATES into:
     zero it before the call ("Grouped GEMM + dGLU (SM100)": dprob must be
     zero-initialized).  amax then holds 2L floats: [2g] over the input-gradient
     blocks, [2g + 1] over the gate-gradient blocks of group g. */
  const void* saved_c;
  const float* beta;
  float* dprob;
  /* want_rht only: the RHT output; SFRHT and rht_norm_const (1 float) for an
     NVFP4 RHT. */
  void* rht;
  void* sfrht;
  const float* rht_norm_const;
  /* Backward epilogues, optional: dbias (L, 2N) float, ACCUMULATED like dprob
     (zero it before the call): dbias[g][n] += sum over the rows of group g of
     D[m][n] before any output conversion ("Grouped GEMM + dGLU (SM100)": the
     per-expert row reduction of the interleaved D).  NULL = not computed. */
  float* dbias;
} bsgg_args;

typedef struct bsgg_plan bsgg_plan;

/* Validate `desc` and build a plan (kernel choice, launch shape, a 16-byte
 * device status word).  The plan belongs to the device that is current at
 * creation.  Returns BSGG_ERR_INVALID_ARG / BSGG_ERR_UNSUPPORTED for
 * descriptions the pages or this library reject; *plan is NULL then. */
BSGG_API bsgg_status bsgg_create(const bsgg_desc* desc, bsgg_plan** plan);

/* Enqueue one grouped GEMM on `stream` (asynchronous, no host sync, graph
 * capturable).  Checks pointers for presence and 16-byte alignment. */
BSGG_API bsgg_status bsgg_run(bsgg_plan* plan, const bsgg_args* args, void* stream);

/* End-to-end call with HOST buffers: `host` holds host pointers (pinned for
 * speed) for every input and output to move; `dev` holds device buffers of the
 * same shapes.  Inputs present in `host` are copied into `dev`, the kernel runs
 * on the `dev` buffers, outputs present in `host` are copied back, and the
 * stream is synchronized.  An input left NULL in `host` is taken as already
 * resident in `dev`.  Bytes moved are returned in *h2d_bytes / *d2h_bytes
 * (either may be NULL).  Allocates nothing.  In discrete weight mode the
 * experts' weights are taken as resident (dev->b_ptrs / dev->sfb_ptrs; host->b
 * and host->sfb must be NULL). */
BSGG_API bsgg_status bsgg_run_host(bsgg_plan* plan, const bsgg_args* host, const bsgg_args* dev,
                          void* stream, uint64_t* h2d_bytes, uint64_t* d2h_bytes);

/* bsgg_run_host without the final synchronization (the pages have no
 * counterpart): the copies in, the kernel and the copies out are enqueued on
 * `stream` and the call returns.  The host buffers (pinned, or the copies are
 * synchronous on the host side) and the device buffers must stay valid, and
 * the outputs in `host` are complete only once the stream's work has
 * finished.  Lets a caller keep several batches in flight on several streams,
 * so that one batch's outputs travel to the host while the next batch's
 * inputs travel to the device and its kernel runs; each stream in flight
 * needs its own `dev` buffers, its own output buffers in `host` and its own
 * plan (the status word is per plan).  Same arguments, byte counts and errors
 * as bsgg_run_host. */
BSGG_API bsgg_status bsgg_run_host_async(bsgg_plan* plan, const bsgg_args* host, const bsgg_args* dev,
                                void* stream, uint64_t* h2d_bytes, uint64_t* d2h_bytes);

/* Number of kernel launches one bsgg_run of this plan enqueues (the pages have
 * no counterpart): 1, or 2 in discrete weight mode (the per-expert descriptor
 * kernel, then the GEMM).  -1 for a null plan. */
BSGG_API int32_t bsgg_launches_per_run(const bsgg_plan* plan);

/* Synchronize `stream`, then read and clear the plan's device status word:
 * BSGG_OK, BSGG_ERR_DEVICE_TIMEOUT, BSGG_ERR_BAD_OFFSETS or BSGG_ERR_BAD_POINTERS
 * (a status bit the library does not define reads as BSGG_ERR_CUDA). */
BSGG_API bsgg_status bsgg_query_device_status(bsgg_plan* plan, void* stream);

/* Test hook for the failure path; the pages have no counterpart.  With enable =
 * 1, every later bsgg_run / bsgg_run_host of this plan launches a kernel whose
 * MMA thread first waits on a barrier that nothing completes, with every
 * barrier wait bounded by 50 ms instead of 2 s: each role gives up, drains its
 * in-flight work and returns, no output is complete, and the status word reads
 * BSGG_ERR_DEVICE_TIMEOUT; the CUDA context stays usable.  enable = 0 restores
 * normal launches.  Errors: BSGG_ERR_INVALID_ARG (null plan, enable not 0/1). */
BSGG_API bsgg_status bsgg_debug_force_timeout(bsgg_plan* plan, int32_t enable);

BSGG_API void bsgg_destroy(bsgg_plan* plan);
BSGG_API const char* bsgg_status_string(bsgg_status status);

/* Bytes of the swizzled SF(rows, cols) layout with L slices and vector v:
 * 512 * L * ceil(rows/128) * ceil(ceil(cols/v)/4). */
BSGG_API uint64_t bsgg_sf_bytes(int64_t rows, int64_t cols, int32_t sf_vec, int32_t num_slices);

/* Byte offset of the scale of (row, k-block, slice l) in that layout, where
 * kblocks = ceil(cols/v).  Pure host function. */
BSGG_API int64_t bsgg_sf_offset(int64_t row, int64_t kblk, int64_t l, int64_t rows, int64_t kblocks);

/* Pack row-major scale codes (L, rows, kblocks) into the swizzled layout,
 * writing every byte (padding = 0, "Grouped GEMM + SwiGLU (SM100)", JAX
 * execution: untouched SF padding is zero).  Device pointers; asynchronous. */
BSGG_API bsgg_status bsgg_pack_sf(const uint8_t* rowmajor, uint8_t* swizzled, int64_t rows,
                         int64_t kblocks, int32_t num_slices, void* stream);

/* Size of the library-owned device scratch used by bsgg_run_noalloc. */
#define BSGG_NOALLOC_SCRATCH_BYTES 256

/* Allocation-free run (the pages have no counterpart; this is a library
 * convenience).  Same computation, arguments and validation as bsgg_create +
 * bsgg_run + bsgg_destroy, but it creates no plan and never calls cudaMalloc
 * or cudaFree.  It is for callers that cannot allocate device memory at the
 * point of the call: a framework whose own pool has already reserved the
 * device memory (a raw cudaMalloc would fail or fragment it), a serving loop
 * that must not let cudaMalloc/cudaFree synchronize the device, or a plug-in
 * inside a host application that owns memory management.
 *
 * The kernel's only scratch, its device status word (16 bytes with the record a
 * range-checking build keeps behind it), lives in a file-scope static device
 * array of BSGG_NOALLOC_SCRATCH_BYTES bytes that every GPU which loads the
 * library holds until the process exits.  A call whose scratch need exceeds
 * that array is rejected with BSGG_ERR_UNSUPPORTED: the need is those 16 bytes,
 * except in discrete weight mode, whose per-expert descriptors (256 * L + 256
 * bytes) never fit, so discrete_b = 1 is rejected.
 *
 * The first call on a device looks up the array's device address with that
 * device current (cudaGetSymbolAddress) and remembers it with the id of the
 * device's context; a call that finds a different context (after
 * cudaDeviceReset, say) looks it up again.  Make the first call on a device,
 * and the first after a reset, before any stream capture.  Every call clears
 * the 16 status bytes on `stream` before its kernel.  All calls share the array, which keeps the last call's contents:
 * calls whose kernels overlap on the GPU (several streams, several host
 * threads) race on it, so run them on one stream when the status matters.
 * With wait_status != 0 the call synchronizes `stream` after the launch and
 * returns the device status as bsgg_query_device_status would (BSGG_OK,
 * BSGG_ERR_DEVICE_TIMEOUT or BSGG_ERR_BAD_OFFSETS; a status bit the library
 * does not define reads as BSGG_ERR_CUDA); with 0 it returns once the kernel
 * is enqueued. */
BSGG_API bsgg_status bsgg_run_noalloc(const bsgg_desc* desc, const bsgg_args* args, void* stream,
                             int32_t wait_status);

/* Range-checking build; the pages have no counterpart.  The library is also
 * built as libbsgg_debug.so with every TMA box origin (A rows, K offset, B row
 * and slice, scale-factor atoms), every output index (D and D_col rows and
 * columns, SFD_row / SFD_col offsets, C, the Hadamard output, dbias) and every
 * per-row / per-group read (prob, alpha) checked against the problem's extents
 * before use.  A failed check skips the access, records the first failure and
 * raises a status bit that bsgg_query_device_status returns as
 * BSGG_ERR_DEVICE_BOUNDS; a failure in the operand loads also makes every role
 * of the CTA give up and drain as after a timeout.  No trap, no fault.  The
 * release build compiles the checks away.
 *
 * bsgg_debug_bounds_checked: 1 in the range-checking build, 0 otherwise.
 * bsgg_debug_bounds_margin: test hook: later launches of the plan check rows
 *   against m_pad - rows instead of m_pad (rows: a multiple of 128 below m_pad),
 *   so that in-range accesses fail their checks without any out-of-range access
 *   being made; barrier waits are then bounded by 50 ms.  0 restores the checks.
 *   BSGG_ERR_UNSUPPORTED in the release build; BSGG_ERR_INVALID_ARG for other rows.
 * bsgg_debug_bounds_violation: the failure recorded by the last
 *   bsgg_query_device_status that returned BSGG_ERR_DEVICE_BOUNDS (site code,
 *   value, limit; all 0 if none).  Site codes: 1 A rows, 2 B n-tile, 3 B slice,
 *   4 SFA atom, 5 SFB row block, 6 K offset, 10 D row, 11 D column, 12 SFD_row,
 *   13 SFD_col, 15 C column, 16 Hadamard output, 18 dbias column, 19 group. */
BSGG_API int32_t bsgg_debug_bounds_checked(void);
BSGG_API bsgg_status bsgg_debug_bounds_margin(bsgg_plan* plan, int32_t rows);
BSGG_API bsgg_status bsgg_debug_bounds_violation(const bsgg_plan* plan, uint32_t* site, uint32_t* value, uint32_t* limit);

/* Measurement utility; the pages have no counterpart.  Measures the dense
 * block-scaled tensor-core throughput of the current device, the denominator of
 * the kernel's roofline: one CTA per SM issues `mmas_per_sm` tcgen05.mma
 * block_scale instructions (M = 128, N = tile_n, K = 32 for MXFP8 or 64 for
 * NVFP4) on operands and unit scales resident in shared memory, with no loads and
 * no epilogue, timed with CUDA events on `stream`.  Synchronizes the stream.
 * in_format: a bsgg_in_format; tile_n: 128 or 256; mmas_per_sm: 4 .. 2^22.
 * Writes TFLOP/s (2*M*N*K per instruction) to *tflops.  Allocates and frees a
 * 4-byte status word.  Errors: BSGG_ERR_INVALID_ARG for other arguments,
 * BSGG_ERR_CUDA for a failed CUDA call, BSGG_ERR_DEVICE_TIMEOUT if the final
 * wait ran out (2 s). */
BSGG_API bsgg_status bsgg_measure_mma_peak(int32_t in_format, int32_t tile_n, int64_t mmas_per_sm, double* tflops,
                                  void* stream);

/* Measurement utility; the pages have no counterpart.  The same measurement for
 * either instruction form the GEMM issues: tile_m = 128 is bsgg_measure_mma_peak
 * (cta_group::1, M = 128, one issuing CTA per SM, tile_n 128 or 256); tile_m = 256
 * is cta_group::2 with M = 256, N = 256 (tile_n must be 256): clusters of two
 * CTAs, each holding its 128 rows of A and half of B's rows, the even CTA issuing
 * `mmas` instructions for the pair, on floor(SMs / 2) pairs.  Each CTA reserves
 * 120 KB of shared memory so that every SM holds one.  TFLOP/s counts 2*M*N*K per
 * instruction.  Synchronizes the stream; allocates and frees a 4-byte status
 * word.  Errors: BSGG_ERR_INVALID_ARG for tile_m not 128 or 256 and the
 * arguments bsgg_measure_mma_peak refuses (mmas: 4 .. 2^22 per issuing thread),
 * BSGG_ERR_UNSUPPORTED for tile_m = 256 with tile_n = 128, BSGG_ERR_CUDA for a
 * failed CUDA call, BSGG_ERR_DEVICE_TIMEOUT if the final wait ran out (2 s). */
BSGG_API bsgg_status bsgg_measure_mma_peak_tile(int32_t in_format, int32_t tile_m, int32_t tile_n, int64_t mmas,
                                       double* tflops, void* stream);

/* ------------------------------------------------------------------------
 * The operators around the grouped GEMM of an expert layer (the pages start at
 * its operands; these have no counterpart there): the router's top-k, the sort
 * of tokens by expert into rows padded to 128 per expert, the quantization of
 * tokens into A and SFA, the way back to tokens, the dense layers beside the
 * experts, and their gradients.
 *
 * They hold no plan: every call is described by its desc, validated on the
 * host, enqueued on `stream` and returns (asynchronous, no allocation, graph
 * capturable).  Formats "f" below are bsgg_out_format values BSGG_OUT_BF16,
 * BSGG_OUT_F16 or BSGG_OUT_F32.  Pointers are device pointers; rows of
 * vectors are read in 16-byte pieces, so the tensors of tokens and rows need
 * 16-byte aligned bases and row pitches (BSGG_ERR_INVALID_ARG otherwise).  No
 * output may overlap an input unless its entry says so.  Sums, softmax
 * statistics and products are accumulated in 32 bits and rounded once at the
 * end; results do not depend on the order in which blocks run.
 *
 * A SLOT is one choice of one token: slot = token * topk + j.  A ROW is a row
 * of the grouped GEMM's A (and D).  row_of_slot (tokens, topk) names a slot's
 * row and slot_of_row (m_pad) a row's slot; -1 stands for a slot that is not
 * routed and for a padding row.  Entries outside the ranges count as -1. */

/* Softmax top-k router.  For a row l of logits, m = max l:
 *   ids     = the topk largest logits, largest first; equal ones by lowest index
 *   weights = exp(l_id - m) / S,  S = the sum of exp(l - m) over all experts
 *             (normalize = 0) or over the chosen ones (normalize = 1)
 * A logit of -inf is never chosen: where fewer than topk are left the id is -1
 * and its weight 0 (a row of -inf only: every id -1).  A NaN logit counts as the
 * largest and makes the row's weights NaN. */
typedef struct {
  int64_t tokens;         /* >= 0; 0 launches nothing */
  int64_t ld;             /* row pitch of logits and dlogits in elements, >= num_experts */
  int32_t num_experts;    /* 1..1024 */
  int32_t topk;           /* 1..min(32, num_experts) */
  int32_t logit_format;   /* f: logits, and dlogits of the backward */
  int32_t normalize;      /* 0 or 1 */
} bsgg_route_desc;

BSGG_API bsgg_status bsgg_route(const bsgg_route_desc* desc, const void* logits, int32_t* ids, float* weights,
                                void* stream);

/* Gradient of bsgg_route with respect to the logits, given ids and weights it
 * returned and g = dweights: inner = sum_j g_j w_j;
 *   normalize = 1: dlogits_i = w_i (g_i - inner) for the chosen i, 0 elsewhere
 *   normalize = 0: dlogits_i = p_i (g_i [i chosen] - inner), p = softmax(l)
 * dweights is (tokens, topk); with row_of_slot given (not NULL) it is instead a
 * per-row gradient of m_pad floats (the backward GEMM's dprob) and slot s reads
 * dweights[row_of_slot[s]], 0 for a slot without a row. */
BSGG_API bsgg_status bsgg_route_backward(const bsgg_route_desc* desc, const void* logits, const int32_t* ids,
                                         const float* weights, const float* dweights, const int32_t* row_of_slot,
                                         int64_t m_pad, void* dlogits, void* stream);

/* Tokens sorted by expert: slots in order of expert, then of slot (stable); each
 * expert's rows padded to a multiple of 128.  An id outside [0, num_experts)
 * is a slot without a row (-1: a masked choice; ids of another process's
 * experts).  Outputs:
 *   padded_offsets (num_experts)  end of each expert's rows; the last one is
 *                                 m_pad, as bsgg_run wants it (rows past the
 *                                 sizes' sum are padding rows of the last expert)
 *   row_of_slot (slots), slot_of_row (m_pad)
 *   prob (m_pad)                  weights[slot] of each row, 0 for padding rows
 *                                 (NULL: not wanted; weights NULL = ones)
 *   rows_used (1)                 the padded sizes' sum, the least m_pad that
 *                                 holds them (NULL: not wanted)
 * slots: 2^30 at most (BSGG_ERR_UNSUPPORTED beyond).
 * m_pad: a positive multiple of 128; bsgg_sort_rows gives one that always
 * suffices.  Where it is too small the slots that do not fit get no row, offsets
 * are cut at m_pad, and BSGG_ERR_BAD_OFFSETS is reported in `status`.
 * workspace: bsgg_sort_workspace_bytes(slots, num_experts) bytes (0: may be
 * NULL).  status: a device word (NULL: not reported) that kernels only ever OR
 * bits into; see bsgg_query_status_word. */
BSGG_API int64_t bsgg_sort_rows(int64_t slots, int32_t num_experts);
BSGG_API uint64_t bsgg_sort_workspace_bytes(int64_t slots, int32_t num_experts);
BSGG_API bsgg_status bsgg_sort_tokens(int64_t slots, int32_t num_experts, int64_t m_pad, const int32_t* ids,
                                      const float* weights, int32_t* padded_offsets, int32_t* row_of_slot,
                                      int32_t* slot_of_row, float* prob, int32_t* rows_used, void* workspace,
                                      uint32_t* status, void* stream);

/* Format of the rows that dispatch and combine_backward write: a bsgg_in_format
 * (BSGG_IN_BF16: bfloat16 values, no scale factors), or float16 values. */
#define BSGG_ROW_F16 6

/* Description of the three operators between tokens and rows. */
typedef struct {
  int64_t tokens;         /* >= 0 */
  int64_t hidden;         /* vector length; a multiple of 8, and of 16 (FP8) or 32 (FP4) for
                             those row formats */
  int64_t m_pad;          /* rows: a positive multiple of 128 */
  int64_t ld_token;       /* row pitch of x, y or dy in elements, >= hidden */
  int64_t ld_residual;    /* row pitch of the residual (combine), >= hidden; 0 without one */
  int32_t topk;           /* 1..32; tokens * topk < 2^31 */
  int32_t token_format;   /* f: x, dy; y and the residual */
  int32_t row_format;     /* dispatch, combine_backward: format of A / dD, as above */
  int32_t d_format;       /* f: D (combine, combine_backward) */
} bsgg_tokens_desc;

/* A[row] = x[token of the row], quantized to row_format with its scale
 * factors in the swizzled SF(m_pad, hidden) layout; padding rows are 0 with
 * scale 1.  Scales: UE8M0 2^ceil(log2(amax / q_max)) per 32 (16) values, E4M3
 * RN(amax / 6) per 16 for NVFP4; an all-zero block (or an E4M3 scale that rounds
 * to 0) has scale 1; codes are RNE(x / scale), saturating.  A block with an
 * infinity or a NaN gets the NaN scale (UE8M0 0xFF, E4M3 0x7F) and zero codes.
 * a: (m_pad, hidden) codes; sfa: bsgg_sf_bytes(m_pad, hidden, v, 1) bytes, every
 * one written (NULL for bfloat16 and float16 rows).  The two maps are each
 * other's inverses, as bsgg_sort_tokens writes them.  The gradient of a dispatch is
 * bsgg_combine without weights. */
BSGG_API bsgg_status bsgg_dispatch(const bsgg_tokens_desc* desc, const void* x, const int32_t* row_of_slot,
                                   const int32_t* slot_of_row, void* a, void* sfa, void* stream);

/* y[t] = residual[t] + sum_j weights[t, j] * D[row_of_slot[t, j]] over the slots
 * that have a row, j ascending.  weights (tokens, topk) float; NULL = ones
 * (where the GEMM's epilogue already multiplied by prob).  residual may be NULL
 * and may be y itself. */
BSGG_API bsgg_status bsgg_combine(const bsgg_tokens_desc* desc, const void* d, const int32_t* row_of_slot,
                                  const float* weights, const void* residual, void* y, void* stream);

/* Gradient of bsgg_combine (that of the residual is dy itself):
 *   dD[row]        = weights[slot of the row] * dy[its token], 0 for padding rows,
 *                    in row_format with scale factors as bsgg_dispatch writes them
 *   dweights[t, j] = <dy[t], D[row_of_slot[t, j]]>, 0 for a slot without a row
 * dd (and sfd) NULL: not wanted; dweights NULL: not wanted, d is then not read. */
BSGG_API bsgg_status bsgg_combine_backward(const bsgg_tokens_desc* desc, const void* dy, const void* d,
                                           const int32_t* row_of_slot, const int32_t* slot_of_row,
                                           const float* weights, void* dd, void* sfd, float* dweights,
                                           void* stream);

/* Activations of the dense layer; gelu is z * Phi(z), srelu max(z, 0)^2. */
typedef enum {
  BSGG_ACT_NONE = 0, BSGG_ACT_RELU = 1, BSGG_ACT_SRELU = 2, BSGG_ACT_SILU = 3, BSGG_ACT_GELU = 4
} bsgg_activation;

/* Dense layer: z = x W^T + bias, y = act(z) + residual.  x (m, k), W (n, k) and
 * the residual (m, n) are in in_format, bias (n) in bias_format, y (m, n) in
 * out_format, z (m, n), kept for the backward, in in_format; each rounded once
 * from the 32-bit accumulator.  Sizes are free (m = 0 launches nothing); x and W
 * are fetched by TMA: 16-byte aligned bases, pitches ldx, ldw multiples of 8.
 * The other tensors need only their element's alignment.  residual may be y. */
typedef struct {
  int64_t m, n, k;
  int64_t ldx, ldw, ld_residual, ldy, ldz;   /* row pitches in elements (0 for an absent tensor) */
  int32_t in_format;      /* BSGG_OUT_BF16 or BSGG_OUT_F16 */
  int32_t out_format;     /* f */
  int32_t bias_format;    /* f (when bias) */
  int32_t activation;     /* bsgg_activation */
} bsgg_linear_desc;

BSGG_API bsgg_status bsgg_linear(const bsgg_linear_desc* desc, const void* x, const void* w, const void* bias,
                                 const void* residual, void* y, void* z, uint32_t* status, void* stream);

/* Gradient of the dense layer: dz = dy * act'(z), dbias = sum over rows of dz,
 *   dx = dz W,   dw = dz^T x  (accumulate_dw = 1: dw += dz^T x, read and
 * rounded once).  dz is kept in in_format (its rounding enters dx and dw; dbias
 * sums the unrounded values in 32 bits) in the caller's buffer of m rows of pitch
 * ld_dz; without an activation dz is dy itself, z and dz are NULL and nothing is
 * rounded.  dx, dw and dbias (float) may each be NULL: not wanted.  dy, z, dz, x
 * and w: 16-byte aligned bases, pitches multiples of 8.  The gradient of the
 * residual is dy. */
typedef struct {
  int64_t m, n, k;
  int64_t ld_dy, ldz, ld_dz, ldx, ldw, ld_dx, ld_dw;
  int32_t in_format;      /* BSGG_OUT_BF16 or BSGG_OUT_F16: dy, z, dz, x, w */
  int32_t dx_format;      /* f */
  int32_t dw_format;      /* f */
  int32_t activation;
  int32_t accumulate_dw;  /* 0 or 1 */
} bsgg_linear_bwd_desc;

BSGG_API bsgg_status bsgg_linear_backward(const bsgg_linear_bwd_desc* desc, const void* dy, const void* x,
                                          const void* w, const void* z, void* dz, void* dx, void* dw,
                                          float* dbias, uint32_t* status, void* stream);

/* Synchronize `stream`, then read a status word that the operators above were
 * given and clear what was read (a report that a kernel on another stream makes
 * meanwhile stays for the next call): BSGG_OK, BSGG_ERR_BAD_OFFSETS (m_pad too
 * small for the sort), BSGG_ERR_DEVICE_TIMEOUT (a wait of bsgg_linear ran out; its
 * outputs are incomplete), or BSGG_ERR_CUDA. */
BSGG_API bsgg_status bsgg_query_status_word(uint32_t* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BSGG_H */
