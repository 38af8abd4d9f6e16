/*
 * w4a16.h - C ABI of the W4A16 fused dequantize-GEMM library for MI355X (gfx950).
 *
 * Operation ("4.3 Weight-only INT4", section 1, W4A16 storage and compute; section 4,
 * Marlin): y[M,N] = x[M,K] * W_hat[K,N], where W_hat is rebuilt on-chip from 4-bit codes
 * and per-group metadata, multiplied with 16-bit activations, accumulated in fp32.
 * K is the reduction axis (input features), N the output features.
 *
 *   affine:  W_hat[k,n] = RN_t((q[k,n] - z[k/g,n]) * s[k/g,n])     (one rounding)
 *   NF4:     W_hat[k,n] = RN_t(c[q[k,n]] * a[k/64,n])
 *
 * with t the activation type (fp16 or bf16), RN round-to-nearest-even, q the 4-bit code,
 * s the group scale, z the 4-bit zero-point (8 when qzeros is NULL: symmetric codes
 * -8..7 stored offset-binary), c a 16-entry fp16 codebook and a an fp16 absmax.
 *
 * Canonical input formats ("INT4 and Low-Bit Inference", section 6-9, packed layout):
 *   qweight  int32 [K/8][N]     eight codes along K per word, code j in bits 4j..4j+3
 *   scales   t     [K/g][N]     one scale per group of g consecutive k, per column
 *   qzeros   int32 [K/g][N/8]   eight zero-points along N per word, same nibble order
 *
 * Conventions for every entry point
 *   - All tensor pointers are DEVICE pointers owned by the caller. The library never
 *     allocates, frees or synchronizes; all work is enqueued on `stream` (a hipStream_t;
 *     NULL = the null stream) and is complete only when the caller synchronizes it.
 *   - Arrays are dense and row-major. x, out and the packed weight need 16-byte aligned
 *     base addresses; scales 2-byte; qzeros 4-byte.
 *   - Arguments are checked on the host before anything is enqueued. A bad argument
 *     returns W4A16_ERR_ARG, a shape the kernels do not implement W4A16_ERR_UNSUPPORTED;
 *     nothing is launched in either case. A failed launch returns W4A16_ERR_HIP.
 *     Faults during execution surface at the caller's next synchronization.
 *   - There is no slow or CPU fallback path.
 *   - The only global state is a per-device cache of the compute-unit count. Calls on
 *     different streams may run concurrently if they use distinct workspaces.
 *
 * Supported shapes: K % 32 == 0, K % group_size == 0, N % 16 == 0, M >= 0, K, N > 0,
 * group_size in {32, 64, 128}; K * N < 2^34 (packed weight below 8 GiB).
 */
#ifndef W4A16_H
#define W4A16_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* W4A16_E4M3: 8-bit floating point codes (OCP e4m3: largest 448, no infinities), one a byte, with
 * scales of their own; only the calls that name it take it. */
typedef enum { W4A16_F16 = 0, W4A16_BF16 = 1, W4A16_F32 = 2, W4A16_E4M3 = 3 } w4a16_dtype;

typedef enum {
  W4A16_OK = 0,
  W4A16_ERR_ARG = 1,          /* null pointer, misalignment, inconsistent shape or dtype */
  W4A16_ERR_UNSUPPORTED = 2,  /* well-formed but not implemented (e.g. N % 16 != 0)    */
  W4A16_ERR_HIP = 3,          /* the HIP runtime rejected a launch                       */
  W4A16_ERR_WORKSPACE = 4     /* workspace missing, misaligned or smaller than required  */
} w4a16_status;

/* Bytes of the device-layout weight for a K x N matrix: K_pad * N / 2 with
 * K_pad = K rounded up to a multiple of 128. Returns 0 for unsupported shapes. */
size_t w4a16_packed_bytes(int K, int N);

/* Load-time re-layout of the weight codes ("INT4 and Low-Bit Inference", section 5,
 * Marlin's tricks: weights are re-ordered once at load so run-time unpacking is
 * branch-free and reads are coalesced; "4.3 Weight-only INT4", section 4).
 *   qweight   [in]  canonical int32 [K/8][N]
 *   packed    [out] w4a16_packed_bytes(K, N) bytes; an opaque order private to this
 *                   library, read only by the GEMM and dequant entry points below.
 * Must not alias qweight. */
w4a16_status w4a16_pack(const int32_t* qweight, int K, int N, int32_t* packed, void* stream);

/* Bytes of scratch device memory w4a16_gemm / w4a16_gemm_nf4 need for this shape on the
 * current device: zero for the decode kernel (M <= 16, see w4a16_gemm); for the batched kernel
 * zero unless it splits K across workgroups, then the fp32 partial tiles of the K slices
 * (summed in slice order by a second kernel on the same stream). The caller allocates it;
 * it needs no initialization and holds nothing between calls. Calls that may run
 * concurrently (different streams) need distinct workspaces. Returns 0 for bad shapes. */
size_t w4a16_workspace_bytes(int M, int K, int N, int group_size);

/* The W4A16 GEMM with affine (asymmetric) or symmetric INT4 weights.
 *   x         [in]  act [M][K], act = W4A16_F16 or W4A16_BF16
 *   packed    [in]  output of w4a16_pack for this K, N
 *   scales    [in]  act [K/group_size][N]
 *   qzeros    [in]  int32 [K/group_size][N/8], or NULL for symmetric codes (zero 8)
 *   out       [out] out_dtype [M][N], out_dtype = act or W4A16_F32
 *   workspace [in/out] >= w4a16_workspace_bytes(M, K, N, group_size) bytes, 256-byte
 *                   aligned (may be NULL when that size is 0)
 * M = 0 is a no-op. Results are deterministic: partial sums are combined in a fixed
 * order, never with floating-point atomics. Three kernels share the work, chosen by shape
 * (w4a16_kernel_name names the one a shape gets): the memory-bound decode kernel for up to 16
 * rows (and up to 32 on weights with K * N < 2^24, one launch per 16 rows); the skinny kernel
 * (K split across the waves of one workgroup) for about 4..256 rows on weights at most 8192
 * deep whose 64-column workgroups fill the chip in one to four launch rounds; the batched MFMA
 * kernel for the other shapes past 16 rows, and for 12..16 rows on weights with K * N >= 2^27
 * deeper than 8192 whose activations do not fit the decode kernel's LDS staging. */
w4a16_status w4a16_gemm(const void* x, int M, int K, int N, w4a16_dtype act,
                        const int32_t* packed, const void* scales, const int32_t* qzeros,
                        int group_size, void* out, w4a16_dtype out_dtype, void* workspace,
                        size_t workspace_bytes, void* stream);

/* The W4A16 GEMM with NF4 weights ("INT4 and Low-Bit Inference", section 5, The formats;
 * "INT4", section INT4, FP4, and NF4 are not identical).
 *   absmax    [in]  fp16 [K/block_size][N] per-block absmax scales
 *   codebook  [in]  16 fp16 values (device memory), code i -> codebook[i]
 *   block_size      32, 64 or 128
 * Other arguments as for w4a16_gemm. */
w4a16_status w4a16_gemm_nf4(const void* x, int M, int K, int N, w4a16_dtype act,
                            const int32_t* packed, const uint16_t* absmax,
                            const uint16_t* codebook, int block_size, void* out,
                            w4a16_dtype out_dtype, void* workspace, size_t workspace_bytes,
                            void* stream);

/* The fused gate+up projection of a gated MLP with its SwiGLU epilogue: the kernels form
 * g = x W_gate and u = x W_up in fp32 and store only h = SiLU(g) * u = g / (1 + exp(-g)) * u
 * (the pages' next step after the linear layer, "4.3 Weight-only INT4", closing section:
 * operator fusion; the MLP is the Llama one whose shapes the pages' decode examples use).
 *   packed, scales, qzeros  the (K, N2) weight holding W_gate in columns [0, N2/2) and W_up
 *                   in [N2/2, N2), packed and laid out exactly as for w4a16_gemm
 *   out       [out] out_dtype [M][N2/2]
 *   workspace       >= w4a16_workspace_bytes(M, K, N2, group_size) bytes (as for w4a16_gemm)
 * N2 must be a multiple of 32 (W4A16_ERR_UNSUPPORTED otherwise). Other arguments, errors and
 * determinism as for w4a16_gemm; one launch per call for M <= 16 (two with a K split). */
w4a16_status w4a16_gemm_swiglu(const void* x, int M, int K, int N2, w4a16_dtype act,
                               const int32_t* packed, const void* scales, const int32_t* qzeros,
                               int group_size, void* out, w4a16_dtype out_dtype, void* workspace,
                               size_t workspace_bytes, void* stream);

/* Maximum scratch of w4a16_gemm_static, in bytes (a static device array on each GPU). */
#define W4A16_STATIC_SCRATCH_BYTES (64u << 20)

/* w4a16_gemm for callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc): the same kernels and results as
 * w4a16_gemm, bit for bit, with the split-K scratch taken from a file-scope device array of
 * W4A16_STATIC_SCRATCH_BYTES per GPU instead of a workspace argument. The array is held by
 * each GPU the library runs on until the process ends; the first call on a device looks up
 * its address (hipGetSymbolAddress). The call allocates and frees nothing.
 *   Arguments, checks and errors as for w4a16_gemm, plus W4A16_ERR_WORKSPACE when the shape
 *   needs more scratch than W4A16_STATIC_SCRATCH_BYTES (w4a16_workspace_bytes gives the
 *   need), and W4A16_ERR_HIP when the array's address cannot be obtained.
 * Every call on one GPU shares that GPU's array and the array keeps the last call's partial
 * sums; nothing in it needs to start at zero (each call writes every partial it reads). Calls
 * whose executions overlap on one GPU (different streams, or concurrent host threads) race
 * on it and give wrong results: serialize them, or use w4a16_gemm with one workspace each. */
w4a16_status w4a16_gemm_static(const void* x, int M, int K, int N, w4a16_dtype act,
                               const int32_t* packed, const void* scales, const int32_t* qzeros,
                               int group_size, void* out, w4a16_dtype out_dtype, void* stream);

/* Bytes of scratch device memory w4a16_gemm_awq needs for this shape on the current device:
 * as w4a16_workspace_bytes, plus room for the scaled activations where they are formed by a
 * pre-pass: M * K * 2 bytes (256-byte multiples) for decode shapes (M <= 16) whose
 * activations do not fit the kernel's LDS staging, and for batched shapes on the 128 x 512
 * tile. Returns 0 for bad shapes. */
size_t w4a16_awq_workspace_bytes(int M, int K, int N, int group_size);

/* The W4A16 GEMM of AWQ-scaled activations ("4.3 Weight-only INT4", section 3.2: the weight
 * is deployed as the regular INT4 format of S W, and the product is Y_hat = (X S^-1) D(Q(S W))
 * with S = diag(s) one factor per input channel):
 *   y = x' @ W_hat,  x'[m][k] = RN_act(x[m][k] * s_inv[k])
 * one round-to-nearest-even of the exact product of two act values, formed as x is staged
 * for the MFMAs (decode shapes whose x does not fit in LDS, and batched shapes on the
 * 128 x 512 tile: by a first small kernel into the workspace).
 *   s_inv     [in]  act [K], the per-input-channel S^-1, 16-byte aligned
 *   workspace [in/out] >= w4a16_awq_workspace_bytes(M, K, N, group_size) bytes, 256-byte
 *                   aligned (may be NULL when that size is 0)
 * Other arguments, errors and determinism as for w4a16_gemm (s_inv NULL with M > 0, or
 * misaligned: W4A16_ERR_ARG). */
w4a16_status w4a16_gemm_awq(const void* x, const void* s_inv, int M, int K, int N,
                            w4a16_dtype act, const int32_t* packed, const void* scales,
                            const int32_t* qzeros, int group_size, void* out,
                            w4a16_dtype out_dtype, void* workspace, size_t workspace_bytes,
                            void* stream);

/* Bytes of scratch device memory w4a16_gemm_w4a8 needs on the current device: the INT8
 * activations (M * K), their scales and code sums (M * 4 each), and, when the shape's output
 * tiles leave compute units idle and K is split into S slices, the slices' int32 sums
 * (S * M * N * 4); each part 256-byte aligned. 0 for M = 0 or bad shapes. */
size_t w4a16_w4a8_workspace_bytes(int M, int K, int N);

/* Name of the W4A8 GEMM configuration a shape gets ("w4a8_64x256", "w4a8_128x512", with
 * "_splitk" when K is split); "none" for bad shapes. */
const char* w4a16_w4a8_kernel_name(int M, int K, int N);

/* W4A8: INT4 weights with per-token INT8 activations on the integer MFMA ("INT4 LLMs: What
 * 4-Bit Quantization Means…", weight-only section: [-8, 7] weights unpacked to INT8, an
 * INT8 x INT8 product, the result dequantized with the input and per-channel scales; "INT8 vs
 * INT4 Quantization, in depth", section "Two regimes": past the crossover only the math rate
 * counts).
 *   y[m][n] = sx[m] * sw[n] * sum_k xq[m][k] * (u[k][n] - 8)
 *   sx[m] = RN_f32(max_k |x[m][k]| / 127),  xq = clip(rint(RN_f32(x / sx)), -127, 127)
 * The integer sum is exact; the epilogue multiplies it by the two scales in fp32. With K split,
 * the slices' int32 sums are added exactly by a second kernel before the same epilogue, so the
 * result does not depend on the split.
 *   x         [in]  act [M][K], finite (quantized per row by a first kernel into the workspace)
 *   packed    [in]  output of w4a16_pack of symmetric codes (u = q + 8, as for w4a16_gemm with
 *                   qzeros = NULL)
 *   wscale    [in]  act [N], one scale per output channel
 *   out       [out] out_dtype [M][N], out_dtype = act or W4A16_F32
 *   workspace [in/out] >= w4a16_w4a8_workspace_bytes(M, K, N), 256-byte aligned
 * K % 32 == 0 (else W4A16_ERR_UNSUPPORTED); other arguments and errors as for w4a16_gemm. */
w4a16_status w4a16_gemm_w4a8(const void* x, int M, int K, int N, w4a16_dtype act,
                             const int32_t* packed, const void* wscale, void* out,
                             w4a16_dtype out_dtype, void* workspace, size_t workspace_bytes,
                             void* stream);

/* Test hook: the per-token INT8 quantization w4a16_gemm_w4a8 applies, in k order.
 *   xq [out] int8 [M][K] (8-byte aligned), sx [out] float [M]. K % 8 == 0. */
w4a16_status w4a16_quantize_act_int8(const void* x, int M, int K, w4a16_dtype act, int8_t* xq,
                                     float* sx, void* stream);

/* NF4 counterpart of w4a16_gemm_swiglu (absmax [K/block_size][N2] fp16, codebook as for
 * w4a16_gemm_nf4). */
w4a16_status w4a16_gemm_nf4_swiglu(const void* x, int M, int K, int N2, w4a16_dtype act,
                                   const int32_t* packed, const uint16_t* absmax,
                                   const uint16_t* codebook, int block_size, void* out,
                                   w4a16_dtype out_dtype, void* workspace, size_t workspace_bytes,
                                   void* stream);

/* Test hook: write W_hat[K][N] (row-major, in `wdtype` = F16 or BF16) using the same
 * device dequantization routine the GEMM kernels use where they form W_hat (the batched
 * kernel, and the decode kernel for bf16 activations and NF4). The fp16 affine decode
 * kernel multiplies the exact integers (q - z) and applies s to the fp32 sum of each
 * group, which skips W_hat's rounding to fp16: its result differs from the rounded-W_hat
 * product by rounding noise only, within the 1e-3 bound. scales are in wdtype. */
w4a16_status w4a16_dequant(const int32_t* packed, const void* scales, const int32_t* qzeros,
                           int K, int N, int group_size, w4a16_dtype wdtype, void* w_out,
                           void* stream);

/* Test hook: NF4 counterpart of w4a16_dequant (absmax and codebook are fp16). */
w4a16_status w4a16_dequant_nf4(const int32_t* packed, const uint16_t* absmax,
                               const uint16_t* codebook, int K, int N, int block_size,
                               w4a16_dtype wdtype, void* w_out, void* stream);

/* ------------------------------------------------------------------------------------------
 * Routed operators: rows of one batch that go to different weights.
 *
 * A slot i = t * topk + j is choice j of token t; ids[i] is its group (an expert, or with topk 1
 * a request's adapter). A group outside [0, groups) is none: the slot's row is zeros where rows
 * are written, and adds nothing where rows come back. S = tokens * topk.
 * Limits: 1 <= topk, 1 <= groups <= W4A16_MAX_GROUPS, S <= W4A16_MAX_SLOTS, and what one launch
 * can hold (2^32 threads: about 2^24 tokens or 2^26 kilobytes of a token's rows; rows of at most
 * 2^31 - 2048 elements): W4A16_ERR_UNSUPPORTED past them. tokens = 0 is a no-op for every call
 * but w4a16_route, whose plan then holds zero offsets.
 * ------------------------------------------------------------------------------------------ */
#define W4A16_MAX_GROUPS 1024
#define W4A16_MAX_SLOTS (1 << 26)

/* Bytes of a plan for this many tokens, choices and groups; 0 for bad arguments. */
size_t w4a16_route_bytes(int tokens, int topk, int groups);

/* The plan of a batch: its slots sorted by group (a stable sort), as int32 words in `plan`:
 *   offsets [groups + 1]  at word 0: group e's sorted rows are [offsets[e], offsets[e + 1])
 *   order   [S]           at word r(groups + 1): the slot of each sorted row; the slots of no
 *                         group come last, in rows [offsets[groups], S)
 *   slot    [tokens][topk] at word r(groups + 1) + r(S): the sorted row of each slot, or -1
 * with r(n) = n rounded up to a multiple of 64; the words after them are private to the
 * library. The plan depends on the ids only: calls on any number of tensors may share it.
 *   ids   [in]  int32 [tokens][topk], 4-byte aligned
 *   plan  [out] >= w4a16_route_bytes(tokens, topk, groups) bytes, 256-byte aligned */
w4a16_status w4a16_route(const int32_t* ids, int tokens, int topk, int groups, int32_t* plan,
                         size_t plan_bytes, void* stream);

/* Rows into sorted order: xs[p] = x[order[p] / topk], zeros in the rows of no group.
 *   x   [in]  dtype [tokens][width], any dtype, element-aligned (as are all rows below)
 *   xs  [out] dtype [S][width]; must not overlap x
 * The plan's tokens, topk and groups must be those it was made with (for every call below). */
w4a16_status w4a16_dispatch(const void* x, const int32_t* plan, int tokens, int topk, int groups,
                            int width, w4a16_dtype dtype, void* xs, void* stream);

/* Gradient of w4a16_dispatch: dx[t] = sum_j dxs[slot[t][j]], summed in fp32, j ascending. */
w4a16_status w4a16_dispatch_backward(const void* dxs, const int32_t* plan, int tokens, int topk,
                                     int groups, int width, w4a16_dtype dtype, void* dx, void* stream);

/* Sorted rows back to their tokens, weighted: y[t] = sum_j weights[t][j] ys[slot[t][j]], summed
 * in fp32, j ascending, rounded once.
 *   ys      [in]  dtype [S][width];  weights [in] float [tokens][topk], 4-byte aligned
 *   y       [out] out_dtype [tokens][width], out_dtype = dtype, or any type for fp32 ys;
 *           must not overlap an input */
w4a16_status w4a16_combine(const void* ys, const int32_t* plan, int tokens, int topk, int groups,
                           const float* weights, int width, w4a16_dtype dtype, void* y,
                           w4a16_dtype out_dtype, void* stream);

/* Gradients of w4a16_combine: dys[slot[t][j]] = weights[t][j] dy[t] (zeros in the rows of no
 * group) and dweights[t][j] = sum_n dy[t][n] ys[slot[t][j]][n] in fp32 (0 for a slot of no
 * group).
 *   dy [in] dtype [tokens][width], ys [in] dtype [S][width], dys [out] dtype [S][width],
 *   dweights [out] float [tokens][topk]; neither may overlap an input */
w4a16_status w4a16_combine_backward(const void* dy, const void* ys, const int32_t* plan, int tokens,
                                    int topk, int groups, const float* weights, int width,
                                    w4a16_dtype dtype, void* dys, float* dweights, void* stream);

/* The W4A16 GEMM of sorted rows with their groups' weights: out[p] = row(p) * W_hat[e] for the
 * rows p of group e, zeros for the rows of no group.
 *   x       [in]  act [tokens][K] with gather != 0: row(p) = x[order[p] / topk], read in place
 *                 (tokens * K * 2 < 2^31, else W4A16_ERR_UNSUPPORTED); else act [S][K]: row(p) = x[p]
 *   packed  [in]  w4a16_packed_bytes(K, N) bytes a group, one after another
 *   scales  [in]  act [groups][K/group_size][N]
 *   qzeros  [in]  int32 [groups][K/group_size][N/8], or NULL for symmetric codes
 *   out     [out] out_dtype [S][N]; must not overlap an input
 * swiglu != 0: each weight is a fused gate+up projection (as for w4a16_gemm_swiglu, N % 32 == 0)
 * and out is [S][N/2]. Other arguments, errors and determinism as for w4a16_gemm. */
w4a16_status w4a16_gemm_grouped(const void* x, const int32_t* plan, int tokens, int topk, int groups,
                                int gather, int K, int N, w4a16_dtype act, const int32_t* packed,
                                const void* scales, const int32_t* qzeros, int group_size, int swiglu,
                                void* out, w4a16_dtype out_dtype, void* stream);

/* NF4 counterpart of w4a16_gemm_grouped: absmax fp16 [groups][K/block_size][N], one codebook. */
w4a16_status w4a16_gemm_grouped_nf4(const void* x, const int32_t* plan, int tokens, int topk, int groups,
                                    int gather, int K, int N, w4a16_dtype act, const int32_t* packed,
                                    const uint16_t* absmax, const uint16_t* codebook, int block_size,
                                    int swiglu, void* out, w4a16_dtype out_dtype, void* stream);

/* Name of the kernel w4a16_gemm_grouped launches for S = tokens * topk rows over this many
 * groups (static string; "none" for bad shapes). */
const char* w4a16_grouped_kernel_name(int S, int K, int N, int groups, int group_size);

/* Bytes of scratch w4a16_lora_add needs on the current device (`planned`: with a plan given);
 * 0 for bad shapes. */
size_t w4a16_lora_workspace_bytes(int M, int K, int N, int adapters, int rank, int planned);

/* Low-rank adapters of many requests beside a projection all rows share:
 *   out[m] = y[m] + scaling[a] (x[m] A[a]^T) B[a]^T, a = ids[m]; out[m] = y[m] where a is none
 * for any shared projection y = x W (w4a16_gemm, NF4, AWQ, ...). t = x A^T is summed in fp32 and
 * enters the second product as a sum of 16-bit parts: bf16 with 16 significant bits of each t
 * (24 where y is fp32), fp16 to 2^-22 of each t or 2^-25 of the row's largest |t|, whichever is
 * more. out is rounded once.
 *   x        [in]  act [M][K], act = W4A16_F16 or W4A16_BF16; K % 32 == 0
 *   y        [in]  y_dtype [M][N], y_dtype = act or W4A16_F32; N % 16 == 0
 *   lora_a   [in]  act [adapters][rank][K];  lora_b [in] act [adapters][N][rank]
 *                  rank a multiple of 8 up to 256 (W4A16_ERR_UNSUPPORTED otherwise; smaller
 *                  adapters are padded with zeros); adapters <= W4A16_MAX_GROUPS
 *   ids      [in]  int32 [M], each row's adapter; read only where plan is NULL
 *   scaling  [in]  float [adapters]
 *   plan     [in]  of w4a16_route(ids, M, 1, adapters), for calls that share it; or NULL
 *   out      [out] y_dtype [M][N]; may be y (then rows of no adapter are left alone), must not
 *                  overlap an input otherwise
 *   workspace [in/out] >= w4a16_lora_workspace_bytes(...), 256-byte aligned
 * x, y, out, lora_a and lora_b need 16-byte alignment. M = 0 is a no-op. Deterministic. */
w4a16_status w4a16_lora_add(const void* x, const void* y, int M, int K, int N, w4a16_dtype act,
                            w4a16_dtype y_dtype, const void* lora_a, const void* lora_b, int adapters,
                            int rank, const int32_t* ids, const float* scaling, const int32_t* plan,
                            void* out, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------------------------
 * 8-bit floating point operators: e4m3 codes with one fp32 scale for each 128 values along the
 * product's depth (activations and gradients), or for each block of 128 x 128 (weights).
 *
 *   scale = max(RN_f32(max |v| / 448), 2^-126)      code = RN_e4m3(RN_f32(v / scale))
 *
 * over the group's values (the last group of a row, column or weight may be short): two correctly
 * rounded fp32 steps and one rounding to 8 bits, ties to even. A group of zeros has the least scale
 * and zero codes. A group that holds an infinity or a NaN has a NaN scale and NaN codes, so that
 * every result it enters is NaN.
 * Products: the codes' products of a block of 128 k are summed on the matrix cores, the block's sum
 * is multiplied by its two scales and added to the result in fp32, which is rounded once. The two scales
 * are multiplied first: where their product passes 2^128 a block's part is infinite or NaN, and under
 * 2^-126 it loses bits. SiLU(g) is 0 where exp(-g) passes 2^128 (g under -88.7). Results are deterministic. A block's sum is an fp32 one for fp32 results, for h that leaves as codes and in
 * the kernels w4a16_fp8_16 and w4a16_fp8_32. For other 16-bit results it comes from the 8-bit MFMA,
 * which drops product bits about 17 below the block's largest: the sum is off by at most 2^-10 of its
 * largest product, on normal operands 1.5e-5 of the result, an eighth of what rounding to fp16 costs.
 * Limits, else W4A16_ERR_UNSUPPORTED: a product's depth is a multiple of 16; operands whose
 * offsets 31 bits hold (K < 2^23; rows * K / 32 < 2^31; a SwiGLU weight below 2 GiB a group);
 * up to 2^30 columns of a result; launches of fewer than 2^32 threads: of rows that are quantized
 * ceil(rows / 8) * ceil(K / 512) < 2^24, of columns and blocks fewer than 2^24 tiles of 128 x 128, and where
 * a second kernel adds slices of k or quantizes h, rows * ceil(columns / 512) < 2^25.
 * Codes, 16-bit x and dy need 16-byte alignment, other arrays that of their elements (outputs of
 * products 16 bytes).
 * ------------------------------------------------------------------------------------------ */

/* Rows to codes, for the operand of a product of depth K: one scale for 128 values of a row.
 *   x       [in]  dtype [M][K], K % 16 == 0
 *   codes   [out] [M][K]
 *   scales  [out] float [ceil(K/128)][M] */
w4a16_status w4a16_quantize_fp8(const void* x, int M, int K, w4a16_dtype dtype, uint8_t* codes,
                                float* scales, void* stream);

/* Columns to codes, transposed, for an operand whose depth is the rows (a weight's gradient): one
 * scale for 128 values of a column.
 *   x       [in]  dtype [M][K], element-aligned
 *   codes   [out] [K][M rounded up to a multiple of 16], zeros past M; 16-byte aligned
 *   scales  [out] float [ceil(M/128)][K] */
w4a16_status w4a16_quantize_fp8_columns(const void* x, int M, int K, w4a16_dtype dtype, uint8_t* codes,
                                        float* scales, void* stream);

/* A weight to codes: one scale for a block of 128 x 128.
 *   w        [in]  dtype [N][K], element-aligned
 *   codes    [out] [N][K];  scales [out] float [ceil(N/128)][ceil(K/128)]
 *   codes_t, scales_t [out] the same transposed ([K][N] and [ceil(K/128)][ceil(N/128)]), the weight
 *                    that gradients are multiplied with; both or neither may be NULL */
w4a16_status w4a16_quantize_fp8_weight(const void* w, int N, int K, w4a16_dtype dtype, uint8_t* codes,
                                       float* scales, uint8_t* codes_t, float* scales_t, void* stream);

/* Bytes of scratch w4a16_gemm_fp8 needs on the current device: the codes and scales of a 16-bit x
 * (M * K and about M * K / 32 bytes; none for one or two rows that the kernel quantizes by itself),
 * fp32 sums of every slice where the depth is cut, and for e4m3 out of shapes whose kernel cannot
 * quantize it h in fp32. 0 for M = 0 or bad shapes. */
size_t w4a16_fp8_workspace_bytes(int M, int K, int N, w4a16_dtype x_dtype, int swiglu,
                                 w4a16_dtype out_dtype);

/* y = x W^T for 8-bit weights.
 *   x         [in]  [M][K]: F16 or BF16 (quantized first, or by the kernel), or E4M3
 *                   codes with x_scales, as w4a16_quantize_fp8 writes them (NULL for 16-bit x)
 *   codes     [in]  [N][K], one row an output feature;  scales [in] float [ceil(N/128)][ceil(K/128)]
 *   out       [out] out_dtype [M][N]: x's 16-bit type or F32; any of F16, BF16, F32 for E4M3 x
 * swiglu != 0: the weight is a fused gate+up projection, gate rows first (N % 2 == 0), each half
 * with blocks of its own (scales [2 ceil(N/256)][ceil(K/128)]: for N % 256 == 0 those of the whole),
 * and out is h = SiLU(g) u, [M][N/2]; out_dtype E4M3 then gives h as codes with out_scales (float
 * [ceil(N/256)][M], N % 32 == 0), quantized from the fp32 h as w4a16_quantize_fp8 does.
 *   workspace [in/out] >= w4a16_fp8_workspace_bytes(...), 256-byte aligned (may be NULL when 0)
 * M = 0 is a no-op. out must not overlap an input. */
w4a16_status w4a16_gemm_fp8(const void* x, w4a16_dtype x_dtype, const float* x_scales, int M, int K, int N,
                            const uint8_t* codes, const float* scales, int swiglu, void* out,
                            w4a16_dtype out_dtype, float* out_scales, void* workspace,
                            size_t workspace_bytes, void* stream);

/* Name of the kernel w4a16_gemm_fp8 launches for the product's 16-bit result ("none" for bad shapes). */
const char* w4a16_fp8_kernel_name(int M, int K, int N, int swiglu);

/* w4a16_gemm_fp8 of a plan's sorted rows with their groups' weights (codes [groups][N][K], scales
 * [groups][...], as there); the rows of no group are zeros (E4M3 out: zero codes, least scales).
 *   x, gather as for w4a16_gemm_grouped: the tokens' rows (tokens * K < 2^31) or the sorted rows;
 *             x_scales has as many rows as x
 *   out       [S][N] or [S][N/2], out_scales [ceil(N/256)][S] */
size_t w4a16_fp8_grouped_workspace_bytes(int tokens, int topk, int groups, int gather, int K, int N,
                                         w4a16_dtype x_dtype, int swiglu, w4a16_dtype out_dtype);
w4a16_status w4a16_gemm_fp8_grouped(const void* x, w4a16_dtype x_dtype, const float* x_scales,
                                    const int32_t* plan, int tokens, int topk, int groups, int gather, int K,
                                    int N, const uint8_t* codes, const float* scales, int swiglu, void* out,
                                    w4a16_dtype out_dtype, float* out_scales, void* workspace,
                                    size_t workspace_bytes, void* stream);

/* Gradients of y = x W^T: dx = dy W, with dy quantized by rows, and dw = dy^T x, with both quantized
 * by columns (each call quantizes them anew; dy is read once for both).
 *   dy       [in]  act [M][N], x [in] act [M][K]; N % 16 == 0, K % 16 == 0
 *   codes_t, scales_t [in] the transposed weight's [K][N] and float [ceil(K/128)][ceil(N/128)]
 *   dx       [out] act [M][K], or NULL;  dw [out] float [N][K], or NULL (x is read for dw alone,
 *                  codes_t and scales_t for dx alone)
 *   workspace [in/out] >= w4a16_fp8_backward_workspace_bytes(...) whichever are asked for, 256-byte
 *                  aligned: dy's row codes, both operands' column codes, and slices' sums
 * M = 0: dw is cleared. */
size_t w4a16_fp8_backward_workspace_bytes(int M, int K, int N);
w4a16_status w4a16_gemm_fp8_backward(const void* dy, const void* x, int M, int K, int N, w4a16_dtype act,
                                     const uint8_t* codes_t, const float* scales_t, void* dx, float* dw,
                                     void* workspace, size_t workspace_bytes, void* stream);

/* The same for sorted rows (dy [S][N], x [S][K]) and their groups' weights: dx [S][K] has zeros in the
 * rows of no group, dw [groups][N][K] zeros for a group of no rows. For dw a group's rows are cut in
 * 128s from its first one. */
size_t w4a16_fp8_grouped_backward_workspace_bytes(int tokens, int topk, int groups, int K, int N);
w4a16_status w4a16_gemm_fp8_grouped_backward(const void* dy, const void* x, const int32_t* plan, int tokens,
                                             int topk, int groups, int K, int N, w4a16_dtype act,
                                             const uint8_t* codes_t, const float* scales_t, void* dx,
                                             float* dw, void* workspace, size_t workspace_bytes,
                                             void* stream);

/* Name of the kernel w4a16_gemm / w4a16_gemm_nf4 launch for this shape (static string),
 * so a caller can log which path ran ("4.3 Weight-only INT4", section 4.1). */
const char* w4a16_kernel_name(int M, int K, int N, int group_size);

/* Static description of a status code. */
const char* w4a16_status_string(w4a16_status status);

/* Measurement hook, not part of the GEMM path: the device's practical HBM read ceiling, for
 * reporting beside the published peak. Reads every 16-byte chunk of buf[0, bytes) once, each
 * wave streaming a contiguous run with the 16-byte non-temporal loads the GEMM kernels use for
 * the packed codes, and XORs folds of the words into the sink words (so no load is dead code):
 * afterwards the XOR of the 256 sink words has changed by the XOR of all words of buf.
 *   buf   [in]     device buffer, 16-byte aligned; bytes a multiple of 16 (0: no-op)
 *   sink  [in/out] 256 device uint32 words, 4-byte aligned
 * Bad arguments return W4A16_ERR_ARG before anything is launched. */
w4a16_status w4a16_read_probe(const void* buf, size_t bytes, uint32_t* sink, void* stream);

/* Library version string. */
const char* w4a16_version(void);

#ifdef __cplusplus
}
#endif

#endif /* W4A16_H */
