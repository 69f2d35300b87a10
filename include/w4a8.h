/*
 * w4a8.h — C ABI of the MI355X (gfx950) W4A8 linear layer.
 *
 * The operation is the W4A8 GEMM of QServe/QoQ (page "[Feature] Support
 * W4A8KV4 Quantization(QServe/QoQ)", quoted abstract): 4-bit weights reached
 * by a progressive (two-level) quantization, 8-bit per-token activations, an
 * 8-bit integer matrix product, and no dequantization of partial sums.
 * The pages give no formula; this library implements the reading below.
 *
 *   level 1 (per output row n):  s1[n] = fp16(absmax_k |W[n,k]| / 119),
 *                                W8 = clamp(rint(W * fp32(1/s1)), -119, 119)
 *   level 2 (per group of g k):  s2 = max(1, ceil((hi-lo)/15)) in [1,16],
 *                                z = rne(-lo/s2) in [0,15], with lo/hi the
 *                                group's min/max widened to include 0,
 *                                q = clamp(rne(W8/s2) + z, 0, 15)
 *   decode (in the GEMM):        W8^ = (q - z) * s2, always inside int8
 *   per-channel mode (g = K):    s1[n] = fp16((hi-lo)/15) over the row, q and z
 *                                per row, s2 = 1
 *   activations (per token m):   s_a[m] = fp16(absmax_k |A[m,k]| / 127),
 *                                A8 = clamp(rint(A * fp32(1/s_a)), -127, 127)
 *   GEMM:                        acc[m,n] = sum_k A8[m,k] * W8^[n,k]  (int32, exact)
 *                                Y[m,n]   = fp16(acc * s_a[m] * s1[n])  (fp32 math)
 *
 * Conventions for every entry point
 *   - All matrices are row-major.  W is N x K (output x input, as a linear
 *     layer stores it), A is M x K, Y is M x N.
 *   - fp16 values are passed as raw IEEE binary16 bit patterns (uint16_t).
 *   - Pointers named *_dev are device (HBM) pointers; all others are host.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).
 *     GPU entry points only enqueue work: they do not synchronize, allocate,
 *     free, or keep state between calls.  The caller owns every buffer.  They
 *     launch on the current device, which must be the buffers' and the stream's.
 *   - Arguments are validated on the host before any HIP call.  A rejected
 *     call returns an error status and touches no memory.  A failed kernel
 *     launch returns W4A8_ERR_DEVICE; faults inside a kernel surface at the
 *     caller's next synchronization, as usual for HIP.
 *   - No entry point throws.
 */
#ifndef W4A8_H
#define W4A8_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  W4A8_OK = 0,
  W4A8_ERR_INVALID_ARGUMENT = 1,   /* null pointer, negative size, ld too small, misaligned */
  W4A8_ERR_UNSUPPORTED = 2,        /* shape or group size outside what the kernels handle */
  W4A8_ERR_BUFFER_TOO_SMALL = 3,   /* blob or workspace smaller than required */
  W4A8_ERR_NONFINITE = 4,          /* w4a8_pack: a weight is NaN or infinite */
  W4A8_ERR_RANGE = 5,              /* w4a8_pack: a scale overflows fp16 */
  W4A8_ERR_LAYOUT = 6,             /* blob header magic/version/shape mismatch */
  W4A8_ERR_DEVICE = 7              /* a HIP call failed */
} w4a8_status;

/* Group-size value that selects per-channel mode (one scale and zero per row). */
#define W4A8_GROUP_PER_CHANNEL 0

/* Group-size value that selects the non-uniform codebook mode (the
 * LUT-quantized, NormalFloat-style weights of the FLUTE page): per row the
 * level-1 int8 quantization (fp16 s1), then each int8 value replaced by the
 * code of the nearest of 16 fixed int8 levels (ties to the lower code):
 *   -119 -84 -65 -50 -37 -26 -15 -5 5 15 26 37 50 65 84 119
 * (standard-normal quantiles at (i + 1/2)/16 scaled to 119).  W8^ = level[q];
 * the decode is a register table lookup.  No groups, no meta section. */
#define W4A8_CODEBOOK_NF 1

/* Shape limits.  K must be a multiple of W4A8_K_QUANTUM, N of W4A8_N_QUANTUM;
 * K <= W4A8_K_MAX keeps every int32 accumulator exact (127*128*K < 2^31).
 * g must be 32, 64 or 128 (and divide K), W4A8_GROUP_PER_CHANNEL (or K), or
 * W4A8_CODEBOOK_NF. */
#define W4A8_K_QUANTUM 128
#define W4A8_N_QUANTUM 16
#define W4A8_K_MAX 131072

/* Upper bounds on the other sizes, so that every launch's grid and every
 * index fits its integer type: tokens m <= W4A8_M_MAX (and output columns
 * n <= W4A8_N_MAX) in every entry point, and rows of at most
 * W4A8_ACT_K_MAX values in the activation quantizers.  Larger sizes are
 * rejected (INVALID_ARGUMENT for m and the quantizers' k, UNSUPPORTED for n). */
#define W4A8_M_MAX (1 << 22)
#define W4A8_N_MAX (1 << 22)
#define W4A8_ACT_K_MAX (1 << 30)

/* Upper bound on the row strides of the activations the GEMM entry points
 * read (lda8 of the int8 A8, lda of the fp16 A), in elements.  The tiled
 * kernels address a 256-row activation tile through one buffer descriptor
 * with a 32-bit range; larger strides are rejected with INVALID_ARGUMENT. */
#define W4A8_LD_MAX (1 << 22)

const char* w4a8_status_string(w4a8_status s);

/* Text of the HIP error behind the most recent W4A8_ERR_DEVICE returned to
 * the calling thread ("no error" if there was none).  Static storage. */
const char* w4a8_last_device_error(void);

/* ------------------------------------------------------------------ packing
 * Packed weight blob ("layout v1").  A 256-byte header (magic, version, n, k,
 * g) is followed by three sections at offsets that depend only on (n, k, g):
 *   q     N*K/2 bytes: uint4 codes in the gfx950 register order.  For output
 *         column tile t (16 rows of W) and k-block b (128 k), 1 KiB holds, for
 *         lane l = 0..63, 16 bytes covering row 16t + (l % 16) and
 *         k = 128b + 64h + 16(l / 16) + j  (h = 0,1; j = 0..15): dword 2h
 *         holds j = 0..7, dword 2h+1 holds j = 8..15, and within a dword
 *         byte i carries j = i (low nibble) and j = i + 4 (high nibble).
 *   meta  N*G4 bytes, G4 = (groups per row) rounded up to a multiple of 4:
 *         row n holds one byte per group (low nibble z, high nibble s2 - 1)
 *         at n*G4 + group; padding bytes are 0.  Per-channel mode: 1 group.
 *         Codebook mode: empty (the header holds the 16 levels at byte 56).
 *   s1    N fp16 row scales.
 * The blob is position independent: copy it verbatim to device memory and
 * pass that copy to w4a8_gemm.  Device code never reads the header.       */

/* Bytes of the blob for (n, k, g); 0 if the shape is unsupported.  (The
 * blob layout above; the quantization it stores is w4a8_pack's.) */
size_t w4a8_packed_size(int n, int k, int g);

/* Quantize W (n x k fp32, row stride ldw >= k elements) and write the blob.
 * Defining passages: the progressive quantization of the QServe/QoQ abstract
 * (read as: weights first to int8 per output channel, then to 4 bits per
 * group, so that dequantization in the W4A8 GEMM is cheap integer work), and
 * the offline weight reordering of the same abstract (compute-aware
 * reordering), the QUICK abstract (interleaving that skips the shared-memory
 * write-back after dequantization) and the FLUTE page ("方法详解"): the codes
 * are stored in the order the matrix-core operand wants them, so the kernel
 * never rearranges them through shared memory.
 * Host only, synchronous, thread-safe.  n_threads <= 0 uses all hardware
 * threads; the output bytes do not depend on the thread count.
 * Errors: INVALID_ARGUMENT, UNSUPPORTED, BUFFER_TOO_SMALL, NONFINITE, RANGE. */
w4a8_status w4a8_pack(const float* w, int n, int k, int ldw, int g,
                      void* blob, size_t blob_bytes, int n_threads);

/* Read (n, k, g) from a blob header (g is reported as W4A8_GROUP_PER_CHANNEL
 * in per-channel mode).  Errors: INVALID_ARGUMENT, LAYOUT. */
w4a8_status w4a8_blob_info(const void* blob, size_t blob_bytes,
                           int* n, int* k, int* g);

/* Decode a host blob back to logical arrays (for checking): q[n*k] codes,
 * z[n*G] and s2[n*G] per group (G = k/g, or 1 per channel, or 0 in codebook
 * mode: nothing written), s1[n] fp16 bits.  Any output pointer may be NULL
 * to skip it.  Errors: INVALID_ARGUMENT, LAYOUT. */
w4a8_status w4a8_unpack(const void* blob, size_t blob_bytes,
                        uint8_t* q, uint8_t* z, uint8_t* s2, uint16_t* s1);

/* ----------------------------------------------------- activation quantizer
 * Per-token int8 quantization of A (m x k fp16, row stride lda elements) into
 * a8_dev (m x k int8, row stride lda8 bytes) and s_a_dev (m fp16 scales).
 * Defining passages: the 8-bit activations of the QServe/QoQ abstract, with
 * the per-token dynamic scale that the PrefixQuant page ("Key Findings")
 * names as the usual practice.
 * m == 0 is a no-op.  k is any size from 1 to W4A8_ACT_K_MAX.  NaN/inf inputs give
 * unspecified outputs (no device-side check).
 * Errors: INVALID_ARGUMENT (null pointer, m < 0, k <= 0, lda < k, lda8 < k,
 * m > W4A8_M_MAX, k > W4A8_ACT_K_MAX), DEVICE. */
w4a8_status w4a8_quant_act(const uint16_t* a_dev, int m, int k, int lda,
                           int8_t* a8_dev, int lda8, uint16_t* s_a_dev,
                           void* stream);

/* Static per-tensor variant (the static alternative to per-token scaling on
 * the PrefixQuant page, "Key Findings"): one fp16 scale for the whole tensor,
 * fixed ahead of time, so no reduction runs.
 *   A8 = clamp(rint(A * fp32(1 / scale)), +-127)  (0 when scale == 0)
 *   s_a_dev[m] = scale for every row, so w4a8_gemm consumes it unchanged.
 * scale_f16 is the fp16 bit pattern of a finite value >= 0.  Layouts as for
 * w4a8_quant_act.  Errors: INVALID_ARGUMENT (as w4a8_quant_act, or a negative,
 * infinite or NaN scale), DEVICE. */
w4a8_status w4a8_quant_act_static(const uint16_t* a_dev, int m, int k, int lda,
                                  uint16_t scale_f16, int8_t* a8_dev, int lda8,
                                  uint16_t* s_a_dev, void* stream);

/* -------------------------------------------------------------- W4A8 GEMM
 * Y = fp16(s_a[m] * s1[n] * sum_k A8[m,k] * W8^[n,k]) with int32 accumulation.
 * Defining passages: the QServe/QoQ abstract (the int8 product runs on the
 * matrix cores and no partial sum is dequantized), and the LiquidGEMM page
 * ("Метод": each 4-bit weight is decoded to int8 in registers by a few
 * integer instructions that cannot overflow, feeding the int8 MMA directly).
 * Small M streams the weights (the FLUTE page's small-batch regime, abstract:
 * moving weights from global memory dominates); large M is bound by the
 * int8 matrix cores, the regime of the kernel speedups the LiquidGEMM page
 * reports ("Результаты").
 *   a8_dev    m x k int8, row stride lda8 bytes (k <= lda8 <= W4A8_LD_MAX,
 *             lda8 % 16 == 0, 16-byte aligned)
 *   s_a_dev   m fp16 per-token scales
 *   blob_dev  device copy of a w4a8_pack blob for (n, k, g)
 *   y_dev     m x n fp16 output, row stride ldy elements (ldy >= n)
 *   acc_dev   optional (may be NULL): m x n int32 raw accumulators, row
 *             stride ldacc elements (ldacc >= n)
 *   workspace_dev / workspace_bytes: 16-byte aligned device scratch of at
 *             least w4a8_gemm_workspace_size(m, n, k, g, opts) bytes (the
 *             same opts); may be NULL when that size is 0.  Owned by the
 *             caller; it needs no initialisation, the call overwrites it,
 *             and two calls in flight at once need two workspaces.
 *   opts      NULL for the automatic choice; otherwise forces the kernel
 *             variant and its split of K (tests and sweeps only).  Results
 *             are identical for every choice: integer partial sums are
 *             added exactly.
 * m == 0 is a no-op.  Errors: INVALID_ARGUMENT, UNSUPPORTED (k % 128, n % 16,
 * k > W4A8_K_MAX, bad g), BUFFER_TOO_SMALL, DEVICE. */
typedef struct {
  int variant;   /* 0 auto, 1 skinny (intra-workgroup split-K), 2 tiled;
                    w4a8_linear only: 3 fused quantization + skinny */
  int k_split;   /* skinny: waves that split K inside a workgroup (1..8);
                    tiled: wave groups that split the k-blocks inside a
                    workgroup (1, or 2: m_tiles x n_tiles 8 x 4 or 4 x 4
                    with 2 stages, 8 x 2 with 2-3, 4 x 2 with 2-4);
                    0 = auto */
  int n_tiles;   /* 16-column tiles per wave: skinny 1, 2 or 4; tiled 2 or 4; 0 = auto */
  int m_tiles;   /* tiled: 16-row tiles per wave (4 or 8), 0 = auto */
  int stages;    /* tiled: LDS pipeline stages, 0 = auto; four-wave tiles
                    (m_tiles x n_tiles) 8 x 4: 2-4, 4 x 4: 2-5, 8 x 2: 2-6,
                    4 x 2: 2, 3, 4, 6 or 8; eight-wave tiles as below */
  int row_groups;/* tiled: waves along M per workgroup: 1 (4 waves) or 2
                    (8 waves, 256 x 256 tiles, m_tiles 8 and 3 stages only),
                    0 = auto */
  int slices;    /* tiled: workgroups that split K of one tile (1..16), their
                    int32 partial sums going through the workspace, which
                    must then hold slices * m * n * 4 bytes; 0 = auto */
  int workgroups;/* w4a8_linear's fused kernel: workgroups of its persistent
                    grid, each walking column-tile groups (1 .. the number of
                    groups; larger values are clamped), 0 = auto */
} w4a8_gemm_opts;

/* Workspace bytes w4a8_gemm needs for these arguments (0 when it needs none,
 * or when the shape is not supported).  Host only, no HIP call. */
size_t w4a8_gemm_workspace_size(int m, int n, int k, int g, const w4a8_gemm_opts* opts);

w4a8_status w4a8_gemm(const int8_t* a8_dev, int lda8, const uint16_t* s_a_dev,
                      int m, const void* blob_dev, int n, int k, int g,
                      uint16_t* y_dev, int ldy, int32_t* acc_dev, int ldacc,
                      void* workspace_dev, size_t workspace_bytes,
                      const w4a8_gemm_opts* opts, void* stream);

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): w4a8_gemm
 * with no workspace argument.  When the plan splits K over workgroups, the
 * int32 partial sums go to one static device array of W4A8_SCRATCH_BYTES
 * that the library holds on each GPU it runs on until the process ends;
 * nothing is allocated or freed by the call.
 *   - Arguments and results are as for w4a8_gemm (bit-identical outputs).
 *   - The automatic plan narrows its K split until the partial sums
 *     (slices * m * n * 4 bytes) fit the array; a split forced through
 *     opts->slices that does not fit returns W4A8_ERR_BUFFER_TOO_SMALL.
 *   - Every call on one GPU shares that GPU's array, which keeps the last
 *     call's contents (nothing in it needs to start at zero).  Calls that
 *     overlap in time on one GPU (other streams, other threads) race on it:
 *     order them on one stream.
 *   - The first call on each device looks the array's address up
 *     (hipGetSymbolAddress, a host-side query); make that first call
 *     outside stream capture.
 * m == 0 is a no-op.  Errors as w4a8_gemm. */
#define W4A8_SCRATCH_BYTES (64u << 20)
w4a8_status w4a8_gemm_noalloc(const int8_t* a8_dev, int lda8, const uint16_t* s_a_dev,
                              int m, const void* blob_dev, int n, int k, int g,
                              uint16_t* y_dev, int ldy, int32_t* acc_dev, int ldacc,
                              const w4a8_gemm_opts* opts, void* stream);

/* ------------------------------------------------------------ whole layer
 * The W4A8 linear layer from fp16 activations: per-token quantization of A
 * (as w4a8_quant_act) followed by the GEMM (as w4a8_gemm), with A8 and s_a
 * written to a8_dev / s_a_dev as well.  Defining passage: the W4A8 layer of
 * the QServe/QoQ abstract, 8-bit activations included; fusing the
 * quantization into the small-M GEMM is this library's choice (it saves a
 * launch where the whole GEMM takes a few microseconds).  For up to 57344 activations
 * (m * k; e.g. up to 14 tokens at k = 4096, 4 at k = 14336), or 65536 on
 * layers of at least 16384 columns, both steps run in one kernel:
 * each workgroup of a persistent grid quantizes the rows itself while its
 * first weight loads are in flight, then walks several column tiles, which
 * saves a launch and a round trip of A8 through memory; otherwise it makes
 * the two calls in order on `stream`.  (opts->variant = 3 forces the fused
 * kernel for up to 16 tokens, when m rounded up to a power of two times the
 * 128-k blocks of each wave's K range is at most 64, each wave's range at
 * most 16 blocks; opts->workgroups sets its grid.)
 * Outputs are bit-identical either way (Y to the last bit: the same int32
 * sums, scales and epilogue).
 *   a_dev     m x k fp16, row stride lda elements (k <= lda <= W4A8_LD_MAX,
 *             lda % 8 == 0, 16-byte aligned)
 *   a8_dev, s_a_dev   outputs, as w4a8_quant_act (k <= lda8 <= W4A8_LD_MAX,
 *             lda8 % 16 == 0, 16-byte aligned)
 *   other arguments as w4a8_gemm; opts->variant may also be 3 to force the
 *   fused kernel (UNSUPPORTED where it does not apply); the workspace is the
 *   one w4a8_gemm_workspace_size gives for the same arguments.
 * m == 0 is a no-op.  Errors as w4a8_gemm. */
w4a8_status w4a8_linear(const uint16_t* a_dev, int lda, int m, int k,
                        const void* blob_dev, int n, int g, uint16_t* y_dev, int ldy,
                        int8_t* a8_dev, int lda8, uint16_t* s_a_dev,
                        int32_t* acc_dev, int ldacc, void* workspace_dev,
                        size_t workspace_bytes, const w4a8_gemm_opts* opts, void* stream);

/* ----------------------------------------------------- W4A16 comparison
 * The weight-only baseline the pages measure W4A8 against (the AWQ-style
 * W4A16 of the QServe/QoQ abstract, the mixed-precision kernels of the QUICK
 * abstract, FLUTE's weight-only GEMM), here on the same blob:
 * fp16 activations times the fp16 weights W16^[n,k] = fp16(s1[n] * W8^[n,k])
 * (one rounding), summed in fp32 on the fp16 MFMA:
 *   Y[m,n] = fp16(sum_k A[m,k] * W16^[n,k])
 * There is no activation quantization and no s_a.
 *   a_dev   m x k fp16, row stride lda elements (k <= lda <= W4A8_LD_MAX,
 *           lda % 8 == 0, 16-byte aligned); y_dev m x n fp16, row stride
 *           ldy >= n.
 *   opts    NULL for the automatic choice (the skinny kernel up to 64
 *           tokens, and up to 128 where the tiled grid would hold fewer than
 *           128 tiles; the tiled one above); variant 1 forces the skinny
 *           kernel (m <= 128; n_tiles / k_split as for the skinny W4A8
 *           kernel), variant 2 the tiled kernel (256 x 128 tiles, any m).
 * Results are within the fp32 summation bound of the exact sum, not
 * bit-exact across choices.  The codebook mode is not supported.
 * Errors: INVALID_ARGUMENT, UNSUPPORTED (shape, codebook blob, variant 1
 * with m > 128), DEVICE. */
w4a8_status w4a16_gemm(const uint16_t* a_dev, int lda, int m, int k,
                       const void* blob_dev, int n, int g, uint16_t* y_dev, int ldy,
                       const w4a8_gemm_opts* opts, void* stream);

/* Kernel launches w4a8_linear makes for these arguments: 1 (fused), 2
 * (quantizer + GEMM) or 3 (quantizer + GEMM split over K + reduction); 0 if
 * the call would be rejected.  Host only, no HIP call. */
int w4a8_linear_launches(int m, int n, int k, int g, const w4a8_gemm_opts* opts);

/* --------------------------------------------- int8 inputs of the linears
 * Two operators of a decoder layer that produce a linear layer's int8 input
 * directly, so that no fp16 copy of it is written: their a8 / s_a go to
 * w4a8_gemm as they are.  Values are taken in fp32 from the fp16 inputs and
 * quantized per token as in w4a8_quant_act:
 *   s_a[m] = fp16(max_k |y[m,k]| / 127),
 *   A8 = clamp(rint(y * fp32(1/s_a)), -127, 127)   (0 where s_a == 0)
 * Rows of any k from 1 to W4A8_ACT_K_MAX and any row strides >= k; rows whose
 * pointers are 16-byte aligned (a8: 8), with strides and k multiples of 8,
 * take 16-byte loads.  m == 0 is a no-op. */

/* Root-mean-square norm with the residual's addition:
 *   h = fp16(x + residual)                (h = x without a residual)
 *   y = h * weight / sqrt(mean_k(h^2) + eps)
 *   residual_dev  m x k fp16, or NULL
 *   weight_dev    k fp16
 *   h_dev         m x k fp16, the new residual stream: required with a
 *                 residual, optional (may be NULL, then not written) without.
 *                 It may be x_dev or residual_dev (same stride).
 * The norm is taken of the rounded h, the value the next layer's residual
 * addition reads.  A row whose h holds a NaN or an infinity gets s_a = NaN, so
 * that what the linear makes of it is NaN as well (its codes are
 * unspecified); a non-finite weight gives unspecified outputs.
 * Errors: INVALID_ARGUMENT (null pointer, m < 0, k <= 0, a stride < k, eps
 * negative or not finite, a residual without h_dev, m > W4A8_M_MAX,
 * k > W4A8_ACT_K_MAX), DEVICE. */
w4a8_status w4a8_rms_norm_quant(const uint16_t* x_dev, int ldx,
                                const uint16_t* residual_dev, int ldr,
                                const uint16_t* weight_dev, float eps, int m, int k,
                                uint16_t* h_dev, int ldh, int8_t* a8_dev, int lda8,
                                uint16_t* s_a_dev, void* stream);

/* The gated activation in front of the down projection:
 *   y = gate / (1 + exp(-gate)) * up
 * gate_dev and up_dev are m x k fp16 with strides of their own, so the two
 * halves of one gate-and-up output serve as they are (up_dev = gate_dev + k,
 * both strides 2k).  A row with a NaN (or infinity * 0) in y gets s_a = NaN.
 * Errors: INVALID_ARGUMENT (null pointer, m < 0, k <= 0, a stride < k,
 * m > W4A8_M_MAX, k > W4A8_ACT_K_MAX), DEVICE. */
w4a8_status w4a8_silu_mul_quant(const uint16_t* gate_dev, int ldg,
                                const uint16_t* up_dev, int ldu, int m, int k,
                                int8_t* a8_dev, int lda8, uint16_t* s_a_dev,
                                void* stream);

/* ---------------------------------------------------- paged int8 KV cache
 * Keys and values of past tokens in pages of page_size token slots, int8
 * with one fp16 scale for each (page, keys or values, kv head):
 *   data   [num_pages][2][kv_heads][page_size][head_dim] int8 (0: keys,
 *          1: values), pages page_stride bytes apart
 *   scale  [num_pages][2][kv_heads] fp16, pages scale_stride values apart
 * A value is code * scale; scales are not negative (a negative one gives
 * unspecified results).  Strides larger than a page let the layers of a model
 * share one allocation.  The pool needs no initialisation.
 *
 * A batch of sequences with new tokens is described by
 *   block_table  [batch][block_table_ld] int32: entry (b, i) is the page that
 *                holds positions [i * page_size, (i + 1) * page_size) of
 *                sequence b; the first max_pages entries of a row count
 *   seq_lens     [batch] int32: tokens of each sequence with its new ones
 *   cu_q         [batch + 1] int32: sequence b's new tokens are the rows
 *                [cu_q[b], cu_q[b + 1]) of q, k, v and of the outputs, the
 *                last at position seq_lens[b] - 1; cu_q[0] = 0, ascending,
 *                cu_q[batch] = total_q.  NULL: one new token each
 *                (total_q == batch).
 * These tables are read on the device when the kernels run.  Whatever they
 * hold, nothing outside the pool and the rows is read or written: lengths are
 * clamped to max_pages * page_size, offsets to total_q, page numbers outside
 * [0, num_pages) count as absent (nothing is written there, its keys are not
 * seen).  Apart from absent pages such contents give unspecified results. */
#define W4A8_HEAD_DIM_MAX 256
#define W4A8_HEADS_MAX 4096
typedef struct {
  int8_t* data_dev;            /* 16-byte aligned */
  uint16_t* scale_dev;
  long long page_stride;       /* bytes, a multiple of 16, >= 2 * kv_heads * page_size * head_dim */
  long long scale_stride;      /* fp16 values, >= 2 * kv_heads */
  int num_pages;
  int page_size;               /* 16, 32, 64, ... 1024 */
  int kv_heads;
  int head_dim;                /* a multiple of 16 up to W4A8_HEAD_DIM_MAX */
  const int32_t* block_table_dev;
  int block_table_ld;          /* >= max_pages */
  int max_pages;               /* max_pages * page_size < 2^31 - page_size */
  const int32_t* seq_lens_dev;
  const int32_t* cu_q_dev;     /* may be NULL */
  int batch;
  int total_q;
} w4a8_kv_view;

/* Rotary positions on the new tokens' queries and keys, and their keys and
 * values appended to the cache, in one launch.
 *   pair (a, b) at angle index i:  (a cos - b sin, b cos + a sin)
 *   half layout         a = x[i], b = x[i + rotary_dim / 2]
 *   interleaved layout  a = x[2i], b = x[2i + 1]
 * with cos = cos_sin[pos][i], sin = cos_sin[pos][rotary_dim / 2 + i], so that
 * any frequencies and long-context scalings are the table's; values from
 * rotary_dim on stay as they are.
 *   q_dev, k_dev, v_dev   rows of q_heads * head_dim and kv_heads * head_dim
 *                fp16, strides of their own (the parts of one QKV output)
 *   cos_sin_dev  [max_pos][rotary_dim] fp32, 16-byte aligned; positions beyond
 *                max_pos - 1 take its last row.  May be NULL if rotary_dim is 0.
 *   rotary_dim   a multiple of 16 from 0 to head_dim
 *   q_out_dev    rotated queries, fp16; may be q_dev (same stride)
 * Rotation and quantization are fp32 on the fp16 inputs: keys are rounded
 * once, to int8.  For every (page, keys or values, kv head) that gets new
 * tokens, with s the scale it has, if slots before the first new one are in
 * use, else 0:
 *   s' = max(s, fp16(amax of the new values / 127))
 *   old codes (only if s' > s): rint(code * fp32(s / s'))
 *   new codes: clamp(rint(v * fp32(1 / s')), -127, 127)   (0 where s' == 0)
 * so a page's scale grows with its tokens, and each time it does the codes
 * before are off by at most half a step more.  A NaN or infinity among the new
 * values makes the block's scale NaN or infinite, and what is read from it NaN.
 * No page may be written by two sequences of one call.
 * Rows are 16-byte aligned with strides a multiple of 8.  batch or total_q
 * of 0 is a no-op.
 * Errors: INVALID_ARGUMENT (null or misaligned pointer, stride too small, bad
 * size), UNSUPPORTED (head_dim, page_size, rotary_dim, more than
 * W4A8_HEADS_MAX heads, more work than one launch holds), DEVICE. */
w4a8_status w4a8_rope_append(const uint16_t* q_dev, int ldq, const uint16_t* k_dev, int ldk,
                             const uint16_t* v_dev, int ldv, int q_heads,
                             const float* cos_sin_dev, int rotary_dim, int max_pos,
                             int interleaved, const w4a8_kv_view* view,
                             uint16_t* q_out_dev, int ldqo, void* stream);

/* Attention of the new tokens' queries over the cache (which holds the new
 * tokens already: w4a8_rope_append first):
 *   o = sum_t softmax_t(scale * q . k_t) v_t
 * over the positions t <= pos of the sequence (its query's own position),
 * and t > pos - window where window > 0.  Query head h reads kv head
 * h / (q_heads / kv_heads).  A row that sees no key is 0; one that sees a key
 * and whose query holds a NaN or an infinity is NaN.
 *   q_dev, out_dev  rows of q_heads * head_dim fp16, 16-byte aligned, strides
 *                   a multiple of 8
 *   max_q, max_len  the most new tokens of one sequence and the longest
 *                   sequence the caller expects (its host-side bounds): they
 *                   choose the kernel, the split of long sequences and so the
 *                   workspace.  Results stay right where the device's tables
 *                   hold more, only slower.
 *   workspace_dev   16-byte aligned, w4a8_paged_attention_workspace_size(view,
 *                   q_heads, max_q, max_len) bytes (host only; pointers in the view
 *                   are only checked for null); may be NULL when that is 0.
 *                   No initialisation; calls in flight at once need one each.
 * Scores, softmax statistics and sums are fp32.  The softmax weights, times
 * their page's value scale, enter the second product as fp16: rounded to 11
 * bits, or to steps of 2^-34 of the row's largest where those are coarser.
 * Results do not depend on scheduling (no atomics).
 * batch or total_q of 0 is a no-op.
 * Errors: INVALID_ARGUMENT, UNSUPPORTED (as w4a8_rope_append; q_heads not a
 * multiple of kv_heads; more row tiles than one launch holds),
 * BUFFER_TOO_SMALL, DEVICE. */
size_t w4a8_paged_attention_workspace_size(const w4a8_kv_view* view, int q_heads, int max_q,
                                           int max_len);
w4a8_status w4a8_paged_attention(const uint16_t* q_dev, int ldq, int q_heads,
                                 const w4a8_kv_view* view, int max_q, int max_len, float scale,
                                 int window, uint16_t* out_dev, int ldo, void* workspace_dev,
                                 size_t workspace_bytes, void* stream);

/* ------------------------------------------------------- measurement aid
 * Not part of the layer.  A read-only stream over `bytes` of device memory
 * (16-byte aligned, a multiple of 16) by `workgroups` x 512 threads, with
 * four non-temporal 16-byte loads in flight per thread: the practical HBM
 * read ceiling that the weight-streaming regime (the FLUTE page, abstract:
 * at small batch, moving the weights from global memory dominates) is
 * measured against.  sink_dev holds `workgroups` uint32 values that are
 * written only in the rare case a workgroup's folded value equals a fixed
 * constant (so the loads cannot be optimised away); their contents mean
 * nothing.  bytes == 0 is a no-op.
 * Errors: INVALID_ARGUMENT (null pointer, misaligned or ragged size,
 * workgroups outside 1..65536), DEVICE. */
w4a8_status w4a8_read_probe(const void* src_dev, size_t bytes, int workgroups,
                            uint32_t* sink_dev, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* W4A8_H */
