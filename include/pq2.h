/*
 * pq2.h — C ABI of libpq2, the GB300 (sm_103a) library for the small-batch
 * and prefill matrix multiply of a ternary-quantised LLM ("PQ2" weights).
 *
 * The method (pages "Kernel experiments: recorded evidence", abbreviated KE,
 * and "Baseline and the integer breakthrough", abbreviated BIB):
 *   * weights: each row of K weights is K/128 blocks of 34 bytes — an fp16
 *     scale s_w followed by 32 code bytes; weight k of a block is the 2-bit
 *     field k%4 of code byte k/4, and code c means weight c-1 (KE Test 1,
 *     Diagram 1; BIB "Unpack four weights with fewer instructions").
 *   * activations: each group of 128 consecutive activations of a row is
 *     quantised to INT8 with s_x = max|x|/127 (fp32), q = clamp(round half to
 *     even(x / s_x), -127, 127) (KE Test 6; BIB "Calculate with small
 *     integers", step 1).
 *   * output: y[m][n] = sum over groups g of dot_g * s_x[m][g] * s_w[n][g],
 *     dot_g the exact int32 dot of the group's weights and q (BIB steps 3-4),
 *     accumulated in fp32.
 *
 * Conventions shared by every entry point:
 *   * Pointers marked (device) are CUDA device pointers owned by the caller;
 *     the library never allocates, frees or keeps them.  Buffers passed to
 *     one call must not overlap unless stated.  The activations x and the
 *     output y of pq2_quantize_act, pq2_mmv and pq2_linear are read and
 *     written with plain loads and stores, so they may also be pinned host
 *     memory that the device addresses at its own address (unified
 *     addressing, e.g. over NVLink-C2C); weights and q must be device
 *     memory (tensor-memory-access copies).
 *   * `stream` is a cudaStream_t (NULL = the legacy default stream).  Work is
 *     enqueued on it; no call synchronises the host with the device.
 *   * Shapes: K > 0 and K % 128 == 0, N >= 1, M in the entry point's range.
 *   * Argument errors are returned before anything is enqueued.  A launch
 *     failure returns PQ2_ERR_LAUNCH.  Device-side waits are bounded: a wait
 *     that gives up writes PQ2_ERR_TIMEOUT to *dev_status (when given) and
 *     the kernel returns early; results are then invalid.
 *   * The library only runs on compute capability 10.3 (GB300); any other
 *     device returns PQ2_ERR_ARCH.  Inputs must be finite (NaN/Inf in x
 *     give unspecified q).
 */
#ifndef PQ2_H
#define PQ2_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes returned by every entry point (and written to dev_status). */
enum {
  PQ2_OK = 0,
  PQ2_ERR_NULL = 1,      /* a required pointer is NULL                       */
  PQ2_ERR_SHAPE = 2,     /* M, N, K, a stride or a size is out of range      */
  PQ2_ERR_ALIGN = 3,     /* a pointer or stride breaks its alignment rule    */
  PQ2_ERR_DTYPE = 4,     /* unknown dtype or layout enum                     */
  PQ2_ERR_ARCH = 5,      /* current device is not compute capability 10.3   */
  PQ2_ERR_LAUNCH = 6,    /* the CUDA launch reported an error                */
  PQ2_ERR_TIMEOUT = 7,   /* a bounded device wait gave up (dev_status only)  */
  PQ2_ERR_CUDA = 8       /* a CUDA runtime query failed (no device, ...)     */
};

/* Element types of activations (x) and outputs (y); PQ2_I8 is the type of an
 * 8-bit key-value cache (pq2_kv_cache) only. */
enum { PQ2_BF16 = 0, PQ2_F16 = 1, PQ2_F32 = 2, PQ2_I8 = 3 };

/* Layouts of the quantised activations written by pq2_quantize_act.
 *  PQ2_Q_ROWS   int8 q[M][K], row-major, natural order.
 *  PQ2_Q_PLANES int8, plane order inside every 128-group: element i of a
 *               group is stored at (i%4)*32 + i/4 (KE Test 21, plane-order
 *               quantisation), so that plane s of a 4-byte code word meets
 *               one contiguous 4-byte slice of q.  Operand of pq2_mmv.
 *  PQ2_Q_F16    fp16, the same integer values widened exactly (|q| <= 127),
 *               in the K order pq2_mm's weight decode produces: inside every
 *               16 consecutive elements (the 16 weights of one 4-byte code
 *               word), element 4b + s (code byte b, field s) is stored at
 *               position 4s + 2(b & 1) + (b >> 1).  Operand of pq2_mm: sm_103a
 *               has no 8-bit integer tcgen05 MMA, so the prefill contraction
 *               runs on the fp16 tensor path, whose fp32 sums of integer
 *               products below 2^24 are exact.
 *  PQ2_Q_F8     two e4m3 planes per 128-group (2 bytes per element, the size
 *               of PQ2_Q_F16): q = 16a + b with a = q >> 4 in [-8, 7] and
 *               b = q & 15 in [0, 15], both exact in e4m3; bytes 0..127 of a
 *               group hold e4m3(16a), bytes 128..255 hold e4m3(b), each in
 *               the K order of pq2_mm_f8's weight decode: inside every 16
 *               consecutive elements, element 8h + 2e + o (h, o in {0, 1},
 *               e = 0..3) is stored at position 4(2h + o) + e.  Operand of
 *               pq2_mm_f8 (the 8-bit tensor path, two MMAs per K step).
 *  PQ2_Q_MMV16  fp16 [M][K], the B operand of the small-batch tensor-core
 *               GEMV pq2_mmv_tc, 128-groups only: inside every group,
 *               position 32t + 4j + 2r + e (t, j, r, e = 0..3, 0..7, 0..1,
 *               0..1) holds element i = 16(t + 4(j/4)) + 8e + f with
 *               f = 2(j%4) + r, divided by 4^f for f <= 4 and by 4^(f-3) for
 *               f >= 5 (exact: powers of two).  With this layout qsum does
 *               not receive sum(q) but the group's offset correction
 *               sum_i q_i (1 + 1024 / scale_i), scale_i that element's
 *               divisor (an exact integer, |.| < 2^22). */
enum { PQ2_Q_ROWS = 0, PQ2_Q_PLANES = 1, PQ2_Q_F16 = 2, PQ2_Q_F8 = 3, PQ2_Q_MMV16 = 4 };

/* Version of the prepared plane layout; bump whenever what a kernel reads
 * changes, so callers can key caches on it (BIB: a layout switch must change
 * the compile identity). */
int pq2_layout_version(void);

/* Static, never-NULL description of a status code. */
const char *pq2_status_string(int status);

/* Bytes of a prepared matrix: codes N*K/4 plus scales N*(K/128)*2 — still
 * exactly 34 bytes per 128 weights (KE Test 4).  0 if the shape is invalid. */
size_t pq2_prepared_bytes(int64_t N, int64_t K);

/* pq2_prepare — split raw blocks into a code plane and a scale plane
 * (KE Test 1 prepare_pq2 with separate buffers; Test 4 shared prepared
 * layout).  A pure byte move: values are unchanged.
 *   raw            (device) u8, N rows of K/128 blocks of 34 bytes, rows
 *                  raw_row_stride bytes apart (>= K/128*34).
 *   codes          (device) u8[N][K/4]; 16-byte aligned.
 *   scales         (device) fp16 bit patterns [N][K/128]; 2-byte aligned.
 * raw must not overlap codes or scales. */
int pq2_prepare(const uint8_t *raw, int64_t raw_row_stride, int64_t N,
                int64_t K, uint8_t *codes, uint16_t *scales, void *stream);

/* pq2_quantize_act — per-128-group INT8 quantisation of activations
 * (KE Test 6 _quantize; BIB "Calculate with small integers", step 1):
 *   s = max|x| / 127 (fp32 IEEE division); d = s > 0 ? s : 1;
 *   q = clamp(round-half-even(x / d), -127, 127) (IEEE division).
 *   x        (device) x_dtype [M][ldx], ldx >= K elements.
 *   M        1 .. 1<<20.
 *   q        (device) written in q_layout: int8 [M][K] for ROWS/PLANES,
 *            fp16 [M][K] for F16 and MMV16, bytes [M][2K] for F8; 16-byte
 *            aligned.
 *   sx       (device) fp32 [M][K/128] activation scales; 4-byte aligned.
 *   qsum     (device, may be NULL) int32 [M][K/128], sum of q per group
 *            (KE Test 21, the correction for the codes' -1 offset). */
int pq2_quantize_act(const void *x, int x_dtype, int64_t ldx, int64_t M,
                     int64_t K, void *q, int q_layout, float *sx,
                     int32_t *qsum, void *stream);

/* Decoders of the 2-bit codes used by the small-batch kernel; both give the
 * same exact int32 group dots.
 *  PQ2_DECODE_ADDXOR  the pages' add/XOR expansion (KE Test 1 _expand_byte;
 *                     BIB "Unpack four weights with fewer instructions"):
 *                     four codes spread one per byte, + 0x7F7F7F7F,
 *                     ^ 0x80808080, giving signed bytes c-1 for a signed
 *                     dp4a.
 *  PQ2_DECODE_PLANES  masked planes (KE Test 21): byte & (3 << 2s) = c*4^s
 *                     for an unsigned x signed dp4a, each plane shifted back
 *                     and the -1 offset removed once per group with sum(q). */
enum { PQ2_DECODE_ADDXOR = 0, PQ2_DECODE_PLANES = 1 };

/* pq2_mmv — small-batch (M = 1..8) ternary x INT8 GEMV with weight reuse
 * (BIB "Calculate with small integers"; KE Tests 6, 12, 14): every packed
 * weight byte is read from HBM once and used for all M columns; codes are
 * decoded in registers and multiplied with dp4a 4-way int8 dot products,
 * 32 per 128-group, into an exact int32 group dot, which is then scaled as
 * (float(dot) * s_x) * s_w and added in fp32.  The decoder is chosen from M
 * only (see pq2_mmv_decoder); pq2_mmv_ex takes it explicitly.
 *   q_planes (device) int8 [M][K] in PQ2_Q_PLANES order; 16-byte aligned.
 *   sx       (device) fp32 [M][K/128]; 4-byte aligned.
 *   qsum     (device) int32 [M][K/128] group sums of q (from
 *            pq2_quantize_act); 4-byte aligned.
 *   codes    (device) u8 [N][K/4] from pq2_prepare; 16-byte aligned.
 *   scales   (device) fp16 [N][K/128] from pq2_prepare; 2-byte aligned.
 *   y        (device) y_dtype [M][N] (PQ2_F32 or PQ2_BF16, bf16 = round to
 *            nearest even of the fp32 result); aligned to its element.
 *   dev_status (device, may be NULL) int32; PQ2_ERR_TIMEOUT is stored there
 *            if a device wait gives up; never cleared by the library.
 * Batch invariance: the fp32 operation sequence of output column m depends
 * only on (N, K) and the device's SM count, never on M, and the group dots
 * are exact, so column m is bit-identical for every M that contains it. */
int pq2_mmv(const int8_t *q_planes, const float *sx, const int32_t *qsum,
            const uint8_t *codes, const uint16_t *scales, void *y,
            int y_dtype, int64_t M, int64_t N, int64_t K, int32_t *dev_status,
            void *stream);

/* Flags of pq2_mmv_ex.  Every libpq2 kernel is launched with programmatic
 * dependent launch: it may start before the kernel enqueued before it on the
 * stream completes, and waits for it before reading anything that kernel may
 * write.  pq2_quantize_act, pq2_mmv, pq2_mmv_ex and pq2_mmv_gated release
 * the next kernel as soon as they start; pq2_mm releases it only once the kernel before it
 * has completed.  So the kernels that may still run when a call starts are
 * those enqueued at or after the latest "ordering point" before it: a
 * pq2_mm call, a host synchronisation, an event wait, a copy, or a kernel
 * launched without programmatic dependent launch (pq2_prepare is one).
 * Without flags a call needs nothing of this.
 *  PQ2_MMV_OVERLAP_WEIGHTS  the call may stream codes and scales from HBM
 *      before earlier kernels complete.  Legal when no kernel that may still
 *      run writes codes or scales (e.g. the weights were prepared before the
 *      latest ordering point).
 *  PQ2_MMV_INDEPENDENT      the call reads every input early and computes
 *      before earlier kernels complete.  Legal when no kernel that may still run writes any input of this call
 *      (e.g. back-to-back projections of the same quantised activations).
 *      y is always written only after the kernel before the call has
 *      completed. */
enum { PQ2_MMV_OVERLAP_WEIGHTS = 1, PQ2_MMV_INDEPENDENT = 2 };

/* pq2_mmv with an explicit decoder (PQ2_DECODE_ADDXOR or PQ2_DECODE_PLANES)
 * and flags; results are bit-identical to pq2_mmv for every decoder. */
int pq2_mmv_ex(const int8_t *q_planes, const float *sx, const int32_t *qsum,
               const uint8_t *codes, const uint16_t *scales, void *y,
               int y_dtype, int64_t M, int64_t N, int64_t K, int decode,
               int flags, int32_t *dev_status, void *stream);

/* pq2_mmv_tc — the small-batch GEMV (M = 1..8) on the legacy tensor-core
 * path (mma.sync m16n8k16, fp16 operands, fp32 accumulation): the same
 * output as pq2_mmv, bit for bit, at an arithmetic cost that does not grow
 * with M.  Each code word is expanded in registers, one logic operation per
 * two weights, into the exact fp16 values 1024 + c * 4^f; the activations
 * come divided by the same powers of four (PQ2_Q_MMV16), so every product is
 * an integer and the fp32 sum of a group is exact; subtracting the group's
 * correction leaves the exact dot of BIB step 3.  The split of the groups,
 * the scaling (float(dot) * s_x) * s_w and the order of the fp32 additions
 * are pq2_mmv's (a function of N, K and the SM count only), hence the same
 * bits and the same batch invariance.
 *   q_mmv16  (device) fp16 [M][K] from pq2_quantize_act(PQ2_Q_MMV16);
 *            16-byte aligned.
 *   sx       (device) fp32 [M][K/128] from the same call.
 *   qcorr    (device) int32 [M][K/128], the corrections that call writes to
 *            its qsum argument.
 *   codes, scales, y, y_dtype, M, N, K, flags, dev_status as for pq2_mmv_ex
 *            (flags: the same stream contract).
 * Returns PQ2_ERR_SHAPE for shapes whose per-CTA tiling it does not cover
 * (none of the library's geometries), else as pq2_mmv_ex. */
int pq2_mmv_tc(const uint16_t *q_mmv16, const float *sx, const int32_t *qcorr,
               const uint8_t *codes, const uint16_t *scales, void *y, int y_dtype,
               int64_t M, int64_t N, int64_t K, int flags, int32_t *dev_status,
               void *stream);

/* 1 if pq2_linear runs the tensor-core GEMV (pq2_mmv_tc on PQ2_Q_MMV16) for
 * M columns of an N x K matrix on a device with sm_count SMs, 0 if it runs
 * pq2_mmv (host only, no CUDA call); the results are the same.  The choice
 * follows the two kernels' measured cost: the tensor-core GEMV from M = 6,
 * and at M = 5 where a CTA of pq2_mmv_geometry holds at most 72 rows in at
 * most 8 splits. */
int pq2_linear_tensor_gemv(int64_t M, int64_t N, int64_t K, int sm_count);

/* pq2_linear — the complete projection y = x W^T (quantise, then the GEMV),
 * as the pages time it ("complete call", KE Tests 3, 6): pq2_quantize_act
 * into the caller's workspace, then pq2_mmv (M = 1..8; pq2_mmv_tc on
 * PQ2_Q_MMV16 for the M where pq2_linear_tensor_gemv says so, with the same
 * bits) with PQ2_MMV_OVERLAP_WEIGHTS, so that it streams the weights while
 * the quantisation and the kernel before it finish, or pq2_mm_f8 on PQ2_Q_F8
 * (M >= 9; bit-identical to pq2_mm, faster).  Hence
 * codes and scales must not be written by a kernel that may still run when
 * the call starts (see the flags of pq2_mmv_ex).
 * Results are bit-identical to pq2_quantize_act + pq2_mmv / pq2_mm_f8.
 * The workspace holds q with one byte per element for M <= 4 and two
 * otherwise (the tensor-core GEMV and the prefill GEMM take 16-bit q).
 *   x         (device) x_dtype [M][ldx], ldx >= K; M 1 .. 1<<20 (M 9..15,
 *             between the pages' GEMV and prefill sizes, run as the prefill
 *             GEMM's one partial token tile).
 *   workspace (device) pq2_linear_workspace_bytes(M, K) bytes, 256-byte
 *             aligned, holding q, s_x and sum(q); contents are scratch.
 *   codes, scales, y, y_dtype, dev_status as for pq2_mmv. */
int pq2_linear(const void *x, int x_dtype, int64_t ldx, int64_t M, int64_t N,
               int64_t K, const uint8_t *codes, const uint16_t *scales,
               void *y, int y_dtype, void *workspace, size_t workspace_bytes,
               int32_t *dev_status, void *stream);

/* Workspace bytes pq2_linear needs for M columns of K inputs (0 if the
 * shape is invalid). */
size_t pq2_linear_workspace_bytes(int64_t M, int64_t K);

/* Activation groups of 64 or 32 (page "Kernel experiments: recorded
 * evidence", Test 9, "Smaller Q8 activation groups"): the activations get
 * one scale per act_group elements, the weights keep their 128-groups and
 * scales, and each 128-group's dot splits into 128 / act_group partial dots,
 * each scaled by its own activation scale:
 *   y[m][n] = sum_g sum_{h < 128/A} (float(dot_gh) * s_x[m][g*128/A + h])
 *             * s_w[n][g]        (fp32, each operation rounded to nearest)
 * act_group = 128 is exactly pq2_quantize_act / pq2_mmv.
 *
 * pq2_quantize_act_grouped — pq2_quantize_act with activation groups of
 * act_group (128, 64, 32) elements; sx and qsum are [M][K / act_group].
 * q keeps the layouts of pq2_quantize_act. */
int pq2_quantize_act_grouped(const void *x, int x_dtype, int64_t ldx,
                             int64_t M, int64_t K, int act_group, void *q,
                             int q_layout, float *sx, int32_t *qsum,
                             void *stream);

/* pq2_mmv_grouped — pq2_mmv_ex (masked-plane decoder, flags) on activations
 * quantised by pq2_quantize_act_grouped with the same act_group; M 1..8.
 * The kernel holds four columns' partial sums at most: M = 5..8 runs as two
 * passes over the weights (columns 0..3, then 4..M-1), with the same bits as
 * one pass (a column's result does not depend on the others).  Batch
 * invariant like pq2_mmv.  Returns PQ2_ERR_SHAPE for M > 8 or another
 * act_group, else as pq2_mmv_ex. */
int pq2_mmv_grouped(const int8_t *q_planes, const float *sx,
                    const int32_t *qsum, const uint8_t *codes,
                    const uint16_t *scales, void *y, int y_dtype, int64_t M,
                    int64_t N, int64_t K, int act_group, int flags,
                    int32_t *dev_status, void *stream);

/* The exact partial dots of pq2_mmv_grouped, dots[m][n][j] = sum over k in
 * [j*A, j*A + A) of (c_{n,k} - 1) q_{m,k}, from the same device code, for
 * parity checks (M 1..8, q in PQ2_Q_PLANES order, qsum from
 * pq2_quantize_act_grouped).  dots (device) int32 [M][N][K / A]. */
int pq2_debug_group_dots_grouped(const int8_t *q_planes, const int32_t *qsum,
                                 const uint8_t *codes, int64_t M, int64_t N,
                                 int64_t K, int act_group, int32_t *dots,
                                 int32_t *dev_status, void *stream);

/* PTQ1_0 weights (page "KERNEL_REPORT: PTQ1_0 small-batch decoding on the
 * PrismML fork, RTX 3060 12GB", "What the source said"): each row of K
 * weights is K/128 blocks of 28 bytes: qs (bytes 0-23, five trits per byte),
 * qh (bytes 24-25, four trits per byte), the fp16 scale d (bytes 26-27,
 * little-endian).  Trit n (0 first) of a byte b is floor(b * 3^(n+1) / 256)
 * mod 3, the digit left above the low byte after n + 1 multiplications by 3;
 * trit t means weight t - 1.  Weight order inside a block (the page does
 * not fix it; this library's reading): trit n of qs byte j is weight 24n + j,
 * trit n of qh byte j is weight 120 + 2n + j.
 *
 * pq2_ptq_prepare — raw blocks (device, N rows, row stride raw_row_stride
 * bytes >= 28 K/128) -> qs plane u8[N][24 K/128] (16-byte aligned) and side
 * plane u32[N][K/128] (8-byte aligned): bits 0-15 qh (byte 24 low), bits
 * 16-31 d.  A byte move; K % 256 == 0. */
int pq2_ptq_prepare(const uint8_t *raw, int64_t raw_row_stride, int64_t N,
                    int64_t K, uint8_t *qs, uint32_t *side, void *stream);

/* pq2_ptq_mmv — y[m][n] = sum_g d_g * sum_h float(dot_gh) * s_x[m][g*128/A+h]
 * for M = 1..4 columns of activations quantised by pq2_quantize_act_grouped
 * with the same act_group A (128, 64 or 32; PQ2_Q_ROWS layout, sum(q)
 * required), dot_gh the exact integer dot of activation group h of block g:
 * fp32, each operation rounded to nearest, a fixed order that depends on
 * (N, K, SM count) only, so column m is bit-identical for every M.
 * y fp32 or bf16 (RNE of the fp32 result) [M][N].  flags as pq2_mmv_ex
 * (PQ2_MMV_OVERLAP_WEIGHTS, PQ2_MMV_INDEPENDENT, same stream contract).
 * K % 256 == 0; the kernel has no waits that can time out. */
int pq2_ptq_mmv(const int8_t *q_rows, const float *sx, const int32_t *qsum,
                const uint8_t *qs, const uint32_t *side, void *y, int y_dtype,
                int64_t M, int64_t N, int64_t K, int act_group, int flags,
                void *stream);

/* pq2_ptq_linear — the complete PTQ1_0 projection: pq2_quantize_act_grouped
 * (PQ2_Q_ROWS, act_group) into the caller's workspace, then pq2_ptq_mmv with
 * PQ2_MMV_OVERLAP_WEIGHTS (the GEMV streams its weights while the
 * quantisation runs; qs and side must not be written by a kernel that may
 * still run).  Bit-identical to the two calls.
 *   x         (device or device-addressable host) x_dtype [M][ldx], M 1..4.
 *   workspace (device) pq2_ptq_linear_workspace_bytes(M, K, act_group)
 *             bytes, 256-byte aligned; contents are scratch.
 * Returns PQ2_ERR_SHAPE for a workspace that is too small, else as the two
 * calls. */
size_t pq2_ptq_linear_workspace_bytes(int64_t M, int64_t K, int act_group);
int pq2_ptq_linear(const void *x, int x_dtype, int64_t ldx, int64_t M,
                   int64_t N, int64_t K, const uint8_t *qs, const uint32_t *side,
                   int act_group, void *y, int y_dtype, void *workspace,
                   size_t workspace_bytes, void *stream);

/* The exact partial dots of pq2_ptq_mmv, dots[m][n][j] = sum over k in
 * [jA, jA + A) of (t_{n,k} - 1) q_{m,k}, from the same device code (parity
 * checks).  dots (device) int32 [M][N][K / A]. */
int pq2_debug_ptq_dots(const int8_t *q_rows, const int32_t *qsum,
                       const uint8_t *qs, const uint32_t *side, int64_t M,
                       int64_t N, int64_t K, int act_group, int32_t *dots,
                       void *stream);

/* pq2_mmv_gated — the gate/up projection with its gated activation in the
 * GEMV's epilogue (page "Kernel experiments: recorded evidence", Test 12,
 * "gated" fusion screen: the projection's output z = x W^T of width N is
 * split in halves, gate = z[:, :N/2], up = z[:, N/2:], and the result is
 * silu(gate) * up computed in fp32 and rounded to the output type):
 *   out[m][n] = silu(y[m][n]) * y[m][n + N/2],  n < N/2,
 *   silu(v)   = v / (1 + exp(-v)),
 * each operation in fp32 with round-to-nearest (exp: CUDA's expf, 2 ulp),
 * where y is the fp32 sum pq2_mmv forms for those rows, with the same
 * operation order (the split count comes from all N rows), so gate and up
 * are bit-identical to pq2_mmv's y.  Batch invariant like pq2_mmv.  Gate
 * row n and up row n + N/2 are streamed by the same CTA; the N/2 x M
 * intermediate never exists.
 *   q_planes, sx, qsum, codes, scales, M, K, flags, dev_status as for
 *            pq2_mmv_ex (masked-plane decoder).  codes/scales hold N rows:
 *            the gate rows, then the up rows.
 *   N        even, 2 .. 1<<30.
 *   out      (device) out_dtype [M][N/2] (PQ2_F32 or PQ2_BF16).
 * Returns PQ2_ERR_SHAPE for an odd N, else as pq2_mmv_ex. */
int pq2_mmv_gated(const int8_t *q_planes, const float *sx, const int32_t *qsum,
                  const uint8_t *codes, const uint16_t *scales, void *out,
                  int out_dtype, int64_t M, int64_t N, int64_t K, int flags,
                  int32_t *dev_status, void *stream);

/* pq2_linear_gated — the complete gated call for M = 1..8:
 * pq2_quantize_act into the workspace, then pq2_mmv_gated with
 * PQ2_MMV_OVERLAP_WEIGHTS (the stream contract of pq2_linear).  Results are
 * bit-identical to pq2_quantize_act + pq2_mmv_gated.
 *   x, x_dtype, ldx, workspace as for pq2_linear (M 1..8 only);
 *   N, codes, scales, out, out_dtype, dev_status as for pq2_mmv_gated. */
int pq2_linear_gated(const void *x, int x_dtype, int64_t ldx, int64_t M,
                     int64_t N, int64_t K, const uint8_t *codes,
                     const uint16_t *scales, void *out, int out_dtype,
                     void *workspace, size_t workspace_bytes,
                     int32_t *dev_status, void *stream);

/* Size of the static device scratch of pq2_linear_static (1 MiB). */
#define PQ2_STATIC_SCRATCH_BYTES ((size_t)1 << 20)

/* pq2_linear_static — pq2_linear for callers that cannot allocate device
 * memory (for example code running where cudaMalloc is not allowed, or
 * runtimes whose allocator owns all device memory).  The pages have no
 * counterpart: this is a deployment convenience, not a step of the method.
 * The call allocates nothing (no cudaMalloc, cudaFree or allocating library
 * routine): its workspace (q, s_x and sum(q), laid out as for pq2_linear) is
 * a file-scope static device array of PQ2_STATIC_SCRATCH_BYTES in every
 * device's context, which each device holds until the process exits.  Its
 * device address is looked up (cudaGetSymbolAddress) with the device current
 * on the first call on that device, which also creates the device's primary
 * context, and again whenever the current context differs from the one the
 * address was found in (after a device reset).  Make the first call on a
 * device before capturing any stream into a graph.
 *   Arguments, results and errors as for pq2_linear, without the workspace;
 *   errors in pq2_linear's order (NULL, dtype, shape).
 *   stream   must belong to the current device (NULL is the current
 *            device's legacy default stream): the scratch address is the
 *            current device's.  Another device's stream returns PQ2_ERR_CUDA.
 *   Returns PQ2_ERR_SHAPE, before any CUDA call, when
 *   pq2_linear_workspace_bytes(M, K) exceeds PQ2_STATIC_SCRATCH_BYTES (for
 *   example M = 4 with K above 246,656, M = 8 with K above 63,488, or
 *   M = 16 with K above 31,744);
 *   PQ2_ERR_CUDA if the scratch address cannot be obtained.
 * Every call on a device shares the one scratch array, which keeps the last
 * call's contents.  Nothing in it needs to start at zero: each call writes
 * all of it that it reads.  Calls that may run at the same time on the GPU
 * (for example on two streams) race on it; calls in order on one stream do
 * not. */
int pq2_linear_static(const void *x, int x_dtype, int64_t ldx, int64_t M,
                      int64_t N, int64_t K, const uint8_t *codes,
                      const uint16_t *scales, void *y, int y_dtype,
                      int32_t *dev_status, void *stream);

/* The decoder pq2_mmv uses for M columns (host only). */
int pq2_mmv_decoder(int64_t M);

/* Largest K pq2_norm_hadamard_quantize takes (a row's fp32 copy stays in
 * shared memory). */
#define PQ2_PREP_MAX_K 32768

/* pq2_norm_hadamard_quantize — the activations' preparation fused into one
 * kernel (page "Kernel experiments: recorded evidence", Test 18, "RMSNorm +
 * Hadamard + Q8 fusion"), per row m of K columns:
 *   h    = x (+ residual), fp32
 *   S    = sum of h^2: partial i (0..2047) sums h[j]^2 for j = i mod 2048 in
 *          increasing j, then p[i] += p[i + len] for len = 1024, 512, .., 1
 *          (fp32; S = p[0])
 *   inv  = 1 / sqrt(S / K + eps)            (IEEE square root and division)
 *   n    = bf16((h * inv) * (w + 1))         (norm weight w, applied as w + 1)
 *   v    = n * sign                          (sign +1 / -1 per column)
 *   v    = bf16(WHT(v)) per 1024-column block, WHT the orthonormal
 *          Walsh-Hadamard transform (butterfly passes of half-width 1, 2, ..,
 *          512 in fp32, then the exact factor 1/32)
 *   q, sx, qsum = pq2_quantize_act of v (group 128, same rounding)
 * Every fp32 operation rounds to nearest; the codes are therefore a function
 * of the inputs alone (bit-exact against the CPU oracle).
 *   x            (device) bf16 [M][K].
 *   residual     (device, may be NULL) bf16 [M][K], added to x first.
 *   residual_out (device, may be NULL) bf16 [M][K] <- bf16(h).
 *   w            (device) bf16 [K]; sign (device) int8 [K], each +1 or -1.
 *   eps          0 <= eps <= 1.
 *   M            1 .. 1<<20;  K a multiple of 1024, 1024 .. PQ2_PREP_MAX_K.
 *   norm_out     (device, may be NULL) bf16 [M][K] <- n.
 *   q, q_layout, sx, qsum as for pq2_quantize_act.
 * Returns PQ2_ERR_SHAPE for K or eps out of range, else as
 * pq2_quantize_act; launched with programmatic dependent launch like it. */
int pq2_norm_hadamard_quantize(const uint16_t *x, const uint16_t *residual,
                               uint16_t *residual_out, const uint16_t *w,
                               const int8_t *sign, float eps, int64_t M,
                               int64_t K, uint16_t *norm_out, void *q,
                               int q_layout, float *sx, int32_t *qsum,
                               void *stream);

/* pq2_mm — prefill (M >= 16; any M >= 1) ternary x INT8 matmul as a dense tensor-core
 * contraction (KE Test 7 "INT8 tensor-core MMQ prefill"; BIB "Use matrix
 * hardware for prefill"): per 128-group the exact dot of q and the decoded
 * codes is formed on tcgen05 tensor cores (fp16 operands holding integer
 * values, fp32 accumulation confined to one group, hence exact), then scaled
 * by s_x * s_w into an fp32 accumulator.
 *   q_f16    (device) fp16 [M][K] from pq2_quantize_act(PQ2_Q_F16);
 *            16-byte aligned.
 *   sx       (device) fp32 [M][K/128].
 *   qsum     (device) int32 [M][K/128] group sums of q.
 *   codes, scales as for pq2_mmv.
 *   y        (device) y_dtype [M][N] (PQ2_F32 or PQ2_BF16).
 *   M        1 .. 1<<20 (the prefill sizes are M >= 16; a smaller M is one
 *            partial 128-token tile).
 *   dev_status as for pq2_mmv. */
int pq2_mm(const uint16_t *q_f16, const float *sx, const int32_t *qsum,
           const uint8_t *codes, const uint16_t *scales, void *y, int y_dtype,
           int64_t M, int64_t N, int64_t K, int32_t *dev_status, void *stream);

/* pq2_mm_f8 — pq2_mm on the 8-bit tensor path: the weights decode to e4m3
 * (-1, 0, +1; code 3 gives +2) and q comes as the two exact e4m3 planes of
 * PQ2_Q_F8; each K step is two kind::f8f6f4 MMAs (16a and b) accumulating
 * into the same fp32 group tile, whose integer sums stay below 2^24, so the
 * group dot is exact and y is bit-identical to pq2_mm's.
 *   q_f8     (device) [M][2K] bytes from pq2_quantize_act(PQ2_Q_F8);
 *            16-byte aligned.  Other arguments as for pq2_mm. */
int pq2_mm_f8(const uint8_t *q_f8, const float *sx, const int32_t *qsum,
              const uint8_t *codes, const uint16_t *scales, void *y,
              int y_dtype, int64_t M, int64_t N, int64_t K,
              int32_t *dev_status, void *stream);

/* pq2_mm_grouped, pq2_mm_f8_grouped — pq2_mm and pq2_mm_f8 on activations
 * quantised by pq2_quantize_act_grouped with activation groups of act_group
 * A = 128, 64 or 32 elements (KE Test 9, "Smaller Q8 activation groups":
 * the weights and their 128-weight scales stay as they are, each weight
 * group's dot splits into 128 / A separately scaled partial dots):
 *   y[m][n] = sum over weight groups g, then over h = 0 .. 128/A - 1, of
 *             (dot_gh * s_x[m][g*128/A + h]) * s_w[n][g]
 * with dot_gh the exact integer dot of activation group h of block g, each
 * a separate tensor-core accumulation (exact, as for pq2_mm), scaled in fp32.
 *   q_f16 / q_f8 as for pq2_mm / pq2_mm_f8, from pq2_quantize_act_grouped
 *            (PQ2_Q_F16 / PQ2_Q_F8, the same act_group).
 *   sx, qsum (device) [M][K / act_group].
 * act_group 128 gives exactly pq2_mm / pq2_mm_f8.  Returns PQ2_ERR_SHAPE for
 * another act_group, else as pq2_mm. */
int pq2_mm_grouped(const uint16_t *q_f16, const float *sx, const int32_t *qsum,
                   const uint8_t *codes, const uint16_t *scales, void *y,
                   int y_dtype, int64_t M, int64_t N, int64_t K, int act_group,
                   int32_t *dev_status, void *stream);
int pq2_mm_f8_grouped(const uint8_t *q_f8, const float *sx, const int32_t *qsum,
                      const uint8_t *codes, const uint16_t *scales, void *y,
                      int y_dtype, int64_t M, int64_t N, int64_t K,
                      int act_group, int32_t *dev_status, void *stream);

/* pq2_linear_grouped — the complete projection with activation groups of
 * act_group elements (128, 64, 32; KE Test 9 times exactly this call at
 * M = 128 and 512): pq2_quantize_act_grouped into the caller's workspace,
 * then pq2_mmv_grouped (M = 1..8, masked-plane decoder, weights streamed
 * while the quantisation runs) or pq2_mm_f8_grouped (M >= 9).
 * Bit-identical to those calls.
 *   x, ldx, codes, scales, y, y_dtype, dev_status as for pq2_linear.
 *   workspace (device) pq2_linear_grouped_workspace_bytes(M, K, act_group)
 *             bytes, 256-byte aligned; contents are scratch.
 * pq2_linear_grouped_workspace_bytes returns 0 for invalid arguments.
 * Returns PQ2_ERR_SHAPE for a workspace that is too small or another
 * act_group, else as the calls it makes. */
size_t pq2_linear_grouped_workspace_bytes(int64_t M, int64_t K, int act_group);
int pq2_linear_grouped(const void *x, int x_dtype, int64_t ldx, int64_t M,
                       int64_t N, int64_t K, const uint8_t *codes,
                       const uint16_t *scales, int act_group, void *y,
                       int y_dtype, void *workspace, size_t workspace_bytes,
                       int32_t *dev_status, void *stream);

/* Matrix-vector products with 4-bit weights and group scales: the output
 * head (or any projection that ternary weights are too coarse for).
 * Row n holds K codes of 4 bits, each G of them with an fp16 scale s and,
 * with zero points, a zero point z in 0..15 (without them z = 8):
 *   y[m][n] = sum_g s[n][g] * sum_{k in g} (c[n][k] - z[n][g]) * x[m][k]
 * G = group = 128, 64 or 32;  K >= G a multiple of G (not of 128).
 *
 * pq2_w4_prepare — lays the weights out once in the order the kernel streams
 * them.  A move of bits: values are unchanged.  It is an ordering point (see
 * pq2_mmv_ex).
 *   codes    (device) u8, N rows of K/2 bytes, ldc bytes apart (>= K/2);
 *            column 2j is the low half of byte j, column 2j + 1 the high.
 *   scales   (device) fp16 [N][K/G].
 *   zeros    (device, NULL = no zero points) u8 [N][K/G]; only the low four
 *            bits are read.
 *   plane    (device) pq2_w4_plane_bytes(N, K, group, zeros != NULL) bytes,
 *            16-byte aligned.
 * pq2_w4_plane_bytes returns 0 for invalid arguments. */
size_t pq2_w4_plane_bytes(int64_t N, int64_t K, int group, int zeros);
int pq2_w4_prepare(const uint8_t *codes, int64_t ldc, const uint16_t *scales,
                   const uint8_t *zeros, int64_t N, int64_t K, int group,
                   uint8_t *plane, void *stream);

/* pq2_w4_mmv — y = x W^T for M = 1..32.  c - z is exact, x is taken in fp16:
 * an fp16 x as it is; a bf16 x scaled by a power of two per 256 columns at
 * most (exact down to 2^-28 of the largest |x| among them, within 2^-39 of it
 * below); a 32-bit x as the sum of two such parts (within 2^-23 of its value,
 * or within 2^-51 of the largest |x| among them where that is more).
 * Products are exact, sums and y fp32.  Infinities and NaN in x come
 * out as the formula has them.
 *   x        (device, or pinned host memory as for pq2_mmv) x_dtype
 *            [M][ldx], ldx >= K; PQ2_BF16, PQ2_F16 or PQ2_F32.
 *   zeros    non-zero if the plane was prepared with zero points.
 *   plane    (device) from pq2_w4_prepare with the same N, K, group, zeros.
 *   y        (device) y_dtype [M][N]; PQ2_F32, PQ2_BF16 or PQ2_F16, the fp32
 *            result rounded to nearest even.
 *   flags    PQ2_MMV_OVERLAP_WEIGHTS, PQ2_MMV_INDEPENDENT as for pq2_mmv_ex
 *            (plane in the place of codes and scales); the kernel releases
 *            the next one as soon as it starts.
 * The weights are read once for M <= 8 (4 with a 32-bit x), above that once per
 * 8 to 32 columns (4 to 16): as many as fit shared memory beside the split of K,
 * which follows N and K (on 152 SMs 32 for K = 4160 .. 8192, 8 for K = 4096).
 * Column m is bit-identical for every M that contains it: the order of its
 * additions depends on (N, K, group) and the device's SM count only. */
int pq2_w4_mmv(const void *x, int x_dtype, int64_t ldx, int64_t M, int64_t N,
               int64_t K, int group, int zeros, const uint8_t *plane, void *y,
               int y_dtype, int flags, void *stream);

/* Most alternatives per row that pq2_token_logprobs returns. */
#define PQ2_MAX_TOP 32

/* pq2_token_logprobs — per row of logits x, with t = scale * x and
 * log p = t - log sum exp t:
 *   token_logprobs[m][j] = log p[tokens[m][j]]
 *   entropy[m]           = -sum p log p
 *   top_ids[m][0..k)     = the k largest logits, descending, equal ones by
 *                          the lower index;  top_logprobs their log p.
 * A logit of -inf is excluded (p = 0).  A row that has only those: every log
 * p is -inf, the entropy 0, top_ids 0..k-1.  A NaN or +inf in a row makes its
 * log p and entropy NaN; in the order of the alternatives NaN is last.
 *   logits   (device) dtype [M][ldl], ldl >= V; PQ2_BF16, PQ2_F16, PQ2_F32.
 *   M        1 .. 1<<20;  V 1 .. 1<<30.
 *   scale    1 / temperature, 0 < scale <= 1e6.
 *   tokens   (device) int64 [M][T], T >= 0 (may be NULL when T = 0).  A
 *            negative id marks no token (log p 0), an id >= V gives NaN.
 *   token_logprobs (device) fp32 [M][T].
 *   entropy  (device, may be NULL) fp32 [M].
 *   k        0 .. min(V, PQ2_MAX_TOP).
 *   top_ids, top_logprobs (device; may be NULL when k = 0) int64 and fp32
 *            [M][k].
 * Sums in fp32 in a fixed order: the same call gives the same bits.  The order
 * follows M, V and the device's SM count (they decide how many CTAs share a
 * row), so the log p and entropy of a row may differ in their last bits between
 * calls with other numbers of rows; the ids do not.  Runs
 * after the kernel before it on the stream and releases the next one as soon
 * as it starts. */
int pq2_token_logprobs(const void *logits, int dtype, int64_t ldl, int64_t M,
                       int64_t V, float scale, const int64_t *tokens,
                       int64_t T, float *token_logprobs, float *entropy,
                       int k, int64_t *top_ids, float *top_logprobs,
                       void *stream);

/* pq2_norm_gate_residual — the RMS norms after a block and before the next
 * one, fused with the block's gate and residual scale, per row of K columns:
 *   p  = z / sqrt(mean z^2 + eps) * (w_post + w_offset)   (p = z if w_post
 *        is NULL)
 *   h' = h + alpha * gate * p         (no gate if NULL; h' = h if z is NULL)
 *   n  = h' / sqrt(mean h'^2 + eps) * (w_pre + w_offset)
 * in fp32 (1 / sqrt is CUDA's rsqrtf, 2 ulp); h' is rounded for h_out only.
 *   z, h     (device) dtype [M][ldz], [M][ldh], both strides >= K; z NULL
 *            gives the plain norm of h (then no w_post, gate or h_out).
 *   w_post, w_pre (device) dtype [K]; w_pre may be NULL if n_out is.
 *   gate     (device, may be NULL) dtype, row m uses row m / rows_per_gate,
 *            ldg >= K apart: rows_per_gate 1 is a gate per token, M one for
 *            all, S one per sequence of S tokens.
 *   w_offset added to both weights (1 for weights stored about 0).
 *   eps      0 <= eps <= 1.
 *   M        1 .. 1<<20;  K 1 .. PQ2_PREP_MAX_K.
 *   h_out, n_out (device, one of them may be NULL) dtype [M][K].  h_out may
 *            be h (when ldh = K); no other buffers may overlap.
 * A missing operand of a part that is asked for is PQ2_ERR_NULL.  Runs after
 * the kernel before it and releases the next one as soon as it starts. */
int pq2_norm_gate_residual(const void *z, int64_t ldz, const void *h,
                           int64_t ldh, int dtype, const void *w_post,
                           const void *gate, int64_t ldg,
                           int64_t rows_per_gate, float alpha,
                           const void *w_pre, float w_offset, float eps,
                           int64_t M, int64_t K, void *h_out, void *n_out,
                           void *stream);

/* A paged key-value cache: the keys and values of `pages` pages of page_size
 * token slots, for `heads` heads of `dim` elements.
 *   k, v      (device) dtype; element (page, head, slot, d) lies at
 *             page * page_stride + head * head_stride + slot * token_stride
 *             + d, strides in elements and the same for k and v, so that
 *             [pages][heads][page_size][dim], [pages][page_size][heads][dim]
 *             and pages that hold k and v in turn are all possible.
 *   k_scales, v_scales (device, PQ2_I8 only, else NULL) fp32
 *             [pages][heads][page_size].
 *   dtype     PQ2_BF16, PQ2_F16 or PQ2_I8: an element of an 8-bit cache
 *             stands for its integer times the scale of its token and head,
 *             s = max|x| / 127, q = clamp(round-half-even(x / s), -127, 127)
 *             (IEEE division; s = 0 divides as 1): pq2_quantize_act's rule
 *             over the dim elements of a token and head.  An infinity or NaN
 *             among them reads back as NaN in all of them.
 *   pages 1 .. 1<<30; heads 1 .. 1<<16; page_size a multiple of 16 up to
 *   1<<20; dim 64, 128 or 256; k, v and the scales 16-byte aligned, the
 *   strides multiples of 16 bytes, below 2^40 bytes and not negative; heads,
 *   slots and pages must not overlap.
 * A sequence's position p lies in slot p % page_size of page
 * table[b][p / page_size].  A call that meets an entry that is no page of the
 * cache, or a position behind the table's width, does not follow it: nothing
 * is stored there, and it reads as zeros. */
typedef struct pq2_kv_cache {
  void *k, *v;
  float *k_scales, *v_scales;
  int dtype;
  int64_t pages, heads, page_size, dim;
  int64_t page_stride, head_stride, token_stride;
} pq2_kv_cache;

/* pq2_kv_store — writes the keys and values of the newest tokens of B
 * sequences into the cache, rounded to nearest even (16 bits) or quantised.
 * Row i of sequence b, cu[b] <= i < cu[b + 1], is its position
 *   lens[b] - (cu[b + 1] - cu[b]) + (i - cu[b]):
 * lens counts the new tokens already.
 *   k, v     (device) dtype PQ2_BF16, PQ2_F16 or PQ2_F32, element (row, head,
 *            d) at row * token_stride + head * head_stride + d (strides in
 *            elements, one pair for each).  Any alignment of whole elements;
 *            16-byte aligned pointers and strides are faster.
 *   tokens   rows of k and v, 0 .. 1<<24 (0: nothing is done, k and v may be
 *            NULL); rows outside every sequence are not read.
 *   cache    (host) its description; pages, tables and scales are device
 *            memory.
 *   table    (device) int32 [B][table_width], rows table_stride apart.
 *   cu       (device, may be NULL) int32 [B + 1], not decreasing; NULL: the
 *            rows are split evenly, tokens / B to each (tokens % B = 0).
 *   lens     (device) int32 [B];  B 1 .. 1<<20.
 * Two rows for one position are the caller's error: which one stays is not
 * defined.  Runs after the kernel before it on the stream and releases the
 * next one as soon as it starts; so does pq2_kv_load. */
int pq2_kv_store(const void *k, int64_t k_token_stride, int64_t k_head_stride,
                 const void *v, int64_t v_token_stride, int64_t v_head_stride,
                 int dtype, int64_t tokens, const pq2_kv_cache *cache,
                 const int32_t *table, int64_t table_stride,
                 int64_t table_width, const int32_t *cu, const int32_t *lens,
                 int64_t B, void *stream);

/* pq2_kv_load — the same rows the other way: reads the last
 * cu[b + 1] - cu[b] positions of each sequence back, packed as
 * pq2_attn_prefill takes them (with cu the running sums of lens: all of
 * them).
 *   k, v     (device) dtype PQ2_BF16, PQ2_F16 or PQ2_F32 [tokens][heads][dim],
 *            16-byte aligned.  Rows outside every sequence stay as they
 *            were; a position that is not in the cache gives zeros. */
int pq2_kv_load(const pq2_kv_cache *cache, const int32_t *table,
                int64_t table_stride, int64_t table_width, const int32_t *cu,
                const int32_t *lens, int64_t B, void *k, void *v, int dtype,
                int64_t tokens, void *stream);

/* pq2_attn_decode — attention of the T newest tokens of each of B sequences
 * over the cache, which holds their own keys and values already
 * (pq2_kv_store).  Query head h uses key head h / (q_heads / heads).  With
 * s_j = scale * q . k_j over the positions j < lens[b] - T + t + 1:
 *   out[b][t][h] = sum_j exp(s_j) v_j / sum_j exp(s_j)
 *   lse[b][t][h] = log sum_j exp(s_j)
 * A row that sees no position (lens[b] = 0, or T > lens[b]) gives 0 and -inf.
 * Positions that a row does not see take no part, whatever they hold.
 *   q        (device) dtype PQ2_BF16 or PQ2_F16, element (b, t, h, d) at
 *            b * batch_stride + t * token_stride + h * head_stride + d
 *            (elements); 4-byte aligned, even strides.
 *   cache    of q's dtype, or PQ2_I8.
 *   q_heads  a multiple of cache->heads, at most 256 times it; T 1 .. 64;
 *            B 1 .. 1<<16.
 *   scale    -1e6 .. 1e6.
 *   lens     (device) int32 [B]; below 0 as 0, above 1<<30 as that.
 *   out      (device) dtype [B][T][q_heads][dim], 16-byte aligned.
 *   lse      (device, may be NULL) fp32 [B][T][q_heads].
 *   workspace (device) pq2_attn_decode_workspace_bytes (positions =
 *            table_width * page_size), 16-byte aligned; NULL where that is 0.
 *            Its contents need not be kept between calls.  Calls that may run
 *            at the same time, or that two threads make on one stream (a call
 *            may launch two kernels), need one each.
 * Scores, the softmax and all sums are fp32.  The weights are rounded to the
 * type in which the tensor cores take them (a 16-bit cache: q's; an 8-bit one:
 * fp16, times the value's scale and in units of the row's largest such product),
 * keys and values not at all.  Over a 16-bit cache the sums of n weights times
 * values are in range for values up to 2^119 / n.  A row that sees an infinity
 * or NaN is infinite or NaN in that column.  The order of the sums follows B, T,
 * lens, table_width, the heads and the SM count; the same call gives the same bits.
 * pq2_attn_decode_workspace_bytes returns 0 for short tables and few sequences,
 * which need none, and for invalid arguments. */
size_t pq2_attn_decode_workspace_bytes(int64_t B, int64_t T, int64_t q_heads,
                                       int64_t heads, int64_t dim,
                                       int64_t positions);
int pq2_attn_decode(const void *q, int dtype, int64_t batch_stride,
                    int64_t token_stride, int64_t head_stride, int64_t B,
                    int64_t T, int64_t q_heads, const pq2_kv_cache *cache,
                    const int32_t *table, int64_t table_stride,
                    int64_t table_width, const int32_t *lens, float scale,
                    void *out, float *lse, void *workspace,
                    size_t workspace_bytes, int32_t *dev_status, void *stream);

/* pq2_attn_prefill — attention over packed sequences: rows cu_q[b] ..
 * cu_q[b + 1] of q attend rows cu_k[b] .. cu_k[b + 1] of k and v.  With
 * causal, counted from the ends: row t of n_q sees keys j < n_k - n_q + t + 1
 * (a chunk after what its prompt has so far; n_q = n_k: a whole prompt).
 * out, lse, scale, heads and the rows that see nothing as in pq2_attn_decode.
 *   q, k, v  (device) dtype PQ2_BF16 or PQ2_F16, element (row, head, d) at
 *            row * token_stride + head * head_stride + d; 16-byte aligned,
 *            strides multiples of 8 elements, below 2^39 and not negative.
 *   q_heads  a multiple of heads, at most 128 times it; dim 64, 128 or 256.
 *   q_rows, k_rows  rows of q and of k and v, 1 .. 1<<24 (k_rows may be 0
 *            when k and v are NULL).
 *   cu_q, cu_k (device) int32 [B + 1], not decreasing, B 1 .. 1<<16; values
 *            outside 0 .. rows are taken as the nearest one inside.
 *   out      (device) dtype [q_rows][q_heads][dim], 16-byte aligned; rows
 *            outside every sequence stay as they were, in lse as well.
 *   lse      (device, may be NULL) fp32 [q_rows][q_heads].
 *   workspace (device) pq2_attn_prefill_workspace_bytes, 16-byte aligned, as
 *            in pq2_attn_decode; may be NULL where that is 0.
 * Keys and values that a row does not see take no part, whatever they hold.
 * Rows whose maximum of |scale * q . k| passes 2^23, and rows before a value
 * that is infinite or NaN in the same 128 keys, are computed again one at a time:
 * a row takes about 0.2 us a key then. */
size_t pq2_attn_prefill_workspace_bytes(int64_t B, int64_t q_rows,
                                        int64_t k_rows, int64_t q_heads,
                                        int64_t heads, int64_t dim);
int pq2_attn_prefill(const void *q, int64_t q_token_stride,
                     int64_t q_head_stride, const void *k,
                     int64_t k_token_stride, int64_t k_head_stride,
                     const void *v, int64_t v_token_stride,
                     int64_t v_head_stride, int dtype, int64_t q_rows,
                     int64_t k_rows, int64_t q_heads, int64_t heads,
                     int64_t dim, const int32_t *cu_q, const int32_t *cu_k,
                     int64_t B, float scale, int causal, void *out, float *lse,
                     void *workspace, size_t workspace_bytes,
                     int32_t *dev_status, void *stream);

/* Paths of pq2_debug_group_dots. */
enum { PQ2_PATH_MMV_ADDXOR = 0, PQ2_PATH_MM = 1, PQ2_PATH_MMV_PLANES = 2,
       PQ2_PATH_MM_F8 = 3, PQ2_PATH_MMV_TC = 4 };

/* pq2_debug_group_dots — the exact per-group int32 dots
 * dots[m][n][g] = sum_{k in g} (c_{n,k} - 1) q_{m,k} computed by the SAME
 * device decode and dot code as pq2_mmv with either decoder (paths 0 and 2,
 * q int8 in PQ2_Q_PLANES order, qsum required for path 2, M 1..8) or as
 * pq2_mm (path 1, q fp16 PQ2_Q_F16 and qsum, M >= 1) or pq2_mm_f8 (path 3,
 * q PQ2_Q_F8 and qsum, M >= 1) or pq2_mmv_tc (path 4, q PQ2_Q_MMV16 and
 * its corrections in qsum, M 1..8), for parity checks.
 *   dots (device) int32 [M][N][K/128]. */
int pq2_debug_group_dots(const void *q, const int32_t *qsum,
                         const uint8_t *codes, int64_t M, int64_t N, int64_t K,
                         int path, int32_t *dots, int32_t *dev_status,
                         void *stream);

/* pq2_debug_mm_dots_grouped — the exact partial dots of pq2_mm_grouped
 * (path PQ2_PATH_MM, q PQ2_Q_F16) or pq2_mm_f8_grouped (PQ2_PATH_MM_F8,
 * q PQ2_Q_F8) from the same device code, for parity checks:
 * dots[m][n][j] = sum over k in [j*A, j*A + A) of (c_{n,k} - 1) q_{m,k}.
 *   q from pq2_quantize_act_grouped with the same act_group; M >= 1.
 *   dots (device) int32 [M][N][K / act_group]. */
int pq2_debug_mm_dots_grouped(const void *q, int path, const uint8_t *codes,
                              int64_t M, int64_t N, int64_t K, int act_group,
                              int32_t *dots, int32_t *dev_status,
                              void *stream);

/* pq2_debug_mmv_drop_arrival — a test of the bounded device waits (the
 * status convention above), not a step of the method: pq2_mmv (masked-plane
 * decoder, no flags) in which one consumer warp does not release the first
 * ring stage of its weight pipeline, so the producer's wait for that slot,
 * limited here to wait_limit_cycles SM clocks (1000 .. 2^32), gives up.  The
 * producer then issues no further copy, waits (bounded) until every copy it
 * issued has landed, and tells the consumers to stop; the kernel writes
 * PQ2_ERR_TIMEOUT to *dev_status (required here) and returns.  y is
 * unspecified afterwards; the device and its context stay usable.  Returns
 * PQ2_ERR_SHAPE when (N, K) gives a pipeline whose slots are never reused
 * (nothing to wait for), else as pq2_mmv. */
int pq2_debug_mmv_drop_arrival(const int8_t *q_planes, const float *sx,
                               const int32_t *qsum, const uint8_t *codes,
                               const uint16_t *scales, void *y, int y_dtype,
                               int64_t M, int64_t N, int64_t K,
                               int64_t wait_limit_cycles, int32_t *dev_status,
                               void *stream);

/* pq2_mmv_geometry — the launch geometry pq2_mmv uses for (N, K) on a device
 * with sm_count SMs (host only, no CUDA call): CTAs, threads per CTA,
 * interleaved K splits per row and row count of the largest CTA.  It does
 * not depend on M. Returns PQ2_ERR_SHAPE for invalid shapes. */
int pq2_mmv_geometry(int64_t N, int64_t K, int sm_count, int *ctas,
                     int *threads, int *splits, int *rows_max);

#ifdef __cplusplus
}
#endif
#endif /* PQ2_H */
