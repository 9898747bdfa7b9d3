/*
 * lowbit.h -- C ABI of liblowbit: matrix products over group-scaled binary
 * {-1,+1} and ternary {-1,0,+1} weights on AMD Instinct MI355X (gfx950).
 *
 * Pages cited, by title (a citation names the page's tag and a section of it
 * in the page's own words):
 *   [RM] richmindsetzone.com: "瀏覽器生圖技術內幕：1-bit diffusion 點樣將 3GB
 *        模型塞入 WebGPU？"
 *   [KC] kongchang.com: "三值权重压缩：27B模型缩至6GB，可在浏览器本地运行"
 *   [OB] ainewscove.com: "我开源了 OpenBonsai：把你自己的 BF16 模型与微调压缩成约
 *        2 GB 的三值 GGUF"
 *   [XH] best.xiaohu.ai: "PrismMLが27BモデルをiPhoneに押し込んだ。しかも頭の良さは
 *        ほぼ落ちていない"
 *
 * What is computed:
 *   - Each weight is a sign (binary) or one of {-1,0,+1} (ternary), and every
 *     group of weights shares one FP16 scale ([RM] section "1-bit 嘅數學：
 *     點解唔爆鑊？"; effective widths 1.125 bits binary, 1.71 ternary).
 *   - The group holds 128 weights, one FP16 scale each ([OB], the method list
 *     of the paragraph "工作原理").
 *   - Multiplying by -1/0/+1 is an add or a sign flip ([KC] section
 *     "精度保留了多少"); a binary product can be done with XOR + popcount
 *     ([RM] section "1-bit 嘅數學：點解唔爆鑊？", the paragraph comparing
 *     binary and ternary).
 *   - Batch-1 decode streams every weight once per token and is bound by
 *     memory bandwidth; prefill is a dense contraction ([XH] sections
 *     "ローカル27Bを阻む第一の壁：「1語生成するたびに全身を運び直す」" and
 *     "速度は二層：低ビット搬送と、CUDA上の草稿加速").
 *
 * Dense (unpacked) meaning of the operands, shared by every entry point:
 *   W       [N][K] weights, row n = output feature, k = reduction index.
 *   codes   int8 [N][K] row-major: binary in {-1,+1}, ternary in {-1,0,+1}.
 *   scales  IEEE binary16 bits, uint16 [N][G], G = K/128; group g of row n
 *           covers k in [128g, 128g+128).  W[n][k] = scale[n][k/128]*code[n][k].
 *           There is no zero point.  Scales must be finite (any sign, 0 ok).
 *   X       [M][K] activations, row-major.  Y = X * W^T, Y is [M][N].
 *   K must be a positive multiple of 128; N, M >= 1.
 *
 * Every pointer is caller-owned device memory unless stated.  Every call is
 * asynchronous on `stream` (a hipStream_t passed as void*, NULL = the null
 * stream) on the current device.  Argument errors are returned synchronously
 * before any HIP call.  A launch failure returns LOWBIT_E_HIP.  No entry
 * point waits for the GPU except lowbit_chain_status, lowbit_chain_destroy
 * and lowbit_release_workspaces, which say so.
 *
 * Streams, workspaces and graphs.  lowbit_gemv, lowbit_gemm, lowbit_gemm_mxfp4,
 * lowbit_attention_kv8, lowbit_attention_kv8_prefix, lowbit_kv8_fork and
 * lowbit_kv8_compact use a device workspace that the library owns, one
 * per (device, stream).  Calls on one stream are ordered and share it; calls on
 * different streams never share one.  A call that needs more than its stream's workspace holds allocates a
 * larger one (hipMalloc, which may synchronize the device as HIP does) and
 * keeps the smaller one allocated until lowbit_release_workspaces, because
 * kernels already queued, and graphs captured earlier, may still use it; no
 * call waits on the stream.  A stream that is being captured into a HIP graph
 * cannot grow its workspace: such a call returns LOWBIT_E_NOMEM, so reserve
 * the workspace first (lowbit_workspace_bytes + lowbit_reserve_workspace, or
 * one eager call of the largest captured product on that stream;
 * the calls beyond products have a ..._workspace call each).
 * A captured graph keeps the workspace address it was captured with; replaying it is
 * valid until lowbit_release_workspaces.  Replays of graphs captured on one
 * stream must run in order on one stream (they share its workspace).  The
 * kernels leave the workspace's counters as they found them, so a replay
 * needs no reset.  No call records a memset into a capture.
 *
 * =====================  PACKED LAYOUT (gfx950)  ===========================
 * Rows are tiled in row-blocks of 16 (NB = ceil(N/16), rows >= N are padding
 * with code 0 / +1 and scale 0).  Inside a row-block, row r = n % 16 and the
 * 128 weights of a group are split over four quarters q = 0..3; the pair
 * (r, q) is the lane L = r + 16q of a 64-wide wavefront.  Quarter q of a
 * group holds 32 weights in slots i = 0..31; slot i of quarter q is the
 * weight at k = 128g + KMAP(q, i) with
 *     KMAP(q, i) = 64*(q & 1) + 16*(q >> 1) + 32*(i >> 4) + (i & 15).
 * (This is the order in which the fp4 B operand of the gfx950
 * 16x16x128 f8f6f4 MFMA consumes k, so one lane's 32 weights are one MFMA
 * fragment.)
 *
 * LOWBIT_BINARY (1 bit / weight).  One 32-bit word per (row, group, quarter);
 *   bit b of the word holds slot  i = 8*(3 - (b & 3)) + (b >> 2),  bit value
 *   1 means -1 and 0 means +1.  Words are stored as
 *     word[((rb * GQ + g/4) * 64 + L) * 4 + (g % 4)],   GQ = ceil(G/4),
 *   so a wavefront reading one 16-byte vector per lane reads 1 KiB contiguous
 *   (16 rows x 4 groups).  Code bytes: NB * GQ * 1024.
 *
 * LOWBIT_TERNARY_2BIT (2 bits / weight, bit-sliced).  Two words P0, P1 per
 *   (row, group, quarter).  Each weight has a "nonzero" bit z and a "negative"
 *   bit s (code = z * (1 - 2s); z = 0 with s = 1 is reserved and never
 *   written).  For slot i = 8j + p (j = 0..3, p = 0..7):
 *     j = 0: P0 bit 4p+1 = z, P0 bit 4p+3 = s      j = 1: P0 bit 4p = z, P0 bit 4p+2 = s
 *     j = 2: P1 bit 4p+1 = z, P1 bit 4p+3 = s      j = 3: P1 bit 4p = z, P1 bit 4p+2 = s
 *   Words are stored as
 *     word[((rb * GP + g/2) * 64 + L) * 4 + 2*(g % 2) + t],  t = 0 (P0), 1 (P1),
 *   GP = ceil(G/2).  Code bytes: NB * GP * 1024.
 *
 * LOWBIT_TERNARY_BASE3 (5 trits / byte, 1.625 bits / weight).  Trit
 *   t = code + 1 in {0,1,2}; a byte holding trits t_0..t_{d-1} has value
 *   sum t_e * 3^e (t_0 is the least-significant digit).  Groups are handled
 *   in octets o = g/8 (GO = ceil(G/8)).  Lane L of octet o owns 52 bytes
 *   B[0..51] covering the 8 groups j = 0..7 (g = 8o + j) of its quarter:
 *     slots 0..29 of group j -> bytes 6j .. 6j+5, slot i in byte 6j + i/5,
 *                                digit i % 5;
 *     slots 30, 31 of group j -> byte 48 + j/2, digits 2*(j%2) + (i-30).
 *   (Bytes 0..47 hold 5 trits, bytes 48..51 hold 4.)  An octet block of a
 *   row-block is 3328 bytes: for s = 0..2 the 1024 bytes at 1024s hold
 *   B[16s .. 16s+15] of lane L at offset 1024s + 16L, and the 256 bytes at
 *   3072 hold B[48..51] of lane L at 3072 + 4L.  Block (rb, o) starts at
 *   byte (rb * GO + o) * 3328.  Code bytes: NB * GO * 3328.  Byte values
 *   >= 243 (>= 81 in bytes 48..51) are invalid.
 *
 * Scales, all formats: fp16 bits stored as
 *     scale[((rb * GQ + g/4) * 16 + r) * 4 + (g % 4)],
 *   i.e. 128 bytes per (row-block, 4 groups).  Scale bytes: NB * GQ * 128.
 *   Padding groups (g >= G) and padding rows hold code 0 (+1 binary) and
 *   scale 0.
 *
 * Bits per weight when N % 16 == 0 and G % 8 == 0: binary 1 + 0.125 = 1.125,
 * ternary 2-bit 2.125, ternary base-3 1.625 + 0.125 = 1.75 (all at or above
 * the information bound log2(3) + 0.125 = 1.70996 for ternary).
 * ========================================================================= */
#ifndef LOWBIT_H
#define LOWBIT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LOWBIT_ABI_VERSION 3

enum lowbit_status {
  LOWBIT_OK = 0,
  LOWBIT_E_NULL = -1,        /* a required pointer is NULL                    */
  LOWBIT_E_SHAPE = -2,       /* K % 128 != 0 (MXFP4: % 32), a size < 1 or too
                                large                                         */
  LOWBIT_E_ALIGN = -3,       /* pointer not aligned as documented             */
  LOWBIT_E_UNSUPPORTED = -4, /* format / dtype combination not provided       */
  LOWBIT_E_BADCODE = -5,     /* reserved for callers that check the flag     */
  LOWBIT_E_HIP = -6,         /* a HIP runtime call or launch failed           */
  LOWBIT_E_NOMEM = -7,       /* the library could not allocate its workspace  */
  LOWBIT_E_TOO_LARGE = -8    /* lowbit_gemv_noalloc: the product needs more
                                scratch than the library's static array       */
};

enum lowbit_format {
  LOWBIT_BINARY = 1,
  LOWBIT_TERNARY_2BIT = 2,
  LOWBIT_TERNARY_BASE3 = 3
};

enum lowbit_dtype {
  LOWBIT_F32 = 1,   /* IEEE binary32                                          */
  LOWBIT_BF16 = 2,  /* bfloat16 bits (uint16)                                 */
  LOWBIT_I8 = 3,    /* int8 with a float scale: value = scale * q             */
  LOWBIT_SIGN1 = 4, /* packed sign bits, K/8 bytes per row, bit k%8 of byte
                       k/8 (LSB first); bit 1 means -alpha, 0 means +alpha     */
  LOWBIT_I32 = 5,   /* int32 output of the exact integer paths               */
  LOWBIT_MXFP4 = 6  /* packed MXFP4 activations (lowbit_gemm_mxfp4 only)     */
};

/* ABI version of the loaded library (LOWBIT_ABI_VERSION).  Library
 * bookkeeping; no passage of the pages. */
int lowbit_abi_version(void);

/* Static text for a status code; never NULL.  Library bookkeeping. */
const char* lowbit_status_str(int status);

/* Bytes of the packed code and scale buffers for an N x K matrix in `fmt`
 * (layout above; storage of [RM] section "1-bit 嘅數學：點解唔爆鑊？" and
 * the ternary width of [KC] section "精度保留了多少").  Host-only, no HIP
 * call.  Errors: E_NULL, E_SHAPE, E_UNSUPPORTED. */
int lowbit_packed_bytes(int fmt, int64_t N, int64_t K, size_t* code_bytes,
                        size_t* scale_bytes);

/* Pack dense codes [N][K] (int8) and scales [N][G] (fp16 bits) into the
 * layout above, writing every byte of pcodes/pscales (padding included).
 * Group-scaled weights of [RM] section "1-bit 嘅數學：點解唔爆鑊？" with the
 * group of 128 of [OB] paragraph "工作原理".
 * pcodes and pscales must be 16-byte aligned.  Codes outside the format's
 * value set are counted into *bad_code_count (device int32, atomically
 * added; pass NULL to skip); their packed value is unspecified.  The count is
 * not cleared by the call. */
int lowbit_pack(int fmt, int64_t N, int64_t K, const int8_t* codes,
                const uint16_t* scales, void* pcodes, void* pscales,
                int32_t* bad_code_count, void* stream);

/* Inverse of lowbit_pack (same passages): writes codes [N][K] and scales
 * [N][G].  A weight
 * decoded from a reserved 2-bit pattern or an out-of-range base-3 byte is
 * written as 0 and counted (one per weight) into *bad_code_count (device
 * int32, atomically added, nullable). */
int lowbit_unpack(int fmt, int64_t N, int64_t K, const void* pcodes,
                  const void* pscales, int8_t* codes, uint16_t* scales,
                  int32_t* bad_code_count, void* stream);

/* Per-row absmax int8 quantization of bf16 X [M][K] (the pages fix no
 * activation format; an 8-bit activation is the plainest reading of the
 * integer product of [KC] section "精度保留了多少".  fp32 arithmetic, no
 * fused operations): a = max_k |x|; if a == 0 then q = 0 and s_x = 0, else
 * inv = 127.0f / a, q = clamp(rint(x * inv), -127, 127) with ties to even,
 * s_x = a / 127.0f.  Writes Q [M][K] and s_x [M]. */
int lowbit_quantize_act_i8(int64_t M, int64_t K, const uint16_t* X_bf16,
                           int8_t* Q, float* s_x, void* stream);

/* Batch-1 product y[n] = sum_k W[n][k] * x[k] for n < N: the per-token
 * product of decode ([XH] section "ローカル27Bを阻む第一の壁：「1語生成する
 * たびに全身を運び直す」") over the weights of [RM] section "1-bit 嘅數學：
 * 點解唔爆鑊？".
 *   x_dtype F32 / BF16: x holds K values.
 *   x_dtype I8: x holds K int8 q; the result is multiplied by x_scale.
 *   x_dtype SIGN1 (binary weights only, K <= 393216): x holds K/8 bytes of
 *     sign bits; the result is multiplied by x_scale (alpha).  Runs as one
 *     launch without the workspace.
 *   y_dtype F32 or BF16 (round to nearest even).  y_dtype I32 is allowed
 *   only for x_dtype I8 / SIGN1 with pscales == NULL: y = exact integer
 *   sum_k code * q (or the signed bit agreement count), x_scale ignored.
 * Alignment: pcodes, pscales, x 16 bytes; y 4 bytes.  Uses the stream's
 * workspace (see "Streams, workspaces and graphs" above; E_NOMEM if it must
 * grow during capture or cannot be allocated). */
int lowbit_gemv(int fmt, int64_t N, int64_t K, const void* pcodes,
                const void* pscales, int x_dtype, const void* x, float x_scale,
                int y_dtype, void* y, void* stream);

/* Allocation-free lowbit_gemv, for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc).  Arguments, results and errors as lowbit_gemv, which it
 * equals bit for bit (the same kernels), plus LOWBIT_E_TOO_LARGE.  Instead of
 * the per-stream workspace it uses a static device array of 4 MiB per GPU
 * (held until the process ends), enough for every product whose workspace
 * (lowbit_workspace_bytes with M = 1) is at most 4 MiB -- every N <= 65536
 * with K <= 65536, and the 27B-class layer shapes; larger products return
 * LOWBIT_E_TOO_LARGE before any launch.  It calls no hipMalloc or hipFree.
 * The first call on a device looks the array up and clears its counter
 * block with a small kernel on `stream`.  All calls on one GPU share the
 * array: calls that may overlap in time on one GPU (different streams, or
 * replays of graphs holding this call on different streams) race and give
 * wrong results; order them on one stream.  Sign activations (SIGN1) use no
 * scratch. */
int lowbit_gemv_noalloc(int fmt, int64_t N, int64_t K, const void* pcodes,
                        const void* pscales, int x_dtype, const void* x, float x_scale,
                        int y_dtype, void* y, void* stream);

/* Product Y[m][n] = sum_k W[n][k] * X[m][k] for m < M, n < N: the dense
 * contraction of prefill and of a denoising step ([XH] section "速度は二層：
 * 低ビット搬送と、CUDA上の草稿加速"; [RM] section "1-bit 嘅數學：點解唔爆鑊？").
 * M <= 16 / (activation split terms) runs the small-M GEMV path (8 rows for
 * binary bf16, 5 for ternary bf16, 8 for int8).
 *   x_dtype BF16: X bf16 [M][K], fp32 accumulation.
 *   x_dtype I8: X int8 [M][K] (e.g. from lowbit_quantize_act_i8) with
 *     x_scales[M] (device fp32); per 128-group integer sums are exact in int32
 *     and Y[m][n] = x_scales[m] * sum_g scale[n][g] * A[m][n][g].
 *     y_dtype I32 requires pscales == NULL and returns sum_g A[m][n][g].
 *   x_dtype SIGN1 (batched sign activations, any weight format): X holds
 *     K/8 bytes of sign bits per row (bit k%8 of byte k/8, 1 = negative) and
 *     x_scales[M] the per-row magnitude alpha_m (device fp32), so that
 *     x[m][k] = alpha_m (-1)^bit.  Per group D[m][n][g] = sum_k code * sign
 *     is an exact integer (for binary weights 128 - 2 popcount(w XOR x) per
 *     group, the XOR + popcount product of [RM] section "1-bit 嘅數學：點解唔爆鑊？") and Y = alpha_m sum_g scale[n][g] D[m][n][g];
 *     y_dtype I32 requires pscales == NULL and returns sum_g D (x_scales
 *     ignored).
 *   y_dtype F32 or BF16 (or I32 as above).
 * K <= 2^36 (E_SHAPE beyond).  Alignment: pcodes, pscales, X, Y 16 bytes.
 * Uses the stream's workspace as lowbit_gemv does. */
int lowbit_gemm(int fmt, int64_t M, int64_t N, int64_t K, const void* pcodes,
                const void* pscales, int x_dtype, const void* X,
                const float* x_scales, int y_dtype, void* Y, void* stream);

/* Workspace management (library bookkeeping, no passage of the pages).
 * lowbit_workspace_bytes: host-only; *bytes = the workspace a lowbit_gemm
 *   call with these arguments needs (M = 1: also bounds lowbit_gemv's).
 *   Errors: E_NULL, E_UNSUPPORTED, E_SHAPE.
 * lowbit_reserve_workspace: makes the stream's workspace on the current
 *   device hold at least `bytes` (grows it as a product call would; E_NOMEM
 *   during capture or when hipMalloc fails).  Call before capturing.
 * lowbit_release_workspaces: waits for each device that holds one, then frees
 *   every workspace, current and retired, of every stream and device.  Call
 *   it only when no queued kernel and no graph that will be replayed uses one;
 *   later calls allocate afresh.  Errors: E_HIP. */
int lowbit_workspace_bytes(int fmt, int64_t M, int64_t N, int64_t K, int x_dtype,
                           size_t* bytes);
int lowbit_reserve_workspace(size_t bytes, void* stream);
int lowbit_release_workspaces(void);

/* ---- chains of batch-1 products in one persistent launch ------------------
 * Batch-1 decode streams every weight of every layer once per token and is
 * bound by memory bandwidth, so the cost that matters is the one paid per
 * token ([XH] sections "ローカル27Bを阻む第一の壁：「1語生成するたびに全身を運び
 * 直す」" and "速度は二層：低ビット搬送と、CUDA上の草稿加速").
 * A chain runs a fixed list of batch-1 products of one weight format as one
 * cooperative launch whose workgroups stream the weights of later products
 * while earlier ones finish.  Stage i with wait_prev != 0 reads its x only
 * after every output of stage i-1 has been written (so x may be, or be
 * computed from, an earlier stage's y); its weights may be read earlier.
 * Outputs are written with device-coherent stores. */
typedef struct lowbit_gemv_stage {
  int fmt;              /* any lowbit_format, equal for all stages                */
  int64_t N, K;         /* W is N x K, K % 128 == 0                                */
  const void* pcodes;   /* packed codes (16-byte aligned)                          */
  const void* pscales;  /* packed fp16 scales (16-byte aligned)                    */
  const void* x;        /* rows x K activations of the chain's x_dtype (row-major,
                           16-byte aligned; rows = 1 unless created with rows)      */
  void* y;              /* rows x N outputs of the chain's y_dtype (4-byte aligned) */
  int wait_prev;        /* 1: read x only after stage i-1 is complete (then rows
                           times K times the x element size must stay below 2^31
                           bytes)                                                  */
  int epilogue;         /* LOWBIT_EPI_NONE or LOWBIT_EPI_SILU_MUL (see below)      */
} lowbit_gemv_stage;

/* Stage epilogues.  LOWBIT_EPI_SILU_MUL: the stage is a fused gate/up
 * product of a gated FFN (the compressed models keep their base model's
 * architecture: [KC] section "三值权重（Ternary）到底做了什么") whose N rows (N % 16 == 0) are ordered so that in every 16-row
 * block rows 0..7 are gate rows 8b..8b+7 and rows 8..15 the up rows
 * 8b..8b+7; y then receives N/2 values z[i] = silu(g[i]) u[i],
 * silu(v) = v / (1 + e^-v), computed in fp32 from the fp32 products and
 * stored in the chain's y_dtype -- the input of the down projection, which a
 * later stage (wait_prev = 1, K = N/2, x = this y when y_dtype equals
 * x_dtype) reads. */
#define LOWBIT_EPI_NONE 0
#define LOWBIT_EPI_SILU_MUL 1

typedef struct lowbit_chain lowbit_chain; /* opaque */

/* Plan a chain of n_stages products on the current device: copies the stage
 * list (pointers are used as given at every run), allocates the chain's
 * device descriptors, counters and split-K partial sums (owned by the chain
 * until lowbit_chain_destroy).  x_dtype F32 or BF16; y_dtype F32 or BF16.
 * Errors: E_NULL, E_SHAPE, E_ALIGN, E_UNSUPPORTED, E_HIP, E_NOMEM. */
int lowbit_chain_create(int n_stages, const lowbit_gemv_stage* stages, int x_dtype,
                        int y_dtype, lowbit_chain** chain);

/* The same with `rows` activation rows per product (1 <= rows <= 8 for BF16 x,
 * <= 4 for F32 x; every stage takes rows x K activations and writes rows x N
 * outputs): a small-M chain such as one pass that verifies rows - 1 drafted
 * tokens and the next one through every product of a model ([XH] section
 * "速度は二層：低ビット搬送と、CUDA上の草稿加速": drafts are checked by the
 * target model in one pass).  The SiLU-mul epilogue needs rows == 1.  Errors as
 * lowbit_chain_create (E_SHAPE for rows out of range). */
int lowbit_chain_create_rows(int n_stages, const lowbit_gemv_stage* stages, int64_t rows,
                             int x_dtype, int y_dtype, lowbit_chain** chain);

/* Run every stage once, asynchronously on `stream`.  Runs of one chain must
 * not overlap (they share its counters); run it on one stream at a time. */
int lowbit_chain_run(lowbit_chain* chain, void* stream);

/* Synchronous: *failed_waits != 0 if a stage ever gave up waiting for its
 * predecessor (a bounded wait of about a second; its outputs are then not
 * meaningful).  Never expected when runs do not overlap. */
int lowbit_chain_status(lowbit_chain* chain, int* failed_waits);

/* Frees the chain's device memory (synchronizes the device first).  Library
 * bookkeeping. */
int lowbit_chain_destroy(lowbit_chain* chain);

/* Data-free quantizer front end (the signed Hadamard rotation and the
 * FP16 scale per 128 weights of the method list of [OB] paragraph
 * "工作原理"; its calibrated GPTQ step needs data and is
 * not part of it).  From bf16 weights W [N][K] writes dense codes [N][K]
 * (int8, the input of lowbit_pack) and fp16 scales [N][K/128].  Per row and
 * group of 128: v = W * d (signs d[K], int8 +-1; signs == NULL: no
 * rotation), u = H v with H[i][j] = (-1)^popcount(i & j), t = u r with
 * r = 1/sqrt(128) as an fp64 number, s16 = fp16((sum |u| / 128) r) (round to
 * nearest even); ternary formats: c = +1 if t > s16/2, -1 if t < -s16/2,
 * else 0; binary: c = -1 if t < 0 else +1; s16 = 0 gives codes 0 / +1.
 * Computed in fp64 (sums exact while a group's magnitudes span less than
 * 2^38, so the result does not depend on the summation order).  Rotated
 * weights expect rotated activations (lowbit_rotate_act with the same
 * signs).  Alignment: W, signs and codes 16 bytes, scales 2 bytes.
 * Errors: E_NULL, E_UNSUPPORTED, E_SHAPE, E_ALIGN, E_HIP. */
int lowbit_quantize_weights(int fmt, int64_t N, int64_t K, const uint16_t* W_bf16,
                            const int8_t* signs, int8_t* codes, uint16_t* scales,
                            void* stream);

/* Activations for rotated weights ([OB] paragraph "工作原理", the signed
 * Hadamard rotation): per row of bf16 X [M][K] and block of 128,
 * X_rot = H (d * x) / sqrt(128) in fp32 (signs as given to
 * lowbit_quantize_weights), so that products with the rotated weights
 * equal those with the original ones.  Output fp32 [M][K].
 * Errors: E_NULL, E_SHAPE, E_ALIGN, E_HIP. */
int lowbit_rotate_act(int64_t M, int64_t K, const uint16_t* X_bf16, const int8_t* signs,
                      float* X_rot, void* stream);

/* Measurement helper, not part of the matrix-product path (the bandwidth
 * bound of [XH] section "ローカル27Bを阻む第一の壁：「1語生成するたびに全身を
 * 運び直す」"): reads the
 * `bytes` (a positive multiple of 16) at src once with 16-byte streaming
 * loads spread over the whole device and XORs the data into *out (device
 * uint32, caller-initialised), so the sustained HBM read rate can be timed
 * beside the decode kernels.  src 16-byte aligned, out 4-byte aligned.
 * Errors: E_NULL, E_SHAPE, E_ALIGN, E_HIP. */
int lowbit_hbm_read_probe(const void* src, int64_t bytes, uint32_t* out, void* stream);

/* =====================  MXFP4  ===========================================
 * Matrices in the OCP microscaling format MXFP4: every 32 consecutive values
 * of a row share one power of two 2^e (E8M0: the byte e + 127; 255 is NaN)
 * and each value is an e2m1 code (bit 3 the sign, magnitudes 0, 0.5, 1, 1.5,
 * 2, 3, 4, 6), 4.25 bits a value.  Not from the pages: the 4-bit format that
 * gfx950's matrix cores take directly, for the layers that one or two bits
 * lose too much of, with lowbit_gemm's meaning of W, X and Y.
 *
 * Packed layout.  Rows in row-blocks of 16 (NB = ceil(rows/16)), k in groups
 * of 128 (G = ceil(K/128)), groups in quads (GQ = ceil(G/4)); lane L = r + 16 q
 * owns row r = n % 16 and block q of a group, k = 128 g + 32 q + i.
 *   code byte  ((rb * G + g) * 64 + L) * 16 + i/2 holds values i (low nibble)
 *              and i + 1 for even i;                       NB * G * 1024 bytes
 *   scale byte ((rb * GQ + g/4) * 64 + L) * 4 + g % 4;    NB * GQ * 256 bytes
 * Padding rows, blocks and groups hold codes 0 and scale 127.
 * ====================================================================== */

/* Bytes of the packed code and scale buffers of a rows x K matrix (K a
 * positive multiple of 32; rows, K <= 2^30, rows * K <= 2^38).  Host-only.
 * Errors: E_NULL, E_SHAPE. */
int lowbit_mxfp4_bytes(int64_t rows, int64_t K, size_t* code_bytes, size_t* scale_bytes);

/* Row-major MXFP4 (codes [rows][K/2], two values a byte with the even k in the
 * low nibble; scales [rows][K/32]) into the packed layout, every byte of it
 * (padding included).  codes, pcodes and pscales 16-byte aligned.
 * Errors: E_NULL, E_SHAPE, E_ALIGN, E_HIP. */
int lowbit_pack_mxfp4(int64_t rows, int64_t K, const uint8_t* codes, const uint8_t* scales,
                      void* pcodes, void* pscales, void* stream);

/* Quantizes X [rows][K] (x_dtype F32 or BF16, rows x_stride elements apart)
 * into the packed layout: per block a = max |x|, e = max(floor(log2 a) - 2,
 * -127), codes x / 2^e rounded to nearest even and limited to 6; a zero block
 * has e = -127; a block that holds an infinity or a NaN has scale 255 and
 * codes 0, so every product that reads it is NaN.  values, if not NULL,
 * receives what the codes stand for, [rows][K] in x_dtype.  Weights (once) and
 * activations (per call) alike.  X, pcodes, pscales, values 16-byte aligned,
 * x_stride >= K and rows 16-byte aligned; the buffers do not overlap.  rows <=
 * 2^30 - 64.
 * Errors: E_NULL, E_UNSUPPORTED, E_SHAPE, E_ALIGN, E_HIP. */
int lowbit_quantize_mxfp4(int64_t rows, int64_t K, int x_dtype, const void* X, int64_t x_stride,
                          void* pcodes, void* pscales, void* values, void* stream);

/* Y[m][n] = sum_k W[n][k] X[m][k], W MXFP4, for any M >= 1 (one token to
 * whole prompts), fp32 accumulation, Y [M][N] in y_dtype F32 or BF16.
 *   x_dtype BF16: X bf16, rows x_stride elements apart (>= K, a multiple of
 *     8); the products of each pair are exact in fp32.  Weights below 2^-126
 *     in magnitude may count as 0, of 2^128 and more (bytes 253, 254, which
 *     lowbit_quantize_mxfp4 does not write) as infinities.
 *   x_dtype MXFP4: X packed codes and x_pscales its packed scales
 *     (lowbit_quantize_mxfp4 of the M x K activations); x_stride ignored.
 * All pointers 16-byte aligned.  N <= 2^26, ceil(M/128) * ceil(N/128) <= 2^23
 * (BF16 X: < 2^23).
 * Sums are added in a fixed order: repeated calls give the same bits.  Uses
 * the stream's workspace as lowbit_gemm does where K is split over workgroups
 * (lowbit_gemm_mxfp4_workspace: its bytes, 0 where none; reserve it before a
 * capture).
 * Errors: E_NULL, E_UNSUPPORTED, E_SHAPE, E_ALIGN, E_NOMEM, E_HIP. */
int lowbit_gemm_mxfp4(int64_t M, int64_t N, int64_t K, const void* pcodes, const void* pscales,
                      int x_dtype, const void* X, int64_t x_stride, const void* x_pscales, int y_dtype,
                      void* Y, void* stream);
int lowbit_gemm_mxfp4_workspace(int64_t M, int64_t N, int64_t K, int x_dtype, size_t* bytes);

/* =====================  8-bit paged cache and attention  ==================
 * Between the q/k/v and the o product of a layer ([XH] section "ローカル27Bを
 * 阻む第一の壁：「1語生成するたびに全身を運び直す」": what a token re-reads):
 * keys and values as e4m3 codes in pages of 16, 32, 64 or 128 tokens, one
 * power of two per page and head for the keys and one for the values (bytes
 * e + 127, 0 .. 247 where tokens lie).  Head sizes 64, 128, 256.
 *   k_codes  [n_pages][kv_heads][page_tokens][head_dim]
 *   v_codes  [n_pages][kv_heads][head_dim][page_tokens]   (transposed)
 *   k_scales, v_scales  [n_pages][kv_heads]
 * All memory is the caller's. */
typedef struct lowbit_kv8 {
  int64_t n_pages;
  int page_tokens, kv_heads, head_dim;
  void* k_codes;      /* 16-byte aligned */
  void* v_codes;      /* 16-byte aligned */
  uint8_t* k_scales;
  uint8_t* v_scales;
} lowbit_kv8;

/* The sequences of one call.  Sequence b holds kv_lens[b] tokens, the call's
 * new ones last; token t lies in page page_table[b][t /
 * page_tokens].  Its new tokens are rows q_starts[b] .. q_starts[b + 1] - 1 of
 * the queries (keys, values); q_starts NULL: max_q rows each, in order.
 * max_q and max_kv bound the new tokens and the lengths of any one sequence;
 * they size the launch, so keep them close.  The arrays are read on the
 * device when the call runs (a graph's replay sees their new contents).  What
 * they hold can not lead a kernel outside the buffers: lengths are cut to
 * max_kv, rows to total_q and max_q, and tokens in a page whose index is not
 * in 0 .. n_pages - 1 are not written and not seen, counted in *bad_pages
 * (device int32, atomically added, once or more for each; not cleared; NULL
 * to skip).  A sequence may be empty (length 0 or no new tokens). */
typedef struct lowbit_kv8_batch {
  int64_t n_seqs;
  const int32_t* page_table; /* device [n_seqs][table_width] */
  int64_t table_width;
  const int32_t* kv_lens;    /* device [n_seqs] */
  const int32_t* q_starts;   /* device [n_seqs + 1], or NULL */
  int64_t total_q;           /* rows in all (q_starts NULL: n_seqs * max_q) */
  int64_t max_q;
  int64_t max_kv;            /* at most table_width * page_tokens */
  int32_t* bad_pages;        /* device, or NULL */
} lowbit_kv8_batch;

/* Writes the new tokens' keys and values (dtype BF16 or F32, [total_q]
 * [kv_heads][head_dim] with tokens k_stride / v_stride elements apart, so they
 * may lie in a fused projection's output) into the cache.  Per page and head:
 * e(a) = the smallest e >= -127 with a <= 448 2^e, a the largest finite
 * magnitude of the page's new tokens; a page that already holds tokens of the
 * sequence keeps e = max(e_old, e(a)), and where that rises its earlier codes
 * are rescaled (times 2^(e_old - e), rounded to nearest even: exact above
 * e4m3's subnormal range).  code = x / 2^e to nearest even, infinities to
 * +-448, NaN to NaN; at e = 120, where larger codes would stand for infinities,
 * codes end at +-240.  Bytes behind a sequence's last token stay as they were.
 * A page that receives tokens must belong to one sequence of the batch and
 * stand in its table once (full pages may be shared by any number).  New tokens
 * that lie before the sequence's start (more of them than kv_lens) are not
 * written.  Writing the same tokens again changes nothing.  K, V 16-byte
 * aligned, rows 16-byte aligned; n_seqs * kv_heads * (pages that max_q tokens
 * can touch) <= 2^23, below it where page_tokens * head_dim is 16384 and below
 * 2^22 where it is 32768.
 * Errors: E_NULL, E_UNSUPPORTED (dtype, page_tokens, head_dim), E_SHAPE,
 * E_ALIGN, E_HIP. */
int lowbit_kv8_append(const lowbit_kv8* cache, const lowbit_kv8_batch* batch, int dtype, const void* K,
                      const void* V, int64_t k_stride, int64_t v_stride, void* stream);

/* O = softmax(softmax_scale Q K^T) V over the cache: query row i of sequence b
 * stands at position p = kv_lens[b] - (new tokens) + i and sees tokens
 * j < kv_lens[b] with j <= p (causal != 0) and j > p - window (window > 0).
 * Q [total_q][q_heads][head_dim] bf16, q_heads a multiple of kv_heads (head h
 * reads key head h / (q_heads / kv_heads)), tokens q_stride elements apart; O
 * likewise, o_stride apart.  lse, if not NULL, receives [total_q][q_heads] the
 * natural logarithm of the softmax sum.  A row that sees no token gets O = 0
 * and lse = -infinity (so does one whose scores are all -infinity, which takes
 * an infinity in Q); what lies in tokens a row does not see (NaN codes too)
 * does not reach it.  With causal == 0 the cache may hold another sequence (an
 * encoder's states) of its own length.  Sums and
 * statistics are fp32.  Weights enter the second product as bf16: in two terms
 * (16 bits) in calls of few rows a sequence and key head, such as single
 * tokens, rounded once (8 bits, as O) in calls of many (with heads of 256 and at
 * most 16 rows also where n_seqs * kv_heads * ceil(max_kv / 64) <= 512).  Results do not depend
 * on the order in which workgroups run.  Rows of sequences behind the last
 * q_starts entry are not written.
 * One call runs one kernel for all its sequences, chosen by max_q * q_heads /
 * kv_heads and max_kv: long contexts with single tokens and prompts of many
 * rows are faster as two calls, each with a max_q of its own.
 * max_q * q_heads / kv_heads <= 2^30, and n_seqs * kv_heads * ceil(max_q *
 * q_heads / kv_heads / 128) <= 2^22 (calls of few rows: any).  O does not overlap
 * Q or the cache.  Keys and values below 2^-126 in magnitude may count as 0.
 * Q, O 16-byte aligned, strides multiples of 8.  Uses the stream's workspace
 * (lowbit_attention_kv8_workspace bytes) as lowbit_gemv does; reserve it
 * before a capture.  A smaller call may need more, as its tiles are cut into more
 * parts: ask for each shape that is captured.
 * Errors: E_NULL, E_UNSUPPORTED (page_tokens, head_dim, softmax_scale
 * log2(e) not finite), E_SHAPE, E_ALIGN, E_NOMEM, E_HIP. */
int lowbit_attention_kv8(const lowbit_kv8* cache, const lowbit_kv8_batch* batch, int64_t q_heads,
                         const uint16_t* Q_bf16, int64_t q_stride, float softmax_scale, int causal,
                         int64_t window, uint16_t* O_bf16, int64_t o_stride, float* lse, void* stream);
int lowbit_attention_kv8_workspace(const lowbit_kv8* cache, const lowbit_kv8_batch* batch, int64_t q_heads,
                                   size_t* bytes);

/* Sequences that begin with the same tokens (answers to one prompt, prompts behind
 * one instruction): group g's sequences are seq_starts[g] .. seq_starts[g + 1] - 1
 * of the batch (no sequence in two groups), so that its rows lie in order, and the tokens they share are
 * the first lens[g] of the pages in page_table's row g.  seq_starts NULL: n_seqs
 * / n_groups each, in order.  max_seqs and max_len bound the sequences of any one
 * group and its lengths; they size the launch, so keep them close.  Arrays are read
 * on the device, as those of lowbit_kv8_batch, and can not lead a kernel outside the
 * buffers either: lengths are cut to max_len, sequences to the batch's.  q_starts may
 * leave rows between the sequences (more than max_q for one: its first max_q are its
 * tokens); such rows, and sequences beyond max_seqs, cost time and change no result. */
typedef struct lowbit_kv8_prefix {
  int64_t n_groups;
  const int32_t* page_table; /* device [n_groups][table_width] */
  int64_t table_width;
  const int32_t* lens;       /* device [n_groups], 0 allowed */
  const int32_t* seq_starts; /* device [n_groups + 1], or NULL */
  int64_t max_seqs;          /* seq_starts NULL: ignored */
  int64_t max_len;           /* at most table_width * page_tokens */
} lowbit_kv8_prefix;

/* lowbit_attention_kv8 for sequences behind shared prefixes: every row of a
 * sequence sees all tokens of its group's prefix, and of its own tokens what a
 * row of lowbit_attention_kv8 sees (window 0).  The batch describes the own tokens
 * alone: kv_lens counts them, page_table holds their pages (its table_width is the
 * distance of two rows, so it may point into rows that begin with the prefix's
 * pages: page_table + k, kv_lens less k * page_tokens, max_kv at most
 * (table_width - k) * page_tokens).  A prefix need not end with a page.  Each
 * prefix is read once for all rows of its group, as a prompt's tokens are (in tiles
 * of 128 or 256 rows; 16 or 32 where the group has few); one row's sums over prefix
 * and own tokens are joined in fp32.  Weights enter the second product in two bf16
 * terms wherever max_q * q_heads / kv_heads is at most 64; with more rows they may be
 * rounded once.  Sequences of no group have no
 * prefix.  Rows of a sequence behind its first max_q are left as they were,
 * should q_starts have more.  Everything else is as lowbit_attention_kv8 says, limits included, for the
 * groups too (their rows: min(total_q, max_seqs * max_q)); max_len + max_kv <=
 * 2^30; total_q * q_heads * (head_dim + 4) <= 2^38.
 * Needs workspace in every case (lowbit_attention_kv8_prefix_workspace: with the
 * same heads no more for a call with smaller bounds, sequences, groups or rows).
 * Errors: as lowbit_attention_kv8. */
int lowbit_attention_kv8_prefix(const lowbit_kv8* cache, const lowbit_kv8_prefix* prefix,
                                const lowbit_kv8_batch* batch, int64_t q_heads, const uint16_t* Q_bf16,
                                int64_t q_stride, float softmax_scale, int causal, uint16_t* O_bf16,
                                int64_t o_stride, float* lse, void* stream);
int lowbit_attention_kv8_prefix_workspace(const lowbit_kv8* cache, const lowbit_kv8_prefix* prefix,
                                          const lowbit_kv8_batch* batch, int64_t q_heads, size_t* bytes);

/* What lowbit_attention_kv8_prefix runs for these arguments (host-only): the
 * bounds decide, so this shows what a loose one costs. */
typedef struct lowbit_kv8_prefix_plan {
  int launches;     /* 1: prefix and own tokens together; 2: the groups over their prefixes, then the sequences */
  int tile_rows;    /* of the first: 16 or 32 read by each wave from the cache, or 128 or 256 of a workgroup */
  int tile_parts;   /* that a tile's tokens are cut into at most; 0: as equal shares of all tokens fall */
  int whole_tiles;  /* of a key head that are not cut (launches 1, tile_rows from 128) */
  int own_rows;     /* launches 2: tile_rows and tile_parts of the second; else 0 */
  int own_parts;
  int weight_terms; /* bf16 terms of a weight, 1 or 2 */
} lowbit_kv8_prefix_plan;
int lowbit_attention_kv8_prefix_launches(const lowbit_kv8* cache, const lowbit_kv8_prefix* prefix,
                                         const lowbit_kv8_batch* batch, int64_t q_heads, lowbit_kv8_prefix_plan* plan);

/* =====================  heads of queries and keys  ========================
 * Between a fused q/k/v product and lowbit_kv8_append / lowbit_attention_kv8
 * (or a diffusion transformer's attention): each head's norm and its rotation
 * by the token's position, in one pass over queries and keys. */
typedef struct lowbit_rope {
  int64_t tokens;
  int head_dim;             /* D, a multiple of 8, at most 256 */
  int n_pairs;              /* rotated pairs, a multiple of 4, 2 n_pairs <= D; 0: no rotation */
  int adjacent;             /* 0: pairs (i, i + n_pairs), else (2 i, 2 i + 1), of the first 2 n_pairs dims */
  int n_axes;               /* at least 1 */
  const int32_t* positions; /* device [n_axes][pos_stride], of any sign */
  int64_t pos_stride;       /* at least tokens (n_axes = 1: ignored) */
  const double* freqs;      /* device [n_pairs], radians for one step of the position */
  const int32_t* pair_axis; /* device [n_pairs], each pair's axis; NULL: axis 0.  A pair whose axis
                               is not in 0 .. n_axes - 1 is not rotated */
} lowbit_rope;

/* For every token and head x of Q [tokens][q_heads][D] and K [tokens][kv_heads]
 * [D] (x_dtype F32 or BF16): y = x w / sqrt(mean of x^2 + eps) with w =
 * q_weight / k_weight [D] (fp32; NULL: y = x, w of 1 + v is the caller's to
 * add); then each pair (a, b) becomes (a cos t - b sin t, b cos t + a sin t),
 * t = positions[axis][token] freqs[pair], reduced in fp64 (off by 2^-51 of the
 * angle).  Everything else is fp32 (squares beyond its range overflow, below it they are 0),
 * rounded once to y_dtype F32 or BF16.  Q, K and the outputs lie with tokens
 * the given strides (in elements) apart, heads contiguous: a fused projection's
 * output as it is.  Q_out may be Q and K_out may be K where x_dtype = y_dtype
 * and the strides agree; otherwise outputs share no byte with an input or each
 * other (refused; rows may lie between another tensor's).  K NULL (kv_heads 0):
 * queries alone.
 * Several axes (time, height, width): each pair turns by one of them.
 * All of Q, K, Q_out, K_out 16-byte aligned, strides multiples of 8; freqs 8 bytes,
 * positions, pair_axis and weights 4.  tokens <= 2^30, q_heads, kv_heads <= 2^16,
 * tokens * stride <= 2^46.
 * eps finite, >= 0.
 * Errors: E_NULL, E_UNSUPPORTED (types, head_dim, n_pairs, eps, overlaps),
 * E_SHAPE, E_ALIGN, E_HIP. */
int lowbit_qk_norm_rope(const lowbit_rope* rope, int x_dtype, const void* Q, int64_t q_heads, int64_t q_stride,
                        const float* q_weight, const void* K, int64_t kv_heads, int64_t k_stride,
                        const float* k_weight, float eps, int y_dtype, void* Q_out, int64_t qo_stride, void* K_out,
                        int64_t ko_stride, void* stream);

/* =====================  pages of the cache  ===============================
 * Who holds which page, decided on the device, so that a step whose new
 * sequences are chosen there (beams, samples) needs no copy to the host.
 * A sequence of n tokens holds the first ceil(n / page_tokens) pages of its
 * table row.  refs [n_pages] counts the holders of each page (a store of prompts
 * may hold pages too); 0: free.  The caches of one call are a model's layers:
 * the same n_pages and page_tokens, one set of tables for all (heads and sizes
 * of head may differ).  Arrays are int32 on the device; the library keeps
 * nothing between calls, and results do not depend on the order in which
 * workgroups run. */

/* The next batch from this one: new sequence i takes over parents[i]'s tokens
 * (0 .. n_seqs - 1; any other number: none) and gets room for grow[i] tokens
 * more (grow NULL: max_grow each; cut to 0 .. max_grow).  new_lens[i] counts them
 * already, as lowbit_kv8_append and lowbit_attention_kv8 want it.  Sequences with
 * several children are forked, those with one go on, those with none are freed.
 *   - Pages are shared.  A partly filled one that new tokens will be written to
 *     stays with the first of the children that will, if nobody else holds it;
 *     every other one gets a copy (codes and exponents, of all layers).
 *   - Copies and further pages are the free ones (after the old batch's pages
 *     were given back) in ascending order, for the children in turn.
 *   - new_refs = refs without the old batch's holders, with the new one's.
 *   - new_table rows end with -1 behind their pages.  A page number outside
 *     0 .. n_pages - 1 in a row becomes -1 and counts for nobody.
 * Where pages do not suffice, *failed is the number that lacks (else 0), no page
 * is written, and the other outputs do not stand: the inputs do.  A child that
 * has more than new_width pages, or 2^30 tokens, is cut to them: its new_lens is less
 * than its parent's and grow together, and appending as many tokens as it asked for
 * would overwrite its last ones, in pages that others may hold.
 * lowbit_kv8_fork_cut is the same call and counts the children that were cut in
 * *cut (device int32, set, not added; NULL to skip).
 * n_seqs 0 (nothing yet: parents are none) and n_new 0 (everything freed) are
 * fine, their arrays may be NULL.  Outputs overlap no input and not each other
 * (refused; that they lie outside the caches is the caller's care); new_refs 16-byte aligned.
 * n_pages <= 2^26; n_seqs, n_new <= 2^20; table widths <= 2^26; max_grow <= 2^30;
 * n_new * (max_grow / page_tokens + 2) <= 2^30, n_new * ceil(new_width / 1024) < 2^24 - 2048;
 * n_caches <= 4096.  One workgroup plans: time grows with n_new and with the
 * entries of the sequences that do not go on as one.  Uses the stream's workspace
 * (lowbit_kv8_fork_workspace bytes); reserve it before a capture.
 * Errors: E_NULL, E_UNSUPPORTED (page_tokens, head_dim, overlaps), E_SHAPE, E_ALIGN,
 * E_NOMEM, E_HIP. */
int lowbit_kv8_fork(const lowbit_kv8* caches, int64_t n_caches, int64_t n_seqs, const int32_t* page_table,
                    int64_t table_width, const int32_t* kv_lens, const int32_t* refs, int64_t n_new,
                    const int32_t* parents, const int32_t* grow, int64_t max_grow, int32_t* new_table,
                    int64_t new_width, int32_t* new_lens, int32_t* new_refs, int32_t* failed, void* stream);
int lowbit_kv8_fork_cut(const lowbit_kv8* caches, int64_t n_caches, int64_t n_seqs, const int32_t* page_table,
                        int64_t table_width, const int32_t* kv_lens, const int32_t* refs, int64_t n_new,
                        const int32_t* parents, const int32_t* grow, int64_t max_grow, int32_t* new_table,
                        int64_t new_width, int32_t* new_lens, int32_t* new_refs, int32_t* failed, int32_t* cut,
                        void* stream);
int lowbit_kv8_fork_workspace(int64_t n_pages, int page_tokens, int64_t n_caches, int64_t n_seqs, int64_t n_new,
                              int64_t max_grow, size_t* bytes);

/* Closes the cache up: with *live pages in use (refs > 0), the k-th page in use
 * at or behind *live moves to the k-th free page before it, so that the pages
 * from *live on are free (in all layers).  remap [n_pages] receives where each
 * page is now (-1: it was free), for tables that are not in the call; new_table
 * is page_table so rewritten (-1 behind a sequence's pages), new_refs the counts.
 * n_seqs may be 0 (the tables then NULL).  Outputs as lowbit_kv8_fork's.  Limits as
 * lowbit_kv8_fork, and ceil(n_pages / 1024) + n_seqs * ceil(table_width / 1024) <
 * 2^24 - 2048.  Uses the stream's workspace (lowbit_kv8_compact_workspace bytes).
 * Errors as lowbit_kv8_fork. */
int lowbit_kv8_compact(const lowbit_kv8* caches, int64_t n_caches, int64_t n_seqs, const int32_t* page_table,
                       int64_t table_width, const int32_t* kv_lens, const int32_t* refs, int32_t* new_table,
                       int32_t* new_refs, int32_t* remap, int32_t* live, void* stream);
int lowbit_kv8_compact_workspace(int64_t n_pages, int64_t n_caches, size_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* LOWBIT_H */
