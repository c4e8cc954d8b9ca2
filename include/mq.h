/*
 * mq.h -- C ABI of the microscaling-quantized convolution library for MI355X (gfx950).
 *
 * The library implements the hot path of MicroQonv (onedev.kr paper digest "합성곱 텐서 레이아웃
 * 재배열로 마이크로스케일링 양자화의 이중 연산과 메모리 이동을 줄이는 MicroQonv"): every convolution
 * tensor is quantized exactly once, before any im2col expansion, into a channel-batch-first layout
 * with 4x4 square-block scaling, and all three convolution GEMMs run directly on the quantized
 * data with the im2col matrix formed on chip only.
 *
 * Conventions shared by every call:
 *   - Every pointer argument named *_dev, and every pointer inside mq_qtensor, is device memory
 *     on the current HIP device. The caller allocates and owns all memory; the library
 *     allocates nothing and keeps no state between calls (the one exception is the device
 *     array of mq_conv_backward_noalloc, part of the library's code object on each GPU).
 *   - Every call is asynchronous on `stream` (0 = the null stream). The return value reports
 *     only synchronous host-side argument validation and launch errors; no call synchronizes.
 *   - Data problems are not reported through the status: a tensor containing NaN or Inf
 *     quantizes to T = NaN, scales 0x7F (E4M3 NaN) and codes 0, and any convolution that
 *     consumes it produces NaN.
 *   - Calls that overlap on one stream are ordered; calls on different streams that share a
 *     buffer race.
 */
#ifndef MQ_H
#define MQ_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MQ_OK = 0,
    MQ_ERR_ARG = 1,         /* null pointer, non-positive size, unknown enum value */
    MQ_ERR_SHAPE = 2,       /* tensor shapes do not match the convolution / each other */
    MQ_ERR_UNSUPPORTED = 3, /* valid request outside the implemented set (see each call) */
    MQ_ERR_WORKSPACE = 4,   /* workspace missing or smaller than required */
    MQ_ERR_LAUNCH = 5       /* a kernel launch failed (hipGetLastError) */
} mq_status;

/* Element formats (onedev.kr digest, sections "How it differs" and "How it is used"):
 * NVFP4 = E2M1 elements, NVFP6 = E2M3 elements; both with one E4M3 scale per 4x4 square and one
 * fp32 tensor scale. */
typedef enum { MQ_NVFP4 = 4, MQ_NVFP6 = 6 } mq_format;

/* Role of a quantized tensor; fixes the meaning of its four dimensions (o0, o1, r, s):
 *   MQ_ROLE_ACT    activation X          (Hin,  Win,  Cin,  N)   channel-batch-first
 *   MQ_ROLE_WEIGHT weight W              (Kh,   Kw,   Cout, Cin) one Cout x Cin matrix per tap
 *   MQ_ROLE_GRAD   output gradient G_Y   (Hout, Wout, Cout, N)   channel-batch-first */
typedef enum { MQ_ROLE_ACT = 0, MQ_ROLE_WEIGHT = 1, MQ_ROLE_GRAD = 2 } mq_role;

/* Element rounding: round-to-nearest-even (weights, activations) or stochastic (gradients),
 * per the onedev.kr digest, section "How it differs". */
typedef enum { MQ_RNE = 0, MQ_SR = 1 } mq_round;

/*
 * A quantized tensor: logical shape [o0][o1][r][s] (s fastest), cut into 4x4 squares over
 * (r, s) with r and s zero-padded up to multiples of 4. With R4 = ceil(r/4), S4 = ceil(s/4):
 *   square t = ((i0*o1 + i1)*R4 + ir/4)*S4 + is/4, element e = (ir%4)*4 + is%4;
 *   codes:  NVFP4 8 bytes per square, element e = nibble (e%2) of byte 8t + e/2 (low first);
 *           NVFP6 12 bytes per square, element e = bits [6e, 6e+6) of the little-endian
 *           96-bit word at byte 12t;
 *           code bits: NVFP4 s|ee|m (bias 1), NVFP6 s|ee|mmm (bias 1); padded slots are 0;
 *   scales: 1 byte per square, E4M3 s|eeee|mmm (bias 7, subnormals, 0x7E = 448, 0x7F = NaN);
 *   tscale: one fp32, the tensor scale T.
 * Value of an element: decode(code) * decode(scale) * T.
 * fmt and role hold mq_format / mq_role values. codes must be 16-byte aligned, scales and tscale
 * 4-byte aligned (device allocations are); other pointers give MQ_ERR_ARG. The convolutions may
 * read the up to 3 bytes that follow the last scale byte in its aligned 4-byte word (never
 * beyond it) and ignore them.
 */
typedef struct {
    int32_t o0, o1, r, s;
    int32_t fmt;
    int32_t role;
    uint8_t *codes;
    uint8_t *scales;
    float *tscale;
} mq_qtensor;

/* One 2-D convolution (groups 1, dilation 1, zero padding). Output size
 * Hout = (H + 2*pad_h - Kh)/stride_h + 1, Wout likewise. */
typedef struct {
    int32_t N, Cin, H, W, Cout, Kh, Kw, stride_h, stride_w, pad_h, pad_w;
} mq_conv;

/* Human-readable name of a status code (static string, never NULL). */
const char *mq_status_str(mq_status st);

/* Bytes needed for the code stream / scale bytes of a quantized tensor with the given logical
 * shape and format: squares * (8 | 12) and squares * 1. Returns 0 for invalid arguments. */
size_t mq_codes_bytes(int32_t o0, int32_t o1, int32_t r, int32_t s, int32_t fmt);
size_t mq_scales_bytes(int32_t o0, int32_t o1, int32_t r, int32_t s);

/*
 * Tensor-amax workspace (mq_quantize, and optionally the relayouts): device scratch of at least
 * MQ_QUANTIZE_WS_BYTES bytes, 4-byte aligned. Word 0 holds the number P of partial maxima,
 * words 1..P the partials (max |x| per part of the tensor, as fp32 bit patterns). Calls on one
 * stream may share a workspace; calls that can run concurrently must not.
 */
#define MQ_QUANTIZE_WS_BYTES 8192

/*
 * mq_relayout_cbf: NCHW fp32 <-> channel-batch-first fp32.
 * Channel-batch-first X_{Cin,N} (onedev.kr digest, section "How it works"): for each pixel
 * (h, w) all channels and all batch elements are contiguous; here [H][W][C][N], N fastest.
 *   inverse = 0: dst[h][w][c][n] = src[n][c][h][w]
 *   inverse = 1: dst[n][c][h][w] = src[h][w][c][n]
 * src_dev, dst_dev: N*C*H*W floats each, must not overlap.
 * amax_ws_dev: null, or a tensor-amax workspace that receives the partial maxima of the tensor
 *          (the relayout reads every element anyway), so that mq_quantize of dst_dev can pass
 *          MQ_QUANTIZE_AMAX_READY and skip its own pass over the tensor. amax_ws_bytes is
 *          ignored when amax_ws_dev is null.
 * Errors: MQ_ERR_ARG for null pointers, non-positive sizes or a misaligned workspace;
 *         MQ_ERR_WORKSPACE for a workspace below MQ_QUANTIZE_WS_BYTES; MQ_ERR_UNSUPPORTED for
 *         C > 65535.
 */
mq_status mq_relayout_cbf(const float *src_dev, float *dst_dev, int32_t N, int32_t C, int32_t H,
                          int32_t W, int32_t inverse, uint32_t *amax_ws_dev, size_t amax_ws_bytes,
                          hipStream_t stream);

/*
 * mq_relayout_weight: OIHW fp32 <-> tap-major [Kh][Kw][Cout][Cin] fp32, the layout of the 2-D
 * weight matrix W_{fCout,Cin} (Cout x Kh*Kw*Cin; onedev.kr digest, section "How it differs")
 * with one Cout x Cin block per tap.
 *   inverse = 0: dst[kh][kw][co][ci] = src[co][ci][kh][kw];  inverse = 1: the reverse.
 * amax_ws_dev, amax_ws_bytes: as for mq_relayout_cbf.
 * Errors: MQ_ERR_ARG for null pointers, non-positive sizes or a misaligned workspace;
 *         MQ_ERR_WORKSPACE for a workspace below MQ_QUANTIZE_WS_BYTES.
 */
mq_status mq_relayout_weight(const float *src_dev, float *dst_dev, int32_t Cout, int32_t Cin,
                             int32_t Kh, int32_t Kw, int32_t inverse, uint32_t *amax_ws_dev,
                             size_t amax_ws_bytes, hipStream_t stream);

/* mq_quantize flag: amax_ws_dev already holds the partial maxima of this tensor's values (from a
 * relayout that wrote src_dev, earlier on the same stream); the amax pass is skipped. */
#define MQ_QUANTIZE_AMAX_READY 1u

/*
 * mq_quantize: quantize one fp32 tensor, exactly once, with the NVFP4 / NVFP6 recipe of the
 * onedev.kr digest, section "How it differs":
 *   amax = max |x| over the tensor;
 *   T    = amax / (448 * Emax)                              (Emax = 6 for E2M1, 7.5 for E2M3)
 *   per 4x4 square: B = CastE4M3(max|x_i| / (T * Emax))    (nearest-even, saturating at 448)
 *   per element:    code = Round(x_i / (B * T))            (RNE, or SR for rnd = MQ_SR)
 * All scale arithmetic is IEEE fp32 in the written order. Stochastic rounding rounds |q| up
 * from its lower grid neighbour lo to hi iff u16 < ((|q|-lo)/(hi-lo)) * 65536, with u16 the
 * (e%2)-th 16-bit half of word (e%8)/2 of Philox4x32-10(counter = (2t + e/8, 0, 0, 0),
 * key = seed) for element e of square t. Codes keep the sign bit of x. Squares with B = 0 hold
 * codes 0; a tensor with T = 0 holds scales 0 and codes 0.
 *
 * src_dev: the tensor as dense fp32 [o0][o1][r][s] (for activations and gradients this is the
 *          channel-batch-first layout).
 * dst:     host struct describing the destination; dst->codes, dst->scales, dst->tscale are
 *          device buffers of mq_codes_bytes / mq_scales_bytes / 4 bytes.
 * amax_ws_dev / amax_ws_bytes: a tensor-amax workspace (overwritten unless flags has
 *          MQ_QUANTIZE_AMAX_READY, then read).
 * flags:   0 or MQ_QUANTIZE_AMAX_READY.
 * Errors: MQ_ERR_ARG (null pointer, bad enum or flag, non-positive dims, misaligned pointer),
 *         MQ_ERR_WORKSPACE (amax_ws_dev null or smaller than MQ_QUANTIZE_WS_BYTES),
 *         MQ_ERR_UNSUPPORTED (2^31 squares or more).
 */
mq_status mq_quantize(const float *src_dev, const mq_qtensor *dst, int32_t rnd, uint64_t seed,
                      uint32_t *amax_ws_dev, size_t amax_ws_bytes, uint32_t flags,
                      hipStream_t stream);

/*
 * mq_quantize_nchw: quantize an NCHW fp32 activation or output gradient straight into its
 * channel-batch-first quantized layout (onedev.kr digest, section "How it works": the layout
 * change happens before quantization, which then runs once, section "How it differs"). The
 * codes, scales and T are those of mq_relayout_cbf (inverse = 0) followed by mq_quantize on its
 * output, with the same recipe, rounding and random draws (square t of the channel-batch-first
 * tensor), without writing the fp32 channel-batch-first copy: an amax pass over src_dev (unless
 * flags has MQ_QUANTIZE_AMAX_READY), then one quantizing pass that reads NCHW and writes squares.
 * src_dev: N*C*H*W floats [n][c][h][w] with (H, W, C, N) = (dst->o0, dst->o1, dst->r, dst->s).
 * dst:     role MQ_ROLE_ACT or MQ_ROLE_GRAD, buffers as for mq_quantize.
 * amax_ws_dev / amax_ws_bytes / flags: as for mq_quantize (the partial maxima may come from any
 *          layout of the same values).
 * Errors: MQ_ERR_ARG (null pointer, bad enum or flag, non-positive dims, misaligned pointer),
 *         MQ_ERR_SHAPE (role MQ_ROLE_WEIGHT), MQ_ERR_WORKSPACE (as for mq_quantize),
 *         MQ_ERR_UNSUPPORTED (the source zero-padded to whole squares, 16*ceil(N/4)*ceil(C/4)*H*W
 *         floats, reaches 2^31 bytes).
 */
mq_status mq_quantize_nchw(const float *src_dev, const mq_qtensor *dst, int32_t rnd, uint64_t seed,
                           uint32_t *amax_ws_dev, size_t amax_ws_bytes, uint32_t flags,
                           hipStream_t stream);

/* Source order of a batched quantization job (mq_quant_job.layout). */
typedef enum {
    MQ_SRC_DENSE = 0, /* [o0][o1][r][s] as stored by the quantized layout (mq_quantize) */
    MQ_SRC_NCHW = 1,  /* NCHW activation or gradient, dst (o0, o1, r, s) = (H, W, C, N) */
    MQ_SRC_OIHW = 2   /* OIHW weight, dst (o0, o1, r, s) = (Kh, Kw, Cout, Cin) */
} mq_source_layout;

#define MQ_QUANTIZE_BATCH_MAX 4

/* One tensor of mq_quantize_batch: what mq_quantize (MQ_SRC_DENSE), mq_quantize_nchw
 * (MQ_SRC_NCHW) or mq_quantize_weight (MQ_SRC_OIHW) would take, with its own workspace. */
typedef struct {
    const float *src;     /* device fp32 source in the order `layout` names */
    int32_t layout;       /* mq_source_layout */
    int32_t rnd;          /* mq_round */
    uint64_t seed;        /* SR seed (ignored for MQ_RNE) */
    uint32_t flags;       /* 0 or MQ_QUANTIZE_AMAX_READY */
    mq_qtensor dst;       /* destination (device buffers) */
    uint32_t *amax_ws;    /* this tensor's amax workspace, device, 4-byte aligned */
    size_t amax_ws_bytes; /* >= MQ_QUANTIZE_WS_BYTES */
} mq_quant_job;

/*
 * mq_quantize_batch: quantize up to MQ_QUANTIZE_BATCH_MAX tensors of one format with one amax
 * launch and one quantizing launch, each exactly as the single-tensor call for its layout would
 * (same recipe of the onedev.kr digest, section "How it differs"; same codes, scales, T and
 * stochastic draws). Batching lets a small tensor share the launches of a large one: the
 * forward pass of a layer quantizes X (NCHW) and W (OIHW) together.
 * jobs: host array of njobs (1..MQ_QUANTIZE_BATCH_MAX) job descriptions; every job needs its own
 *       amax workspace (the same pointer twice is MQ_ERR_ARG).
 * Errors: MQ_ERR_ARG (null pointer, bad enum or flag, misaligned pointer, non-positive dims,
 *         shared workspace), MQ_ERR_SHAPE (formats differ between jobs; an NCHW job with a
 *         weight destination or an OIHW job with another role), MQ_ERR_WORKSPACE (a workspace
 *         missing or below MQ_QUANTIZE_WS_BYTES), MQ_ERR_UNSUPPORTED (more than
 *         MQ_QUANTIZE_BATCH_MAX jobs, 2^31 squares or more, or an NCHW source that reaches 2^31
 *         bytes once zero-padded to whole squares).
 */
mq_status mq_quantize_batch(const mq_quant_job *jobs, int32_t njobs, hipStream_t stream);

/*
 * mq_quantize_weight: quantize an OIHW fp32 weight straight into the tap-major quantized layout
 * [Kh][Kw][Cout][Cin] of the 2-D weight matrix (onedev.kr digest, section "How it differs"),
 * with the same amax, T, square scales and codes as mq_relayout_weight followed by mq_quantize
 * on its output (the recipe above), without writing the fp32 tap-major copy. A weight of at
 * most 65536 elements takes one launch (every workgroup reduces the whole tensor's amax itself,
 * then quantizes its share of the squares); a larger one runs the amax pass into amax_ws_dev and
 * a quantizer that gathers from OIHW.
 * w_oihw_dev: Cout*Cin*Kh*Kw floats, [co][ci][kh][kw].
 * dst:     role MQ_ROLE_WEIGHT with (o0, o1, r, s) = (Kh, Kw, Cout, Cin).
 * rnd, seed: as for mq_quantize.
 * amax_ws_dev / amax_ws_bytes: a tensor-amax workspace (overwritten; untouched for a small
 *          weight, but required either way).
 * Errors: MQ_ERR_ARG (null pointer, bad enum, misaligned pointer), MQ_ERR_SHAPE (dst role not
 *         MQ_ROLE_WEIGHT), MQ_ERR_WORKSPACE (workspace null or smaller than
 *         MQ_QUANTIZE_WS_BYTES), MQ_ERR_UNSUPPORTED (2^31 squares or more).
 */
mq_status mq_quantize_weight(const float *w_oihw_dev, const mq_qtensor *dst, int32_t rnd,
                             uint64_t seed, uint32_t *amax_ws_dev, size_t amax_ws_bytes,
                             hipStream_t stream);

/*
 * mq_conv_fwd: forward GEMM Y = W . X' (onedev.kr digest, section "How it differs") with the
 * im2col matrix X' formed on chip from the channel-batch-first quantized X (section "How it
 * works"):
 *   Y[ho][wo][co][n] = T_W * T_X * sum_{kh,kw,ci} Wq[kh][kw][co][ci]
 *                                               * Xq[ho*sh - ph + kh][wo*sw - pw + kw][ci][n]
 * (zero outside the input), accumulated in fp32 from exact fp16 (or bf16) products.
 * x: MQ_ROLE_ACT tensor of shape (H, W, Cin, N); w: MQ_ROLE_WEIGHT tensor (Kh, Kw, Cout, Cin);
 * same format. y_dev: fp32 channel-batch-first [Hout][Wout][Cout][N], fully overwritten.
 * Errors: MQ_ERR_ARG, MQ_ERR_SHAPE (dims or formats disagree with p), MQ_ERR_UNSUPPORTED.
 */
mq_status mq_conv_fwd(const mq_conv *p, const mq_qtensor *x, const mq_qtensor *w, float *y_dev,
                      hipStream_t stream);

/* Bytes of device workspace mq_conv_wgrad needs for this convolution (0 on invalid input). */
size_t mq_wgrad_workspace_bytes(const mq_conv *p);

/*
 * mq_conv_wgrad: weight-gradient GEMM G_W = G_Y . X'^T (onedev.kr digest, section "How it
 * differs"), reading the quantized G_Y and X along their batch-contiguous direction:
 *   G_W[kh][kw][co][ci] = T_G * T_X * sum_{ho,wo,n} Gq[ho][wo][co][n]
 *                                               * Xq[ho*sh - ph + kh][wo*sw - pw + kw][ci][n]
 * gy: MQ_ROLE_GRAD (Hout, Wout, Cout, N); x: MQ_ROLE_ACT (H, W, Cin, N); same format.
 * gw_dev: fp32 [Kh][Kw][Cout][Cin], fully overwritten.
 * ws_dev / ws_bytes: device scratch of at least mq_wgrad_workspace_bytes(p) bytes (split-K
 * partial sums; summed in a fixed order, so results are deterministic).
 * Errors: MQ_ERR_ARG, MQ_ERR_SHAPE, MQ_ERR_WORKSPACE, MQ_ERR_UNSUPPORTED.
 */
mq_status mq_conv_wgrad(const mq_conv *p, const mq_qtensor *gy, const mq_qtensor *x,
                        float *gw_dev, void *ws_dev, size_t ws_bytes, hipStream_t stream);

/*
 * mq_conv_dgrad: input-gradient GEMM G_X' = W^T . G_Y (onedev.kr digest, section "How it
 * differs") with the col2im sum fused, so the Kh*Kw-inflated G_X' never exists in memory:
 *   G_X[h][w][ci][n] = T_W * T_G * sum_{kh,kw,co} Wq[kh][kw][co][ci] * Gq[ho][wo][co][n]
 *       over (ho, wo) with ho*sh - ph + kh = h and wo*sw - pw + kw = w.
 * w: MQ_ROLE_WEIGHT (Kh, Kw, Cout, Cin); gy: MQ_ROLE_GRAD (Hout, Wout, Cout, N); same format.
 * gx_dev: fp32 channel-batch-first [H][W][Cin][N], fully overwritten.
 * Errors: MQ_ERR_ARG, MQ_ERR_SHAPE, MQ_ERR_UNSUPPORTED.
 */
mq_status mq_conv_dgrad(const mq_conv *p, const mq_qtensor *w, const mq_qtensor *gy,
                        float *gx_dev, hipStream_t stream);

/*
 * mq_conv_backward: both gradients of one convolution, G_W as mq_conv_wgrad and G_X as
 * mq_conv_dgrad compute them (same values, bit for bit), for the backward pass that needs both.
 * For the tuned shapes the weight gradient's split sum runs inside the input-gradient launch, on
 * workgroups of its own (when the CUs that launch leaves idle finish it in a few passes), instead
 * of as a launch between the two GEMMs. gw_dev, gx_dev and ws_dev must not overlap.
 * w: MQ_ROLE_WEIGHT (Kh, Kw, Cout, Cin); gy: MQ_ROLE_GRAD (Hout, Wout, Cout, N);
 * x: MQ_ROLE_ACT (H, W, Cin, N); one format.
 * gw_dev: fp32 [Kh][Kw][Cout][Cin]; gx_dev: fp32 [H][W][Cin][N]; both fully overwritten.
 * ws_dev / ws_bytes: as for mq_conv_wgrad (mq_wgrad_workspace_bytes(p)).
 * Errors: MQ_ERR_ARG, MQ_ERR_SHAPE, MQ_ERR_WORKSPACE, MQ_ERR_UNSUPPORTED.
 */
mq_status mq_conv_backward(const mq_conv *p, const mq_qtensor *w, const mq_qtensor *gy,
                           const mq_qtensor *x, float *gw_dev, float *gx_dev, void *ws_dev,
                           size_t ws_bytes, hipStream_t stream);

/*
 * mq_conv_fwd_amax: mq_conv_fwd (same Y, bit for bit) whose epilogue also writes the tensor-amax
 * partial maxima of |Y| into amax_ws_dev, in the format mq_quantize reads with
 * MQ_QUANTIZE_AMAX_READY. When Y is the next tensor to be quantized (the next layer's activation
 * with nothing elementwise in between), mq_quantize of Y (channel-batch-first, dense source)
 * then skips its own read of Y: the tensor amax of the NVFP4 / NVFP6 recipe (onedev.kr digest,
 * section "How it differs": T = max|X| / (448 * Emax)) comes from the producer of the tensor.
 * The workgroups of the tuned kernels each write one partial; other shapes run the amax pass over
 * Y after the convolution (same partials format, same result).
 * amax_ws_dev / amax_ws_bytes: a tensor-amax workspace (MQ_QUANTIZE_WS_BYTES, 4-byte aligned),
 *          overwritten; pass it to mq_quantize of Y with MQ_QUANTIZE_AMAX_READY, later on the same
 *          stream.
 * Errors: as mq_conv_fwd; MQ_ERR_WORKSPACE (workspace null or below MQ_QUANTIZE_WS_BYTES),
 *         MQ_ERR_ARG (misaligned workspace).
 */
mq_status mq_conv_fwd_amax(const mq_conv *p, const mq_qtensor *x, const mq_qtensor *w,
                           float *y_dev, uint32_t *amax_ws_dev, size_t amax_ws_bytes,
                           hipStream_t stream);

/*
 * mq_conv_backward_amax: mq_conv_backward (same G_W and G_X, bit for bit) whose input-gradient
 * epilogue also writes the tensor-amax partial maxima of |G_X| into gx_amax_ws_dev (format as for
 * mq_conv_fwd_amax). G_X is the output gradient of the layer before when nothing elementwise sits
 * between, so its stochastic quantization (mq_quantize, MQ_QUANTIZE_AMAX_READY) skips its amax
 * pass.
 * gx_amax_ws_dev / gx_amax_ws_bytes: a tensor-amax workspace, overwritten.
 * Errors: as mq_conv_backward; MQ_ERR_WORKSPACE / MQ_ERR_ARG for the amax workspace as above.
 */
mq_status mq_conv_backward_amax(const mq_conv *p, const mq_qtensor *w, const mq_qtensor *gy,
                                const mq_qtensor *x, float *gw_dev, float *gx_dev, void *ws_dev,
                                size_t ws_bytes, uint32_t *gx_amax_ws_dev, size_t gx_amax_ws_bytes,
                                hipStream_t stream);

/*
 * Size of the device array that mq_conv_backward_noalloc keeps the weight gradient's split-K
 * partial sums in (one array per GPU, held until the process ends).
 */
#define MQ_NOALLOC_SCRATCH_BYTES (32u << 20)

/*
 * mq_conv_backward_noalloc: mq_conv_backward (same kernels, same G_W and G_X bit for bit) for
 * callers that cannot allocate memory: code under HIP graph capture, tight serving loops and
 * harnesses that forbid hipMalloc. The weight gradient's split-K partial sums go to a
 * library-owned device array of MQ_NOALLOC_SCRATCH_BYTES on the current device instead of a
 * caller workspace; the call allocates nothing (no hipMalloc, no allocating library routine).
 * The caller still provides every input and output as for mq_conv_backward, on the current HIP
 * device (stream must belong to it).
 * Every call on one GPU shares that GPU's array: calls that can overlap on one GPU (different
 * streams, or threads without ordering between their calls) race and must not be issued;
 * calls ordered on one stream are fine.
 * Errors: as mq_conv_backward; MQ_ERR_UNSUPPORTED when mq_wgrad_workspace_bytes(p) exceeds
 *         MQ_NOALLOC_SCRATCH_BYTES; MQ_ERR_LAUNCH when the device array cannot be located.
 */
mq_status mq_conv_backward_noalloc(const mq_conv *p, const mq_qtensor *w, const mq_qtensor *gy,
                                   const mq_qtensor *x, float *gw_dev, float *gx_dev,
                                   hipStream_t stream);

/* ---- attention over an 8-bit key/value cache ------------------------------------------------
 *
 * A decoder's serving path around one paged cache: attention over whole prompts
 * (mq_attn_prompt), the quantizing write of their keys and values (mq_kv_append), attention of
 * the newly generated tokens over the cache (mq_attn_cached), and the eviction of the cached
 * tokens that received the least attention (mq_kv_evict). The cache follows the library's block
 * scaling: E4M3 codes, one scale per block of tokens and head.
 */

/* Element type of queries, keys, values and outputs. */
typedef enum { MQ_F16 = 1, MQ_BF16 = 2 } mq_dtype;

/* Tokens that share one scale of the cache. */
#define MQ_KV_BLOCK 16

/*
 * Token vectors: `tokens` rows of `heads` vectors of `head_dim` elements of type `dtype`
 * (mq_dtype). Element (t, h, d) is data[t * token_stride + h * head_stride + d] (strides in
 * elements, so that the three parts of one fused projection can be passed as they lie). data
 * must be 16-byte aligned and both strides multiples of 8 (MQ_ERR_ARG otherwise).
 */
typedef struct {
    void *data;
    int64_t token_stride, head_stride;
    int32_t tokens, heads, head_dim, dtype;
} mq_rows;

/*
 * A paged cache of keys and values in 8 bits. num_pages pages of page_size tokens (a multiple
 * of MQ_KV_BLOCK); head_dim 64, 96, 128, 192 or 256. With NB = page_size / 16:
 *   k_codes  [num_pages][kv_heads][page_size][head_dim]   E4M3 (s|eeee|mmm, bias 7)
 *   v_codes  [num_pages][kv_heads][NB][head_dim][16]      E4M3, the 16 tokens of a block together
 *   k_scales, v_scales [num_pages][kv_heads][NB]          one byte e per block: the scale 2^(e-127)
 * A key element's value is decode(code) * 2^(e-127). Scale bytes written by this library lie in
 * [10, 247]; 255 marks a block that received a NaN or an infinity: its codes are 0, and every
 * attention row that sees a token of the block is NaN.
 * Token t of a sequence lies in page table[t / page_size], slot t % page_size. A table entry
 * outside [0, num_pages) holds no tokens: nothing is read from it or written to it, and its
 * tokens take no part in attention.
 * k_codes and v_codes must be 16-byte aligned (MQ_ERR_ARG otherwise). No two sequences may share
 * a page that one of them writes (mq_kv_append, and the new pages of mq_kv_evict).
 */
typedef struct {
    int32_t num_pages, page_size, kv_heads, head_dim;
    uint8_t *k_codes, *v_codes, *k_scales, *v_scales;
} mq_kv_cache;

/*
 * mq_kv_append: quantize new keys and values into the cache behind each sequence's tokens.
 * Sequence s has lens[s] tokens in the cache and receives rows [cu[s], cu[s+1]) of k and v
 * (cu[0..n_seqs] ascending from 0 to k->tokens). Each block of 16 tokens and head that receives a
 * token: with amax the largest magnitude of the new tokens in it,
 *   e    = max(10, the smallest e with amax <= 448 * 2^(e-127), e_held)
 *   code = CastE4M3(x * 2^(127-e))                 new tokens (nearest, ties to even)
 *   code = CastE4M3(value(code) * 2^(e_held-e))    tokens that the block held
 * (e_held, and held tokens, only where the block held tokens); slots of the block after its last
 * token become 0. A NaN or an infinity among the new values, or e_held = 255, gives e = 255 and
 * codes 0. Scaling by powers of two is exact, so each code is rounded once for each time its
 * block's scale grows. Appending the same tokens to the same lens again changes nothing.
 * table_dev: [n_seqs][max_pages] page numbers. lens_dev is not changed. Tokens whose position
 *          reaches max_pages * page_size are dropped.
 * Errors: MQ_ERR_ARG (null or misaligned pointer, negative size, unknown dtype, page_size no
 *         multiple of 16), MQ_ERR_SHAPE (k, v and the cache disagree), MQ_ERR_UNSUPPORTED
 *         (head_dim outside the set, 2^31 or more work items).
 */
mq_status mq_kv_append(const mq_kv_cache *cache, const mq_rows *k, const mq_rows *v,
                       const int32_t *table_dev, const int32_t *lens_dev, const int32_t *cu_dev,
                       int32_t n_seqs, int32_t max_pages, hipStream_t stream);

/* Bytes of device workspace mq_attn_cached needs for these sizes (0 on invalid input, and where
 * none is needed), and for any call with the same heads and fewer sequences, new tokens or a
 * smaller max_len, with or without weights. max_len: the call's, or max_pages * page_size where the
 * call passes 0. weights: 1 if a call adds up attention weights. */
size_t mq_attn_cached_workspace_bytes(int32_t n_seqs, int32_t q_heads, int32_t kv_heads,
                                      int32_t head_dim, int32_t q_len, int32_t max_len,
                                      int32_t weights);

/*
 * mq_attn_cached: attention of each sequence's last q_len tokens over its cached tokens.
 * Sequence s holds lens[s] tokens, its new ones (already appended) included. Row i of sequence s,
 * i in [0, q_len), sees tokens t <= lens[s] - q_len + i; query head h reads key/value head
 * h / (q_heads / kv_heads):
 *   p[t] = softmax_t(scale * sum_d q[d] * K[t][d])     out[d] = sum_t p[t] * V[t][d]
 * with the softmax and both sums in fp32 from exact products of the cache's values; p is held to
 * 2^-16 of itself for the second product. A row that sees no token is 0.
 * q, out:  n_seqs * q_len rows, sequence by sequence.
 * max_len: no sequence holds more tokens than this (longer ones are read up to it); 0 stands for
 *          max_pages * page_size. It sizes the launch and the workspace.
 * weights_dev: null, or fp32 [num_pages][kv_heads][page_size]: for each cached token and
 *          key/value head, p summed over the head's query heads and the q_len rows is added to
 *          the token's place. Sequences may read the same pages: the places gain what all of them
 *          give. The order is fixed, so results are deterministic, where such a page lies at the
 *          same place of their rows of table_dev (a common beginning); what a page gains at
 *          different places of the table is added in any order.
 * ws_dev / ws_bytes: device scratch, 16-byte aligned, of at least
 *          mq_attn_cached_workspace_bytes(...) bytes (may be null where that is 0).
 * Errors: MQ_ERR_ARG, MQ_ERR_SHAPE (q, out and the cache disagree; q_heads no multiple of
 *         kv_heads), MQ_ERR_WORKSPACE, MQ_ERR_UNSUPPORTED (as for mq_kv_append).
 */
mq_status mq_attn_cached(const mq_kv_cache *cache, const mq_rows *q, const mq_rows *out,
                         const int32_t *table_dev, const int32_t *lens_dev, int32_t n_seqs,
                         int32_t max_pages, int32_t q_len, int32_t max_len, float scale,
                         float *weights_dev, void *ws_dev, size_t ws_bytes, hipStream_t stream);

/*
 * mq_attn_prompt: causal attention over whole prompts, packed one after another. Sequence s has
 * rows [cu[s], cu[s+1]) of q, k, v and out; row i of a sequence sees its rows j <= i; query head
 * h reads key/value head h / (q_heads / kv_heads):
 *   p[j] = softmax_j(scale * sum_d q[d] * k[j][d])     out[d] = sum_j p[j] * v[j][d]
 * with the softmax and both sums in fp32 and p rounded to dtype for the second product: by 2^-8 of
 * itself at most for MQ_BF16; for MQ_F16 by 2^-11 of itself, or where that is more by 2^-28 of the
 * largest p in the row's same 64 tokens (64 i <= j < 64 (i + 1)).
 * max_len: no sequence is longer than this (rows past it are neither read nor written).
 * Errors: as for mq_attn_cached (without a workspace); MQ_ERR_UNSUPPORTED also for a token_stride
 *         of k or v above 2^24.
 */
mq_status mq_attn_prompt(const mq_rows *q, const mq_rows *k, const mq_rows *v, const mq_rows *out,
                         const int32_t *cu_dev, int32_t n_seqs, int32_t max_len, float scale,
                         hipStream_t stream);

/*
 * mq_kv_evict: cut each sequence's cache back to at most `keep` tokens, head by head. Of a
 * sequence's lens[s] tokens (all of them where lens[s] <= keep) each key/value head keeps the
 * last min(recent, keep), and of the others those with the largest weights (equal weights: the
 * lower position first; a NaN weight is below every other), in their order. They are copied to
 * the first min(lens[s], keep) slots of new_table's pages:
 *   e    = max of the scale bytes that the kept tokens of a new block come with
 *   code = CastE4M3(value(code) * 2^(e_src - e))   (unchanged where e_src = e; all 0 if e = 255)
 * and their weights with them; slots of a new block after its last token become 0 (weights too).
 * new_table's pages must not be pages of `table_dev` or of each other. The old pages are left
 * as they are, for the caller to free.
 * weights_dev: fp32 [num_pages][kv_heads][page_size], as mq_attn_cached adds them up.
 * table_dev [n_seqs][max_pages]; new_table_dev [n_seqs][new_max_pages], with
 *          keep <= new_max_pages * page_size.
 * new_lens_dev: [n_seqs], receives min(lens[s], keep); not lens_dev itself (MQ_ERR_ARG).
 * kept_dev: [n_seqs][kv_heads][keep], receives the kept tokens' former positions, ascending, -1
 *          after the last.
 * A kept token whose old page is outside [0, num_pages) is copied as code 0 with scale byte 10.
 * Errors: MQ_ERR_ARG, MQ_ERR_SHAPE (keep does not fit new_table), MQ_ERR_UNSUPPORTED (also keep
 *         above 2^30).
 */
mq_status mq_kv_evict(const mq_kv_cache *cache, float *weights_dev, const int32_t *table_dev,
                      const int32_t *lens_dev, const int32_t *new_table_dev,
                      int32_t *new_lens_dev, int32_t *kept_dev, int32_t n_seqs,
                      int32_t max_pages, int32_t new_max_pages, int32_t keep, int32_t recent,
                      hipStream_t stream);

/* ---- microscaled 4-bit linear layers ---------------------------------------------------------
 *
 * The linear layers of a transformer block on E2M1 elements with one power-of-two scale per 32 of
 * them along the contracted dimension, the operands that the scaled matrix instructions take:
 * quantization along rows and columns from one read (mq_mx4_quantize, read back by
 * mq_mx4_dequantize), the product of two quantized matrices (mq_mx4_matmul), a linear layer on a
 * quantized weight (mq_mx4_linear) and its gradients (mq_mx4_linear_backward), and the gated
 * feed-forward product silu(x Wg^T) * (x Wu^T) (mq_mx4_gated) and its gradients
 * (mq_mx4_gated_backward). Each tensor is quantized once for each direction that it is contracted
 * along, and read once for both.
 *
 * Every product is exact and summed in fp32 (in an order that the sizes alone fix: results repeat
 * bit for bit); a sum below 2^-126 in magnitude may become 0. Outputs and workspaces must not
 * overlap inputs or each other, and calls that can run at the same time must not share a workspace;
 * a workspace holds nothing from one call to the next.
 */

/* mq_matrix.dtype: an mq_dtype, or fp32. */
#define MQ_F32 3

/* Elements that share one scale, and columns that lie together (mq_mx4). */
#define MQ_MX4_BLOCK 32
#define MQ_MX4_PIECE 256

/* A dense matrix: element (r, c) is data[r * stride + c]. data must be aligned to the element's
 * size (16-byte alignment, and a stride that keeps it, is faster). stride in elements, >= cols.
 * A matrix without elements may be null. */
typedef struct {
    void *data;
    int64_t stride;
    int32_t rows, cols, dtype;
} mq_matrix;

/*
 * A quantized matrix of rows x cols, with blocks of 32 along a row. Rows are cut into
 * P = ceil(cols / 256) pieces of 256 columns (8 blocks), the last one filled up with zeros:
 *   codes   [P][rows][128]  E2M1 (s|ee|m, bias 1); element j of a piece in byte j / 2, the even
 *                           one in the low half
 *   scales  [P][rows][8]    one byte e for a block of 32: the scale 2^(e-127)
 * An element's value is decode(code) * 2^(e-127). Scale bytes written by this library lie in
 * [2, 252]; 255 marks a block that received a NaN or an infinity: its codes are 0, and every sum
 * that it takes part in is NaN. Elements past cols must have code 0, and no scale byte of 255.
 * codes must be 16-byte aligned, scales 8-byte aligned (MQ_ERR_ARG otherwise).
 */
typedef struct {
    int32_t rows, cols;
    uint8_t *codes, *scales;
} mq_mx4;

/* Bytes of the codes and of the scales of a quantized matrix (0 for invalid arguments, and for a
 * matrix without elements). */
size_t mq_mx4_codes_bytes(int32_t rows, int32_t cols);
size_t mq_mx4_scales_bytes(int32_t rows, int32_t cols);

/*
 * mq_mx4_quantize: x along its rows, its columns, or both from one read. With amax the largest
 * magnitude of a block,
 *   e    = the smallest byte with amax <= 6 * 2^(e-127), but in [2, 252]
 *   code = CastE2M1(x * 2^(127-e))
 * (the scale is rounded up, so that nothing but amax past 6 * 2^125 saturates; the OCP microscaling
 * text takes the largest power of two up to amax / 4 and lets what lies past 6 of it saturate).
 * CastE2M1 is to nearest, ties to the even code, saturating at 6 (MQ_RNE), or stochastic (MQ_SR): up
 * from the neighbour below in magnitude iff u < frac * 65536, where frac is the distance to it in
 * steps and u a 16-bit draw: of element j (of 32) of block t = row * ceil(cols / 32) + block, the
 * (j%2)-th half of word (j%8)/2 of Philox4x32-10(counter = (4t + j/8 as 64 bits, low word first;
 * d; 0), key = seed) with d = 0 for rows and 1 for columns. A code keeps its element's sign.
 * row: null, or rows x cols. col: null, or cols x rows, the transposed matrix along its rows.
 * Errors: MQ_ERR_ARG (null, misaligned, negative, unknown dtype or rounding, neither row nor col),
 *         MQ_ERR_SHAPE, MQ_ERR_UNSUPPORTED (a dimension of 2^30 or more, or more work than a grid
 *         holds).
 */
mq_status mq_mx4_quantize(const mq_matrix *x, const mq_mx4 *row, const mq_mx4 *col, int32_t rnd,
                          uint64_t seed, hipStream_t stream);

/* mq_mx4_dequantize: the values of q, rounded once to out's type. Errors: as mq_mx4_quantize. */
mq_status mq_mx4_dequantize(const mq_mx4 *q, const mq_matrix *out, hipStream_t stream);

/*
 * mq_mx4_matmul: y = a b^T, y[m][n] = sum_k a[m][k] * b[n][k], rounded once to y's type.
 * a: M x K, b: N x K, y: M x N (K = 0 gives zeros).
 * ws_dev / ws_bytes: not used: mq_mx4_matmul_workspace_bytes is 0 for all sizes, and ws_dev may be
 *          null. Of the calls below: device scratch, 16-byte aligned, of at least
 *          mq_mx4_..._workspace_bytes(M, N, K) bytes (may be null where that is 0). What suffices
 *          for M rows suffices for fewer.
 * Errors: MQ_ERR_ARG (ws_dev not 16-byte aligned among them), MQ_ERR_SHAPE, MQ_ERR_UNSUPPORTED
 *         (as mq_mx4_quantize); of the calls below also MQ_ERR_WORKSPACE.
 */
size_t mq_mx4_matmul_workspace_bytes(int32_t m, int32_t n, int32_t k);
mq_status mq_mx4_matmul(const mq_mx4 *a, const mq_mx4 *b, const mq_matrix *y, void *ws_dev,
                        size_t ws_bytes, hipStream_t stream);

/*
 * mq_mx4_linear: y = Q(x) w^T, x quantized along its rows (MQ_RNE) on the way.
 * x: M x K (M may be 0), w: N x K, y: M x N; the types of x and y are independent.
 * x_col: null, or K x M: receives x quantized along its columns, which the weight's gradient reads.
 * Errors: as mq_mx4_matmul.
 */
size_t mq_mx4_linear_workspace_bytes(int32_t m, int32_t n, int32_t k);
mq_status mq_mx4_linear(const mq_matrix *x, const mq_mx4 *w, const mq_matrix *y,
                        const mq_mx4 *x_col, void *ws_dev, size_t ws_bytes, hipStream_t stream);

/*
 * mq_mx4_linear_backward: the gradients of y = x w^T for dy: M x N,
 *   dx = Q(dy) w        M x K, from w_col (K x N), the weight quantized along its columns
 *   dw = Q(dy^T) x      N x K, from x_col (K x M)
 * with dy quantized along its rows and its columns, rounded as `rnd` says (see mq_mx4_quantize).
 * dx or dw may be null, and with it w_col or x_col. M = 0 gives dw = 0.
 * Errors: as mq_mx4_matmul; MQ_ERR_ARG also where dx and dw are both null.
 */
size_t mq_mx4_linear_backward_workspace_bytes(int32_t m, int32_t n, int32_t k);
mq_status mq_mx4_linear_backward(const mq_matrix *dy, const mq_mx4 *x_col, const mq_mx4 *w_col,
                                 const mq_matrix *dx, const mq_matrix *dw, int32_t rnd,
                                 uint64_t seed, void *ws_dev, size_t ws_bytes, hipStream_t stream);

/*
 * mq_mx4_gated: h = silu(G) * U with G = Q(x) wg^T, U = Q(x) wu^T, silu(z) = z / (1 + exp(-z));
 * the two products and the activation stay in fp32, h is rounded once.
 * x: M x K, wg and wu: F x K, h: M x F. g, u: both null, or M x F of h's type: receive G and U,
 * rounded, for the backward pass (in f16, one that rounds past 65504 becomes an infinity, and makes the
 * gradients of its blocks NaN). x_col: as for mq_mx4_linear.
 * Errors: as mq_mx4_matmul.
 */
size_t mq_mx4_gated_workspace_bytes(int32_t m, int32_t f, int32_t k);
mq_status mq_mx4_gated(const mq_matrix *x, const mq_mx4 *wg, const mq_mx4 *wu, const mq_matrix *h,
                       const mq_matrix *g, const mq_matrix *u, const mq_mx4 *x_col, void *ws_dev,
                       size_t ws_bytes, hipStream_t stream);

/*
 * mq_mx4_gated_backward: the gradients of mq_mx4_gated for dh: M x F, from the g and u that it kept
 * (all three of one type). With s = 1 / (1 + exp(-g)),
 *   dg = dh * u * s * (1 + g * (1 - s))     du = dh * g * s      (fp32, never stored)
 *   dx = Q(dg) wg + Q(du) wu     M x K, from wg_col and wu_col (K x F)
 *   dwg = Q(dg^T) x, dwu = Q(du^T) x      F x K, both of one type, from x_col (K x M)
 * dg and du are quantized along rows and columns, rounded as `rnd` says; a stochastic draw of du is
 * that of dg's with d + 2 in the counter. dx may be null, and with it wg_col and wu_col; dwg and dwu
 * may both be null, and with them x_col. M = 0 gives dwg = dwu = 0.
 * Errors: as mq_mx4_linear_backward.
 */
size_t mq_mx4_gated_backward_workspace_bytes(int32_t m, int32_t f, int32_t k);
mq_status mq_mx4_gated_backward(const mq_matrix *dh, const mq_matrix *g, const mq_matrix *u,
                                const mq_mx4 *x_col, const mq_mx4 *wg_col, const mq_mx4 *wu_col,
                                const mq_matrix *dx, const mq_matrix *dwg, const mq_matrix *dwu,
                                int32_t rnd, uint64_t seed, void *ws_dev, size_t ws_bytes,
                                hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MQ_H */
