/*
 * autoround_hip.h - C ABI of the MI355X (gfx950) AutoRound per-Linear tuning library.
 *
 * AutoRound tunes, per weight group, a rounding offset V in [-0.5, 0.5] and two
 * clip factors (alpha on the group minimum, beta on the group maximum) by
 * SignSGD so that the fake-quantized weight Ŵ = s*(clamp(rint(W/s + V) + zp) - zp)
 * reproduces the layer output X·Wᵀ on calibration tokens; the final integer codes
 * are then packed into 32-bit words.
 *
 * Sources (page title, section):
 *   [LLMC]  "[llm-compressor] AutoRound: 부호 경사 하강법으로 라운딩 최적화":
 *           paper-core equations (RTN, learnable offset, SignSGD), constructor
 *           parameter table, the per-module tuning loop, _fake_quantize_with_offset.
 *   [INTEL] "Introducing AutoRound: Intel's Advanced Quantization for LLMs and VLMs":
 *           section 2 (rounding and clipping range tuned jointly), section 4
 *           (zero iterations = RTN; 8/4/3/2-bit).
 *   [SGL]   "[SGLang] AutoRound: 자동 라운딩 최적화 양자화": "1. AutoRoundConfig"
 *           (bits {2,3,4,8}, sym, pack_factor = Fraction(32, bits)), "설계 근거"
 *           (GPTQ/AWQ packing reuse).
 *
 * Conventions for every entry point:
 *   - Every array pointer is a caller-owned DEVICE pointer (hipMalloc / torch),
 *     row-major and contiguous, 16-byte aligned. The library never allocates
 *     device memory; scratch space comes in through (ws, ws_bytes).
 *   - `stream` is a hipStream_t (NULL = default stream). All device work is
 *     enqueued asynchronously on it, except where an entry point says it blocks.
 *   - Arguments are validated before anything is enqueued; on any error status
 *     nothing has been written. No C++ exception crosses this interface.
 *   - Shapes: W is [N, K] (N out features, K in features, torch Linear layout).
 *     K must be a multiple of 8 and of group_size; G = K / group_size groups per
 *     row (group_size = -1: one group of K per row). group_size must be a
 *     multiple of 8. N >= 1 and K >= 8, except where an entry point accepts N*K = 0.
 *   - bf16 data is passed as uint16 bit patterns.
 */
#ifndef AUTOROUND_HIP_H
#define AUTOROUND_HIP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  AR_OK = 0,
  AR_ERR_INVALID_ARG = 1,   /* null pointer, bad hyper-parameter, misaligned pointer */
  AR_ERR_UNSUPPORTED = 2,   /* bits not in {2,3,4,8} (16 = "leave unquantized"), bad dtype */
  AR_ERR_SHAPE = 3,         /* size constraint violated */
  AR_ERR_WORKSPACE = 4,     /* ws_bytes smaller than the *_workspace_size result */
  AR_ERR_NONFINITE = 5,     /* check_finite set and an input holds NaN or Inf */
  AR_ERR_HIP = 6            /* a HIP runtime call or kernel launch failed */
} ar_status;

typedef enum { AR_F32 = 0, AR_BF16 = 1 } ar_dtype;

/* Tuning hyper-parameters; names as on the [LLMC] constructor parameter table. */
typedef struct {
  int32_t bits;          /* {2,3,4,8}: [SGL] 1. AutoRoundConfig SUPPORTED_BITS            */
  int32_t group_size;    /* input channels per group; -1 = whole row                      */
  int32_t sym;           /* 0: asymmetric (zero-point from the range), 1: symmetric        */
  int32_t nsamples;      /* calibration samples ([LLMC] default 128)                       */
  int32_t seqlen;        /* tokens per sample ([LLMC] default 2048)                        */
  int32_t batch_samples; /* samples per SignSGD step; nsamples % batch_samples == 0        */
  int32_t iters;         /* SignSGD steps ([LLMC] default 200); 0 = RTN ([INTEL] sec. 4)   */
  float lr;              /* offset step ([LLMC] default 0.005)                             */
  float minmax_lr;       /* clip-factor step; < 0 means "unset" = lr ([LLMC] minmax_lr)    */
  float minmax_shrink;   /* initial alpha = beta ([LLMC] minmax_shrink, default 1.0)       */
  float clip_lo;         /* alpha/beta lower clamp (default 0.5)                           */
  float clip_hi;         /* alpha/beta upper clamp (default 1.0)                           */
  int32_t init_scale;    /* initial alpha = beta ([LLMC] tuning loop: "Min-Max or MSE"):
                            0: minmax_shrink (Min-Max); 1: MSE, per group the shrink p of
                            the grid p_j = float32(1 - j/mse_grid) inside [clip_lo, clip_hi]
                            whose round-to-nearest quantization has the smallest sum of
                            squared weight errors (float32 errors, float64 sum, first
                            minimum on ties)                                              */
  int32_t mse_grid;      /* grid steps per unit shrink for init_scale = 1 (default 100)   */
  int32_t check_finite;  /* 0 (default): no check. A NaN or Inf in the data then makes
                            the loss of every step that reads it NaN: such a step is
                            never taken as the best (the comparison is a strict <), and
                            its non-finite gradients move nothing (sgn(NaN) = 0), so the
                            returned state stays finite. The [LLMC] tuning loop reads
                            each batch loss on the host; this loop does not.
                            1: the tuning entry points (ar_tune_step, ar_tune_linear and
                            their Gram and no-allocation forms) first scan their inputs
                            (W, X, Y; the step also V, alpha, beta) on the device and
                            return AR_ERR_NONFINITE, with no output written, when any
                            element is NaN or infinite. The call then blocks until the
                            scan's result is on the host, so it cannot be captured in a
                            HIP graph. ar_tune_block passes it to each Linear's tuning. */
} ar_config;

/* Per-kernel device time of one ar_tune_linear call, measured with HIP events
   recorded on the call's stream around the kernels of every sample_every-th
   SignSGD step (milliseconds, summed over the timed steps). */
typedef struct {
  int32_t sample_every;  /* input: time steps i with i % sample_every == 0 (<= 1: every step) */
  double fwd_gemm_ms;    /* Y' = X_b·Ŵᵀ with the residual / dY / R² epilogue               */
  double wgrad_gemm_ms;  /* G = (2/(T_b·N))·dYᵀ·X_b, with the loss reduction and best-loss
                            decision in its prologue                                        */
  double ste_update_ms;  /* straight-through fold + SignSGD update + next fake-quant         */
  int64_t steps;         /* output: number of SignSGD steps timed                          */
} ar_kernel_times;

/* Fill *cfg with the [LLMC] defaults: bits 4, group_size 128, asym, nsamples 128,
   seqlen 2048, batch_samples 8, iters 200, lr 0.005, minmax_lr unset (-1),
   minmax_shrink 1.0, clip range [0.5, 1.0], Min-Max initial scale (mse_grid 100).
   Returns AR_ERR_INVALID_ARG on NULL. */
ar_status ar_config_default(ar_config* cfg);

/* Static, NUL-terminated description of a status code (never NULL). */
const char* ar_status_string(int32_t status);

/* Bytes of device workspace ar_tune_linear needs for this problem (X is
   [nsamples*seqlen, K] bf16, Y is [nsamples*seqlen, N] of dtype ydt). */
ar_status ar_workspace_size(const ar_config* cfg, int64_t N, int64_t K, int32_t ydt,
                            size_t* bytes);

/* Bytes of device workspace ar_tune_step needs for a minibatch of Tb tokens. */
ar_status ar_step_workspace_size(const ar_config* cfg, int64_t N, int64_t K, int64_t Tb,
                                 int32_t ydt, size_t* bytes);

/* Initial clip factors of every group ([LLMC] tuning loop, initial scale):
   alpha = beta = minmax_shrink (init_scale 0) or the MSE shrink (init_scale 1).
   alpha, beta [N, G] float32, required. N*K = 0 is a no-op. */
ar_status ar_init_clip(const ar_config* cfg, int32_t wdt, const void* W, int64_t N, int64_t K,
                       float* alpha, float* beta, void* stream);

/* Round-to-nearest quantization ([LLMC] paper-core RTN equation): V = 0 and
   the initial clip factors of ar_init_clip; group min/max from W ([LLMC] tuning
   loop, initial scale).
   W      [N, K] of dtype wdt (AR_F32 or AR_BF16)
   codes  [N, K] uint8 in [0, 2^bits-1]        (nullable)
   scale  [N, G] float32                       (nullable)
   zp     [N, G] uint8 zero-points              (nullable)
   Wq     [N, K] of dtype wdt, s*(code - zp)    (nullable)
   N*K = 0 is a no-op. */
ar_status ar_rtn_quant(const ar_config* cfg, int32_t wdt, const void* W, int64_t N, int64_t K,
                       uint8_t* codes, float* scale, uint8_t* zp, void* Wq, void* stream);

/* Fake-quantization with learnable offset and clip factors ([LLMC] paper-core
   offset equation and _fake_quantize_with_offset; [INTEL] sec. 2 clip range):
   per group lo = min(alpha*wmin, 0), hi = max(beta*wmax, 0), s = (hi-lo)/maxq,
   zp = clamp(rint(-lo/s), 0, maxq)  (sym: s = 2*max(|alpha*wmin|, |beta*wmax|)/maxq,
   zp = 2^(bits-1)); per element code = clamp(rint(W/s + V) + zp, 0, maxq),
   Ŵ = s*(code - zp). A zero-range group uses s = 1. All float32, rint = half-even.
   V [N, K] float32; alpha, beta [N, G] float32.
   Wq_bf16 [N, K] bf16 Ŵ (nullable); codes, scale, zp as in ar_rtn_quant (nullable).
   N*K = 0 is a no-op. */
ar_status ar_fakequant_fwd(const ar_config* cfg, int32_t wdt, const void* W, int64_t N,
                           int64_t K, const float* V, const float* alpha, const float* beta,
                           uint16_t* Wq_bf16, uint8_t* codes, float* scale, uint8_t* zp,
                           void* stream);

/* Tuning state of one Linear, all device pointers owned by the caller. */
typedef struct {
  const void* W;       /* [N, K] weight, dtype wdt          */
  int32_t wdt;         /* AR_F32 or AR_BF16                  */
  int64_t N, K;
  float* V;            /* [N, K] offsets, updated in place   */
  float* alpha;        /* [N, G] min clip factors, in place  */
  float* beta;         /* [N, G] max clip factors, in place  */
  float* best_V;       /* [N, K] best-state snapshot   (nullable: no snapshot; the four
                          best_* pointers are all set or all NULL) */
  float* best_alpha;   /* [N, G]                              */
  float* best_beta;    /* [N, G]                              */
  float* best_loss;    /* device scalar; caller initialises it to +inf */
} ar_state;

/* One SignSGD iteration on one minibatch ([LLMC] tuning loop; [LLMC] SignSGD
   equation). From the current state: Ŵ (bf16 operand), Y' = Xb·Ŵᵀ (bf16 MFMA,
   float32 accumulation), R = Y' - Yb, loss = sum(R²)/(Tb·N) -> loss_out[0];
   dY = bf16(R); G = (2/(Tb·N))·dYᵀ·Xb; straight-through fold to dL/dV, dL/dalpha,
   dL/dbeta. If best_* are set and loss < *best_loss, the current (pre-update)
   state is copied to best_* and *best_loss = loss. If apply_update != 0:
   V <- clamp(V - lr·sgn(dL/dV), -0.5, 0.5), alpha/beta <- clamp(· - minmax_lr·sgn, clip_lo, clip_hi).
   Xb [Tb, K] bf16; Yb [Tb, N] of dtype ydt; Tb > 0, Tb % 8 == 0.
   loss_out: device float (required). gV [N, K], galpha/gbeta [N, G] float32:
   pre-update gradients (nullable). ws: ar_step_workspace_size bytes. */
ar_status ar_tune_step(const ar_config* cfg, const ar_state* state, const uint16_t* Xb,
                       const void* Yb, int32_t ydt, int64_t Tb, float* loss_out, float* gV,
                       float* galpha, float* gbeta, int32_t apply_update, void* ws,
                       size_t ws_bytes, void* stream);

/* ar_tune_step for callers that cannot allocate device memory (code under HIP
   graph capture, tight loops, harnesses that forbid allocation): the same
   arguments without (ws, ws_bytes), and the same kernels, results and errors.
   Its scratch is a fixed array of AR_NOALLOC_SCRATCH_BYTES in each GPU's
   memory, set up on the first call on that device (the device current at the
   call, which must be the stream's) and held until the process ends. A problem
   whose ar_step_workspace_size exceeds AR_NOALLOC_SCRATCH_BYTES returns
   AR_ERR_WORKSPACE before anything is enqueued. The call makes no device
   allocation. Every call on one GPU shares that GPU's array: calls that may
   overlap on one GPU (other streams, other host threads) race and must be
   serialised by the caller. Each call writes every part of the array it reads
   before reading it, so what an earlier call left there does not matter. */
#define AR_NOALLOC_SCRATCH_BYTES ((size_t)64 * 1024 * 1024)
ar_status ar_tune_step_noalloc(const ar_config* cfg, const ar_state* state, const uint16_t* Xb,
                               const void* Yb, int32_t ydt, int64_t Tb, float* loss_out,
                               float* gV, float* galpha, float* gbeta, int32_t apply_update,
                               void* stream);

/* The whole per-Linear tuning loop ([LLMC] tuning loop with best-loss snapshot):
   V = 0, alpha and beta from ar_init_clip; step i uses minibatch b = i mod
   (nsamples/batch_samples), i.e. rows [b*Tb, (b+1)*Tb) of X and Y with
   Tb = batch_samples*seqlen; after cfg->iters steps the state with the lowest
   loss (strictly lower than all before it, evaluated before its update) is
   restored and quantized. iters = 0 gives RTN ([INTEL] section 4).
   W [N, K] wdt; X [nsamples*seqlen, K] bf16; Y [nsamples*seqlen, N] ydt.
   Outputs: codes [N, K] uint8, scale [N, G] float32, zp [N, G] uint8 (required);
   Wq [N, K] wdt (nullable); V_out [N, K], alpha_out/beta_out [N, G] float32 final
   (restored) state (nullable); losses [iters] float32 per-step loss (nullable).
   ws: ar_workspace_size bytes. times: when non-NULL, per-kernel device times of
   every times->sample_every-th step are measured with HIP events and, with
   iters > 0, the call blocks until the stream has drained (iters = 0 leaves the
   times at zero and does not block). */
ar_status ar_tune_linear(const ar_config* cfg, int32_t wdt, const void* W, int64_t N, int64_t K,
                         const uint16_t* X, const void* Y, int32_t ydt, uint8_t* codes,
                         float* scale, uint8_t* zp, void* Wq, float* V_out, float* alpha_out,
                         float* beta_out, float* losses, void* ws, size_t ws_bytes,
                         ar_kernel_times* times, void* stream);

/* ---- W{2,3,4,8} x bf16 product on the packed format ------------------------
   Y = X·bf16(Ŵ)ᵀ with Ŵ = s·(q - zp) read from ar_pack's format ([SGL] "설계
   근거": AutoRound checkpoints reuse GPTQ/AWQ packing; [LLMC]
   _fake_quantize_with_offset for the dequantisation): the deployment side of the
   tuned codes. The bf16 Ŵ is the operand the tuning loop's forward product uses.
   X [M, K] bf16 row-major; qweight [K*bits/32, N] int32 and qzeros
   [G, N*bits/32] int32 as ar_pack writes them (qzeros NULL: symmetric grid,
   zp = 2^(bits-1)); scale [N, G] float32 (ar_tune_linear's layout); Y [M, N]
   row-major, ydt AR_F32 or AR_BF16. float32 accumulation. group_size as in
   ar_config (-1: whole row); K*bits % 32 == 0, K % group = 0, group % 8 == 0;
   with qzeros N*bits % 32 == 0. M <= 16 streams the packed words once,
   dequantizing each code once for all M rows (split-K, slices summed in a fixed
   order); larger M dequantizes once into a blocked bf16 operand and runs the
   MFMA product. M = 0 or N = 0 is a no-op. The workspace size depends on bits,
   group_size and the shape (the split-K slice length follows the group size);
   ar_dequant_gemm_workspace_size validates them as ar_dequant_gemm does. */
ar_status ar_dequant_gemm_workspace_size(int32_t bits, int32_t group_size, int64_t M, int64_t N,
                                         int64_t K, size_t* bytes);
ar_status ar_dequant_gemm(int32_t bits, int32_t group_size, const uint16_t* X, int64_t M,
                          int64_t K, const int32_t* qweight, const int32_t* qzeros,
                          const float* scale, int64_t N, void* Y, int32_t ydt, void* ws,
                          size_t ws_bytes, void* stream);

/* ---- e4m3 operands and their product ---------------------------------------
   The 8-bit-float path of a decoder layer: both sides of a Linear in e4m3 (the
   OCP format: no infinities, largest value 448) with float32 scales per block of
   128 input channels. ar_fp8_quant_weight stands beside ar_rtn_quant,
   ar_rmsnorm_fp8 beside the block's RMSNorm, ar_fp8_gemm and
   ar_fp8_gemm_grouped beside ar_dequant_gemm. Codes are passed as uint8 bit
   patterns. KB = ceil(K/128) and NB = ceil(N/128); K (and D) must be a multiple
   of 16 below 2^22, rows and N stay below 2^23, and a last block may be shorter
   than 128; other sizes are AR_ERR_SHAPE. Scale and index arrays need 4-byte
   alignment, the others 16.

   Scale of a block: s = 1 if its largest magnitude amax is 0, else
   max(amax/448, 2^-126); code = e4m3(x/s), round to nearest even. Both quotients
   are float32, rounded once (to 2^-46). A NaN gives a NaN code and does not enter
   amax. An infinity makes s infinite and its own code NaN, and with s every
   product of the block NaN. */

/* Activations: q [M, K], scale [KB, M] (one row of scales per block of 128
   channels). gate = 0: the codes of X [M, K]. gate = 1: X is [M, 2K] and the
   codes are those of SiLU(X[:, :K])·X[:, K:], computed in float32 and not rounded
   before. xdt: AR_F32 or AR_BF16. M*K = 0 is a no-op; M*K < 2^36. */
ar_status ar_fp8_quant_act(int32_t xdt, const void* X, int32_t gate, int64_t M, int64_t K,
                           uint8_t* q, float* scale, void* stream);

/* Weights of E layers (E = 1: one Linear; more: the experts of a fused layer):
   W [E, N, K] -> q [E, N, K], scale [E, NB, KB], one scale per 128 x 128 block.
   E*N*K = 0 is a no-op; E*NB*KB < 2^24. */
ar_status ar_fp8_quant_weight(int32_t wdt, const void* W, int64_t E, int64_t N, int64_t K,
                              uint8_t* q, float* scale, void* stream);

/* RMSNorm with the residual's addition and an e4m3 output: v = x + residual
   rounded to dt (residual NULL: v = x), y = (v / sqrt(mean(v²) + eps))·w (sum of
   squares in float64, y in float32), q [D per row] and scale [KB, M] of the
   unrounded y as ar_fp8_quant_act forms them. x, residual [M, D] and w [D] of
   dtype dt (AR_F32 or AR_BF16). h [M, D] dt: v (nullable, needs residual; may be
   x or residual itself, for a residual stream kept in place). y [M, D] dt: the
   norm's output rounded (nullable). eps >= 0 and finite. M*D = 0 is a no-op. */
ar_status ar_rmsnorm_fp8(int32_t dt, const void* x, const void* residual, const void* w, int64_t M,
                         int64_t D, float eps, void* h, void* y, uint8_t* q, float* scale,
                         void* stream);

/* Y [M, N] = Σ_j xs[j, m]·ws[n/128, j]·Σ_{k in block j} Xq[m, k]·Wq[n, k]: Xq
   [M, K] with xs [KB, M] (ar_fp8_quant_act or ar_rmsnorm_fp8), Wq [N, K] with ws
   [NB, KB] (ar_fp8_quant_weight, E = 1). float32 accumulation, in a fixed order;
   ydt AR_F32 or AR_BF16. M = 0 or N = 0 is a no-op; K = 0 is AR_ERR_SHAPE, and so
   is a product whose launch would pass 2^32 threads (M*N beyond 2^36 or so). No
   workspace. The scales may be any float32: where the product of two leaves the
   normal range, the block's term is formed without it.
   A float32 Y is summed in float32 throughout. For a bf16 Y the matrix unit adds
   the products of 8 neighbouring channels with 13 bits below the largest one's
   exponent, cutting the rest off, and everything else in float32: off by up to
   4e-5 of a block's sum for products of like sizes, far below a bf16 rounding.
   Where large products cancel within 8 channels and the small ones are what
   counts, take a float32 Y, or AR_BF16 | AR_F32_SUMS for ydt: a bf16 Y summed like
   a float32 one and rounded once, at half the matrix rate. */
#define AR_F32_SUMS 0x100
ar_status ar_fp8_gemm(const uint8_t* Xq, const float* xs, int64_t M, int64_t K, const uint8_t* Wq,
                      const float* ws, int64_t N, void* Y, int32_t ydt, void* stream);

/* The product by expert: rows offsets[e] <= r < offsets[e+1] of Y [R, N] are
   X_row(r)·Wq[e]ᵀ as above, ydt too, with Wq [E, N, K], ws [E, NB, KB], Xq [T, K], xs [KB, T].
   offsets [E+1] int32 on the device, non-decreasing, in [0, R]; an expert may have
   no rows; rows outside [offsets[0], offsets[E]) keep what they held. row_index
   [R] int32 on the device: row(r) = row_index[r], so a token's codes serve each of
   its experts (an entry may occur any number of times; one outside [0, T) gives
   a row of zeros); NULL: row(r) = r, and T must equal R. The contents of offsets
   are not checked on the host: offsets outside [0, R] are clamped to it, and
   with decreasing ones the rows of Y are unspecified, but nothing outside the
   arrays is read or written. 1 <= E <= 8192; with row_index T*K < 2^32, and T >= 1
   where R is. R = 0 or N = 0 is a no-op. No workspace and no host synchronisation: the call can be
   captured in a HIP graph and replayed with other offsets. */
ar_status ar_fp8_gemm_grouped(const uint8_t* Xq, const float* xs, int64_t T, int64_t K,
                              const uint8_t* Wq, const float* ws, int64_t E, int64_t N,
                              const int32_t* offsets, const int32_t* row_index, int64_t R, void* Y,
                              int32_t ydt, void* stream);

/* ---- Attention and the 4-bit key/value cache --------------------------------
   What a decoder layer needs between its q/k/v product and its o product, in serving and
   on calibration sequences of different lengths: attention over whole prompts beside
   ar_attention, which takes one length and as many key heads as query heads; a cache that
   holds keys and values on the integer grid of ar_rtn_quant (asymmetric, 4 bits); and
   attention of new tokens straight from it. q, k and v come as products of ar_fp8_gemm or
   ar_dequant_gemm leave them, rotated where the model rotates.

   heads query heads share kv_heads key heads, heads/kv_heads neighbours each (heads must
   be a multiple, the quotient at most 256). head_dim is 64 or 128. q, k and v are
   [tokens, heads, head_dim] with a stride in elements between tokens (a multiple of 8, at
   least heads*head_dim, below 2^22), so they may be parts of one q|k|v product. bf16 unless
   said otherwise; float32 softmax and sums; outputs bf16, contiguous, apart from the inputs and
   the workspace. scale multiplies q·k and must be positive and, times log2(e), a finite
   float32. lse (nullable): the natural logarithm of the row's sum of exponentials, [tokens,
   heads] float32. A row that sees no key is 0, its lse minus infinity. What a row does not see
   may hold anything, NaN too. Index arrays need 4-byte alignment, the others 16. */

/* Bytes of device workspace of ar_attention_packed. */
ar_status ar_attention_packed_workspace_size(int64_t B, int64_t Tq, int64_t Tk, int64_t heads,
                                             int64_t kv_heads, int64_t head_dim, size_t* bytes);

/* Causal attention within each of B sequences packed one behind the other: sequence b's
   queries are the tokens q_offsets[b] .. q_offsets[b+1] of q [Tq], its keys and values
   the tokens k_offsets[b] .. k_offsets[b+1] of k and v [Tk] (k_offsets NULL: q_offsets,
   and Tq = Tk). Query i of Lq sees the keys 0 .. i + Lk - Lq: all of them at the last
   query, so a chunk of a prompt takes the keys of what came before it too. Offsets
   [B+1] int32 on the device, non-decreasing; a sequence may have no queries, or fewer keys
   than queries. Rows of out [Tq, heads, head_dim] and lse outside [q_offsets[0],
   q_offsets[B]) keep what they held. Contents of the offsets are not checked on the host:
   they are clamped to [0, Tq] and [0, Tk], and with decreasing ones rows of out are
   unspecified, but nothing outside the arrays is read or written. The weights are rounded
   to bf16 for their product with v, and keys of less than 2^-117 of the largest weight may be
   lost. Tq = 0 or B = 0 is a no-op; B <= 65536, Tq and Tk < 2^30, Tq*heads < 2^30,
   min(B, Tq)*kv_heads < 2^22. No host synchronisation: the call can be captured in a HIP graph and
   replayed with other offsets. Two calls that may overlap need workspaces of their own. */
ar_status ar_attention_packed(const uint16_t* q, int64_t q_stride, const uint16_t* k,
                              int64_t k_stride, const uint16_t* v, int64_t v_stride, int64_t Tq,
                              int64_t Tk, int64_t heads, int64_t kv_heads, int64_t head_dim,
                              const int32_t* q_offsets, const int32_t* k_offsets, int64_t B,
                              float scale, uint16_t* out, float* lse, void* ws, size_t ws_bytes,
                              void* stream);

/* The same, same workspace, with float32 weights in their product with v (three bf16 parts), as
   ar_attention has them, at up to twice the time. */
ar_status ar_attention_packed_f32(const uint16_t* q, int64_t q_stride, const uint16_t* k,
                                  int64_t k_stride, const uint16_t* v, int64_t v_stride, int64_t Tq,
                                  int64_t Tk, int64_t heads, int64_t kv_heads, int64_t head_dim,
                                  const int32_t* q_offsets, const int32_t* k_offsets, int64_t B,
                                  float scale, uint16_t* out, float* lse, void* ws,
                                  size_t ws_bytes, void* stream);

/* A cache of pages of page_size tokens (16, 32, 64, 128 or 256). Slot p*page_size + t is
   token t of page p. Per token, head and group of group_size channels (32, 64 or 128, a
   divisor of head_dim), for keys and for values, in float32, each step rounded once:
     lo = min(x, 0), hi = max(x, 0), s = max((hi - lo)/15, 2^-100),
     zp = clamp(rint(-lo/s), 0, 15), s' = s with its four lowest mantissa bits replaced by zp,
     code = clamp(rint(x/s') + zp, 0, 15); the value held is s'·(code - zp).
   A NaN or an infinity, or a range beyond float32, makes s' NaN and with it the group.
   codes [pages, 2, heads, page_size, head_dim/2] uint8, two codes a byte, the even channel
   in the low half: the keys' (first) bytes in order; of the values, byte 32·b + 16·c + n
   of token t at [t/8][b][n][t%8][c]. scale [pages, 2, heads, page_size,
   head_dim/group_size] float32: s'. pages*page_size < 2^31. */
typedef struct {
  uint8_t* codes;
  float* scale;
  int64_t pages;
  int64_t heads;        /* key heads */
  int32_t head_dim;
  int32_t page_size;
  int32_t group_size;
} ar_kv4_cache;

/* Quantize k and v [T, cache heads, head_dim] (dt AR_F32 or AR_BF16; strides as above)
   into slots [T] int32 on the device; tokens whose slot lies outside the cache (-1, say)
   are left out. Where two tokens of one call name the same slot, what that slot then
   holds is unspecified (every other slot is as it should be). T = 0 is a no-op;
   T <= 2^28 - 16. */
ar_status ar_kv4_write(const ar_kv4_cache* cache, int32_t dt, const void* k, int64_t k_stride,
                       const void* v, int64_t v_stride, const int32_t* slots, int64_t T,
                       void* stream);

/* The values held in slots [T] int32 (any number of times each), to k and v [T, cache heads,
   head_dim] of dtype dt, contiguous; zeros for a slot outside the cache. A bf16 output is
   rounded once. T = 0 is a no-op; T <= 2^28 - 16. */
ar_status ar_kv4_read(const ar_kv4_cache* cache, const int32_t* slots, int64_t T, int32_t dt,
                      void* k, void* v, void* stream);

/* Bytes of device workspace of ar_kv4_attention (of cache, its sizes only are read). */
ar_status ar_kv4_attention_workspace_size(const ar_kv4_cache* cache, int64_t B, int64_t new_tokens,
                                          int64_t heads, int64_t max_len, size_t* bytes);

/* Attention of the newest new_tokens tokens of each of B sequences over its cached tokens,
   theirs among them: q [B*new_tokens, heads, head_dim]; sequence b's token t lies in page
   table[b, t / page_size] at t % page_size (table [B, width] int32), and it has
   lengths[b] (int32) of them, so its new token i sees those before lengths[b] -
   new_tokens + 1 + i. Both arrays are on the device and not checked on the host: a length
   is taken as min(max(length, 0), max_len), and tokens of a page that is not of the cache (-1, say)
   take no part. max_len (the largest length to come; at most width*page_size, below
   2^30) decides whether long sequences are divided, and with it the workspace. out [B*new_tokens,
   heads, head_dim], lse [B*new_tokens, heads]. The weights, each with its value's
   scale, are rounded to f16, and the matrix unit cuts products off: a score is off by up to
   2^-17 of a key's scale times the largest |q| for each channel, an output by 2^-13 of the
   largest weight times scale of 8 neighbouring tokens for each token, of those that the row sees;
   what is below 2^-30 of the row's largest weight times scale may be lost, and so may keys of less
   than 2^-117 of the largest weight. B*new_tokens = 0 is a no-op;
   new_tokens <= 256, B*heads*new_tokens < 2^31, and B*(cache heads)*ceil(rows/16) < 2^23 for
   the new_tokens*heads/(cache heads) rows of a key head. No host synchronisation: the call can
   be captured in a HIP graph and replayed with other lengths and tables. Two calls that may
   overlap need workspaces of their own. */
ar_status ar_kv4_attention(const ar_kv4_cache* cache, const uint16_t* q, int64_t q_stride,
                           int64_t B, int64_t new_tokens, int64_t heads, const int32_t* table,
                           int64_t width, const int32_t* lengths, int64_t max_len, float scale,
                           uint16_t* out, float* lse, void* ws, size_t ws_bytes, void* stream);

/* ---- Sequential block-wise tuning with quantized inputs --------------------
   [LLMC] tuning loop (each Linear of a subgraph tuned in turn on its captured
   inputs and targets), parameter table and "enable_quanted_input 모드" (the
   previous layers' quantized output as input), design point 3 (layer by
   layer). The pages do not show the block; a Llama-style decoder block is
   used: a = RMSNorm(h); q, k, v = a·W{q,k,v}ᵀ; rotate-half rotary embedding
   on q and k (theta rope_theta, position = token index within its sequence);
   causal softmax(q·kᵀ/sqrt(Dh))·v per sequence and head; h1 = h + attn·Woᵀ;
   m = RMSNorm(h1); z = SiLU(m·Wgᵀ)·(m·Wuᵀ); out = h1 + z·Wdᵀ. bf16
   activations between operations. */
typedef struct {
  int64_t hidden;       /* D                                  */
  int64_t heads;        /* H; head_dim D/H must be 64 or 128  */
  int64_t inter;        /* F (MLP width)                      */
  int64_t seqlen;       /* tokens per calibration sequence    */
  int64_t nsamples;     /* calibration sequences              */
  float rms_eps;
  float rope_theta;
} ar_block_dims;

typedef struct {        /* bf16 [out, in] row-major; norms bf16 [D] */
  const uint16_t *Wq, *Wk, *Wv, *Wo, *Wg, *Wu, *Wd;
  const uint16_t *norm_attn, *norm_mlp;
} ar_block_weights;

/* Per Linear, in the order q, k, v, o, gate, up, down: codes [N, K] uint8,
   scale [N, G] float32, zp [N, G] uint8, Wq [N, K] bf16 (all required),
   losses [iters] float32 (nullable). out_fp / out_q [M, D] bf16: the block
   output with the original / the tuned weights (nullable). */
typedef struct {
  uint8_t* codes[7];
  float* scale[7];
  uint8_t* zp[7];
  uint16_t* Wq[7];
  float* losses[7];
  uint16_t* out_fp;
  uint16_t* out_q;
} ar_block_outputs;

/* Workspace bytes for ar_block_forward (cfg NULL) or ar_tune_block (cfg set;
   cfg->nsamples * cfg->seqlen must equal the block's token count). */
ar_status ar_block_workspace_size(const ar_config* cfg, const ar_block_dims* dims, size_t* bytes);

/* The block's forward on h [nsamples*seqlen, D] bf16 -> out (same shape). */
ar_status ar_block_forward(const ar_block_dims* dims, const ar_block_weights* w,
                           const uint16_t* h, uint16_t* out, void* ws, size_t ws_bytes,
                           void* stream);

/* The block's attention step alone: out = causal softmax(q·kᵀ/sqrt(Dh))·v per
   sequence (dims->seqlen consecutive rows) and head (dims->heads column groups
   of Dh = hidden/heads, 64 or 128), with q and k already rotated. q, k, v, out
   [nsamples·seqlen, hidden] bf16 row-major, 16-byte aligned; float32
   accumulation and softmax, bf16 output. No workspace. */
ar_status ar_attention(const ar_block_dims* dims, const uint16_t* q, const uint16_t* k,
                       const uint16_t* v, uint16_t* out, void* stream);

/* Tune the block's seven Linears in order q, k, v, o, gate, up, down, each with
   ar_tune_linear on target Y = its full-precision output (the block with the
   original weights on h) and input X = its input in the quantized pipeline
   (quanted_input != 0: the block on h_q with the Linears tuned so far replaced
   by their bf16 Ŵ; h_q NULL means h) or in the full-precision pipeline
   (quanted_input = 0). cfg as for ar_tune_linear with nsamples*seqlen = the
   block's tokens. Blocks until the host has enqueued all work. */
ar_status ar_tune_block(const ar_config* cfg, const ar_block_dims* dims,
                        const ar_block_weights* w, const uint16_t* h, const uint16_t* h_q,
                        int32_t quanted_input, const ar_block_outputs* outs, void* ws,
                        size_t ws_bytes, void* stream);

/* ---- Per-layer configuration ([SGL] "2. 레이어별 개별 설정", "3. 정규식 기반
   레이어 매칭", "4. FusedMoE와 Fused QKV 처리"). Host-only calls: strings and
   arrays are host memory, nothing touches the GPU. -------------------------- */

/* One per-layer rule. The key is an exact layer name, or a pattern when it
   contains any of the characters * + ? ^ $ ( ) [ ] { } | \ (ECMAScript regular
   expression, matched against the whole name). */
typedef struct {
  const char* key;
  int32_t bits;         /* < 0: not set                      */
  int32_t group_size;   /* 0: not set (-1 is "whole row")    */
  int32_t sym;          /* < 0: not set, else 0 / 1          */
} ar_layer_rule;

typedef struct {
  int32_t bits;         /* 16: leave the layer unquantized   */
  int32_t group_size;
  int32_t sym;
} ar_layer_qconfig;

/* Config of layer `name`. quantized = 0 marks a layer outside the quantized
   set: with no rule, or an exact-name rule leaving fields unset, it gets
   bits 16, group_size -1, sym 1. Order: exact key, then the first pattern key
   that fully matches (keys that do not compile are skipped; unset fields from
   *defaults), then the fallback. AR_ERR_INVALID_ARG on NULL arguments. */
ar_status ar_resolve_layer_config(const ar_layer_rule* rules, int32_t nrules,
                                  const ar_layer_qconfig* defaults, int32_t quantized,
                                  const char* name, ar_layer_qconfig* out);

/* Config of a fused layer: every sub-layer must resolve to the same config,
   else AR_ERR_INVALID_ARG. With sub_names set (nsub > 0) the sub-layers are
   sub_names (a fused q/k/v-style layer). With sub_names NULL (nsub = 0) they
   are the rule keys that start with layer_name (a fused expert layer); with
   no such key, layer_name itself. sub_names set with nsub = 0 (an empty
   sub-layer list) is AR_ERR_INVALID_ARG, as is sub_names NULL with nsub > 0. */
ar_status ar_resolve_fused_config(const ar_layer_rule* rules, int32_t nrules,
                                  const ar_layer_qconfig* defaults, int32_t quantized,
                                  const char* layer_name, const char* const* sub_names,
                                  int32_t nsub, ar_layer_qconfig* out);

/* ---- Gram form (same-input Linears) --------------------------------------
   For one Linear the quantized and the reference outputs see the same tokens,
   so the minibatch loss and its gradient depend on the tokens only through
   H = Xbᵀ·Xb (the Hessian weight of the layer objective, ADMM-Q page "1. 문제
   공식화"), Cn = (Xb·Wᵀ - Yb)ᵀ·Xb and e2 = |Xb·Wᵀ - Yb|²: with D = bf16(Ŵ) - W,
     sum(R²) = Σ D∘(D·H) + 2·Σ D∘Cn + e2,   dL/dŴ = (2/(Tb·N))·(D·H + Cn).
   This is the [LLMC] output-reconstruction loss with the residual kept
   unrounded (the token form rounds dY to bf16), at 2·N·K·3K product FLOP per
   step instead of 4·Tb·K·N: D·H runs as bf16 MFMA on a hi/lo split
   (D_hi·H_hi + D_hi·H_lo + D_lo·H_hi, float32 accumulation). The statistics
   are computed once per minibatch (three products of the minibatch's tokens).
   Everything else (quantizer, straight-through fold, SignSGD, snapshot,
   finalisation) is the token form's. */

/* Bytes of device workspace for ar_tune_linear_gram (wdt: dtype of W). */
ar_status ar_gram_workspace_size(const ar_config* cfg, int32_t wdt, int64_t N, int64_t K,
                                 int32_t ydt, size_t* bytes);

/* Bytes of device workspace for ar_tune_step_gram with a minibatch of Tb tokens. */
ar_status ar_gram_step_workspace_size(const ar_config* cfg, int32_t wdt, int64_t N, int64_t K,
                                      int64_t Tb, int32_t ydt, size_t* bytes);

/* ar_tune_step in the Gram form: same arguments, state semantics and outputs
   (loss_out = sum(R²)/(Tb·N) with R unrounded; gradients from D·H + Cn). The
   minibatch's statistics are computed inside the call. ws:
   ar_gram_step_workspace_size bytes. */
ar_status ar_tune_step_gram(const ar_config* cfg, const ar_state* state, const uint16_t* Xb,
                            const void* Yb, int32_t ydt, int64_t Tb, float* loss_out, float* gV,
                            float* galpha, float* gbeta, int32_t apply_update, void* ws,
                            size_t ws_bytes, void* stream);

/* ar_tune_linear in the Gram form: same arguments and outputs. ws:
   ar_gram_workspace_size bytes (the per-minibatch H and Cn live there: nb·(6·K·K
   + 4·N·K) bytes for nb = nsamples/batch_samples minibatches). With times,
   fwd_gemm_ms is the product D·H, ste_update_ms the update kernel and
   wgrad_gemm_ms is 0. */
ar_status ar_tune_linear_gram(const ar_config* cfg, int32_t wdt, const void* W, int64_t N,
                              int64_t K, const uint16_t* X, const void* Y, int32_t ydt,
                              uint8_t* codes, float* scale, uint8_t* zp, void* Wq, float* V_out,
                              float* alpha_out, float* beta_out, float* losses, void* ws,
                              size_t ws_bytes, ar_kernel_times* times, void* stream);

/* Pack codes into 32-bit words ([SGL] pack_factor = Fraction(32, bits); GPTQ-style
   layout): code (n, k) occupies bits [k*bits, (k+1)*bits) of the bit string of
   column n, least significant bit first, so word w of column n is
   qweight[w, n] (a 3-bit code that straddles two words is split, low bits first).
   codes [N, K] uint8 -> qweight [K*bits/32, N] int32.
   zp [N, G] uint8 -> qzeros [G, N*bits/32] int32, same scheme along N (zp and
   qzeros nullable together). Requires K*bits % 32 == 0, and N*bits % 32 == 0
   when zp is given. N*K = 0 is a no-op. */
ar_status ar_pack(int32_t bits, const uint8_t* codes, const uint8_t* zp, int64_t N, int64_t K,
                  int64_t G, int32_t* qweight, int32_t* qzeros, void* stream);

/* Inverse of ar_pack (same shapes and constraints). */
ar_status ar_unpack(int32_t bits, const int32_t* qweight, const int32_t* qzeros, int64_t N,
                    int64_t K, int64_t G, uint8_t* codes, uint8_t* zp, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* AUTOROUND_HIP_H */
