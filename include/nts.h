/*
 * nts.h -- C ABI of libnts, GB300 (sm_103a) kernels for per-token RMS
 * normalization: split-H layerwise QK-RMSNorm, fused RMSNorm + MX cast, and
 * MXNorm + MX cast; and for the QKV projection between them: block-128 E4M3
 * casts, the block-scaled 8-bit matrix product, products of few rows with
 * 4-bit weights, the residual's addition with RMSNorm and the cast, and headwise
 * QK-RMSNorm with the rotary position embedding of one or several axes, the
 * last two forward and backward.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Pointers named *_dev are device pointers (cudaMalloc'd, or owned by a
 *    framework such as PyTorch); pointers named *_host are host pointers
 *    (pinned memory gives asynchronous copies).  Entry points without a
 *    suffix take device pointers only.  The caller owns every buffer; the
 *    library allocates no device memory at run time.  Its static device
 *    state: one status word per kernel family, a 512 KB pool of tile
 *    counters (a pair per stream, and one per launch recorded into a CUDA
 *    graph), and the 16 MiB staging array of nts_mxnorm_cast_host_noalloc.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream).  Calls only enqueue work and return; results are ready once
 *    the stream has reached that point.  Kernels are launched as
 *    programmatic dependents: one may be scheduled while the previous
 *    kernel in the stream drains, but it touches no global memory before
 *    that kernel has completed, so stream order holds as usual.
 *  - Matrices are row-major with one token per row: element (t, j) of a
 *    [T, H] matrix is at index t*H + j.  bf16 means IEEE-style bfloat16
 *    (uint16 storage).  Device pointers must be 16-byte aligned.
 *  - Return value: an nts_status.  Nothing is launched when the status is
 *    not NTS_OK, and no call aborts or throws.  nts_last_error() gives a
 *    human-readable detail for the calling thread.
 *  - T == 0 is valid and launches nothing; the data pointers may then be
 *    NULL (an empty tensor's storage), the other arguments are still checked.
 *
 * Sources (web pages), by title and section:
 *   SwiftQK: Fast and Communication-Efficient Tensor Parallelism for
 *   Query-Key Normalization (IEEE CAL) -- Eq. (1), Sec. III.A-D, Algorithm 1;
 *   the SwiftQK reading notes (zhongzhuzhou.org) -- Eq. (1), Sec. 3, Sec. 4b;
 *   the MXNorm paper card (arXiv 2603.13180) -- abstract, Fig. 1 caption,
 *   Fig. 8, Fig. A.1.
 */
#ifndef NTS_H
#define NTS_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define NTS_API __attribute__((visibility("default")))
#else
#define NTS_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    NTS_OK = 0,
    NTS_ERR_INVALID_ARG = 1, /* null required pointer, bad size/shape/eps/N/B/fmt/p; from
                                nts_check_status: a position outside the rotation table */
    NTS_ERR_UNSUPPORTED = 2, /* valid request this build cannot run: misaligned
                                pointer, row too wide, cluster not launchable */
    NTS_ERR_CUDA = 3,        /* a CUDA runtime call, a launch, or the host's own part
                                of one failed */
    NTS_ERR_TIMEOUT = 4      /* a kernel's bounded wait expired (nts_check_status) */
} nts_status;

typedef enum {
    NTS_FMT_E4M3 = 0, /* OCP E4M3: 1 byte per element, max 448; E8M0 scales (MXFP8) */
    NTS_FMT_E2M1 = 1, /* OCP E2M1: 4 bits per element, max 6; E8M0 scales (MXFP4) */
    NTS_FMT_NVFP4 = 2 /* E2M1 elements, B = 16, one E4M3 scale per block (NVFP4) */
} nts_elem_fmt;

typedef enum {
    NTS_OUT_BF16 = 0,
    NTS_OUT_FP32 = 1
} nts_out_type;

/* Codes of 4-bit weights, two to a byte, the even one's in bits 0 to 3: E2M1, or
   two's complement. */
typedef enum {
    NTS_W4_E2M1 = 0,
    NTS_W4_INT4 = 1
} nts_w4_fmt;

/* Library version, major*10000 + minor*100 + patch. */
NTS_API int nts_version(void);

/* Static string naming a status code. */
NTS_API const char *nts_status_string(int status);

/* Detail of the calling thread's most recent failure ("" if none). */
NTS_API const char *nts_last_error(void);

/*
 * nts_qknorm_rms -- layerwise QK-RMSNorm of every token row, computed as
 * split-H scalar partial sums (SwiftQK Eq. (1) and Algorithm 1):
 *
 *     S_k    = sum over columns [k*H/N, (k+1)*H/N) of x_j^2    (Phase A, fp32)
 *     S      = S_0 + ... + S_{N-1}                            (rank order)
 *     rinv   = 1 / sqrt(S / H + eps)          (H is the FULL row width)
 *     y_j    = bf16_rne((x_j * gamma_j) * rinv)                (Phases B, C)
 *
 * The N shards of a row are N CTAs of one thread-block cluster; each keeps
 * its shard on chip, exchanges its partial sum through distributed shared
 * memory, and forms x*gamma while the exchange is in flight.  N changes only
 * the work decomposition and the fp32 summation order, never the result's
 * definition.
 *
 *   X_dev      bf16 [T, H], read.            gamma_dev  fp32 [H], read.
 *   Y_dev      bf16 [T, H], written.  Y_dev == X_dev (in place) is allowed;
 *              any other overlap is undefined.
 *   rinv_dev   fp32 [T], written, or NULL.
 *   T >= 0; H >= 8; H % N == 0; (H / N) % 8 == 0; H / N <= 30720;
 *   eps > 0 and finite; N in {1, 2, 4, 8}.
 * Errors: INVALID_ARG (null X/gamma/Y, T < 0, H <= 0, H % N, bad eps or N),
 *         UNSUPPORTED ((H/N) % 8 != 0, slice too wide, unaligned pointer,
 *         cluster shape not launchable), CUDA (launch failure).
 */
NTS_API int nts_qknorm_rms(const void *X_dev, const float *gamma_dev, void *Y_dev,
                   float *rinv_dev, int64_t T, int64_t H, float eps, int N,
                   void *stream);

/*
 * nts_qknorm_rms_fp8 -- nts_qknorm_rms on FP8-E4M3 activations (SwiftQK
 * Sec. IV.C evaluates bf16 and FP8-E4M3 activations; the squares and the
 * combine stay fp32).  X_dev holds OCP E4M3 codes, uint8 [T, H]; the
 * activation is code * x_scale (a per-tensor dequantization scale, > 0 and
 * finite).  gamma, Y (bf16), rinv, N and the errors are those of
 * nts_qknorm_rms, plus UNSUPPORTED when (H / N) % 16 != 0 (a shard's row must
 * be a whole number of 16-byte vectors).  Y must not overlap X.
 */
NTS_API int nts_qknorm_rms_fp8(const void *X_dev, float x_scale, const float *gamma_dev,
                               void *Y_dev, float *rinv_dev, int64_t T, int64_t H, float eps,
                               int N, void *stream);

/*
 * nts_qknorm_rms_heads -- headwise QK-Norm (SwiftQK Sec. II.A: one
 * normalization factor per attention head instead of one per projected
 * vector).  X holds T tokens of H = nheads * head_dim values, the heads one
 * after another; head h of token t is normalized over its own head_dim
 * values:  rinv[t][h] = 1/sqrt((1/head_dim) sum x^2 + eps),
 * y = bf16_rne((x * gamma) * rinv), with gamma of head_dim entries shared by
 * all heads.  N splits every head across the CTAs of a cluster exactly as in
 * nts_qknorm_rms (head_dim % N == 0, (head_dim / N) % 8 == 0).
 *   X_dev, Y_dev  bf16 [T, H] (in place allowed); gamma_dev fp32 [head_dim];
 *   rinv_dev      fp32 [T, H/head_dim] or NULL.
 * Errors: as nts_qknorm_rms, plus INVALID_ARG for head_dim <= 0 or
 * H % head_dim != 0.
 */
NTS_API int nts_qknorm_rms_heads(const void *X_dev, const float *gamma_dev, void *Y_dev,
                                 float *rinv_dev, int64_t T, int64_t H, int64_t head_dim,
                                 float eps, int N, void *stream);

/*
 * nts_layernorm_split -- LayerNorm with the split-H statistic exchange
 * (SwiftQK reading notes, Sec. 5e: the variance is (1/H) sum x^2 - mu^2, so
 * a shard needs only two additive scalars, its sum and its sum of squares,
 * and the Phase A/B/C structure of nts_qknorm_rms carries over with two
 * scalars per shard instead of one):
 *
 *     s1_k, s2_k = sums over shard k of x_j and x_j^2            (fp32)
 *     mu    = (s1_0 + ... + s1_{N-1}) / H
 *     var   = max((s2_0 + ... + s2_{N-1}) / H - mu^2, 0)
 *     rstd  = 1 / sqrt(var + eps)
 *     y_j   = bf16_rne((x_j * rstd - mu * rstd) * gamma_j + beta_j)
 *
 * which is (x_j - mu) * rstd * gamma_j + beta_j (fp32 fused multiply-adds).  The one-pass variance
 * loses relative accuracy when |mu| is large against the spread of the row
 * (fp32 cancellation in s2/H - mu^2); the pages' formulation is kept.
 *   X_dev      bf16 [T, H], read.     gamma_dev  fp32 [H], read.
 *   beta_dev   fp32 [H], read, or NULL (no shift).
 *   Y_dev      bf16 [T, H], written (Y == X allowed).
 *   mean_dev   fp32 [T], written, or NULL.   rstd_dev  fp32 [T], or NULL.
 *   Limits as nts_qknorm_rms, except H / N <= 20480 when beta is given (the
 *   shard's gamma and beta both stay in shared memory).
 * Errors: as nts_qknorm_rms.
 */
NTS_API int nts_layernorm_split(const void *X_dev, const float *gamma_dev,
                                const float *beta_dev, void *Y_dev, float *mean_dev,
                                float *rstd_dev, int64_t T, int64_t H, float eps, int N,
                                void *stream);

/*
 * nts_qknorm_rms_qk -- nts_qknorm_rms of a token batch's Q and K in ONE
 * launch (one persistent grid walks the tiles of both tensors).  Q and K may
 * have different widths (Hq, Hk: e.g. grouped-query attention, where K is
 * narrower) and their own gains; they share T, eps and N.  Each tensor obeys
 * the argument rules of nts_qknorm_rms (in-place Yq == Q, Yk == K allowed;
 * rinv_* nullable); the same errors apply.  Layerwise QK-Norm normalizes Q
 * and K separately (SwiftQK Sec. II.A); fusing the two calls halves the
 * launches, which dominate at decode sizes.
 */
NTS_API int nts_qknorm_rms_qk(const void *Q_dev, const float *gamma_q_dev, void *Yq_dev,
                              float *rinv_q_dev, const void *K_dev,
                              const float *gamma_k_dev, void *Yk_dev, float *rinv_k_dev,
                              int64_t T, int64_t Hq, int64_t Hk, float eps, int N,
                              void *stream);

/*
 * nts_qknorm_rms_mxcast -- layerwise QK-RMSNorm with the split-H exchange of
 * nts_qknorm_rms, whose normalized rows leave as an MX (or NVFP4) block cast
 * instead of bf16: the QK path's Phase C feeds the block stage of
 * nts_rmsnorm_mxcast (SwiftQK Sec. III.C writes only the final normalized
 * shard; the MXNorm card, Fig. 8, fuses normalization and cast into one
 * kernel).  With w_j = fp32(x_j * gamma_j) and rinv = 1/sqrt(S/H + eps),
 * S = S_0 + ... + S_{N-1} in rank order as in nts_qknorm_rms, the scales and
 * codes are exactly those nts_rmsnorm_mxcast defines for this w and rinv
 * (E8M0 scales for E4M3/E2M1, E4M3 scales for NVFP4).  Each block's absmax
 * is taken while the exchange is in flight; blocks never straddle shards.
 *   X_dev       bf16 [T, H], read.         gamma_dev  fp32 [H], read.
 *   codes_dev   uint8 [T, H] (E4M3) or [T, H/2] (E2M1, NVFP4), written,
 *               16-byte aligned.
 *   scales_dev  uint8 [T, H/B], written.   rinv_dev   fp32 [T] or NULL.
 *   Limits of nts_qknorm_rms, plus B in {16, 32, 64} (16 for NVFP4) and
 *   (H / N) % B == 0.
 * Errors: as nts_qknorm_rms; INVALID_ARG also for a null scales_dev, a bad
 *         B or fmt; UNSUPPORTED for (H / N) % B != 0.
 */
NTS_API int nts_qknorm_rms_mxcast(const void *X_dev, const float *gamma_dev,
                                  uint8_t *codes_dev, uint8_t *scales_dev, float *rinv_dev,
                                  int64_t T, int64_t H, float eps, int N, int B, int fmt,
                                  void *stream);

/*
 * nts_qknorm_rms_qk_mxcast -- nts_qknorm_rms_mxcast of a token batch's Q and
 * K in ONE launch, as nts_qknorm_rms_qk fuses nts_qknorm_rms: Q and K may
 * have different widths (Hq, Hk) and their own gains; they share T, eps, N,
 * B and fmt.  Each tensor's codes, scales and rinv follow the definition of
 * nts_qknorm_rms_mxcast.  Both tensors take the thread layout of the wider
 * shard: with Hq == Hk every result equals that of a one-tensor call bit for
 * bit; otherwise the narrower tensor's fp32 sum of squares may be added in
 * another order (rinv within fp32 rounding of the one-tensor call; its scales
 * and codes are decided with that rinv).  Each tensor obeys the argument
 * rules of nts_qknorm_rms_mxcast, and the same errors apply, for either.
 */
NTS_API int nts_qknorm_rms_qk_mxcast(const void *Q_dev, const float *gamma_q_dev,
                                     uint8_t *codes_q_dev, uint8_t *scales_q_dev,
                                     float *rinv_q_dev, const void *K_dev,
                                     const float *gamma_k_dev, uint8_t *codes_k_dev,
                                     uint8_t *scales_k_dev, float *rinv_k_dev, int64_t T,
                                     int64_t Hq, int64_t Hk, float eps, int N, int B, int fmt,
                                     void *stream);

/*
 * nts_rmsnorm_mxcast -- RMSNorm fused with the MX cast (MXNorm card,
 * Fig. 1 caption, left graph; Fig. 8, where the normalization and the cast
 * are one fused kernel):
 *
 *     rinv     = 1 / sqrt((1/D) sum_j x_j^2 + eps)      (statistic of x, fp32)
 *     w_j      = fp32(x_j * gamma_j), or x_j when gamma_dev is NULL
 *     amax_k   = max over block k (B contiguous elements) of |w_j|
 *     e_k      = round(log2(fp32(amax_k * rinv))) - emax, clamped to
 *                [-127, 127], where round() is to the nearest integer in the
 *                log2 domain (mantissa >= sqrt 2 rounds up) and emax = 8
 *                (E4M3: the scale divides the absmax by 256) or 2 (E2M1)
 *     scale_k  = e_k + 127                                   (E8M0 byte)
 *     code_j   = cast_rne_satfinite(fp32(w_j * rinv) * 2^-e_k)
 *
 *   X_dev       bf16 [T, D], read.    gamma_dev fp32 [D], read, or NULL.
 *   codes_dev   E4M3: uint8 [T, D]; E2M1: uint8 [T, D/2] with element 2i in
 *               bits 0-3 and element 2i+1 in bits 4-7 of byte i.  Written.
 *   scales_dev  uint8 [T, D/B] E8M0 codes (2^(code-127)), row-major. Written.
 *   rinv_dev    fp32 [T] or NULL.   amax_dev  fp32 [T, D/B] block absmaxes
 *               of w (before normalization) or NULL.
 *   T >= 0; D % B == 0; B in {16, 32, 64}; D <= 32768; eps > 0 and finite;
 *   fmt in nts_elem_fmt.
 *
 * fmt = NTS_FMT_NVFP4 (B must be 16; the MXNorm card lists NVFP4 among its
 * kernel cases, Table 4, without its rules; this is the reading taken):
 *     s_k      = E4M3_rne_satfinite(fp32(fp32(amax_k * rinv) / 6))
 *     scale_k  = the E4M3 code of s_k
 *     code_j   = E2M1_rne_satfinite(fp32(fp32(w_j * rinv) * fp32(1 / s_k))),
 *                or 0 for every element of a block whose s_k is 0;
 * codes are laid out as for E2M1; no per-tensor second-level scale.
 * Errors: INVALID_ARG (null X/codes/scales, T < 0, D <= 0, D % B, bad B,
 *         eps or fmt, NVFP4 with B != 16), UNSUPPORTED (row too wide,
 *         unaligned pointer), CUDA (launch failure).
 */
NTS_API int nts_rmsnorm_mxcast(const void *X_dev, const float *gamma_dev,
                       uint8_t *codes_dev, uint8_t *scales_dev,
                       float *rinv_dev, float *amax_dev, int64_t T, int64_t D,
                       float eps, int B, int fmt, void *stream);

/*
 * nts_mxnorm_cast -- MXNorm (MXNorm card, abstract and Fig. 1 caption,
 * right graph): the RMS is estimated from the K = D/B block absmaxes that the
 * MX cast computes anyway,
 *
 *     rho~  = c(B, p) * ((1/K) sum_k amax_k^p)^(1/p),   p in {1, 2}
 *     rinv  = 1 / sqrt(rho~^2 + eps)
 *
 * then the block stage of nts_rmsnorm_mxcast runs with this rinv (the
 * normalized block absmax is amax_k * rinv, so no second reduction).  w, the
 * tensor whose absmaxes are taken and which is cast, is x (gamma_dev NULL,
 * the gain folded into the next Linear layer) or fp32(x * gamma).
 * c(B, p) = E[max of B i.i.d. |N(0,1)|^p]^(-1/p) (nts_mxnorm_correction).
 * Arguments, layouts and errors as nts_rmsnorm_mxcast, plus p in {1, 2}
 * (INVALID_ARG otherwise).
 */
NTS_API int nts_mxnorm_cast(const void *X_dev, const float *gamma_dev,
                    uint8_t *codes_dev, uint8_t *scales_dev, float *rinv_dev,
                    float *amax_dev, int64_t T, int64_t D, float eps, int B,
                    int fmt, int p, void *stream);

/*
 * nts_mxnorm_postround_cast -- the "post-round" MXNorm scheme (MXNorm card,
 * Fig. A.4, which names it and reports it trains unstably; reading): the RMS
 * estimate takes every block absmax after the E8M0 power-of-two rounding,
 *     rho~ = c(B, p) * ((1/K) sum_k (2^round(log2 amax_k))^p)^(1/p),
 * with the same c(B, p); the cast (scales and codes from amax_k * rinv) is
 * that of nts_mxnorm_cast.  Arguments, layouts and errors as
 * nts_mxnorm_cast; the rounding is that of E8M0 scales, so fmt =
 * NTS_FMT_NVFP4 is INVALID_ARG here.
 */
NTS_API int nts_mxnorm_postround_cast(const void *X_dev, const float *gamma_dev,
                                      uint8_t *codes_dev, uint8_t *scales_dev,
                                      float *rinv_dev, float *amax_dev, int64_t T, int64_t D,
                                      float eps, int B, int fmt, int p, void *stream);

/*
 * nts_mxnorm_correction -- the correction factor c(B, p) used by
 * nts_mxnorm_cast (MXNorm card, Fig. 1 caption: the scalar making the
 * estimate equal the RMS for i.i.d. Gaussian rows), computed on the host by
 * quadrature.  B >= 1, p in {1, 2}; *c_out receives the value.
 * Errors: INVALID_ARG.
 */
NTS_API int nts_mxnorm_correction(int B, int p, double *c_out);

/*
 * nts_rope_table_host -- the table of nts_qknorm_rope, on the host: row pos
 * holds the cosines of the rot_dim/2 angles pos * base^(-2i/rot_dim), then
 * their sines, each formed in double precision (far positions keep their
 * angle) and rounded once to fp32.
 *   table_host  fp32 [P, rot_dim], written.   base > 0 and finite.
 * Errors: INVALID_ARG.
 */
NTS_API int nts_rope_table_host(int64_t P, int64_t rot_dim, double base, float *table_host);

/*
 * nts_qknorm_rope -- headwise QK-RMSNorm (nts_qknorm_rms_heads) of a token
 * batch's Q and K with the rotary position embedding in the same pass, one
 * launch.  Per head of head_dim = d values of the token at position pos:
 *
 *     rinv = 1 / sqrt((1/d) sum x^2 + eps)                       (fp32)
 *     n_j  = (x_j * gamma_j) * rinv                              (fp32)
 *     y_a  = n_a c - n_b s,   y_b = n_b c + n_a s     for every pair (a, b)
 *            of the first rot_dim values, with c = table[pos][i] and
 *            s = table[pos][rot_dim/2 + i], i the pair's number
 *     y_j  = n_j                                      for j >= rot_dim
 *
 * and one rounding to bf16.  Pair i is (i, i + rot_dim/2), or (2i, 2i + 1)
 * when `interleaved` is not 0.
 *
 *   Q_dev, K_dev    bf16, row t at t*ldq (t*ldk) elements: nheads_q (nheads_k)
 *                   heads of head_dim values one after another.  Row strides
 *                   let both be columns of one packed QKV buffer.
 *   Yq_dev, Yk_dev  the same layout with strides ldyq, ldyk.  Y == X with the
 *                   same stride (in place) is allowed; any other overlap is
 *                   undefined.  Values between the rows are left alone.
 *   gamma_*_dev     fp32 [head_dim].
 *   rinv_*_dev      fp32 [T, nheads] or NULL.
 *   positions_dev   int64 [T].  A negative position marks a padding row: its
 *                   Q and K may hold anything, its Y is zeros and its rinv 0.
 *                   A position >= P gives the same zeros and is reported by
 *                   nts_check_status (INVALID_ARG).
 *   table_dev       fp32 [P, rot_dim], P >= 1 (nts_rope_table_host).
 *   T >= 0; head_dim a multiple of 16 up to 512; rot_dim a multiple of 16,
 *   0 < rot_dim <= head_dim; strides multiples of 8.
 * Errors: INVALID_ARG (null required pointer, bad sizes, eps, odd rot_dim or
 *         one beyond head_dim, a stride below the row), UNSUPPORTED (other
 *         head_dim or rot_dim, unaligned rows, T >= 2^31, more than 65536
 *         heads, T times the warp items of a token from 2^31: a warp takes
 *         32 / l heads of Q or of K, l the power of two from head_dim / 16
 *         up), CUDA.
 */
NTS_API int nts_qknorm_rope(const void *Q_dev, int64_t ldq, const float *gamma_q_dev,
                            void *Yq_dev, int64_t ldyq, float *rinv_q_dev, const void *K_dev,
                            int64_t ldk, const float *gamma_k_dev, void *Yk_dev, int64_t ldyk,
                            float *rinv_k_dev, const int64_t *positions_dev,
                            const float *table_dev, int64_t P, int64_t T, int64_t nheads_q,
                            int64_t nheads_k, int64_t head_dim, int64_t rot_dim,
                            int interleaved, float eps, void *stream);

/*
 * nts_qknorm_rope_backward -- the gradient of nts_qknorm_rope.  With g the
 * rotation of dy by the opposite angles and u_j = g_j gamma_j:
 *
 *     dx_j      = rinv (u_j - x_j rinv^2 (1/d) sum u x)          (bf16)
 *     dgamma_j  = sum over tokens and heads of g_j x_j rinv      (fp32)
 *
 * rinv is formed again from Q and K (the forward pass's inputs).  Padding
 * rows, and rows whose position lies outside the table, get zeros and add
 * nothing to dgamma; so does a head whose sum of squares is beyond fp32, with
 * rinv = 0.  The sums have a fixed order: equal calls give equal bits.
 *   dYq_dev, dYk_dev, dQ_dev, dK_dev  bf16, laid out as Q and K, each with its
 *                   own row stride; dQ == dYq or dQ == Q with the same stride
 *                   is allowed (dK likewise).
 *   dgamma_*_dev    fp32 [head_dim], overwritten (zeros when T == 0).
 *   workspace_dev   scratch of at least nts_qknorm_rope_backward_workspace()
 *                   bytes, 4-byte aligned, contents arbitrary before and
 *                   after; calls that overlap in time need one each.
 * Other arguments, limits and errors as nts_qknorm_rope; INVALID_ARG also for
 * a missing or short workspace, UNSUPPORTED for an eps below 2^-126.
 */
NTS_API int nts_qknorm_rope_backward(const void *dYq_dev, int64_t lddyq, const void *dYk_dev,
                                     int64_t lddyk, const void *Q_dev, int64_t ldq,
                                     const float *gamma_q_dev, const void *K_dev, int64_t ldk,
                                     const float *gamma_k_dev, const int64_t *positions_dev,
                                     const float *table_dev, int64_t P, void *dQ_dev,
                                     int64_t lddq, void *dK_dev, int64_t lddk,
                                     float *dgamma_q_dev, float *dgamma_k_dev,
                                     void *workspace_dev, int64_t workspace_bytes, int64_t T,
                                     int64_t nheads_q, int64_t nheads_k, int64_t head_dim,
                                     int64_t rot_dim, int interleaved, float eps, void *stream);

/* Workspace bytes of nts_qknorm_rope_backward.  Errors: INVALID_ARG. */
NTS_API int nts_qknorm_rope_backward_workspace(int64_t head_dim, int64_t *bytes_out);

/*
 * nts_qknorm_rope_axes, nts_qknorm_rope_axes_backward -- nts_qknorm_rope and
 * its gradient for tokens with a position on each of several axes (time,
 * height and width of images and video): pair i turns by the position on its
 * own axis,
 *
 *     c = table[pos_a][i],  s = table[pos_a][rot_dim/2 + i],
 *     pos_a = positions[t][a],  a = pair_axis[i].
 *
 * The table is the caller's: nts_rope_table_host's, whose pair i has one
 * frequency on every axis, or one whose columns start their frequencies anew
 * on each axis.
 *   positions_dev    int64, token t's on axis a at t*pos_stride_t +
 *                    a*pos_stride_a elements (strides >= 0): [T, naxes] or
 *                    [naxes, T].  A token with a negative position on any axis
 *                    is a padding row; one with none and a position >= P on an
 *                    axis gives the same zeros and is reported by
 *                    nts_check_status.
 *   naxes            1 to 4.
 *   pair_axis_host   uint8 [rot_dim/2] on the host, each below naxes, read
 *                    before the call returns.
 * Other arguments, limits and errors as nts_qknorm_rope and
 * nts_qknorm_rope_backward (its workspace too); INVALID_ARG also for another
 * naxes, an axis out of range or a negative stride, UNSUPPORTED for a table of
 * 2^31 values or more or a stride whose last position lies beyond 64-bit
 * addresses.
 */
NTS_API int nts_qknorm_rope_axes(const void *Q_dev, int64_t ldq, const float *gamma_q_dev,
                                 void *Yq_dev, int64_t ldyq, float *rinv_q_dev,
                                 const void *K_dev, int64_t ldk, const float *gamma_k_dev,
                                 void *Yk_dev, int64_t ldyk, float *rinv_k_dev,
                                 const int64_t *positions_dev, int64_t pos_stride_t,
                                 int64_t pos_stride_a, int naxes,
                                 const uint8_t *pair_axis_host, const float *table_dev,
                                 int64_t P, int64_t T, int64_t nheads_q, int64_t nheads_k,
                                 int64_t head_dim, int64_t rot_dim, int interleaved, float eps,
                                 void *stream);

NTS_API int nts_qknorm_rope_axes_backward(
    const void *dYq_dev, int64_t lddyq, const void *dYk_dev, int64_t lddyk, const void *Q_dev,
    int64_t ldq, const float *gamma_q_dev, const void *K_dev, int64_t ldk,
    const float *gamma_k_dev, const int64_t *positions_dev, int64_t pos_stride_t,
    int64_t pos_stride_a, int naxes, const uint8_t *pair_axis_host, const float *table_dev,
    int64_t P, void *dQ_dev, int64_t lddq, void *dK_dev, int64_t lddk, float *dgamma_q_dev,
    float *dgamma_k_dev, void *workspace_dev, int64_t workspace_bytes, int64_t T,
    int64_t nheads_q, int64_t nheads_k, int64_t head_dim, int64_t rot_dim, int interleaved,
    float eps, void *stream);

/*
 * nts_rmsnorm_blockcast -- RMSNorm fused with the cast to E4M3 codes that
 * carry one fp32 scale per block of 128 contiguous values (the last block of
 * a row may be shorter), the operand of nts_gemm_blockscaled:
 *
 *     rinv    = 1 / sqrt((1/D) sum_j x_j^2 + eps)                (fp32)
 *     w_j     = fp32(fp32(x_j * gamma_j) * rinv), or fp32(x_j * rinv)
 *     scale_k = fp32(max(absmax of block k, 2^-100) / 448)
 *     code_j  = E4M3_rne_satfinite(fp32(w_j * fp32(1 / scale_k)))
 *
 * so code * scale stands for w.  A NaN keeps its place as the NaN code; a
 * block that holds an infinity gets an infinite scale.
 *   X_dev       bf16 [T, D], read.       gamma_dev   fp32 [D] or NULL.
 *   codes_dev   uint8 [T, D], written.   scales_dev  fp32 [T, ceil(D/128)].
 *   rinv_dev    fp32 [T] or NULL.
 *   T >= 0; D a multiple of 16 up to 32768; eps > 0 and finite.
 * Errors: INVALID_ARG (null X/codes/scales, T < 0, D <= 0, bad eps),
 *         UNSUPPORTED (D % 16, D too wide, T >= 2^31, unaligned pointer), CUDA.
 */
NTS_API int nts_rmsnorm_blockcast(const void *X_dev, const float *gamma_dev, uint8_t *codes_dev,
                                  float *scales_dev, float *rinv_dev, int64_t T, int64_t D,
                                  float eps, void *stream);

/*
 * nts_add_rmsnorm_blockcast -- nts_rmsnorm_blockcast of the sum of a layer's
 * output and the residual stream, which is written too:
 *
 *     h_j  = round(x_j + r_j) to the stream's type
 *     rinv = 1 / sqrt((1/D) sum_j h_j^2 + eps)                   (fp32)
 *
 * and w, scales and codes of h as there (the order of the sum may differ by
 * fp32 roundings).  A row whose sum of squares is beyond fp32 gets rinv = 0.
 *   X_dev          bf16 [T, D].      residual_dev  [T, D], bf16 or fp32
 *                                    (residual_type, an nts_out_type).
 *   gamma_dev      fp32 [D] or NULL.
 *   H_dev          [T, D] in the stream's type; may be residual_dev, or X_dev
 *                  when that is its type too; any other overlap is undefined.
 *   codes_dev      uint8 [T, D].     scales_dev    fp32 [T, ceil(D/128)].
 *   rinv_dev       fp32 [T] or NULL.
 *   T >= 0; D a multiple of 16 up to 32768; eps > 0 and finite.
 * Errors: as nts_rmsnorm_blockcast; INVALID_ARG also for another type.
 */
NTS_API int nts_add_rmsnorm_blockcast(const void *X_dev, const void *residual_dev,
                                      const float *gamma_dev, void *H_dev, uint8_t *codes_dev,
                                      float *scales_dev, float *rinv_dev, int residual_type,
                                      int64_t T, int64_t D, float eps, void *stream);

/*
 * nts_add_rmsnorm_backward -- the gradient of nts_add_rmsnorm_blockcast, the
 * cast taken as exact.  With dy the gradient of w, u_j = dy_j gamma_j and e the
 * gradient of h from the layers behind:
 *
 *     dres_j   = rinv u_j - h_j rinv^3 (1/D) sum u h + e_j
 *     dgamma_j = sum over the rows of dy_j h_j rinv              (fp32)
 *
 * dres is the gradient of x and of the residual alike; that of a row with
 * rinv = 0 is e.  The sums have a fixed order: equal calls give equal bits.
 *   dY_dev         bf16 [T, D].      rinv_dev      fp32 [T], the forward pass's.
 *   H_dev, dH_dev  [T, D] in the stream's type (residual_type); dH (e) or NULL.
 *   gamma_dev      fp32 [D] or NULL.
 *   dres_dev       [T, D] in the stream's type; may be dH_dev or H_dev, or
 *                  dY_dev when that is its type too.
 *   dX_dev         bf16 [T, D] or NULL: dres of an fp32 stream rounded once
 *                  more, for the product behind; may be dY_dev.
 *   dgamma_dev     fp32 [D], overwritten (zeros when T == 0), or NULL.
 *   workspace_dev  with dgamma: scratch of at least
 *                  nts_add_rmsnorm_backward_workspace() bytes, 16-byte aligned,
 *                  contents arbitrary before and after; calls that overlap in
 *                  time need one each.
 *   T, D as above.
 * Errors: INVALID_ARG (null required pointer, bad sizes or type, dX of a bf16
 *         stream, dgamma without gamma, a missing or short workspace),
 *         UNSUPPORTED (D % 16, D too wide, T >= 2^31, unaligned pointer), CUDA.
 */
NTS_API int nts_add_rmsnorm_backward(const void *dY_dev, const void *H_dev, const float *rinv_dev,
                                     const float *gamma_dev, const void *dH_dev, void *dres_dev,
                                     void *dX_dev, float *dgamma_dev, void *workspace_dev,
                                     int64_t workspace_bytes, int residual_type, int64_t T,
                                     int64_t D, void *stream);

/* Workspace bytes of nts_add_rmsnorm_backward.  Errors: INVALID_ARG. */
NTS_API int nts_add_rmsnorm_backward_workspace(int64_t D, int64_t *bytes_out);

/*
 * nts_blockcast -- the cast of nts_rmsnorm_blockcast without the norm
 * (w = x), in blocks of block_rows x 128 values: 1 for activations and
 * gradients, 128 for weights.
 *   codes_dev   uint8 [T, D].
 *   scales_dev  fp32 [ceil(T / block_rows), ceil(D / 128)].
 *   D a multiple of 16; block_rows 1 or 128.
 * Errors: as nts_rmsnorm_blockcast, but D and T only have to stay below 2^31;
 * INVALID_ARG also for another block_rows, UNSUPPORTED also for 2^31 blocks of
 * 128 x 128 or more.
 */
NTS_API int nts_blockcast(const void *X_dev, uint8_t *codes_dev, float *scales_dev, int64_t T,
                          int64_t D, int block_rows, void *stream);

/*
 * nts_blockcast_t -- the transpose of X [T, D], cast in blocks of 128 tokens
 * of one column: the operands of a weight gradient, whose sums run over the
 * tokens.
 *   codes_dev   uint8 [D, Tp], Tp = T rounded up to a multiple of 16; the
 *               codes of the Tp - T tokens beyond T are zero.
 *   scales_dev  fp32 [D, ceil(T / 128)].
 *   D a multiple of 16; T at most 65535 * 128 = 8388480.
 * Errors: as nts_rmsnorm_blockcast, but D only has to stay below 2^31;
 * UNSUPPORTED also for more tokens.
 */
NTS_API int nts_blockcast_t(const void *X_dev, uint8_t *codes_dev, float *scales_dev, int64_t T,
                            int64_t D, void *stream);

/*
 * nts_gemm_blockscaled -- matrix product of E4M3 operands with one fp32 scale
 * per block of 128 values along K, on the tensor cores:
 *
 *     Y[m][n] = sum_kb a_scales[m][kb] w_scales[n'][kb]
 *                   sum_{k in block kb} A[m][k] W[n][k]
 *
 * with n' = n / 128 (w_block_rows = 128: weights in 128 x 128 blocks) or n
 * (w_block_rows = 1).  Sums in fp32, one rounding to the output type.  For
 * Y = X W^T take A = the cast of X and W = nts_blockcast(.., 128); the
 * gradient of X is the same product of dY with the transposed weights (their
 * 128 x 128 scales transposed too); the gradient of W is the product of
 * nts_blockcast_t(dY) with nts_blockcast_t(X), w_block_rows = 1.
 *   A_codes_dev  uint8 [M, K].   a_scales_dev  fp32 [M, ceil(K/128)].
 *   W_codes_dev  uint8 [N, K].   w_scales_dev  fp32 [ceil(N/128) or N,
 *                                              ceil(K/128)].
 *   Y_dev        bf16 or fp32 [M, N] (out_type, an nts_out_type), written;
 *                overlaps no operand.
 *   M >= 0; N > 0; K a positive multiple of 16 (the last block may be
 *   shorter than 128).
 * The order of the sums depends on the shape alone: equal calls give equal
 * bits.
 * Errors: INVALID_ARG (null pointer, bad sizes, w_block_rows or out_type),
 *         UNSUPPORTED (K % 16, unaligned codes or Y, sizes from 2^31 - 256),
 *         CUDA.
 */
NTS_API int nts_gemm_blockscaled(const uint8_t *A_codes_dev, const float *a_scales_dev,
                                 const uint8_t *W_codes_dev, const float *w_scales_dev,
                                 int w_block_rows, void *Y_dev, int out_type, int64_t M,
                                 int64_t N, int64_t K, void *stream);

/*
 * nts_gemv_groupscaled -- product of few rows with weights of 4 bits, which
 * carry a bf16 scale per group of 32, 64 or 128 values along K (the last group
 * of a row may be shorter):
 *
 *     Y[m][n] = sum_g w_scales[n][g] sum_{k in group g} A[m][k] W[n][k]
 *
 * Sums in fp32, one rounding to the output type.  Up to 8 rows cost what one
 * does; 16 are one pass over the weights, more are passes of 16, or of 32 with
 * more than 4096 x 4096 weights.  From 9 rows on weights of 8 bits and
 * nts_gemm_blockscaled take less time, at twice the memory.
 * What may leave fp32's range on the way though the output would not: in passes
 * of 16, outputs of group scales above 2^102 (128 values along K are raised to
 * 2^14 and more by a power of two that comes off behind the scales); in those
 * of 32, bf16 values from about 2^117 on (a group's products are summed before
 * its scale multiplies them).
 *   A_dev         with a_scales NULL: bf16, row m at m*lda elements, a value that
 *                 is below 2^-31 of the largest of its 128 neighbours along K
 *                 off by up to 2^-39 of that one; otherwise E4M3 codes (uint8)
 *                 with one fp32 scale per 128 values, as nts_gemm_blockscaled
 *                 takes them.
 *   a_scales_dev  fp32 [M, ceil(K/128)] or NULL.
 *   W_codes_dev   uint8 [N, K/2] (fmt, an nts_w4_fmt).
 *   w_scales_dev  bf16 [N, ceil(K/group)].
 *   Y_dev         bf16 or fp32 [M, N] (out_type, an nts_out_type), written;
 *                 overlaps no operand.
 *   M >= 0; N > 0; K a positive multiple of 32 up to 32768; lda >= K, a multiple
 *   of 16 bytes.
 * The order of the sums depends on the shape alone: equal calls give equal
 * bits.
 * Errors: INVALID_ARG (null pointer, bad sizes, group, fmt or out_type, a stride
 *         below the row), UNSUPPORTED (K % 32, K too long, unaligned rows,
 *         codes, scales or Y, M above 65535 * 16, N from 2^31 - 256), CUDA.
 */
NTS_API int nts_gemv_groupscaled(const void *A_dev, int64_t lda, const float *a_scales_dev,
                                 const uint8_t *W_codes_dev, const void *w_scales_dev, int group,
                                 int fmt, void *Y_dev, int out_type, int64_t M, int64_t N,
                                 int64_t K, void *stream);

/*
 * nts_groupcast_host -- weights [N, K] to the operand of nts_gemv_groupscaled,
 * on the host:
 *
 *     scale = bf16(fp32(max(absmax of the group, 2^-100) / top)),
 *             top = 6 (E2M1) or 7 (int4)
 *     code  = the value nearest to fp32(w / scale), ties to the even code,
 *             saturating (int4: -7 to 7)
 *
 *   W_host       bf16 [N, K], finite.   codes_host   uint8 [N, K/2], written.
 *   scales_host  bf16 [N, ceil(K/group)], written.
 * Errors: INVALID_ARG (null pointer, bad sizes, group or fmt, a weight that is
 *         not finite), UNSUPPORTED (K % 32).
 */
NTS_API int nts_groupcast_host(const void *W_host, uint8_t *codes_host, void *scales_host,
                               int64_t N, int64_t K, int group, int fmt);

/*
 * nts_check_status -- synchronizes `stream`, then reads and clears the
 * device status words.  Returns NTS_ERR_TIMEOUT if any kernel since the last
 * check gave up on a bounded wait (its outputs are then undefined),
 * NTS_ERR_INVALID_ARG if a rotation call met a position outside its table,
 * NTS_ERR_CUDA if the stream reported an error, NTS_OK otherwise.
 */
NTS_API int nts_check_status(void *stream);

/*
 * Host-buffer forms: the same operations for callers whose inputs and
 * outputs live in host memory.  Each enqueues the host->device copy of the
 * input rows, the kernel, and the device->host copies of the outputs, all
 * ordered on `stream`: the caller synchronizes the stream before reading
 * *_host outputs.  Calls of more than 32 MB move their rows in up to 16
 * chunks through two internal copy streams (one per direction, created on
 * the first such call on a device) while the kernels run on `stream`, so
 * both copy directions and the kernels overlap; the enqueueing of such calls
 * from several host threads is serialized.  Host buffers should be pinned
 * for the copies to run asynchronously.
 * The device staging buffers (*_dev) are caller-owned and sized like the
 * corresponding host buffers; gamma stays a device pointer (a parameter,
 * uploaded once).  Optional outputs follow the device forms: a NULL *_host
 * output skips that output (its *_dev may then be NULL too).
 * Errors: as the device forms; CUDA also covers a failed copy.
 */
NTS_API int nts_qknorm_rms_host(const void *X_host, const float *gamma_dev,
                        void *Y_host, float *rinv_host, void *X_dev,
                        void *Y_dev, float *rinv_dev, int64_t T, int64_t H,
                        float eps, int N, void *stream);

/*
 * nts_qknorm_rms_qk_host -- nts_qknorm_rms_qk on host buffers: the copies of
 * Q and K to the device, the one launch that normalizes both, and the copies
 * of Yq and Yk back, enqueued as nts_qknorm_rms_host enqueues its work (in
 * row chunks through the library's copy streams for large calls; the
 * caller's stream is ordered after the last copy back).
 *   Q_host bf16 [T, Hq], K_host bf16 [T, Hk]: read.
 *   Yq_host, Yk_host: written once the stream reaches the end of the call.
 *   Q_dev, Yq_dev, K_dev, Yk_dev: caller-owned device staging of the same
 *   sizes (16-byte aligned); gamma_q_dev, gamma_k_dev: device gains.
 * Errors: as nts_qknorm_rms_qk; CUDA also covers a failed copy.
 */
NTS_API int nts_qknorm_rms_qk_host(const void *Q_host, const float *gamma_q_dev,
                                   void *Yq_host, const void *K_host,
                                   const float *gamma_k_dev, void *Yk_host, void *Q_dev,
                                   void *Yq_dev, void *K_dev, void *Yk_dev, int64_t T,
                                   int64_t Hq, int64_t Hk, float eps, int N, void *stream);

NTS_API int nts_rmsnorm_mxcast_host(const void *X_host, const float *gamma_dev,
                            uint8_t *codes_host, uint8_t *scales_host,
                            void *X_dev, uint8_t *codes_dev,
                            uint8_t *scales_dev, int64_t T, int64_t D,
                            float eps, int B, int fmt, void *stream);

NTS_API int nts_mxnorm_cast_host(const void *X_host, const float *gamma_dev,
                         uint8_t *codes_host, uint8_t *scales_host,
                         void *X_dev, uint8_t *codes_dev, uint8_t *scales_dev,
                         int64_t T, int64_t D, float eps, int B, int fmt,
                         int p, void *stream);

/*
 * nts_mxnorm_cast_host_noalloc -- nts_mxnorm_cast_host with no caller-owned
 * device buffers: the device staging for X, gamma, codes and scales is a
 * fixed 16 MiB array inside the library (one per device).  The pages have
 * no counterpart; it serves callers that cannot allocate device memory at
 * the call: processes whose device memory another framework's pool has
 * already reserved, latency-bound loops that must not call the allocator
 * after start-up (cudaFree synchronizes the device, cudaMalloc may), and
 * host-only callers with no device allocator.
 *
 *   X_host      bf16 [T, D], read.   gamma_host  fp32 [D], read, or NULL.
 *   codes_host, scales_host: as nts_mxnorm_cast_host, written once the
 *   stream reaches the end of the call's work.  Other arguments as
 *   nts_mxnorm_cast.
 *
 * Set-up: the first call on each device looks up the array's device address
 * (and fills the library's host-side launch caches: device facts, kernel
 * attributes, c(B, p), the stream's tile counters).  Its copies and its
 * kernel all run on `stream` in one piece, never chunked, so it never
 * creates the copy streams of the other host-buffer forms.  Make that first
 * call before any stream capture; later calls on that device and stream
 * allocate nothing, host or device.
 * Sharing: every call on a device uses the same array, so calls that overlap
 * in time (other streams, unordered host threads) race and corrupt each
 * other's staging; serialize them.  Nothing in the array needs to start at
 * zero: each call copies in all the kernel reads.
 * Errors: as nts_mxnorm_cast_host, and every argument is checked before
 * anything is enqueued; UNSUPPORTED when the call needs more than 16 MiB of
 * staging (2*T*D bytes of X, 4*D of gamma, T*D or T*D/2 of codes,
 * T*D/B of scales, each rounded up to 256 bytes), or for a device ordinal
 * of 64 or more.
 */
NTS_API int nts_mxnorm_cast_host_noalloc(const void *X_host, const float *gamma_host,
                                         uint8_t *codes_host, uint8_t *scales_host, int64_t T,
                                         int64_t D, float eps, int B, int fmt, int p,
                                         void *stream);

#ifdef __cplusplus
}
#endif

#endif /* NTS_H */
