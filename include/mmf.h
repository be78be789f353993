/*
 * mmf.h -- C ABI of the fused RMSNorm + BitLinear library for NVIDIA B200
 * (sm_100a).  Library: bitlinear_rmsnorm_quant_b200/libmmf.so.
 *
 * The layer is the BitLinear dense layer of the MatMul-free language model
 * ("Scalable MatMul-free Language Modeling", Zhu et al.):
 *   - weights are ternary {-1, 0, +1}, obtained from full-precision latent
 *     weights by absmean quantisation (datacamp.com, section "Thay MatMul bằng
 *     các phép toán tam phân"; jiqizhixin.com, section "具有三值权重的
 *     MatMul-free 密集层"), so the product needs only additions and
 *     subtractions (ld246.com, section "三值权重的应用");
 *   - the activations pass through RMSNorm before quantisation (datacamp.com,
 *     component figure, item "RMS norm"), and RMSNorm and quantisation are one
 *     fused operation that reads x from HBM once (ld246.com, section "融合
 *     BitLinear 层的创新"; jiqizhixin.com, Algorithm 1);
 *   - activations are quantised per token to int8 by absmax, accumulated in
 *     int32, and rescaled by (absmax/127) * mean|W|.  The pages give no
 *     formula; these are the plain definitions, stated per function below.
 *
 * Conventions for every entry point:
 *   - Pointers are DEVICE pointers owned by the caller unless stated.  The
 *     library never allocates, frees or caches device memory and keeps no
 *     pointer after a call returns.
 *   - Every pointer must be 16-byte aligned (TMA and 128-bit loads).
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Calls are asynchronous and ordered on that stream; results
 *     are ready when the stream has reached the call.
 *   - bf16 tensors are passed as uint16_t bit patterns.
 *   - Shapes: M tokens (0 <= M <= 16,776,960 = 65535 * 256; the scan states
 *     its own sizes), K = d_in (128 <= K <= 65536,
 *     K % 128 == 0), N = d_out (0 <= N < 2^31).  M == 0 or N == 0 is a no-op
 *     returning MMF_OK once the scalar arguments and K are valid; the buffer
 *     pointers of an empty problem are not checked and may be NULL.
 *   - Argument errors return synchronously and launch nothing.  A failed
 *     launch returns MMF_ERR_CUDA.  A device-side wait that timed out (every
 *     wait inside the kernels is bounded, about one second) is recorded in a
 *     device error word, and the kernel that gave up returns without writing
 *     its outputs; mmf_check_async reports (MMF_ERR_TIMEOUT) and clears it.
 *   - The first call on a device does a one-time set-up (device properties,
 *     kernel attributes, the driver's tensor-map entry point); make that
 *     first call outside any CUDA graph capture.
 *   - Entry points are thread-safe; calls that overlap on the GPU must not
 *     write the same output or workspace buffer.
 */
#ifndef MMF_H
#define MMF_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mmf_status {
    MMF_OK = 0,
    MMF_ERR_INVALID_ARG = 1,       /* null pointer, negative size, bad eps */
    MMF_ERR_UNSUPPORTED_SHAPE = 2, /* K not a multiple of 128 in [128, 65536], or too large */
    MMF_ERR_MISALIGNED = 3,        /* a pointer is not 16-byte aligned */
    MMF_ERR_WORKSPACE = 4,         /* workspace missing or smaller than mmf_workspace_bytes */
    MMF_ERR_CUDA = 5,              /* a CUDA runtime call or launch failed */
    MMF_ERR_TIMEOUT = 6,           /* a bounded device-side wait ran out */
    MMF_ERR_NO_DEVICE = 7          /* no sm_100 device is current */
} mmf_status;

/* Human-readable name of a status code; never NULL. */
const char* mmf_status_string(int status);

/* Library version string, e.g. "mmf 0.1.0 sm_100a". */
const char* mmf_version(void);

/* Number of kernel launches one mmf_bitlinear_fwd_group call with `count`
 * non-empty projections of N rows in total issues for this (M, K): 1 on the
 * fused decode path (1 .. 3 tokens), 2 (quantiser + contraction) for
 * 4 .. 32 tokens, 1 + count on the large-M path; 0 for an invalid or empty
 * shape.  A single mmf_bitlinear_fwd is count = 1. */
int mmf_fwd_launches(int64_t M, int64_t K, int64_t N, int count);

/* Bytes of the packed ternary matrix for an N x K weight: N * K / 4. */
size_t mmf_packed_bytes(int64_t N, int64_t K);

/* Bytes of device workspace mmf_bitlinear_fwd and mmf_ternary_acc need for
 * this shape; 0 when the shape takes the fused decode path (1 .. 3 tokens),
 * which needs none.  For 4 .. 32 tokens it holds the codes in the decode
 * tensor-core kernel's operand layout (16 or 32 token rows per 128-wide K
 * chunk) and the per-token absmax and code sums; for more tokens the codes in
 * row-major order and the same sums.  Depends only on (M, K, N). */
size_t mmf_workspace_bytes(int64_t M, int64_t K, int64_t N);

/*
 * mmf_pack_ternary -- absmean ternarisation and 2-bit packing of a latent
 * weight matrix (datacamp.com, "Thay MatMul bằng các phép toán tam phân": the
 * full-precision weights are scaled by their mean absolute value and rounded
 * to the nearest of -1, 0, +1; read as a division, since a product would round
 * every weight of a N(0, 0.02) matrix to 0).
 *
 *   beta   = mean over all N*K of |W|, summed in fp64 in a fixed order and
 *            rounded once to fp32; written to scale[0].
 *   w~     = clamp(rint(W / (beta + eps_w)), -1, 1), the division in fp32
 *            (IEEE, round to nearest even), rint ties to even.
 *   packed = uint32 [N][K/16], row-major, row pitch K/4 bytes.  Word j of row n
 *            holds weights k = 16j + i, i = 0..15; weight i occupies bits
 *            [8*(i%4) + 2*(i/4), +2) and stores the code w~ + 1
 *            (0 = -1, 1 = 0, 2 = +1; 3 is never written).
 *
 * W: fp32 [N][K] row-major (nn.Linear layout, y = x W~^T).  eps_w >= 0.
 * `packed` is also used as scratch before it receives the codes, so it must
 * not alias W.  Deterministic: the same W gives the same bits on every run.
 */
int mmf_pack_ternary(const float* W, int64_t N, int64_t K, float eps_w,
                     uint32_t* packed, float* scale, void* stream);

/*
 * mmf_quantize_act -- RMSNorm followed by per-token absmax int8 quantisation,
 * one fused pass over x (the same arithmetic as inside mmf_bitlinear_fwd):
 *   ms     = (float)(sum_k x_k^2 / K)      sum and quotient in fp64
 *   inv    = 1 / sqrt(ms + eps)            fp32, correctly rounded
 *   r_k    = (x_k * inv) * gamma_k         fp32, two roundings in this order
 *   absmax = max(max_k |r_k|, 1e-5)        written to absmax[m]
 *   q_k    = clamp(rint(r_k * (127/absmax)), -127, 127)
 * x: bf16 [M][K]; gamma: fp32 [K]; q: int8 [M][K]; absmax: fp32 [M].
 * eps >= 0.  x and q must not alias.
 */
int mmf_quantize_act(const uint16_t* x, const float* gamma, float eps,
                     int64_t M, int64_t K, int8_t* q, float* absmax, void* stream);

/*
 * mmf_ternary_acc -- the ternary contraction alone, for parity checks:
 *   acc[m][n] = sum over k with w~[n][k] = +1 of q[m][k]
 *             - sum over k with w~[n][k] = -1 of q[m][k]      (int32, exact)
 * q: int8 [M][K] (values in [-127, 127]); packed as from mmf_pack_ternary;
 * acc: int32 [M][N].  Takes the same kernel path mmf_bitlinear_fwd takes for
 * this (M, K, N), so it needs the same workspace.
 */
int mmf_ternary_acc(const int8_t* q, const uint32_t* packed, int64_t M,
                    int64_t K, int64_t N, int32_t* acc, void* workspace,
                    size_t workspace_bytes, void* stream);

/*
 * mmf_bitlinear_fwd -- the fused BitLinear forward:
 *   (q, absmax) = RMSNorm + quantisation of x, as in mmf_quantize_act
 *   acc         = ternary contraction of q with the packed weights
 *   y[m][n]     = bf16_rn((float)acc[m][n] * ((absmax[m] / 127) * scale[0]))
 * x: bf16 [M][K]; gamma: fp32 [K]; packed/scale as from mmf_pack_ternary;
 * y: bf16 [M][N].  workspace: device buffer of at least
 * mmf_workspace_bytes(M, K, N) bytes (may be NULL when that is 0); it holds
 * the int8 codes between the two kernels of the large-M path.  x, y and the
 * workspace must not overlap.
 */
int mmf_bitlinear_fwd(const uint16_t* x, const float* gamma, float eps,
                      const uint32_t* packed, const float* scale, int64_t M,
                      int64_t K, int64_t N, uint16_t* y, void* workspace,
                      size_t workspace_bytes, void* stream);

/*
 * mmf_bitlinear_fwd_glu -- the down projection of the GLU channel mixer with
 * its gating fused in (datacamp.com, section "Các thành phần lõi: MLGRU và
 * GLU": the input goes through two BitLinear layers, one output through
 * SiLU, multiplied element-wise by the other, and the product through a
 * third BitLinear layer).  The input of the fused forward is
 *   p[m][k] = bf16_rn(SiLU(g[m][k]) * u[m][k]),  SiLU(v) = v * (1 / (1 + e^-v)),
 * each step rounded to fp32; then as mmf_bitlinear_fwd with x = p.  p never
 * goes to memory: the kernels form it while normalising.
 * g, u: bf16 [M][K] (the gate and up projections' outputs); other arguments,
 * workspace (mmf_workspace_bytes(M, K, N)) and errors as mmf_bitlinear_fwd;
 * flags: 0 or MMF_FWD_PDL (g and u are then read only after the kernel before
 * has finished, like x).  g, u, y and the workspace must not overlap.
 */
int mmf_bitlinear_fwd_glu(const uint16_t* g, const uint16_t* u,
                          const float* gamma, float eps, const uint32_t* packed,
                          const float* scale, int64_t M, int64_t K, int64_t N,
                          uint16_t* y, void* workspace, size_t workspace_bytes,
                          unsigned flags, void* stream);

/*
 * mmf_mlgru_scan -- the MLGRU token mixer's element-wise recurrence between
 * its f/c/g projections and its o projection (datacamp.com, section "Các
 * thành phần lõi: MLGRU và GLU": tokens taken one at a time, gates in (0, 1)
 * deciding how much of the previous hidden state and of the current token is
 * kept).  For every sequence b and channel k, from h = h0[b][k] (0 when h0 is
 * NULL), token by token:
 *   f = sigma(f_pre), c = SiLU(c_pre), g = sigma(g_pre),  sigma(v) = 1/(1 + e^-v)
 *   h = f * h + (1 - f) * c          (fp32)
 *   o[b][t][k] = bf16_rn(g * h)      (the o projection's input)
 * and h_last[b][k] = h after the last token (may be NULL).  Tokens are split
 * into chunks combined through their linear maps h -> A h + B, and sigma uses
 * the hardware exponential and reciprocal (a few ulp), so the result matches
 * the token-by-token recurrence to a few fp32 ulps per token, not bit for bit.
 * f_pre, c_pre, g_pre, o: bf16 [B][T][D] (the projections' y layout with
 * M = B * T); h0, h_last: fp32 [B][D].  D must be even, B <= 65535; pointers
 * 16-byte aligned; o must not overlap the inputs.  T = 0 copies h0 (or zeros)
 * to h_last.
 */
int mmf_mlgru_scan(const uint16_t* f_pre, const uint16_t* c_pre,
                   const uint16_t* g_pre, const float* h0, int64_t B, int64_t T,
                   int64_t D, uint16_t* o, float* h_last, void* stream);

/*
 * mmf_bitlinear_bwd -- backward of mmf_bitlinear_fwd with the straight-through
 * estimator (ld246.com, section "训练与优化：新的策略": the non-differentiable
 * ternary weights and quantisation are back-propagated with a surrogate
 * gradient, read as passing gradients through both quantisers unchanged).
 * With x_q = q * (absmax / 127) (the forward's codes) and W_q = w~ * beta:
 *   dr = dy . W_q,  dW = dy^T . x_q,
 *   dx = inv * gamma * dr - x * inv^3 * (sum_k gamma_k dr_k x_k) / K,
 *   dgamma = sum over tokens of dr * x * inv,  inv = 1 / sqrt(sum x^2 / K + eps).
 * dy: bf16 [M][N]; x, gamma, eps, packed, scale as for the forward;
 * dx: bf16 [M][K]; dgamma: fp32 [K]; dW: fp32 [N][K] (the latent weights'
 * gradient); all overwritten.  The two products run on the tensor cores in
 * this library's own kernel (bf16 operands, fp32 accumulation): for dr the
 * ternary weights are unpacked from the 2-bit codes (exact), for dW each
 * token's codes are scaled by absmax / 127 and rounded to bf16 as they are
 * loaded.  An empty contraction gives zeros (M == 0: dW = 0, dgamma = 0;
 * N == 0: dx = 0).  workspace: at least mmf_bwd_workspace_bytes(M, K, N)
 * bytes, no initialisation needed.  Sizes as the forward, with N a multiple
 * of 8 (dy rows are read by TMA), and M <= 4194240 when K > 8192; buffers of an empty extent
 * (x, dx and workspace when M == 0; dW when N == 0; dy and packed when either
 * is 0) may be NULL.
 */
size_t mmf_bwd_workspace_bytes(int64_t M, int64_t K, int64_t N);
int mmf_bitlinear_bwd(const uint16_t* dy, const uint16_t* x, const float* gamma,
                      float eps, const uint32_t* packed, const float* scale,
                      int64_t M, int64_t K, int64_t N, uint16_t* dx,
                      float* dgamma, float* dW, void* workspace,
                      size_t workspace_bytes, void* stream);

/*
 * mmf_embed_fwd -- the model's embedding: lookup with scaling, the x of its
 * first layer (nothing on the pages fixes it; the plain definition):
 *   x[m][k] = bf16_rn(scale * table[ids[m]][k])          (the product in fp32)
 * ids: int32 [M], or int64 [M] with MMF_EMBED_IDS64; table: fp32 [V][K], or
 * bf16 [V][K] with MMF_EMBED_TABLE_BF16; x: bf16 [M][K].  An id outside
 * [0, V) (the usual -1 of a padded place) gives a row of zeros.  K % 8 == 0,
 * 8 <= K <= 65536, V < 2^31 - 1, M as above; scale finite.  x must not overlap
 * the inputs (refused, as for the gradients below).
 */
#define MMF_EMBED_IDS64 1u       /* ids are int64 (else int32) */
#define MMF_EMBED_TABLE_BF16 2u  /* mmf_embed_fwd: the table is bf16 (else fp32) */
#define MMF_EMBED_ACCUMULATE 4u  /* mmf_embed_bwd: add to dtable (else overwrite it) */
int mmf_embed_fwd(const void* ids, const void* table, float scale, int64_t V,
                  int64_t M, int64_t K, uint16_t* x, unsigned flags, void* stream);

/*
 * mmf_embed_bwd -- gradient of mmf_embed_fwd for the table:
 *   dtable[v][k] = scale * sum over the tokens m with ids[m] = v of dx[m][k]
 * in fp32; with MMF_EMBED_ACCUMULATE the sum is added to dtable[v][k], and rows
 * no token names are not touched (without the flag they become zeros).  The
 * tokens are sorted by id and each row's are added in their order in a fixed
 * grouping: the same ids and dx give the same bits on every run.  A place whose
 * id is outside [0, V) takes no part.
 * ids as above; dx: bf16 [M][K] (as from mmf_bitlinear_bwd); dtable: fp32
 * [V][K].  workspace: at least mmf_embed_bwd_workspace_bytes(V, M, K) bytes, no
 * initialisation needed; fewer tokens never need more.  dtable and the workspace
 * must not overlap the inputs or one another.  M == 0 without the flag writes
 * zeros.
 */
size_t mmf_embed_bwd_workspace_bytes(int64_t V, int64_t M, int64_t K);
int mmf_embed_bwd(const void* ids, const uint16_t* dx, float scale, int64_t V,
                  int64_t M, int64_t K, float* dtable, void* workspace,
                  size_t workspace_bytes, unsigned flags, void* stream);

/*
 * mmf_mlgru_scan_bwd -- gradient of mmf_mlgru_scan.  The states are recomputed
 * from the pre-activations; nothing of the forward has to be kept but its
 * inputs.  With f, c, g, h as there and s = sigma(c_pre), from dh_T = dh_last
 * (0 when NULL) + do_T g_T, the tokens taken backwards:
 *   dh_t   = do_t g_t + f_{t+1} dh_{t+1},          dh0 = f_1 dh_1
 *   df_pre = bf16_rn(dh_t (h_{t-1} - c_t) f (1 - f))
 *   dc_pre = bf16_rn(dh_t (1 - f) s (1 + c_pre (1 - s)))
 *   dg_pre = bf16_rn(do h_t g (1 - g))
 * in fp32, sigma by the hardware exponential and reciprocal as there.
 * Pre-activations below -28 (-infinity too) count as -28, as there: gates of
 * less than 7e-13 are off by up to that much, and the outputs they scale by up
 * to 2e-11 of the state's and the gradient's size, relative to themselves without
 * bound.  A NaN reaches the outputs that these formulas make NaN and no others;
 * an infinite input's outputs may be NaN where the formulas make them infinite.
 * f_pre, c_pre, g_pre, d_o (the gradient of o) and the outputs
 * df_pre, dc_pre, dg_pre: bf16 [B][T][D]; h0, dh_last (may be NULL) and dh0
 * (may be NULL: not wanted): fp32 [B][D].  Sizes as mmf_mlgru_scan.  The
 * outputs and the workspace must not overlap the inputs or one another.  T = 0 copies dh_last
 * (or zeros) to dh0.  workspace: at least
 * mmf_mlgru_scan_bwd_workspace_bytes(B, T, D) bytes, no initialisation needed;
 * fewer or shorter sequences never need more.
 */
size_t mmf_mlgru_scan_bwd_workspace_bytes(int64_t B, int64_t T, int64_t D);
int mmf_mlgru_scan_bwd(const uint16_t* f_pre, const uint16_t* c_pre,
                       const uint16_t* g_pre, const uint16_t* d_o,
                       const float* h0, const float* dh_last, int64_t B,
                       int64_t T, int64_t D, uint16_t* df_pre, uint16_t* dc_pre,
                       uint16_t* dg_pre, float* dh0, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * mmf_adamw_step -- one AdamW step over `count` tensors at once (the pages name
 * no optimiser; the plain definition, decoupled weight decay).  Per element:
 *   g' = g * grad_scale
 *   m  = beta1 * m + (1 - beta1) * g'
 *   v  = beta2 * v + (1 - beta2) * g'^2
 *   p  = p * (1 - lr * weight_decay)
 *        - lr / (1 - beta1^step) * m / (sqrt(v / (1 - beta2^step)) + eps)
 * in fp32 (m and v as separately rounded products and sums, so their bits are
 * those of the elementwise fp32 operations).  p: fp32 [n], updated in place;
 * p_bf16: bf16 [n] copy of the new p, or NULL; g: fp32 [n], or bf16 [n] with
 * MMF_ADAMW_GRAD_BF16.
 * m, v: fp32 [n], or with MMF_ADAMW_STATE8 8-bit floats [n] in blocks of
 * MMF_ADAMW_BLOCK consecutive elements (the last block may be short), m as
 * e4m3 codes and v as e5m2 codes, the values code * m_scale[block] and
 * code * v_scale[block] (fp32 [ceil(n / 256)], powers of two).  With 2^e <=
 * the block's largest |m| < 2^(e+1), e taken as at least -90, m_scale =
 * 2^(e-7), and v_scale = 2^(e-14) likewise.  The codes are rounded up or down
 * at random, with the right mean: 16 bits per moment from draw floor(i / 2) of
 * the SplitMix64 stream (seed, index of the tensor in the call) for element i,
 * all 64 bits of the seed taken;
 * p is updated with the moments before they are rounded.  |m| below the
 * smallest normal code becomes 0; a positive v is kept at least at the
 * smallest normal code.  A block in which a moment is 2^127 or more, infinite
 * or NaN reads as NaN from then on.  All zeros are the fresh states of either
 * kind.
 * With MMF_ADAMW_STATE8 the seed must be another at every step of a run (the
 * step's number will do): with one that stays, an element draws the same bits
 * each time, which is a fixed threshold to round at, and its moments are biased
 * for good (after some hundred steps v is 3 times too large in the median, 10
 * times once the gradients have halved).  A graph that is captured without
 * `scalars` repeats its step's seed, and its bias corrections, on every replay.
 *
 * tensors: HOST array, read during the call only; n == 0 is skipped (its
 * pointers may be NULL).  p, p_bf16, m, v, m_scale and v_scale of one call must
 * not overlap one another (checked, MMF_ERR_INVALID_ARG) nor any g.  Launches
 * one kernel per 256 tensors.
 *
 * hyper: HOST struct, read during the call only.  0 <= beta < 1, eps >= 2^-126,
 * lr >= 0, step >= 1 (the count that includes this step), everything finite.
 * scalars: NULL, or a DEVICE copy (16-byte aligned) of what
 * mmf_adamw_scalars_at fills: the kernel then takes lr, the bias corrections,
 * grad_scale and the seed from there and not from hyper, so a captured graph
 * takes each replay's values from memory (a gradient-clipping factor computed
 * on the device may be written there too).
 */
#define MMF_ADAMW_STATE8 1u     /* m, v in 8 bits */
#define MMF_ADAMW_GRAD_BF16 2u  /* g is bf16 (else fp32) */
#define MMF_ADAMW_BLOCK 256     /* elements that share m_scale and v_scale */

typedef struct mmf_adamw_tensor {
    float* p;
    const void* g;
    void* m;
    void* v;
    float* m_scale;     /* NULL without MMF_ADAMW_STATE8 */
    float* v_scale;
    uint16_t* p_bf16;   /* may be NULL */
    int64_t n;
    float weight_decay; /* >= 0 */
    unsigned flags;
} mmf_adamw_tensor;

typedef struct mmf_adamw_hyper {
    double lr, beta1, beta2, eps, grad_scale;
    int64_t step;
    uint64_t seed;       /* MMF_ADAMW_STATE8: another at every step, as of `step` */
} mmf_adamw_hyper;

typedef struct mmf_adamw_scalars {
    float lr;
    float alpha;         /* lr / (1 - beta1^step) */
    float inv_sqrt_bc2;  /* 1 / sqrt(1 - beta2^step) */
    float grad_scale;
    uint64_t seed;
    uint64_t reserved;
} mmf_adamw_scalars;

int mmf_adamw_step(const mmf_adamw_tensor* tensors, int count,
                   const mmf_adamw_hyper* hyper,
                   const mmf_adamw_scalars* scalars, void* stream);

/* Fills *out (HOST) with the scalars of a step; launches nothing. */
int mmf_adamw_scalars_at(const mmf_adamw_hyper* hyper, mmf_adamw_scalars* out);

/* Flags of mmf_bitlinear_fwd_group. */
#define MMF_FWD_PDL 1u   /* launch as a programmatic dependent of the kernel before it on the stream (see below) */
#define MMF_MAX_GROUP 8  /* projections per mmf_bitlinear_fwd_group call */

/* One projection of a group: its packed weights and scale (as from
 * mmf_pack_ternary for an N x K matrix) and its output y, bf16 [M][N]. */
typedef struct mmf_projection {
    const uint32_t* packed;
    const float* scale;
    uint16_t* y;
    int64_t N;
} mmf_projection;

/*
 * mmf_bitlinear_fwd_group -- the fused forward of `count` (1..MMF_MAX_GROUP)
 * projections that read the same x: the token mixer's gate projections and
 * the channel mixer's gate/up pair each share one normalised, quantised input
 * (jiqizhixin.com, section "MatMul-free 语言模型架构"; datacamp.com, section
 * "Các thành phần lõi: MLGRU và GLU").  x is normalised and quantised once;
 * each projection i then gets y_i exactly as mmf_bitlinear_fwd would compute
 * it (same bits).  On the small-M path all projections run in one launch.
 *
 * proj: HOST array of `count` descriptors (read during the call only); an
 * entry with N == 0 is skipped.  workspace: at least
 * mmf_workspace_bytes(M, K, sum of N) bytes.
 *
 * flags: 0 or MMF_FWD_PDL.  With MMF_FWD_PDL the kernels are launched as
 * programmatic dependents of the kernel before them on the stream: packed
 * weights, scales and gamma are fetched BEFORE that kernel has finished (x is
 * read, and y written, only after it), so the caller guarantees that the
 * immediately preceding kernel on the stream does not write packed, scale or
 * gamma.  Without the flag the launches are ordinary stream-ordered launches.
 */
int mmf_bitlinear_fwd_group(const uint16_t* x, const float* gamma, float eps,
                            int64_t M, int64_t K, const mmf_projection* proj,
                            int count, void* workspace, size_t workspace_bytes,
                            unsigned flags, void* stream);

/*
 * mmf_bitlinear_fwd_noalloc -- mmf_bitlinear_fwd without a caller-supplied
 * workspace; nothing on the pages corresponds to it (it is an interface
 * convenience, not part of the method).
 *
 * Some callers cannot allocate device memory: a plug-in hosted by another
 * runtime that owns all device memory through its own pool (a raw cudaMalloc
 * would bypass that pool's accounting and may fail or fragment it), or a
 * latency-critical caller that must not block in cudaMalloc / cudaFree, which
 * can synchronise the device.  This entry point serves them: the caller passes
 * only inputs and outputs, exactly as for mmf_bitlinear_fwd (same arguments
 * minus the workspace, same results bit for bit), and the large-M workspace
 * comes from a static device array inside the library instead.
 *
 * Limits and behaviour:
 *   - The static scratch holds MMF_NOALLOC_SCRATCH_BYTES bytes (64 MiB);
 *     shapes with mmf_workspace_bytes(M, K, N) above that return
 *     MMF_ERR_WORKSPACE and launch nothing.  Every GPU that loads the library
 *     holds the 64 MiB until the process exits.
 *   - No call allocates or frees device memory.
 *   - The first call on a device (with a workspace-needing shape) looks up
 *     the scratch's device address for that device; make that first call
 *     before any stream capture on the device.
 *   - All calls on a device share the one scratch array.  Calls whose kernels
 *     overlap on the GPU (different streams, or threads with their own
 *     streams) race on it and give wrong results; order them, e.g. on one
 *     stream.  Nothing in the scratch needs clearing between calls: each call
 *     rewrites every byte it reads.
 */
#define MMF_NOALLOC_SCRATCH_BYTES (64u << 20)
int mmf_bitlinear_fwd_noalloc(const uint16_t* x, const float* gamma, float eps,
                              const uint32_t* packed, const float* scale,
                              int64_t M, int64_t K, int64_t N, uint16_t* y,
                              void* stream);

/*
 * mmf_hbm_copy -- streaming device-to-device copy of `bytes` bytes (a multiple
 * of 16) with 128-bit loads and stores.  Measurement kernel: it gives the HBM
 * bandwidth the roofline fractions are stated against.  src and dst must not
 * overlap.
 */
int mmf_hbm_copy(const void* src, void* dst, size_t bytes, void* stream);

/*
 * mmf_selftest_timeout -- failure-detection self-test (no counterpart on the
 * pages).  Launches one thread that waits on a shared-memory barrier nothing
 * arrives at, with the same bounded wait the kernels use but a limit of
 * limit_ns (0 < limit_ns <= 1e9).  The wait gives up, records a timeout in the
 * device error word (so the next mmf_check_async returns MMF_ERR_TIMEOUT),
 * writes 1 to *waited_out if waited_out is not NULL (device pointer, 4-byte
 * aligned), and the kernel returns.  Nothing hangs or faults.
 */
int mmf_selftest_timeout(uint64_t limit_ns, int32_t* waited_out, void* stream);

/*
 * mmf_check_async -- synchronises `stream`, then reads and clears the device
 * error word of the current device.  Returns MMF_ERR_TIMEOUT if a bounded
 * wait in any earlier kernel ran out, MMF_ERR_CUDA if the stream reports an
 * error, else MMF_OK.
 */
int mmf_check_async(void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MMF_H */
