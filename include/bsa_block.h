/*
 * bsa_block.h -- C ABI of the operators around the attention of a diffusion transformer's
 * block (libbsa.so; the attention itself is in bsa.h).
 *
 *   bsa_rotary      -- Q, K, V from the projection's layout to the attention's: per-head RMS
 *                      norm of Q and K, rotary positions with several axes (time, height,
 *                      width), and the change of layout, in one pass
 *   bsa_gated_norm  -- the step between two sub-blocks: norm of the branch, gate, residual add,
 *                      norm of the sum, scale and shift, in one pass
 * and the backward pass of each.
 *
 * The conventions of bsa.h hold: the caller owns every buffer; no call allocates, frees or
 * synchronises; work is enqueued on `stream` of the current device, where every buffer lives;
 * argument checks run on the host before any launch, and a failed check enqueues nothing;
 * workspaces are 256-byte aligned. Differences: these calls raise no error on the device, and
 * their workspaces need no zero fill (each call writes what it reads).
 *
 * Tensors are given by a pointer and element strides; channels are contiguous. Pointers are
 * 16-byte aligned and strides non-negative multiples of 16 bytes (the stride of a dimension of
 * length one is not looked at). An input may have a stride of zero (a broadcast input). An
 * output (gradients and the workspace count) must not overlap itself, another output or an
 * input that the call reads (weights, modulations and positions count), except that an output may
 * be the input that its own comment names (the same pointer, strides and dtype). Views of the
 * same strides that interleave in one buffer (Q, K and V of a fused projection, a slice of the
 * channels or tokens) are told apart; otherwise the address ranges must be disjoint.
 */
#ifndef BSA_BLOCK_H_
#define BSA_BLOCK_H_

#include "bsa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ rotary positions */

#define BSA_ROTARY_MAX_AXES 4

typedef enum {
    BSA_ROTARY_INTERLEAVED = 0, /* pair p is channels (2p, 2p + 1) */
    BSA_ROTARY_HALVES = 1       /* pair p is channels (p, p + rot / 2) */
} bsa_rotary_pairing;

/* Which channels turn with which axis, and how fast. The axes take axis_dim[a] channels each,
 * one after another: rot = their sum, rot <= d. Axis a owns axis_dim[a] / 2 consecutive pairs;
 * its pair j turns by scale[a] * theta[a]^(-2 j / axis_dim[a]) radians per position, or by
 * inv_freq[p] (p: the pair's index over all axes) when inv_freq is given. Channels from rot
 * on do not turn. */
typedef struct {
    int n_axes;                           /* 1 .. BSA_ROTARY_MAX_AXES */
    int axis_dim[BSA_ROTARY_MAX_AXES];    /* even, >= 2; HALVES: the sum a multiple of 16 */
    double theta[BSA_ROTARY_MAX_AXES];    /* finite, > 0; not read with inv_freq */
    double scale[BSA_ROTARY_MAX_AXES];    /* finite; not read with inv_freq */
    int pairing;                          /* bsa_rotary_pairing */
    const double *inv_freq;               /* host, rot / 2 finite values, or NULL */
} bsa_rotary_spec;

/* The frequencies of a spec, made once on the host (bsa_rotary_plan_init) and passed to every
 * call by value: nothing of it lives on the device. Frequencies are kept in 2^-64 turns per
 * position, so that position * frequency modulo one turn is one wrapping 64-bit product, exact
 * for every int32 position; the frequency itself is within 2^-51 of its value plus 2^-65 turns. */
typedef struct {
    uint32_t magic;
    int32_t d, rot, n_axes, pairing;
    uint64_t turns[64];  /* pair p */
    uint8_t axis[64];    /* pair p */
} bsa_rotary_plan;

/* Host-only. d in {64, 128} (BSA_ERR_SHAPE). BSA_ERR_INVALID_ARG: null pointers, axes or
 * pairing out of range, a theta, scale or frequency that is not finite (theta > 0). */
bsa_status bsa_rotary_plan_init(const bsa_rotary_spec *spec, int d, bsa_rotary_plan *plan);

/* One of Q, K, V: `heads` heads of d channels per token, from src to dst. Strides in elements.
 * dst may be src. */
typedef struct {
    const void *src;
    int64_t src_batch, src_token, src_head;
    void *dst;
    int64_t dst_batch, dst_token, dst_head;
    const float *weight; /* device fp32 [d], the RMS norm's weight, or NULL (all ones) */
    int heads;
} bsa_heads;

/*
 * bsa_rotary -- per token n, head and pair (a, b) of axis s, for Q and K:
 *   u = norm ? x * rsqrt(mean_c x_c^2 + eps) * weight : x          (over the head's d channels)
 *   t = positions[n][s] * frequency
 *   y_a = u_a cos t - u_b sin t,   y_b = u_b cos t + u_a sin t;   channels from rot on: y = u
 * and V is copied. fp32 throughout, one rounding to dt. With dst strides of [B][H][N][d] the
 * results are bsa_forward's Q, K, V.
 *   plan        host (bsa_rotary_plan_init)
 *   q, k, v     host descriptors; any may be NULL, not all three. heads may differ (shared
 *               keys and values); weight is not read for v, nor when norm == 0
 *   dt          BSA_BF16 or BSA_FP32, of every src and dst
 *   positions   device int32 [B or 1][N][n_axes], n_axes contiguous per token; pos_batch is
 *               the batch stride in elements (0: one set for all). Any value, negative too.
 *               Not read (may be NULL) when only v is given
 *   norm, eps   norm != 0 selects the RMS norm; eps >= 0, finite
 * One launch. Errors: BSA_ERR_SHAPE (B, N, heads < 1, B * N > INT32_MAX, heads > 65535),
 * BSA_ERR_DTYPE, BSA_ERR_INVALID_ARG (null or misaligned pointers, strides, overlaps, eps, a
 * plan that bsa_rotary_plan_init did not make), BSA_ERR_CUDA.
 */
bsa_status bsa_rotary(const bsa_rotary_plan *plan, const bsa_heads *q, const bsa_heads *k, const bsa_heads *v,
                      int dt, int B, int N, const int32_t *positions, int64_t pos_batch, int norm, float eps,
                      void *stream);

/* The gradient of one of Q, K, V. dx may be x. */
typedef struct {
    const void *dy;  /* arriving at bsa_rotary's dst */
    int64_t dy_batch, dy_token, dy_head;
    const void *x;   /* bsa_rotary's src; read (and its strides looked at) only for q, k with norm */
    int64_t x_batch, x_token, x_head;
    void *dx;        /* written */
    int64_t dx_batch, dx_token, dx_head;
    const float *weight;
    float *dweight;  /* device fp32 [d] (written), or NULL; q, k with norm only */
    int heads;
} bsa_heads_grad;

/*
 * bsa_rotary_backward -- the gradients of bsa_rotary, with g the arriving gradient turned back
 * by -t and r = rsqrt(mean x^2 + eps):
 *   norm == 0: dx = g.   norm != 0: v = g * weight, dx = r (v - x r^2 mean(v x)),
 *   dweight = sum over batch, tokens and heads of g x r
 * V's gradient is copied. Sums run in fp32 in an order fixed by the shape: the same call gives
 * the same bits.
 *   workspace   device, >= bsa_rotary_workspace_size bytes; needed when a dweight is asked for
 * One launch, two with a dweight. Errors: as bsa_rotary; BSA_ERR_WORKSPACE.
 */
bsa_status bsa_rotary_backward(const bsa_rotary_plan *plan, const bsa_heads_grad *q, const bsa_heads_grad *k,
                               const bsa_heads_grad *v, int dt, int B, int N, const int32_t *positions,
                               int64_t pos_batch, int norm, float eps, void *workspace, size_t workspace_bytes,
                               void *stream);

/* Host-only: workspace bytes of bsa_rotary_backward. Errors: BSA_ERR_SHAPE, BSA_ERR_INVALID_ARG. */
bsa_status bsa_rotary_workspace_size(int B, int N, int d, size_t *bytes);

/* ------------------------------------------------------------------ gated norm */

typedef enum {
    BSA_NORM_NONE = 0,
    BSA_NORM_RMS = 1,  /* n = t * rsqrt(mean t^2 + eps) */
    BSA_NORM_LAYER = 2 /* n = (t - mean t) * rsqrt(mean (t - mean t)^2 + eps) */
} bsa_norm_kind;

/* norm(t) = n * weight + bias over the C channels of a row; NULL weight: ones, NULL bias: zeros */
typedef struct {
    int kind;  /* bsa_norm_kind */
    float eps; /* >= 0, finite */
    const float *weight, *bias; /* device fp32 [C], 16-byte aligned */
} bsa_norm;

/* [B][N][C] tensor: element strides of batch and token; ptr NULL where a call allows none */
typedef struct {
    void *ptr;
    int64_t batch, token;
} bsa_rows;

/* A modulation [B][F][C] of dtype mod_dt: tokens [f * N / F, (f + 1) * N / F) of a batch share
 * row f (F = 1: one row per batch; F = frames of a video; F = N: one per token). NULL: none. */
typedef struct {
    const void *ptr;
    int64_t batch, frame;
} bsa_modulation;

typedef struct {
    int B, N, C, F;     /* C a multiple of 8, 8 .. 8192; F divides N */
    int stream_dt;      /* dtype of x, h (and dh, dx): the residual stream */
    int branch_dt;      /* dtype of y, z (and dz, dy); BSA_FP32 only with an fp32 stream */
    int mod_dt;         /* dtype of gate, scale, shift and their gradients */
    float alpha;        /* finite */
    bsa_norm post, pre; /* norm of the branch, norm of the sum */
    bsa_modulation gate, scale, shift;
} bsa_gated_norm_desc;

/*
 * bsa_gated_norm -- per token:
 *   u = post(y)                    (kind NONE: u = y)
 *   h = x + alpha * gate * u       (gate NULL: ones)
 *   z = pre(h) * (1 + scale) + shift
 * fp32 throughout; z comes from h before h is rounded. Each output is rounded once.
 *   x           read
 *   y           NULL ptr: no branch, h = x (h->ptr is then NULL, post NONE, gate NULL)
 *   h           written; may be x
 *   z           written when pre.kind is not NONE, else its ptr is NULL; may be y
 * y, h, z may be null pointers in place of a NULL ptr. scale and shift need a pre norm, and
 * gate and post a y. One launch. Errors: BSA_ERR_SHAPE (B, N < 1, B * N > INT32_MAX, C, F),
 * BSA_ERR_DTYPE, BSA_ERR_INVALID_ARG (null or misaligned pointers, strides, overlaps, alpha,
 * eps, kind, outputs and inputs that do not go together, neither a branch nor a pre norm),
 * BSA_ERR_CUDA.
 */
bsa_status bsa_gated_norm(const bsa_gated_norm_desc *desc, const bsa_rows *x, const bsa_rows *y,
                          const bsa_rows *h, const bsa_rows *z, void *stream);

/* Inputs and outputs of bsa_gated_norm_backward */
typedef struct {
    bsa_rows dh; /* arriving at h from where h goes on; NULL ptr: zero */
    bsa_rows dz; /* arriving at z; needed with a pre norm, NULL ptr without */
    bsa_rows h;  /* bsa_gated_norm's h (its x without a branch); needed with a pre norm */
    bsa_rows y;  /* bsa_gated_norm's y; needed when dy, or the gradient of gate or post, is asked for */
    bsa_rows dx; /* written (the gradient of x is that of h); may be dh or h; NULL ptr: not wanted */
    bsa_rows dy; /* written; may be y or dz; NULL ptr: not wanted */
    void *dgate, *dscale, *dshift;                          /* mod_dt [B][F][C], contiguous, or NULL */
    float *dpost_weight, *dpost_bias, *dpre_weight, *dpre_bias; /* fp32 [C], or NULL */
} bsa_gated_norm_grads;

/*
 * bsa_gated_norm_backward -- the gradients of bsa_gated_norm at (h, y):
 *   n, r: pre's normalised row and 1 / its scale;  a = dz * weight * (1 + scale)
 *   dx = dh + r (a - [mean a] - n mean(a n))                       ([...]: LAYER only)
 *   m, r2: post's;  b = alpha * gate * dx * weight
 *   dy = r2 (b - [mean b] - m mean(b m))                           (post NONE: dy = b)
 *   dshift = sum dz,  dscale = sum dz * (n * weight + bias),  dgate = alpha sum dx * u
 *   dpre_weight = sum dz (1 + scale) n,  dpre_bias = sum dz (1 + scale)
 *   dpost_weight = alpha sum gate dx m,  dpost_bias = alpha sum gate dx
 * (sums over the tokens that share the value). Statistics are computed again from h and y as
 * stored. fp32 throughout; sums run in an order fixed by the shape: the same call gives the
 * same bits. The gradient of a parameter that the forward did not have (NULL ptr in desc) is
 * BSA_ERR_INVALID_ARG for gate, scale and shift; for a weight or bias it is the gradient at
 * one or zero. A modulation whose gradient is asked for is not broadcast (BSA_ERR_INVALID_ARG).
 *   workspace   device, >= bsa_gated_norm_workspace_size bytes; needed when a gradient of a
 *               modulation, weight or bias is asked for
 * One launch, two with those gradients. Errors: as bsa_gated_norm; BSA_ERR_WORKSPACE.
 */
bsa_status bsa_gated_norm_backward(const bsa_gated_norm_desc *desc, const bsa_gated_norm_grads *grads,
                                   void *workspace, size_t workspace_bytes, void *stream);

/* Host-only: workspace bytes of bsa_gated_norm_backward. Errors: BSA_ERR_SHAPE, BSA_ERR_INVALID_ARG. */
bsa_status bsa_gated_norm_workspace_size(int B, int N, int C, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* BSA_BLOCK_H_ */
