/*
 * conv_train.h -- C ABI of the training-side operators that stand next to
 * the convolutions of conv_nhwc.h, for fitting a head on the maps a stack of
 * layers produces: group norm with its activation over NHWC maps (forward
 * and gradients), the softmax cross entropy of a 1x1 head over a large set
 * of classes (forward and gradients) and the orthogonalised update of weight
 * matrices.
 *
 * Conventions as in conv_nhwc.h: device buffers are owned by the caller, an
 * entry point validates on the host, returns a negative conv_status without
 * enqueueing anything when it refuses, and otherwise only enqueues kernels
 * on the given stream (no allocation, no synchronisation, nothing cached
 * between calls, no memset node), so every call can be captured into a HIP
 * graph. A call that needs scratch memory takes it as `ws` (256-byte
 * aligned); the *_ws_bytes function of the operator gives its size, 0 when
 * none is needed (ws may then be NULL), or a negative conv_status for a
 * description the operator refuses. ws holds nothing between calls; calls
 * that may run at the same time need a ws each. Too small a ws is
 * CONV_E_SCRATCH. Every result is the same on every run: no atomic adds.
 * An output overlapping an input, another output or ws is CONV_E_ALIAS.
 * Each tensor must be smaller than 2^31 bytes (CONV_E_UNSUPPORTED); ws may
 * be larger.
 */
#ifndef CONV_TRAIN_H
#define CONV_TRAIN_H

#include "conv_nhwc.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations of the norm: those of conv_act, and SiLU(v) = v / (1 + e^-v). */
enum { CONV_ACT_SILU = 4 };

/* Group norm over an NHWC map, then an activation:
 *   mean, var over the h * w * (c / groups) values of (image, group),
 *   xhat = (x - mean) / sqrt(var + eps)        (var the biased variance)
 *   y    = act(gamma[ch] * xhat + beta[ch]). */
typedef struct conv_norm_desc {
  int64_t n, h, w, c;
  int64_t x_pixel_stride; /* elements from one pixel of x to the next, >= c; 0 = c. A
                             channel slice of a wider map is read in place. */
  int32_t groups;         /* divides c */
  int32_t dtype;          /* of x, y, dy, dx: CONV_F32 or CONV_BF16 (one RNE
                             rounding; all arithmetic and sums in fp32) */
  int32_t act;            /* conv_act or CONV_ACT_SILU */
  float eps;              /* >= 0, finite */
} conv_norm_desc;

/* Scratch of conv_group_norm (grad = 0) or conv_group_norm_grad (grad = 1). */
int64_t conv_group_norm_ws_bytes(const conv_norm_desc* d, int32_t grad);

/* Human-readable description of the launch that x, y, dy and dx of the given
 * common byte alignment (1 .. 16) take, as conv_describe writes it for a layer. */
conv_status conv_group_norm_describe(const conv_norm_desc* d, int32_t grad, int32_t align, char* buf, int32_t len);

/*   x           : device [n][h][w] pixels x_pixel_stride elements apart
 *   gamma, beta : device float[c], or NULL for 1 and 0
 *   y           : device [n][h][w][c] of dtype
 *   stats       : device float[n][groups][2], receives (mean, 1/sqrt(var + eps))
 *                 for the gradients, or NULL
 * Pointers aligned to their element (16-byte aligned x and y with c and
 * x_pixel_stride whole 16-byte chunks run fastest), ws to 256 bytes.
 * CONV_E_SHAPE: a size or groups <= 0, c not divisible by groups,
 * x_pixel_stride < c, eps negative or not finite. CONV_E_UNSUPPORTED: dtype,
 * act, n > 65535 or a size limit. */
conv_status conv_group_norm(const conv_norm_desc* d, const void* x, const float* gamma, const float* beta, void* y,
                            float* stats, void* ws, int64_t ws_bytes, void* stream);

/* Gradients of conv_group_norm for the upstream gradient dy, from its x,
 * stats, gamma and beta:
 *   dz = dy * act'(z), z = gamma * xhat + beta,
 *   dbeta[ch] = sum dz, dgamma[ch] = sum dz * xhat  over images and pixels,
 *   dx = rstd * (gamma dz - m1 - xhat m2), m1 and m2 the means of gamma dz and
 *        gamma dz xhat over the (image, group).
 * act' of ReLU is 1 for z > 0, of ReLU6 1 for 0 < z < 6, else 0.
 *   dy, dx        : device [n][h][w][c] of dtype
 *   dgamma, dbeta : device float[c], either may be NULL
 * Errors as conv_group_norm. */
conv_status conv_group_norm_grad(const conv_norm_desc* d, const void* x, const void* dy, const float* stats,
                                 const float* gamma, const float* beta, void* dx, float* dgamma, float* dbeta,
                                 void* ws, int64_t ws_bytes, void* stream);

/* Softmax cross entropy of a 1x1 head: rows are the pixels (n * h * w) of a
 * map of c channels, the head has one weight row per class.
 *   s[r][v] = sum_k x[r][k] w[v][k]
 *   loss[r] = log(sum_v e^s[r][v]) - s[r][labels[r]]
 *   total   = sum_r weight[r] loss[r]
 * A row whose label lies outside 0 .. classes-1 (-100, say) is left out:
 * its loss is 0, its gradient row is 0, and its x is not used (whatever it
 * holds). weights NULL takes the mean: 1 / (rows not left out), and a total
 * of 0 when all are. The logits are never stored: the forward pass keeps one
 * (maximum, sum of exponentials) per row and run of classes; the gradient
 * computes them again, a piece of the classes at a time. */
typedef struct conv_head_desc {
  int64_t rows, c, classes;
  int32_t dtype;       /* of x, w, dx, dw: CONV_BF16 */
  int32_t label_bytes; /* 4 (int32) or 8 (int64) */
} conv_head_desc;

/* Scratch of conv_head_loss (grad = 0) or conv_head_loss_grad (grad = 1). */
int64_t conv_head_loss_ws_bytes(const conv_head_desc* d, int32_t grad);

/* The products' tiles for x and w of the given common alignment, as conv_describe. */
conv_status conv_head_loss_describe(const conv_head_desc* d, int32_t grad, int32_t align, char* buf, int32_t len);

/*   x       : device [rows][c] (an NHWC map)
 *   w       : device [classes][c] (OHWI of a 1x1 layer)
 *   labels  : device int32 or int64 [rows]
 *   weights : device float[rows] or NULL
 *   loss    : device float[rows]
 *   total   : device float[1]
 * Logits, sums and losses in fp32 from the bf16 products. Alignment: x, w to
 * 2 bytes (16 with c % 8 == 0 is read in place, otherwise through a copy in
 * ws), ws to 256. CONV_E_SHAPE: a size <= 0. CONV_E_UNSUPPORTED: dtype,
 * label_bytes, c over 65536, rows or classes over 2^22 - 64, 2^24 tiles of
 * logits or more (128 x 128, or 256 x 256 above 256 channels), or a size limit. */
conv_status conv_head_loss(const conv_head_desc* d, const void* x, const void* w, const void* labels,
                           const float* weights, float* loss, float* total, void* ws, int64_t ws_bytes,
                           void* stream);

/* The same and the gradients of total:
 *   g[r][v] = weight[r] (softmax(s[r])[v] - [v == labels[r]])
 *   dx[r]   = sum_v g[r][v] w[v],   dw[v] = sum_r g[r][v] x[r]
 *   dx : device [rows][c], dw : device [classes][c], bf16
 * g is rounded to bf16 once for the two products (half a bf16 step of each
 * term), but what that leaves out of a row's label entry is kept in fp32 and
 * added back; the sums run in fp32 and are rounded to bf16 once. */
conv_status conv_head_loss_grad(const conv_head_desc* d, const void* x, const void* w, const void* labels,
                                const float* weights, float* loss, float* total, void* dx, void* dw, void* ws,
                                int64_t ws_bytes, void* stream);

/* Orthogonalised update of weight matrices (the update of the Muon
 * optimiser): with X0 = G / (|G|_F + eps), m <= n after transposing a tall G,
 *   X <- a X + (b A + c A A) X,  A = X X^T,  `steps` times,
 * which drives every singular value of X towards 1, one matrix per batch
 * entry. A convolution's OHWI weights are the matrix [c_out][kh kw c_in]. */
typedef struct conv_ortho_desc {
  int64_t batch, rows, cols;
  int32_t dtype; /* of g: CONV_F32 or CONV_BF16; the result is CONV_BF16 */
  int32_t steps; /* 1 .. 100 */
  float a, b, c; /* finite */
  float eps;     /* >= 0, finite */
} conv_ortho_desc;

int64_t conv_orthogonalize_ws_bytes(const conv_ortho_desc* d);

/* The kernels and tiles it takes, as conv_describe. */
conv_status conv_orthogonalize_describe(const conv_ortho_desc* d, char* buf, int32_t len);

/*   g   : device [batch][rows][cols] of dtype
 *   out : device [batch][rows][cols] bf16 (one RNE rounding)
 * Matrices whose shorter side is at most 64 and longer at most 1024 need no
 * scratch. The products run on fp16 matrix instructions with fp32 sums; X is
 * held as a pair of fp16 (22 bits; fp32 without scratch), the diagonals of A and
 * of the polynomial in fp32. Besides its bf16 rounding the result is then off, in
 * the Frobenius norm, by a fifth to three quarters of that rounding after five
 * steps of a, b, c = 3.4445, -4.7750, 2.0315 (0.21 for 700 x 900, 0.30 for
 * 64 x 576, 0.73 for 16 x 1000), by up to 1.4 of it after eight, and by less than
 * a third for coefficients under which the singular values converge. Values are
 * scaled by powers of two to stay in fp16's range. Coefficients that between two
 * steps take an entry of X to 255 (singular values up to 2 do not), or off the
 * diagonal one of A to 16 or one of b A + c A A to 64, leave that range and give
 * infinities or NaN, also where fp32 would hold them. The norm is summed in 64 bits. A zero matrix with eps > 0 gives zeros.
 * CONV_E_SHAPE: a size <= 0, steps or a coefficient out of range.
 * CONV_E_UNSUPPORTED: dtype, batch > 65535, a side over 32768, a size limit. */
conv_status conv_orthogonalize(const conv_ortho_desc* d, const void* g, void* out, void* ws, int64_t ws_bytes,
                               void* stream);

#ifdef __cplusplus
}
#endif

#endif /* CONV_TRAIN_H */
