/*
 * norm_w4.h — C ABI of the operators around the NF4-LoRA linear (lora_nf4.h): the
 * root-mean-square norm in front of it, with its gradient for training and an 8-bit
 * output for serving, and the product with a 4-bit group-scaled weight that serves
 * the merged weight (lora_nf4_merge) without adapters. Part of liblora_nf4.so.
 *
 * Conventions as in lora_nf4.h: device pointers owned by the caller (16-byte
 * aligned, workspaces 256-byte), dense row-major matrices, bf16 as uint16_t bit
 * patterns, work enqueued on `stream` of the current device, nothing allocated or
 * synchronized, arguments checked on the host before any HIP call (ln_status codes),
 * outputs disjoint from inputs and from each other (LN_EALIAS), no state kept
 * between calls. T = 0 is an empty batch: sizes are checked, nothing is computed
 * except where noted, and token operands may be NULL. Floating-point inputs must be
 * finite (not checked).
 */
#ifndef NORM_W4_H
#define NORM_W4_H

#include <stddef.h>
#include <stdint.h>

#include "lora_nf4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* 8-bit formats, beside ln_dtype's LN_F32 and LN_BF16: OCP FP8 E4M3 ("E4M3FN", largest
   448) and two's complement integers. */
typedef enum { LN_E4M3 = 2, LN_I8 = 3 } ln_qtype;

#define LN_NORM_MAX_D (1 << 20)  /* widest row of the norm */
#define LN_W4_MAX_D_IN (1 << 22) /* widest d_in of a 4-bit weight */

/*
 * rmsnorm_fwd — the norm of T rows of d values, with the residual's addition:
 *     h = x + residual      (the float32 sum rounded to dtype; h = x without a residual)
 *     y = h rstd w,   rstd = 1 / sqrt(mean(h^2) + eps)        per row
 * The sum of squares runs over the rounded h in float32 (where it overflows, |h| above 1e19 /
 * sqrt(d), rstd is 0); y is rounded once.
 *   dtype     LN_BF16 or LN_F32, of x, residual, w, h and y
 *   eps       > 0, finite
 *   x, residual, h, y   [T, d]; residual and h both given or both NULL
 *   w         [d]
 *   rstd      float32 [T] (output; may be NULL); rmsnorm_bwd reads it
 * T >= 0, 1 <= d <= LN_NORM_MAX_D, any width (fastest where a row is a multiple of 16
 * bytes, so that every row starts aligned). A row of NaN or infinities affects itself only.
 */
int rmsnorm_fwd(int64_t T, int64_t d, int dtype, float eps, const void* x, const void* residual,
                const void* w, void* h, void* y, float* rstd, void* stream);

/*
 * rmsnorm_fwd_quant — the same norm with its output in 8 bits and one scale a row, as
 * w4_matvec reads it:
 *     scale = max_j |y_j| / top,   q_j = y_j / scale in q_type    (top 448 or 127)
 * to the nearest level, halves to the even one; a row of zeros has scale 0 and q 0. The quotient
 * y_j / scale is formed as (h w)_j (top / max |h w|), for bf16 rows exactly (h w is exact, and
 * a quotient next to the middle of two levels is on its side of it), for float32 rows from
 * the rounded h w and off by at most 3 2^-24 of it before it goes to its level. A scale in float32's
 * subnormal range is rounded up, so that no level passes top; the levels are those of the
 * scale as it is stored.
 *   q         [T, d] of q_type (LN_E4M3 or LN_I8), q_scale float32 [T] (outputs)
 *   the other arguments as for rmsnorm_fwd.
 */
int rmsnorm_fwd_quant(int64_t T, int64_t d, int dtype, float eps, const void* x, const void* residual,
                      const void* w, void* h, int q_type, void* q, float* q_scale, void* stream);

/*
 * rmsnorm_bwd — gradients of rmsnorm_fwd. With g = dy w and n = h rstd,
 *     dx = dh + rstd (g - n mean(g n)),      dw = sum over rows of dy n
 * dx is the gradient of x and of the residual alike (h is their sum).
 *   dy, h     [T, d] (h as rmsnorm_fwd left it; x where there was no residual)
 *   dh        [T, d], the gradient that reaches h from its other readers, or NULL
 *   rstd      float32 [T] from rmsnorm_fwd
 *   dx        [T, d];  dw [d] or NULL (a frozen weight); both of dtype, rounded once
 *   workspace rmsnorm_bwd_workspace_bytes(T, d) bytes where dw is given (float32 sums
 *             of row blocks, joined in a fixed order: dw does not depend on the run),
 *             not needed otherwise
 * T = 0 sets dw to zero.
 */
int rmsnorm_bwd(int64_t T, int64_t d, int dtype, const void* dy, const void* dh, const void* h,
                const void* w, const float* rstd, void* dx, void* dw, void* workspace,
                size_t workspace_bytes, void* stream);

/* Workspace bytes rmsnorm_bwd needs with dw (0 if the sizes are invalid or T = 0). */
size_t rmsnorm_bwd_workspace_bytes(int64_t T, int64_t d);

/*
 * The packed 4-bit weight. A weight of d_out rows and d_in columns is held as
 *     w[n][k] = (c[n][k] - z[n][k / group]) s[n][k / group],   c, z in 0 .. 15
 * with group 32, 64 or 128, d_in a multiple of 64 and of group, any d_out >= 1, fewer than
 * 2^24 tiles in all (see below). z is 8 everywhere where no zero points are stored. Codes lie in tiles of 16 rows x 128
 * columns, so that one wave reads a tile as 1024 consecutive bytes and each lane's 16
 * bytes are matrix-instruction operands in place:
 *   codes   uint8 [ceil(d_out / 16)][ceil(d_in / 128)][1024]; byte 256 g + 16 r + 4 q + i
 *           of a tile holds row r, column 32 q + 8 g + i in its low nibble and column
 *           32 q + 8 g + i + 4 in its high nibble (g, q, i in 0 .. 3, r in 0 .. 15)
 *   scales  bf16 [ceil(d_out / 16)][d_in / group][16], the last index the row of the tile
 *   zeros   uint8 of scales' shape, values 0 .. 15, or NULL
 * Rows past d_out and columns past d_in exist in codes and scales only as padding:
 * w4_quantize writes zeros there, readers ignore what they hold.
 */

/*
 * w4_quantize — packs w [d_out, d_in] (LN_F32 or LN_BF16), round to nearest-even:
 *   zeros NULL: s = bf16(f32(max|w| / 7)),  c = clamp(rint(f32(w / s)), -8, 7) + 8
 *   zeros:      lo = min(w, 0), hi = max(w, 0) over the group, s = bf16(f32(f32(hi - lo) / 15)),
 *               z = clamp(rint(f32(-lo / s)), 0, 15),  c = clamp(rint(f32(w / s)) + z, 0, 15)
 * A group with s = 0 has c = z (8, or 0 with zero points). hi - lo must be finite in float32.
 */
int w4_quantize(const void* w, int w_dtype, int64_t d_out, int64_t d_in, int32_t group, uint8_t* codes,
                uint16_t* scales, uint8_t* zeros, void* stream);

/* w4_dequantize — out [d_out, d_in] = (c - z) s, rounded once to out_dtype (LN_F32: exact). */
int w4_dequantize(const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros, int64_t d_out,
                  int64_t d_in, int32_t group, int out_dtype, void* out, void* stream);

/*
 * w4_matvec — y = x W^T for a few rows of x and a packed weight W:
 *     y[t][n] = x_scale[t] sum_groups s (sum_k x[t][k] c[n][k] - z sum_k x[t][k])
 * in float32 (8-bit integers: int32 inside a group, exact), rounded once to y_dtype.
 *   x         [T, d_in] of x_dtype: LN_BF16, LN_E4M3 or LN_I8
 *   x_scale   float32 [T], one factor a row (rmsnorm_fwd_quant's q_scale), or NULL (1)
 *   y         [T, d_out] of y_dtype: LN_BF16 or LN_F32
 *   workspace w4_matvec_workspace_bytes(T, d_in, d_out) bytes (0 unless d_in is split
 *             across workgroups, where the float32 sums of the splits meet in it, added in
 *             a fixed order); may be NULL when that is 0
 *             (two calls that may run at the same time need a workspace each)
 * 0 <= T <= 2^21, T d_out <= 2^35 - 16 T; made for up to 64 rows, where reading the packed weight bounds it. More
 * rows run as blocks of 64, each reading the weight again.
 */
int w4_matvec(int64_t T, int64_t d_in, int64_t d_out, int32_t group, int x_dtype, const void* x,
              const float* x_scale, const uint8_t* codes, const uint16_t* scales, const uint8_t* zeros,
              int y_dtype, void* y, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes w4_matvec needs (0 if the sizes are invalid, T = 0, or none is needed). */
size_t w4_matvec_workspace_bytes(int64_t T, int64_t d_in, int64_t d_out);

/*
 * w4_matvec_multi — w4_matvec of n_proj weights that read the same x (q/k/v, gate/up)
 * in one launch (and one more where d_in is split).
 *   d_out, codes, scales, zeros, y   HOST arrays [n_proj] (1 .. LN_MAX_PROJ), read
 *             during the call only; zeros NULL: no weight has zero points, otherwise
 *             every entry is given
 *   workspace as for w4_matvec, sized by w4_matvec_multi_workspace_bytes
 * All weights share d_in and group. (The values are those of single calls up to the
 * order of float32 additions, where the two split d_in differently.)
 */
int w4_matvec_multi(int64_t T, int64_t d_in, int32_t n_proj, const int64_t* d_out, int32_t group,
                    int x_dtype, const void* x, const float* x_scale, const uint8_t* const* codes,
                    const uint16_t* const* scales, const uint8_t* const* zeros, int y_dtype,
                    void* const* y, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes w4_matvec_multi needs (0 if the sizes are invalid, T = 0, or none is needed). */
size_t w4_matvec_multi_workspace_bytes(int64_t T, int64_t d_in, int32_t n_proj, const int64_t* d_out);

#ifdef __cplusplus
}
#endif

#endif /* NORM_W4_H */
