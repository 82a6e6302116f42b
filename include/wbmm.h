/*
 * wbmm.h — C ABI of libwbmm: WBMM (Windowed Batch Matrix Multiplication) on AMD MI355X (gfx950).
 *
 * WBMM cuts a feature map into non-overlapping w x w windows (d = w*w pixels), builds for every
 * channel c a d x d matrix M_c from a compact (2w-1) x (2w-1) relative-position table T_c, and
 * mixes every window of every image with one shared matmul out = M_c . x, with no softmax
 * [gecl.asia reading notes, "Core Idea"; arxivdaily abstract; pith page, Fig. 1 caption].
 *
 * Conventions shared by every entry point:
 *   - Index orientation: M_c[i][j] = T_c[(y_i - y_j) + w - 1][(x_i - x_j) + w - 1], in-window
 *     position i = y_i * w + x_i (row-major); the table's first axis is vertical.
 *   - Every pointer argument named as device memory must be a device (HBM) address on the current
 *     HIP device, aligned to its element size (workspaces: see each call).
 *   - The caller owns every buffer. The library never allocates or frees device memory and never
 *     synchronizes: all work is enqueued on `stream` (a hipStream_t passed as void*; NULL = the
 *     default stream) and runs asynchronously.
 *   - Arguments are validated on the host before anything is enqueued. On any status other than
 *     WBMM_OK nothing has been enqueued (except WBMM_E_HIP, which reports a failed launch) and
 *     wbmm_last_error() returns a message for the calling thread.
 *   - Outputs are overwritten, never accumulated into.
 *   - Tensor layouts: feature maps are (B, C, H, W) in WBMM_NCHW or (B, H, W, C) in WBMM_NHWC,
 *     dense, no strides. Tables are (C, 2w-1, 2w-1), matrices (C, d, d), mix weights (C, 3, 3),
 *     all dense row-major.
 *   - H and W need not be multiples of w: the map is treated as zero-padded at the bottom and
 *     right to the next multiple of w, and outputs are cropped back to H x W.
 */
#ifndef WBMM_H
#define WBMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define WBMM_ABI_VERSION 1

typedef enum wbmm_status {
  WBMM_OK = 0,
  WBMM_E_INVALID = 1,      /* a size, pointer or combination of arguments is invalid          */
  WBMM_E_UNSUPPORTED = 2,  /* valid request this build does not provide (e.g. misalignment)   */
  WBMM_E_WORKSPACE = 3,    /* workspace missing or smaller than the matching *_bytes query    */
  WBMM_E_HIP = 4           /* a HIP launch failed; wbmm_last_error() carries HIP's message    */
} wbmm_status;

typedef enum wbmm_dtype { WBMM_F32 = 0, WBMM_BF16 = 1 } wbmm_dtype;
typedef enum wbmm_layout { WBMM_NCHW = 0, WBMM_NHWC = 1 } wbmm_layout;

/* ABI version this library was built with (WBMM_ABI_VERSION). */
int wbmm_abi_version(void);

/* Message for the last non-OK status returned on the calling thread ("" if none). The pointer
 * stays valid until the next wbmm_* call on the same thread. */
const char* wbmm_last_error(void);

/*
 * wbmm_build_index — relative-position index of one window.
 * Defines: the table lookup that turns an in-window pair (i, j) into a table entry
 *          [gecl.asia reading notes, "Core Idea" and "Method" point 2].
 *   idx[i*d + j] = ((y_i - y_j) + w - 1) * (2w - 1) + ((x_i - x_j) + w - 1)   (int32, d x d)
 * w:   window side, 1 <= w <= 32.
 * idx: device, int32 [d*d], written.
 * Bit-exact. Errors: WBMM_E_INVALID for w out of range or idx == NULL.
 */
wbmm_status wbmm_build_index(int w, int32_t* idx, void* stream);

/*
 * wbmm_build_matrix — materialize M_c from the table (the pages' inference caching of the
 * constructed weights) [gecl.asia reading notes, "Core Idea"; "Method", last sentence].
 *   M[c][i][j] = T[c][idx[i][j]]   (an exact copy in the table's dtype)
 * T: device [C][2w-1][2w-1], dtype `dtype` (WBMM_F32 or WBMM_BF16).
 * M: device [C][d][d], same dtype, written. Must not overlap T.
 * Bit-exact. Errors: WBMM_E_INVALID for C < 1, w out of range, NULL pointers, bad dtype.
 */
wbmm_status wbmm_build_matrix(const void* T, int C, int w, int dtype, void* M, void* stream);

/*
 * wbmm_fold_hier — fold an s x s sub-window table into a w x w window matrix (hierarchical
 * window reparameterization, zero inference cost) [gecl.asia reading notes, "Method" point 4;
 * arxivdaily abstract].
 *   For pairs (i, j) in the same s x s sub-window (sub-windows tile the window from its origin):
 *     M_out[c][i][j] = M_in[c][i][j] + T_sub[c][idx_s(i, j)]   (one add in `dtype`, RNE)
 *   otherwise M_out[c][i][j] = M_in[c][i][j]; idx_s is wbmm_build_index's formula with s for w
 *   applied to the in-sub-window coordinates (y mod s, x mod s).
 * M_in:  device [C][d][d]; T_sub: device [C][2s-1][2s-1]; M_out: device [C][d][d], written;
 *        M_out may equal M_in (in place) but must not partially overlap it.
 * s must divide w and 1 <= s < w. dtype WBMM_F32 or WBMM_BF16 (bf16 adds round to bf16, RNE).
 * Bit-exact. Errors: WBMM_E_INVALID for bad sizes, s not dividing w, NULL pointers.
 */
wbmm_status wbmm_fold_hier(const void* M_in, const void* T_sub, int C, int w, int s, int dtype,
                           void* M_out, void* stream);

/*
 * wbmm_forward_workspace_bytes — device workspace wbmm_forward needs for these arguments
 * (0 when none), the largest need over fp32 and bf16 inputs and outputs (a bf16 z_save with the
 * mix in window mode takes the fp32 pre-mix map through the workspace; bf16 maps with the mix
 * on the fast bf16 shapes keep z there when no z_save is given). Returns 0 for invalid
 * arguments as well; wbmm_forward reports those.
 */
size_t wbmm_forward_workspace_bytes(int B, int C, int H, int W, int w, int layout, int has_mix,
                                    int has_z_save);

/*
 * wbmm_forward — the WBMM layer forward [gecl.asia reading notes, "Core Idea", "Method";
 * pith page, "Core claim"; arxivdaily abstract].
 *   z = crop(reverse(M_c . partition(pad(x))))   for every channel c, window and image;
 *   y = mix3x3(z, mix_w) if mix_w != NULL, else y = z.
 * mix3x3 is the inter-block 3x3 depthwise cross-correlation, zero padding 1, stride 1, no bias:
 *   y[b,c,h,v] = sum_{u,t in 0..2} mix_w[c,u,t] * z[b,c,h+u-1,v+t-1]  (z = 0 outside the map)
 *   [gecl.asia reading notes, "Method" point 3].
 * Sizes: B, C, H, W >= 1; 1 <= w <= 32.
 * layout:    WBMM_NCHW or WBMM_NHWC (x, y and z_save share it).
 * in_dtype:  WBMM_F32 or WBMM_BF16 for x and for T/M. Products accumulate in fp32.
 * out_dtype: WBMM_F32 or WBMM_BF16 for y and z_save (bf16 outputs are rounded RNE from fp32).
 * x:      device map, in_dtype.
 * T, M:   exactly one non-NULL. T: device [C][2w-1][2w-1] — M_c is formed on chip from T_c.
 *         M: device [C][d][d] — the cached (possibly folded) matrices are read from memory.
 * mix_w:  device fp32 [C][3][3] or NULL. The mix runs in fp32 on the fp32 pre-mix map; with
 *         bf16 output, y and z_save are rounded from it (RNE).
 * z_save: device map in out_dtype receiving the pre-mix output z (for the backward), or NULL.
 * y:      device map in out_dtype, written; must not overlap x, T, M, mix_w or z_save.
 * workspace / workspace_bytes: device scratch of at least wbmm_forward_workspace_bytes(...)
 *         bytes (may be NULL when that is 0).
 * Errors: WBMM_E_INVALID (sizes, pointers, both or neither of T/M, overlap of y with x),
 *         WBMM_E_UNSUPPORTED (misaligned pointer), WBMM_E_WORKSPACE, WBMM_E_HIP.
 */
wbmm_status wbmm_forward(int B, int C, int H, int W, int w, int layout, int in_dtype,
                         int out_dtype, const void* x, const void* T, const void* M,
                         const float* mix_w, void* z_save, void* y, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * wbmm_backward_workspace_bytes — device workspace wbmm_backward needs (per-workgroup fp64
 * partial tables, and a dz buffer when the mix cannot be fused). Returns 0 for invalid arguments.
 */
size_t wbmm_backward_workspace_bytes(int B, int C, int H, int W, int w, int layout, int has_mix);

/*
 * wbmm_backward — gradients of wbmm_forward (fp32). The pages train with the operator but do not
 * write out its backward; it follows from the forward by the chain rule:
 *   dz    = mix3x3 adjoint of dy (correlation with the 180-degree rotated mix_w), or dy if no mix;
 *   dmix_w[c,u,t] = sum_{b,h,v} dy[b,c,h,v] * z[b,c,h+u-1,v+t-1];
 *   G_c   = partition(pad(dz));  dx = crop(reverse(M_c^T . G_c));
 *   dT[c][k] = sum over pairs (i,j) with idx[i][j] = k of (G_c . X_c^T)[i][j].
 * x, dy:   device fp32 maps in `layout`.
 * T, M:    exactly one non-NULL (as in wbmm_forward; with M, dT is the gradient with respect to
 *          the table that M was gathered from).
 * mix_w:   device fp32 [C][3][3] or NULL; z_saved (the forward's z_save) is required iff mix_w.
 * dx:      device fp32 map, written, or NULL to skip.
 * dT:      device fp32 [C][2w-1][2w-1], written, or NULL to skip.
 * dmix_w:  device fp32 [C][3][3], written, or NULL to skip (ignored without mix_w).
 * workspace / workspace_bytes: device scratch of at least wbmm_backward_workspace_bytes(...)
 *          bytes, 256-byte aligned; no initial contents are required. Calls that share a
 *          workspace must be ordered on one stream.
 * dT and dmix_w are reduced in a fixed order (fp64 per-workgroup partials summed by a second,
 * small kernel; no floating-point atomics): results are bitwise reproducible run to run.
 * Windows 1 <= w <= 32 (16 < w <= 32: dx through the forward contraction with the table
 * rotated by 180 degrees or the matrix transposed, whose matrix is M^T; dT from row-pair tiles
 * of 32 x 32, with the windows as the sum dimension).
 * Errors: WBMM_E_INVALID, WBMM_E_UNSUPPORTED (misaligned pointer), WBMM_E_WORKSPACE,
 *         WBMM_E_HIP.
 */
wbmm_status wbmm_backward(int B, int C, int H, int W, int w, int layout, const float* x,
                          const float* T, const float* M, const float* mix_w,
                          const float* z_saved, const float* dy, float* dx, float* dT,
                          float* dmix_w, void* workspace, size_t workspace_bytes, void* stream);

/*
 * wbmm_backward_noalloc — wbmm_backward for callers that cannot allocate device memory (code
 * under HIP graph capture, tight serving or training loops, harnesses that forbid hipMalloc):
 * the same gradients, arguments and errors, minus the workspace. The scratch that the backward
 * needs (per-workgroup fp64 partials, a dz map) is a fixed device array inside the library, one
 * copy per GPU, held until the process ends: WBMM_NOALLOC_SCRATCH_BYTES bytes. A problem whose
 * wbmm_backward_workspace_bytes(...) exceeds that is rejected with WBMM_E_UNSUPPORTED. The call
 * allocates and frees nothing and needs no initial contents in the scratch. Every call on one
 * GPU shares that GPU's scratch: calls that may overlap on one GPU (other streams, other host
 * threads) race and must be ordered by the caller; calls on one stream are ordered.
 */
#define WBMM_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
wbmm_status wbmm_backward_noalloc(int B, int C, int H, int W, int w, int layout, const float* x,
                                  const float* T, const float* M, const float* mix_w,
                                  const float* z_saved, const float* dy, float* dx, float* dT,
                                  float* dmix_w, void* stream);

/*
 * wbmm_forward_hier_workspace_bytes — device workspace wbmm_forward_hier needs (0 when none, and
 * 0 for invalid arguments, which wbmm_forward_hier reports).
 */
size_t wbmm_forward_hier_workspace_bytes(int B, int C, int H, int W, int w, int s, int layout,
                                         int has_mix, int has_z_save);

/*
 * wbmm_forward_hier — the layer forward with the hierarchical reparameterization folded on chip
 * [gecl.asia reading notes, "Method" point 4: a sub-window table overlays 7x7 structure in a
 * 14x14 window at no inference cost]. The matrix is
 *   M'_c[i][j] = M_c[i][j] + T_sub[c][idx_s(i, j)]   for pairs i, j in one s x s sub-window,
 *   M'_c[i][j] = M_c[i][j]                           otherwise,
 * each sum one fp32 add (RNE): exactly what wbmm_fold_hier stores. Then z and y as in
 * wbmm_forward. fp32 only; s divides w and s < w. For w = 2s (the sub-windows are the window's
 * quadrants) the fold happens on chip and M' is never formed in memory; for other s, M' is
 * built and folded in the workspace (C w^4 floats) and read as a cached matrix.
 * x, y, z_save: device fp32 maps in `layout`; T: device fp32 [C][2w-1][2w-1];
 * T_sub: device fp32 [C][2s-1][2s-1]; mix_w, z_save, workspace as in wbmm_forward
 * (workspace size from wbmm_forward_hier_workspace_bytes).
 * Errors: WBMM_E_INVALID (sizes, s not dividing w or not below it, NULL or overlapping
 *         pointers), WBMM_E_UNSUPPORTED (no launch shape, misaligned pointer), WBMM_E_WORKSPACE,
 *         WBMM_E_HIP.
 */
wbmm_status wbmm_forward_hier(int B, int C, int H, int W, int w, int s, int layout, const float* x,
                              const float* T, const float* T_sub, const float* mix_w,
                              float* z_save, float* y, void* workspace, size_t workspace_bytes,
                              void* stream);

/*
 * wbmm_backward_hier_workspace_bytes — device workspace wbmm_backward_hier needs (0 for invalid
 * arguments).
 */
size_t wbmm_backward_hier_workspace_bytes(int B, int C, int H, int W, int w, int s, int layout,
                                          int has_mix);

/*
 * wbmm_backward_hier — gradients of wbmm_forward_hier (fp32). As wbmm_backward with M' in place
 * of M, and in addition the sub-table's gradient:
 *   dx = crop(reverse(M'_c^T . G_c));   dT[c][k] = sum over pairs (i,j) with idx[i][j] = k of
 *   (G_c . X_c^T)[i][j];   dT_sub[c][k'] = the same sum over the pairs inside one s x s
 *   sub-window with idx_s[i][j] = k'.
 * T, T_sub: as in wbmm_forward_hier. dx, dT, dT_sub, dmix_w: written, or NULL to skip
 * (dT_sub: device fp32 [C][2s-1][2s-1]). mix_w, z_saved, dy, workspace as in wbmm_backward.
 * dT, dT_sub and dmix_w are reduced in a fixed order: bitwise reproducible run to run.
 * Any s dividing w with s < w, 1 <= w <= 32: for w = 2s on chip; for other s with M' built in
 * the workspace, dX and dT from the cached-matrix backward, and dT_sub as the table gradient of
 * an s-window layer on the same G and x (a pair of one sub-window is a pair of one window of
 * the s-grid, which the w-grid subdivides).
 * Errors: WBMM_E_INVALID (as wbmm_forward_hier), WBMM_E_UNSUPPORTED (no launch shape,
 *         misaligned pointer), WBMM_E_WORKSPACE, WBMM_E_HIP.
 */
wbmm_status wbmm_backward_hier(int B, int C, int H, int W, int w, int s, int layout,
                               const float* x, const float* T, const float* T_sub,
                               const float* mix_w, const float* z_saved, const float* dy,
                               float* dx, float* dT, float* dT_sub, float* dmix_w,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * wbmm_forward_shifted_workspace_bytes / wbmm_forward_shifted — wbmm_forward on a window grid
 * offset by (oy, ox), 0 <= oy, ox < w: the interleaved grid that alternate layers can use so
 * that information crosses window borders [gecl.asia reading notes, "Limitations": interleaving
 * windows between layers]. Window (wy, wx) covers map rows wy*w - oy .. wy*w - oy + w - 1 and
 * columns wx*w - ox .. wx*w - ox + w - 1; the pixels of a border window that lie outside the map
 * are zeros (no cyclic roll), and only positions inside the map are written. (0, 0) is exactly
 * wbmm_forward. Every other argument, layout, dtype and error as in wbmm_forward; an offset
 * outside [0, w) is WBMM_E_INVALID.
 */
size_t wbmm_forward_shifted_workspace_bytes(int B, int C, int H, int W, int w, int oy, int ox,
                                            int layout, int has_mix, int has_z_save);
wbmm_status wbmm_forward_shifted(int B, int C, int H, int W, int w, int oy, int ox, int layout,
                                 int in_dtype, int out_dtype, const void* x, const void* T,
                                 const void* M, const float* mix_w, void* z_save, void* y,
                                 void* workspace, size_t workspace_bytes, void* stream);

/*
 * wbmm_backward_shifted_workspace_bytes / wbmm_backward_shifted — the gradients of
 * wbmm_forward_shifted (dx, dT, dmix_w), with the arguments, outputs and errors of wbmm_backward
 * plus the grid offset (oy, ox) of the forward. The padding pixels are constants: dT sums the
 * pair products of the map's own pixels only.
 */
size_t wbmm_backward_shifted_workspace_bytes(int B, int C, int H, int W, int w, int oy, int ox,
                                             int layout, int has_mix);
wbmm_status wbmm_backward_shifted(int B, int C, int H, int W, int w, int oy, int ox, int layout,
                                  const float* x, const float* T, const float* M,
                                  const float* mix_w, const float* z_saved, const float* dy,
                                  float* dx, float* dT, float* dmix_w, void* workspace,
                                  size_t workspace_bytes, void* stream);

/*
 * wbmm_dwconv_forward — the standard k x k depthwise convolution (DW-Std) that the pages time
 * WBMM against: every output gathers the k*k neighbours around its own position in its own
 * channel [pith page, Fig. 1 and Fig. 2 captions; operator benchmark, Fig. 3 caption]. Not part of
 * a WBMM layer; provided so the comparison runs on the same hardware.
 *   y[b,c,h,v] = sum_{u,t in 0..k-1} w_dw[c,u,t] * x[b,c,h+u-p,v+t-p],  p = k / 2,
 *   x taken as 0 outside the map (cross-correlation, stride 1, no bias: the frameworks' form).
 * Sizes: B, C, H, W >= 1; k odd, 3 <= k <= 13 (WBMM_E_UNSUPPORTED otherwise, and for rows too
 *         long for one workgroup's staging buffer, about 600 pixels).
 * x:    device fp32 NCHW [B][C][H][W].
 * w_dw: device fp32 [C][k][k].
 * y:    device fp32 NCHW [B][C][H][W], written; must not overlap x or w_dw.
 * Accumulates in fp32 (one fma per tap, taps in row-major order). Enqueued on `stream`; no
 * workspace. Errors: WBMM_E_INVALID (sizes, even k, NULL, overlap), WBMM_E_UNSUPPORTED (k or
 * row length out of range, misaligned pointers), WBMM_E_HIP (launch failure).
 */
wbmm_status wbmm_dwconv_forward(int B, int C, int H, int W, int k, const float* x,
                                const float* w_dw, float* y, void* stream);

/*
 * wbmm_backward_bf16_workspace_bytes / wbmm_backward_bf16 — the layer backward with bf16 maps
 * (mixed-precision training): x, dy, z_saved and dx in bf16, T in bf16 (the forward's table),
 * dT and dmix_w in fp32. Same gradients as wbmm_backward (derived by the chain rule; the pages
 * train with the operator [arxivdaily abstract]):
 *   G = mix adjoint of dy (kept as a bf16 map, RNE), or dy itself without a mix;
 *   dx = M_c^T G per window (bf16 matrix cores, fp32 accumulation, RNE to bf16);
 *   dT_c[k] = sum over pairs with idx = k of (G X^T)[i][j] (bf16 products, fp32 sums over a
 *   group of windows, fp64 across groups in a fixed order); dmix_w as in wbmm_backward.
 * Any 1 <= w <= 32, NCHW or NHWC (`layout`), any map size; w = 14 on NCHW 28x28 or 56x56 maps
 * runs the bf16 matrix-core kernels, other shapes the fp32 kernels on the bf16 values (widened
 * exactly), with dx rounded to bf16 (RNE).
 * mix_w / z_saved: both or neither. dx, dT, dmix_w may each be NULL (skipped). bf16 maps and T
 * must be 16-byte aligned. workspace: at least wbmm_backward_bf16_workspace_bytes(...) bytes,
 * 256-byte aligned (never NULL: the dT partials live there). Errors as in wbmm_backward.
 */
size_t wbmm_backward_bf16_workspace_bytes(int B, int C, int H, int W, int w, int layout,
                                          int has_mix);
wbmm_status wbmm_backward_bf16(int B, int C, int H, int W, int w, int layout, const void* x,
                               const void* T, const float* mix_w, const void* z_saved,
                               const void* dy, void* dx, float* dT, float* dmix_w,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * 8-bit activation checkpoints: what a training step keeps of a map between forward and backward.
 * A tensor of n elements is n code bytes and ceil(n / WBMM_CKPT_GROUP) scale bytes, one per group
 * of WBMM_CKPT_GROUP elements in memory order (the last group may be short):
 *   value = q(code) * 2^(byte - 127);   byte 255: every value of the group is NaN,
 * q(code) the int8 value (WBMM_CKPT_INT8) or the OCP 8-bit float 4-3 value (WBMM_CKPT_E4M3).
 * int8 spreads its steps evenly below the group's largest magnitude, e4m3 keeps a relative error
 * of at most 2^-4 for magnitudes down to 2^-13 of it. Decoded values are exact in bf16 and fp32,
 * results outside their range aside: in bf16 the smallest codes under bytes 0 to 2; and the largest
 * magnitudes, above 127/64 2^127 in int8 and from 31/16 2^127 in e4m3, whose nearest code stands
 * for 2^128, which reads back as an infinity.
 */
#define WBMM_CKPT_GROUP 32
typedef enum wbmm_ckpt_format { WBMM_CKPT_INT8 = 0, WBMM_CKPT_E4M3 = 1 } wbmm_ckpt_format;

/*
 * wbmm_ckpt_pack — tensor to checkpoint. Per group, with amax the largest magnitude and top = 127
 * (int8) or 448 (e4m3): e is the least integer >= -126 with amax <= top 2^e, the byte e + 127, and
 * a code the nearest to x 2^-e, ties to even. A group that holds an infinity or a NaN gets byte
 * 255 (codes 0).
 * x:      device, n elements of `dtype`, any layout (dense).
 * codes:  device, n bytes, written. scales: device, ceil(n / WBMM_CKPT_GROUP) bytes, written.
 * wbmm_ckpt_unpack — the inverse: x = the values, in `dtype`.
 * Any pointer alignment down to the element works; x aligned to 16 and codes to 8 bytes takes the
 * wide accesses. Bit-exact. Errors: WBMM_E_INVALID (n < 1, dtype, fmt, NULL or overlapping
 * buffers), WBMM_E_UNSUPPORTED (n > 2^35, x not aligned to its elements), WBMM_E_HIP.
 */
wbmm_status wbmm_ckpt_pack(const void* x, int64_t n, int dtype, int fmt, uint8_t* codes,
                           uint8_t* scales, void* stream);
wbmm_status wbmm_ckpt_unpack(const uint8_t* codes, const uint8_t* scales, int64_t n, int dtype,
                             int fmt, void* x, void* stream);

/*
 * wbmm_backward_ckpt_workspace_bytes / wbmm_backward_ckpt — wbmm_backward with the two maps that
 * a training step keeps, x and the pre-mix z, as checkpoints in `fmt` (packed in the maps' own
 * memory order, B C H W elements). dT sums over the checkpoint's x, dmix_w over its z; dx needs
 * neither. Every other argument, output, rule and error as in wbmm_backward (table input).
 * dtype:   of T, dy and dx: WBMM_F32, or WBMM_BF16 (widened exactly). mix_w, dT and dmix_w are
 *          fp32 in both, and so is G, dy after the mix adjoint; dT's and dmix_w's products and sums
 *          are in fp32 and fp64 for either type, dx's in fp32. For WBMM_BF16 with the mix G enters
 *          dx's products as the sum of two bf16 numbers, to 2^-17 of itself: an error of dx of up
 *          to 2^-17 sum |T| |G| over its window, before the one rounding to bf16 (RNE), which is
 *          up to 2^-8 |dx|.
 * x_codes, x_scales, z_codes, z_scales: as wbmm_ckpt_pack writes them; z_* exactly with mix_w.
 * dx, dT, dmix_w: written, or NULL to skip. workspace: 256-byte aligned. For w = 1, w > 16 and
 * most maps of 33 C H W >= 2^30 it holds the decoded maps beside wbmm_backward's own: 4 bytes an element for x,
 * for z with the mix, and for WBMM_BF16 for dy and dx as well, so that a call needs more memory
 * than the checkpoints save.
 * For 2 <= w <= 16 (very large images, 33 C H W >= 2^30, aside) every other fp32 operand enters the
 * products as the sum of three bf16 numbers, which an infinity has not, nor has a finite magnitude
 * of (2 - 2^-8) 2^127 or more: such entries of T or G make the results that they reach NaN. Other
 * windows run wbmm_backward's kernels, in fp32 throughout.
 * Errors as in wbmm_backward; also WBMM_E_INVALID for an unknown fmt.
 */
size_t wbmm_backward_ckpt_workspace_bytes(int B, int C, int H, int W, int w, int layout, int dtype,
                                          int has_mix);
wbmm_status wbmm_backward_ckpt(int B, int C, int H, int W, int w, int layout, int dtype, int fmt,
                               const uint8_t* x_codes, const uint8_t* x_scales, const void* T,
                               const float* mix_w, const uint8_t* z_codes,
                               const uint8_t* z_scales, const void* dy, void* dx, float* dT,
                               float* dmix_w, void* workspace, size_t workspace_bytes,
                               void* stream);

/*
 * wbmm_scan_forward_workspace_bytes / wbmm_scan_forward — gated linear recurrence along one axis: a mixer
 * of any reach, next to the windowed one and on the same maps. Tensors are dense (outer, len,
 * inner); the recurrence runs along len, independently for every (outer, inner):
 *   a_t = sigmoid(g_t),   h_t = a_t h_{t-1} + (1 - a_t) u_t,   h_{-1} = h0.
 * A map in raster order is (B C, H W, 1) in NCHW and (B, H W, C) in NHWC; its columns in NCHW are
 * (B C, H, W), its rows (B C H, W, 1). A serving step is len = 1 with h0 and h_last.
 * dtype:    of g, u and h: WBMM_F32 or WBMM_BF16. The recurrence itself is fp32.
 * reverse:  nonzero: sequences run from their last position to their first.
 * h0:       device fp32 [outer][inner], or NULL for zeros.
 * lens:     device int32 [n_lens], n_lens dividing outer, or NULL (n_lens ignored): sequence o has
 *           lens[o / (outer / n_lens)] positions, held to [0, len]. Positions past it are not
 *           used, whatever they hold, and h is 0 there; a reversed sequence starts at its own last
 *           position.
 * h:        device map, written.
 * h_last:   device fp32 [outer][inner], or NULL: the state after the last step (h0 for an empty
 *           sequence). May be h0 itself (updated in place).
 * states:   device fp32 [outer][ceil(len / WBMM_SCAN_CHUNK)][inner], or NULL: the state before
 *           steps 0, WBMM_SCAN_CHUNK, 2 WBMM_SCAN_CHUNK, ... in the order the sequence runs (its
 *           last state past its end). The backward starts from them.
 * workspace: wbmm_scan_forward_workspace_bytes(...) bytes, 16-byte aligned (NULL when 0; needed only
 *           where few columns make the axis run in segments). Calls that share one must be ordered
 *           on one stream.
 * An infinity in h0 or u makes h from there on, in its own column, infinite or NaN (the runs of
 * steps are joined by products of their a_t, which may underflow to 0: NaN where a product with the
 * infinity would be one). Gates: a_t and 1 - a_t are held at 1.6e-38 from below; a NaN in g or u is
 * a NaN in h from there on.
 * No atomics: bitwise reproducible. Errors: WBMM_E_INVALID (sizes, dtype, n_lens, NULL or
 * overlapping buffers), WBMM_E_UNSUPPORTED (outer * inner >= 2^26, len > 2^30, more than 2^38
 * elements, misaligned pointer), WBMM_E_WORKSPACE, WBMM_E_HIP.
 */
#define WBMM_SCAN_CHUNK 32
size_t wbmm_scan_forward_workspace_bytes(int64_t outer, int64_t len, int64_t inner);
wbmm_status wbmm_scan_forward(int64_t outer, int64_t len, int64_t inner, int dtype, int reverse,
                              const void* g, const void* u, const float* h0, const int32_t* lens,
                              int64_t n_lens, void* h, float* h_last, float* states,
                              void* workspace, size_t workspace_bytes, void* stream);

/*
 * wbmm_scan_backward_workspace_bytes / wbmm_scan_backward — gradients of wbmm_scan_forward, from the last step to the first:
 *   G_t = dh_t + a_{t+1} G_{t+1}   (dh_last in place of a_n G_n at the last step),
 *   du_t = (1 - a_t) G_t,   dg_t = a_t (1 - a_t) (h_{t-1} - u_t) G_t,   dh0 = a_0 G_0
 * (dh0 = dh_last for an empty sequence). The h_{t-1} are run again from `states`, in fp32.
 * g, reverse, lens, sizes: as in the forward.
 * u:        the forward's u, or its checkpoint's codes when u_scales is given (u_fmt: the
 *           checkpoint's format; ignored without u_scales).
 *           A checkpoint's groups run through the whole tensor: with lens, the padding that was
 *           packed has to be finite, or its group's other values read back as NaN.
 * states:   as the forward wrote them, or NULL: the call then runs the recurrence for them first,
 *           on the u that it is given, from h0 (device fp32 [outer][inner], or NULL for zeros; NULL
 *           with states), into its workspace, reading g and u a second time. With a checkpointed u
 *           and the forward's states, each run of WBMM_SCAN_CHUNK steps starts from the state of
 *           the forward's own u.
 * dh:       device map in dtype. dh_last: device fp32 [outer][inner], the gradient of h_last, or
 *           NULL for zeros.
 * dg, du:   device maps in dtype, written; 0 past the end of a sequence. dh0: device fp32
 *           [outer][inner], written, or NULL.
 * workspace: wbmm_scan_backward_workspace_bytes(...) bytes, 16-byte aligned (NULL when 0).
 * Infinities and NaN as in the forward: those of dh and dh_last reach the earlier steps' dg, du and
 * dh0, those of the state only dg.
 * Errors as in the forward; also WBMM_E_INVALID for an unknown u_fmt, or h0 beside states.
 */
size_t wbmm_scan_backward_workspace_bytes(int64_t outer, int64_t len, int64_t inner,
                                          int has_states);
wbmm_status wbmm_scan_backward(int64_t outer, int64_t len, int64_t inner, int dtype, int reverse,
                               int u_fmt, const void* g, const void* u, const uint8_t* u_scales,
                               const float* states, const float* h0, const void* dh,
                               const float* dh_last, const int32_t* lens, int64_t n_lens, void* dg,
                               void* du, float* dh0, void* workspace, size_t workspace_bytes,
                               void* stream);

/*
 * wbmm_rmsnorm_forward — root-mean-square norm along one axis with the residual's addition in front:
 * what stands before a mixer. Tensors are dense (outer, len, inner) and normed over len, for every
 * (outer, inner): the channels of a map are (B, C, H W) in NCHW, (B H W, C, 1) in NHWC.
 *   t = x + residual,   y = t weight / sqrt(mean_len(t^2) + eps).
 * t is formed in fp32 and normed as it is, its squares summed and y's products formed in fp64; s and y are
 * rounded once (RNE; a bf16 y by way of fp32). An infinity or NaN in t reaches its own (outer, inner) only,
 * one in a weight its own entries only.
 * dtype:    of x, residual, s and y: WBMM_F32 or WBMM_BF16.
 * residual: device tensor, or NULL. weight: device fp32 [len], or NULL for ones.
 * s:        device tensor, t in dtype (what the backward takes), or NULL. May be x or residual itself.
 * y:        device tensor, written.
 * codes, scales: the checkpoint of y in `fmt`, exactly what wbmm_ckpt_pack makes of it (n bytes and
 *           ceil(n / WBMM_CKPT_GROUP) bytes), or both NULL (fmt ignored). In the same launch where the
 *           groups do not run across rows (len a multiple of 32 at inner = 1, or inner a multiple of 32)
 *           and addresses are aligned to 16 bytes (codes to 8), else by a second launch over y.
 * Any pointer alignment down to the element works. No workspace, no atomics: bitwise reproducible.
 * Errors: WBMM_E_INVALID (sizes, dtype, fmt, eps, NULL or overlapping buffers), WBMM_E_UNSUPPORTED (len >
 * 2^20, outer * inner > 2^25 (2^23 for inner = 1 and len > 1536), more than 2^35 elements, misaligned
 * pointer), WBMM_E_HIP.
 */
wbmm_status wbmm_rmsnorm_forward(int64_t outer, int64_t len, int64_t inner, int dtype, float eps,
                                 const void* x, const void* residual, const float* weight, void* s,
                                 void* y, int fmt, uint8_t* codes, uint8_t* scales, void* stream);

/*
 * wbmm_rmsnorm_backward_workspace_bytes / wbmm_rmsnorm_backward — gradients of wbmm_rmsnorm_forward at
 * the sum that it stored:
 *   r = 1 / sqrt(mean(s^2) + eps),   h = s r,
 *   dx = ds + r (weight dy - h mean(weight dy h)),   dweight = sum over (outer, inner) of dy h.
 * The two sums over len and r are fp64, so that s may be as large or as small as fp32 goes, as in the
 * forward; weight dy, h and the mean are fp32.
 * s:       the forward's s (its x where there was no residual). dy: gradient of y.
 * ds:      gradient of s from elsewhere (the residual's further way), or NULL for zeros.
 * dx:      device tensor in dtype, the gradient of x and of residual alike, or NULL to skip.
 * dweight: device fp32 [len], or NULL to skip. Summed in fp64 in a fixed order.
 * workspace: wbmm_rmsnorm_backward_workspace_bytes(...) bytes, 16-byte aligned; not needed without
 *          dweight. Calls that share one must be ordered on one stream.
 * Errors as in the forward, and WBMM_E_WORKSPACE.
 */
size_t wbmm_rmsnorm_backward_workspace_bytes(int64_t outer, int64_t len, int64_t inner);
wbmm_status wbmm_rmsnorm_backward(int64_t outer, int64_t len, int64_t inner, int dtype, float eps,
                                  const void* s, const float* weight, const void* dy,
                                  const void* ds, void* dx, float* dweight, void* workspace,
                                  size_t workspace_bytes, void* stream);

/*
 * wbmm_adamw_plan / wbmm_adamw_step — one AdamW step over all parameters of a model in one launch, from
 * the gradients that the backward calls write. For every element, with t the step's number:
 *   g = grad_factor grad,   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2,
 *   p = (1 - lr wd) p - lr / (1 - beta1^t) m / (sqrt(v) / sqrt(1 - beta2^t) + eps).
 * Everything is fp32 and rounded operation by operation; the factors of lr, beta and t are formed in
 * fp64 and rounded once.
 * A wbmm_adamw_tensor is one parameter, dense, all pointers to device memory:
 *   p:        fp32, updated. g: fp32 or bf16 (g_dtype), read. n: elements. weight_decay: wd.
 *   m, v:     fp32, updated; or, with m_scales and v_scales, 8-bit states: m and the root of v as
 *             checkpoints in WBMM_CKPT_E4M3 (n code bytes and ceil(n / WBMM_CKPT_GROUP) scale bytes each;
 *             all zero bytes are zero states). They are read as wbmm_ckpt_unpack gives them. What is
 *             stored is rounded to one of the two neighbouring code values at random, to the value
 *             itself on average; but a root above zero never to 0: one below the least code, 2^-17 of its
 *             group's largest, is held at that code until the group's scale falls. v, the root's square, moves
 *             further than unrounded, on average, as the root's variance joins it: by up to 1/16 where the
 *             codes are normal (roots from 2^-13 of their group's largest on, at least), by 1 / (2 n) at the
 *             n-th of the 8 least. Random words are Philox 4x32 with 7 rounds, counter (index / 4 as 64
 *             bits, tensor, t), key `seed`, word index % 4, its low 16 bits for m and its high ones for the
 *             root. A group that holds an infinity or a NaN becomes NaN, as in wbmm_ckpt_pack.
 *   p_bf16:   a copy of p in bf16 (RNE), written, or NULL: what a bf16 forward reads.
 * wbmm_adamw_plan checks `count` such tensors and lays out a table for them in HOST memory (table_bytes
 *   at least wbmm_adamw_plan_bytes(...), 8-byte aligned); the caller copies it to the device and keeps
 *   both it and the tensors where they are. *chunks is what the step wants back. No GPU work.
 *   Overlapping buffers are refused, two gradients aside.
 * wbmm_adamw_step: table: the device copy, 8-byte aligned; count, chunks: the plan's (a table of other
 *   counts is left alone: nothing is written).
 *   step:     t, from 1 to 2^31 - 1; with step_dev, a device int32 read by the kernel, `step` is ignored
 *             (a captured graph counts on the device; it must hold at least 1).
 *   lr_factor, grad_factor: device fp32 that lr and the gradients are multiplied by, or NULL.
 * 1 <= t; 0 <= beta < 1; eps >= 0. Any alignment down to the element works; 16 bytes (codes 8) takes the
 * wide accesses. Bitwise reproducible, and the same for any alignment.
 * Errors: WBMM_E_INVALID, WBMM_E_UNSUPPORTED (more than 2^36 elements, misaligned pointers),
 * WBMM_E_WORKSPACE (table too small), WBMM_E_HIP.
 */
typedef struct wbmm_adamw_tensor {
  float* p;
  const void* g;
  void* m;
  void* v;
  uint8_t* m_scales;
  uint8_t* v_scales;
  uint16_t* p_bf16;
  int64_t n;
  double weight_decay;
  int32_t g_dtype;
  int32_t reserved;
} wbmm_adamw_tensor;
size_t wbmm_adamw_plan_bytes(const wbmm_adamw_tensor* tensors, int64_t count);
wbmm_status wbmm_adamw_plan(const wbmm_adamw_tensor* tensors, int64_t count, void* table,
                            size_t table_bytes, int64_t* chunks);
wbmm_status wbmm_adamw_step(const void* table, int64_t count, int64_t chunks, double lr,
                            double beta1, double beta2, double eps, int64_t step,
                            const int32_t* step_dev, const float* lr_factor,
                            const float* grad_factor, uint64_t seed, void* stream);

/*
 * wbmm_delta_forward_workspace_bytes / wbmm_delta_forward — gated delta rule: the recurrence beside
 * wbmm_scan_forward whose state is a matrix S (dk x dv) per head, for long sequences, maps in raster
 * order (a map in NHWC is (B, H W, heads, channels of a head) as it lies) and single steps:
 *   a_t = sigmoid(g_t),   b_t = sigmoid(beta_t),
 *   S_t = a_t (I - b_t k_t k_t^T) S_{t-1} + b_t k_t v_t^T,   o_t = scale S_t^T q_t,   S_{-1} = s0.
 * Keys are taken as they are; the rule contracts for |k| <= 1 (wbmm_rmsnorm_forward over a key's entries,
 * with weights of dk^-1/2, gives length 1).
 * Sizes:    B, L, Hk, H >= 1, Hk dividing H; 1 <= dk, dv <= 128.
 * dtype:    of q, k, v, g, beta and o: WBMM_F32 or WBMM_BF16. Sums and the state are fp32, products good
 *           to 2^-24 of their factors. A bf16 call gives what the fp32 call of the same values gives,
 *           rounded (RNE).
 * reverse:  nonzero: sequences run from their last position to their first.
 * q, k:     device [B][L][Hk][dk]; head h uses key head h / (H / Hk). v: device [B][L][H][dv].
 * g, beta:  device [B][L][H]. g is held to [-87, 87].
 * s0:       device fp32 [B][H][dk][dv], or NULL for zeros.
 * lens:     device int32 [B], or NULL: sequence b has lens[b] positions, held to [0, L]. Positions past
 *           it are not used, whatever they hold, and o is 0 there; a reversed sequence starts at its own
 *           last position.
 * o:        device [B][L][H][dv], written.
 * s_last:   device fp32 [B][H][dk][dv], or NULL: the state after the last step (s0 for an empty
 *           sequence). May be s0 itself (updated in place).
 * states:   device fp32 [B][H][ceil(L / WBMM_DELTA_CHUNK)][dk][dv], or NULL: the state before steps 0,
 *           WBMM_DELTA_CHUNK, ... in the order the sequence runs (its last state past its end).
 * workspace: wbmm_delta_forward_workspace_bytes(...) bytes, 16-byte aligned (NULL when 0: up to 8
 *           steps). Calls that share one must be ordered on one stream.
 * An infinity or NaN in q reaches its own o; one in k, v or the state, and a NaN in g or beta (infinite ones are
 * gates as any other), makes o of the head NaN from the chunk of WBMM_DELTA_CHUNK steps on that it lies in
 * (in v and in a column of the state: in its own column). fp32 numbers that bf16 has no finite value for
 * (3.39e38 and more) may count as infinite. No atomics: bitwise reproducible.
 * Errors: WBMM_E_INVALID (sizes, dtype, scale, NULL or overlapping buffers), WBMM_E_UNSUPPORTED (dk or dv >
 * 128, Hk dk or H dv > 2^22, more than 2^22 chunks over all heads, L > 2^28, misaligned pointer),
 * WBMM_E_WORKSPACE, WBMM_E_HIP.
 */
#define WBMM_DELTA_CHUNK 64
size_t wbmm_delta_forward_workspace_bytes(int64_t B, int64_t L, int Hk, int H, int dk, int dv,
                                          int dtype);
wbmm_status wbmm_delta_forward(int64_t B, int64_t L, int Hk, int H, int dk, int dv, int dtype,
                               int reverse, float scale, const void* q, const void* k,
                               const void* v, const void* g, const void* beta, const float* s0,
                               const int32_t* lens, void* o, float* s_last, float* states,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * wbmm_delta_backward_workspace_bytes / wbmm_delta_backward — gradients of wbmm_delta_forward. With D_t
 * the gradient of S_t (D of the last step has ds_last added), e_t = v_t - a_t S_{t-1}^T k_t:
 *   D_t += scale q_t do_t^T,   dq_t = scale S_t do_t,   dv_t = b_t D_t^T k_t,
 *   dk_t = b_t (D_t e_t - a_t S_{t-1} D_t^T k_t),   D_{t-1} = a_t (I - b_t k_t k_t^T) D_t,
 *   db_t = (D_t^T k_t) . e_t,   da_t = <(I - b_t k_t k_t^T) S_{t-1}, D_t>,   ds0 = D_{-1},
 * dg and dbeta through the sigmoids. dq and dk of a shared key head are the sums over its heads, in order.
 * q, k, v, g, beta, lens, reverse, scale, sizes: as in the forward.
 * states:   as the forward wrote them, or NULL: the call then forms them first, from s0 (device fp32
 *           [B][H][dk][dv], or NULL for zeros; NULL with states), in its workspace.
 * dout:     device [B][L][H][dv], gradient of o. ds_last: device fp32 [B][H][dk][dv], gradient of s_last,
 *           or NULL for zeros.
 * dq, dk, dv, dg, dbeta: device tensors in dtype, written; 0 past the end of a sequence. ds0: device fp32
 *           [B][H][dk][dv], written, or NULL; may be ds_last itself.
 * workspace: wbmm_delta_backward_workspace_bytes(...) bytes, 16-byte aligned.
 * An infinity or NaN makes the gradients of its head NaN where they depend on it, in whole chunks (g and
 * beta: a NaN). dg is (1 - a) times a sum over a chunk's steps, good to the last bits of its largest terms:
 * where a gate forgets nearly everything (g below -10) the sum itself may be smaller than those.
 * Errors as in the forward; also WBMM_E_INVALID for s0 beside states.
 */
size_t wbmm_delta_backward_workspace_bytes(int64_t B, int64_t L, int Hk, int H, int dk, int dv,
                                           int dtype, int has_states);
wbmm_status wbmm_delta_backward(int64_t B, int64_t L, int Hk, int H, int dk, int dv, int dtype,
                                int reverse, float scale, const void* q, const void* k,
                                const void* v, const void* g, const void* beta,
                                const float* states, const float* s0, const void* dout,
                                const float* ds_last, const int32_t* lens, void* dq, void* dkey,
                                void* dval, void* dg, void* dbeta, float* ds0, void* workspace,
                                size_t workspace_bytes, void* stream);

/*
 * wbmm_probe_mfma — measurement aid, not part of the method: a matrix-core peak probe. Launches
 * `blocks` workgroups of 4 waves; every wave runs `iters` rounds of 8 independent MFMA
 * accumulation chains on register operands (dtype WBMM_F32: v_mfma_f32_16x16x4f32, WBMM_BF16:
 * v_mfma_f32_16x16x32_bf16) and writes one float per lane to out (device, blocks * 256 floats),
 * so the sustained matrix rate on this part and clock can be set beside the datasheet peak.
 * wbmm_probe_mfma_flops returns the flops of such a launch (0 for invalid arguments).
 * wbmm_set_launch_events attaches to it like to the main kernel of the other calls.
 * Errors: WBMM_E_INVALID (dtype, blocks or iters < 1, NULL or misaligned out), WBMM_E_HIP.
 */
double wbmm_probe_mfma_flops(int dtype, int blocks, int iters);
wbmm_status wbmm_probe_mfma(int dtype, int blocks, int iters, float* out, void* stream);

/*
 * wbmm_set_launch_events — measurement aid, not part of the method. The next wbmm_forward,
 * wbmm_backward (or their _hier, _shifted, _bf16 and _ckpt forms), wbmm_dwconv_forward or wbmm_probe_mfma
 * call made on the calling thread
 * attaches `before` and `after` (hipEvent_t
 * handles passed as void*) to the dispatch of its main contraction kernel (hipExtLaunchKernel's
 * start and stop events), so their elapsed time is that kernel's execution; the pair is then
 * cleared. Both NULL clears a pending pair. The caller owns the events. Errors: WBMM_E_INVALID
 * when exactly one of the two is NULL.
 */
wbmm_status wbmm_set_launch_events(void* before, void* after);

#ifdef __cplusplus
}
#endif

#endif /* WBMM_H */
