/*
 * seam_blend.h -- C ABI of the MI355X (gfx950) tiled-VAE decode-assembly library.
 *
 * Two operations, each behind one entry point:
 *
 *  vae_tile_blend_stitch  -- crossfade overlapping decoded tiles along rows
 *      (blend_v), columns (blend_h) and frames (blend_t), crop every tile to the
 *      row limit and stitch the result into one output, written once.
 *      Defined by: diffusers issue "[Proposal] Vectorize tiled VAE blending
 *      while preserving rounding and CUDA graph replay", section "Proposed
 *      scope" (blend_v / blend_h / blend_t; extent clamping from diffusers
 *      #2660; in-place output; per-product rounding; coefficients from float64
 *      division).
 *
 *  patch_groupnorm -- GroupNorm of a tensor viewed as spatial patches: per-patch
 *      (count, mean, M2) statistics merged with Chan's formula so that the
 *      result equals unsplit GroupNorm (global mean, variance divided by the
 *      count).  Defined by: DistVAE PR "Add tiled VAE parallelism & extended
 *      model support", the PatchGroupNorm commits and the Patchify commit
 *      (first patches one band longer).
 *
 *
 * Beside them, operators of the transformer over latent tokens that makes the
 * latents those tiles are decoded from: layer norm (forward and backward),
 * rotary position embedding, and the gradient norm with clipping.
 *
 * Conventions shared by every entry point
 *  - Pointers named "device" are HIP device pointers (any device memory the
 *    current device can read/write); everything else is host memory read
 *    during the call only.  The caller owns and allocates every buffer.  The
 *    library allocates no device memory, never synchronises the stream and
 *    keeps no state other than a thread-local error message.
 *  - All work is enqueued on `stream` (a hipStream_t; NULL = the null stream),
 *    on the device that is current when the call is made.  Results are ready
 *    when the stream reaches that point.
 *  - Return value: 0 on success, or a negative SB_E* code; the message is then
 *    available from seamblend_last_error().  Argument and geometry errors are
 *    detected on the host before anything is enqueued.  Faults during
 *    execution surface asynchronously on the stream, as for any HIP kernel.
 *  - Tensors are dense, contiguous, row-major (last index fastest), except
 *    where an entry point takes strides.
 *  - What a call writes (outputs, workspace) overlaps nothing else that it reads
 *    or writes, except where an entry point says so; what is checked of that is
 *    said there.
 */
#ifndef SEAM_BLEND_H
#define SEAM_BLEND_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* storage dtype of every tile / tensor in one call */
typedef enum { SB_F32 = 0, SB_F16 = 1, SB_BF16 = 2 } sb_dtype;

/* return codes */
#define SB_OK 0
#define SB_EARG (-1)       /* bad argument: null pointer, unknown dtype, bad rank ... */
#define SB_EGEOM (-2)      /* geometry outside what the data-parallel kernel supports */
#define SB_EWORKSPACE (-3) /* workspace smaller than patch_groupnorm_workspace_bytes() */
#define SB_ELAUNCH (-4)    /* the HIP runtime rejected a launch (message from hipGetErrorString) */

/*
 * Output extents of vae_tile_blend_stitch for a tile grid, after the same
 * validation the entry point performs (host only, no device work).
 *   grid[6]        {ndim (4 or 5), N, C, n_t, n_h, n_w}; n_t must be 1 when ndim == 4.
 *   tile_extents   n_t + n_h + n_w entries: t_0..t_{n_t-1}, h_0.., w_0..
 *                  (t_0 must be 1 when ndim == 4).
 *   blend_extent   {E_t, E_h, E_w} >= 0; E_t is ignored when ndim == 4.
 *   row_limit      {R_t, R_h, R_w} >= 1: stride between tile origins along
 *                  each axis, and the crop of every tile but the last.
 *   out_extents    receives {L_t, L_h, L_w}, L = (n - 1) * R + (last extent).
 * Geometry preconditions (else SB_EGEOM): every non-last tile is >= R long;
 * with e(k) = min(E, ext(k-1), ext(k)) the blend extent between tiles k-1 and
 * k (e(0) = 0), every tile satisfies ext(k) >= e(k) + e(k+1), so a tile's head
 * seam and tail never overlap; at most 64 tiles per axis; output planes and
 * tiles below 2^31 elements per (n, c) plane.
 */
int vae_tile_blend_stitch_output_extents(const int64_t grid[6], const int64_t *tile_extents,
                                         const int64_t blend_extent[3],
                                         const int64_t row_limit[3], int64_t out_extents[3]);

/*
 * Blend + crop + stitch of a tile grid into `out`.
 *   tiles        host array of n_t*n_h*n_w device pointers in raster order
 *                (tau, i, j): tile (tau, i, j) is a contiguous
 *                [N, C, t_tau, h_i, w_j] array (ndim 5) or [N, C, h_i, w_j]
 *                (ndim 4) of `dtype`.  Tiles are only read.
 *   grid, tile_extents, blend_extent, row_limit: as above.
 *   dtype        SB_F32, SB_F16 or SB_BF16 (tiles and output alike).
 *   out          device pointer to a contiguous [N, C, L_t, L_h, L_w] (ndim 5)
 *                or [N, C, L_h, L_w] (ndim 4) array of `dtype`; must not
 *                overlap any tile (checked, SB_EARG).
 *   stream       hipStream_t or NULL.
 * Result: for each temporal tile, tiles are blended in raster order, row seam
 * (with the tile above, as already blended) before column seam (with the tile
 * to the left, as already blended), each seam element
 *   RN_T( RN_T(a * w_a[k]) + RN_T(b * w_b[k]) ),  w_b[k] = fp32(k/e),
 *   w_a[k] = fp32(1 - k/e) from double, products and sum in fp32 without
 *   fusion;
 * every tile is cropped to R except the last along each axis; then each
 * stitched temporal chunk is blended with the previous stitched chunk (as
 * already blended) along frames and cropped.  Bit-exact for every dtype.
 * Each output element is written exactly once; no scratch memory.
 * N*C == 0 is a no-op that accepts null tile and output pointers.
 * Limits (SB_EGEOM beyond them, before any launch): clamped blend extents up
 * to 4096; a launch window takes at most 192 tile pointers, a window's tile
 * rows with the row above and its temporal tiles with the one before, so up
 * to 48 tile columns always fit and more may be refused when there are several
 * tile rows or temporal tiles; when every W seam and crop is narrower than 16
 * vectors (the narrow-seam layout) a launch window of more than 2^24 - 1
 * output frames is refused; otherwise any frame count is taken, in several
 * launches.
 */
int vae_tile_blend_stitch(const void *const *tiles, const int64_t grid[6],
                          const int64_t *tile_extents, const int64_t blend_extent[3],
                          const int64_t row_limit[3], int dtype, void *out, void *stream);

/*
 * Device workspace (bytes) patch_groupnorm needs for this problem; 0 with an
 * error message for invalid arguments.  shape: ndim entries {N, C, spatial..}.
 */
size_t patch_groupnorm_workspace_bytes(int ndim, const int64_t *shape, int64_t groups,
                                       int split_axis, int64_t n_patches);

/*
 * GroupNorm of x viewed as n_patches patches along split_axis.
 *   x            device pointer, contiguous [N, C, spatial...] of dtype, ndim 3..5.
 *   shape        host array of ndim extents; C % groups == 0; N*C < 2^31,
 *                each group (C/G * spatial elements) < 2^31 elements and the
 *                tensor < 2^56 bytes (else SB_EGEOM).
 *   split_axis   2 <= split_axis < ndim: the spatial axis the patches cut.
 *   n_patches    1..64.  Patch p covers [s_p, s_p + len_p) along split_axis
 *                with the first (L mod P) patches one longer (empty patches
 *                allowed when P > L).
 *   eps          added to the variance (fp32), >= 0.
 *   gamma, beta  device pointers to [C] of dtype, or NULL (1 and 0).
 *   out          device pointer like x; may be x itself (in place).
 *   workspace    device scratch of at least patch_groupnorm_workspace_bytes(),
 *                16-byte aligned; caller-owned, contents need not be initialised.
 *   patch_stats  optional device pointer to N*G*P*3 floats, or NULL: receives
 *                per-patch (count, mean, M2), M2 = sum of squared deviations
 *                about the patch mean, merged in fp32 over that patch's chunks;
 *                (0, 0, 0) for an empty patch.
 *   stream       hipStream_t or NULL.
 * Result: per (n, g), mean and M2 over the C/G channels and all spatial
 * positions, obtained by merging fp32 partial statistics in a fixed order:
 * count, mean = sum n_k mean_k / count, M2 = sum (M2_k + n_k (mean_k -
 * mean)^2) over the partials (Chan's merge taken over many sets at once);
 * var = M2 / count; rstd = 1/sqrt(var+eps);
 * y = (x - mean) * rstd * gamma_c + beta_c in fp32, rounded once to dtype.
 * Each thread folds its values into (count, mean, M2) a batch at a time: the
 * batch's mean and squared deviations by two passes, then a Chan merge
 * (Welford's update), so M2 is never a difference of power sums.  Statistics
 * are taken about a shift K_g (the median of five of the group's elements,
 * spread over it), so the mean is carried as K_g + m and x - mean is formed as
 * (x - K_g) - m: inputs whose mean is large against their spread keep full
 * fp32 accuracy, and up to two outlying samples never become the shift.
 * Deterministic: the same inputs give the same bits on every call.
 */
int patch_groupnorm(const void *x, int ndim, const int64_t *shape, int64_t groups,
                    int split_axis, int64_t n_patches, float eps, const void *gamma,
                    const void *beta, int dtype, void *out, void *workspace,
                    size_t workspace_bytes, float *patch_stats, void *stream);

/*
 * patch_groupnorm for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * the same computation, kernels and results, with the statistics partials in
 * a static scratch array the library holds on each GPU instead of a
 * caller-given workspace.  The caller still passes x, out (and gamma, beta,
 * patch_stats).  Allocates nothing and calls no allocating routine; its first
 * call on a device looks the array's device address up once.
 *   Limit: problems whose partials exceed SB_GN_STATIC_SCRATCH_BYTES
 *   (patch_groupnorm_workspace_bytes() > 1 MiB, i.e. N*groups*patches*chunks
 *   above 65536) return SB_EWORKSPACE before anything is enqueued.
 *   Every call on one GPU shares that GPU's array: calls that overlap on one
 *   GPU (for example on two streams) race and must be ordered by the caller.
 * Arguments, layout and errors otherwise as patch_groupnorm.
 */
#define SB_GN_STATIC_SCRATCH_BYTES (1u << 20)
int patch_groupnorm_noalloc(const void *x, int ndim, const int64_t *shape, int64_t groups,
                            int split_axis, int64_t n_patches, float eps, const void *gamma,
                            const void *beta, int dtype, void *out, float *patch_stats,
                            void *stream);

/*
 * Normalised-ramp blend of wide tiles (unsloth Studio PR "size seam-free VAE
 * tiles from measured peaks", the Qwen-Image-2.1 wide-tile commit, which
 * the later commits extend to every image VAE and to the tiled encode).
 * A tile has no weight within `margin` positions of an edge it shares with
 * another tile (an edge inside the canvas) and ramps linearly to full weight
 * over the next `ramp`: at whole distance d from such an edge the factor is
 * clamp((d - margin) / ramp, 0, 1); a tile's weight along an axis is the
 * product of its two edges' factors and its 2-D weight the product of its
 * axes'.  Weights are normalised to 1 at every position; the sum of weight
 * times value is accumulated in fp32 and rounded once to the storage type.
 *   tiles:        n_h * n_w device pointers, raster order (i, j); tile (i, j) is a
 *                 contiguous [N, C, (T,) h_i, w_j] array of dtype (frames are not tiled).
 *   grid:         {ndim (4 | 5), N, C, 1, n_h, n_w}, n_h and n_w in 1..48.
 *   tile_origins: 1 + n_h + n_w positions: 0 (frames), then the row origins, then the
 *                 column origins; each axis starts at 0 and increases.
 *   tile_extents: 1 + n_h + n_w extents: T (1 when ndim == 4), then h_i, then w_j.  The
 *                 canvas along an axis ends where its last tile ends (< 2^20).
 *   margin, ramp: per axis (t, h, w) in positions; [0] is ignored; margin >= 0, ramp >= 1.
 *   out:          contiguous [N, C, (T,) L_h, L_w] of dtype; must not overlap a tile.
 * Every position needs a tile with weight (overlaps wider than twice the margin),
 * and at most 4 tiles may carry weight at one position of an axis: else SB_EGEOM.
 * Enqueued on `stream`; allocates nothing; N * C == 0 is a no-op.
 */
int vae_tile_ramp_blend(const void *const *tiles, const int64_t grid[6], const int64_t *tile_origins,
                        const int64_t *tile_extents, const int64_t margin[3], const int64_t ramp[3],
                        int dtype, void *out, void *stream);

/*
 * Tile layout along one axis of a canvas of L latents (host only): writes the
 * origin and extent of each tile and their count.  Defined by the unsloth
 * Studio PR "size seam-free VAE tiles from measured peaks", sections "Problem"
 * and "Change" and its commit log (stock tiles with edge slivers; 32-latent
 * tiles with at least 16-latent overlaps spread evenly so the last ends at the
 * edge at full size; a canvas within one tile is one tile; at a sliver, the
 * fewest decoder calls, then the widest tile, decoding no more latents per
 * side than the stock loop; the earlier fewest tiles of the smallest side).
 *   rule / params:
 *     SB_LAYOUT_STOCK          {T, S}: a tile of T at every multiple of S below L,
 *                              the last cut short by the edge.
 *     SB_LAYOUT_EDGE_ALIGNED   {t, ov}: the fewest tiles of side t whose neighbours
 *                              overlap by >= ov, origin_k = floor(k (L - t) / (n - 1));
 *                              one tile of L when L <= t (whatever ov: a single tile
 *                              has no neighbour); otherwise ov < t (SB_EARG).
 *     SB_LAYOUT_FEWEST_CALLS   {T, S, ov, M}: the fewest tiles, then the widest side
 *                              t <= M, with n * t <= B, the latents the stock (T, S) loop
 *                              decodes along the axis, and overlaps >= ov; spread evenly.
 *                              Up to rounding: when no whole side fits B but the exact
 *                              covering does (L + (n - 1) ov <= B), the smallest covering
 *                              side is taken.
 *     SB_LAYOUT_SMALLEST_SIDE  {ov, M}: the fewest tiles of side <= M covering with
 *                              overlaps >= ov, then the smallest such side; spread evenly.
 *     SB_LAYOUT_AUTO           {T, S, floor_tile, floor_overlap}: the stock tiles when
 *                              every one is >= floor_tile and every overlap >=
 *                              floor_overlap, else EDGE_ALIGNED with
 *                              t = max(floor_tile, T), ov = max(floor_overlap, T - S).
 *   max_tiles: capacity of origins[] and extents[] (SB_EARG if exceeded).
 * Returns 0, SB_EARG for bad parameters, SB_EGEOM if no layout satisfies the rule.
 */
typedef enum {
  SB_LAYOUT_STOCK = 0,
  SB_LAYOUT_EDGE_ALIGNED = 1,
  SB_LAYOUT_FEWEST_CALLS = 2,
  SB_LAYOUT_SMALLEST_SIDE = 3,
  SB_LAYOUT_AUTO = 4
} sb_layout_rule;

int vae_tile_layout(int64_t L, int rule, const int64_t params[4], int64_t max_tiles,
                    int64_t *origins, int64_t *extents, int64_t *n_tiles);

/*
 * Layer norm of rows of D elements (the transformer over latent tokens):
 *   m = sum x / D, v = sum (x - m)^2 / D, r = 1 / sqrt(v + eps),
 *   out = (x - m) r gamma + beta.
 *   shape        {outer, inner, D}: outer * inner rows (< 2^31), D in 1..2^28.
 *   *_stride     {outer, inner} strides in elements, 0..2^40; the D elements of a
 *                row are contiguous.  Views of a packed projection need no copy.
 *   gamma, beta  device pointers to [D] of weight_dtype, or NULL (1 and 0).
 *   dtype        of x and out; weight_dtype: dtype, or SB_F32.
 *   out          each element held once; x itself (same pointer and strides), or
 *                sharing no element with it (checked; SB_EARG).
 *   workspace    caller-owned device scratch of layer_norm_forward_workspace_bytes()
 *                bytes, 16-byte aligned; not looked at where that is 0 (rows of
 *                up to 64 KiB).
 * Any element alignment is taken; 16-byte aligned rows are fastest.  Statistics
 * are fp32 and corrected two-pass (sums about a first mean, then its rounding
 * error taken out), so a mean that is large against the spread costs no
 * accuracy; one rounding to dtype.  Deterministic.  No rows: no-op.
 */
int layer_norm_forward(const void *x, const int64_t x_stride[2], const int64_t shape[3], float eps,
                       const void *gamma, const void *beta, int dtype, int weight_dtype, void *out,
                       const int64_t out_stride[2], void *workspace, size_t workspace_bytes, void *stream);

/* Device workspace (bytes) layer_norm_forward needs: 0 for rows of up to 64
 * KiB; (size_t)-1 with an error message for invalid arguments. */
size_t layer_norm_forward_workspace_bytes(const int64_t shape[3], int dtype);

/* Device workspace (bytes) layer_norm_backward needs; 0 with an error message
 * for invalid arguments. */
size_t layer_norm_backward_workspace_bytes(const int64_t shape[3], int dtype);

/*
 * Gradient of layer_norm_forward: with h = (x - m) r and g = dy gamma,
 *   dx = r (g - mean(g) - h mean(g h)),
 *   dgamma = sum over rows of dy h,  dbeta = sum over rows of dy.
 * The statistics are formed again from x: nothing is kept from the forward
 * pass.  dy, x, dx: rows as above; dx may be dy or x themselves, else it
 * shares no element with them.  gamma: NULL for 1.  dgamma, dbeta: device
 * pointers to [D] of weight_dtype, or NULL where not wanted; they are written,
 * not added to (zeros without rows).  workspace: caller-owned device scratch,
 * 16-byte aligned, contents need not be initialised.  Sums over rows are fp32
 * in a fixed order.
 */
int layer_norm_backward(const void *dy, const int64_t dy_stride[2], const void *x, const int64_t x_stride[2],
                        const int64_t shape[3], float eps, const void *gamma, int dtype, int weight_dtype,
                        void *dx, const int64_t dx_stride[2], void *dgamma, void *dbeta, void *workspace,
                        size_t workspace_bytes, void *stream);

/* which elements of a head's rotated part make pair i of n */
#define SB_ROTARY_HALF 0        /* i and i + n */
#define SB_ROTARY_INTERLEAVED 1 /* 2i and 2i + 1 */

/*
 * Rotary position embedding of query heads and, in the same launch, key heads:
 * pair i of every head of token t turns by a = position * freqs[i],
 *   (u, v) -> scale (u cos a - v sin a, u sin a + v cos a),
 * and the head's elements from rot_dim on are copied.  transpose != 0 turns by
 * -a: the gradient of the forward call.
 *   q, k         device tensors [B, T, heads, D]; q_heads or k_heads may be 0
 *                (then its pointers and strides are not read).
 *   shape        {B, T, D}: B * T < 2^31, D <= 2^13, at most 2^12 heads each.
 *   *_stride     {B, T, head} strides in elements, 0..2^40; D is contiguous.
 *   *_out        each element held once; q_out is q itself or shares no element
 *                with q (k alike), and no output one with the other tensor's
 *                input or output (SB_EARG).  Views of one packed projection are
 *                told apart exactly; tensors of unlike strides whose memory
 *                interleaves are refused.
 *   freqs        device pointer to rot_dim / 2 doubles: radians per position.
 *   positions    device pointer to 4- or 8-byte signed integers, strides
 *                {axis, B, T} in elements, 0..2^40 (0 broadcasts).
 *   sections     n_sections (1..4) pair counts that add up to rot_dim / 2:
 *                consecutive pairs turn by the positions of axis 0, 1, ...
 * The angle is formed and reduced in 64 bits, cosine and sine in fp32, one
 * rounding to dtype.  No tokens or no heads: no-op.
 */
int rotary_apply(const void *q, const int64_t q_stride[3], void *q_out, const int64_t q_out_stride[3],
                 int64_t q_heads, const void *k, const int64_t k_stride[3], void *k_out,
                 const int64_t k_out_stride[3], int64_t k_heads, const int64_t shape[3], int dtype,
                 const double *freqs, int64_t rot_dim, int layout, const void *positions, int position_bytes,
                 const int64_t position_stride[3], const int64_t *sections, int n_sections, float scale,
                 int transpose, void *stream);

/* Device workspace (bytes) of grad_norm and grad_norm_clip for n tensors of
 * these element counts; 0 with an error message for invalid arguments. */
size_t grad_norm_workspace_bytes(const int64_t *numels, int64_t n);

/*
 * norm = sqrt(sum of g^2 over every element of n tensors), written to a device
 * float.  grads: host array of device pointers, each to numels[k] contiguous
 * elements of dtypes[k] (not read where numels[k] == 0); at most 2^16 tensors
 * and 2^44 elements.  Squares are formed and summed in 64 bits, in a fixed
 * order.  workspace: device scratch, 16-byte aligned.
 */
int grad_norm(const void *const *grads, const int64_t *numels, const int *dtypes, int64_t n, float *norm,
              void *workspace, size_t workspace_bytes, void *stream);

/*
 * grad_norm, and every gradient times c = min(1, max_norm / (norm + eps)): in
 * place where outs is NULL, else into outs[k] of out_dtypes[k] (dtypes[k], or
 * SB_F32), which is the gradient itself or shares no memory with any gradient.
 * No two tensors that are written share memory (both checked; SB_EARG); what is
 * only read may.  In place nothing is written when c is 1.  A norm
 * that is NaN or infinite scales by NaN or 0, as the formula says; the host is
 * not told (no synchronisation).  c is formed from the 64-bit norm, so finite
 * gradients whose norm is past fp32 (it is written as infinite) are scaled as
 * well.  max_norm >= 0.
 */
int grad_norm_clip(const void *const *grads, void *const *outs, const int64_t *numels, const int *dtypes,
                   const int *out_dtypes, int64_t n, float max_norm, float eps, float *norm, void *workspace,
                   size_t workspace_bytes, void *stream);

/* Thread-local message describing the last non-zero return on this thread. */
const char *seamblend_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* SEAM_BLEND_H */
