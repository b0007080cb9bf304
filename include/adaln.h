/*
 * libadaln — fused AdaLN (LayerNorm-Modulate) forward and backward for GB300 (sm_103a).
 *
 * The operator is the fused normalisation + modulation node of video / MMDiT diffusion
 * transformers described in "AdaptiveLoad: Towards Efficient Video Diffusion Transformer
 * Training" (technical summary, section 2.B "Fused LayerNorm-Modulate CUDA kernels").
 * The pages name the operator without printing its formula; this library computes, for
 * every token row x of width D that is modulated by row m of the shift/scale tables:
 *
 *     mean = (1/D) sum_d x_d,   var = (1/D) sum_d (x_d - mean)^2   (biased)
 *     rstd = 1 / sqrt(var + eps),   xhat = (x - mean) * rstd       (no LayerNorm affine)
 *     y    = xhat * (1 + scale[m]) + shift[m]
 *
 * and the gradients of a loss L with dL/dy = dy:
 *
 *     dx        = rstd * (g - mean_d(g) - xhat * mean_d(g * xhat)),  g = dy * (1 + scale[m])
 *     dshift[m] = sum over tokens of m of dy,   dscale[m] = sum over tokens of m of dy * xhat
 *
 * The backward reduces dshift/dscale with threads pinned to a feature index d that
 * accumulate down the sequence (the section's "D-tile coalesced reduction"), into per-tile
 * fp32 partials that a second, fixed-order stage sums: results are bitwise reproducible
 * run to run on the same device with the same arguments. No float atomics are used whose order
 * could show (the vocabulary loss adds each later piece's part of dx in place, one addition to an
 * element and launch).
 *
 * Layouts (all row-major, D contiguous):
 *   x, y, dy, dx      [R, D]   in `dtype`       R = Bt*N (dense) or total_tokens (packed)
 *   shift, scale      [nmod, D] in `dtype`      dense: nmod = Bt, token (b, n) uses row b
 *   mean, rstd        [R]      fp32
 *   dshift, dscale    [nmod, D] fp32            (always fp32, also for bf16 I/O)
 *   cu_seqlens        [nseg+1] int32 (device)   packed: cu_seqlens[0] = 0, non-decreasing,
 *                                               cu_seqlens[nseg] = total_tokens
 *   mod_idx           [nseg]   int32 (device)   segment s uses modulation row mod_idx[s]
 *
 * Ownership and execution. The caller owns every buffer. Every call is asynchronous and
 * ordered on the caller's `stream`; nothing synchronises except adaln_read_status. The
 * library allocates no device memory and keeps no state beyond cached device properties
 * (adaln_bwd_noalloc's fixed scratch array, below, is part of the loaded module).
 * Inputs and outputs must not alias.
 *
 * Preconditions (checked on the host; a violation returns a status and launches nothing):
 *   - x, y, dy, dx, shift, scale, dshift, dscale: 16-byte aligned; mean, rstd: 4-byte
 *     aligned; workspace: 256-byte aligned.
 *   - 8 <= D <= 16384 and D % 8 == 0; eps > 0 and finite.
 *   - Bt, N, total_tokens, nseg, nmod >= 0 (empty problems are valid: a backward with no
 *     tokens writes zero gradients).
 *
 * Data errors in device-resident tables (cu_seqlens not starting at 0, decreasing, or not
 * ending at total_tokens; mod_idx outside [0, nmod)) cannot be seen by the host. The
 * kernels detect them, skip the affected rows without any out-of-range access, and record
 * a code in the workspace; adaln_read_status returns it.
 *
 * Workspace. The packed forward and both backwards take a caller-allocated device
 * workspace of at least the size the matching *_workspace_size function returns for the
 * CURRENT device (the size depends on its SM count). It needs no initialisation. With the other
 * arguments the same, a size never falls as Bt, N, total_tokens or R grows: a workspace
 * for the largest batch serves every smaller one.
 * Determinism holds for a fixed device model: the tile split follows its SM count.
 */
#ifndef ADALN_H_
#define ADALN_H_

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { ADALN_F32 = 0, ADALN_BF16 = 1 } adaln_dtype;

typedef enum {
    ADALN_OK = 0,
    ADALN_ERR_INVALID_ARG = 1,  /* null pointer, negative size, bad eps or dtype       */
    ADALN_ERR_UNSUPPORTED = 2,  /* D outside [8, 16384] or not a multiple of 8; a dtype the
                                   call does not take                                   */
    ADALN_ERR_ALIGNMENT = 3,    /* a pointer violates the alignment above               */
    ADALN_ERR_WORKSPACE = 4,    /* workspace null or smaller than required              */
    ADALN_ERR_CUDA = 5,         /* a CUDA runtime call or kernel launch failed          */
    ADALN_ERR_BAD_SEQLENS = 6,  /* device data: cu_seqlens malformed (adaln_read_status) */
    ADALN_ERR_BAD_MOD_IDX = 7,  /* device data: mod_idx out of range (adaln_read_status) */
    ADALN_ERR_TIMEOUT = 8,      /* a kernel gave up waiting (1 s) for a bulk copy of its
                                   input rows, for the row sums of the other CTA of its
                                   cluster (fp32 rows wider than 14336) or for a matrix
                                   product; its outputs from then on are not valid
                                   (adaln_read_status) */
    ADALN_ERR_BAD_TARGET = 9    /* device data: a target neither in [0, V) nor ignore_index
                                   (adaln_read_status)                                  */
} adaln_status;

/* Forward, dense batch x[Bt, N, D]; token (b, n) uses shift[b], scale[b].
 * Writes y, mean, rstd. Section 2.B, forward-pass bullet: statistics stay on chip, the
 * row is reduced by warp shuffles then a block reduction, and the modulation is applied
 * on a later pass over the row held in registers. One launch. */
int adaln_fwd(const void* x, const void* shift, const void* scale, void* y, float* mean,
              float* rstd, int64_t Bt, int64_t N, int64_t D, float eps, adaln_dtype dtype,
              cudaStream_t stream);

/* Workspace bytes adaln_bwd needs on the current device. */
size_t adaln_bwd_workspace_size(int64_t Bt, int64_t N, int64_t D, adaln_dtype dtype);

/* Backward, dense batch. Reads dy, x, the forward's mean/rstd and scale; writes dx [Bt,N,D]
 * and dshift/dscale [Bt, D] (fp32, overwritten). Section 2.B, backward-pass bullet ("D-tile
 * coalesced reduction"): each row's dx is computed from the saved statistics while threads
 * pinned to feature indices accumulate dy and dy*xhat down their tile of rows; per-tile
 * partials are summed by a second, fixed-order stage. Two launches on `stream`; for fp32
 * rows wider than 14336 the first is a launch of two-CTA thread-block clusters (each CTA
 * half of every row), so such calls need a device and context that allow clusters. */
int adaln_bwd(const void* dy, const void* x, const float* mean, const float* rstd,
              const void* scale, void* dx, float* dshift, float* dscale, void* workspace,
              size_t workspace_bytes, int64_t Bt, int64_t N, int64_t D, adaln_dtype dtype,
              cudaStream_t stream);

/* The two stages of adaln_bwd as separate calls, taking adaln_bwd's exact arguments:
 * adaln_bwd_partials launches only the fused dx + per-tile partial kernel (writes dx and the
 * workspace partials; dshift/dscale untouched), adaln_bwd_reduce only the fixed-order
 * second stage (reads the workspace partials, writes dshift/dscale). Calling both in this
 * order on one stream is exactly adaln_bwd; they exist so each stage can be timed alone. */
int adaln_bwd_partials(const void* dy, const void* x, const float* mean, const float* rstd,
                       const void* scale, void* dx, float* dshift, float* dscale, void* workspace,
                       size_t workspace_bytes, int64_t Bt, int64_t N, int64_t D, adaln_dtype dtype,
                       cudaStream_t stream);
int adaln_bwd_reduce(const void* dy, const void* x, const float* mean, const float* rstd,
                     const void* scale, void* dx, float* dshift, float* dscale, void* workspace,
                     size_t workspace_bytes, int64_t Bt, int64_t N, int64_t D, adaln_dtype dtype,
                     cudaStream_t stream);

/* Workspace bytes adaln_fwd_varlen needs (a small status area). */
size_t adaln_fwd_varlen_workspace_size(int64_t total_tokens, int32_t nseg, int64_t D,
                                       adaln_dtype dtype);

/* Forward, packed mixed-length segments (x[total_tokens, D]); segment s uses modulation
 * row mod_idx[s] of shift/scale [nmod, D]. Same math as adaln_fwd. Section 2.A batches
 * sequences of very different lengths into buckets (B sequences of length S each); the pages
 * print no interface for feeding such a bucket to the operator. This call is the library's
 * reading: the bucket's sequences packed back to back, delimited by the prefix sums
 * cu_seqlens (segment s = rows [cu_seqlens[s], cu_seqlens[s+1])), each sequence with its
 * own modulation row (the timestep / condition embedding of its sample), as section 2.B's
 * per-sample modulation requires. The workspace receives the per-CTA status words. */
int adaln_fwd_varlen(const void* x, const void* shift, const void* scale, void* y, float* mean,
                     float* rstd, const int32_t* cu_seqlens, const int32_t* mod_idx, int32_t nseg,
                     int64_t total_tokens, int64_t nmod, int64_t D, float eps, void* workspace,
                     size_t workspace_bytes, adaln_dtype dtype, cudaStream_t stream);

/* Workspace bytes adaln_bwd_varlen needs on the current device. */
size_t adaln_bwd_varlen_workspace_size(int64_t total_tokens, int32_t nseg, int64_t nmod,
                                       int64_t D, adaln_dtype dtype);

/* Backward, packed segments (the layout of adaln_fwd_varlen, section 2.A buckets).
 * dshift/dscale [nmod, D]: row m sums every token of every segment with mod_idx == m, in a
 * fixed order; rows no segment uses are written as 0. Section 2.B, backward-pass bullet:
 * the D-tile reduction runs down each (row tile, segment) piece, and the pieces of every
 * modulation row are summed by the fixed-order second stage. */
int adaln_bwd_varlen(const void* dy, const void* x, const float* mean, const float* rstd,
                     const void* scale, void* dx, float* dshift, float* dscale,
                     const int32_t* cu_seqlens, const int32_t* mod_idx, int32_t nseg,
                     int64_t total_tokens, int64_t nmod, int64_t D, void* workspace,
                     size_t workspace_bytes, adaln_dtype dtype, cudaStream_t stream);

/* The two stages of adaln_bwd_varlen, with its exact arguments (see adaln_bwd_partials). */
int adaln_bwd_varlen_partials(const void* dy, const void* x, const float* mean, const float* rstd,
                              const void* scale, void* dx, float* dshift, float* dscale,
                              const int32_t* cu_seqlens, const int32_t* mod_idx, int32_t nseg,
                              int64_t total_tokens, int64_t nmod, int64_t D, void* workspace,
                              size_t workspace_bytes, adaln_dtype dtype, cudaStream_t stream);
int adaln_bwd_varlen_reduce(const void* dy, const void* x, const float* mean, const float* rstd,
                            const void* scale, void* dx, float* dshift, float* dscale,
                            const int32_t* cu_seqlens, const int32_t* mod_idx, int32_t nseg,
                            int64_t total_tokens, int64_t nmod, int64_t D, void* workspace,
                            size_t workspace_bytes, adaln_dtype dtype, cudaStream_t stream);

/* Backward without saved statistics, for callers that do not keep the forward's mean and
 * rstd (8 bytes a row of activation memory): they are first recomputed from x with the
 * forward's row mapping and arithmetic (bitwise the values the forward wrote, for the same
 * eps), into the end of the workspace, then the backward runs as adaln_bwd /
 * adaln_bwd_varlen. It costs one more read of x.
 * The workspace must hold the *_recompute_workspace_size bytes (which include the
 * backward's own); arguments and errors otherwise as adaln_bwd / adaln_bwd_varlen. */
size_t adaln_bwd_recompute_workspace_size(int64_t Bt, int64_t N, int64_t D, adaln_dtype dtype);
int adaln_bwd_recompute(const void* dy, const void* x, const void* scale, void* dx, float* dshift,
                        float* dscale, void* workspace, size_t workspace_bytes, int64_t Bt, int64_t N,
                        int64_t D, float eps, adaln_dtype dtype, cudaStream_t stream);
size_t adaln_bwd_varlen_recompute_workspace_size(int64_t total_tokens, int32_t nseg, int64_t nmod,
                                                 int64_t D, adaln_dtype dtype);
int adaln_bwd_varlen_recompute(const void* dy, const void* x, const void* scale, void* dx,
                               float* dshift, float* dscale, const int32_t* cu_seqlens,
                               const int32_t* mod_idx, int32_t nseg, int64_t total_tokens, int64_t nmod,
                               int64_t D, float eps, void* workspace, size_t workspace_bytes,
                               adaln_dtype dtype, cudaStream_t stream);

/* Synchronises `stream`, then returns the device-side status recorded in `workspace` by
 * the last packed forward/backward (or backward, or vocabulary loss) that used it: ADALN_OK,
 * ADALN_ERR_BAD_SEQLENS, ADALN_ERR_BAD_MOD_IDX, ADALN_ERR_BAD_TARGET or ADALN_ERR_TIMEOUT, in that order of
 * precedence (ADALN_ERR_CUDA if the copy fails, ADALN_ERR_WORKSPACE if the workspace holds
 * no status). Every wait a kernel makes on its own bulk copies is bounded (1 s); a kernel
 * that runs out of time stops, drains the copies it started and records the timeout. The
 * dense forward takes no workspace, so it has nowhere to record one. */
int adaln_read_status(const void* workspace, cudaStream_t stream);

/* Bytes of the fixed scratch array adaln_bwd_noalloc uses on every device that loads the
 * library (16 MiB). */
#define ADALN_NOALLOC_SCRATCH_BYTES (16u << 20)

/* adaln_bwd for callers that cannot allocate device memory (no caller workspace).
 * The paper has no counterpart to this call; it exists for callers such as a host framework
 * that only hands out the tensors it owns, code that runs under an allocator that must not
 * grow, or a plain C program without a device allocator. Same arguments and results as
 * adaln_bwd minus the workspace: the scratch is a fixed array of ADALN_NOALLOC_SCRATCH_BYTES
 * inside this library, held by every GPU that loads the library until the process exits.
 *   - Allocates nothing (no cudaMalloc, no cudaFree, no allocating library routine).
 *   - Problems whose scratch need, adaln_bwd_workspace_size(Bt, N, D, dtype), exceeds
 *     ADALN_NOALLOC_SCRATCH_BYTES are rejected with ADALN_ERR_WORKSPACE before any launch.
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current; make that first call before any
 *     stream capture.
 *   - Every call on a device shares the one array, which keeps the last call's contents;
 *     nothing in it needs to start at zero. Calls that overlap on the GPU (different
 *     streams, or different host threads, without ordering between them) race on it and
 *     give wrong gradients: order them on one stream.
 *   - The device address is cached per device index for the life of the process; it does
 *     not survive cudaDeviceReset (or any teardown of the device's primary context), after
 *     which this call must not be used in that process.
 *   - The kernels record device-side errors (a timed-out wait) in the array, where
 *     adaln_read_status cannot see them: read them with adaln_noalloc_read_status. */
int adaln_bwd_noalloc(const void* dy, const void* x, const float* mean, const float* rstd,
                      const void* scale, void* dx, float* dshift, float* dscale, int64_t Bt,
                      int64_t N, int64_t D, adaln_dtype dtype, cudaStream_t stream);

/* adaln_read_status for adaln_bwd_noalloc: synchronises `stream`, then returns the device-side
 * status the last adaln_bwd_noalloc on the current device recorded in the library's fixed
 * array (ADALN_OK or ADALN_ERR_TIMEOUT; ADALN_ERR_WORKSPACE before the first such call on the
 * device, ADALN_ERR_CUDA if the copy fails). It copies a few bytes to the host and allocates
 * nothing on the device. Like adaln_bwd_noalloc, this call has no counterpart in the paper. */
int adaln_noalloc_read_status(cudaStream_t stream);

/* ---- Affine layer norm ------------------------------------------------------------------
 * The network's norms with a learned weight and bias [D] (in `dtype`) in place of a
 * conditioned modulation row, e.g. the final norm before a vocabulary head:
 *     y  = xhat * weight + bias                     (null weight: 1, null bias: 0)
 *     dx = rstd * (g - mean_d(g) - xhat * mean_d(g * xhat)),  g = dy * weight
 *     dweight = sum over rows of dy * xhat,  dbias = sum over rows of dy    (fp32, overwritten)
 * x, y, dy, dx [R, D]; mean, rstd [R] as in adaln_fwd. dweight and dbias may each be null (not
 * wanted; with both null the reduction is not launched). R = 0 is valid: the forward does
 * nothing, the backward writes zero dweight and dbias. Checks, reduction order, launches and
 * status as adaln_fwd / adaln_bwd. */
int adaln_layernorm_fwd(const void* x, const void* weight, const void* bias, void* y, float* mean,
                        float* rstd, int64_t R, int64_t D, float eps, adaln_dtype dtype,
                        cudaStream_t stream);
size_t adaln_layernorm_bwd_workspace_size(int64_t R, int64_t D, adaln_dtype dtype);
int adaln_layernorm_bwd(const void* dy, const void* x, const float* mean, const float* rstd,
                        const void* weight, void* dx, float* dweight, float* dbias, void* workspace,
                        size_t workspace_bytes, int64_t R, int64_t D, adaln_dtype dtype,
                        cudaStream_t stream);

/* ---- Softmax cross entropy over a vocabulary ---------------------------------------------
 * The loss of a vocabulary head: hidden rows x [N, D], the head's weight [V, D] (bf16), targets
 * [N] (device int64). The logits are never kept: the forward reduces tiles of them as they are
 * computed, the backward computes them again, a piece of the vocabulary at a time.
 *     z = x weight^T,  lse[i] = log sum_v exp(z[i, v]),  loss[i] = lse[i] - z[i, target[i]]
 *     dz[i, v] = exp(z[i, v] - lse[i]) * (dloss[i] + dlse[i]) - (v == target[i]) * dloss[i]
 *     dx = dz weight,  dweight = dz^T x
 * Rows with target == ignore_index carry no loss: their loss, lse and dx are 0, they add
 * nothing to dweight whatever x holds there, and they cost no products. A target outside
 * [0, V) that is not ignore_index is treated the same and recorded (ADALN_ERR_BAD_TARGET in
 * adaln_read_status, after the forward or the backward).
 *
 * x, weight, dx, dweight: `dtype` ADALN_BF16 (ADALN_F32 is ADALN_ERR_UNSUPPORTED: the products
 * run on the tensor cores, whose operands are bf16), 16-byte aligned, contiguous; loss, lse,
 * dloss, dlse: fp32. Products accumulate in fp32 on the tensor cores, which cut sums towards zero
 * after every 16 terms (losses are good to 1e-6 of themselves at D = 2048). dz is rounded to bf16
 * before its two products, but the target's remainder is added to both in fp32; dx and dweight are
 * rounded once at the end. The loss is taken from the distance to the row's largest logit, so it
 * is not negative and small losses are exact to fp32. Results are bitwise reproducible.
 * N >= 0, 1 <= V, D as everywhere. dlse may be null (lse is not differentiated); dx or dweight
 * may be null (not wanted). With N = 0 the backward writes zero dweight. The backward takes the
 * forward's lse and must get its ignore_index. Workspace as *_workspace_size says (they do not
 * depend on the device); it keeps nothing between calls. */
size_t adaln_linear_xent_fwd_workspace_size(int64_t N, int64_t V, int64_t D, adaln_dtype dtype);
int adaln_linear_xent_fwd(const void* x, const void* weight, const int64_t* target, float* loss, float* lse,
                          int64_t N, int64_t V, int64_t D, int64_t ignore_index, void* workspace,
                          size_t workspace_bytes, adaln_dtype dtype, cudaStream_t stream);
size_t adaln_linear_xent_bwd_workspace_size(int64_t N, int64_t V, int64_t D, adaln_dtype dtype);
int adaln_linear_xent_bwd(const void* x, const void* weight, const int64_t* target, const float* lse,
                          const float* dloss, const float* dlse, void* dx, void* dweight, int64_t N, int64_t V,
                          int64_t D, int64_t ignore_index, void* workspace, size_t workspace_bytes,
                          adaln_dtype dtype, cudaStream_t stream);

/* ---- Head norms with rotation by positions -----------------------------------------------
 * Queries and keys on their way from a projection into attention: an RMS norm of each head, and the
 * rotation of its pairs of neighbouring elements by angles that follow from the row's positions, in
 * one pass over both.
 *     xhat = x / sqrt(mean_d(x^2) + eps),  y = xhat * weight                (norm != 0; else y = x)
 *     out[2i] = y[2i] cos t - y[2i+1] sin t,  out[2i+1] = y[2i] sin t + y[2i+1] cos t
 *     t = pos[r, a] * theta^(-2j / axes[a])     for the pair j = 0 .. axes[a] / 2 - 1 of axis a
 * and, with dy the outputs' gradient turned back by t,
 *     dweight = sum over rows and heads of dy * xhat,  dx = rstd (g - xhat mean_d(g xhat)), g = dy * weight
 *
 * q [R, Hq, d] and k [R, Hk, d], d contiguous, heads d apart, rows *_ld elements apart (so that they may
 * be parts of a joint projection's rows); outputs and gradients likewise, each with a row distance of
 * its own. 8 <= d <= 256, d % 8 == 0; ADALN_F32 or ADALN_BF16, fp32 arithmetic, one rounding at the end.
 * Row distances are multiples of 8 and at least H * d; pointers are 16-byte aligned (pos and the weights'
 * gradients 4). Hq or Hk may be 0 (its pointers are not looked at): queries and keys with positions of
 * their own are two calls.
 *   - q_weight, k_weight [d], in `dtype`, each may be null (ones); without a norm both must be.
 *   - pos [R, naxes] (device int32), any values; null: no rotation. axes[naxes] (host, at most 8): the even
 *     widths of the axes, side by side from element 0; a head's elements behind them are not
 *     rotated. theta >= 1. Angles are good to 2^-25 of a turn (half of it the fp32 argument of sine and cosine)
 *     and the frequencies' own rounding (2^-50 of the angle), at any position.
 *   - dq_weight, dk_weight [d] fp32, overwritten; each may be null (not wanted). Without a norm q and k
 *     of the backward are not looked at.
 * R = 0 is valid (zero weight gradients). One launch forward, two backward (one without weight
 * gradients); sums are added in a fixed order. */
int adaln_qk_norm_rope_fwd(const void* q, const void* k, const void* q_weight, const void* k_weight,
                           const int32_t* pos, void* q_out, void* k_out, int64_t R, int32_t Hq, int32_t Hk,
                           int32_t d, int64_t q_ld, int64_t k_ld, int64_t q_out_ld, int64_t k_out_ld,
                           const int32_t* axes, int32_t naxes, double theta, float eps, int norm,
                           adaln_dtype dtype, cudaStream_t stream);
size_t adaln_qk_norm_rope_bwd_workspace_size(int64_t R, int32_t Hq, int32_t Hk, int32_t d, adaln_dtype dtype);
int adaln_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q, const void* k,
                           const void* q_weight, const void* k_weight, const int32_t* pos, void* dq, void* dk,
                           float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes, int64_t R,
                           int32_t Hq, int32_t Hk, int32_t d, int64_t dq_out_ld, int64_t dk_out_ld, int64_t q_ld,
                           int64_t k_ld, int64_t dq_ld, int64_t dk_ld, const int32_t* axes, int32_t naxes,
                           double theta, float eps, int norm, adaln_dtype dtype, cudaStream_t stream);

/* ---- Attention over packed sequences -----------------------------------------------------
 * Softmax attention of every segment's queries over the same segment's keys, without the scores:
 *     z = scale q k^T,  lse = log sum_j exp(z_j),  p = exp(z - lse),  o = p v
 *     dv = p^T dout,  dz = p (dout v^T - rowsum(dout o)),  dq = scale dz k,  dk = scale dz^T q
 * q, o, dout, dq [Rq, Hq, d]; k, v, dk, dv [Rk, Hk, d], d contiguous, heads d apart, rows *_ld elements
 * apart (parts of a joint projection's rows go as they are); lse [Hq, Rq] fp32. Heads are grouped: query
 * head h meets key head h / (Hq / Hk), and dk, dv are sums over the group.
 *   - cu_q, cu_k [nseg + 1] (device int32, as cu_seqlens everywhere): segment s has the queries
 *     cu_q[s] .. and the keys cu_k[s] ..; both tables may be the same. A null table: nseg segments of
 *     Rq / nseg (Rk / nseg) rows. Lengths may be 0 and differ between the two sides.
 *   - causal != 0: query i of a segment of n queries and m keys sees the keys j <= i + m - n (the last
 *     query sees all).
 *   - A query that sees no key has o = 0, lse = -inf and dq = 0, and adds nothing to dk and dv, whatever it
 *     and its dout hold.
 *   - scale > 0.
 * bf16 only (ADALN_F32 is ADALN_ERR_UNSUPPORTED: the products run on the tensor cores); 8 <= d <= 128,
 * d % 8 == 0; Hq a multiple of Hk; Rq, Rk, nseg <= 2^30. Row distances are multiples of 8 and at least
 * H * d; pointers 16-byte aligned (lse and the tables 4). Products accumulate in fp32; maxima, sums and lse
 * are fp32; p and dz are rounded to bf16 as operands of the next product; o, dq, dk and dv once at
 * the end. What lies behind a segment's last row reaches nothing of it, NaN included; NaN or infinity in a
 * key or value reaches the rows of its own segment, in a query that sees a key or its dout dk and dv of the
 * segment's keys (masked ones too). Results are bitwise reproducible; a segment's may differ in the last bits
 * with what it is packed with (the tiles follow the call's sizes), not with what the other segments hold.
 * The backward takes the forward's o and lse (rowsum(dout o) of queries that see at most 32 keys from the
 * scores: a rounded o is too far off where few keys share a row). dq may be null, or dk and dv both (not wanted).
 * Malformed tables are recorded (ADALN_ERR_BAD_SEQLENS in adaln_read_status) and nothing is computed:
 * outputs stay as they were. Two or three launches either way. */
size_t adaln_attention_fwd_workspace_size(int64_t nseg, int64_t Rq, int64_t Rk, int32_t Hq, int32_t Hk, int32_t d,
                                          adaln_dtype dtype);
int adaln_attention_fwd(const void* q, const void* k, const void* v, void* o, float* lse, const int32_t* cu_q,
                        const int32_t* cu_k, int64_t nseg, int64_t Rq, int64_t Rk, int32_t Hq, int32_t Hk, int32_t d,
                        int64_t q_ld, int64_t k_ld, int64_t v_ld, int64_t o_ld, float scale, int causal,
                        void* workspace, size_t workspace_bytes, adaln_dtype dtype, cudaStream_t stream);
size_t adaln_attention_bwd_workspace_size(int64_t nseg, int64_t Rq, int64_t Rk, int32_t Hq, int32_t Hk, int32_t d,
                                          adaln_dtype dtype);
int adaln_attention_bwd(const void* dout, const void* q, const void* k, const void* v, const void* o, const float* lse,
                        void* dq, void* dk, void* dv, const int32_t* cu_q, const int32_t* cu_k, int64_t nseg,
                        int64_t Rq, int64_t Rk, int32_t Hq, int32_t Hk, int32_t d, int64_t dout_ld, int64_t q_ld,
                        int64_t k_ld, int64_t v_ld, int64_t o_ld, int64_t dq_ld, int64_t dk_ld, int64_t dv_ld,
                        float scale, int causal, void* workspace, size_t workspace_bytes, adaln_dtype dtype,
                        cudaStream_t stream);

/* ---- Row sharding across ranks ----------------------------------------------------------
 * A batch can be split into contiguous, segment-aligned row shards, one per rank (the pages
 * train on 8- and 16-GPU clusters, AdaptiveLoad technical summary sections 2.A and 4). The
 * forward needs no exchange; each rank's backward gives dshift/dscale over its own tokens,
 * and the batch's gradients are their sum over ranks. adaln_sum_ranks forms that sum from
 * the ranks' fp32 gradients stacked on one device, parts[world][n] (e.g. after an
 * all-gather), always adding in rank order 0, 1, ..., world - 1:
 *     out[i] = parts[0][i] + parts[1][i] + ... + parts[world - 1][i]
 * so every rank that runs it gets the same bits, whatever moved the data. parts and out are
 * device pointers, 16-byte aligned, not overlapping; n elements each. One launch on
 * `stream`. Returns ADALN_ERR_INVALID_ARG for world < 1 or n < 0. */
int adaln_sum_ranks(const float* parts, float* out, int32_t world, int64_t n, cudaStream_t stream);

/* ---- Debug build --------------------------------------------------------------------------
 * The library can be built a second time with -DADALN_DEBUG (libadaln_debug.so; the package's
 * build(debug=True)). In that build every kernel checks each computed index of a global or
 * shared-memory access against the extent of its buffer before the access; a failed check
 * skips the access (a load yields zeros) and sets the access's class bit in a device-side
 * debug word, without trapping. adaln_debug_read waits for the device (cudaDeviceSynchronize)
 * and stores in *word the OR of the bits set since the last reset (0: no check failed); with
 * reset != 0 it also clears them. Returns ADALN_ERR_INVALID_ARG for a null word, ADALN_ERR_CUDA
 * if the device reports an error, and ADALN_ERR_UNSUPPORTED from the release build, which
 * compiles the checks away. */
#define ADALN_DEBUG_ROWS     1u   /* x, dy, y, dx: row in [0, R), bytes within the row        */
#define ADALN_DEBUG_STATS    2u   /* mean, rstd: row in [0, R)                                */
#define ADALN_DEBUG_MOD      4u   /* shift, scale: modulation row in [0, nmod)                */
#define ADALN_DEBUG_PARTIALS 8u   /* backward partials: slot in [0, tiles + nseg), column < D */
#define ADALN_DEBUG_SEGMENTS 16u  /* cu_seqlens[0 .. nseg], mod_idx[0 .. nseg)                */
#define ADALN_DEBUG_SHARED   32u  /* shared memory: within the CTA's allocation               */
#define ADALN_DEBUG_GRADS    64u  /* dshift, dscale: [0, nmod) x [0, D)                       */
#define ADALN_DEBUG_RANKS    128u /* adaln_sum_ranks: [0, n) of each rank's row              */
#define ADALN_DEBUG_STATUS   256u /* workspace status words                                   */
#define ADALN_DEBUG_LOSS     512u /* vocabulary loss: rows, packed rows, partials, gradients  */
#define ADALN_DEBUG_HEADS    1024u /* head norm and rotation: rows, heads, positions          */
#define ADALN_DEBUG_ATTN     2048u /* attention: rows, heads, work items, partial results     */
int adaln_debug_read(uint32_t* word, int reset);

/* Dual-constraint bucket size, AdaptiveLoad technical summary section 2.A:
 *     B = max(1, min(floor(M_mem / S), floor(M_comp / S^p)))
 * with exact integer arithmetic (S^p is never formed past M_comp). Host only.
 * Returns B >= 1, or -ADALN_ERR_INVALID_ARG when S, M_mem or M_comp <= 0 or p < 1. */
int64_t adaln_bucket_batch(int64_t S, int64_t M_mem, int64_t M_comp, int32_t p);

/* ---- Host-side scheduling half of section 2.A (host only, no device work) ------------- */

/* adaln_bucket_batch with a real exponent p > 0, as a fitted exponent is. An integral p in
 * [1, 64] takes the exact integer path; otherwise S^p is evaluated in double precision and
 * floor(M_comp / S^p) can differ by one from the exact value when M_comp / S^p lies within
 * about 1e-13 (relative) of an integer. Returns B >= 1, or -ADALN_ERR_INVALID_ARG when S,
 * M_mem or M_comp <= 0 or p is not positive and finite. */
int64_t adaln_bucket_batch_real(int64_t S, int64_t M_mem, int64_t M_comp, double p);

/* Shape-Benchmarking cost fit, section 2.A: the least-squares fit of the step-time model
 *     t = a + b * B * S^p
 * to n measured (B[i], S[i], t[i]) samples, p searched in [p_lo, p_hi] (for each p the
 * model is linear in a and b, solved exactly; the residual is then minimised over p by a
 * grid bracket and golden-section refinement to 1e-12 in p). With a step-time budget
 * t_budget > a, the compute bound follows as M_comp = floor((t_budget - a) / b).
 * Writes out[0..4] = a, b, p, root-mean-square residual, M_comp (M_comp = 0 when
 * t_budget <= a or b <= 0). Returns ADALN_OK, or ADALN_ERR_INVALID_ARG for n < 3, a null
 * pointer, B or S <= 0, a non-finite t, or not 0 < p_lo < p_hi. */
int adaln_fit_step_cost(const int64_t* B, const int64_t* S, const double* t, int64_t n,
                        double p_lo, double p_hi, double t_budget, double* out);

/* Compute-load imbalance of a bucketing rule, the quantity section 2.A's scheduler lowers
 * (the results report its coefficient of variation across batches). Each of the n sample
 * lengths goes to the smallest of the nbuckets increasing bucket lengths that holds it; a
 * bucket's samples, in input order, fill batches of its batch size, the last one possibly
 * partial. Batch size: rule 0 = the equal-token rule max(1, floor(M_mem / S)); rule 1 =
 * the dual constraint adaln_bucket_batch_real(S, M_mem, M_comp, p). A batch of k samples of
 * bucket S costs k * S^p. Writes out[0..2] = coefficient of variation (population standard
 * deviation / mean) of the batch costs, number of batches, mean cost. Returns ADALN_OK, or
 * ADALN_ERR_INVALID_ARG for a null pointer, n < 1, nbuckets < 1, buckets not increasing and
 * positive, a length <= 0 or above the largest bucket, M_mem or M_comp <= 0, a bad p or rule. */
int adaln_bucket_load_cv(const int64_t* lengths, int64_t n, const int64_t* buckets,
                         int32_t nbuckets, int64_t M_mem, int64_t M_comp, double p, int32_t rule,
                         double* out);

/* Static, human-readable name of a status code. */
const char* adaln_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* ADALN_H_ */
