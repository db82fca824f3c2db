/*
 * gs_net.h -- C ABI of the network operators of libgs103.so.
 *
 * A network that predicts Gaussians from views works on tokens (one per
 * GS_TILE x GS_TILE pixel block) and writes the GS_NPARAM parameters that
 * gs_project reads; gs_project_bwd gives the gradient that its backward
 * starts from.  These are the operators of such a network that pass over all
 * tokens, forward and backward:
 *   gs_rope                 rotary positions with several axes
 *   gs_gated_norm_fwd/_bwd  norm after a block, gate, residual scale,
 *                           residual sum and norm before the next block
 *   gs_act8_*, gs_glu_*     activation checkpoints in 8 bits and their use in
 *                           the backward pass
 *
 * Conventions as in gs.h: the caller owns every buffer; pointers are device
 * pointers unless marked (host); work is enqueued on `stream`; arguments are
 * checked on the host before anything is enqueued.  Tensors here are
 * matrices or [tokens][heads][dim] arrays with strides in ELEMENTS; the last
 * axis is contiguous.  A data pointer needs the alignment of its element
 * only, and rows may start anywhere; 16-byte aligned rows are the fast case.
 * Sums, statistics and weights are fp32.  A call with zero tokens is valid
 * (sums over the tokens are then written as zeros).
 */
#ifndef GS_NET_H
#define GS_NET_H

#include "gs.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gs_dtype { GS_BF16 = 0, GS_F16 = 1, GS_F32 = 2 } gs_dtype;

/* ---------------------------------------------------------------------- */
/* Rotary positions with several axes (view, row, column, ...).  The first
 * sum(dims) channels of a head are split into n_axes sections; section a of
 * dims[a] channels holds dims[a] / 2 pairs, pair j rotated by the angle
 *   positions[t][a] * scale[a] * base[a] ^ (-2 j / dims[a])
 * as (u, v) -> (u cos - v sin, u sin + v cos).  The remaining channels pass
 * through.  A pair is (j, j + dims[a] / 2) within its section, or
 * (2 j, 2 j + 1) when interleaved.  The inverse rotation is the backward
 * pass: the gradient of the inputs from that of the outputs. */
#define GS_ROPE_MAX_AXES 4
#define GS_ROPE_MAX_DIM 256

/* gs_rope_turns -- turns[] (host, sum(dims) / 2 entries): each pair's
 * frequency as a 64-bit fraction of a turn, f / 2 pi * 2^64 mod 2^64 to within
 * 1.  A position times this, modulo 2^64, is the angle's phase, off by 2^-64 of
 * a turn for each unit of the position.  1 <= n_axes <= GS_ROPE_MAX_AXES,
 * dims[a] even and >= 0, 2 <= sum(dims) <= GS_ROPE_MAX_DIM, base[a] > 0,
 * scale[a] and every frequency finite. */
gs_status gs_rope_turns(int32_t n_axes, const int32_t* dims, const double* base,
                        const double* scale, uint64_t* turns);

/* One set of heads (queries, or keys): in and out [tokens][heads][head_dim].
 * out may equal in with the same strides (in place; others are refused). */
typedef struct gs_heads {
  const void* in;
  void* out;
  int64_t in_token, in_head, out_token, out_head; /* strides, elements */
  int32_t heads;
} gs_heads;

/* gs_rope -- rotates one or two sets of heads in one launch.
 *   dims, turns  (host) as given to and by gs_rope_turns
 *   positions    [tokens][n_axes] int32, any values
 *   sets         (host) n_sets = 1 or 2 sets, 0 <= heads <= 65536
 *   dtype        gs_dtype of the heads; the rotation is computed in fp32 */
gs_status gs_rope(int64_t tokens, int32_t n_axes, const int32_t* dims, const uint64_t* turns,
                  int32_t interleaved, int32_t inverse, const int32_t* positions,
                  int32_t head_dim, int32_t dtype, const gs_heads* sets, int32_t n_sets,
                  void* stream);

/* ---------------------------------------------------------------------- */
/* The join of two blocks of a residual network, per token (row) with C
 * channels:
 *   u  = w_post * norm(block)      (post; u = block without, whatever w_post)
 *   x' = x + res_scale * gate[g] * u
 *   y  = w_pre * norm(x')
 * norm(v) = v * rsqrt(mean(v^2) + eps), or with GS_NORM_CENTER
 * (v - mean) * rsqrt(mean((v - mean)^2) + eps).  w_post, w_pre, res_scale
 * [C] fp32 or NULL (ones); gate [groups][C] or NULL (ones), where row t
 * belongs to group g with group_offsets[g] <= t < group_offsets[g + 1]
 * (int32, ascending from 0 to tokens; a group may be empty; NULL with one
 * group: all rows).  x and x' are of type res_dtype, everything else of type
 * dtype; res_dtype is dtype or GS_F32.  1 <= C <= GS_NORM_MAX_C. */
#define GS_NORM_MAX_C 8192
#define GS_NORM_POST 1    /* norm after the block                             */
#define GS_NORM_CENTER 2  /* centred norms                                    */

typedef struct gs_norm {
  int64_t tokens;
  int32_t channels, groups;  /* groups: 1 without a gate                      */
  int32_t flags;             /* GS_NORM_*                                     */
  int32_t dtype, res_dtype;
  float eps;
  const float *w_pre, *w_post, *res_scale;
  const void* gate;
  const int32_t* group_offsets;
} gs_norm;

/* gs_gated_norm_fwd
 *   x, block    [tokens][C]; block NULL: no sum, y = w_pre * norm(x) (x_out
 *               NULL)
 *   x_out, y    outputs; y NULL: no norm before (the network's last sum);
 *               x_out may equal x (same strides)
 *   stats       [tokens][4] fp32 output: mean and 1/deviation of block, mean
 *               and 1/deviation of x' (0 where not computed)
 *   y_q, y_e    y's checkpoint (see gs_act8_encode; the bytes are those of
 *               encoding y as stored), or NULL both */
gs_status gs_gated_norm_fwd(const gs_norm* p, const void* x, int64_t x_stride, const void* block,
                            int64_t block_stride, void* x_out, int64_t x_out_stride, void* y,
                            int64_t y_stride, float* stats, int8_t* y_q, int64_t q_stride,
                            uint8_t* y_e, int64_t e_stride, void* stream);

/* gs_gated_norm_bwd -- with d = dx_out + (gradient through norm(x')):
 *   dx = d, dblock = gradient through gate, scale and norm, and the sums over
 *   rows dw_pre, dw_post, dres_scale [C], dgate [groups][C] (fp32 outputs,
 *   overwritten, NULL where not wanted; the order of summation is fixed;
 *   without GS_NORM_POST dw_post is zeros).
 *   x_out    [tokens][C] x' as the forward wrote it
 *   block, stats  the forward's; block NULL as there (dblock NULL)
 *   dx_out   gradient of x' from the rest of the network, or NULL (0)
 *   dy       gradient of y, or NULL (0; then dw_pre is zeros)
 *   dx       may equal dx_out, dblock may equal dy (same strides)
 *   workspace  gs_gated_norm_workspace_bytes(channels, groups) bytes, 16-byte
 *              aligned, no initialisation */
size_t gs_gated_norm_workspace_bytes(int32_t channels, int32_t groups);
gs_status gs_gated_norm_bwd(const gs_norm* p, const void* x_out, int64_t x_stride,
                            const void* block, int64_t block_stride, const float* stats,
                            const void* dx_out, int64_t dx_out_stride, const void* dy,
                            int64_t dy_stride, void* dx, int64_t dx_stride, void* dblock,
                            int64_t dblock_stride, float* dw_pre, float* dw_post, float* dgate,
                            float* dres_scale, void* workspace, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------- */
/* Activation checkpoints in 8 bits.  Channels [32 i, 32 i + 32) of a row share
 * one exponent e; a value is q * 2^(e - 127), with e the smallest exponent
 * >= 1 for which the group's largest magnitude is at most 127 * 2^(e - 127)
 * and q rounded to nearest (ties to even), |q| <= 127.  Such a value is exact
 * in bf16 and fp32; where only that rounding carried it past the largest number
 * of the type that it is read in, gs_act8_decode and gs_glu_bwd (fp32) read that
 * number (above 65024 in fp16, above 127 * 2^121 in bf16 and fp32).  Only a group with an infinity or a NaN,
 * which has e = 255 and q = 0, reads back as NaN.  Storage: q int8 [tokens][ld], e uint8 [tokens][ld / 32]
 * with ld = C rounded up to 32 (the padding is zero); q rows are 16-byte
 * aligned (q_stride a multiple of 16, at least ld; e_stride at least ld / 32). */
#define GS_ACT8_GROUP 32

gs_status gs_act8_encode(int64_t tokens, int32_t channels, int32_t dtype, const void* x,
                         int64_t x_stride, int8_t* q, int64_t q_stride, uint8_t* e,
                         int64_t e_stride, void* stream);
gs_status gs_act8_decode(int64_t tokens, int32_t channels, int32_t dtype, const int8_t* q,
                         int64_t q_stride, const uint8_t* e, int64_t e_stride, void* x,
                         int64_t x_stride, void* stream);

/* A gated unit h = act(gate) * up (up NULL: h = act(gate)), act GS_ACT_SILU
 * v / (1 + e^-v) or GS_ACT_GELU v Phi(v).
 * gs_glu_fwd writes h from the exact inputs and their checkpoints; gs_glu_bwd
 * takes the derivative at the values that the checkpoints hold:
 *   dgate = dh * up * act'(gate), dup = dh * act(gate)
 * and, with h_q and h_e, writes the checkpoint of h at those values, from
 * which the next product's weight gradient is taken.  dgate may equal dh
 * (same strides). */
#define GS_ACT_SILU 0
#define GS_ACT_GELU 1

typedef struct gs_ckpt {  /* a checkpoint's arrays; q NULL: none              */
  int8_t* q;
  uint8_t* e;
  int64_t q_stride, e_stride;
} gs_ckpt;

gs_status gs_glu_fwd(int64_t tokens, int32_t channels, int32_t dtype, int32_t act,
                     const void* gate, int64_t gate_stride, const void* up, int64_t up_stride,
                     void* h, int64_t h_stride, const gs_ckpt* gate8, const gs_ckpt* up8,
                     void* stream);
gs_status gs_glu_bwd(int64_t tokens, int32_t channels, int32_t dtype, int32_t act,
                     const gs_ckpt* gate8, const gs_ckpt* up8, const void* dh, int64_t dh_stride,
                     void* dgate, int64_t dgate_stride, void* dup, int64_t dup_stride,
                     const gs_ckpt* h8, void* stream);

/* gs_act8_wgrad -- the weight gradient of a linear layer y = x w^T from the
 * checkpoint of its input: dw[n][k] = sum_t dy[t][n] * x8[t][k], n < rows,
 * k < channels, summed in fp32; accumulate != 0 adds to dw (the sum is
 * formed in fp32 and rounded once).
 *   dy          [tokens][rows] of type dtype; used exactly in every type (of
 *               an fp32 gradient what lies below 2^-133 is cut)
 *   q, e        the checkpoint; its values are used exactly, as bf16 (64
 *               steps of 2^122, a magnitude above 127 * 2^121 that was
 *               rounded up, are an infinity there)
 *   dw          [rows][channels] of type out_dtype (GS_F32 or GS_BF16)
 *   tokens      times the bf16 terms of dy's type (1 bf16, 2 fp16, 3 fp32) at
 *               most 2^31 - 64 when rounded up to 64
 *   workspace   gs_act8_wgrad_workspace_bytes(...) bytes (0: refused), 16-byte aligned;
 *               its first 256 bytes must be zero before the first call
 *               (gs_workspace_status reads them) and calls on one workspace
 *               must not overlap */
size_t gs_act8_wgrad_workspace_bytes(int64_t tokens, int32_t rows, int32_t channels,
                                     int32_t dtype);
gs_status gs_act8_wgrad(int64_t tokens, int32_t rows, int32_t channels, int32_t dtype,
                        const void* dy, int64_t dy_stride, const int8_t* q, int64_t q_stride,
                        const uint8_t* e, int64_t e_stride, void* dw, int64_t dw_stride,
                        int32_t out_dtype, int32_t accumulate, void* workspace, size_t ws_bytes,
                        void* stream);

/* Self-test of gs_act8_wgrad's bounded waits: the call in bf16 with contiguous
 * arrays and an fp32 dw, whose exponents stop after `steps` steps of 64 tokens
 * per pair of SMs (in eights), so that its waits run out, after 100 ms instead of
 * two seconds; the kernel waits for its copies under way, flags the error and
 * ends, and the call synchronises and returns GS_ERR_TIMEOUT (GS_OK where
 * `steps` were enough).  dw is left undefined, the context stays usable. */
gs_status gs_selftest_wgrad_timeout(int64_t tokens, int32_t rows, int32_t channels,
                                    const void* dy, const int8_t* q, const uint8_t* e, void* dw,
                                    void* workspace, size_t ws_bytes, int32_t steps, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* GS_NET_H */
