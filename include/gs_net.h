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
 *   gs_ffn_fwd/_bwd         the gated feed-forward block: both projections,
 *                           the activation and the product in one kernel
 *   gs_linear_attn_*        linear attention with a decay for each head, in
 *                           chunks or token by token
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

/* ---------------------------------------------------------------------- */
/* The gated feed-forward block up to its last projection: both first ones, the
 * activation and the product in one kernel on the tensor cores.  With w [2 hidden][channels],
 * the gate's rows and then up's:
 *   gate = x w_gate^T, up = x w_up^T, h = act(gate) * up
 * Neither gate nor up is written; gs_ffn_bwd forms them again from x.  x, w,
 * h, dh and dx are of one type, GS_BF16 or GS_F16; sums are fp32 (the tensor
 * cores cut them, by 2^-23 at most after every 16 terms; dw's in runs of 2048
 * tokens, which are added with rounding).  h may not
 * overlap the inputs, nor may dx or dw overlap them or one another (an address
 * that is still read while it would be written is refused).
 *   workspace   gs_ffn_workspace_bytes(...) bytes (0: refused), 16-byte
 *               aligned; its first 256 bytes must be zero before the first
 *               call (gs_workspace_status reads them) and calls on one
 *               workspace must not overlap
 * tokens <= 2^31 - 512; channels, hidden <= 2^20. */
size_t gs_ffn_workspace_bytes(int64_t tokens, int32_t channels, int32_t hidden, int32_t backward);
gs_status gs_ffn_fwd(int64_t tokens, int32_t channels, int32_t hidden, int32_t dtype, int32_t act,
                     const void* x, int64_t x_stride, const void* w, int64_t w_stride, void* h,
                     int64_t h_stride, void* workspace, size_t ws_bytes, void* stream);

/* gs_ffn_bwd -- from the gradient of h:
 *   dgate = dh * up * act'(gate), dup = dh * act(gate)  (rounded to dtype)
 *   dx = dgate w_gate + dup w_up,  dw = [dgate | dup]^T x
 *   dx        [tokens][channels], or NULL where not wanted
 *   dw        [2 hidden][channels] of type dw_dtype (dtype or GS_F32), or
 *             NULL; accumulate != 0 adds to dw (the sum is formed in fp32
 *             and rounded once).  The order of summation is fixed. */
gs_status gs_ffn_bwd(int64_t tokens, int32_t channels, int32_t hidden, int32_t dtype, int32_t act,
                     const void* x, int64_t x_stride, const void* w, int64_t w_stride,
                     const void* dh, int64_t dh_stride, void* dx, int64_t dx_stride, void* dw,
                     int64_t dw_stride, int32_t dw_dtype, int32_t accumulate, void* workspace,
                     size_t ws_bytes, void* stream);

/* Self-test of the block's bounded waits: the forward call in bf16 (silu) with
 * contiguous arrays, whose operands stop after `steps` steps of 64 channels per
 * pair of SMs, so that its waits run out, after 100 ms instead of two seconds;
 * the kernel waits for its copies under way, flags the error and ends, and the
 * call synchronises and returns GS_ERR_TIMEOUT (GS_OK where `steps` were
 * enough).  h is left undefined, the context stays usable. */
gs_status gs_selftest_ffn_timeout(int64_t tokens, int32_t channels, int32_t hidden, const void* x,
                                  const void* w, void* h, void* workspace, size_t ws_bytes,
                                  int32_t steps, void* stream);

/* ---------------------------------------------------------------------- */
/* Linear attention with a decay for each head.  A head has a state S
 * [dim][vdim], and from token to token
 *   S_t = d S_{t-1} + k_t v_t^T,  o_t = scale * q_t S_t,  d = e^log_decay
 * Tokens come in groups (views, streams): group g is the tokens
 * [group_offsets[g], group_offsets[g + 1]) and goes from its state to its
 * last state.  Query head h reads key (and value) head h / (q_heads /
 * k_heads), and has a decay and a state of its own.  Tokens outside the
 * groups (behind the last one) are neither read nor written.
 * q, k, v and what is written for them are of one type, GS_BF16 or GS_F16;
 * states and sums are fp32.  The chunked calls round two things to the type on
 * the way, once each: the decayed products of queries and keys (backward also
 * of values and dout), and the states where they are multiplied by a query or
 * by dout, both in fp16 brought into its range by powers of two.  Outputs and
 * gradients are then off by about sqrt(2) times their last rounding; states that
 * are handed on have no such rounding.  An infinity or a NaN in a token spreads
 * to the outputs and gradients of its group, some of those before it among
 * them.  1 <= dim, vdim <= GS_LINEAR_ATTN_MAX_DIM. */
#define GS_LINEAR_ATTN_MAX_DIM 128

typedef struct gs_linear_attn {
  int64_t tokens;
  int32_t q_heads, k_heads;      /* k_heads divides q_heads                   */
  int32_t dim, vdim;             /* channels of queries and keys, of values   */
  int32_t groups;                /* 1 without offsets                         */
  int32_t dtype;
  float scale;
  const float* log_decay;        /* [q_heads], 0 or less                      */
  const int32_t* group_offsets;  /* [groups + 1] ascending from 0, or NULL    */
  const float* state;            /* [groups][q_heads][dim][vdim], or NULL (0) */
} gs_linear_attn;

typedef struct gs_attn_heads {   /* [tokens][heads][channels]                 */
  void* p;
  int64_t token, head;           /* strides, elements                         */
} gs_attn_heads;

/* gs_linear_attn_fwd -- all tokens of the groups, in chunks.
 *   heads       (host) four: q, k, v, out; out may not overlap the inputs (the
 *               same address is refused)
 *   state_out   [groups][q_heads][dim][vdim] fp32: the states after the
 *               groups' last tokens (a group's own state where it has none),
 *               or NULL; may equal state
 *   workspace   at most gs_linear_attn_workspace_bytes(a, backward) bytes (0:
 *               refused; rows of q, k, v and dout that do not start on 16-byte
 *               boundaries, or are no multiple of 8 long, are copied there
 *               first), 16-byte aligned, no initialisation; calls on one
 *               workspace must not overlap.  In the backward pass of shared
 *               key heads dk and dv of each query head lie there in fp32, for
 *               as many tokens at a time as there is room for: with less room
 *               (two segments of at most 2048 tokens at least) there are more
 *               launches, and the same results */
size_t gs_linear_attn_workspace_bytes(const gs_linear_attn* a, int32_t backward);
gs_status gs_linear_attn_fwd(const gs_linear_attn* a, const gs_attn_heads* heads,
                             float* state_out, void* workspace, size_t ws_bytes, void* stream);

/* gs_linear_attn_bwd -- heads (host): q, k, v, dout, dq, dk, dv; dq, dk and dv
 * may not overlap the inputs or one another (the same address is refused).  From the
 * gradients of the outputs and (dstate_out, or NULL: 0) of the last states: dq,
 * dk, dv (summed over the query heads that share a key head) and dstate, the
 * gradient of the first states (or NULL; may equal dstate_out).  The decays get
 * no gradient. */
gs_status gs_linear_attn_bwd(const gs_linear_attn* a, const gs_attn_heads* heads,
                             const float* dstate_out, float* dstate, void* workspace,
                             size_t ws_bytes, void* stream);

/* gs_linear_attn_step -- one token of each of a->tokens streams; heads (host):
 * q, k, v, out; state [tokens][q_heads][dim][vdim] fp32, read and updated in
 * place.  out may lie where q does, or k or v where key heads are not shared,
 * with the same strides; else it may not overlap them.  a->state and
 * a->group_offsets are not used. */
gs_status gs_linear_attn_step(const gs_linear_attn* a, const gs_attn_heads* heads, float* state,
                              void* stream);

/* Every wait of the chunked kernels for the tensor cores is bounded: a block waits
 * for two seconds in all, then issues no more products, waits (again for two
 * seconds at most) for its copies and products under way and ends; results are
 * undefined.  gs_linear_attn_status synchronises the stream and returns
 * GS_ERR_TIMEOUT if that happened on the current device, on any stream, since the
 * last such call. */
gs_status gs_linear_attn_status(void* stream);

/* Self-test: gs_linear_attn_fwd (or, backward != 0, _bwd, with state_out its dstate)
 * with segments of `chunks` chunks of 128 tokens (1 to 16; 0: as many as
 * gs_selftest_linear_attn_chunks says are chosen).  products >= 0: each block's tensor
 * cores get no more than that many sets of products, so that its waits run out, after
 * 20 ms instead of two seconds.  Synchronises, and returns what gs_linear_attn_status does;
 * after GS_ERR_TIMEOUT the results are undefined, the context stays usable. */
int32_t gs_selftest_linear_attn_chunks(const gs_linear_attn* a, int32_t backward, int32_t states);
gs_status gs_selftest_linear_attn(const gs_linear_attn* a, const gs_attn_heads* heads, int32_t backward,
                                  const float* dstate_out, float* state_out, void* workspace,
                                  size_t ws_bytes, int32_t chunks, int32_t products, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* GS_NET_H */
