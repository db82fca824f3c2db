// act8.cu -- activation checkpoints in 8 bits: gs_act8_encode, gs_act8_decode
// and the gated unit's two directions (gs_glu_fwd, gs_glu_bwd).
//
// 32 channels share a power-of-two step, so a value q * step is exact in bf16
// and in fp32 and the choice of q is the same in every implementation.  All
// four kernels are single passes bound by memory.  A lane has eight channels:
// WIDE, where rows start on 16-byte boundaries, eight neighbours (16-byte
// accesses of 16-bit types; a group is four lanes); otherwise eight channels 32
// apart (a warp's accesses are then runs of 32 elements at any alignment, and a
// group is the warp).
#include "net_common.cuh"

namespace gs {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;              // channels of a lane
constexpr int kUnitsPerBlock = 2048;  // lanes' worth of work

struct Act8K {
  int8_t* q;
  uint8_t* e;
  int64_t qs, es;
};

struct RowsK {
  int64_t tokens;
  int32_t C;
  int32_t upr;   // units (WIDE: lanes, else warps) per row, padding included
  int32_t rows;  // rows per block
};

template <bool WIDE>
__device__ __forceinline__ int channel(int c, int j) {
  return WIDE ? c + j : c + 32 * j;
}

// Writes eight channels' bytes and their groups' exponents.  Every lane of the
// warp calls it; channels from `end` on are not stored.
template <bool WIDE>
__device__ __forceinline__ void put8(const float (&v)[kPer], const Act8K& k, int64_t t, int c,
                                     int end) {
  int8_t* q = k.q + t * k.qs;
  uint8_t* ep = k.e + t * k.es;
  if (WIDE) {
    uint32_t mag = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) mag = max(mag, __float_as_uint(v[j]) & 0x7fffffffu);
    mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 1));
    mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 2));
    if (c >= end) return;
    const uint32_t e = act8_exponent(mag);
    const float inv = act8_inverse(e);
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t lo = __byte_perm(act8_quantise(v[4 * h], inv, e),
                                      act8_quantise(v[4 * h + 1], inv, e), 0x0040);
      const uint32_t hi = __byte_perm(act8_quantise(v[4 * h + 2], inv, e),
                                      act8_quantise(v[4 * h + 3], inv, e), 0x0040);
      w[h] = __byte_perm(lo, hi, 0x5410);
    }
    *reinterpret_cast<uint2*>(q + c) = make_uint2(w[0], w[1]);
    if (c % GS_ACT8_GROUP == 0) ep[c / GS_ACT8_GROUP] = (uint8_t)e;
  } else {
    uint32_t mine = 0;  // lane j keeps group j's exponent
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const uint32_t e =
          act8_exponent(__reduce_max_sync(0xffffffffu, __float_as_uint(v[j]) & 0x7fffffffu));
      if (c + 32 * j < end) q[c + 32 * j] = (int8_t)(act8_quantise(v[j], act8_inverse(e), e) & 0xff);
      if (lane == j) mine = e;
    }
    const int g = (c - lane) / GS_ACT8_GROUP + lane;
    if (lane < kPer && g * GS_ACT8_GROUP < end) ep[g] = (uint8_t)mine;
  }
}

template <bool WIDE>
__device__ __forceinline__ void get8(float (&v)[kPer], const Act8K& k, int64_t t, int c, int end) {
  const int8_t* q = k.q + t * k.qs;
  const uint8_t* ep = k.e + t * k.es;
  if (WIDE) {
    if (c >= end) return;
    const uint2 w = *reinterpret_cast<const uint2*>(q + c);
    const float step = act8_step(ep[c / GS_ACT8_GROUP]);
    const uint32_t x[2] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u};
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[j] = act8_value(x[j >> 2], j & 3, step);
  } else {
    uint32_t b[kPer], e[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (c + 32 * j < end) {
        b[j] = (uint8_t)q[c + 32 * j];
        e[j] = ep[(c + 32 * j) / GS_ACT8_GROUP];
      }
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (c + 32 * j < end) v[j] = act8_value(b[j] ^ 0x80u, 0, act8_step(e[j]));
  }
}

template <typename T, bool WIDE>
__device__ __forceinline__ void get(float (&v)[kPer], const T* row, int c, int C) {
  if (WIDE) {
    if (c >= C) return;
    const Pack<T, kPer> w = load_pack<T, kPer>(row + c);
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[j] = to_f32(w.v[j]);
  } else {
    T w[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (c + 32 * j < C) w[j] = row[c + 32 * j];
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (c + 32 * j < C) v[j] = to_f32(w[j]);
  }
}
template <typename T, bool WIDE>
__device__ __forceinline__ void put(const float (&v)[kPer], T* row, int c, int C) {
  if (WIDE) {
    if (c >= C) return;
    Pack<T, kPer> w;
#pragma unroll
    for (int j = 0; j < kPer; ++j) w.v[j] = from_f32<T>(v[j]);
    store_pack<T, kPer>(row + c, w);
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (c + 32 * j < C) row[c + 32 * j] = from_f32<T>(v[j]);
  }
}

// Runs f(t, c, end) for the block's units, c the lane's first channel and end
// the row's width with its padding (0 for lanes with nothing to do); whole
// warps take part in each step.
template <bool WIDE, typename F>
__device__ __forceinline__ void each_unit(const RowsK& r, F f) {
  const int64_t row0 = (int64_t)blockIdx.x * r.rows;
  const int n = r.upr * (int)min((int64_t)r.rows, r.tokens - row0);
  const int end = (r.C + GS_ACT8_GROUP - 1) / GS_ACT8_GROUP * GS_ACT8_GROUP;
  const int lane = threadIdx.x & 31;
  if (WIDE) {
    for (int at = threadIdx.x; at - lane < n; at += kThreads) {
      const int row = at / r.upr;
      f(row0 + row, (at - row * r.upr) * kPer, at < n ? end : 0);
    }
  } else {
    for (int at = threadIdx.x >> 5; at < n; at += kThreads / 32) {
      const int row = at / r.upr;
      f(row0 + row, (at - row * r.upr) * (32 * kPer) + lane, end);
    }
  }
}

template <typename T, bool WIDE>
__global__ void __launch_bounds__(kThreads) encode_kernel(RowsK r, const T* x, int64_t xs,
                                                          Act8K k) {
  each_unit<WIDE>(r, [&](int64_t t, int c, int end) {
    float v[kPer] = {};
    get<T, WIDE>(v, x + t * xs, c, min(r.C, end));
    put8<WIDE>(v, k, t, c, end);
  });
}

template <typename T, bool WIDE>
__global__ void __launch_bounds__(kThreads) decode_kernel(RowsK r, Act8K k, T* x, int64_t xs) {
  each_unit<WIDE>(r, [&](int64_t t, int c, int end) {
    float v[kPer];
    get8<WIDE>(v, k, t, c, end);
    put<T, WIDE>(v, x + t * xs, c, min(r.C, end));
  });
}

// act(v) and its derivative.  Phi comes from Abramowitz and Stegun's formula
// 7.1.26 for the error function (absolute error below 1.5e-7, half of that in
// Phi), which needs the one exponential that the derivative has too.
struct Phi {
  float p, density;  // Phi(v), phi(v)
};
__device__ __forceinline__ Phi normal(float v) {
  const float z = fabsf(v) * 0.70710678118654752f;
  const float t = __fdividef(1.f, fmaf(0.3275911f, z, 1.f));
  const float ex = __expf(-z * z);
  float q = fmaf(1.061405429f, t, -1.453152027f);
  q = fmaf(q, t, 1.421413741f);
  q = fmaf(q, t, -0.284496736f);
  q = fmaf(q, t, 0.254829592f);
  const float tail = 0.5f * q * t * ex;
  return Phi{v < 0.f ? tail : 1.f - tail, ex * 0.39894228040143268f};
}
template <int ACT>
__device__ __forceinline__ float act_value(float v) {
  if (ACT == GS_ACT_SILU) return __fdividef(v, 1.f + __expf(-v));
  return v * normal(v).p;
}
template <int ACT>
__device__ __forceinline__ void act_both(float v, float& f, float& df) {
  if (ACT == GS_ACT_SILU) {
    const float s = __fdividef(1.f, 1.f + __expf(-v));
    f = v * s;
    df = s * (1.f + v * (1.f - s));
  } else {
    const Phi n = normal(v);
    f = v * n.p;
    df = fmaf(v, n.density, n.p);
  }
}

template <typename T, bool WIDE, int ACT, bool GATED>
__global__ void __launch_bounds__(kThreads) glu_fwd_kernel(RowsK r, const T* gate, int64_t gs,
                                                           const T* up, int64_t us, T* h,
                                                           int64_t hs, Act8K g8, Act8K u8) {
  each_unit<WIDE>(r, [&](int64_t t, int c, int end) {
    const int C = min(r.C, end);
    float g[kPer] = {}, u[kPer] = {}, o[kPer];
    get<T, WIDE>(g, gate + t * gs, c, C);
    if (GATED) get<T, WIDE>(u, up + t * us, c, C);
#pragma unroll
    for (int j = 0; j < kPer; ++j) o[j] = act_value<ACT>(g[j]) * (GATED ? u[j] : 1.f);
    put<T, WIDE>(o, h + t * hs, c, C);
    if (g8.q) put8<WIDE>(g, g8, t, c, end);
    if (GATED && u8.q) put8<WIDE>(u, u8, t, c, end);
  });
}

template <typename T, bool WIDE, int ACT, bool GATED>
__global__ void __launch_bounds__(kThreads) glu_bwd_kernel(RowsK r, Act8K g8, Act8K u8,
                                                           const T* dh, int64_t dhs, T* dgate,
                                                           int64_t dgs, T* dup, int64_t dus,
                                                           Act8K h8) {
  each_unit<WIDE>(r, [&](int64_t t, int c, int end) {
    const int C = min(r.C, end);
    float g[kPer] = {}, u[kPer] = {}, d[kPer] = {};
    get8<WIDE>(g, g8, t, c, end);
    if (GATED) get8<WIDE>(u, u8, t, c, end);
    get<T, WIDE>(d, dh + t * dhs, c, C);
    float o[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      float f, df;
      act_both<ACT>(g[j], f, df);
      const float w = GATED ? u[j] : 1.f;
      o[j] = channel<WIDE>(c, j) < C ? f * w : 0.f;
      g[j] = d[j] * w * df;
      u[j] = d[j] * f;
    }
    put<T, WIDE>(g, dgate + t * dgs, c, C);
    if (GATED) put<T, WIDE>(u, dup + t * dus, c, C);
    if (h8.q) put8<WIDE>(o, h8, t, c, end);
  });
}

RowsK make_rows(int64_t tokens, int32_t C, bool wide) {
  RowsK r{tokens, C, 0, 1};
  const int lanes = (int)div_up(C, GS_ACT8_GROUP) * (GS_ACT8_GROUP / kPer);
  r.upr = wide ? lanes : (int)div_up(lanes, 32);
  const int per_block = wide ? kUnitsPerBlock : kUnitsPerBlock / 32;
  r.rows = r.upr >= per_block ? 1 : per_block / r.upr;
  const int64_t spread = div_up(tokens, (int64_t)device_sms() * 4);  // few tokens: use every SM
  if (r.rows > spread) r.rows = (int32_t)spread;
  return r;
}

unsigned blocks_of(const RowsK& r) { return (unsigned)div_up(r.tokens, r.rows); }

bool shape_ok(int64_t tokens, int32_t C, int32_t dtype) {
  return tokens >= 0 && tokens < ((int64_t)1 << 31) && C >= 1 && C <= (1 << 24) && dtype_ok(dtype);
}
bool ckpt_ok(const Act8K& k, int32_t C) {
  return k.q && k.e && aligned16(k.q) && k.qs % 16 == 0 &&
         k.qs >= div_up(C, GS_ACT8_GROUP) * GS_ACT8_GROUP;
}
Act8K ckpt_of(const gs_ckpt* c) {
  return c ? Act8K{c->q, c->e, c->q_stride, c->e_stride} : Act8K{nullptr, nullptr, 0, 0};
}

#define GS_ACT8_TYPES(dtype, ...)                     \
  do {                                                \
    if ((dtype) == GS_BF16) {                         \
      using T = __nv_bfloat16;                        \
      __VA_ARGS__;                                    \
    } else if ((dtype) == GS_F16) {                   \
      using T = __half;                               \
      __VA_ARGS__;                                    \
    } else {                                          \
      using T = float;                                \
      __VA_ARGS__;                                    \
    }                                                 \
  } while (0)

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" gs_status gs_act8_encode(int64_t tokens, int32_t channels, int32_t dtype, const void* x,
                                    int64_t x_stride, int8_t* q, int64_t q_stride, uint8_t* e,
                                    int64_t e_stride, void* stream) {
  if (!shape_ok(tokens, channels, dtype)) return GS_ERR_INVALID_ARG;
  if (tokens == 0) return GS_OK;
  const Act8K k{q, e, q_stride, e_stride};
  const int el = dtype_size(dtype);
  if (!x || !aligned_to(x, el) || !ckpt_ok(k, channels)) return GS_ERR_INVALID_ARG;
  const bool wide = channels % 8 == 0 && rows_aligned(x, x_stride, el, 16);
  const RowsK r = make_rows(tokens, channels, wide);
  cudaStream_t st = (cudaStream_t)stream;
  GS_ACT8_TYPES(dtype, if (wide) encode_kernel<T, true><<<blocks_of(r), kThreads, 0, st>>>(
                           r, (const T*)x, x_stride, k);
                else encode_kernel<T, false><<<blocks_of(r), kThreads, 0, st>>>(r, (const T*)x,
                                                                            x_stride, k));
  GS_CHECK_LAUNCH();
  return GS_OK;
}

extern "C" gs_status gs_act8_decode(int64_t tokens, int32_t channels, int32_t dtype,
                                    const int8_t* q, int64_t q_stride, const uint8_t* e,
                                    int64_t e_stride, void* x, int64_t x_stride, void* stream) {
  if (!shape_ok(tokens, channels, dtype)) return GS_ERR_INVALID_ARG;
  if (tokens == 0) return GS_OK;
  const Act8K k{const_cast<int8_t*>(q), const_cast<uint8_t*>(e), q_stride, e_stride};
  const int el = dtype_size(dtype);
  if (!x || !aligned_to(x, el) || !ckpt_ok(k, channels)) return GS_ERR_INVALID_ARG;
  const bool wide = channels % 8 == 0 && rows_aligned(x, x_stride, el, 16);
  const RowsK r = make_rows(tokens, channels, wide);
  cudaStream_t st = (cudaStream_t)stream;
  GS_ACT8_TYPES(dtype, if (wide) decode_kernel<T, true><<<blocks_of(r), kThreads, 0, st>>>(
                           r, k, (T*)x, x_stride);
                else decode_kernel<T, false><<<blocks_of(r), kThreads, 0, st>>>(r, k, (T*)x,
                                                                            x_stride));
  GS_CHECK_LAUNCH();
  return GS_OK;
}

extern "C" gs_status gs_glu_fwd(int64_t tokens, int32_t channels, int32_t dtype, int32_t act,
                                const void* gate, int64_t gate_stride, const void* up,
                                int64_t up_stride, void* h, int64_t h_stride,
                                const gs_ckpt* gate8, const gs_ckpt* up8, void* stream) {
  if (!shape_ok(tokens, channels, dtype) || (act != GS_ACT_SILU && act != GS_ACT_GELU))
    return GS_ERR_INVALID_ARG;
  if (tokens == 0) return GS_OK;
  const Act8K g8 = ckpt_of(gate8), u8 = ckpt_of(up8);
  const int el = dtype_size(dtype);
  if (!gate || !h || !aligned_to(gate, el) || !aligned_to(up, el) || !aligned_to(h, el) ||
      (g8.q && !ckpt_ok(g8, channels)) || (u8.q && (!up || !ckpt_ok(u8, channels))))
    return GS_ERR_INVALID_ARG;
  const bool wide = channels % 8 == 0 && rows_aligned(gate, gate_stride, el, 16) &&
                    rows_aligned(up, up_stride, el, 16) && rows_aligned(h, h_stride, el, 16);
  const RowsK r = make_rows(tokens, channels, wide);
  cudaStream_t st = (cudaStream_t)stream;
#define GS_GLU(WIDE, ACT)                                                                   \
  do {                                                                                      \
    if (up)                                                                                 \
      glu_fwd_kernel<T, WIDE, ACT, true><<<blocks_of(r), kThreads, 0, st>>>(                \
          r, (const T*)gate, gate_stride, (const T*)up, up_stride, (T*)h, h_stride, g8, u8); \
    else                                                                                    \
      glu_fwd_kernel<T, WIDE, ACT, false><<<blocks_of(r), kThreads, 0, st>>>(               \
          r, (const T*)gate, gate_stride, nullptr, 0, (T*)h, h_stride, g8, u8);             \
  } while (0)
  GS_ACT8_TYPES(dtype, if (act == GS_ACT_SILU) {
    if (wide) GS_GLU(true, GS_ACT_SILU); else GS_GLU(false, GS_ACT_SILU);
  } else {
    if (wide) GS_GLU(true, GS_ACT_GELU); else GS_GLU(false, GS_ACT_GELU);
  });
#undef GS_GLU
  GS_CHECK_LAUNCH();
  return GS_OK;
}

extern "C" gs_status gs_glu_bwd(int64_t tokens, int32_t channels, int32_t dtype, int32_t act,
                                const gs_ckpt* gate8, const gs_ckpt* up8, const void* dh,
                                int64_t dh_stride, void* dgate, int64_t dgate_stride, void* dup,
                                int64_t dup_stride, const gs_ckpt* h8, void* stream) {
  if (!shape_ok(tokens, channels, dtype) || (act != GS_ACT_SILU && act != GS_ACT_GELU))
    return GS_ERR_INVALID_ARG;
  if (tokens == 0) return GS_OK;
  const Act8K g8 = ckpt_of(gate8), u8 = ckpt_of(up8), o8 = ckpt_of(h8);
  const int el = dtype_size(dtype);
  if (!ckpt_ok(g8, channels) || (u8.q && !ckpt_ok(u8, channels)) || (o8.q && !ckpt_ok(o8, channels)) || (!u8.q != !dup) ||
      !dh || !dgate || !aligned_to(dh, el) || !aligned_to(dgate, el) || !aligned_to(dup, el))
    return GS_ERR_INVALID_ARG;
  const bool wide = channels % 8 == 0 && rows_aligned(dh, dh_stride, el, 16) &&
                    rows_aligned(dgate, dgate_stride, el, 16) &&
                    rows_aligned(dup, dup_stride, el, 16);
  const RowsK r = make_rows(tokens, channels, wide);
  cudaStream_t st = (cudaStream_t)stream;
#define GS_GLU(WIDE, ACT)                                                                   \
  do {                                                                                      \
    if (dup)                                                                                \
      glu_bwd_kernel<T, WIDE, ACT, true><<<blocks_of(r), kThreads, 0, st>>>(                \
          r, g8, u8, (const T*)dh, dh_stride, (T*)dgate, dgate_stride, (T*)dup, dup_stride, \
          o8);                                                                              \
    else                                                                                    \
      glu_bwd_kernel<T, WIDE, ACT, false><<<blocks_of(r), kThreads, 0, st>>>(               \
          r, g8, u8, (const T*)dh, dh_stride, (T*)dgate, dgate_stride, nullptr, 0, o8);     \
  } while (0)
  GS_ACT8_TYPES(dtype, if (act == GS_ACT_SILU) {
    if (wide) GS_GLU(true, GS_ACT_SILU); else GS_GLU(false, GS_ACT_SILU);
  } else {
    if (wide) GS_GLU(true, GS_ACT_GELU); else GS_GLU(false, GS_ACT_GELU);
  });
#undef GS_GLU
  GS_CHECK_LAUNCH();
  return GS_OK;
}
