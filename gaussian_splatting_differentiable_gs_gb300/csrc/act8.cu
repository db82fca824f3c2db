// act8.cu -- activation checkpoints in 8 bits: gs_act8_encode, gs_act8_decode
// and the gated unit's two directions (gs_glu_fwd, gs_glu_bwd).
//
// 32 channels share a power-of-two step, so a value q * step is exact in bf16
// and in fp32 and the choice of q is the same in every implementation.  All
// four kernels are single passes bound by memory: a block takes a few whole
// rows as one run of units of V channels (V = 8: 16-byte accesses of 16-bit
// types; V = 1 where a row starts off such a boundary), and a group's 32 / V
// lanes agree on its magnitude by shuffles.
#include "net_common.cuh"

namespace gs {
namespace {

constexpr int kThreads = 256;
constexpr int kUnitsPerBlock = 2048;

struct Act8K {
  int8_t* q;
  uint8_t* e;
  int64_t qs, es;
};

struct RowsK {
  int64_t tokens;
  int32_t C;
  int32_t upr;   // units per row, padding included (whole groups)
  int32_t rows;  // rows per block
};

template <int V>
__device__ __forceinline__ uint32_t group_exponent(const float (&v)[V]) {
  uint32_t mag = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) mag = max(mag, __float_as_uint(v[j]) & 0x7fffffffu);
#pragma unroll
  for (int o = 1; o < GS_ACT8_GROUP / V; o <<= 1)
    mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, o));
  return act8_exponent(mag);
}

// Writes a unit's bytes (and, once per group, the exponent).  Every lane of
// the warp calls it; only lanes with `in` store.
template <int V>
__device__ __forceinline__ void put8(const float (&v)[V], const Act8K& k, int64_t t, int c,
                                     bool in) {
  const uint32_t e = group_exponent<V>(v);
  if (!in) return;
  const float inv = act8_inverse(e);
  Pack<int8_t, V> q;
#pragma unroll
  for (int j = 0; j < V; ++j) q.v[j] = (int8_t)act8_quantise(v[j], inv, e);
  store_pack<int8_t, V>(k.q + t * k.qs + c, q);
  if (c % GS_ACT8_GROUP == 0) k.e[t * k.es + c / GS_ACT8_GROUP] = (uint8_t)e;
}

template <int V>
__device__ __forceinline__ void get8(float (&v)[V], const Act8K& k, int64_t t, int c) {
  const Pack<int8_t, V> q = load_pack<int8_t, V>(k.q + t * k.qs + c);
  const float step = act8_step(k.e[t * k.es + c / GS_ACT8_GROUP]);
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = (float)q.v[j] * step;
}

template <typename T, int V>
__device__ __forceinline__ void get(float (&v)[V], const T* p) {
  const Pack<T, V> w = load_pack<T, V>(p);
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = to_f32(w.v[j]);
}
template <typename T, int V>
__device__ __forceinline__ void put(const float (&v)[V], T* p) {
  Pack<T, V> w;
#pragma unroll
  for (int j = 0; j < V; ++j) w.v[j] = from_f32<T>(v[j]);
  store_pack<T, V>(p, w);
}

// Runs f(t, c, in) for the block's units; whole warps take part in each step.
template <int V, typename F>
__device__ __forceinline__ void each_unit(const RowsK& r, F f) {
  const int64_t row0 = (int64_t)blockIdx.x * r.rows;
  const int n = r.upr * (int)min((int64_t)r.rows, r.tokens - row0);
  for (int at = threadIdx.x; at - (int)(threadIdx.x & 31) < n; at += kThreads) {
    const int row = at / r.upr;
    f(row0 + row, (at - row * r.upr) * V, at < n);
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) encode_kernel(RowsK r, const T* x, int64_t xs,
                                                          Act8K k) {
  each_unit<V>(r, [&](int64_t t, int c, bool in) {
    float v[V] = {};
    if (in && c < r.C) get<T, V>(v, x + t * xs + c);
    put8<V>(v, k, t, c, in);
  });
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads) decode_kernel(RowsK r, Act8K k, T* x, int64_t xs) {
  each_unit<V>(r, [&](int64_t t, int c, bool in) {
    if (!in || c >= r.C) return;
    float v[V];
    get8<V>(v, k, t, c);
    put<T, V>(v, x + t * xs + c);
  });
}

// act(v) and its derivative.
template <int ACT>
__device__ __forceinline__ float act_value(float v) {
  if (ACT == GS_ACT_SILU) return __fdividef(v, 1.f + __expf(-v));
  return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
}
template <int ACT>
__device__ __forceinline__ void act_both(float v, float& f, float& df) {
  if (ACT == GS_ACT_SILU) {
    const float s = __fdividef(1.f, 1.f + __expf(-v));
    f = v * s;
    df = s * (1.f + v * (1.f - s));
  } else {
    const float p = 0.5f * (1.f + erff(v * 0.70710678118654752f));
    f = v * p;
    df = p + v * __expf(-0.5f * v * v) * 0.39894228040143268f;
  }
}

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads) glu_fwd_kernel(RowsK r, const T* gate, int64_t gs,
                                                           const T* up, int64_t us, T* h,
                                                           int64_t hs, Act8K g8, Act8K u8) {
  each_unit<V>(r, [&](int64_t t, int c, bool in) {
    float g[V] = {}, u[V] = {};
    const bool live = in && c < r.C;
    if (live) get<T, V>(g, gate + t * gs + c);
    if (live && up) get<T, V>(u, up + t * us + c);
    if (live) {
      float o[V];
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = act_value<ACT>(g[j]) * (up ? u[j] : 1.f);
      put<T, V>(o, h + t * hs + c);
    }
    if (g8.q) put8<V>(g, g8, t, c, in);
    if (u8.q) put8<V>(u, u8, t, c, in);
  });
}

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(kThreads) glu_bwd_kernel(RowsK r, Act8K g8, Act8K u8,
                                                           const T* dh, int64_t dhs, T* dgate,
                                                           int64_t dgs, T* dup, int64_t dus,
                                                           Act8K h8) {
  each_unit<V>(r, [&](int64_t t, int c, bool in) {
    float o[V] = {};
    if (in && c < r.C) {
      float g[V], u[V], d[V], dg[V], du[V];
      get8<V>(g, g8, t, c);
      if (u8.q) get8<V>(u, u8, t, c);
      get<T, V>(d, dh + t * dhs + c);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float f, df;
        act_both<ACT>(g[j], f, df);
        const float w = u8.q ? u[j] : 1.f;
        dg[j] = d[j] * w * df;
        du[j] = d[j] * f;
        o[j] = f * w;
      }
      put<T, V>(dg, dgate + t * dgs + c);
      if (dup) put<T, V>(du, dup + t * dus + c);
    }
    if (h8.q) put8<V>(o, h8, t, c, in);
  });
}

RowsK make_rows(int64_t tokens, int32_t C, int V) {
  RowsK r{tokens, C, (int32_t)(div_up(C, GS_ACT8_GROUP) * (GS_ACT8_GROUP / V)), 1};
  r.rows = r.upr >= kUnitsPerBlock ? 1 : kUnitsPerBlock / r.upr;
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
  const RowsK r = make_rows(tokens, channels, wide ? 8 : 1);
  cudaStream_t st = (cudaStream_t)stream;
  GS_ACT8_TYPES(dtype, if (wide) encode_kernel<T, 8><<<blocks_of(r), kThreads, 0, st>>>(
                           r, (const T*)x, x_stride, k);
                else encode_kernel<T, 1><<<blocks_of(r), kThreads, 0, st>>>(r, (const T*)x,
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
  const RowsK r = make_rows(tokens, channels, wide ? 8 : 1);
  cudaStream_t st = (cudaStream_t)stream;
  GS_ACT8_TYPES(dtype, if (wide) decode_kernel<T, 8><<<blocks_of(r), kThreads, 0, st>>>(
                           r, k, (T*)x, x_stride);
                else decode_kernel<T, 1><<<blocks_of(r), kThreads, 0, st>>>(r, k, (T*)x,
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
  const RowsK r = make_rows(tokens, channels, wide ? 8 : 1);
  cudaStream_t st = (cudaStream_t)stream;
#define GS_GLU(V, ACT)                                                                      \
  glu_fwd_kernel<T, V, ACT><<<blocks_of(r), kThreads, 0, st>>>(                             \
      r, (const T*)gate, gate_stride, (const T*)up, up_stride, (T*)h, h_stride, g8, u8)
  GS_ACT8_TYPES(dtype, if (act == GS_ACT_SILU) {
    if (wide) GS_GLU(8, GS_ACT_SILU); else GS_GLU(1, GS_ACT_SILU);
  } else {
    if (wide) GS_GLU(8, GS_ACT_GELU); else GS_GLU(1, GS_ACT_GELU);
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
  const RowsK r = make_rows(tokens, channels, wide ? 8 : 1);
  cudaStream_t st = (cudaStream_t)stream;
#define GS_GLU(V, ACT)                                                                       \
  glu_bwd_kernel<T, V, ACT><<<blocks_of(r), kThreads, 0, st>>>(                              \
      r, g8, u8, (const T*)dh, dh_stride, (T*)dgate, dgate_stride, (T*)dup, dup_stride, o8)
  GS_ACT8_TYPES(dtype, if (act == GS_ACT_SILU) {
    if (wide) GS_GLU(8, GS_ACT_SILU); else GS_GLU(1, GS_ACT_SILU);
  } else {
    if (wide) GS_GLU(8, GS_ACT_GELU); else GS_GLU(1, GS_ACT_GELU);
  });
#undef GS_GLU
  GS_CHECK_LAUNCH();
  return GS_OK;
}
