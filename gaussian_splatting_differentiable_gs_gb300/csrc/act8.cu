// act8.cu -- activation checkpoints in 8 bits: gs_act8_encode, gs_act8_decode
// and the gated unit's two directions (gs_glu_fwd, gs_glu_bwd).
//
// 32 channels share a power-of-two step, so a value q * step is exact in bf16
// and in fp32 and the choice of q is the same in every implementation.  All
// four kernels are single passes.  A lane has eight neighbouring channels (a group
// is four lanes).  Where rows start on 16-byte boundaries the kernels are bound by
// memory (a gated unit of 32640 x 2816 bf16, both directions: 230 us, 6.4 TB/s).
// Where they do not, a lane reads the aligned 16-byte granules that its channels
// touch and shifts them into place; for stores a granule is put together from two
// lanes, and only a run's two ends are written element by element.  That form is
// bound by instructions (8160 x 1361 fp16: 72 us, of which storing is 20, the
// checkpoints 14 and the error function 10).  Loads of single words in place of
// granules: no change; a warp that walks along a row and keeps its last lane's
// words, so that only rows' ends are split: 2 us more.
#include <type_traits>

#include "net_common.cuh"

namespace gs {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;               // channels of a lane
constexpr int kUnitsPerBlock = 2048;  // lanes' worth of work
// Blocks an SM: 48 warps hide the memory latency of the aligned form (both directions
// of a gated unit of 32640 x 2816 bf16: six blocks 230 us, eight 232, five 242); the
// other form needs more registers than that leaves (8160 x 1361 fp16: five 78 us,
// four 80, six 95).
template <bool WIDE>
constexpr int kBlocks = WIDE ? 6 : 5;

struct Act8K {
  int8_t* q;
  uint8_t* e;
  int64_t qs, es;
};

struct RowsK {
  int64_t tokens;
  int32_t C;
  int32_t upr;   // units (lanes) per row, padding included
  int32_t rows;  // rows per block
};

// The larger one; a NaN if there is one (whose bits, without the sign, are above
// any number's).
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// Writes eight channels' bytes and, once per group, the exponent.  Every lane of
// the warp calls it; lanes with c >= end store nothing.
__device__ __forceinline__ void put8(const float (&v)[kPer], const Act8K& k, int64_t t, int c,
                                     int end) {
  float top = fabsf(v[0]);
#pragma unroll
  for (int j = 1; j < kPer; ++j) top = max_nan(top, fabsf(v[j]));
  uint32_t mag = __float_as_uint(top);
  mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 1));
  mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 2));
  if (c >= end) return;
  const uint32_t e = act8_exponent(mag);
  const float inv = act8_inverse(e);
  const uint32_t keep = e == 255u ? 0u : 0xffffffffu;
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __byte_perm(act8_round(v[4 * h], inv), act8_round(v[4 * h + 1], inv), 0x0040);
    const uint32_t hi =
        __byte_perm(act8_round(v[4 * h + 2], inv), act8_round(v[4 * h + 3], inv), 0x0040);
    w[h] = __byte_perm(lo, hi, 0x5410) & keep;
  }
  *reinterpret_cast<uint2*>(k.q + t * k.qs + c) = make_uint2(w[0], w[1]);
  if (c % GS_ACT8_GROUP == 0) k.e[t * k.es + c / GS_ACT8_GROUP] = (uint8_t)e;
}

// Eight channels of a checkpoint as they lie in memory: all of a unit's loads
// are issued before the first value is used.
struct Held8 {
  uint2 q;
  uint32_t e;
};
__device__ __forceinline__ Held8 load8(const Act8K& k, int64_t t, int c) {
  return Held8{*reinterpret_cast<const uint2*>(k.q + t * k.qs + c),
               k.e[t * k.es + c / GS_ACT8_GROUP]};
}
__device__ __forceinline__ float held8(const Held8& h, int j, float step) {
  return act8_value((j < 4 ? h.q.x : h.q.y) ^ 0x80808080u, j & 3, step);
}
// The step for arithmetic in fp32.  From kAct8Top on it is the next number below, which
// makes 64 steps of 2^122 fp32's largest number in place of an infinity (whose product
// with a derivative of 0 would be a NaN); other values of such a group lose a last place
// at most.
__device__ __forceinline__ float held_step(const Held8& h) {
  // signed, with one more in the exponent: 255 (a NaN) is the least then, and stays
  const int bits = (int)((h.e + 1) << 23), top = (int)((kAct8Top<float> + 1) << 23) - 1;
  return __int_as_float(min(bits, top) - (1 << 23));
}

// The first N words of z (N + 4 words) shifted down by s bytes (0 <= s < 16, even).
template <int N>
__device__ __forceinline__ void shift_down(uint32_t (&z)[N + 4], int s) {
#pragma unroll
  for (int i = 0; i < N + 2; ++i) z[i] = s & 8 ? z[i + 2] : z[i];
#pragma unroll
  for (int i = 0; i < N + 1; ++i) z[i] = s & 4 ? z[i + 1] : z[i];
  const int bits = (s & 2) * 8;
#pragma unroll
  for (int i = 0; i < N; ++i) z[i] = __funnelshift_r(z[i], z[i + 1], bits);
}

// A matrix whose rows start anywhere, or (WIDE) on 16-byte boundaries.  `edge`:
// that many first and last rows may lie within 16 bytes of the matrix' ends.
template <typename T>
struct Mat {
  T* p;
  int64_t stride, edge;
};

// Element j of 32-bit words, and two values as a word (fp32: one).
template <typename T>
__device__ __forceinline__ float word_value(const uint32_t* w, int j);
template <>
__device__ __forceinline__ float word_value<float>(const uint32_t* w, int j) {
  return __uint_as_float(w[j]);
}
template <>
__device__ __forceinline__ float word_value<__nv_bfloat16>(const uint32_t* w, int j) {
  return __uint_as_float(j & 1 ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16);
}
template <>
__device__ __forceinline__ float word_value<__half>(const uint32_t* w, int j) {
  return __half2float(__ushort_as_half((unsigned short)(j & 1 ? w[j >> 1] >> 16 : w[j >> 1])));
}
__device__ __forceinline__ uint32_t bits_of(float v) { return __float_as_uint(v); }
__device__ __forceinline__ uint32_t bits_of(__nv_bfloat16 v) { return __bfloat16_as_ushort(v); }
__device__ __forceinline__ uint32_t bits_of(__half v) { return __half_as_ushort(v); }

template <typename T>
__device__ __forceinline__ void words_of(const float (&v)[kPer], uint32_t* w) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) w[j] = __float_as_uint(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < kPer / 2; ++j) w[j] = pair_word<T>(v[2 * j], v[2 * j + 1]);
  }
}

// Eight channels of a matrix from c on (zeros from C on); c < C.
template <typename T, bool WIDE>
struct Held {
  static constexpr int kWords = kPer * sizeof(T) / 4;
  uint32_t w[kWords + (WIDE ? 0 : 4)];
  __device__ __forceinline__ void load(const Mat<const T>& m, const RowsK& r, int64_t t, int c) {
    const T* p = m.p + t * m.stride + c;
    if constexpr (WIDE) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) granule(i, reinterpret_cast<const uint4*>(p) + i / 4);
    } else {
      const int n = min(kPer, r.C - c) * (int)sizeof(T);
      // granules reach up to 14 bytes out of the row: not out of the matrix
      if ((c > 0 || t >= m.edge) && (c + 2 * kPer <= r.C || t < r.tokens - m.edge)) {
        const int d = (int)((uintptr_t)p & 15);
        const char* g = (const char*)p - d;
#pragma unroll
        for (int i = 0; i < kWords + 4; i += 4) {
          w[i] = w[i + 1] = w[i + 2] = w[i + 3] = 0;
          if (4 * i < d + n) granule(i, reinterpret_cast<const uint4*>(g) + i / 4);
        }
        shift_down<kWords>(w, d);
        if (n < 4 * kWords) {
#pragma unroll
          for (int i = 0; i < kWords; ++i)
            w[i] = 4 * i + 4 <= n ? w[i] : 4 * i < n ? w[i] & 0xffffu : 0u;
        }
      } else {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (c + i < r.C)
            w[i * (int)sizeof(T) / 4] |= bits_of(p[i]) << (sizeof(T) == 2 && (i & 1) ? 16 : 0);
      }
    }
  }
  __device__ __forceinline__ float value(int j) const { return word_value<T>(w, j); }

 private:
  __device__ __forceinline__ void granule(int i, const uint4* g) {
    const uint4 v = *g;
    w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
  }
};

// Stores eight channels from c on, those below C.  Every lane of the warp calls
// it; `in`: c < C.
template <typename T, bool WIDE>
__device__ __forceinline__ void put(const float (&v)[kPer], const Mat<T>& m, const RowsK& r,
                                    int64_t t, int c, bool in) {
  constexpr int kWords = kPer * sizeof(T) / 4;
  T* p = m.p + t * m.stride + c;
  if constexpr (WIDE) {
    if (in) {
      uint32_t w[kWords];
      words_of<T>(v, w);
#pragma unroll
      for (int i = 0; i < kWords; i += 4)
        reinterpret_cast<uint4*>(p)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    }
    return;
  }
  uint32_t own[kWords], w[kWords + 4];
  words_of<T>(v, own);
#pragma unroll
  for (int i = 0; i < kWords; ++i) w[4 + i] = own[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __shfl_up_sync(0xffffffffu, w[kWords + i], 1);
  if (!in) return;
  const int lane = threadIdx.x & 31;
  const int d = (int)((uintptr_t)p & 15), n = min(kPer, r.C - c) * (int)sizeof(T);
  // prev: the lane before has this row's channels before c; next: the lane after
  // has enough of the row to store the granule that this lane's last bytes are in
  const bool prev = lane > 0 && c > 0;
  const bool next = lane < 31 && min(kPer, r.C - c - kPer) * (int)sizeof(T) >= 16 - d;
  if (d) {
    shift_down<kWords>(w, 16 - d);
  } else {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = own[i];
  }
  char* g = (char*)p - d;  // granule i: bytes [16 i, 16 i + 16) from here
  int lo = 0, hi = next ? n : min(n, 4 * kWords - d);  // own bytes [0, lo), [hi, n): one by one
  if (d && !prev) lo = min(16 - d, n);
#pragma unroll
  for (int i = 0; i < kWords / 4; ++i) {
    if (16 * (i + 1) - d <= n) {
      if (i > 0 || !d || prev)
        *reinterpret_cast<uint4*>(g + 16 * i) =
            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else {
      hi = min(hi, max(16 * i - d, 0));  // the row ends inside this granule
    }
  }
  if (lo > 0 || hi < n) {
    using U = typename std::conditional<sizeof(T) == 4, uint32_t, uint16_t>::type;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int b = j * (int)sizeof(T);
      if (b < n && (b < lo || b >= hi))
        reinterpret_cast<U*>(p)[j] = (U)(own[b / 4] >> (b % 4 * 8));
    }
  }
}

// Runs f(t, c, end) for the block's units, c the lane's first channel and end
// the row's width with its padding (0 for lanes with nothing to do); whole
// warps take part in each step.
template <typename F>
__device__ __forceinline__ void each_unit(const RowsK& r, F f) {
  launch_dependents();
  wait_for_previous();
  const int64_t row0 = (int64_t)blockIdx.x * r.rows;
  const int n = r.upr * (int)min((int64_t)r.rows, r.tokens - row0);
  const int end = (r.C + GS_ACT8_GROUP - 1) / GS_ACT8_GROUP * GS_ACT8_GROUP;
  const int lane = threadIdx.x & 31;
  const int rows = kThreads / r.upr, units = kThreads - rows * r.upr;  // of one step
  int row = (int)threadIdx.x / r.upr, unit = (int)threadIdx.x - row * r.upr;
  for (int at = threadIdx.x; at - lane < n; at += kThreads) {
    f(row0 + row, unit * kPer, at < n ? end : 0);
    row += rows;
    unit += units;
    if (unit >= r.upr) unit -= r.upr, ++row;
  }
}

template <typename T, bool WIDE>
__global__ void __launch_bounds__(kThreads, kBlocks<WIDE>)
    encode_kernel(RowsK r, Mat<const T> x, Act8K k) {
  each_unit(r, [&](int64_t t, int c, int end) {
    float v[kPer] = {};
    if (c < min(r.C, end)) {
      Held<T, WIDE> h;
      h.load(x, r, t, c);
#pragma unroll
      for (int j = 0; j < kPer; ++j) v[j] = h.value(j);
    }
    put8(v, k, t, c, end);
  });
}

template <typename T, bool WIDE>
__global__ void __launch_bounds__(kThreads, kBlocks<WIDE>)
    decode_kernel(RowsK r, Act8K k, Mat<T> x) {
  each_unit(r, [&](int64_t t, int c, int end) {
    const bool in = c < min(r.C, end);
    float v[kPer];
    if (in) {
      const Held8 h = load8(k, t, c);
#pragma unroll
      for (int j = 0; j < kPer; ++j) v[j] = held8(h, j, act8_step(h.e));
      if (h.e >= kAct8Top<T> && h.e < 255u) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[j] = act8_within<T>(v[j], held8(h, j, 1.f), act8_step(h.e));
      }
    }
    put<T, WIDE>(v, x, r, t, c, in);
  });
}

// 2^v and 1 / v as the hardware's single instructions; results and arguments below
// 2^-126 count as zero, which is below the error of every use here.
__device__ __forceinline__ float power2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float reciprocal(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Phi and its density for two values.  16-bit types take Abramowitz and Stegun's formula
// 7.1.26 for the error function, which needs the one exponential that the derivative has
// too; in this arithmetic Phi is off by up to 2.6e-7, a thousandth of fp16's rounding of
// values near 1 (in the tail, where Phi is small, by up to a third of itself: below that
// rounding of v Phi's terms).  It takes two values an instruction (8160 x 1361 fp16: 72 us,
// 75 without).  The same elsewhere in these kernels costs the aligned form registers, and
// thereby warps: 238 us in place of 230 at 32640 x 2816 bf16.  fp32 takes the complementary
// error function, which keeps its relative accuracy in the tail.
struct Phi {
  float2 p, density;  // Phi(v), phi(v)
};
template <typename T>
__device__ __forceinline__ Phi normal(float2 v) {
  if constexpr (sizeof(T) == 4) {
    const float2 w = mul2(mul2(v, v), both(-0.72134752044448170f));  // -v^2 / 2 in powers of two
    return Phi{make_float2(0.5f * erfcf(v.x * -0.70710678118654752f),
                           0.5f * erfcf(v.y * -0.70710678118654752f)),
               mul2(make_float2(power2(w.x), power2(w.y)), both(0.39894228040143268f))};
  } else {
    const float2 z = make_float2(fabsf(v.x) * 0.70710678118654752f, fabsf(v.y) * 0.70710678118654752f);
    const float2 y = fma2(both(0.3275911f), z, both(1.f));
    const float2 t = make_float2(reciprocal(y.x), reciprocal(y.y));
    const float2 w = mul2(mul2(z, z), both(-1.4426950408889634f));
    const float2 ex = make_float2(power2(w.x), power2(w.y));
    float2 q = fma2(both(0.5f * 1.061405429f), t, both(0.5f * -1.453152027f));
    q = fma2(q, t, both(0.5f * 1.421413741f));
    q = fma2(q, t, both(0.5f * -0.284496736f));
    q = fma2(q, t, both(0.5f * 0.254829592f));
    const float2 tail = mul2(mul2(q, t), ex), rest = fma2(tail, both(-1.f), both(1.f));
    return Phi{make_float2(v.x < 0.f ? tail.x : rest.x, v.y < 0.f ? tail.y : rest.y),
               mul2(ex, both(0.39894228040143268f))};
  }
}
// act(v) and its derivative for two values.
__device__ __forceinline__ float sigmoid(float v) {
  return reciprocal(1.f + power2(v * -1.4426950408889634f));
}
template <typename T, int ACT>
__device__ __forceinline__ float2 act_value(float2 v) {
  if (ACT == GS_ACT_SILU) return make_float2(v.x * sigmoid(v.x), v.y * sigmoid(v.y));
  return mul2(v, normal<T>(v).p);
}
template <typename T, int ACT>
__device__ __forceinline__ void act_both(float2 v, float2& f, float2& df) {
  if (ACT == GS_ACT_SILU) {
    const float s = sigmoid(v.x), u = sigmoid(v.y);
    f = make_float2(v.x * s, v.y * u);
    df = make_float2(s * (1.f + v.x * (1.f - s)), u * (1.f + v.y * (1.f - u)));
  } else {
    const Phi n = normal<T>(v);
    f = mul2(v, n.p);
    df = fma2(v, n.density, n.p);
  }
}

template <typename T, bool WIDE, int ACT, bool GATED>
__global__ void __launch_bounds__(kThreads, kBlocks<WIDE>)
    glu_fwd_kernel(RowsK r, Mat<const T> gate, Mat<const T> up, Mat<T> h, Act8K g8, Act8K u8) {
  each_unit(r, [&](int64_t t, int c, int end) {
    const bool in = c < min(r.C, end);
    float g[kPer] = {}, u[kPer] = {}, o[kPer];
    if (in) {
      Held<T, WIDE> hg, hu;
      hg.load(gate, r, t, c);
      if (GATED) hu.load(up, r, t, c);
#pragma unroll
      for (int j = 0; j < kPer; j += 2) {
        const float2 a = make_float2(hg.value(j), hg.value(j + 1));
        float2 f = act_value<T, ACT>(a);
        g[j] = a.x, g[j + 1] = a.y;
        if (GATED) {
          const float2 b = make_float2(hu.value(j), hu.value(j + 1));
          u[j] = b.x, u[j + 1] = b.y;
          f.x *= b.x, f.y *= b.y;
        }
        o[j] = f.x, o[j + 1] = f.y;
      }
      if (WIDE) put<T, WIDE>(o, h, r, t, c, in);
    }
    if (!WIDE) put<T, WIDE>(o, h, r, t, c, in);
    if (g8.q) put8(g, g8, t, c, end);
    if (GATED && u8.q) put8(u, u8, t, c, end);
  });
}

template <typename T, bool WIDE, int ACT, bool GATED>
__global__ void __launch_bounds__(kThreads, kBlocks<WIDE>)
    glu_bwd_kernel(RowsK r, Act8K g8, Act8K u8, Mat<const T> dh, Mat<T> dgate, Mat<T> dup,
                   Act8K h8) {
  each_unit(r, [&](int64_t t, int c, int end) {
    const bool in = c < min(r.C, end);
    float dg[kPer], du[kPer], o[kPer] = {};
    if (in) {
      const Held8 hg = load8(g8, t, c), hu = GATED ? load8(u8, t, c) : Held8{};
      const float sg = held_step(hg), su = held_step(hu);
      Held<T, WIDE> hd;
      hd.load(dh, r, t, c);
#pragma unroll
      for (int j = 0; j < kPer; j += 2) {
        float2 f, df;
        act_both<T, ACT>(make_float2(held8(hg, j, sg), held8(hg, j + 1, sg)), f, df);
        const float2 d = make_float2(hd.value(j), hd.value(j + 1));
        const float2 w = GATED ? make_float2(held8(hu, j, su), held8(hu, j + 1, su)) : both(1.f);
        o[j] = WIDE || c + j < r.C ? f.x * w.x : 0.f;
        o[j + 1] = WIDE || c + j + 1 < r.C ? f.y * w.y : 0.f;
        dg[j] = d.x * w.x * df.x, dg[j + 1] = d.y * w.y * df.y;
        du[j] = d.x * f.x, du[j + 1] = d.y * f.y;
      }
      if (WIDE) {
        put<T, WIDE>(dg, dgate, r, t, c, in);
        if (GATED) put<T, WIDE>(du, dup, r, t, c, in);
      }
    }
    if (!WIDE) {
      put<T, WIDE>(dg, dgate, r, t, c, in);
      if (GATED) put<T, WIDE>(du, dup, r, t, c, in);
    }
    if (h8.q) put8(o, h8, t, c, end);
  });
}

RowsK make_rows(int64_t tokens, int32_t C) {
  RowsK r{tokens, C, (int32_t)div_up(C, GS_ACT8_GROUP) * (GS_ACT8_GROUP / kPer), 1};
  r.rows = r.upr >= kUnitsPerBlock ? 1 : kUnitsPerBlock / r.upr;
  const int64_t spread = div_up(tokens, (int64_t)device_sms() * 4);  // few tokens: use every SM
  if (r.rows > spread) r.rows = (int32_t)spread;
  return r;
}

unsigned blocks_of(const RowsK& r) { return (unsigned)div_up(r.tokens, r.rows); }

bool shape_ok(int64_t tokens, int32_t C, int32_t dtype) {
  return tokens >= 0 && tokens < ((int64_t)1 << 31) && C >= 1 && C <= (1 << 24) && dtype_ok(dtype);
}
bool ckpt_ok(const Act8K& k, int64_t tokens, int32_t C) {
  return gs::ckpt_ok(tokens, C, k.q, k.qs, k.e, k.es);
}
Act8K ckpt_of(const gs_ckpt* c) {
  return c ? Act8K{c->q, c->e, c->q_stride, c->e_stride} : Act8K{nullptr, nullptr, 0, 0};
}

template <typename T>
Mat<T> mat_of(T* p, int64_t stride, int32_t C) {
  const int64_t apart = stride >= C ? stride * (int64_t)sizeof(T) : 0;
  return {p, stride, apart ? div_up(16, apart) : (int64_t)1 << 31};
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
  if (!x || !aligned_to(x, el) || !ckpt_ok(k, tokens, channels)) return GS_ERR_INVALID_ARG;
  const bool wide = channels % 8 == 0 && rows_aligned(x, x_stride, el, 16);
  const RowsK r = make_rows(tokens, channels);
  cudaStream_t st = (cudaStream_t)stream;
  GS_ACT8_TYPES(dtype, const Mat<const T> m = mat_of((const T*)x, x_stride, channels);
                GS_CUDA(launch_overlapped(wide ? encode_kernel<T, true> : encode_kernel<T, false>,
                                          blocks_of(r), kThreads, 0, st, r, m, k)));
  return GS_OK;
}

extern "C" gs_status gs_act8_decode(int64_t tokens, int32_t channels, int32_t dtype,
                                    const int8_t* q, int64_t q_stride, const uint8_t* e,
                                    int64_t e_stride, void* x, int64_t x_stride, void* stream) {
  if (!shape_ok(tokens, channels, dtype)) return GS_ERR_INVALID_ARG;
  if (tokens == 0) return GS_OK;
  const Act8K k{const_cast<int8_t*>(q), const_cast<uint8_t*>(e), q_stride, e_stride};
  const int el = dtype_size(dtype);
  if (!x || !aligned_to(x, el) || !ckpt_ok(k, tokens, channels)) return GS_ERR_INVALID_ARG;
  const bool wide = channels % 8 == 0 && rows_aligned(x, x_stride, el, 16);
  const RowsK r = make_rows(tokens, channels);
  cudaStream_t st = (cudaStream_t)stream;
  GS_ACT8_TYPES(dtype, const Mat<T> m = mat_of((T*)x, x_stride, channels);
                GS_CUDA(launch_overlapped(wide ? decode_kernel<T, true> : decode_kernel<T, false>,
                                          blocks_of(r), kThreads, 0, st, r, k, m)));
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
      (g8.q && !ckpt_ok(g8, tokens, channels)) || (u8.q && (!up || !ckpt_ok(u8, tokens, channels))))
    return GS_ERR_INVALID_ARG;
  const bool wide = channels % 8 == 0 && rows_aligned(gate, gate_stride, el, 16) &&
                    rows_aligned(up, up_stride, el, 16) && rows_aligned(h, h_stride, el, 16);
  const RowsK r = make_rows(tokens, channels);
  cudaStream_t st = (cudaStream_t)stream;
#define GS_GLU(WIDE, ACT)                                                                    \
  do {                                                                                       \
    const Mat<const T> mg = mat_of((const T*)gate, gate_stride, channels);                   \
    const Mat<const T> mu = mat_of((const T*)up, up_stride, channels);                       \
    const Mat<T> mh = mat_of((T*)h, h_stride, channels);                                     \
    GS_CUDA(launch_overlapped(up ? glu_fwd_kernel<T, WIDE, ACT, true>                        \
                                  : glu_fwd_kernel<T, WIDE, ACT, false>,                     \
                              blocks_of(r), kThreads, 0, st, r, mg, mu, mh, g8, u8));        \
  } while (0)
  GS_ACT8_TYPES(dtype, if (act == GS_ACT_SILU) {
    if (wide) GS_GLU(true, GS_ACT_SILU); else GS_GLU(false, GS_ACT_SILU);
  } else {
    if (wide) GS_GLU(true, GS_ACT_GELU); else GS_GLU(false, GS_ACT_GELU);
  });
#undef GS_GLU
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
  if (!ckpt_ok(g8, tokens, channels) || (u8.q && !ckpt_ok(u8, tokens, channels)) ||
      (o8.q && !ckpt_ok(o8, tokens, channels)) || (!u8.q != !dup) || !dh || !dgate ||
      !aligned_to(dh, el) || !aligned_to(dgate, el) || !aligned_to(dup, el) ||
      !in_place_ok(tokens, dh, dh_stride, dgate, dgate_stride) ||
      !in_place_ok(tokens, dh, dh_stride, dup, dup_stride))
    return GS_ERR_INVALID_ARG;
  const bool wide = channels % 8 == 0 && rows_aligned(dh, dh_stride, el, 16) &&
                    rows_aligned(dgate, dgate_stride, el, 16) &&
                    rows_aligned(dup, dup_stride, el, 16);
  const RowsK r = make_rows(tokens, channels);
  cudaStream_t st = (cudaStream_t)stream;
#define GS_GLU(WIDE, ACT)                                                                    \
  do {                                                                                       \
    const Mat<const T> md = mat_of((const T*)dh, dh_stride, channels);                       \
    const Mat<T> mg = mat_of((T*)dgate, dgate_stride, channels);                             \
    const Mat<T> mu = mat_of((T*)dup, dup_stride, channels);                                 \
    GS_CUDA(launch_overlapped(dup ? glu_bwd_kernel<T, WIDE, ACT, true>                       \
                                   : glu_bwd_kernel<T, WIDE, ACT, false>,                    \
                              blocks_of(r), kThreads, 0, st, r, g8, u8, md, mg, mu, o8));    \
  } while (0)
  GS_ACT8_TYPES(dtype, if (act == GS_ACT_SILU) {
    if (wide) GS_GLU(true, GS_ACT_SILU); else GS_GLU(false, GS_ACT_SILU);
  } else {
    if (wide) GS_GLU(true, GS_ACT_GELU); else GS_GLU(false, GS_ACT_GELU);
  });
#undef GS_GLU
  return GS_OK;
}
