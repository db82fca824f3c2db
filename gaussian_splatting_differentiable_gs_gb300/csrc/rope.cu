// rope.cu -- gs_rope: rotary positions with several axes.
//
// A pair (u, v) of a head's channels turns by the angle position * frequency:
// (u cos - v sin, u sin + v cos); the inverse turns back, and is the backward
// pass (the rotation is orthogonal).  Angles are phases in 64-bit fractions of
// a turn: position * turns modulo 2^64, whose top 32 bits are the signed phase
// in [-1/2, 1/2), so a large position loses nothing and the sine never needs a
// range reduction.  The angle is the same for every head of a token: a thread
// keeps the sines of its pairs and walks heads.
#include <math.h>
#include <string.h>

#include "net_common.cuh"

namespace gs {
namespace {

struct RopeK {
  uint64_t turns[GS_ROPE_MAX_DIM / 2];
  int32_t dims[GS_ROPE_MAX_AXES];
  int32_t n_axes, head_dim;
  int32_t pairs;             // that rotate
  int32_t rot_units, units;  // units that rotate, and with those that copy
  int32_t head_slots, tokens_per_block;
  float sign;
};

struct HeadsK {
  const char* in;
  char* out;
  int64_t in_token, in_head, out_token, out_head;  // bytes
};

#ifndef HBX
#define HBX 2
#define MB 1
#endif
// Heads a thread loads before it stores any.
template <typename T, int VEC>
constexpr int kBatchOf = VEC * sizeof(T) >= 8 && sizeof(T) == 2 ? HBX : 4;
constexpr int kThreads = 256;

// Sine and cosine of a phase in half turns, [-1, 1).  16-bit heads take the
// fast functions (absolute error below 2^-21 on this range, a sixteenth of the
// rounding of an fp16 result), fp32 heads the accurate ones.
template <typename T>
__device__ __forceinline__ void sine(float half_turns, float* s, float* c) {
  if (sizeof(T) == 4) sincospif(half_turns, s, c);
  else __sincosf(half_turns * 3.14159265358979f, s, c);
}

// A unit is VEC pairs (2 VEC channels) of a head; with VEC = 1 the two channels
// move one by one, so that any stride and an odd last channel are served.  Units
// of neighbouring pairs (INTER) may reach over the sections' ends.  Threads: unit
// fastest (a warp reads neighbouring channels), then head slot, then token.
template <typename T, int VEC, bool INTER>
__global__ void __launch_bounds__(kThreads, VEC * sizeof(T) >= 8 && sizeof(T) == 2 ? MB : 1) rope_kernel(
    int64_t tokens, const __grid_constant__ RopeK k, const __grid_constant__ HeadsK s0,
    const __grid_constant__ HeadsK s1, int heads0, int heads, const int32_t* __restrict__ pos) {
  constexpr int kHeadBatch = kBatchOf<T, VEC>;
  const int u = threadIdx.x % k.units;
  const int y = threadIdx.x / k.units;
  const int hs = y % k.head_slots;
  const int64_t t = (int64_t)blockIdx.x * k.tokens_per_block + y / k.head_slots;
  if (t >= tokens) return;

  // the unit's place: its first pair's section, and its two halves' channels
  int axis = 0, at = 0, before = 0;
  auto seek = [&](int pair) {
    while (axis + 1 < k.n_axes && pair - before >= k.dims[axis] / 2) {
      before += k.dims[axis] / 2;
      at += k.dims[axis];
      ++axis;
    }
  };
  int first = 2 * VEC * u, second = first + VEC;
  if (!INTER && u < k.rot_units) {
    seek(u * VEC);
    first = at + u * VEC - before;
    second = first + k.dims[axis] / 2;
  }
  constexpr bool kWide = INTER && VEC > 1;  // both halves in one access
  const bool two = VEC > 1 || second < k.head_dim;

  Pack<T, VEC> a[kHeadBatch], b[kHeadBatch];
  auto load = [&](int h0) {
#pragma unroll
    for (int i = 0; i < kHeadBatch; ++i) {
      const int h = h0 + i * k.head_slots;
      if (h < heads) {
        const bool in0 = h < heads0;
        const HeadsK& s = in0 ? s0 : s1;
        const T* p = reinterpret_cast<const T*>(s.in + t * s.in_token +
                                                (in0 ? h : h - heads0) * s.in_head);
        if (kWide) {
          const Pack<T, 2 * VEC> w = load_pack<T, 2 * VEC>(p + first);
#pragma unroll
          for (int c = 0; c < VEC; ++c) {
            a[i].v[c] = w.v[2 * c];
            b[i].v[c] = w.v[2 * c + 1];
          }
        } else {
          a[i] = load_pack<T, VEC>(p + first);
          if (two) b[i] = load_pack<T, VEC>(p + second);
        }
      }
    }
  };
  load(hs);  // on its way while the angles are computed

  float co[VEC], si[VEC];
  bool rot[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int pair = u * VEC + i;
    rot[i] = INTER ? pair < k.pairs : u < k.rot_units;
    if (rot[i]) {
      if (INTER) seek(pair);
      const int64_t p = pos[t * k.n_axes + axis];
      const uint64_t phase = (uint64_t)p * k.turns[pair];
      sine<T>((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &si[i], &co[i]);  // 2^-31
      si[i] *= k.sign;
    }
  }

  for (int h0 = hs; h0 < heads; h0 += kHeadBatch * k.head_slots) {
    if (h0 != hs) load(h0);
#pragma unroll
    for (int i = 0; i < kHeadBatch; ++i) {
      const int h = h0 + i * k.head_slots;
      if (h < heads) {
        const bool in0 = h < heads0;
        const HeadsK& s = in0 ? s0 : s1;
        T* p = reinterpret_cast<T*>(s.out + t * s.out_token +
                                    (in0 ? h : h - heads0) * s.out_head);
#pragma unroll
        for (int c = 0; c < VEC; ++c) {
          if (rot[c]) {
            const float x = to_f32(a[i].v[c]), z = to_f32(b[i].v[c]);
            a[i].v[c] = from_f32<T>(x * co[c] - z * si[c]);
            b[i].v[c] = from_f32<T>(x * si[c] + z * co[c]);
          }
        }
        if (kWide) {
          Pack<T, 2 * VEC> w;
#pragma unroll
          for (int c = 0; c < VEC; ++c) {
            w.v[2 * c] = a[i].v[c];
            w.v[2 * c + 1] = b[i].v[c];
          }
          store_pack<T, 2 * VEC>(p + first, w);
        } else {
          store_pack<T, VEC>(p + first, a[i]);
          if (two) store_pack<T, VEC>(p + second, b[i]);
        }
      }
    }
  }
}

template <typename T, bool INTER>
void rope_launch(int vec, dim3 grid, int threads, int64_t tokens, const RopeK& k, const HeadsK& s0,
                 const HeadsK& s1, int heads0, int heads, const int32_t* pos, cudaStream_t st) {
  constexpr int kMax = 16 / (int)sizeof(T) / (INTER ? 2 : 1);
  if (kMax >= 8 && vec == 8)
    rope_kernel<T, kMax >= 8 ? 8 : 1, INTER><<<grid, threads, 0, st>>>(tokens, k, s0, s1, heads0, heads, pos);
  else if (kMax >= 4 && vec == 4)
    rope_kernel<T, kMax >= 4 ? 4 : 1, INTER><<<grid, threads, 0, st>>>(tokens, k, s0, s1, heads0, heads, pos);
  else if (vec == 2)
    rope_kernel<T, 2, INTER><<<grid, threads, 0, st>>>(tokens, k, s0, s1, heads0, heads, pos);
  else
    rope_kernel<T, 1, INTER><<<grid, threads, 0, st>>>(tokens, k, s0, s1, heads0, heads, pos);
}

bool dims_ok(int32_t n_axes, const int32_t* dims, int* sum) {
  if (n_axes < 1 || n_axes > GS_ROPE_MAX_AXES || !dims) return false;
  int64_t s = 0;
  for (int a = 0; a < n_axes; ++a) {
    if (dims[a] < 0 || (dims[a] & 1)) return false;
    s += dims[a];
  }
  *sum = (int)s;
  return s >= 2 && s <= GS_ROPE_MAX_DIM;
}

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" gs_status gs_rope_turns(int32_t n_axes, const int32_t* dims, const double* base,
                                   const double* scale, uint64_t* turns) {
  int sum = 0;
  if (!dims_ok(n_axes, dims, &sum) || !base || !scale || !turns) return GS_ERR_INVALID_ARG;
  for (int a = 0; a < n_axes; ++a)
    if (!(base[a] > 0.0) || !isfinite(base[a]) || !isfinite(scale[a])) return GS_ERR_INVALID_ARG;
  int at = 0;
  for (int a = 0; a < n_axes; ++a)
    for (int j = 0; j < dims[a] / 2; ++j) {
      double f = scale[a] * pow(base[a], -2.0 * j / dims[a]) / (2.0 * M_PI);
      if (!isfinite(f)) return GS_ERR_INVALID_ARG;
      f -= floor(f);  // whole turns do not matter
      const double hi = floor(ldexp(f, 32));
      const double lo = nearbyint(ldexp(ldexp(f, 32) - hi, 32));
      turns[at++] = ((uint64_t)hi << 32) + (uint64_t)lo;
    }
  return GS_OK;
}

extern "C" gs_status gs_rope(int64_t tokens, int32_t n_axes, const int32_t* dims,
                             const uint64_t* turns, int32_t interleaved, int32_t inverse,
                             const int32_t* positions, int32_t head_dim, int32_t dtype,
                             const gs_heads* sets, int32_t n_sets, void* stream) {
  int rot = 0;
  if (tokens < 0 || tokens >= ((int64_t)1 << 31) || !dims_ok(n_axes, dims, &rot) || !turns ||
      rot > head_dim || head_dim > GS_ROPE_MAX_DIM || !dtype_ok(dtype) || !sets || n_sets < 1 ||
      n_sets > 2)
    return GS_ERR_INVALID_ARG;
  const int elem = dtype_size(dtype);
  int64_t heads = 0;
  for (int i = 0; i < n_sets; ++i) {
    if (sets[i].heads < 0 || sets[i].heads > 65536) return GS_ERR_INVALID_ARG;
    heads += sets[i].heads;
  }
  if (tokens == 0 || heads == 0) return GS_OK;
  if (!positions || !aligned4(positions)) return GS_ERR_INVALID_ARG;

  // Pairs per unit: the widest that the sections, the strides and the
  // alignment of every set allow, up to 16 bytes per access.
  const int rest = head_dim - rot;
  int vec = 16 / elem / (interleaved ? 2 : 1);
  auto fits = [&](int v) {
    if (interleaved) {
      if (v > 1 && head_dim % (2 * v)) return false;
    } else {
      for (int a = 0; a < n_axes; ++a)
        if ((dims[a] / 2) % v) return false;
      if (v > 1 && rest % (2 * v)) return false;
    }
    const int64_t bytes = (int64_t)v * elem * (interleaved && v > 1 ? 2 : 1);
    for (int i = 0; i < n_sets; ++i) {
      const gs_heads& s = sets[i];
      if (!s.heads) continue;
      if (!aligned_to(s.in, bytes) || !aligned_to(s.out, bytes)) return false;
      for (int64_t stride : {s.in_token, s.in_head, s.out_token, s.out_head})
        if (stride * elem % bytes) return false;
    }
    return true;
  };
  while (vec > 1 && !fits(vec)) vec /= 2;
  bool copies = false;
  for (int i = 0; i < n_sets; ++i) {
    const gs_heads& s = sets[i];
    if (!s.heads) continue;
    if (!s.in || !s.out || !aligned_to(s.in, elem) || !aligned_to(s.out, elem))
      return GS_ERR_INVALID_ARG;
    copies |= s.in != s.out;
  }
  RopeK k{};
  memcpy(k.turns, turns, sizeof(uint64_t) * (rot / 2));
  for (int a = 0; a < n_axes; ++a) k.dims[a] = dims[a];
  k.n_axes = n_axes;
  k.head_dim = head_dim;
  k.pairs = rot / 2;
  k.rot_units = (int)div_up(rot / 2, vec);
  k.units = copies ? (int)div_up(head_dim, 2 * vec) : k.rot_units;
  k.sign = inverse ? -1.f : 1.f;
  const int rows = kThreads / k.units;  // (token, head slot) pairs of a block
  int slots = (int)div_up(heads, elem == 2 && vec >= 4 ? kBatchOf<__half, 4> : 4);
  k.head_slots = slots < rows ? slots : rows;
  k.tokens_per_block = rows / k.head_slots;
  const int threads = k.units * k.head_slots * k.tokens_per_block;
  const int64_t blocks = div_up(tokens, k.tokens_per_block);
  auto make = [&](const gs_heads& s) {
    return HeadsK{(const char*)s.in, (char*)s.out, s.in_token * elem, s.in_head * elem,
                  s.out_token * elem, s.out_head * elem};
  };
  const HeadsK s0 = make(sets[0]), s1 = make(sets[n_sets - 1]);
  const dim3 grid((unsigned)blocks);
  cudaStream_t st = (cudaStream_t)stream;
#define GS_ROPE(T)                                                                            \
  do {                                                                                        \
    if (interleaved)                                                                          \
      rope_launch<T, true>(vec, grid, threads, tokens, k, s0, s1, sets[0].heads, (int)heads,  \
                           positions, st);                                                    \
    else                                                                                      \
      rope_launch<T, false>(vec, grid, threads, tokens, k, s0, s1, sets[0].heads, (int)heads, \
                            positions, st);                                                   \
  } while (0)
  if (dtype == GS_BF16) GS_ROPE(__nv_bfloat16);
  else if (dtype == GS_F16) GS_ROPE(__half);
  else GS_ROPE(float);
#undef GS_ROPE
  GS_CHECK_LAUNCH();
  return GS_OK;
}
