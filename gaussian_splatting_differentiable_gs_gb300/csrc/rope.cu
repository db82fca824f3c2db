// rope.cu -- gs_rope: rotary positions with several axes.
//
// A pair (u, v) of a head's channels turns by the angle position * frequency:
// (u cos - v sin, u sin + v cos); the inverse turns back, and is the backward
// pass (the rotation is orthogonal).  Angles are phases in 64-bit fractions of
// a turn: position * turns modulo 2^64, whose top 32 bits are the signed phase
// in [-1/2, 1/2), so a large position loses nothing and the sine never needs a
// range reduction.  The angle is the same for every head of a token: a block
// computes the sines of its tokens once, a thread keeps those of its channels and
// walks heads.
//
// One read and one write of the heads.  fp32 heads run at 99 % of the copy rate
// (32640 tokens of 24 heads of 80: 75.6 us).  16-bit heads do not: 32640 tokens of 20
// heads of 64 in bf16 take 43 us where the copy rate would allow 25, with DRAM busy for
// 35 % of it and 53 % of the issue slots used; 72 registers a thread leave 22 warps an
// SM, whose largest stall is the wait for their loads.  A thread has a few pairs
// of a head, as vectors of up to 16 bytes, and finds their places once: blocks
// walk over the tokens.  (With a block per group of tokens, every thread computing
// its own sines, 32640 tokens of 20 heads of 64 in bf16 took 53 us, most of them
// in that set-up.  Vectors of 16 neighbouring bytes, whatever the sections, with
// the partners read a second time, took 62 us.)
#include <math.h>
#include <string.h>

#include "net_common.cuh"

namespace gs {
namespace {

struct RopeK {
  uint64_t turns[GS_ROPE_MAX_DIM / 2];
  int32_t dims[GS_ROPE_MAX_AXES];
  int32_t n_axes, head_dim, rot;  // rot: channels that turn
  float sign;
};

struct HeadsK {
  const char* in;
  char* out;
  int64_t in_token, in_head, out_token, out_head;  // bytes
  int32_t heads;
  int32_t units;                  // of VEC pairs of a head: those that turn, or all
  int32_t slots, block_tokens;    // threads: units x slots x block_tokens
};

// Heads a thread loads before it stores any, and blocks an SM that leave it the
// registers for that (32640 tokens, 20 heads of 64 in bf16: 4 heads and 3 blocks
// 45 us, 4 and 4 47, 4 and 2 52, 2 and 4 45; pairs of neighbours, 16 heads of 96
// in fp16: 2 and 4 51 us, 4 and 3 57).
template <typename T, int VEC, bool INTER>
constexpr int kBatchOf = INTER && VEC * sizeof(T) == 8 && sizeof(T) == 2 ? 2 : 4;
template <typename T, int VEC, bool INTER>
constexpr int kBlocksOf = kBatchOf<T, VEC, INTER> == 2 ? 4 : 3;
// Most pairs a thread: 16 bytes of an fp32 head or of neighbours; of either half
// of a 16-bit head 8 bytes, as 16 take so many registers that less is in flight
// (the same heads in sections of 32: 8 bytes 45 us, 16 bytes 49 to 105).
constexpr int most_pairs(int elem, bool interleaved) { return elem == 4 && interleaved ? 2 : 4; }
constexpr int kThreads = 256;
// Sine and cosine of a phase in half turns, [-1, 1).  16-bit heads take the
// fast functions (absolute error below 2^-21 on this range, a sixteenth of the
// rounding of an fp16 result), fp32 heads the accurate ones.
template <typename T>
__device__ __forceinline__ void sine(float half_turns, float* s, float* c) {
  if (sizeof(T) == 4) sincospif(half_turns, s, c);
  else __sincosf(half_turns * 3.14159265358979f, s, c);
}

// VEC pairs a thread: two vectors of VEC channels, or (neighbours, INTER) one of
// 2 VEC; with VEC = 1 the two channels move one by one, so that any stride and an
// odd last channel are served.  Threads: vector fastest, then head slot, then
// token.
template <typename T, int VEC, bool INTER>
__global__ void __launch_bounds__(kThreads, kBlocksOf<T, VEC, INTER>) rope_kernel(
    int64_t tokens, const __grid_constant__ RopeK k, const __grid_constant__ HeadsK q,
    const __grid_constant__ HeadsK kk, const int32_t* pos) {
  constexpr bool kOne = INTER && VEC > 1;  // both channels in one vector
  constexpr int kHeadBatch = kBatchOf<T, VEC, INTER>;
  __shared__ float2 angles[2][kThreads * VEC];  // [token][pair]: cosine, sine
  const HeadsK& s = blockIdx.y ? kk : q;
  const int threads = s.units * s.slots * s.block_tokens;
  if ((int)threadIdx.x >= threads) return;  // (the larger set's blocks have more)
  const int u = threadIdx.x % s.units, y = threadIdx.x / s.units;
  const int hs = y % s.slots, tok = y / s.slots;
  const int pairs = k.rot / 2;

  // the unit's place: its pairs, and its two halves' channels
  const int pair = u * VEC;
  int first = 2 * VEC * u, second = first + (kOne ? 0 : VEC);
  if (!INTER && pair < pairs) {
    int axis = 0, at = 0;
    while (pair - at / 2 >= k.dims[axis] / 2) at += k.dims[axis++];
    first = at + pair - at / 2;
    second = first + k.dims[axis] / 2;
  }
  const bool two = VEC > 1 || second < k.head_dim;
  // the angle that this thread computes for the block (and every `threads`-th after it)
  auto axis_of = [&](int j) {
    int axis = 0;
    while (j >= k.dims[axis] / 2) j -= k.dims[axis++] / 2;
    return axis;
  };
  const int a_tok = threadIdx.x / pairs, a_pair = threadIdx.x - a_tok * pairs;
  const int a_axis = axis_of(a_pair);
  auto compute = [&](float2* to, int64_t row, int axis, int j) {
    if (row >= tokens) return;
    const int64_t p = pos[row * k.n_axes + axis];
    const uint64_t phase = (uint64_t)p * k.turns[j];
    float2 a;
    sine<T>((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &a.y, &a.x);  // 2^-31
    a.y *= k.sign;
    *to = a;
  };

  launch_dependents();
  wait_for_previous();
  const int64_t in_step = s.in_head * s.slots, out_step = s.out_head * s.slots;
  int turn = 0;
  for (int64_t t0 = (int64_t)blockIdx.x * s.block_tokens; t0 < tokens;
       t0 += (int64_t)gridDim.x * s.block_tokens, turn ^= 1) {
    const int64_t t = t0 + tok;
    const char* in = s.in + t * s.in_token + hs * s.in_head;
    char* out = s.out + t * s.out_token + hs * s.out_head;
    Pack<T, kOne ? 2 * VEC : VEC> a[kHeadBatch], b[kOne ? 1 : kHeadBatch];
    auto load = [&](int left) {
      const char* p = in;
#pragma unroll
      for (int i = 0; i < kHeadBatch; ++i, p += in_step)
        if (i * s.slots < left) {
          a[i] = load_pack<T, kOne ? 2 * VEC : VEC>(reinterpret_cast<const T*>(p) + first);
          if (!kOne && two)
            b[kOne ? 0 : i] = load_pack<T, kOne ? 2 * VEC : VEC>(reinterpret_cast<const T*>(p) + second);
        }
    };
    int left = t < tokens ? s.heads - hs : 0;  // heads from this thread's on
    load(left);  // on its way while the angles are computed
    float2* angle = angles[turn];
    if (a_tok < s.block_tokens) compute(angle + threadIdx.x, t0 + a_tok, a_axis, a_pair);
    for (int i = threadIdx.x + threads; i < s.block_tokens * pairs; i += threads) {
      const int j = i % pairs;
      compute(angle + i, t0 + i / pairs, axis_of(j), j);
    }
    // (two tables in turn: one barrier a round is enough)
    asm volatile("bar.sync 1, %0;" ::"r"((threads + 31) / 32 * 32) : "memory");
    float2 cs[VEC];
#pragma unroll
    for (int c = 0; c < VEC; ++c)
      cs[c] = pair + c < pairs ? angle[tok * pairs + pair + c] : make_float2(1.f, 0.f);
    while (left > 0) {
      char* p = out;
#pragma unroll
      for (int i = 0; i < kHeadBatch; ++i, p += out_step)
        if (i * s.slots < left) {
#pragma unroll
          for (int c = 0; c < VEC; ++c)
            if (pair + c < pairs) {
              T& x = a[i].v[kOne ? 2 * c : c];
              T& z = kOne ? a[i].v[kOne ? 2 * c + 1 : 0] : b[kOne ? 0 : i].v[c];
              const float u0 = to_f32(x), v0 = to_f32(z);
              x = from_f32<T>(u0 * cs[c].x - v0 * cs[c].y);
              z = from_f32<T>(u0 * cs[c].y + v0 * cs[c].x);
            }
          store_pack(reinterpret_cast<T*>(p) + first, a[i]);
          if (!kOne && two) store_pack(reinterpret_cast<T*>(p) + second, b[kOne ? 0 : i]);
        }
      left -= kHeadBatch * s.slots;
      in += kHeadBatch * in_step;
      out += kHeadBatch * out_step;
      load(left);
    }
  }
}

template <typename T, bool INTER>
cudaError_t rope_launch(int vec, dim3 grid, int threads, int64_t tokens, const RopeK& k,
                        const HeadsK& s0, const HeadsK& s1, const int32_t* pos, cudaStream_t st) {
  constexpr int kMost = most_pairs(sizeof(T), INTER);
  if (kMost == 4 && vec == 4)
    return launch_overlapped(rope_kernel<T, kMost, INTER>, grid, threads, 0, st, tokens, k, s0, s1, pos);
  if (vec == 2)
    return launch_overlapped(rope_kernel<T, 2, INTER>, grid, threads, 0, st, tokens, k, s0, s1, pos);
  return launch_overlapped(rope_kernel<T, 1, INTER>, grid, threads, 0, st, tokens, k, s0, s1, pos);
}

// ---- frequencies (host) ----------------------------------------------------
// A number as the sum of two doubles, for about 100 bits: a double's 53 would leave a
// frequency off by 2^-56 of a turn, and the angle at position 2^31 by 1.5e-6.  Sums by
// Knuth's exact addition, products by fma (a rounded product too: one that the compiler
// could fuse with the sum after it would spoil that).
struct Wide {
  double hi, lo;
};
Wide sum2(double a, double b) {  // exact
  const double s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
Wide operator+(Wide a, Wide b) {
  const Wide s = sum2(a.hi, b.hi);
  return sum2(s.hi, s.lo + (a.lo + b.lo));
}
Wide operator*(Wide a, Wide b) {
  const double p = fma(a.hi, b.hi, 0.0);
  return sum2(p, fma(a.hi, b.lo, fma(a.lo, b.hi, fma(a.hi, b.hi, -p))));
}
Wide operator/(Wide a, double b) {
  const double q = a.hi / b;
  return sum2(q, (fma(-q, b, a.hi) + a.lo) / b);
}

// e^x: x less whole powers of two, e^r - 1 = y by its series for r / 512, then nine times
// y (2 + y) for twice the argument.
Wide exp_wide(Wide x) {
  constexpr Wide kLn2{0.6931471805599453, 2.3190468138462996e-17};
  const double k = nearbyint(x.hi / kLn2.hi);
  const Wide part = kLn2 * Wide{-k, 0.0}, r0 = x + part, r{r0.hi / 512.0, r0.lo / 512.0};
  Wide p = r / 9.0 + Wide{1.0, 0.0};  // 1 + r / n (1 + r / (n + 1) (...)), |r| < 7e-4
  for (int n = 8; n >= 2; --n) p = r * p / n + Wide{1.0, 0.0};
  Wide y = r * p;
  for (int i = 0; i < 9; ++i) y = y * (y + Wide{2.0, 0.0});
  y = y + Wide{1.0, 0.0};
  return {ldexp(y.hi, (int)k), ldexp(y.lo, (int)k)};
}
// ln x: the double's logarithm y and, as x e^-y is 1 + d with a small d, d - d^2 / 2.
Wide log_wide(double x) {
  const Wide y{log(x), 0.0};
  // e^-y in two factors: each stays a normal number wherever x is
  const Wide half = exp_wide(Wide{-0.5 * y.hi, 0.0});
  const Wide d = half * (half * Wide{x, 0.0}) + Wide{-1.0, 0.0};
  return y + d + Wide{fma(-0.5 * d.hi, d.hi, 0.0), 0.0};
}

// |scale| base^(-2 j / dim) / 2 pi in turns, times 2^64, modulo 2^64; false where it is not
// a finite number.
bool turns_of(double scale, Wide log_base, int j, int dim, uint64_t* turns) {
  constexpr Wide kTurn{0.15915494309189535, -9.839338337591243e-18};  // 1 / 2 pi
  const Wide e = log_base * Wide{-2.0 * j, 0.0} / dim;
  const Wide f = exp_wide(e) * (kTurn * Wide{fabs(scale), 0.0});
  if (!isfinite(f.hi)) return false;
  const double part = ldexp(f.hi - floor(f.hi), 32), hi = floor(part);  // both exact
  const double lo = nearbyint(ldexp((part - hi) + ldexp(f.lo, 32), 32));
  const uint64_t t = ((uint64_t)hi << 32) + (uint64_t)(int64_t)lo;
  *turns = scale < 0.0 ? 0 - t : t;
  return true;
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
  for (int a = 0; a < n_axes; ++a) {
    const Wide log_base = log_wide(base[a]);
    for (int j = 0; j < dims[a] / 2; ++j)
      if (!turns_of(scale[a], log_base, j, dims[a], &turns[at++])) return GS_ERR_INVALID_ARG;
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

  // Pairs per unit: the widest that the sections, the strides and the alignment
  // of every set allow, up to 16 bytes per access.
  const int rest = head_dim - rot;
  bool copies = false;
  int vec = most_pairs(elem, interleaved);
  auto fits = [&](int v) {
    if (v == 1) return true;
    if (interleaved) {
      if (head_dim % (2 * v)) return false;
    } else {
      for (int a = 0; a < n_axes; ++a)
        if ((dims[a] / 2) % v) return false;
      if (rest % (2 * v)) return false;
    }
    const int64_t bytes = (int64_t)v * elem * (interleaved ? 2 : 1);
    for (int i = 0; i < n_sets; ++i) {
      const gs_heads& s = sets[i];
      if (!s.heads) continue;
      if (!aligned_to(s.in, bytes) || !aligned_to(s.out, bytes)) return false;
      for (int64_t stride : {s.in_token, s.in_head, s.out_token, s.out_head})
        if (stride * elem % bytes) return false;
    }
    return true;
  };
  while (!fits(vec)) vec /= 2;
  for (int i = 0; i < n_sets; ++i) {
    const gs_heads& s = sets[i];
    if (!s.heads) continue;
    if (!s.in || !s.out || !aligned_to(s.in, elem) || !aligned_to(s.out, elem))
      return GS_ERR_INVALID_ARG;
    // in place with other strides, a head would be written before another one is read there
    if (s.in == s.out && ((tokens > 1 && s.in_token != s.out_token) ||
                          (s.heads > 1 && s.in_head != s.out_head)))
      return GS_ERR_INVALID_ARG;
    copies |= s.in != s.out;
  }

  RopeK k{};
  memcpy(k.turns, turns, sizeof(uint64_t) * (rot / 2));
  for (int a = 0; a < n_axes; ++a) k.dims[a] = dims[a];
  k.n_axes = n_axes;
  k.head_dim = head_dim;
  k.rot = rot;
  k.sign = inverse ? -1.f : 1.f;
  const int sms = device_sms();
  HeadsK h[2] = {};
  int n = 0, threads = 32;
  int64_t blocks = 1;
  for (int i = 0; i < n_sets; ++i) {
    const gs_heads& s = sets[i];
    if (!s.heads) continue;
    HeadsK& d = h[n++];
    d = HeadsK{(const char*)s.in, (char*)s.out, s.in_token * elem, s.in_head * elem,
               s.out_token * elem, s.out_head * elem, s.heads, 0, 0, 0};
    d.units = (int)div_up(copies ? head_dim : rot, 2 * vec);
    const int rows = kThreads / d.units;  // (token, head slot) pairs of a block
    d.slots = (int)div_up(s.heads, interleaved && elem == 2 && vec == 4 ? 2 : 4);  // as kBatchOf
    if (d.slots > rows) d.slots = rows;
    d.block_tokens = rows / d.slots;
    const int64_t spread = div_up(tokens, sms);  // few tokens: use every SM
    if (d.block_tokens > spread) d.block_tokens = (int)spread;
    const int need = (int)div_up(d.units * d.slots * d.block_tokens, 32) * 32;
    if (need > threads) threads = need;
    const int64_t want = div_up(tokens, d.block_tokens);
    if (want > blocks) blocks = want;
  }
  // blocks of both sets together: as many as run at once
  const int64_t most = (int64_t)sms * (2048 / threads < 32 ? 2048 / threads : 32) / n;
  if (blocks > most) blocks = most;
  const dim3 grid((unsigned)blocks, n);
  cudaStream_t st = (cudaStream_t)stream;
#define GS_ROPE(T)                                                                         \
  GS_CUDA((interleaved ? rope_launch<T, true> : rope_launch<T, false>)(                    \
      vec, grid, threads, tokens, k, h[0], h[1], positions, st))
  if (dtype == GS_BF16) GS_ROPE(__nv_bfloat16);
  else if (dtype == GS_F16) GS_ROPE(__half);
  else GS_ROPE(float);
#undef GS_ROPE
  return GS_OK;
}
