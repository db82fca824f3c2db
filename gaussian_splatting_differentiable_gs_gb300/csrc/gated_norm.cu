// gated_norm.cu -- gs_gated_norm_fwd and gs_gated_norm_bwd: the join of two
// blocks of a residual network.
//
//   u = w_post N(b);  x' = x + s g u;  y = w_pre N(x')
//
// Forward: a row lives in the registers of a team of warps between its one
// read and its one write; the statistics are those of the unrounded sum.
// Backward, with n = N(x'), m = N(b), h = dy w_pre, k = s g w_post:
//   d  = dx' + r_x (h - n mean(h n) [- mean(h)])
//   db = r_b (d k - m mean(d k m) [- mean(d k)]),   dx = d
// and the sums over rows need two column sums only: dw_pre = sum_t dy n, and
// per gate group e_G = sum_{t in G} d m, from which dw_post = sum_G s g_G e_G,
// dres_scale = sum_G g_G w_post e_G and dgate_G = s w_post e_G.
#include <atomic>

#include "net_common.cuh"

namespace gs {
namespace {

constexpr int kNormCtas = 304;      // most row ranges of the backward (column sums)
constexpr int kMaxTeamWarps = 16;
constexpr int kTeamThreads = 512;   // most threads of a CTA
constexpr int kSmemBudget = 224 * 1024;

struct NormK {
  int64_t tokens;
  int32_t C, groups;
  int32_t post, center;
  float eps, inv_c;
  const float *w_pre, *w_post, *scale;
  const void* gate;
  const int32_t* offsets;
};

// Sums of one or two values per thread over a team of `warps` warps, the same
// bits in every thread.  red: two slots of 2 kMaxTeamWarps floats per team,
// used in turn: a slot is written again only after the barrier of the sum in
// between.
struct TeamSum {
  float* red;
  int warps, warp, bar;
  int turn;
  __device__ __forceinline__ void operator()(float& a, float& b, bool both) {
#pragma unroll
    for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if (both) {
#pragma unroll
      for (int o = 16; o; o >>= 1) b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (warps == 1) return;
    float2* r = reinterpret_cast<float2*>(red) + (turn & 1) * kMaxTeamWarps;
    ++turn;
    if ((threadIdx.x & 31) == 0) r[warp] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(warps * 32) : "memory");
    a = b = 0.f;
    for (int i = 0; i < warps; ++i) {
      const float2 v = r[i];
      a += v.x;
      b += v.y;
    }
  }
  __device__ __forceinline__ float operator()(float v) {
    float none = 0.f;
    (*this)(v, none, false);
    return v;
  }
};

__device__ __forceinline__ int find_group(const int32_t* offsets, int groups, int64_t t) {
  if (!offsets) return 0;
  int lo = 0, hi = groups - 1;  // the last group that starts at or before t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (offsets[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// A thread's share of the rows to come.  Rows whose vectors are 4 or 16 bytes
// are copied asynchronously into shared memory, kDepth - 1 rows ahead; every
// thread copies what it reads itself, so nothing but its own copies is waited
// for.  Single 16-bit values (rows that start anywhere) cannot be copied so:
// they are held in registers, one row ahead.
template <typename T, int VEC, int NV>
struct Rows {
  static constexpr int kChunk = VEC * sizeof(T) >= 16 ? 16 : VEC * sizeof(T);
  static constexpr int kPer = VEC * sizeof(T) / kChunk, kChunks = NV * kPer;
  static constexpr bool kRing = kChunk >= 4;
  static constexpr int kBytes = kRing ? kChunks * kChunk : 0;  // per thread and row

  const T* base;  // NULL: zeros
  int64_t stride;
  T held[kRing ? 1 : VEC * NV];

  __device__ __forceinline__ void fetch(char* slot, int64_t t, int first, int step, int C) {
    if (!kRing || !base) return;
    const T* p = base + t * stride;
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(slot) + threadIdx.x * kChunk;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = first + i / kPer * step + i % kPer * (kChunk / (int)sizeof(T));
      if (c < C) {
        if (kChunk == 16)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                           to + i * (int)blockDim.x * kChunk),
                       "l"(p + c)
                       : "memory");
        else
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                           to + i * (int)blockDim.x * kChunk),
                       "l"(p + c)
                       : "memory");
      }
    }
  }
  __device__ __forceinline__ void hold(int64_t t, int first, int step, int C) {
    if (kRing || !base) return;
    const T* p = base + t * stride;
#pragma unroll
    for (int i = 0; i < (kRing ? 0 : VEC * NV); ++i)
      if (first + i * step < C) held[i] = p[first + i * step];
  }
  __device__ __forceinline__ void read(float (&v)[VEC * NV], const char* slot, int first, int step,
                                       int C) const {
    constexpr int kEl = kChunk / (int)sizeof(T);
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = first + i / kPer * step + i % kPer * kEl;
      if (base && c < C) {
        if (kRing) {
          const Pack<T, kEl> w = load_pack<T, kEl>(reinterpret_cast<const T*>(
              slot + (i * (int)blockDim.x + (int)threadIdx.x) * kChunk));
#pragma unroll
          for (int j = 0; j < kEl; ++j) v[i * kEl + j] = to_f32(w.v[j]);
        } else {
          v[i] = to_f32(held[i]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < kEl; ++j) v[i * kEl + j] = 0.f;
      }
    }
  }
};

template <int N>
__device__ __forceinline__ void copies_done_but() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}

template <typename T, int VEC, int NV>
__device__ __forceinline__ void store_row(const float (&v)[VEC * NV], T* p, int first, int step,
                                          int C) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = first + i * step;
    if (c < C) {
      Pack<T, VEC> w;
#pragma unroll
      for (int j = 0; j < VEC; ++j) w.v[j] = from_f32<T>(v[i * VEC + j]);
      store_pack<T, VEC>(p + c, w);
    }
  }
}

// v *= p[channel] (fp32 weights; NULL: ones)
template <typename T, int VEC, int NV>
__device__ __forceinline__ void scale_row(float (&v)[VEC * NV], const T* p, int first, int step,
                                          int C) {
  if (!p) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = first + i * step;
    if (c < C) {
      const Pack<T, VEC> w = load_pack<T, VEC>(p + c);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i * VEC + j] *= to_f32(w.v[j]);
    }
  }
}

// mean and 1/deviation of a row held by a team; v becomes the centred row.
template <int VEC, int NV>
__device__ __forceinline__ void row_stats(float (&v)[VEC * NV], TeamSum& sum, const NormK& k,
                                          int first, int step, float& mean, float& rstd) {
  mean = 0.f;
  if (k.center) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < VEC * NV; ++i) s += v[i];
    mean = sum(s) * k.inv_c;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (first + i * step < k.C) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[i * VEC + j] -= mean;
      }
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < VEC * NV; ++i) s += v[i] * v[i];
  rstd = rsqrtf(sum(s) * k.inv_c + k.eps);
}

// k = res_scale * gate * w_post of a group, per channel
template <typename TB, int VEC, int NV>
__device__ __forceinline__ void group_weights(float (&wk)[VEC * NV], const NormK& k, int g,
                                              int first, int step) {
#pragma unroll
  for (int i = 0; i < VEC * NV; ++i) wk[i] = 1.f;
  scale_row<float, VEC, NV>(wk, k.scale, first, step, k.C);
  if (k.post) scale_row<float, VEC, NV>(wk, k.w_post, first, step, k.C);
  if (k.gate) scale_row<TB, VEC, NV>(wk, (const TB*)k.gate + (int64_t)g * k.C, first, step, k.C);
}

// A CTA takes rows [cta R, cta R + R); its teams take them in turn and keep the
// weights of their channels in registers.
template <typename TB, typename TX, int VEC, int NV, int DEPTH>
__global__ void __launch_bounds__(kTeamThreads, VEC * NV <= 8 ? 2 : 1) norm_fwd_kernel(
    const __grid_constant__ NormK k, const TX* x, int64_t x_stride, const TB* block,
    int64_t block_stride, TX* x_out, int64_t x_out_stride, TB* y, int64_t y_stride, float4* stats,
    int8_t* y_q, int64_t q_stride, uint8_t* y_e, int64_t e_stride, int64_t rows_per_cta,
    int warps) {
  extern __shared__ __align__(16) char smem[];
  constexpr int E = VEC * NV;
  using RX = Rows<TX, VEC, NV>;
  using RB = Rows<TB, VEC, NV>;
  const int warp = threadIdx.x >> 5;
  const int team = warp / warps, teams = (blockDim.x >> 5) / warps;
  const int slot_bytes = (RX::kBytes + RB::kBytes) * blockDim.x;
  TeamSum sum{reinterpret_cast<float*>(smem + DEPTH * slot_bytes) + team * 4 * kMaxTeamWarps, warps,
              warp - team * warps, team + 1, 0};
  const int lane = threadIdx.x - team * warps * 32;
  const int first = lane * VEC, step = warps * 32 * VEC;

  const int64_t begin = (int64_t)blockIdx.x * rows_per_cta + team;
  const int64_t end = min((int64_t)(blockIdx.x + 1) * rows_per_cta, k.tokens);
  RX rx{x, x_stride};
  RB rb{block, block_stride};
  auto ask = [&](int s, int64_t t) {
    if (t < end) {
      rx.fetch(smem + s * slot_bytes, t, first, step, k.C);
      rb.fetch(smem + s * slot_bytes + RX::kBytes * blockDim.x, t, first, step, k.C);
    }
    copies_commit();
  };
  auto hold = [&](int64_t t) {
    if (t < end) {
      rx.hold(t, first, step, k.C);
      rb.hold(t, first, step, k.C);
    }
  };
#pragma unroll
  for (int i = 0; i < DEPTH - 1; ++i) ask(i, begin + (int64_t)i * teams);
  hold(begin);

  float wp[E], wk[E];
#pragma unroll
  for (int i = 0; i < E; ++i) wp[i] = 1.f;
  scale_row<float, VEC, NV>(wp, k.w_pre, first, step, k.C);
  int g = -1;
  int64_t group_end = 0;

  int s = 0;
  for (int64_t t = begin; t < end; t += teams) {
    copies_done_but<DEPTH - 2>();
    float v[E], u[E];
    rx.read(v, smem + s * slot_bytes, first, step, k.C);
    rb.read(u, smem + s * slot_bytes + RX::kBytes * blockDim.x, first, step, k.C);
    ask(s == 0 ? DEPTH - 1 : s - 1, t + (int64_t)(DEPTH - 1) * teams);
    hold(t + teams);
    s = s + 1 == DEPTH ? 0 : s + 1;
    float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
    if (block) {
      if (g < 0 || t >= group_end) {
        g = find_group(k.offsets, k.groups, t);
        group_end = k.offsets && g + 1 < k.groups ? k.offsets[g + 1] : k.tokens;
        group_weights<TB, VEC, NV>(wk, k, g, first, step);
      }
      if (k.post) {
        row_stats<VEC, NV>(u, sum, k, first, step, st.x, st.y);
#pragma unroll
        for (int i = 0; i < E; ++i) u[i] *= st.y;
      }
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] += wk[i] * u[i];
      store_row<TX, VEC, NV>(v, x_out + t * x_out_stride, first, step, k.C);
    }
    if (y) {
      row_stats<VEC, NV>(v, sum, k, first, step, st.z, st.w);
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] *= st.w * wp[i];
      store_row<TB, VEC, NV>(v, y + t * y_stride, first, step, k.C);
      if (y_q) {
        // the checkpoint of y as stored; a group is 32 / VEC lanes of a warp
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          uint32_t mag = 0;
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            v[i * VEC + j] = to_f32(from_f32<TB>(v[i * VEC + j]));
            mag = max(mag, __float_as_uint(v[i * VEC + j]) & 0x7fffffffu);
          }
#pragma unroll
          for (int o = 1; o < GS_ACT8_GROUP / VEC; o <<= 1)
            mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, o));
          const uint32_t e = act8_exponent(mag);
          const float inv = act8_inverse(e);
          const int c = first + i * step;
          if (c < (k.C + GS_ACT8_GROUP - 1) / GS_ACT8_GROUP * GS_ACT8_GROUP) {
            Pack<int8_t, VEC> q;
#pragma unroll
            for (int j = 0; j < VEC; ++j) q.v[j] = (int8_t)act8_quantise(v[i * VEC + j], inv, e);
            store_pack<int8_t, VEC>(y_q + t * q_stride + c, q);
            if (c % GS_ACT8_GROUP == 0) y_e[t * e_stride + c / GS_ACT8_GROUP] = (uint8_t)e;
          }
        }
      }
    }
    if (lane == 0) stats[t] = st;
  }
}

// Rows as in the forward, cut at the groups' ends, with the column sums in
// registers.  The sums of a (CTA, group) pair go to slot cta + group of part_e:
// along the rows either the CTA or the group advances, so no two pairs share a
// slot.
template <typename TB, typename TX, int VEC, int NV, int DEPTH>
__global__ void __launch_bounds__(kTeamThreads, 1) norm_bwd_kernel(
    const __grid_constant__ NormK k, const TX* x, int64_t x_stride, const TB* block,
    int64_t block_stride, const float4* stats, const TX* dx_out, int64_t dx_out_stride,
    const TB* dy, int64_t dy_stride, TX* dx, int64_t dx_stride, TB* dblock, int64_t dblock_stride,
    float* part_pre, float* part_e, int64_t rows_per_cta, int warps) {
  extern __shared__ __align__(16) char smem[];
  constexpr int E = VEC * NV;
  using RX = Rows<TX, VEC, NV>;
  using RB = Rows<TB, VEC, NV>;
  const int warp = threadIdx.x >> 5;
  const int team = warp / warps, teams = (blockDim.x >> 5) / warps;
  const int xb = RX::kBytes * blockDim.x, bb = RB::kBytes * blockDim.x;
  const int slot_bytes = 2 * (xb + bb);
  float* red = reinterpret_cast<float*>(smem + DEPTH * slot_bytes);
  float* join = red + teams * 4 * kMaxTeamWarps;  // [teams][C] column sums of several teams
  TeamSum sum{red + team * 4 * kMaxTeamWarps, warps, warp - team * warps, team + 1, 0};
  const int lane = threadIdx.x - team * warps * 32;
  const int first = lane * VEC, step = warps * 32 * VEC;

  const int64_t begin = (int64_t)blockIdx.x * rows_per_cta;
  const int64_t end = min(begin + rows_per_cta, k.tokens);
  RX rx{dy ? x : nullptr, x_stride}, rd{dx_out, dx_out_stride};
  RB rb{block, block_stride}, ry{dy, dy_stride};
  auto ask = [&](int s, int64_t t) {
    if (t < end) {
      char* at = smem + s * slot_bytes;
      rx.fetch(at, t, first, step, k.C);
      rd.fetch(at + xb, t, first, step, k.C);
      rb.fetch(at + 2 * xb, t, first, step, k.C);
      ry.fetch(at + 2 * xb + bb, t, first, step, k.C);
    }
    copies_commit();
  };
  float4 st_next = make_float4(0.f, 0.f, 0.f, 0.f);
  auto hold = [&](int64_t t) {
    if (t < end) {
      rx.hold(t, first, step, k.C);
      rd.hold(t, first, step, k.C);
      rb.hold(t, first, step, k.C);
      ry.hold(t, first, step, k.C);
      st_next = stats[t];
    }
  };
#pragma unroll
  for (int i = 0; i < DEPTH - 1; ++i) ask(i, begin + team + (int64_t)i * teams);
  hold(begin + team);

  float acc_pre[E], acc_e[E], wp[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    acc_pre[i] = acc_e[i] = 0.f;
    wp[i] = 1.f;
  }
  scale_row<float, VEC, NV>(wp, k.w_pre, first, step, k.C);

  auto flush = [&](const float (&acc)[E], float* to) {
    if (teams == 1) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (first + i * step < k.C) to[first + i * step + j] = acc[i * VEC + j];
      return;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int c = first + i * step + j;
        if (c < k.C) join[team * k.C + c] = acc[i * VEC + j];
      }
    __syncthreads();
    for (int c = threadIdx.x; c < k.C; c += blockDim.x) {
      float s = 0.f;
      for (int i = 0; i < teams; ++i) s += join[i * k.C + c];
      to[c] = s;
    }
  };

  int g = find_group(k.offsets, k.groups, begin);
  int s = 0;
  int64_t t = begin + team;  // this team's next row
  for (int64_t at = begin; at < end;) {
    const int64_t stop =
        k.offsets && g + 1 < k.groups ? min(end, max(at, (int64_t)k.offsets[g + 1])) : end;
    float wk[E];
    group_weights<TB, VEC, NV>(wk, k, g, first, step);
    for (; t < stop; t += teams) {
      if (DEPTH == 1) ask(0, t);
      copies_done_but<(DEPTH > 2 ? DEPTH - 2 : 0)>();
      float d[E], n[E], h[E], m[E];
      const char* slot = smem + s * slot_bytes;
      rx.read(n, slot, first, step, k.C);
      rd.read(d, slot + xb, first, step, k.C);
      rb.read(m, slot + 2 * xb, first, step, k.C);
      ry.read(h, slot + 2 * xb + bb, first, step, k.C);
      const float4 st = st_next;
      if (DEPTH > 1) ask(s == 0 ? DEPTH - 1 : s - 1, t + (int64_t)(DEPTH - 1) * teams);
      hold(t + teams);
      s = s + 1 == DEPTH ? 0 : s + 1;
      if (dy) {
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
          n[i] = (n[i] - st.z) * st.w;
          acc_pre[i] += h[i] * n[i];
          h[i] *= wp[i];
          a += h[i] * n[i];
          b += h[i];
        }
        sum(a, b, k.center);
        a *= k.inv_c;
        b = k.center ? b * k.inv_c : 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) d[i] += st.w * (h[i] - n[i] * a - b);
      }
      store_row<TX, VEC, NV>(d, dx + t * dx_stride, first, step, k.C);
      if (block) {
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (first + i * step < k.C) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
              const int c = i * VEC + j;
              if (k.post) m[c] = (m[c] - st.x) * st.y;
              acc_e[c] += d[c] * m[c];
              d[c] *= wk[c];
              a += d[c] * m[c];
              b += d[c];
            }
          }
        if (k.post) {
          sum(a, b, k.center);
          a *= k.inv_c;
          b = k.center ? b * k.inv_c : 0.f;
#pragma unroll
          for (int i = 0; i < E; ++i) d[i] = st.y * (d[i] - m[i] * a - b);
        }
        store_row<TB, VEC, NV>(d, dblock + t * dblock_stride, first, step, k.C);
      }
    }
    if (block && part_e && stop > at) {
      flush(acc_e, part_e + ((int64_t)blockIdx.x + g) * k.C);
#pragma unroll
      for (int i = 0; i < E; ++i) acc_e[i] = 0.f;
    }
    at = stop;
    if (g + 1 < k.groups) ++g;
  }
  if (part_pre) flush(acc_pre, part_pre + (int64_t)blockIdx.x * k.C);
}

// Joins the CTAs' column sums, 32 columns per block, in a fixed order.
__global__ void __launch_bounds__(1024) norm_sums_kernel(NormK k, int64_t gate_elem,
                                                         int32_t gate_dtype, const float* part_pre,
                                                         const float* part_e, int64_t rows_per_cta,
                                                         int ctas, float* dw_pre, float* dw_post,
                                                         float* dgate, float* dscale) {
  __shared__ float red[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  const bool in = c < k.C;
  auto total = [&](const float* p, int lo, int hi) {  // slots [lo, hi)
    float s = 0.f;
    if (in)
      for (int i = lo + threadIdx.y; i < hi; i += 32) s += p[(int64_t)i * k.C + c];
    __syncthreads();
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    s = red[threadIdx.x][threadIdx.y];
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    __syncthreads();
    if (threadIdx.x == 0) red[0][threadIdx.y] = s;
    __syncthreads();
    return red[0][threadIdx.x];
  };
  if (dw_pre) {
    const float s = total(part_pre, 0, part_pre ? ctas : 0);
    if (in && threadIdx.y == 0) dw_pre[c] = s;
  }
  if (!dw_post && !dgate && !dscale) return;
  const float w = in && k.w_post ? k.w_post[c] : 1.f;
  const float sc = in && k.scale ? k.scale[c] : 1.f;
  float sum_post = 0.f, sum_scale = 0.f;
  for (int g = 0; g < k.groups; ++g) {
    int64_t lo = k.offsets ? k.offsets[g] : 0, hi = k.offsets ? k.offsets[g + 1] : k.tokens;
    lo = max((int64_t)0, lo);
    hi = min(hi, k.tokens);
    float e = 0.f;
    if (part_e && lo < hi)  // the same for the whole block
      e = total(part_e, (int)(lo / rows_per_cta) + g, (int)((hi - 1) / rows_per_cta) + g + 1);
    float gv = 1.f;
    if (in && k.gate) {
      const int64_t at = (int64_t)g * k.C + c;
      gv = gate_dtype == GS_F32    ? ((const float*)k.gate)[at]
           : gate_dtype == GS_BF16 ? to_f32(((const __nv_bfloat16*)k.gate)[at])
                                   : to_f32(((const __half*)k.gate)[at]);
    }
    sum_post += sc * gv * e;
    sum_scale += gv * w * e;
    if (in && dgate && threadIdx.y == 0) dgate[(int64_t)g * k.C + c] = sc * w * e;
  }
  if (in && threadIdx.y == 0) {
    if (dw_post) dw_post[c] = sum_post;
    if (dscale) dscale[c] = sum_scale;
  }
}

bool norm_ok(const gs_norm* p) {
  if (!p || p->tokens < 0 || p->tokens >= ((int64_t)1 << 31) || p->channels < 1 ||
      p->channels > GS_NORM_MAX_C || p->groups < 1 || !dtype_ok(p->dtype) ||
      (p->res_dtype != p->dtype && p->res_dtype != GS_F32) ||
      (p->flags & ~(GS_NORM_POST | GS_NORM_CENTER)) || !(p->eps >= 0.f))
    return false;
  if (p->groups > 1 && (!p->gate || !p->group_offsets)) return false;
  return aligned4(p->w_pre) && aligned4(p->w_post) && aligned4(p->res_scale) &&
         aligned4(p->group_offsets) && aligned_to(p->gate, dtype_size(p->dtype));
}

NormK make_norm(const gs_norm& p) {
  NormK k{};
  k.tokens = p.tokens;
  k.C = p.channels;
  k.groups = p.gate ? p.groups : 1;
  k.post = (p.flags & GS_NORM_POST) != 0;
  k.center = (p.flags & GS_NORM_CENTER) != 0;
  k.eps = p.eps;
  k.inv_c = (float)(1.0 / p.channels);
  k.w_pre = p.w_pre;
  k.w_post = p.w_post;
  k.scale = p.res_scale;
  k.gate = p.gate;
  k.offsets = p.gate ? p.group_offsets : nullptr;
  return k;
}

// 16-byte rows everywhere: the wide accesses may be used.
bool norm_wide(const gs_norm& p, int vec) {
  return p.channels % vec == 0 && aligned16(p.w_pre) && aligned16(p.w_post) &&
         aligned16(p.res_scale) && aligned16(p.gate);
}

struct FwdArgs {
  NormK k;
  const void *x, *block;
  void *x_out, *y;
  int64_t xs, bs, xos, ys;
  float4* stats;
  int8_t* y_q;
  int64_t qs;
  uint8_t* y_e;
  int64_t es;
};

// Rows are 8 channels a thread (16 from 4096 channels on), so a row of 1024 is
// four warps; a CTA holds as many such teams as 512 threads and 15 named
// barriers allow.
struct Shape {
  int warps, teams, threads;
};
template <int VEC, int NV>
Shape norm_shape(const NormK& k) {
  Shape s;
  s.warps = (int)div_up(k.C, 32 * VEC * NV);
  s.teams = kTeamThreads / 32 / s.warps;
  if (s.teams > 8) s.teams = 8;
  s.threads = s.teams * s.warps * 32;
  return s;
}

// Row ranges: `per_sm` CTAs an SM, none without a row for each team.
inline int64_t norm_ranges(int64_t tokens, int teams, int per_sm, int64_t* rows_per_cta) {
  int64_t ctas = (int64_t)device_sms() * per_sm;
  if (ctas > kNormCtas) ctas = kNormCtas;
  const int64_t most = div_up(tokens, teams);
  if (ctas > most) ctas = most;
  *rows_per_cta = div_up(tokens, ctas);
  return div_up(tokens, *rows_per_cta);
}

// Shared memory above 48 KB is asked for once per kernel and device.
template <typename F>
cudaError_t allow_smem(F kernel, std::atomic<uint64_t>& known) {
  int dev = 0;
  const cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess || dev >= 64) return err != cudaSuccess ? err : cudaErrorInvalidDevice;
  if (known.load(std::memory_order_acquire) >> dev & 1) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBudget);
  if (e == cudaSuccess) known.fetch_or(1ull << dev, std::memory_order_release);
  return e;
}

// The deepest ring whose rows fit in shared memory (two CTAs share an SM's).
template <typename TB, typename TX, int VEC, int NV, int DEPTH>
cudaError_t fwd_launch(const FwdArgs& a, cudaStream_t st) {
  constexpr int kPerSm = VEC * NV <= 8 ? 2 : 1;
  const Shape s = norm_shape<VEC, NV>(a.k);
  const size_t smem =
      (size_t)DEPTH * (Rows<TX, VEC, NV>::kBytes + Rows<TB, VEC, NV>::kBytes) * s.threads +
      sizeof(float) * s.teams * 4 * kMaxTeamWarps;
  if constexpr (DEPTH > 2) {
    if (smem > kSmemBudget / kPerSm) return fwd_launch<TB, TX, VEC, NV, DEPTH - 1>(a, st);
  }
  static std::atomic<uint64_t> known{0};
  const auto kernel = norm_fwd_kernel<TB, TX, VEC, NV, DEPTH>;
  const cudaError_t e = allow_smem(kernel, known);
  if (e != cudaSuccess) return e;
  int64_t rows = 0;
  const int64_t ctas = norm_ranges(a.k.tokens, s.teams, kPerSm, &rows);
  kernel<<<(unsigned)ctas, s.threads, smem, st>>>(
      a.k, (const TX*)a.x, a.xs, (const TB*)a.block, a.bs, (TX*)a.x_out, a.xos, (TB*)a.y, a.ys,
      a.stats, a.y_q, a.qs, a.y_e, a.es, rows, s.warps);
  return cudaSuccess;
}

template <typename TB, typename TX, int VEC>
cudaError_t fwd_pick(const FwdArgs& a, cudaStream_t st) {
  if (a.k.C <= 4096) return fwd_launch<TB, TX, VEC, 8 / VEC, 4>(a, st);
  return fwd_launch<TB, TX, VEC, 16 / VEC, 4>(a, st);
}

template <typename TB, typename TX>
cudaError_t fwd_types(const FwdArgs& a, bool wide, cudaStream_t st) {
  return wide ? fwd_pick<TB, TX, 16 / sizeof(TB)>(a, st) : fwd_pick<TB, TX, 1>(a, st);
}

struct BwdArgs {
  NormK k;
  const void *x, *block;
  int64_t xs, bs;
  const float4* stats;
  const void *dx_out, *dy;
  int64_t dxos, dys;
  void *dx, *dblock;
  int64_t dxs, dbs;
  float *part_pre, *part_e;
  int64_t rows_per_cta;
  int ctas;
};

// As the forward; one CTA an SM (its registers hold the column sums), and no
// rows ahead where two do not fit (more than 4096 fp32 channels).
template <typename TB, typename TX, int VEC, int NV, int DEPTH>
cudaError_t bwd_launch(const BwdArgs& a, cudaStream_t st) {
  const Shape s = norm_shape<VEC, NV>(a.k);
  const size_t smem =
      (size_t)DEPTH * 2 * (Rows<TX, VEC, NV>::kBytes + Rows<TB, VEC, NV>::kBytes) * s.threads +
      sizeof(float) * s.teams * (4 * kMaxTeamWarps + (s.teams > 1 ? (size_t)a.k.C : 0));
  if constexpr (DEPTH > 1) {
    if (smem > kSmemBudget) return bwd_launch<TB, TX, VEC, NV, DEPTH - 1>(a, st);
  }
  static std::atomic<uint64_t> known{0};
  const auto kernel = norm_bwd_kernel<TB, TX, VEC, NV, DEPTH>;
  const cudaError_t e = allow_smem(kernel, known);
  if (e != cudaSuccess) return e;
  kernel<<<(unsigned)a.ctas, s.threads, smem, st>>>(
      a.k, (const TX*)a.x, a.xs, (const TB*)a.block, a.bs, a.stats, (const TX*)a.dx_out, a.dxos,
      (const TB*)a.dy, a.dys, (TX*)a.dx, a.dxs, (TB*)a.dblock, a.dbs, a.part_pre, a.part_e,
      a.rows_per_cta, s.warps);
  return cudaSuccess;
}

template <typename TB, typename TX, int VEC, int NV>
cudaError_t bwd_ranges(BwdArgs& a, cudaStream_t st) {
  a.ctas = (int)norm_ranges(a.k.tokens, norm_shape<VEC, NV>(a.k).teams, 1, &a.rows_per_cta);
  return bwd_launch<TB, TX, VEC, NV, 4>(a, st);
}

template <typename TB, typename TX, int VEC>
cudaError_t bwd_pick(BwdArgs& a, cudaStream_t st) {
  if (a.k.C <= 4096) return bwd_ranges<TB, TX, VEC, 8 / VEC>(a, st);
  return bwd_ranges<TB, TX, VEC, 16 / VEC>(a, st);
}

template <typename TB, typename TX>
cudaError_t bwd_types(BwdArgs& a, bool wide, cudaStream_t st) {
  return wide ? bwd_pick<TB, TX, 16 / sizeof(TB)>(a, st) : bwd_pick<TB, TX, 1>(a, st);
}

#define GS_NORM_TYPES(p, f, ...)                                                         \
  ((p)->dtype == GS_F32    ? f<float, float>(__VA_ARGS__)                                \
   : (p)->dtype == GS_BF16 ? ((p)->res_dtype == GS_F32 ? f<__nv_bfloat16, float>(__VA_ARGS__) \
                                                  : f<__nv_bfloat16, __nv_bfloat16>(__VA_ARGS__)) \
                           : ((p)->res_dtype == GS_F32 ? f<__half, float>(__VA_ARGS__)   \
                                                  : f<__half, __half>(__VA_ARGS__)))

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" gs_status gs_gated_norm_fwd(const gs_norm* p, const void* x, int64_t x_stride,
                                       const void* block, int64_t block_stride, void* x_out,
                                       int64_t x_out_stride, void* y, int64_t y_stride,
                                       float* stats, int8_t* y_q, int64_t q_stride, uint8_t* y_e,
                                       int64_t e_stride, void* stream) {
  if (!norm_ok(p)) return GS_ERR_INVALID_ARG;
  if (p->tokens == 0) return GS_OK;
  const int eb = dtype_size(p->dtype), ex = dtype_size(p->res_dtype);
  if (!x || !stats || (!block != !x_out) || (!block && !y) || (!y_q != !y_e) || (y_q && !y) ||
      !aligned16(stats) || !aligned_to(x, ex) || !aligned_to(block, eb) ||
      !aligned_to(x_out, ex) || !aligned_to(y, eb))
    return GS_ERR_INVALID_ARG;
  if (y_q && (!aligned16(y_q) || q_stride % 16 ||
              q_stride < div_up(p->channels, GS_ACT8_GROUP) * GS_ACT8_GROUP)) return GS_ERR_INVALID_ARG;
  const int vec = 16 / eb;
  const bool wide = norm_wide(*p, vec) && rows_aligned(x, x_stride, ex, 16) &&
                    rows_aligned(block, block_stride, eb, 16) &&
                    rows_aligned(x_out, x_out_stride, ex, 16) && rows_aligned(y, y_stride, eb, 16);
  const FwdArgs a{make_norm(*p), x, block, x_out, y, x_stride, block_stride, x_out_stride,
                  y_stride, (float4*)stats, y_q, q_stride, y_e, e_stride};
  cudaStream_t st = (cudaStream_t)stream;
  GS_CUDA(GS_NORM_TYPES(p, fwd_types, a, wide, st));
  GS_CHECK_LAUNCH();
  return GS_OK;
}

extern "C" size_t gs_gated_norm_workspace_bytes(int32_t channels, int32_t groups) {
  if (channels < 1 || channels > GS_NORM_MAX_C || groups < 1) return 0;
  return sizeof(float) * (size_t)channels * ((size_t)2 * kNormCtas + groups);
}

extern "C" gs_status gs_gated_norm_bwd(
    const gs_norm* p, const void* x_out, int64_t x_stride, const void* block, int64_t block_stride,
    const float* stats, const void* dx_out, int64_t dx_out_stride, const void* dy,
    int64_t dy_stride, void* dx, int64_t dx_stride, void* dblock, int64_t dblock_stride,
    float* dw_pre, float* dw_post, float* dgate, float* dres_scale, void* workspace,
    size_t ws_bytes, void* stream) {
  if (!norm_ok(p)) return GS_ERR_INVALID_ARG;
  const int eb = dtype_size(p->dtype), ex = dtype_size(p->res_dtype);
  if ((!block != !dblock) || (dgate && !p->gate) || !aligned4(dw_pre) || !aligned4(dw_post) ||
      !aligned4(dgate) || !aligned4(dres_scale))
    return GS_ERR_INVALID_ARG;
  const bool need_e = dw_post || dgate || dres_scale;
  if (p->tokens > 0 && (!x_out || !stats || !dx || (!dx_out && !dy) || !aligned16(stats) ||
                        !aligned_to(x_out, ex) || !aligned_to(block, eb) ||
                        !aligned_to(dx_out, ex) || !aligned_to(dy, eb) || !aligned_to(dx, ex) ||
                        !aligned_to(dblock, eb)))
    return GS_ERR_INVALID_ARG;
  if ((dw_pre || need_e) &&
      (!workspace || !aligned16(workspace) ||
       ws_bytes < gs_gated_norm_workspace_bytes(p->channels, p->groups)))
    return GS_ERR_INVALID_ARG;
  const int vec = 16 / eb;
  const bool wide = norm_wide(*p, vec) && rows_aligned(x_out, x_stride, ex, 16) &&
                    rows_aligned(block, block_stride, eb, 16) &&
                    rows_aligned(dx_out, dx_out_stride, ex, 16) &&
                    rows_aligned(dy, dy_stride, eb, 16) && rows_aligned(dx, dx_stride, ex, 16) &&
                    rows_aligned(dblock, dblock_stride, eb, 16);
  cudaStream_t st = (cudaStream_t)stream;
  BwdArgs a{make_norm(*p), x_out, block, x_stride, block_stride, (const float4*)stats, dx_out, dy,
            dx_out_stride, dy_stride, dx, dblock, dx_stride, dblock_stride, nullptr, nullptr, 1, 0};
  if (dw_pre && dy) a.part_pre = (float*)workspace;
  if (need_e && block) a.part_e = (float*)workspace + (size_t)kNormCtas * p->channels;
  if (p->tokens > 0) {
    GS_CUDA(GS_NORM_TYPES(p, bwd_types, a, wide, st));
    GS_CHECK_LAUNCH();
  } else {
    a.part_pre = a.part_e = nullptr;
  }
  if (dw_pre || need_e) {
    norm_sums_kernel<<<(unsigned)div_up(p->channels, 32), dim3(32, 32), 0, st>>>(
        a.k, 0, p->dtype, a.part_pre, a.part_e, a.rows_per_cta, a.ctas, dw_pre, dw_post, dgate,
        dres_scale);
    GS_CHECK_LAUNCH();
  }
  return GS_OK;
}
