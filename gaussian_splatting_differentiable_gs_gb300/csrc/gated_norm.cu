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
#include "net_common.cuh"

namespace gs {
namespace {

constexpr int kNormCtas = 304;      // row ranges of the backward (column sums)
constexpr int kMaxTeamWarps = 16;

struct NormK {
  int64_t tokens;
  int32_t C, groups;
  int32_t post, center;
  float eps, inv_c;
  const float *w_pre, *w_post, *scale;
  const void* gate;
  const int32_t* offsets;
};

// Sum of one value per thread over a team of `warps` warps, the same bits in
// every thread.  red: two slots of kMaxTeamWarps floats per team, used in
// turn: a slot is written again only after the barrier of the sum in between.
struct TeamSum {
  float* red;
  int warps, warp, bar;
  int turn;
  __device__ __forceinline__ float operator()(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (warps == 1) return v;
    float* r = red + (turn & 1) * kMaxTeamWarps;
    ++turn;
    if ((threadIdx.x & 31) == 0) r[warp] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(warps * 32) : "memory");
    float s = 0.f;
    for (int i = 0; i < warps; ++i) s += r[i];
    return s;
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

template <typename T, int VEC, int NV>
__device__ __forceinline__ void load_row(float (&v)[VEC * NV], const T* p, int first, int step,
                                         int C) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = first + i * step;
    if (c < C) {
      const Pack<T, VEC> w = load_pack<T, VEC>(p + c);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i * VEC + j] = to_f32(w.v[j]);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i * VEC + j] = 0.f;
    }
  }
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

template <typename TB, typename TX, int VEC, int NV>
__global__ void __launch_bounds__(512) norm_fwd_kernel(
    NormK k, const TX* x, int64_t x_stride, const TB* block, int64_t block_stride, TX* x_out,
    int64_t x_out_stride, TB* y, int64_t y_stride, float4* stats, int8_t* y_q, int64_t q_stride,
    uint8_t* y_e, int64_t e_stride, int warps) {
  __shared__ float red[16][2][kMaxTeamWarps];
  const int warp = threadIdx.x >> 5;
  const int team = warp / warps, teams = (blockDim.x >> 5) / warps;
  TeamSum sum{&red[team][0][0], warps, warp - team * warps, team + 1, 0};
  const int lane = threadIdx.x - team * warps * 32;
  const int first = lane * VEC, step = warps * 32 * VEC;

  for (int64_t t = (int64_t)blockIdx.x * teams + team; t < k.tokens;
       t += (int64_t)gridDim.x * teams) {
    float v[VEC * NV];
    float4 st = make_float4(0.f, 0.f, 0.f, 0.f);
    if (block) {
      float u[VEC * NV];
      load_row<TB, VEC, NV>(u, block + t * block_stride, first, step, k.C);
      load_row<TX, VEC, NV>(v, x + t * x_stride, first, step, k.C);
      if (k.post) {
        row_stats<VEC, NV>(u, sum, k, first, step, st.x, st.y);
#pragma unroll
        for (int i = 0; i < VEC * NV; ++i) u[i] *= st.y;
        scale_row<float, VEC, NV>(u, k.w_post, first, step, k.C);
      }
      scale_row<float, VEC, NV>(u, k.scale, first, step, k.C);
      if (k.gate) {
        const int g = find_group(k.offsets, k.groups, t);
        scale_row<TB, VEC, NV>(u, (const TB*)k.gate + (int64_t)g * k.C, first, step, k.C);
      }
#pragma unroll
      for (int i = 0; i < VEC * NV; ++i) v[i] += u[i];
      store_row<TX, VEC, NV>(v, x_out + t * x_out_stride, first, step, k.C);
    } else {
      load_row<TX, VEC, NV>(v, x + t * x_stride, first, step, k.C);
    }
    if (y) {
      row_stats<VEC, NV>(v, sum, k, first, step, st.z, st.w);
#pragma unroll
      for (int i = 0; i < VEC * NV; ++i) v[i] *= st.w;
      scale_row<float, VEC, NV>(v, k.w_pre, first, step, k.C);
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

// Work of one CTA: rows [cta R, cta R + R), cut at the groups' ends; its teams
// take rows in turn and keep their column sums in registers.  The sums of a
// (CTA, group) pair go to slot cta + group of part_e: along the rows either the
// CTA or the group advances, so no two pairs share a slot.
template <typename TB, typename TX, int VEC, int NV>
__global__ void __launch_bounds__(512) norm_bwd_kernel(
    NormK k, const TX* x, int64_t x_stride, const TB* block, int64_t block_stride,
    const float4* stats, const TX* dx_out, int64_t dx_out_stride, const TB* dy, int64_t dy_stride,
    TX* dx, int64_t dx_stride, TB* dblock, int64_t dblock_stride, float* part_pre, float* part_e,
    int64_t rows_per_cta, int warps) {
  extern __shared__ float smem[];
  constexpr int E = VEC * NV;
  const int warp = threadIdx.x >> 5;
  const int team = warp / warps, teams = (blockDim.x >> 5) / warps;
  TeamSum sum{smem + team * 2 * kMaxTeamWarps, warps, warp - team * warps, team + 1, 0};
  float* join = smem + teams * 2 * kMaxTeamWarps;  // [teams][C] column sums
  const int lane = threadIdx.x - team * warps * 32;
  const int first = lane * VEC, step = warps * 32 * VEC;

  const int64_t begin = (int64_t)blockIdx.x * rows_per_cta;
  const int64_t end = min(begin + rows_per_cta, k.tokens);
  float acc_pre[E], acc_e[E];
#pragma unroll
  for (int i = 0; i < E; ++i) acc_pre[i] = acc_e[i] = 0.f;

  auto flush = [&](const float (&acc)[E], float* to) {
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
  for (int64_t at = begin; at < end;) {
    const int64_t stop =
        k.offsets && g + 1 < k.groups ? min(end, max(at, (int64_t)k.offsets[g + 1])) : end;
    float wk[E];  // k = scale * gate * w_post of this group
#pragma unroll
    for (int i = 0; i < E; ++i) wk[i] = 1.f;
    scale_row<float, VEC, NV>(wk, k.scale, first, step, k.C);
    if (k.post) scale_row<float, VEC, NV>(wk, k.w_post, first, step, k.C);
    if (k.gate) scale_row<TB, VEC, NV>(wk, (const TB*)k.gate + (int64_t)g * k.C, first, step, k.C);
    for (int64_t t = at + team; t < stop; t += teams) {
      float d[E], n[E];
      const float4 st = stats[t];
      if (dx_out) {
        load_row<TX, VEC, NV>(d, dx_out + t * dx_out_stride, first, step, k.C);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) d[i] = 0.f;
      }
      if (dy) {
        float h[E];
        load_row<TB, VEC, NV>(h, dy + t * dy_stride, first, step, k.C);
        load_row<TX, VEC, NV>(n, x + t * x_stride, first, step, k.C);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          n[i] = (n[i] - st.z) * st.w;
          acc_pre[i] += h[i] * n[i];
        }
        scale_row<float, VEC, NV>(h, k.w_pre, first, step, k.C);
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) a += h[i] * n[i], b += h[i];
        a = sum(a) * k.inv_c;
        b = k.center ? sum(b) * k.inv_c : 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) d[i] += st.w * (h[i] - n[i] * a - b);
      }
      store_row<TX, VEC, NV>(d, dx + t * dx_stride, first, step, k.C);
      if (block) {
        float m[E];
        load_row<TB, VEC, NV>(m, block + t * block_stride, first, step, k.C);
        if (k.post) {
#pragma unroll
          for (int i = 0; i < E; ++i) m[i] = (m[i] - st.x) * st.y;
        }
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (first + i * step < k.C) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
              const int c = i * VEC + j;
              acc_e[c] += d[c] * m[c];
              d[c] *= wk[c];
              a += d[c] * m[c];
              b += d[c];
            }
          }
        if (k.post) {
          a = sum(a) * k.inv_c;
          b = k.center ? sum(b) * k.inv_c : 0.f;
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

template <typename TB, typename TX, int VEC, int NV>
void fwd_launch(const FwdArgs& a, cudaStream_t st) {
  const int warps = (int)div_up(a.k.C, 32 * VEC * NV);
  const int teams = warps >= 4 ? 1 : 4 / warps;
  const int64_t want = div_up(a.k.tokens, teams);
  const unsigned blocks = (unsigned)(want < (1 << 30) ? want : (1 << 30));
  norm_fwd_kernel<TB, TX, VEC, NV><<<blocks, teams * warps * 32, 0, st>>>(
      a.k, (const TX*)a.x, a.xs, (const TB*)a.block, a.bs, (TX*)a.x_out, a.xos, (TB*)a.y, a.ys,
      a.stats, a.y_q, a.qs, a.y_e, a.es, warps);
}

// Channels per thread: up to 32, so that a row of 1024 is one warp's.
template <typename TB, typename TX, int VEC>
void fwd_pick(const FwdArgs& a, cudaStream_t st) {
  const int per_lane = (int)div_up(a.k.C, 32);
  if (per_lane <= 8) fwd_launch<TB, TX, VEC, 8 / VEC>(a, st);
  else if (per_lane <= 16) fwd_launch<TB, TX, VEC, 16 / VEC>(a, st);
  else fwd_launch<TB, TX, VEC, 32 / VEC>(a, st);
}

template <typename TB, typename TX>
void fwd_types(const FwdArgs& a, bool wide, cudaStream_t st) {
  if (wide) fwd_pick<TB, TX, 16 / sizeof(TB)>(a, st);
  else fwd_pick<TB, TX, 1>(a, st);
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

template <typename TB, typename TX, int VEC, int NV>
cudaError_t bwd_launch(const BwdArgs& a, cudaStream_t st) {
  const int warps = (int)div_up(a.k.C, 32 * VEC * NV);
  const int teams = warps >= 16 ? 1 : (16 / warps < 8 ? 16 / warps : 8);
  const size_t smem = sizeof(float) * teams * (2 * kMaxTeamWarps + (size_t)a.k.C);
  norm_bwd_kernel<TB, TX, VEC, NV><<<a.ctas, teams * warps * 32, smem, st>>>(
      a.k, (const TX*)a.x, a.xs, (const TB*)a.block, a.bs, a.stats, (const TX*)a.dx_out, a.dxos,
      (const TB*)a.dy, a.dys, (TX*)a.dx, a.dxs, (TB*)a.dblock, a.dbs, a.part_pre, a.part_e,
      a.rows_per_cta, warps);
  return cudaSuccess;
}

template <typename TB, typename TX, int VEC>
cudaError_t bwd_pick(const BwdArgs& a, cudaStream_t st) {
  if (a.k.C <= 4096) return bwd_launch<TB, TX, VEC, 8 / VEC>(a, st);
  return bwd_launch<TB, TX, VEC, 16 / VEC>(a, st);
}

template <typename TB, typename TX>
cudaError_t bwd_types(const BwdArgs& a, bool wide, cudaStream_t st) {
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
  GS_NORM_TYPES(p, fwd_types, a, wide, st);
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
    a.rows_per_cta = div_up(p->tokens, kNormCtas);
    a.ctas = (int)div_up(p->tokens, a.rows_per_cta);
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
