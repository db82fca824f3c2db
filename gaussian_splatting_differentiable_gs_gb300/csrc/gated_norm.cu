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

constexpr int kNormCtas = 304;      // most row ranges (places for their column sums)
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

// Sums of N values per thread over a team of `warps` warps, the same bits in
// every thread.  red: two slots of kRedFloats / 2 floats per team, used in turn:
// a slot is written again only after the barrier of the sum in between.
constexpr int kRedFloats = 2 * 2 * kMaxTeamWarps;
struct Team {
  float* red;
  int warps, warp, bar;
  int turn;
  __device__ __forceinline__ void sync() const {
    if (warps == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(warps * 32) : "memory");
  }
  template <int N>
  __device__ __forceinline__ void sum(float (&v)[N]) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    if (warps == 1) return;
    float* r = red + (turn & 1) * (kRedFloats / 2);
    ++turn;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) r[i * kMaxTeamWarps + warp] = v[i];
    }
    sync();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
    for (int w = 0; w < warps; w += 4)  // places of warps that are not there hold zeros
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float4 u = *reinterpret_cast<const float4*>(r + i * kMaxTeamWarps + w);
        v[i] += (u.x + u.y) + (u.z + u.w);
      }
  }
};

// Zeros in the sums' places, and in the slots where some of a slot is never
// copied to, before any copy is asked for.
__device__ __forceinline__ void clear_shared(char* smem, int slots, int bytes, bool filled) {
  for (int i = (filled ? slots : 0) + threadIdx.x * 16; i < bytes; i += blockDim.x * 16)
    *reinterpret_cast<uint4*>(smem + i) = make_uint4(0, 0, 0, 0);
  __syncthreads();
}

// The last group that starts at or before row t.  Whole warps call it.
__device__ __forceinline__ int find_group(const int32_t* offsets, int groups, int64_t t) {
  if (!offsets) return 0;
  if (groups <= 32) {
    const int lane = threadIdx.x & 31;
    const unsigned below = __ballot_sync(0xffffffffu, lane < groups && offsets[lane] <= t);
    return below ? 31 - __clz(below) : 0;
  }
  int lo = 0, hi = groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (offsets[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// The rows to come are copied asynchronously (cp.async, 16 bytes at a time)
// into shared memory while earlier rows are worked on.  Where rows start on
// 16-byte boundaries (VEC > 1) every thread copies what it reads itself, so it
// waits for nothing but its own copies.  Otherwise a team copies the 16-byte
// granules that its row touches, and meets at a barrier before and after it
// reads them; bytes of the first and last granule that are not the tensor's are
// not read.
template <typename T, int VEC, int NV>
struct Rows {
  static constexpr bool kOwn = VEC > 1;
  static constexpr int kChunk = 16, kEl = kOwn ? kChunk / (int)sizeof(T) : 1;
  static constexpr int kPer = VEC / kEl, kChunks = NV * kPer;
  // bytes of a row's slot for the whole CTA
  __host__ __device__ static int slot(int threads, int teams, int C) {
    return kOwn ? kChunks * kChunk * threads : teams * row_bytes(C);
  }
  __host__ __device__ static int row_bytes(int C) { return (C * (int)sizeof(T) + 31) / 16 * 16; }

  const T* base;  // NULL: zeros
  int64_t stride;

  __device__ __forceinline__ void fetch(char* slot, int64_t t, int first, int step, int C,
                                        int team) const {
    if (!base) return;
    const T* p = base + t * stride;
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(slot);
    if (kOwn) {
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int c = first + i / kPer * step + i % kPer * kEl;
        if (c < C)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                           to + (i * (int)blockDim.x + (int)threadIdx.x) * kChunk),
                       "l"(p + c)
                       : "memory");
      }
    } else {
      const int off = (int)((uintptr_t)p & 15), n = C * (int)sizeof(T);
      int b = first * 16 - off;  // the granule's first byte within the row
      uint32_t at = to + team * row_bytes(C) + first * 16;
      // what lies before the row may not be the tensor's
      if (b < 0 && (stride < C || t * stride * (int64_t)sizeof(T) < 16)) {
        for (int j = 0; j < b + 16 && j < n; j += sizeof(T))
          *reinterpret_cast<T*>(slot + team * row_bytes(C) + off + j) = p[j / (int)sizeof(T)];
        b += step * 16, at += step * 16;
      }
      const char* from = (const char*)p + b;
      for (; b < n; b += step * 16, at += step * 16, from += step * 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(from),
                     "r"(min(n - b, 16))
                     : "memory");
    }
  }
  // Channels from C on and tensors that are not there read as the zeros that the
  // slots began with.
  __device__ __forceinline__ void read(float (&v)[VEC * NV], const char* slot, int64_t t, int first,
                                       int step, int C, int team) const {
    if (kOwn) {
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const Pack<T, kEl> w = load_pack<T, kEl>(reinterpret_cast<const T*>(
            slot + (i * (int)blockDim.x + (int)threadIdx.x) * kChunk));
#pragma unroll
        for (int j = 0; j < kEl; ++j) v[i * kEl + j] = to_f32(w.v[j]);
      }
      return;
    }
    const T* row = reinterpret_cast<const T*>(
        slot + team * row_bytes(C) + ((uintptr_t)(base + t * stride) & 15));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = first + i * step;
      v[i] = base && c < C ? to_f32(row[c]) : 0.f;
    }
  }
};

// Waits until at most n of this thread's latest groups of copies are pending.
__device__ __forceinline__ void copies_pending(int n) {
  switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
  }
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
constexpr int kMaxDepth = 5;  // rows of a team in shared memory

template <typename T, int VEC, int NV>
__device__ __forceinline__ void store_row(const float (&v)[VEC * NV], T* p, int first, int step,
                                          int C) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = first + i * step;
    if (c < C) {
      Pack<T, VEC> w;
      if constexpr (sizeof(T) == 2 && VEC > 1) {
#pragma unroll
        for (int j = 0; j < VEC; j += 2)
          reinterpret_cast<uint32_t*>(&w)[j / 2] = pair_word<T>(v[i * VEC + j], v[i * VEC + j + 1]);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) w.v[j] = from_f32<T>(v[i * VEC + j]);
      }
      store_pack<T, VEC>(p + c, w);
    }
  }
}

// Channels i and i + 1 of a thread's.
template <int E>
__device__ __forceinline__ float2 pair(const float (&v)[E], int i) {
  return make_float2(v[i], v[i + 1]);
}
template <int E>
__device__ __forceinline__ void put_pair(float (&v)[E], int i, float2 a) {
  v[i] = a.x, v[i + 1] = a.y;
}

// Mean and 1/deviation of a team's row; v becomes the centred row.
template <int VEC, int NV>
__device__ __forceinline__ void row_stats(float (&v)[VEC * NV], Team& team, const NormK& k,
                                          int first, int step, float& mean, float& rstd) {
  mean = 0.f;
  if (k.center) {
    float2 all = both(0.f);
#pragma unroll
    for (int i = 0; i < VEC * NV; i += 2) all = add2(all, pair(v, i));
    float s[1] = {all.x + all.y};
    team.sum(s);
    mean = s[0] * k.inv_c;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (first + i * step < k.C) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[i * VEC + j] -= mean;
      }
  }
  float2 all = both(0.f);
#pragma unroll
  for (int i = 0; i < VEC * NV; i += 2) all = fma2(pair(v, i), pair(v, i), all);
  float s[1] = {all.x + all.y};
  team.sum(s);
  rstd = rsqrtf(s[0] * k.inv_c + k.eps);
}

// Per-channel weights in shared memory, in the order in which a team's threads
// read them (16 bytes a thread at a time; every team reads the same): place
// of value j of a thread's vector i.  Channels from C on have weight 0.
template <int VEC, int NV>
struct Weights {
  static constexpr int kEl = VEC >= 4 ? 4 : 1;
  __host__ __device__ static int count(int warps) { return VEC * NV * warps * 32; }
  __device__ __forceinline__ static int place(int i, int j, int lane, int lanes) {
    return ((i * (VEC / kEl) + j / kEl) * lanes + lane) * kEl + j % kEl;
  }
  // f(channel) for every channel, by the whole CTA
  template <typename F>
  __device__ __forceinline__ static void fill(float* w, int C, int lanes, F f) {
    for (int c = threadIdx.x; c < VEC * NV * lanes; c += blockDim.x)
      w[place(c / VEC / lanes, c % VEC, c / VEC % lanes, lanes)] = c < C ? f(c) : 0.f;
  }
  __device__ __forceinline__ static void get(float (&v)[VEC], const float* w, int i, int lane,
                                             int lanes) {
#pragma unroll
    for (int j = 0; j < VEC; j += kEl) {
      const Pack<float, kEl> p = load_pack<float, kEl>(w + place(i, j, lane, lanes));
#pragma unroll
      for (int e = 0; e < kEl; ++e) v[j + e] = p.v[e];
    }
  }
  __device__ __forceinline__ static void get_all(float (&v)[VEC * NV], const float* w, int lane,
                                                 int lanes) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float u[VEC];
      get(u, w, i, lane, lanes);
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i * VEC + j] = u[j];
    }
  }
};

// k = res_scale * gate * w_post of a group's channel c
template <typename TB>
__device__ __forceinline__ float group_weight(const NormK& k, int g, int c) {
  float w = k.scale ? k.scale[c] : 1.f;
  if (k.w_post) w *= k.w_post[c];
  if (k.gate) w *= to_f32(((const TB*)k.gate)[(int64_t)g * k.C + c]);
  return w;
}

// A team's sums of part[0] and, for centred norms, part[1] (0 otherwise).
__device__ __forceinline__ void team_sums(Team& team, float (&part)[2], bool center) {
  if (center) {
    team.sum(part);
  } else {
    float only[1] = {part[0]};
    team.sum(only);
    part[0] = only[0];
    part[1] = 0.f;
  }
}

// Work of a CTA: rows [cta R, cta R + R), cut at the groups' ends; its teams
// take them in turn; the backward keeps its column sums in registers.  A thread has
// up to 32 (backward: 16) channels of a row, so that what a row costs by itself
// (sums over the team, addresses) is spread over many: with 8 the forward took 283
// instructions per 8 x 32 channels and was bound by them.
struct Range {
  int64_t begin, end;
};
__device__ __forceinline__ Range cta_rows(const NormK& k, int64_t rows_per_cta) {
  const int64_t b = (int64_t)blockIdx.x * rows_per_cta;
  return Range{b, min(b + rows_per_cta, k.tokens)};
}

template <typename TB, typename TX, int VEC, int NV>
__global__ void __launch_bounds__(kTeamThreads, 1) norm_fwd_kernel(
    const __grid_constant__ NormK k, const TX* x, int64_t x_stride, const TB* block,
    int64_t block_stride, TX* x_out, int64_t x_out_stride, TB* y, int64_t y_stride, float4* stats,
    int8_t* y_q, int64_t q_stride, uint8_t* y_e, int64_t e_stride, int64_t rows_per_cta, int warps,
    int depth) {
  extern __shared__ __align__(16) char smem[];
  constexpr int E = VEC * NV;
  using RX = Rows<TX, VEC, NV>;
  using RB = Rows<TB, VEC, NV>;
  const int warp = threadIdx.x >> 5;
  const int tm = warp / warps, teams = (blockDim.x >> 5) / warps;
  const int xb = RX::slot(blockDim.x, teams, k.C), bb = RB::slot(blockDim.x, teams, k.C);
  const int slot_bytes = xb + bb;
  float* red = reinterpret_cast<float*>(smem + depth * slot_bytes);
  float* w_pre = red + teams * kRedFloats;
  float* w_k = w_pre + Weights<VEC, NV>::count(warps);
  Team team{red + tm * kRedFloats, warps, warp - tm * warps, tm + 1, 0};
  const int lanes = warps * 32, lane = threadIdx.x - tm * lanes;
  const int first = lane * VEC, step = warps * 32 * VEC;

  launch_dependents();
  const Range rows = cta_rows(k, rows_per_cta);
  const RX rx{x, x_stride};
  const RB rb{block, block_stride};
  int64_t next = rows.begin + tm;  // the next row to ask for
  auto ask = [&](int s) {
    if (next < rows.end) {
      rx.fetch(smem + s * slot_bytes, next, first, step, k.C, tm);
      rb.fetch(smem + s * slot_bytes + xb, next, first, step, k.C, tm);
    }
    copies_commit();
    next += teams;
  };
  clear_shared(smem, depth * slot_bytes, depth * slot_bytes + teams * kRedFloats * (int)sizeof(float),
               !RX::kOwn || (block && k.C == VEC * NV * lanes));
  wait_for_previous();
  for (int i = 0; i < depth; ++i) ask(i);

  Weights<VEC, NV>::fill(w_pre, k.C, lanes,
                         [&](int c) { return k.w_pre ? k.w_pre[c] : 1.f; });

  int g = find_group(k.offsets, k.groups, rows.begin), s = 0;
  int64_t t = rows.begin + tm;
  for (int64_t at = rows.begin; at < rows.end;) {
    const int64_t stop =
        k.offsets && g + 1 < k.groups ? min(rows.end, max(at, (int64_t)k.offsets[g + 1])) : rows.end;
    if (stop > at) {  // the same for the whole CTA
      if (at > rows.begin) __syncthreads();
      Weights<VEC, NV>::fill(w_k, k.C, lanes,
                             [&](int c) { return group_weight<TB>(k, g, c); });
      __syncthreads();
    }
    for (; t < stop; t += teams) {
      copies_pending(depth - 1);
      if (!RX::kOwn) team.sync();
      float v[E], u[E], m0 = 0.f, r0 = 0.f, m1 = 0.f, r1 = 0.f;
      const char* slot = smem + s * slot_bytes;
      rx.read(v, slot, t, first, step, k.C, tm);
      rb.read(u, slot + xb, t, first, step, k.C, tm);
      if (block) {
        if (k.post) {
          row_stats<VEC, NV>(u, team, k, first, step, m0, r0);
#pragma unroll
          for (int i = 0; i < E; i += 2) put_pair(u, i, mul2(pair(u, i), both(r0)));
        }
        float w[E];
        Weights<VEC, NV>::get_all(w, w_k, lane, lanes);
#pragma unroll
        for (int i = 0; i < E; i += 2) put_pair(v, i, fma2(pair(w, i), pair(u, i), pair(v, i)));
        store_row<TX, VEC, NV>(v, x_out + t * x_out_stride, first, step, k.C);
      }
      if (!RX::kOwn) team.sync();
      ask(s);
      s = s + 1 == depth ? 0 : s + 1;
      if (y) {
        row_stats<VEC, NV>(v, team, k, first, step, m1, r1);
        float w[E];
        Weights<VEC, NV>::get_all(w, w_pre, lane, lanes);
#pragma unroll
        for (int i = 0; i < E; i += 2)
          put_pair(v, i, mul2(mul2(both(r1), pair(w, i)), pair(v, i)));
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
              for (int j = 0; j < VEC; ++j)
                q.v[j] = (int8_t)(e == 255u ? 0u : act8_round(v[i * VEC + j], inv) & 0xff);
              store_pack<int8_t, VEC>(y_q + t * q_stride + c, q);
              if (c % GS_ACT8_GROUP == 0) y_e[t * e_stride + c / GS_ACT8_GROUP] = (uint8_t)e;
            }
          }
        }
      }
      if (lane == 0) stats[t] = make_float4(m0, r0, m1, r1);
    }
    at = stop;
    if (g + 1 < k.groups) ++g;
  }
}

// The sums of a (CTA, group) pair go to slot cta + group of part_e: along the
// rows either the CTA or the group advances, so no two pairs share a slot.
template <typename TB, typename TX, int VEC, int NV>
__global__ void __launch_bounds__(kTeamThreads, 1) norm_bwd_kernel(
    const __grid_constant__ NormK k, const TX* x, int64_t x_stride, const TB* block,
    int64_t block_stride, const float4* stats, const TX* dx_out, int64_t dx_out_stride,
    const TB* dy, int64_t dy_stride, TX* dx, int64_t dx_stride, TB* dblock, int64_t dblock_stride,
    float* part_pre, float* part_e, int64_t rows_per_cta, int warps, int depth) {
  extern __shared__ __align__(16) char smem[];
  constexpr int E = VEC * NV;
  using RX = Rows<TX, VEC, NV>;
  using RB = Rows<TB, VEC, NV>;
  const int warp = threadIdx.x >> 5;
  const int tm = warp / warps, teams = (blockDim.x >> 5) / warps;
  const int xb = RX::slot(blockDim.x, teams, k.C), bb = RB::slot(blockDim.x, teams, k.C);
  const int slot_bytes = 2 * (xb + bb);
  float* red = reinterpret_cast<float*>(smem + depth * slot_bytes);
  float* w_pre = red + teams * kRedFloats;
  float* w_k = w_pre + Weights<VEC, NV>::count(warps);
  float* join = w_k + Weights<VEC, NV>::count(warps);  // column sums of several teams, in places
  Team team{red + tm * kRedFloats, warps, warp - tm * warps, tm + 1, 0};
  const int lanes = warps * 32, lane = threadIdx.x - tm * lanes;
  const int first = lane * VEC, step = warps * 32 * VEC;

  launch_dependents();
  const Range rows = cta_rows(k, rows_per_cta);
  const RX rx{dy ? x : nullptr, x_stride}, rd{dx_out, dx_out_stride};
  const RB rb{block, block_stride}, ry{dy, dy_stride};
  int64_t next = rows.begin + tm;
  auto ask = [&](int s) {
    if (next < rows.end) {
      char* at = smem + s * slot_bytes;
      rx.fetch(at, next, first, step, k.C, tm);
      ry.fetch(at + 2 * xb + bb, next, first, step, k.C, tm);
      rd.fetch(at + xb, next, first, step, k.C, tm);
      rb.fetch(at + 2 * xb, next, first, step, k.C, tm);
    }
    copies_commit();
    next += teams;
  };
  clear_shared(smem, depth * slot_bytes, depth * slot_bytes + teams * kRedFloats * (int)sizeof(float),
               !RX::kOwn || (block && dy && dx_out && k.C == VEC * NV * lanes));
  wait_for_previous();
  for (int i = 0; i < depth; ++i) ask(i);
  float4 st_next = make_float4(0.f, 0.f, 0.f, 0.f);
  if (rows.begin + tm < rows.end) st_next = stats[rows.begin + tm];

  float acc_pre[E], acc_e[E];
#pragma unroll
  for (int i = 0; i < E; ++i) acc_pre[i] = acc_e[i] = 0.f;
  Weights<VEC, NV>::fill(w_pre, k.C, lanes,
                         [&](int c) { return k.w_pre ? k.w_pre[c] : 1.f; });

  auto flush = [&](const float (&acc)[E], float* to) {
    if (teams == 1) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (first + i * step < k.C) to[first + i * step + j] = acc[i * VEC + j];
      return;
    }
    using W = Weights<VEC, NV>;
    using P = Pack<float, W::kEl>;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < E; i += W::kEl) {
      P p;
#pragma unroll
      for (int j = 0; j < W::kEl; ++j) p.v[j] = acc[i + j];
      store_pack<float, W::kEl>(join + tm * E * lanes + W::place(i / VEC, i % VEC, lane, lanes), p);
    }
    __syncthreads();
    for (int q = threadIdx.x; q < E / W::kEl * lanes; q += blockDim.x) {
      P sum = load_pack<float, W::kEl>(join + q * W::kEl);
      for (int i = 1; i < teams; ++i) {
        const P p = load_pack<float, W::kEl>(join + i * E * lanes + q * W::kEl);
#pragma unroll
        for (int j = 0; j < W::kEl; ++j) sum.v[j] += p.v[j];
      }
      constexpr int kIn = VEC / W::kEl;  // packs of a vector
      const int r = q / lanes, c = (r / kIn * lanes + q % lanes) * VEC + r % kIn * W::kEl;
      if (c < k.C) store_pack<float, W::kEl>(to + c, sum);
    }
  };

  int g = find_group(k.offsets, k.groups, rows.begin), s = 0;
  int64_t t = rows.begin + tm;  // this team's next row
  for (int64_t at = rows.begin; at < rows.end;) {
    const int64_t stop =
        k.offsets && g + 1 < k.groups ? min(rows.end, max(at, (int64_t)k.offsets[g + 1])) : rows.end;
    if (stop > at) {  // the same for the whole CTA
      if (at > rows.begin) __syncthreads();
      Weights<VEC, NV>::fill(w_k, k.C, lanes,
                             [&](int c) { return group_weight<TB>(k, g, c); });
      __syncthreads();
    }
    for (; t < stop; t += teams) {
      copies_pending(depth - 1);
      if (!RX::kOwn) team.sync();
      const float4 st = st_next;
      if (t + teams < rows.end) st_next = stats[t + teams];
      const char* slot = smem + s * slot_bytes;
      float d[E];
      if (dy) {
        float n[E], h[E], w[E];
        rx.read(n, slot, t, first, step, k.C, tm);
        ry.read(h, slot + 2 * xb + bb, t, first, step, k.C, tm);
        Weights<VEC, NV>::get_all(w, w_pre, lane, lanes);
        float2 hn = both(0.f), h1 = both(0.f);
#pragma unroll
        for (int i = 0; i < E; i += 2) {
          const float2 ni = mul2(add2(pair(n, i), both(-st.z)), both(st.w)), hi = pair(h, i);
          put_pair(acc_pre, i, fma2(hi, ni, pair(acc_pre, i)));
          const float2 hw = mul2(hi, pair(w, i));
          hn = fma2(hw, ni, hn);
          put_pair(n, i, ni);
          put_pair(h, i, hw);
        }
        if (k.center)
#pragma unroll
          for (int i = 0; i < E; i += 2) h1 = add2(h1, pair(h, i));
        float part[2] = {hn.x + hn.y, h1.x + h1.y};
        team_sums(team, part, k.center);
        const float2 a = both(-part[0] * k.inv_c), b = both(-part[1] * k.inv_c);
        rd.read(d, slot + xb, t, first, step, k.C, tm);
        if (k.center)
#pragma unroll
          for (int i = 0; i < E; i += 2) put_pair(h, i, add2(pair(h, i), b));
#pragma unroll
        for (int i = 0; i < E; i += 2)
          put_pair(d, i, fma2(both(st.w), fma2(pair(n, i), a, pair(h, i)), pair(d, i)));
      } else {
        rd.read(d, slot + xb, t, first, step, k.C, tm);
      }
      store_row<TX, VEC, NV>(d, dx + t * dx_stride, first, step, k.C);
      if (block) {
        float m[E], w[E];  // weights: 0 from C on
        rb.read(m, slot + 2 * xb, t, first, step, k.C, tm);
        Weights<VEC, NV>::get_all(w, w_k, lane, lanes);
        if (k.post)
#pragma unroll
          for (int i = 0; i < E; i += 2)
            put_pair(m, i, mul2(add2(pair(m, i), both(-st.x)), both(st.y)));
        float2 dm = both(0.f), d1 = both(0.f);
#pragma unroll
        for (int i = 0; i < E; i += 2) {
          const float2 mi = pair(m, i), di = pair(d, i);
          put_pair(acc_e, i, fma2(di, mi, pair(acc_e, i)));
          const float2 dw = mul2(di, pair(w, i));
          dm = fma2(dw, mi, dm);
          put_pair(d, i, dw);
        }
        if (k.post) {
          if (k.center)
#pragma unroll
            for (int i = 0; i < E; i += 2) d1 = add2(d1, pair(d, i));
          float part[2] = {dm.x + dm.y, d1.x + d1.y};
          team_sums(team, part, k.center);
          const float2 a = both(-part[0] * k.inv_c), b = both(-part[1] * k.inv_c);
          if (k.center)
#pragma unroll
            for (int i = 0; i < E; i += 2) put_pair(d, i, add2(pair(d, i), b));
#pragma unroll
          for (int i = 0; i < E; i += 2)
            put_pair(d, i, mul2(both(st.y), fma2(pair(m, i), a, pair(d, i))));
        }
        store_row<TB, VEC, NV>(d, dblock + t * dblock_stride, first, step, k.C);
      }
      if (!RX::kOwn) team.sync();
      ask(s);
      s = s + 1 == depth ? 0 : s + 1;
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

// Joins the CTAs' column sums, 32 columns per block, in a fixed order: the
// block's 32 warps share out the groups (up to 32 at a time), and a group's
// slots among its warps.
__global__ void __launch_bounds__(1024) norm_sums_kernel(const __grid_constant__ NormK k,
                                                         int32_t gate_dtype, const float* part_pre,
                                                         const float* part_e, int64_t rows_per_cta,
                                                         int ctas, float* dw_pre, float* dw_post,
                                                         float* dgate, float* dscale) {
  __shared__ float red[32][33], red2[32][33];
  const int x = threadIdx.x, y = threadIdx.y;
  const int c = blockIdx.x * 32 + x;
  const bool in = c < k.C;
  launch_dependents();
  // Before anything is read, the weights and offsets too: the row kernel begins early
  // itself, so when this one begins, what runs before that may still be writing them.
  wait_for_previous();
  auto slots = [&](const float* p, int lo, int hi, int from, int by) {
    float s = 0.f;
    if (in && p)
#pragma unroll 8
      for (int i = lo + from; i < hi; i += by) s += p[(int64_t)i * k.C + c];
    return s;
  };
  auto join = [&](float (*m)[33], float* to) {  // one warp
    if (!in || !to) return;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) s += m[i][x];
    to[c] = s;
  };
  if (blockIdx.y == 0) {  // dw_pre's blocks
    if (!dw_pre) return;
    red[y][x] = slots(part_pre, 0, ctas, y, 32);
    __syncthreads();
    if (y == 0) join(red, dw_pre);
    return;
  }
  const float w = in && k.w_post ? k.w_post[c] : 1.f;
  const float sc = in && k.scale ? k.scale[c] : 1.f;
  int64_t lo = 0, hi = 0;  // rows of the group whose slots this warp adds up
  float gv = 1.f;          // gate of the group that it joins
  auto ahead = [&](int g0) {
    const int n = min(32, k.groups - g0), per = 32 / n, g = g0 + y / per;
    lo = 0, hi = y < n * per ? k.tokens : 0;
    if (k.offsets && y < n * per) {
      lo = max(lo, (int64_t)k.offsets[g]);
      hi = min(hi, (int64_t)k.offsets[g + 1]);
    }
    if (y < n && in && k.gate) {
      const int64_t at = (int64_t)(g0 + y) * k.C + c;
      gv = gate_dtype == GS_F32    ? ((const float*)k.gate)[at]
           : gate_dtype == GS_BF16 ? to_f32(((const __nv_bfloat16*)k.gate)[at])
                                   : to_f32(((const __half*)k.gate)[at]);
    }
  };
  ahead(0);
  float post = 0.f, scale = 0.f;
  for (int g0 = 0; g0 < k.groups; g0 += 32) {
    const int n = min(32, k.groups - g0), per = 32 / n, g = g0 + y / per;
    float e = 0.f;
    if (lo < hi)
      e = slots(part_e, (int)(lo / rows_per_cta) + g, (int)((hi - 1) / rows_per_cta) + g + 1,
                y % per, per);
    __syncthreads();
    red[y][x] = e;
    __syncthreads();
    if (y < n) {  // one warp a group
      e = 0.f;
      for (int i = 0; i < per; ++i) e += red[y * per + i][x];
      if (k.post) post += sc * gv * e;  // else u does not depend on w_post
      scale += gv * w * e;
      if (in && dgate) dgate[(int64_t)(g0 + y) * k.C + c] = sc * w * e;
    }
    if (g0 + 32 < k.groups) ahead(g0 + 32);
  }
  __syncthreads();
  red[y][x] = post;
  red2[y][x] = scale;
  __syncthreads();
  if (y == 0) join(red, dw_post);
  if (y == 1) join(red2, dscale);
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
  k.w_post = k.post ? p.w_post : nullptr;  // no norm after the block: no weight
  k.scale = p.res_scale;
  k.gate = p.gate;
  k.offsets = p.gate ? p.group_offsets : nullptr;
  return k;
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

// A team: the warps that a row of VEC * NV channels a thread needs; a CTA: as many
// teams as its threads allow (16 of one warp; several warps need a named barrier).
struct Shape {
  int warps, teams, threads;
};
template <int VEC, int NV>
Shape norm_shape(const NormK& k, int threads) {
  Shape s;
  s.warps = (int)div_up(k.C, 32 * VEC * NV);
  s.teams = threads / 32 / s.warps;
  if (s.teams < 1) s.teams = 1;
  s.threads = s.teams * s.warps * 32;
  return s;
}

// Row ranges: one CTA an SM, none without a row for each team.
inline int64_t norm_ranges(int64_t tokens, int teams, int64_t* rows_per_cta) {
  int64_t ctas = device_sms();
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

// Threads of a CTA and rows of a team in shared memory: 512 threads where that
// leaves a row ahead for each team (or more, up to kMaxDepth), else fewer, as fp32 rows do.
struct Layout {
  Shape s;
  int depth;
  size_t smem;
};
template <typename TB, typename TX, int VEC, int NV>
Layout norm_layout(const NormK& k, int tensors, bool join) {
  Layout l;
  const int sms = device_sms();
  for (int threads = kTeamThreads;; threads /= 2) {
    l.s = norm_shape<VEC, NV>(k, threads);
    const size_t slot = (size_t)tensors * (Rows<TX, VEC, NV>::slot(l.s.threads, l.s.teams, k.C) +
                                           Rows<TB, VEC, NV>::slot(l.s.threads, l.s.teams, k.C));
    const size_t fixed =
        sizeof(float) * ((size_t)l.s.teams * kRedFloats + 2 * Weights<VEC, NV>::count(l.s.warps) +
                         (join && l.s.teams > 1 ? (size_t)l.s.teams * Weights<VEC, NV>::count(l.s.warps) : 0));
    l.depth = kMaxDepth;
    while (l.depth > 1 && l.depth * slot + fixed > (size_t)kSmemBudget) --l.depth;
    l.smem = l.depth * slot + fixed;
    const bool spread = k.tokens >= (int64_t)sms * l.s.teams || threads <= 128;  // every SM has work
    if ((l.depth >= 2 && spread) || l.s.teams == 1) return l;
  }
}

template <typename TB, typename TX, int VEC, int NV>
cudaError_t fwd_launch(const FwdArgs& a, cudaStream_t st) {
  const Layout l = norm_layout<TB, TX, VEC, NV>(a.k, 1, false);
  static std::atomic<uint64_t> known{0};
  const auto kernel = norm_fwd_kernel<TB, TX, VEC, NV>;
  const cudaError_t e = allow_smem(kernel, known);
  if (e != cudaSuccess) return e;
  int64_t rows = 0;
  const int64_t ctas = norm_ranges(a.k.tokens, l.s.teams, &rows);
  return launch_overlapped(kernel, (unsigned)ctas, l.s.threads, l.smem, st, a.k, (const TX*)a.x,
                           a.xs, (const TB*)a.block, a.bs, (TX*)a.x_out, a.xos, (TB*)a.y, a.ys,
                           a.stats, a.y_q, a.qs, a.y_e, a.es, rows, l.s.warps, l.depth);
}

template <typename TB, typename TX, int VEC>
cudaError_t fwd_pick(const FwdArgs& a, cudaStream_t st) {
  if constexpr (VEC > 1) {
    if (a.k.C <= 256) return fwd_launch<TB, TX, VEC, 8 / VEC>(a, st);
    if (a.k.C <= 512) return fwd_launch<TB, TX, VEC, 16 / VEC>(a, st);
    return fwd_launch<TB, TX, VEC, 32 / VEC>(a, st);
  }
  if (a.k.C <= 4096) return fwd_launch<TB, TX, VEC, 8 / VEC>(a, st);  // more would not fit the registers
  return fwd_launch<TB, TX, VEC, 16 / VEC>(a, st);
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

template <typename TB, typename TX, int VEC, int NV>
cudaError_t bwd_launch(BwdArgs& a, cudaStream_t st) {
  const Layout l = norm_layout<TB, TX, VEC, NV>(a.k, 2, true);
  static std::atomic<uint64_t> known{0};
  const auto kernel = norm_bwd_kernel<TB, TX, VEC, NV>;
  const cudaError_t e = allow_smem(kernel, known);
  if (e != cudaSuccess) return e;
  a.ctas = (int)norm_ranges(a.k.tokens, l.s.teams, &a.rows_per_cta);
  return launch_overlapped(kernel, (unsigned)a.ctas, l.s.threads, l.smem, st, a.k, (const TX*)a.x,
                           a.xs, (const TB*)a.block, a.bs, a.stats, (const TX*)a.dx_out, a.dxos,
                           (const TB*)a.dy, a.dys, (TX*)a.dx, a.dxs, (TB*)a.dblock, a.dbs,
                           a.part_pre, a.part_e, a.rows_per_cta, l.s.warps, l.depth);
}

// 16 channels a thread where rows are aligned and that wide (32640 x 1024 bf16: 85 us,
// with 8 a thread 107 us, when that was measured; 76 us now); 8 for rows that start
// anywhere, where 16 cost more in single accesses than they save (5003 x 997 fp32:
// 49 us, 87 us; 45 us now).
template <typename TB, typename TX, int VEC>
cudaError_t bwd_pick(BwdArgs& a, cudaStream_t st) {
  if (a.k.C <= (VEC > 1 ? 256 : 4096)) return bwd_launch<TB, TX, VEC, 8 / VEC>(a, st);
  return bwd_launch<TB, TX, VEC, 16 / VEC>(a, st);
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
      !aligned_to(x_out, ex) || !aligned_to(y, eb) ||
      !in_place_ok(p->tokens, x, x_stride, x_out, x_out_stride))
    return GS_ERR_INVALID_ARG;
  if (y_q && !ckpt_ok(p->tokens, p->channels, y_q, q_stride, y_e, e_stride)) return GS_ERR_INVALID_ARG;
  const int vec = 16 / eb;
  const bool wide = p->channels % vec == 0 && rows_aligned(x, x_stride, ex, 16) &&
                    rows_aligned(block, block_stride, eb, 16) &&
                    rows_aligned(x_out, x_out_stride, ex, 16) && rows_aligned(y, y_stride, eb, 16);
  const FwdArgs a{make_norm(*p), x, block, x_out, y, x_stride, block_stride, x_out_stride,
                  y_stride, (float4*)stats, y_q, q_stride, y_e, e_stride};
  cudaStream_t st = (cudaStream_t)stream;
  GS_CUDA(GS_NORM_TYPES(p, fwd_types, a, wide, st));
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
                        !aligned_to(dblock, eb) ||
                        !in_place_ok(p->tokens, dx_out, dx_out_stride, dx, dx_stride) ||
                        !in_place_ok(p->tokens, dy, dy_stride, dblock, dblock_stride)))
    return GS_ERR_INVALID_ARG;
  if ((dw_pre || need_e) &&
      (!workspace || !aligned16(workspace) ||
       ws_bytes < gs_gated_norm_workspace_bytes(p->channels, p->groups)))
    return GS_ERR_INVALID_ARG;
  const int vec = 16 / eb;
  const bool wide = p->channels % vec == 0 && rows_aligned(x_out, x_stride, ex, 16) &&
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
  } else {
    a.part_pre = a.part_e = nullptr;
  }
  if (dw_pre || need_e) {
    GS_CUDA(launch_overlapped(norm_sums_kernel, dim3((unsigned)div_up(p->channels, 32), need_e ? 2 : 1),
                              dim3(32, 32), 0, st, a.k, p->dtype, a.part_pre, a.part_e,
                              a.rows_per_cta, a.ctas, dw_pre, dw_post, dgate, dres_scale));
  }
  return GS_OK;
}
