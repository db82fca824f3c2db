// linear_attn.cu -- gs_linear_attn_fwd, _bwd, _step: linear attention with a decay for
// each head.
//
//   S_t = d S_{t-1} + k_t v_t^T,  o_t = scale q_t S_t,  d = e^log_decay
//
// In chunks of 64 tokens (n of them, i and j counted from a chunk's start, S its state
// at the start):
//   o_i = scale (d^(i+1) q_i S + sum_{j <= i} d^(i-j) (q_i k_j) v_j)
//   S'  = d^n S + sum_j d^(n-1-j) k_j v_j^T
//
// The backward pass is the same sum three times with the arguments in other places, of
// which two go through the tokens backwards.  With R the gradient of the state after a
// token's update, R_t = d R_{t+1} + scale q_t do_t^T:
//   dq_t = scale S_t do_t   queries do, keys v, values k, state S^T, forwards
//   dk_t = R_t v_t          queries v, keys do, values q, state R^T, backwards
//   dv_t = R_t^T k_t        queries k, keys q, values do, state R, backwards
// Backwards the decay comes after a token's term instead of before it (d^i and d^(n-j)
// in place of d^(i+1) and d^(n-1-j)).
//
// Tokens are split into segments.  One kernel sums each segment's own part of the state,
// a second one goes through the segments' parts and leaves each one's state at its start
// and a group's last state, a third one forms the outputs, segment by segment, with the
// state in registers (fp32) between a segment's chunks.
//
// Products are on the tensor cores (mma.sync: chains of products of 16 x 64 results per
// warp whose operands come from one another's registers), sums and states fp32.  What is
// rounded to the inputs' type on the way: the decayed products q_i k_j, and the state
// where it is multiplied by a query (not where it is kept); each of the two parts of an
// output is rounded once there and once more as the output.  The decayed keys of a
// state's sum are taken as 3 (bf16) or 2 (fp16) terms, exact to fp32's rounding, for the
// states that are handed on, and as 2 terms for those inside a segment.
#include <atomic>
#include <type_traits>

#include "activation.cuh"

namespace gs {
namespace {

constexpr int kL = 64;  // tokens of a chunk
constexpr int kTilesOfRows = kL / 16;
// The padded head (64 or 128 channels) sets the warps: each has 16 rows of the state.
template <int DP>
constexpr int kWarps = DP / 16;
template <int DP>
constexpr int kThreads = 32 * kWarps<DP>;

struct Side {  // heads that are read or written
  void* p;
  int64_t token, head;  // strides, elements
  int32_t dim;
  int32_t of_key;       // one head for rep query heads
  int32_t wide;         // rows start on 16-byte boundaries
};

struct Split {  // tokens in groups, groups in segments
  int64_t tokens;
  const int32_t* offsets;  // NULL: one group
  int32_t groups, seg;
};

// Segment `slot` of the groups one after the other.  Group g's segments begin at slot
// offsets[g] / seg + g, where no other group's can be.
struct Span {
  int32_t group;
  int64_t start;
  int32_t n;      // tokens; 0: none here
};
__device__ __forceinline__ int64_t offset_of(const Split& s, int g) {
  if (!s.offsets) return g ? s.tokens : 0;
  const int64_t o = s.offsets[g];
  return o < 0 ? 0 : o > s.tokens ? s.tokens : o;
}
__device__ __forceinline__ int64_t first_slot(const Split& s, int g) { return offset_of(s, g) / s.seg + g; }
__device__ __forceinline__ Span span_of(const Split& s, int64_t slot) {
  int lo = 0, hi = s.groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first_slot(s, mid) <= slot) lo = mid;
    else hi = mid - 1;
  }
  const int64_t in = slot - first_slot(s, lo), begin = offset_of(s, lo), end = offset_of(s, lo + 1);
  const int64_t start = begin + in * s.seg, left = end - start;
  return Span{lo, start, in < 0 || left <= 0 ? 0 : (int)(left < s.seg ? left : s.seg)};
}

// ---- mma.sync and its operands ---------------------------------------------
__device__ __forceinline__ uint32_t smem_at(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
template <typename T>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Tiles in shared memory: rows of DP 16-bit elements, whose 16-byte granules are swizzled
// by the row.  `at`: the byte address of column c (a multiple of 8) of row r.
template <int DP>
__device__ __forceinline__ uint32_t at(uint32_t base, int r, int c) {
  return base + r * (DP * 2) + (((c >> 3) ^ (r & 7)) << 4);
}
// The four 8 x 8 matrices of a 16 x 16 block at (r0, c0), lane's row address:
// rows first (r0, r0 + 8 at c0, then at c0 + 8) or columns first.
template <int DP>
__device__ __forceinline__ uint32_t block_rows(uint32_t base, int r0, int c0, int lane) {
  return at<DP>(base, r0 + (lane & 15), c0 + (lane >> 4) * 8);
}
template <int DP>
__device__ __forceinline__ uint32_t block_cols(uint32_t base, int r0, int c0, int lane) {
  return at<DP>(base, r0 + (lane & 7) + (lane >> 4) * 8, c0 + (lane >> 3 & 1) * 8);
}

// kL rows (n of them there) of `dim` channels to a tile; zeros elsewhere.  The copies of
// whole granules are asynchronous.
template <typename T, int DP>
__device__ __forceinline__ void load_rows(T* tile, const T* from, int64_t stride, int n, int dim, bool wide) {
  constexpr int kG = DP / 8;
#pragma unroll 4
  for (int i = threadIdx.x; i < kL * kG; i += kThreads<DP>) {
    const int r = i / kG, c = i % kG * 8;
    const uint32_t to = at<DP>(smem_at(tile), r, c);
    const T* p = from + r * stride + c;
    if (r < n && wide && c + 8 <= dim) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p) : "memory");
    } else {
      uint32_t w[4] = {0, 0, 0, 0};
      if (r < n) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < dim)
            w[j / 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(p + j) << (j % 2 * 16);
      }
      asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                   : "memory");
    }
  }
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// d^x with a = log2 d <= 0; a decay that leaves nothing after one token counts as 2^-1000.
__device__ __forceinline__ float log2_decay(const float* log_decay, int h) {
  const float a = log_decay[h] * 1.4426950408889634f;
  return a < -1000.f ? -1000.f : a;
}

// The state's rows 16 w .. past n tokens: st <- decay st + sum_j weight_j key_j value_j^T,
// the weighted keys as TERMS terms.  weight_j = mul d^(n - 1 - j + shift).  In fp16 keys
// and state take a power of two meanwhile, so that the largest key with the largest weight
// is near 2^13: the terms of small ones would be below fp16's range.
template <typename T, int DP, int TERMS>
__device__ __forceinline__ void add_tokens(float (&st)[DP / 8][4], float decay, uint32_t keys, uint32_t values,
                                           int warp, int lane, int n, float a, int shift, float mul) {
  const int t = lane & 3;
  uint32_t raw[kL / 16][4];
  // (row g, tokens 2t..), (g + 8, 2t..), (g, 2t + 8..), (g + 8, 2t + 8..) of each 16 tokens
#pragma unroll
  for (int ks = 0; ks < kL / 16; ++ks) ldm4t(raw[ks], block_cols<DP>(keys, ks * 16, warp * 16, lane));
  float back = 1.f;
  if constexpr (std::is_same<T, __half>::value) {
    uint32_t top = 0;  // magnitudes compare as whole numbers
#pragma unroll
    for (int ks = 0; ks < kL / 16; ++ks)
#pragma unroll
      for (int r = 0; r < 4; ++r) top = max(top, max(raw[ks][r] & 0x7fffu, raw[ks][r] >> 16 & 0x7fffu));
#pragma unroll
    for (int o = 16; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float m = __half2float(__ushort_as_half((unsigned short)top)) * fabsf(mul) * power2(a * (float)shift);
    const int e = m > 0.f ? min(max((int)(__float_as_uint(m) >> 23) - 127 - 13, -100), 100) : 0;
    back = __uint_as_float((uint32_t)(127 + e) << 23);
    const float fit = __uint_as_float((uint32_t)(127 - e) << 23);
    decay *= fit;
    mul *= fit;
  }
#pragma unroll
  for (int i = 0; i < DP / 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) st[i][j] *= decay;
#pragma unroll
  for (int ks = 0; ks < kL / 16; ++ks) {
    if (ks * 16 >= n) break;
    float w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int tok = ks * 16 + 2 * t + (j & 1) + (j >> 1) * 8;
      w[j] = mul * power2(a * (float)(max(n - 1 - tok, 0) + shift));
    }
    uint32_t term[TERMS][4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const Pack<T, 2> e = *reinterpret_cast<const Pack<T, 2>*>(&raw[ks][r]);
      float x = to_f32(e.v[0]) * w[r >> 1 << 1], y = to_f32(e.v[1]) * w[(r >> 1 << 1) + 1];
#pragma unroll
      for (int i = 0; i < TERMS; ++i) {
        term[i][r] = pair_word<T>(x, y);
        const Pack<T, 2> q = *reinterpret_cast<const Pack<T, 2>*>(&term[i][r]);
        x -= to_f32(q.v[0]);
        y -= to_f32(q.v[1]);
      }
    }
#pragma unroll
    for (int c = 0; c < DP; c += 16) {
      uint32_t b[4];
      ldm4t(b, block_rows<DP>(values, ks * 16, c, lane));
#pragma unroll
      for (int i = 0; i < TERMS; ++i) {
        mma16<T>(st[c / 8], term[i], b[0], b[1]);
        mma16<T>(st[c / 8 + 1], term[i], b[2], b[3]);
      }
    }
  }
  if constexpr (std::is_same<T, __half>::value) {
#pragma unroll
    for (int i = 0; i < DP / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) st[i][j] *= back;
  }
}

// ---- each segment's part of the state ---------------------------------------
struct Part {
  Side key, value;
  float mul;
  int32_t back, shift;  // tokens from the last to the first
  float* to;            // [slots][heads][DP][DP]
};
struct PartsArgs {
  Split split;
  int32_t heads, rep;
  const float* log_decay;
  Part part[2];
};

template <typename T>
__device__ __forceinline__ const T* head_at(const Side& s, int h, int rep, int64_t token) {
  return (const T*)s.p + (int64_t)(s.of_key ? h / rep : h) * s.head + token * s.token;
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads<DP>) attn_parts_kernel(const __grid_constant__ PartsArgs p) {
  extern __shared__ __align__(128) uint8_t smem[];
  launch_dependents();
  wait_for_previous();
  T* tiles = (T*)smem;  // [2][keys, values][kL][DP]
  constexpr int kTile = kL * DP;
  const int h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Part& part = p.part[blockIdx.z];
  const Span s = span_of(p.split, blockIdx.x);
  if (s.n == 0) return;
  const float a = log2_decay(p.log_decay, h);
  const int64_t from = part.back ? s.start + s.n - 1 : s.start;
  const int64_t step = part.back ? -1 : 1;
  const T* k = head_at<T>(part.key, h, p.rep, from);
  const T* v = head_at<T>(part.value, h, p.rep, from);
  auto load = [&](int c) {
    T* to = tiles + (c & 1) * 2 * kTile;
    const int n = min(kL, s.n - c * kL);
    load_rows<T, DP>(to, k + step * c * kL * part.key.token, step * part.key.token, n, part.key.dim, part.key.wide);
    load_rows<T, DP>(to + kTile, v + step * c * kL * part.value.token, step * part.value.token, n, part.value.dim,
                     part.value.wide);
    copies_commit();
  };
  float st[DP / 8][4] = {};
  const int chunks = (s.n + kL - 1) / kL;
  load(0);
  for (int c = 0; c < chunks; ++c) {
    copies_wait<0>();
    __syncthreads();
    if (c + 1 < chunks) load(c + 1);
    const int n = min(kL, s.n - c * kL);
    const uint32_t keys = smem_at(tiles + (c & 1) * 2 * kTile);
    add_tokens<T, DP, std::is_same<T, __half>::value ? 2 : 3>(st, power2(a * (float)n), keys, keys + kTile * 2, warp,
                                                               lane, n, a, part.shift, part.mul);
  }
  float* to = part.to + ((int64_t)blockIdx.x * p.heads + h) * DP * DP + (warp * 16 + (lane >> 2)) * DP + (lane & 3) * 2;
#pragma unroll
  for (int i = 0; i < DP / 8; ++i) {
    *reinterpret_cast<float2*>(to + i * 8) = make_float2(st[i][0], st[i][1]);
    *reinterpret_cast<float2*>(to + 8 * DP + i * 8) = make_float2(st[i][2], st[i][3]);
  }
}

// ---- the states at the segments' starts, in place of their parts ---------------
struct Scan {
  const float* edge;  // [groups][heads][D][E] or NULL (zeros)
  float* last;        // likewise, or NULL
  float* parts;
  int32_t back;
};
struct ScanArgs {
  Split split;
  int32_t heads, D, E;
  const float* log_decay;
  Scan scan[2];
  int32_t scans;
};

template <int DP>
__global__ void __launch_bounds__(128) attn_scan_kernel(const __grid_constant__ ScanArgs p) {
  launch_dependents();
  wait_for_previous();
  const Scan& k = p.scan[blockIdx.z];
  const int h = blockIdx.y, i = (blockIdx.x % (DP * DP / 512)) * 512 + threadIdx.x * 4;
  const int g = blockIdx.x / (DP * DP / 512);
  const int row = i / DP, col = i % DP;
  const float a = log2_decay(p.log_decay, h);
  const int64_t begin = offset_of(p.split, g), end = offset_of(p.split, g + 1);
  const int64_t first = begin / p.split.seg + g;
  const int slots = end > begin ? (int)((end - begin + p.split.seg - 1) / p.split.seg) : 0;
  const int tail = (int)(end - begin - (int64_t)(slots - 1) * p.split.seg);
  const int64_t mat = ((int64_t)g * p.heads + h) * p.D * p.E + (int64_t)row * p.E + col;
  float4 s = make_float4(0, 0, 0, 0);
  float* sv = &s.x;
  if (k.edge && row < p.D)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (col + j < p.E) sv[j] = k.edge[mat + j];
  const float full = power2(a * (float)p.split.seg), rest = power2(a * (float)tail);
  const int64_t stride = (int64_t)p.heads * DP * DP;
  float* at = k.parts + (first * p.heads + h) * DP * DP + i;
  const int last = slots - 1;
  constexpr int kAhead = 8;
  for (int b = 0; b < slots; b += kAhead) {
    float4 u[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (b + j < slots) u[j] = *reinterpret_cast<const float4*>(at + stride * (k.back ? last - b - j : b + j));
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (b + j >= slots) break;
      const int slot = k.back ? last - b - j : b + j;
      *reinterpret_cast<float4*>(at + stride * slot) = s;
      const float d = slot == last ? rest : full;
      s.x = s.x * d + u[j].x, s.y = s.y * d + u[j].y, s.z = s.z * d + u[j].z, s.w = s.w * d + u[j].w;
    }
  }
  if (k.last && row < p.D)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (col + j < p.E) k.last[mat + j] = sv[j];
}

// ---- outputs -----------------------------------------------------------------
struct OutArgs {
  Split split;
  int32_t heads, rep;    // query heads
  int32_t shared;        // outputs are summed over the rep query heads of a key head
  Side query, key, value, out;
  const float* log_decay;
  const float* states;   // [slots][heads][DP][DP], NULL: no group has more than one segment
  const float* edge;     // [groups][heads][..] or NULL (zeros)
  int32_t transposed;    // states are stored [values' channels][keys' channels]
  int32_t back, shift;
  float mul_inner, mul_state, mul_key;
  float* sums;           // [tokens][key heads][DP], where shared and rep > 1
};

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads<DP>) attn_out_kernel(const __grid_constant__ OutArgs p) {
  extern __shared__ __align__(128) uint8_t smem[];
  launch_dependents();
  wait_for_previous();
  constexpr bool kHalfType = std::is_same<T, __half>::value;
  constexpr int kTile = kL * DP;
  constexpr int kSplits = kWarps<DP> / kTilesOfRows;  // of the values' channels over warps
  constexpr int kWidth = DP / kSplits;
  T* tiles = (T*)smem;                          // [2][queries, keys, values][kL][DP]
  T* state = tiles + 6 * kTile;                 // [DP][DP]
  __shared__ float top[kWarps<DP>];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rt = warp % kTilesOfRows, col0 = warp / kTilesOfRows * kWidth;
  const Span s = span_of(p.split, blockIdx.x);
  if (s.n == 0) return;
  const int64_t from = p.back ? s.start + s.n - 1 : s.start, step = p.back ? -1 : 1;
  const int chunks = (s.n + kL - 1) / kL;
  const int reps = p.shared ? p.rep : 1;
  const uint32_t state_at = smem_at(state);

  for (int r = 0; r < reps; ++r) {
    const int h = p.shared ? blockIdx.y * p.rep + r : blockIdx.y;
    const float a = log2_decay(p.log_decay, h);
    const T* q = head_at<T>(p.query, h, p.rep, from);
    const T* k = head_at<T>(p.key, h, p.rep, from);
    const T* v = head_at<T>(p.value, h, p.rep, from);
    auto load = [&](int c) {
      T* to = tiles + (c & 1) * 3 * kTile;
      const int n = min(kL, s.n - c * kL);
      const int64_t at = step * c * kL;
      load_rows<T, DP>(to, q + at * p.query.token, step * p.query.token, n, p.query.dim, p.query.wide);
      load_rows<T, DP>(to + kTile, k + at * p.key.token, step * p.key.token, n, p.key.dim, p.key.wide);
      load_rows<T, DP>(to + 2 * kTile, v + at * p.value.token, step * p.value.token, n, p.value.dim, p.value.wide);
      copies_commit();
    };
    __syncthreads();
    load(0);

    // the state: 16 rows (keys' channels) a warp
    float st[DP / 8][4];
    {
      const bool edge = !p.states;
      const int ld = edge ? (p.transposed ? p.key.dim : p.value.dim) : DP;
      const float* src = edge ? (p.edge ? p.edge + ((int64_t)s.group * p.heads + h) * p.key.dim * p.value.dim : nullptr)
                              : p.states + ((int64_t)blockIdx.x * p.heads + h) * DP * DP;
#pragma unroll
      for (int i = 0; i < DP / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = warp * 16 + g + (j >> 1) * 8, col = i * 8 + 2 * t + (j & 1);
          const bool in = src && (!edge || (row < p.key.dim && col < p.value.dim));
          st[i][j] = in ? src[p.transposed ? (int64_t)col * ld + row : (int64_t)row * ld + col] : 0.f;
        }
    }
    // powers of the decay that the thread needs: between rows g, g + 8 and columns 2t, 2t + 1
    const float d8 = power2(a * 8.f), d16 = power2(a * 16.f);
    const float b0 = p.mul_inner * power2(a * (float)(g - 2 * t + 8)), b1 = p.mul_inner * power2(a * (float)(g - 2 * t + 7));
    const bool in0 = g >= 2 * t, in1 = g >= 2 * t + 1;
    const float d0 = p.mul_inner * power2(a * (float)max(g - 2 * t, 0)), d1 = p.mul_inner * power2(a * (float)max(g - 2 * t - 1, 0));
    const float row_first = p.mul_state * power2(a * (float)(rt * 16 + g + 1 - p.shift));

    for (int c = 0; c < chunks; ++c) {
      const int n = min(kL, s.n - c * kL);
      // the state as the products take it; fp16 with a power of two that keeps it in range
      float unscale = 1.f, rescale = 1.f;
      if constexpr (kHalfType) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < DP / 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) m = fmaxf(m, fabsf(st[i][j]));
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) top[warp] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWarps<DP>; ++i) m = fmaxf(m, top[i]);
        const int e = min(max((int)(__float_as_uint(m) >> 23) - 127 - 13, -100), 100);
        rescale = __uint_as_float((uint32_t)(127 - e) << 23);
        unscale = __uint_as_float((uint32_t)(127 + e) << 23);
      }
#pragma unroll
      for (int i = 0; i < DP / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          const int row = warp * 16 + g + (j >> 1) * 8;
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(at<DP>(state_at, row, i * 8) + t * 4),
                       "r"(pair_word<T>(st[i][j] * rescale, st[i][j + 1] * rescale))
                       : "memory");
        }
      copies_wait<0>();
      __syncthreads();
      if (c + 1 < chunks) load(c + 1);
      const uint32_t qs = smem_at(tiles + (c & 1) * 3 * kTile), ks = qs + kTile * 2, vs = ks + kTile * 2;

      // queries times the state
      uint32_t qf[DP / 16][4];
#pragma unroll
      for (int i = 0; i < DP / 16; ++i) ldm4(qf[i], block_rows<DP>(qs, rt * 16, i * 16, lane));
      float o[kWidth / 8][4] = {};
#pragma unroll
      for (int i = 0; i < DP / 16; ++i)
#pragma unroll
        for (int x = 0; x < kWidth; x += 16) {
          uint32_t b[4];
          ldm4t(b, block_rows<DP>(state_at, i * 16, col0 + x, lane));
          mma16<T>(o[x / 8], qf[i], b[0], b[1]);
          mma16<T>(o[x / 8 + 1], qf[i], b[2], b[3]);
        }
      const float f0 = row_first * unscale, f1 = f0 * d8;
#pragma unroll
      for (int i = 0; i < kWidth / 8; ++i) o[i][0] *= f0, o[i][1] *= f0, o[i][2] *= f1, o[i][3] *= f1;

      // queries times keys, decayed, times values: blocks of 16 keys up to the diagonal
      float far = 1.f;  // d^(16 (rt - jb - 1))
      for (int jb = rt; jb >= 0; --jb) {
        float w[2][4] = {};
#pragma unroll
        for (int i = 0; i < DP / 16; ++i) {
          uint32_t b[4];
          ldm4(b, block_cols<DP>(ks, jb * 16, i * 16, lane));
          mma16<T>(w[0], qf[i], b[0], b[1]);
          mma16<T>(w[1], qf[i], b[2], b[3]);
        }
        uint32_t pf[4];
        if (jb == rt) {
          pf[0] = pair_word<T>(in0 ? w[0][0] * d0 : 0.f, in1 ? w[0][1] * d1 : 0.f);
          pf[1] = pair_word<T>(w[0][2] * b0, w[0][3] * b1);
          pf[2] = 0;
          pf[3] = pair_word<T>(in0 ? w[1][2] * d0 : 0.f, in1 ? w[1][3] * d1 : 0.f);
        } else {
          const float f8 = far * d8;
          pf[0] = pair_word<T>(w[0][0] * (b0 * f8), w[0][1] * (b1 * f8));
          pf[1] = pair_word<T>(w[0][2] * (b0 * d8 * f8), w[0][3] * (b1 * d8 * f8));
          pf[2] = pair_word<T>(w[1][0] * (b0 * far), w[1][1] * (b1 * far));
          pf[3] = pair_word<T>(w[1][2] * (b0 * f8), w[1][3] * (b1 * f8));
          far *= d16;
        }
#pragma unroll
        for (int x = 0; x < kWidth; x += 16) {
          uint32_t b[4];
          ldm4t(b, block_rows<DP>(vs, jb * 16, col0 + x, lane));
          mma16<T>(o[x / 8], pf, b[0], b[1]);
          mma16<T>(o[x / 8 + 1], pf, b[2], b[3]);
        }
      }

      if (c + 1 < chunks)
        add_tokens<T, DP, 2>(st, power2(a * (float)n), ks, vs, warp, lane, n, a, p.shift, p.mul_key);

      // the sums over a key head's query heads, one after the other
      const int64_t tok = from + step * c * kL;
      if (reps > 1) {
#pragma unroll
        for (int i = 0; i < kWidth / 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            const int row = rt * 16 + g + (j >> 1) * 8;
            if (row >= n) continue;
            float2* x = reinterpret_cast<float2*>(p.sums + ((tok + step * row) * (p.heads / p.rep) + blockIdx.y) * DP +
                                                  col0 + i * 8 + 2 * t);
            if (r) {
              const float2 y = *x;
              o[i][j] += y.x, o[i][j + 1] += y.y;
            }
            if (r + 1 < reps) *x = make_float2(o[i][j], o[i][j + 1]);
          }
      }
      __syncthreads();  // the state, the queries and the keys have been read
      if (r + 1 < reps) continue;
      // through the queries' tile, whose rows these are, to memory
#pragma unroll
      for (int i = 0; i < kWidth / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; j += 2)
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(at<DP>(qs, rt * 16 + g + (j >> 1) * 8, col0 + i * 8) + t * 4),
                       "r"(pair_word<T>(o[i][j], o[i][j + 1]))
                       : "memory");
      __syncwarp();
      T* to = (T*)p.out.p + (int64_t)blockIdx.y * p.out.head + tok * p.out.token;
#pragma unroll
      for (int i = 0; i < 16 * kWidth / 8 / 32; ++i) {
        const int row = rt * 16 + i * (32 / (kWidth / 8)) + lane / (kWidth / 8), col = col0 + lane % (kWidth / 8) * 8;
        if (row >= n || col >= p.out.dim) continue;
        const uint8_t* e = (const uint8_t*)(tiles + (c & 1) * 3 * kTile) + (at<DP>(0, row, col));
        T* x = to + step * row * p.out.token + col;
        if (p.out.wide && col + 8 <= p.out.dim) {
          *reinterpret_cast<uint4*>(x) = *reinterpret_cast<const uint4*>(e);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (col + j < p.out.dim) x[j] = reinterpret_cast<const T*>(e)[j];
        }
      }
    }
  }
}

// ---- single tokens -------------------------------------------------------------
struct StepArgs {
  Side q, k, v, out;
  int32_t heads, rep;
  const float* log_decay;
  float scale;
  float* state;  // [tokens][heads][D][E]
};

// One head of one token a block: VEC neighbouring columns of the state a thread, whose
// rows the block's threads share out; read, updated, written and multiplied by the query
// in one pass.  Bound by the state's bytes.
template <typename T, int VEC>
__global__ void __launch_bounds__(128) attn_step_kernel(const __grid_constant__ StepArgs p) {
  launch_dependents();
  wait_for_previous();
  __shared__ float sums[128 * VEC];
  __shared__ float qk[2][256];
  const int h = blockIdx.y, D = p.q.dim, E = p.v.dim;
  const int64_t b = blockIdx.x;
  const T* q = head_at<T>(p.q, h, p.rep, b);
  const T* k = head_at<T>(p.k, h, p.rep, b);
  const T* v = head_at<T>(p.v, h, p.rep, b);
  for (int i = threadIdx.x; i < D; i += 128) {
    qk[0][i] = to_f32(q[i]);
    qk[1][i] = to_f32(k[i]);
  }
  const int across = (E + VEC - 1) / VEC;            // threads side by side
  const int down = 128 / across, c = threadIdx.x % across, r0 = threadIdx.x / across;
  const float d = expf(p.log_decay[h]);
  float value[VEC], acc[VEC] = {};
  if (r0 < down)
#pragma unroll
    for (int j = 0; j < VEC; ++j) value[j] = to_f32(v[c * VEC + j]);
  __syncthreads();
  float* s = p.state + (b * p.heads + h) * D * E + c * VEC;
  if (r0 < down) {
    constexpr int kAhead = 8;  // rows under way
    for (int r = r0; r < D; r += kAhead * down) {
      Pack<float, VEC> m[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (r + i * down < D) m[i] = load_pack<float, VEC>(s + (int64_t)(r + i * down) * E);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int row = r + i * down;
        if (row >= D) break;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          m[i].v[j] = d * m[i].v[j] + qk[1][row] * value[j];
          acc[j] += qk[0][row] * m[i].v[j];
        }
        store_pack<float, VEC>(s + (int64_t)row * E, m[i]);
      }
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) sums[r0 * E + c * VEC + j] = acc[j];
  }
  __syncthreads();
  T* out = (T*)p.out.p + (int64_t)h * p.out.head + b * p.out.token;
  for (int i = threadIdx.x; i < E; i += 128) {
    float o = 0.f;
    for (int r = 0; r < down; ++r) o += sums[r * E + i];
    out[i] = from_f32<T>(p.scale * o);
  }
}

// ---- host ------------------------------------------------------------------------
constexpr int64_t kMaxTokens = ((int64_t)1 << 31) - 1;

// Tokens of a segment: long enough that its states' bytes are few beside its tokens', short
// enough that there is work for every SM.
int32_t segment_tokens(int64_t tokens, int32_t heads, bool backward) {
  const int64_t chunks = div_up(tokens, kL) * heads;
  int64_t m = chunks / ((int64_t)device_sms() * 8);
  const int64_t least = backward ? 2 : 1;
  m = m < least ? least : m > 16 ? 16 : m;
  return (int32_t)m * kL;
}

struct Room {
  float *states, *grads, *sums[2];
  size_t bytes;
  Room(void* ws, int64_t slots, int32_t heads, int32_t key_heads, int32_t dp, int64_t tokens, bool backward) {
    char* base = (char*)ws;
    size_t at = 0;
    auto take = [&](size_t n) {
      char* p = base + at;
      at += (n + 255) / 256 * 256;
      return (float*)p;
    };
    const size_t one = sizeof(float) * slots * heads * dp * dp;
    const size_t sum = backward && heads > key_heads ? sizeof(float) * tokens * key_heads * dp : 0;
    states = take(one);
    grads = take(backward ? one : 0);
    sums[0] = take(sum);
    sums[1] = take(sum);
    bytes = at;
  }
};

bool shape_ok(const gs_linear_attn* a) {
  return a->tokens >= 0 && a->tokens <= kMaxTokens && a->q_heads >= 1 && a->q_heads <= 65535 && a->k_heads >= 1 &&
         a->q_heads % a->k_heads == 0 && a->dim >= 1 && a->dim <= GS_LINEAR_ATTN_MAX_DIM && a->vdim >= 1 &&
         a->vdim <= GS_LINEAR_ATTN_MAX_DIM && a->groups >= 1 && a->groups <= (1 << 24) &&
         (a->dtype == GS_BF16 || a->dtype == GS_F16);
}
bool aligned_or_none(const gs_linear_attn* a) {
  return a->log_decay && aligned_to(a->log_decay, 4) && aligned_to(a->group_offsets, 4) && aligned_to(a->state, 4);
}
int padded_dim(const gs_linear_attn* a) { return a->dim <= 64 && a->vdim <= 64 ? 64 : 128; }

bool side(Side* s, const gs_linear_attn* a, const gs_attn_heads* h, int32_t dim, bool of_key, bool output) {
  if (!h || !h->p || !aligned_to(h->p, 2)) return false;
  constexpr int64_t kMost = (int64_t)1 << 40;
  if (h->token >= kMost || h->token <= -kMost || h->head >= kMost || h->head <= -kMost) return false;
  const int32_t heads = of_key ? a->k_heads : a->q_heads;
  if (output) {  // no two elements in one place
    const int64_t t = h->token < 0 ? -h->token : h->token, e = h->head < 0 ? -h->head : h->head;
    const bool many = a->tokens > 1;
    if ((heads > 1 && e < dim) || (many && t < dim)) return false;
    if (heads > 1 && many && !(t >= e * (heads - 1) + dim || e >= t * (a->tokens - 1) + dim)) return false;
  }
  *s = Side{h->p, h->token, h->head, dim, of_key ? 1 : 0,
            aligned16(h->p) && (a->tokens < 2 || h->token % 8 == 0) && (heads < 2 || h->head % 8 == 0) ? 1 : 0};
  return true;
}

template <typename T, int DP>
constexpr int kPartsSmem = 4 * kL * DP * 2;
template <typename T, int DP>
constexpr int kOutSmem = (6 * kL * DP + DP * DP) * 2;

// Dynamic shared memory beyond 48 KB, asked for once per kernel and device.
template <typename F>
bool allow_smem(F kernel, std::atomic<uint64_t>& known, int bytes) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (known.load(std::memory_order_acquire) & bit) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  known.fetch_or(bit, std::memory_order_release);
  return true;
}

template <typename T, int DP>
gs_status run_parts(const PartsArgs& p, int64_t slots, int parts, cudaStream_t st) {
  static std::atomic<uint64_t> known{0};
  if (!allow_smem(attn_parts_kernel<T, DP>, known, kPartsSmem<T, DP>)) {
    (void)cudaGetLastError();
    return GS_ERR_CUDA;
  }
  GS_CUDA(launch_overlapped(attn_parts_kernel<T, DP>, dim3((unsigned)slots, p.heads, parts), dim3(kThreads<DP>),
                            kPartsSmem<T, DP>, st, p));
  return GS_OK;
}
template <int DP>
gs_status run_scan(const ScanArgs& p, cudaStream_t st) {
  const int64_t blocks = (int64_t)p.split.groups * (DP * DP / 512);
  if (blocks > INT32_MAX) return GS_ERR_INVALID_ARG;
  GS_CUDA(launch_overlapped(attn_scan_kernel<DP>, dim3((unsigned)blocks, p.heads, p.scans), dim3(128), 0, st, p));
  return GS_OK;
}
template <typename T, int DP>
gs_status run_out(const OutArgs& p, int64_t slots, cudaStream_t st) {
  static std::atomic<uint64_t> known{0};
  if (!allow_smem(attn_out_kernel<T, DP>, known, kOutSmem<T, DP>)) {
    (void)cudaGetLastError();
    return GS_ERR_CUDA;
  }
  GS_CUDA(launch_overlapped(attn_out_kernel<T, DP>, dim3((unsigned)slots, p.shared ? p.heads / p.rep : p.heads),
                            dim3(kThreads<DP>), kOutSmem<T, DP>, st, p));
  return GS_OK;
}

struct Call {
  Split split;
  int64_t slots;
  int dp, rep;
  Call(const gs_linear_attn* a, bool backward) {
    split = Split{a->tokens, a->group_offsets, a->groups, segment_tokens(a->tokens, a->q_heads, backward)};
    slots = a->tokens / split.seg + a->groups;
    dp = padded_dim(a);
    rep = a->q_heads / a->k_heads;
  }
};

template <typename T, int DP>
gs_status forward(const gs_linear_attn* a, const Call& c, const Side (&s)[4], float* state_out, const Room& room,
                  cudaStream_t st) {
  const bool scan = a->tokens > c.split.seg || state_out;
  if (scan) {
    PartsArgs p{c.split, a->q_heads, c.rep, a->log_decay, {Part{s[1], s[2], 1.f, 0, 0, room.states}, Part{}}};
    gs_status r = run_parts<T, DP>(p, c.slots, 1, st);
    if (r != GS_OK) return r;
    ScanArgs q{c.split, a->q_heads, a->dim, a->vdim, a->log_decay,
               {Scan{a->state, state_out, room.states, 0}, Scan{}}, 1};
    r = run_scan<DP>(q, st);
    if (r != GS_OK) return r;
  }
  OutArgs o{};
  o.split = c.split;
  o.heads = a->q_heads;
  o.rep = c.rep;
  o.query = s[0];
  o.key = s[1];
  o.value = s[2];
  o.out = s[3];
  o.log_decay = a->log_decay;
  o.states = scan ? room.states : nullptr;
  o.edge = a->state;
  o.mul_inner = o.mul_state = a->scale;
  o.mul_key = 1.f;
  return run_out<T, DP>(o, c.slots, st);
}

template <typename T, int DP>
gs_status backward(const gs_linear_attn* a, const Call& c, const Side (&s)[7], const float* dstate_out,
                   float* dstate, const Room& room, cudaStream_t st) {
  const Side &q = s[0], &k = s[1], &v = s[2], &g = s[3];
  const bool scan = a->tokens > c.split.seg || dstate;
  if (scan) {
    PartsArgs p{c.split, a->q_heads, c.rep, a->log_decay,
                {Part{k, v, 1.f, 0, 0, room.states}, Part{q, g, a->scale, 1, 1, room.grads}}};
    gs_status r = run_parts<T, DP>(p, c.slots, 2, st);
    if (r != GS_OK) return r;
    ScanArgs w{c.split, a->q_heads, a->dim, a->vdim, a->log_decay,
               {Scan{a->state, nullptr, room.states, 0}, Scan{dstate_out, dstate, room.grads, 1}}, 2};
    r = run_scan<DP>(w, st);
    if (r != GS_OK) return r;
  }
  OutArgs o{};
  o.split = c.split;
  o.heads = a->q_heads;
  o.rep = c.rep;
  o.log_decay = a->log_decay;
  o.mul_inner = a->scale;
  {
    OutArgs x = o;  // dq
    x.query = g, x.key = v, x.value = k, x.out = s[4];
    x.states = scan ? room.states : nullptr;
    x.edge = a->state;
    x.transposed = 1;
    x.mul_state = a->scale;
    x.mul_key = 1.f;
    const gs_status r = run_out<T, DP>(x, c.slots, st);
    if (r != GS_OK) return r;
  }
  o.back = o.shift = o.shared = 1;
  o.mul_state = 1.f;
  o.mul_key = a->scale;
  o.states = scan ? room.grads : nullptr;
  o.edge = dstate_out;
  {
    OutArgs x = o;  // dk
    x.query = v, x.key = g, x.value = q, x.out = s[5];
    x.transposed = 1;
    x.sums = room.sums[0];
    const gs_status r = run_out<T, DP>(x, c.slots, st);
    if (r != GS_OK) return r;
  }
  OutArgs x = o;  // dv
  x.query = k, x.key = q, x.value = g, x.out = s[6];
  x.sums = room.sums[1];
  return run_out<T, DP>(x, c.slots, st);
}

}  // namespace
}  // namespace gs

using namespace gs;

#define GS_ATTN_CALL(F, ...)                                                      \
  (a->dtype == GS_BF16                                                            \
       ? (c.dp == 64 ? F<__nv_bfloat16, 64>(__VA_ARGS__) : F<__nv_bfloat16, 128>(__VA_ARGS__)) \
       : (c.dp == 64 ? F<__half, 64>(__VA_ARGS__) : F<__half, 128>(__VA_ARGS__)))

extern "C" size_t gs_linear_attn_workspace_bytes(const gs_linear_attn* a, int32_t backward) {
  if (!a || !shape_ok(a)) return 0;
  const Call c(a, backward != 0);
  return Room(nullptr, c.slots, a->q_heads, a->k_heads, c.dp, a->tokens, backward != 0).bytes;
}

extern "C" gs_status gs_linear_attn_fwd(const gs_linear_attn* a, const gs_attn_heads* q, const gs_attn_heads* k,
                                        const gs_attn_heads* v, const gs_attn_heads* out, float* state_out,
                                        void* workspace, size_t ws_bytes, void* stream) {
  if (!a || !shape_ok(a) || !aligned_or_none(a) || (!a->group_offsets && a->groups != 1)) return GS_ERR_INVALID_ARG;
  const Call c(a, false);
  const Room room(workspace, c.slots, a->q_heads, a->k_heads, c.dp, a->tokens, false);
  Side s[4];
  if (!workspace || !aligned16(workspace) || ws_bytes < room.bytes) return GS_ERR_INVALID_ARG;
  if (a->tokens > 0 && (!side(&s[0], a, q, a->dim, false, false) || !side(&s[1], a, k, a->dim, true, false) ||
                        !side(&s[2], a, v, a->vdim, true, false) || !side(&s[3], a, out, a->vdim, false, true)))
    return GS_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  if (a->tokens == 0 && !state_out) return GS_OK;
  if (a->tokens == 0) {
    ScanArgs w{c.split, a->q_heads, a->dim, a->vdim, a->log_decay,
               {Scan{a->state, state_out, room.states, 0}, Scan{}}, 1};
    return c.dp == 64 ? run_scan<64>(w, st) : run_scan<128>(w, st);
  }
  return GS_ATTN_CALL(forward, a, c, s, state_out, room, st);
}

extern "C" gs_status gs_linear_attn_bwd(const gs_linear_attn* a, const gs_attn_heads* q, const gs_attn_heads* k,
                                        const gs_attn_heads* v, const gs_attn_heads* dout,
                                        const gs_attn_heads* dq, const gs_attn_heads* dk, const gs_attn_heads* dv,
                                        const float* dstate_out, float* dstate, void* workspace, size_t ws_bytes,
                                        void* stream) {
  if (!a || !shape_ok(a) || !aligned_or_none(a) || (!a->group_offsets && a->groups != 1)) return GS_ERR_INVALID_ARG;
  const Call c(a, true);
  const Room room(workspace, c.slots, a->q_heads, a->k_heads, c.dp, a->tokens, true);
  Side s[7];
  if (!workspace || !aligned16(workspace) || ws_bytes < room.bytes) return GS_ERR_INVALID_ARG;
  if (a->tokens > 0 &&
      (!side(&s[0], a, q, a->dim, false, false) || !side(&s[1], a, k, a->dim, true, false) ||
       !side(&s[2], a, v, a->vdim, true, false) || !side(&s[3], a, dout, a->vdim, false, false) ||
       !side(&s[4], a, dq, a->dim, false, true) || !side(&s[5], a, dk, a->dim, true, true) ||
       !side(&s[6], a, dv, a->vdim, true, true)))
    return GS_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  if (a->tokens == 0 && !dstate) return GS_OK;
  if (a->tokens == 0) {
    ScanArgs w{c.split, a->q_heads, a->dim, a->vdim, a->log_decay,
               {Scan{dstate_out, dstate, room.grads, 1}, Scan{}}, 1};
    return c.dp == 64 ? run_scan<64>(w, st) : run_scan<128>(w, st);
  }
  return GS_ATTN_CALL(backward, a, c, s, dstate_out, dstate, room, st);
}

extern "C" gs_status gs_linear_attn_step(const gs_linear_attn* a, const gs_attn_heads* q, const gs_attn_heads* k,
                                         const gs_attn_heads* v, const gs_attn_heads* out, float* state,
                                         void* stream) {
  if (!a || !shape_ok(a) || !aligned_or_none(a)) return GS_ERR_INVALID_ARG;
  if (a->tokens == 0) return GS_OK;
  StepArgs p{};
  if (!state || !aligned_to(state, 4) || !side(&p.q, a, q, a->dim, false, false) ||
      !side(&p.k, a, k, a->dim, true, false) || !side(&p.v, a, v, a->vdim, true, false) ||
      !side(&p.out, a, out, a->vdim, false, true))
    return GS_ERR_INVALID_ARG;
  p.heads = a->q_heads;
  p.rep = a->q_heads / a->k_heads;
  p.log_decay = a->log_decay;
  p.scale = a->scale;
  p.state = state;
  cudaStream_t st = (cudaStream_t)stream;
  const dim3 grid((unsigned)a->tokens, a->q_heads);
  const bool vec = a->vdim % 4 == 0 && aligned16(state);
  if (a->dtype == GS_BF16)
    GS_CUDA(vec ? launch_overlapped(attn_step_kernel<__nv_bfloat16, 4>, grid, dim3(128), 0, st, p)
                : launch_overlapped(attn_step_kernel<__nv_bfloat16, 1>, grid, dim3(128), 0, st, p));
  else
    GS_CUDA(vec ? launch_overlapped(attn_step_kernel<__half, 4>, grid, dim3(128), 0, st, p)
                : launch_overlapped(attn_step_kernel<__half, 1>, grid, dim3(128), 0, st, p));
  return GS_OK;
}
