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
constexpr int kV = 64;  // values' channels of a block: wider heads take two blocks
// The keys' channels, padded to KD = 64 or 128, set the warps: each has 16 rows of the state.
template <int KD>
constexpr int kWarps = KD / 16;
template <int KD>
constexpr int kThreads = 32 * kWarps<KD>;

struct Side {  // heads that are read or written
  void* p;
  int64_t token, head;  // strides, elements
  int32_t dim;
  int32_t of_key;       // one head for rep query heads
  int32_t wide;         // whole granules of 16 bytes, on such boundaries
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
// Tiles in shared memory: rows of W 16-bit elements, whose 16-byte granules are swizzled by
// the row's last three bits: granule i of row r is at place i ^ (r % 8).  Tiles begin on
// 256-byte boundaries, so that 16 elements on are an exclusive or with 32.
//
// The lane's row address for the four 8 x 8 matrices of a 16 x 16 block at column 0 of the
// rows from r0 on (a multiple of 8): rows first (r0, r0 + 8 at column 0, then at 8) ...
template <int W>
__device__ __forceinline__ uint32_t rows_first(uint32_t tile, int r0, int lane) {
  return tile + (r0 + (lane & 15)) * (W * 2) + (((lane >> 4) ^ (lane & 7)) << 4);
}
// ... or columns first.
template <int W>
__device__ __forceinline__ uint32_t cols_first(uint32_t tile, int r0, int lane) {
  return tile + (r0 + (lane & 7) + (lane >> 4) * 8) * (W * 2) + (((lane >> 3 & 1) ^ (lane & 7)) << 4);
}

// A chunk's tile.  A chunk of n < kL tokens has them in its last n rows and zeros before
// them, so that a row's distance to the chunk's end is the same in every chunk.  Columns
// from dim on (a multiple of 8) are zeros.
template <typename T, int W, int THREADS>
__device__ __forceinline__ void load_tile(T* tile, const T* from, int64_t stride, int n, int dim) {
  constexpr int kG = W / 8, kRows = THREADS / kG;
  const int r0 = threadIdx.x / kG, c = threadIdx.x % kG, pad = kL - n;
  uint32_t to = smem_at(tile) + r0 * (W * 2) + ((c ^ (r0 & 7)) << 4);
  const T* p = from + (r0 - pad) * stride + c * 8;
  const bool in = c * 8 < dim;
#pragma unroll
  for (int i = 0; i < kL / kRows; ++i) {
    const bool there = in && r0 + i * kRows >= pad;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + i * kRows * W * 2),
                 "l"(there ? p : from), "r"(there ? 16 : 0)
                 : "memory");
    p += kRows * stride;
  }
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// log2 of a head's decay; one that leaves nothing after a token counts as 2^-1000.
__device__ __forceinline__ float log2_decay(const float* log_decay, int h) {
  const float a = log_decay[h] * 1.4426950408889634f;
  return a < -1000.f ? -1000.f : a;
}

template <typename T>
__device__ __forceinline__ float2 unpack(uint32_t w) {
  const Pack<T, 2> e = *reinterpret_cast<const Pack<T, 2>*>(&w);
  return make_float2(to_f32(e.v[0]), to_f32(e.v[1]));
}

// What a thread needs of a decay's powers: the weights of the keys in a chunk's last 16
// rows (tokens 2t, 2t + 1, 2t + 8, 2t + 9), mul d^(15 - token + shift).
struct Weights {
  float w[4];
  float top;  // the largest
  __device__ __forceinline__ Weights(float a, int t, int shift, float mul) : top(mul * power2(a * (float)shift)) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = mul * power2(a * (float)(15 - 2 * t - (j & 1) - (j >> 1) * 8 + shift));
  }
};

// 16 rows of the state past a chunk: st <- decay st + sum_j weight_j key_j value_j^T, the
// weighted keys as TERMS terms.  keys: columns first at the warp's 16 of the keys' channels;
// values: rows first.  In fp16 keys and state take a power of two meanwhile, so that the
// largest key with the largest weight is near 2^13: the terms of small ones would be below
// fp16's range.
template <typename T, int KD, int TERMS>
__device__ __forceinline__ void add_tokens(float (&st)[kV / 8][4], float decay, uint32_t keys, uint32_t values,
                                           const Weights& weights, float d16) {
  float w[4] = {weights.w[0], weights.w[1], weights.w[2], weights.w[3]};
  float back = 1.f;
  if constexpr (std::is_same<T, __half>::value) {
    uint32_t top = 0;  // magnitudes compare as whole numbers
#pragma unroll
    for (int ks = 0; ks < kL / 16; ++ks) {
      uint32_t raw[4];
      ldm4t(raw, keys + ks * 16 * KD * 2);
#pragma unroll
      for (int r = 0; r < 4; ++r) top = max(top, max(raw[r] & 0x7fffu, raw[r] >> 16 & 0x7fffu));
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float m = __half2float(__ushort_as_half((unsigned short)top)) * fabsf(weights.top);
    const int e = m > 0.f ? min(max((int)(__float_as_uint(m) >> 23) - 127 - 13, -100), 100) : 0;
    back = __uint_as_float((uint32_t)(127 + e) << 23);
    const float fit = __uint_as_float((uint32_t)(127 - e) << 23);
    decay *= fit;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] *= fit;
  }
#pragma unroll
  for (int i = 0; i < kV / 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) st[i][j] *= decay;
#pragma unroll
  for (int ks = kL / 16 - 1; ks >= 0; --ks) {
    uint32_t raw[4];
    // (row g, tokens 2t..), (g + 8, 2t..), (g, 2t + 8..), (g + 8, 2t + 8..)
    ldm4t(raw, keys + ks * 16 * KD * 2);
    uint32_t term[TERMS][4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float2 x = mul2(unpack<T>(raw[r]), r < 2 ? make_float2(w[0], w[1]) : make_float2(w[2], w[3]));
#pragma unroll
      for (int i = 0; i < TERMS; ++i) {
        term[i][r] = pair_word<T>(x.x, x.y);
        if (i + 1 < TERMS) x = fma2(unpack<T>(term[i][r]), both(-1.f), x);
      }
    }
#pragma unroll
    for (int c = 0; c < kV; c += 16) {
      uint32_t b[4];
      ldm4t(b, (values ^ (c * 2)) + ks * 16 * kV * 2);
#pragma unroll
      for (int i = 0; i < TERMS; ++i) {
        mma16<T>(st[c / 8], term[i], b[0], b[1]);
        mma16<T>(st[c / 8 + 1], term[i], b[2], b[3]);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] *= d16;
  }
  if constexpr (std::is_same<T, __half>::value) {
#pragma unroll
    for (int i = 0; i < kV / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) st[i][j] *= back;
  }
}

// Powers between rows g, g + 8 and columns 2t, 2t + 1 of a 16 x 16 block, times mul.
struct Powers {
  float b0, b1;  // d^(g - 2t + 8), d^(g - 2t + 7)
  float d0, d1;  // d^(g - 2t), d^(g - 2t - 1) on the diagonal
  float d8, d16;
  bool in0, in1;
  __device__ __forceinline__ Powers(float a, int g, int t, float mul) {
    b0 = mul * power2(a * (float)(g - 2 * t + 8));
    b1 = mul * power2(a * (float)(g - 2 * t + 7));
    in0 = g >= 2 * t;
    in1 = g >= 2 * t + 1;
    d0 = mul * power2(a * (float)max(g - 2 * t, 0));
    d1 = mul * power2(a * (float)max(g - 2 * t - 1, 0));
    d8 = power2(a * 8.f);
    d16 = power2(a * 16.f);
  }
};

// o += (queries times keys, decayed, up to the diagonal) times values, for the 16 rows rt.
// keys: columns first; values: rows first, at the warp's columns.
template <typename T, int KD, int WIDTH>
__device__ __forceinline__ void add_inner(float (&o)[WIDTH / 8][4], const uint32_t (&qf)[KD / 16][4], uint32_t keys,
                                          uint32_t values, int rt, const Powers& p) {
  float far = 1.f;  // d^(16 (rt - jb - 1))
#pragma unroll 1
  for (int jb = rt; jb >= 0; --jb) {
    float w[2][4] = {};
    const uint32_t k = keys + jb * (16 * KD * 2), v = values + jb * (16 * kV * 2);
#pragma unroll
    for (int i = 0; i < KD / 16; ++i) {
      uint32_t b[4];
      ldm4(b, k ^ (i * 32));
      mma16<T>(w[0], qf[i], b[0], b[1]);
      mma16<T>(w[1], qf[i], b[2], b[3]);
    }
    uint32_t pf[4];
    if (jb == rt) {
      pf[0] = pair_word<T>(p.in0 ? w[0][0] * p.d0 : 0.f, p.in1 ? w[0][1] * p.d1 : 0.f);
      pf[1] = pair_word<T>(w[0][2] * p.b0, w[0][3] * p.b1);
      pf[2] = 0;
      pf[3] = pair_word<T>(p.in0 ? w[1][2] * p.d0 : 0.f, p.in1 ? w[1][3] * p.d1 : 0.f);
    } else {
      const float c0 = p.b0 * far, c1 = p.b1 * far, e0 = c0 * p.d8, e1 = c1 * p.d8;
      pf[0] = pair_word<T>(w[0][0] * e0, w[0][1] * e1);
      pf[1] = pair_word<T>(w[0][2] * (e0 * p.d8), w[0][3] * (e1 * p.d8));
      pf[2] = pair_word<T>(w[1][0] * c0, w[1][1] * c1);
      pf[3] = pair_word<T>(w[1][2] * e0, w[1][3] * e1);
      far *= p.d16;
    }
#pragma unroll
    for (int x = 0; x < WIDTH; x += 16) {
      uint32_t b[4];
      ldm4t(b, v ^ (x * 2));
      mma16<T>(o[x / 8], pf, b[0], b[1]);
      mma16<T>(o[x / 8 + 1], pf, b[2], b[3]);
    }
  }
}

// The state as the products take it.  rescale: a power of two.
template <typename T>
__device__ __forceinline__ void put_state(uint32_t tile, const float (&st)[kV / 8][4], int warp, int g, int t,
                                          float rescale) {
  const uint32_t row = tile + (warp * 16 + g) * (kV * 2) + t * 4;
#pragma unroll
  for (int i = 0; i < kV / 8; ++i) {
    const uint32_t to = row + ((i ^ g) << 4);
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(pair_word<T>(st[i][0] * rescale, st[i][1] * rescale)) : "memory");
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + 8 * kV * 2),
                 "r"(pair_word<T>(st[i][2] * rescale, st[i][3] * rescale))
                 : "memory");
  }
}
// fp16: the power of two that brings the block's largest entry of the state near 2^13, as
// an exponent.  top: room for a number a warp, which nobody uses until the next barrier.
__device__ __forceinline__ int state_exponent(const float (&st)[kV / 8][4], float* top, int warps, int warp, int lane) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < kV / 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) m = fmaxf(m, fabsf(st[i][j]));
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) top[warp] = m;
  __syncthreads();
  for (int i = 0; i < warps; ++i) m = fmaxf(m, top[i]);
  return min(max((int)(__float_as_uint(m) >> 23) - 127 - 13, -100), 100);
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// 16 rows of the state from memory: entry (row, col) at src[row * rs + col * cs].
__device__ __forceinline__ void get_state(float (&st)[kV / 8][4], const float* src, int64_t rs, int64_t cs, int row0,
                                          int col0, int rows, int cols, int g, int t) {
#pragma unroll
  for (int i = 0; i < kV / 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = row0 + g + (j >> 1) * 8, col = col0 + i * 8 + 2 * t + (j & 1);
      st[i][j] = src && row < rows && col < cols ? src[row * rs + col * cs] : 0.f;
    }
}

// The warp's 16 rows of outputs through its own rows of a tile (of W columns, whose
// contents it alone uses and needs no more) to memory; the rows from `pad` on are there.
template <typename T, int W, int WIDTH>
__device__ __forceinline__ void put_rows(uint32_t tile, const float (&o)[WIDTH / 8][4], int rt, int col0, T* to,
                                         int64_t stride, int pad, int dim, bool wide, int lane) {
  const int g = lane >> 2, t = lane & 3;
  const uint32_t row = tile + (rt * 16 + g) * (W * 2) + t * 4;
  __syncwarp();
#pragma unroll
  for (int i = 0; i < WIDTH / 8; ++i) {
    const uint32_t at = row + (((col0 / 8 + i) ^ g) << 4);
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(pair_word<T>(o[i][0], o[i][1])) : "memory");
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 8 * W * 2), "r"(pair_word<T>(o[i][2], o[i][3])) : "memory");
  }
  __syncwarp();
  constexpr int kG = WIDTH / 8, kRows = 32 / kG;
  const int r0 = rt * 16 + lane / kG, c = col0 / 8 + lane % kG;
#pragma unroll
  for (int i = 0; i < 16 / kRows; ++i) {
    const int r = r0 + i * kRows;
    if (r < pad || c * 8 >= dim) continue;
    uint32_t w[4];
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(tile + r * (W * 2) + ((c ^ (r & 7)) << 4))
                 : "memory");
    T* x = to + (r - pad) * stride + c * 8;
    if (wide) {
      *reinterpret_cast<uint4*>(x) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c * 8 + j < dim) reinterpret_cast<uint16_t*>(x)[j] = (uint16_t)(w[j / 2] >> (j % 2 * 16));
    }
  }
}
// fp32 sums over a key head's query heads, one head after the other: o += what the heads
// before left, and unless this is the last one, o stays there.
template <int WIDTH>
__device__ __forceinline__ void sum_heads(float (&o)[WIDTH / 8][4], float* to, int64_t stride, int rt, int pad, int g,
                                          int t, bool first, bool last) {
#pragma unroll
  for (int i = 0; i < WIDTH / 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const int r = rt * 16 + g + (j >> 1) * 8;
      if (r < pad) continue;
      float2* x = reinterpret_cast<float2*>(to + (r - pad) * stride + i * 8 + 2 * t);
      if (!first) {
        const float2 y = *x;
        o[i][j] += y.x, o[i][j + 1] += y.y;
      }
      if (!last) *x = make_float2(o[i][j], o[i][j + 1]);
    }
}

template <typename T>
__device__ __forceinline__ T* head_at(const Side& s, int h, int rep, int64_t token) {
  return (T*)s.p + (int64_t)(s.of_key ? h / rep : h) * s.head + token * s.token;
}

// ---- each segment's part of the state ---------------------------------------
struct Part {
  Side key, value;
  float mul;
  int32_t back, shift;  // tokens from the last to the first
  int32_t exact;        // its last states are handed on
  float* to;            // [slots][heads][Dp][Ep]
};
struct PartsArgs {
  Split split;
  int32_t heads, rep;
  int32_t Dp, Ep;  // channels, rounded up to 64
  const float* log_decay;
  Part part[2];
};

template <typename T, int KD>
__global__ void __launch_bounds__(kThreads<KD>, 256 / KD) attn_parts_kernel(const __grid_constant__ PartsArgs p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  launch_dependents();
  wait_for_previous();
  constexpr int kSet = kL * (KD + kV);  // keys, values
  T* tiles = (T*)smem;
  const int h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blocks = p.Ep / kV, e0 = blockIdx.z % blocks * kV;
  const Part& part = p.part[blockIdx.z / blocks];
  const Span s = span_of(p.split, blockIdx.x);
  if (s.n == 0) return;
  const float a = log2_decay(p.log_decay, h);
  const int64_t from = part.back ? s.start + s.n - 1 : s.start;
  const int64_t step = part.back ? -1 : 1;
  const T* k = head_at<T>(part.key, h, p.rep, from);
  const T* v = head_at<T>(part.value, h, p.rep, from) + e0;
  auto load = [&](int c) {
    T* to = tiles + (c & 1) * kSet;
    const int n = min(kL, s.n - c * kL);
    const int64_t at = step * c * kL;
    load_tile<T, KD, kThreads<KD>>(to, k + at * part.key.token, step * part.key.token, n, part.key.dim);
    load_tile<T, kV, kThreads<KD>>(to + kL * KD, v + at * part.value.token, step * part.value.token, n,
                                   part.value.dim - e0);
    copies_commit();
  };
  float st[kV / 8][4] = {};
  const int chunks = (s.n + kL - 1) / kL;
  const Weights weights(a, lane & 3, part.shift, part.mul);
  const float d16 = power2(a * 16.f);
  const uint32_t keys = cols_first<KD>(smem_at(tiles), 0, lane) ^ (warp * 32);
  const uint32_t values = rows_first<kV>(smem_at(tiles) + kL * KD * 2, 0, lane);
  load(0);
  for (int c = 0; c < chunks; ++c) {
    copies_wait<0>();
    __syncthreads();
    if (c + 1 < chunks) load(c + 1);
    const uint32_t set = (c & 1) * kSet * 2;
    const float decay = power2(a * (float)min(kL, s.n - c * kL));
    if (std::is_same<T, __half>::value || !part.exact)
      add_tokens<T, KD, 2>(st, decay, keys + set, values + set, weights, d16);
    else
      add_tokens<T, KD, 3>(st, decay, keys + set, values + set, weights, d16);
  }
  float* to = part.to + (((int64_t)blockIdx.x * p.heads + h) * p.Dp + warp * 16 + (lane >> 2)) * p.Ep + e0 + (lane & 3) * 2;
#pragma unroll
  for (int i = 0; i < kV / 8; ++i) {
    *reinterpret_cast<float2*>(to + i * 8) = make_float2(st[i][0], st[i][1]);
    *reinterpret_cast<float2*>(to + 8 * p.Ep + i * 8) = make_float2(st[i][2], st[i][3]);
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
  int32_t heads, D, E, Dp, Ep;
  const float* log_decay;
  Scan scan[2];
  int32_t scans;
};

// One element of the state a thread, so that there are enough of them to hide the latency
// of the parts' loads (kAhead of them under way).
constexpr int kScanThreads = 256;
template <int AHEAD>
__global__ void __launch_bounds__(kScanThreads) attn_scan_kernel(const __grid_constant__ ScanArgs p) {
  launch_dependents();
  wait_for_previous();
  const Scan& k = p.scan[blockIdx.z];
  const int per = (p.D * p.E + kScanThreads - 1) / kScanThreads, size = p.Dp * p.Ep;
  const int h = blockIdx.y, g = blockIdx.x / per, i = blockIdx.x % per * kScanThreads + threadIdx.x;
  if (i >= p.D * p.E) return;
  const int row = i / p.E, col = i % p.E;
  const float a = log2_decay(p.log_decay, h);
  const int64_t begin = offset_of(p.split, g), end = offset_of(p.split, g + 1);
  const int64_t first = begin / p.split.seg + g;
  const int slots = end > begin ? (int)((end - begin + p.split.seg - 1) / p.split.seg) : 0;
  const int tail = (int)(end - begin - (int64_t)(slots - 1) * p.split.seg);
  const int64_t mat = ((int64_t)g * p.heads + h) * p.D * p.E + i;
  float s = k.edge ? k.edge[mat] : 0.f;
  const float full = power2(a * (float)p.split.seg), rest = power2(a * (float)tail);
  const int last = slots - 1;
  const int64_t stride = (k.back ? -1 : 1) * (int64_t)p.heads * size;
  float* at = k.parts + ((first + (k.back ? last : 0)) * p.heads + h) * size + row * p.Ep + col;
  for (int b = 0; b < slots; b += AHEAD) {
    float u[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
      if (b + j < slots) u[j] = at[stride * (b + j)];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      if (b + j >= slots) break;
      at[stride * (b + j)] = s;
      s = s * ((k.back ? b + j == 0 : b + j == last) ? rest : full) + u[j];
    }
  }
  if (k.last) k.last[mat] = s;
}

// ---- outputs -----------------------------------------------------------------
struct OutArgs {
  Split split;
  int32_t heads, rep;    // query heads
  int32_t shared;        // outputs are summed over the rep query heads of a key head
  Side query, key, value, out;
  const float* log_decay;
  int32_t K, V, Kp, Vp;  // keys' and values' channels, and rounded up to 64 or 128
  const float* states;   // [slots][heads][Kp][Vp], NULL: no group has more than one segment
  const float* edge;     // [groups][heads][..] or NULL (zeros)
  int32_t transposed;    // states are stored [values' channels][keys' channels] (and [Vp][Kp])
  int32_t back, shift;
  float mul_inner, mul_state, mul_key;
  float* sums;           // [tokens][key heads][Vp], where shared and rep > 1
};

// Where a state is read from: a segment's, or without those the group's own.
struct Stored {
  const float* p;
  int64_t rs, cs;  // between rows and columns as they are used
};
__device__ __forceinline__ Stored stored(const float* states, const float* edge, int Kp, int Vp, int kdim, int vdim,
                                         int transposed, int64_t slot, int64_t group) {
  const float* p = states ? states + slot * Kp * Vp : edge ? edge + group * kdim * vdim : nullptr;
  const int ks = states ? Kp : kdim, vs = states ? Vp : vdim;
  return transposed ? Stored{p, 1, ks} : Stored{p, vs, 1};
}

template <typename T, int KD>
__global__ void __launch_bounds__(kThreads<KD>, 256 / KD) attn_out_kernel(const __grid_constant__ OutArgs p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  launch_dependents();
  wait_for_previous();
  constexpr int kKeys = kL * KD, kValues = kL * kV, kSet = 2 * kKeys + kValues;
  constexpr int kSplits = kWarps<KD> / kTilesOfRows;  // of the values' channels over warps
  constexpr int kWidth = kV / kSplits;
  T* tiles = (T*)smem;                          // [2] queries, keys, values
  const uint32_t state = smem_at(tiles + 2 * kSet);  // [KD][kV]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rt = warp % kTilesOfRows, col0 = warp / kTilesOfRows * kWidth;
  const Span s = span_of(p.split, blockIdx.x);
  if (s.n == 0) return;
  const int64_t from = p.back ? s.start + s.n - 1 : s.start, step = p.back ? -1 : 1;
  const int chunks = (s.n + kL - 1) / kL, e0 = blockIdx.z * kV;
  const int reps = p.shared ? p.rep : 1;
  const uint32_t queries = rows_first<KD>(smem_at(tiles), rt * 16, lane);
  const uint32_t keys = cols_first<KD>(smem_at(tiles) + kKeys * 2, 0, lane);
  const uint32_t values = rows_first<kV>(smem_at(tiles) + 4 * kKeys, 0, lane);
  const uint32_t state_rows = rows_first<kV>(state, 0, lane) ^ (col0 * 2);

  for (int r = 0; r < reps; ++r) {
    const int h = p.shared ? blockIdx.y * p.rep + r : blockIdx.y;
    const float a = log2_decay(p.log_decay, h);
    const T* q = head_at<T>(p.query, h, p.rep, from);
    const T* k = head_at<T>(p.key, h, p.rep, from);
    const T* v = head_at<T>(p.value, h, p.rep, from) + e0;
    auto load = [&](int c) {
      T* to = tiles + (c & 1) * kSet;
      const int n = min(kL, s.n - c * kL);
      const int64_t at = step * c * kL;
      load_tile<T, KD, kThreads<KD>>(to, q + at * p.query.token, step * p.query.token, n, p.query.dim);
      load_tile<T, KD, kThreads<KD>>(to + kKeys, k + at * p.key.token, step * p.key.token, n, p.key.dim);
      load_tile<T, kV, kThreads<KD>>(to + 2 * kKeys, v + at * p.value.token, step * p.value.token, n, p.value.dim - e0);
      copies_commit();
    };
    __syncthreads();
    load(0);
    float st[kV / 8][4];  // 16 rows (keys' channels) a warp
    const Stored from_memory = stored(p.states, p.edge, p.Kp, p.Vp, p.K, p.V, p.transposed,
                                      ((int64_t)blockIdx.x * p.heads + h), ((int64_t)s.group * p.heads + h));
    get_state(st, from_memory.p, from_memory.rs, from_memory.cs, warp * 16, e0, p.K, p.V, g, t);
    const Powers powers(a, g, t, p.mul_inner);
    const Weights weights(a, t, p.shift, p.mul_key);

    for (int c = 0; c < chunks; ++c) {
      const int n = min(kL, s.n - c * kL), pad = kL - n;
      const uint32_t set = (c & 1) * kSet * 2;
      float unscale = 1.f, rescale = 1.f;
      if constexpr (std::is_same<T, __half>::value) {
        // (in the other set's values, which are read no more and not yet on their way)
        const int e = state_exponent(st, reinterpret_cast<float*>(tiles + ((c + 1) & 1) * kSet + 2 * kKeys), kWarps<KD>,
                                     warp, lane);
        rescale = power_of_two(-e);
        unscale = power_of_two(e);
      }
      put_state<T>(state, st, warp, g, t, rescale);
      copies_wait<0>();
      __syncthreads();
      if (c + 1 < chunks) load(c + 1);

      // queries times the state
      uint32_t qf[KD / 16][4];
#pragma unroll
      for (int i = 0; i < KD / 16; ++i) ldm4(qf[i], (queries + set) ^ (i * 32));
      float o[kWidth / 8][4] = {};
#pragma unroll
      for (int i = 0; i < KD / 16; ++i)
#pragma unroll
        for (int x = 0; x < kWidth; x += 16) {
          uint32_t b[4];
          ldm4t(b, (state_rows ^ (x * 2)) + i * 16 * kV * 2);
          mma16<T>(o[x / 8], qf[i], b[0], b[1]);
          mma16<T>(o[x / 8 + 1], qf[i], b[2], b[3]);
        }
      // (rows before the chunk's first token are not there)
      const float f0 = p.mul_state * unscale * power2(a * (float)max(rt * 16 + g + 1 - p.shift - pad, 0));
      const float f1 = p.mul_state * unscale * power2(a * (float)max(rt * 16 + g + 9 - p.shift - pad, 0));
#pragma unroll
      for (int i = 0; i < kWidth / 8; ++i) o[i][0] *= f0, o[i][1] *= f0, o[i][2] *= f1, o[i][3] *= f1;
      add_inner<T, KD, kWidth>(o, qf, keys + set, (values + set) ^ (col0 * 2), rt, powers);

      if (c + 1 < chunks)
        add_tokens<T, KD, 2>(st, power2(a * (float)n), (keys + set) ^ (warp * 32), values + set, weights, powers.d16);
      const int64_t tok = from + step * c * kL;
      if (reps > 1)
        sum_heads<kWidth>(o, p.sums + (tok * (p.heads / p.rep) + blockIdx.y) * p.Vp + e0 + col0,
                          step * (p.heads / p.rep) * p.Vp, rt, pad, g, t, r == 0, r + 1 == reps);
      __syncthreads();  // the state, the queries and the keys have been read
      if (r + 1 == reps)
        put_rows<T, KD, kWidth>(smem_at(tiles) + set, o, rt, col0,
                                (T*)p.out.p + (int64_t)blockIdx.y * p.out.head + tok * p.out.token + e0,
                                step * p.out.token, pad, p.out.dim - e0, p.out.wide, lane);
    }
  }
}

// ---- the gradients of keys and values together -----------------------------------
// Heads of up to 64 channels: both go through the tokens backwards with the same state R
// [dim][vdim] (the gradient of the state), which is read as it lies for dv and transposed
// for dk, and updated once.  queries, keys, values, douts as in the call.
struct KvArgs {
  Split split;
  int32_t heads, rep;
  Side q, k, v, g, dk, dv;
  int32_t D, E;
  const float* log_decay;
  const float* states;  // [slots][heads][64][64], NULL: no group has more than one segment
  const float* edge;    // [groups][heads][dim][vdim] or NULL (zeros)
  float scale;
  float* sums[2];       // [tokens][key heads][64], where rep > 1: of dk, of dv
};

template <typename T>
__global__ void __launch_bounds__(kThreads<64>, 4) attn_kv_kernel(const __grid_constant__ KvArgs p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  launch_dependents();
  wait_for_previous();
  constexpr int kTile = kL * 64, kB = kTile * 2;  // keys, values, queries, douts
  T* tiles = (T*)smem;
  const uint32_t state = smem_at(tiles + 4 * kTile);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, rt = warp;
  const Span s = span_of(p.split, blockIdx.x);
  if (s.n == 0) return;
  const int64_t from = s.start + s.n - 1;
  const int chunks = (s.n + kL - 1) / kL, key_heads = p.heads / p.rep;
  const uint32_t rows = rows_first<64>(smem_at(tiles), 0, lane), cols = cols_first<64>(smem_at(tiles), 0, lane);
  const uint32_t own = rt * 16 * 128;
  const uint32_t state_rows = rows_first<64>(state, 0, lane), state_cols = cols_first<64>(state, 0, lane);

  for (int r = 0; r < p.rep; ++r) {
    const int h = blockIdx.y * p.rep + r;
    const float a = log2_decay(p.log_decay, h);
    auto load = [&](int c) {
      T* to = tiles;
      const int n = min(kL, s.n - c * kL);
      const int64_t at = from - (int64_t)c * kL;
      load_tile<T, 64, kThreads<64>>(to, head_at<T>(p.k, h, p.rep, at), -p.k.token, n, p.k.dim);
      load_tile<T, 64, kThreads<64>>(to + kTile, head_at<T>(p.v, h, p.rep, at), -p.v.token, n, p.v.dim);
      load_tile<T, 64, kThreads<64>>(to + 2 * kTile, head_at<T>(p.q, h, p.rep, at), -p.q.token, n, p.q.dim);
      load_tile<T, 64, kThreads<64>>(to + 3 * kTile, head_at<T>(p.g, h, p.rep, at), -p.g.token, n, p.g.dim);
      copies_commit();
    };
    __syncthreads();
    load(0);
    float st[kV / 8][4];
    const Stored from_memory = stored(p.states, p.edge, 64, 64, p.D, p.E, 0, ((int64_t)blockIdx.x * p.heads + h),
                                      ((int64_t)s.group * p.heads + h));
    get_state(st, from_memory.p, from_memory.rs, from_memory.cs, warp * 16, 0, p.D, p.E, g, t);
    const Powers powers(a, g, t, p.scale);
    const Weights weights(a, t, 1, p.scale);

    for (int c = 0; c < chunks; ++c) {
      const int n = min(kL, s.n - c * kL), pad = kL - n;
      float unscale = 1.f, rescale = 1.f;
      if constexpr (std::is_same<T, __half>::value) {
        const int e = state_exponent(st, reinterpret_cast<float*>(tiles + 5 * kTile), kWarps<64>,
                                     warp, lane);
        rescale = power_of_two(-e);
        unscale = power_of_two(e);
      }
      put_state<T>(state, st, warp, g, t, rescale);
      copies_wait<0>();
      __syncthreads();
      const float f0 = unscale * power2(a * (float)max(rt * 16 + g - pad, 0));
      const float f1 = unscale * power2(a * (float)max(rt * 16 + g + 8 - pad, 0));
      const int64_t tok = from - (int64_t)c * kL;
      const int64_t sum = (tok * key_heads + blockIdx.y) * 64, sum_step = -(int64_t)key_heads * 64;
      uint32_t f[4][4];
      {  // dv: keys times R, and keys times queries times douts
#pragma unroll
        for (int i = 0; i < 4; ++i) ldm4(f[i], (rows + own) ^ (i * 32));
        float o[8][4] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int x = 0; x < 64; x += 16) {
            uint32_t b[4];
            ldm4t(b, (state_rows ^ (x * 2)) + i * 16 * 128);
            mma16<T>(o[x / 8], f[i], b[0], b[1]);
            mma16<T>(o[x / 8 + 1], f[i], b[2], b[3]);
          }
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i][0] *= f0, o[i][1] *= f0, o[i][2] *= f1, o[i][3] *= f1;
        add_inner<T, 64, 64>(o, f, cols + 2 * kB, rows + 3 * kB, rt, powers);
        if (p.rep > 1) sum_heads<64>(o, p.sums[1] + sum, sum_step, rt, pad, g, t, r == 0, r + 1 == p.rep);
        if (r + 1 == p.rep)
          put_rows<T, 64, 64>(smem_at(tiles), o, rt, 0, head_at<T>(p.dv, h, p.rep, tok), -p.dv.token, pad,
                              p.dv.dim, p.dv.wide, lane);
      }
      {  // dk: values times R^T, and values times douts times queries
#pragma unroll
        for (int i = 0; i < 4; ++i) ldm4(f[i], (rows + kB + own) ^ (i * 32));
        float o[8][4] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int x = 0; x < 64; x += 16) {
            uint32_t b[4];
            ldm4(b, (state_cols ^ (i * 32)) + x * 128);
            mma16<T>(o[x / 8], f[i], b[0], b[1]);
            mma16<T>(o[x / 8 + 1], f[i], b[2], b[3]);
          }
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i][0] *= f0, o[i][1] *= f0, o[i][2] *= f1, o[i][3] *= f1;
        add_inner<T, 64, 64>(o, f, cols + 3 * kB, rows + 2 * kB, rt, powers);
        if (p.rep > 1) sum_heads<64>(o, p.sums[0] + sum, sum_step, rt, pad, g, t, r == 0, r + 1 == p.rep);
        if (r + 1 == p.rep)
          put_rows<T, 64, 64>(smem_at(tiles) + kB, o, rt, 0, head_at<T>(p.dk, h, p.rep, tok), -p.dk.token, pad,
                              p.dk.dim, p.dk.wide, lane);
      }
      if (c + 1 < chunks)
        add_tokens<T, 64, 2>(st, power2(a * (float)n), (cols + 2 * kB) ^ (warp * 32), rows + 3 * kB, weights,
                             powers.d16);
      __syncthreads();  // the state and the tiles have been read
      if (c + 1 < chunks) load(c + 1);
    }
  }
}

// ---- rows that start anywhere, copied to padded rows --------------------------------
struct RowsArgs {
  Side from[4];
  void* to[4];        // [tokens][heads][dim rounded up to 8]
  int32_t heads[4];
  int64_t tokens;
};
template <typename W>
__global__ void __launch_bounds__(256) attn_rows_kernel(const __grid_constant__ RowsArgs p) {
  launch_dependents();
  wait_for_previous();
  const Side& s = p.from[blockIdx.y];
  const int heads = p.heads[blockIdx.y], granules = (s.dim + 7) / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, r = i / granules, token = r / heads;
  const int c = (int)(i % granules) * 8, h = (int)(r % heads);
  if (token >= p.tokens) return;
  const W* from = (const W*)s.p + token * s.token + h * s.head + c;
  Pack<W, 8> v;
#pragma unroll
  for (int j = 0; j < 8; ++j) v.v[j] = c + j < s.dim ? from[j] : W(0);
  store_pack<W, 8>((W*)p.to[blockIdx.y] + (r * granules) * 8 + c, v);
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

int padded_dim(int32_t dim) { return dim <= 64 ? 64 : 128; }

// Tokens of a segment.  The kernels run in waves of as many blocks as the SMs hold (four
// of four warps each, two of eight), a wave takes as long as a segment, and each segment
// costs about two chunks more for its state.  Where a group is one segment its states need
// neither a sum nor a scan: those two kernels' start is worth about five chunks, and their
// work half of the outputs'.
int32_t segment_tokens(const gs_linear_attn* a, bool backward) {
  // (the groups' lengths are on the device: taken as equal)
  const int64_t chunks = div_up(div_up(a->tokens, a->groups), kL), resident = (int64_t)device_sms() * (256 / padded_dim(a->dim));
  const int64_t blocks = (int64_t)a->groups * a->q_heads * (padded_dim(a->vdim) / kV);
  const int least = backward ? 2 : 1, most = 32;
  int best = least;
  int64_t cost = INT64_MAX;
  for (int m = least; m <= most; ++m) {
    const int64_t waves = div_up(div_up(chunks, m) * blocks, resident);
    const int64_t c = chunks <= m ? 2 * waves * (chunks + 2) : 3 * waves * (m + 2) + 10;
    if (c < cost) cost = c, best = m;
  }
  return best * kL;
}

struct Room {
  float *states, *grads, *sums[2];
  void* rows[4];
  size_t bytes;
  // copied: the inputs (q, k, v, dout) whose rows have to be copied, a bit each
  Room(void* ws, const gs_linear_attn* a, int64_t slots, bool backward, int copied) {
    char* base = (char*)ws;
    size_t at = 0;
    auto take = [&](size_t n) {
      char* p = base + at;
      at += (n + 255) / 256 * 256;
      return (float*)p;
    };
    const size_t d = padded_dim(a->dim), e = padded_dim(a->vdim);
    const size_t one = sizeof(float) * slots * a->q_heads * d * e;
    const size_t sum = backward && a->q_heads > a->k_heads ? sizeof(float) * a->tokens * a->k_heads : 0;
    states = take(one);
    grads = take(backward ? one : 0);
    sums[0] = take(sum * d);
    sums[1] = take(sum * e);
    const size_t row[4] = {(size_t)a->q_heads * div_up(a->dim, 8), (size_t)a->k_heads * div_up(a->dim, 8),
                           (size_t)a->k_heads * div_up(a->vdim, 8), (size_t)a->q_heads * div_up(a->vdim, 8)};
    for (int i = 0; i < 4; ++i) rows[i] = take(copied >> i & 1 ? 16 * row[i] * a->tokens : 0);
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
            dim % 8 == 0 && aligned16(h->p) && (a->tokens < 2 || h->token % 8 == 0) && (heads < 2 || h->head % 8 == 0)
                ? 1 : 0};
  return true;
}

template <int KD>
constexpr int kPartsSmem = 2 * kL * (KD + kV) * 2;
template <int KD>
constexpr int kOutSmem = (2 * kL * (2 * KD + kV) + KD * kV) * 2;

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

// Inputs whose rows the kernels can't read as they lie.
int to_copy(const Side* s, int n) {
  int bits = 0;
  for (int i = 0; i < n; ++i) bits |= (s[i].wide ? 0 : 1) << i;
  return bits;
}
gs_status copy_rows(const gs_linear_attn* a, Side* s, int n, const Room& room, cudaStream_t st) {
  RowsArgs p{};
  p.tokens = a->tokens;
  int count = 0;
  int64_t most = 0;
  for (int i = 0; i < n; ++i) {
    if (s[i].wide) continue;
    const int32_t heads = s[i].of_key ? a->k_heads : a->q_heads;
    const int64_t granules = div_up(s[i].dim, 8);
    p.from[count] = s[i];
    p.to[count] = room.rows[i];
    p.heads[count++] = heads;
    if (a->tokens * heads * granules > most) most = a->tokens * heads * granules;
    s[i] = Side{room.rows[i], heads * granules * 8, granules * 8, (int32_t)granules * 8, s[i].of_key, 1};
  }
  if (!count) return GS_OK;
  const int64_t blocks = div_up(most, 256);
  if (blocks > INT32_MAX) return GS_ERR_INVALID_ARG;
  GS_CUDA(launch_overlapped(attn_rows_kernel<uint16_t>, dim3((unsigned)blocks, count), dim3(256), 0, st, p));
  return GS_OK;
}

template <typename T, int KD>
gs_status run_parts(const PartsArgs& p, int64_t slots, int parts, cudaStream_t st) {
  static std::atomic<uint64_t> known{0};
  if (!allow_smem(attn_parts_kernel<T, KD>, known, kPartsSmem<KD>)) {
    (void)cudaGetLastError();
    return GS_ERR_CUDA;
  }
  GS_CUDA(launch_overlapped(attn_parts_kernel<T, KD>, dim3((unsigned)slots, p.heads, parts * (p.Ep / kV)),
                            dim3(kThreads<KD>), kPartsSmem<KD>, st, p));
  return GS_OK;
}
gs_status run_scan(const ScanArgs& p, cudaStream_t st) {
  const int64_t blocks = p.split.groups * div_up(p.D * p.E, kScanThreads);
  if (blocks > INT32_MAX) return GS_ERR_INVALID_ARG;
  GS_CUDA(launch_overlapped(attn_scan_kernel<16>, dim3((unsigned)blocks, p.heads, p.scans), dim3(kScanThreads), 0, st,
                            p));
  return GS_OK;
}
template <typename T, int KD>
gs_status run_out_of(const OutArgs& p, int64_t slots, cudaStream_t st) {
  static std::atomic<uint64_t> known{0};
  if (!allow_smem(attn_out_kernel<T, KD>, known, kOutSmem<KD>)) {
    (void)cudaGetLastError();
    return GS_ERR_CUDA;
  }
  GS_CUDA(launch_overlapped(attn_out_kernel<T, KD>,
                            dim3((unsigned)slots, p.shared ? p.heads / p.rep : p.heads, p.Vp / kV),
                            dim3(kThreads<KD>), kOutSmem<KD>, st, p));
  return GS_OK;
}
constexpr int kKvSmem = 5 * kL * 64 * 2 + 64;  // four tiles, the state, a number a warp
template <typename T>
gs_status run_kv(const KvArgs& p, int64_t slots, cudaStream_t st) {
  static std::atomic<uint64_t> known{0};
  if (!allow_smem(attn_kv_kernel<T>, known, kKvSmem)) {
    (void)cudaGetLastError();
    return GS_ERR_CUDA;
  }
  GS_CUDA(launch_overlapped(attn_kv_kernel<T>, dim3((unsigned)slots, p.heads / p.rep), dim3(kThreads<64>), kKvSmem, st,
                            p));
  return GS_OK;
}
template <typename T>
gs_status run_out(const OutArgs& p, int64_t slots, cudaStream_t st) {
  return p.Kp == 64 ? run_out_of<T, 64>(p, slots, st) : run_out_of<T, 128>(p, slots, st);
}

struct Call {
  Split split;
  int64_t slots;
  int Dp, Ep, rep;
  Call(const gs_linear_attn* a, bool backward) {
    split = Split{a->tokens, a->group_offsets, a->groups, segment_tokens(a, backward)};
    slots = a->tokens / split.seg + a->groups;
    Dp = padded_dim(a->dim);
    Ep = padded_dim(a->vdim);
    rep = a->q_heads / a->k_heads;
  }
};

// The states at the segments' starts (and, with two parts, the gradients at their ends).
template <typename T>
gs_status states_of(const gs_linear_attn* a, const Call& c, const Part (&part)[2], const Scan (&scan)[2], int n,
                    cudaStream_t st) {
  const PartsArgs p{c.split, a->q_heads, c.rep, c.Dp, c.Ep, a->log_decay, {part[0], part[1]}};
  const gs_status r = c.Dp == 64 ? run_parts<T, 64>(p, c.slots, n, st) : run_parts<T, 128>(p, c.slots, n, st);
  if (r != GS_OK) return r;
  return run_scan(ScanArgs{c.split, a->q_heads, a->dim, a->vdim, c.Dp, c.Ep, a->log_decay, {scan[0], scan[1]}, n}, st);
}

template <typename T>
gs_status forward(const gs_linear_attn* a, const Call& c, Side (&s)[4], float* state_out, const Room& room,
                  cudaStream_t st) {
  const bool scan = a->tokens > c.split.seg || state_out;
  const gs_status copied = copy_rows(a, s, 3, room, st);
  if (copied != GS_OK) return copied;
  if (scan) {
    const gs_status r = states_of<T>(a, c, {Part{s[1], s[2], 1.f, 0, 0, state_out != nullptr, room.states}, Part{}},
                                     {Scan{a->state, state_out, room.states, 0}, Scan{}}, 1, st);
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
  o.K = a->dim, o.V = a->vdim, o.Kp = c.Dp, o.Vp = c.Ep;
  o.mul_inner = o.mul_state = a->scale;
  o.mul_key = 1.f;
  return run_out<T>(o, c.slots, st);
}

template <typename T>
gs_status backward(const gs_linear_attn* a, const Call& c, Side (&s)[7], const float* dstate_out,
                   float* dstate, const Room& room, cudaStream_t st) {
  const gs_status copied = copy_rows(a, s, 4, room, st);
  if (copied != GS_OK) return copied;
  const Side &q = s[0], &k = s[1], &v = s[2], &g = s[3];
  const bool scan = a->tokens > c.split.seg || dstate;
  if (scan) {
    const gs_status r =
        states_of<T>(a, c, {Part{k, v, 1.f, 0, 0, 0, room.states},
                          Part{q, g, a->scale, 1, 1, dstate != nullptr, room.grads}},
                     {Scan{a->state, nullptr, room.states, 0}, Scan{dstate_out, dstate, room.grads, 1}}, 2, st);
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
    x.K = a->vdim, x.V = a->dim, x.Kp = c.Ep, x.Vp = c.Dp;
    x.states = scan ? room.states : nullptr;
    x.edge = a->state;
    x.transposed = 1;
    x.mul_state = a->scale;
    x.mul_key = 1.f;
    const gs_status r = run_out<T>(x, c.slots, st);
    if (r != GS_OK) return r;
  }
  if (c.Dp == 64 && c.Ep == 64)
    return run_kv<T>(KvArgs{c.split, a->q_heads, c.rep, q, k, v, g, s[5], s[6], a->dim, a->vdim, a->log_decay,
                            scan ? room.grads : nullptr, dstate_out, a->scale, {room.sums[0], room.sums[1]}},
                     c.slots, st);
  o.back = o.shift = o.shared = 1;
  o.mul_state = 1.f;
  o.mul_key = a->scale;
  o.states = scan ? room.grads : nullptr;
  o.edge = dstate_out;
  {
    OutArgs x = o;  // dk
    x.query = v, x.key = g, x.value = q, x.out = s[5];
    x.K = a->vdim, x.V = a->dim, x.Kp = c.Ep, x.Vp = c.Dp;
    x.transposed = 1;
    x.sums = room.sums[0];
    const gs_status r = run_out<T>(x, c.slots, st);
    if (r != GS_OK) return r;
  }
  OutArgs x = o;  // dv
  x.query = k, x.key = q, x.value = g, x.out = s[6];
  x.K = a->dim, x.V = a->vdim, x.Kp = c.Dp, x.Vp = c.Ep;
  x.sums = room.sums[1];
  return run_out<T>(x, c.slots, st);
}

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" size_t gs_linear_attn_workspace_bytes(const gs_linear_attn* a, int32_t backward) {
  if (!a || !shape_ok(a)) return 0;
  const Call c(a, backward != 0);
  return Room(nullptr, a, c.slots, backward != 0, backward ? 15 : 7).bytes;
}

extern "C" gs_status gs_linear_attn_fwd(const gs_linear_attn* a, const gs_attn_heads* q, const gs_attn_heads* k,
                                        const gs_attn_heads* v, const gs_attn_heads* out, float* state_out,
                                        void* workspace, size_t ws_bytes, void* stream) {
  if (!a || !shape_ok(a) || !aligned_or_none(a) || (!a->group_offsets && a->groups != 1)) return GS_ERR_INVALID_ARG;
  const Call c(a, false);
  Side s[4] = {};
  if (a->tokens > 0 && (!side(&s[0], a, q, a->dim, false, false) || !side(&s[1], a, k, a->dim, true, false) ||
                        !side(&s[2], a, v, a->vdim, true, false) || !side(&s[3], a, out, a->vdim, false, true)))
    return GS_ERR_INVALID_ARG;
  const Room room(workspace, a, c.slots, false, a->tokens > 0 ? to_copy(s, 3) : 0);
  if (!workspace || !aligned16(workspace) || ws_bytes < room.bytes) return GS_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  if (a->tokens == 0 && !state_out) return GS_OK;
  if (a->tokens == 0) {
    return run_scan(ScanArgs{c.split, a->q_heads, a->dim, a->vdim, c.Dp, c.Ep, a->log_decay,
                             {Scan{a->state, state_out, room.states, 0}, Scan{}}, 1}, st);
  }
  return a->dtype == GS_BF16 ? forward<__nv_bfloat16>(a, c, s, state_out, room, st)
                             : forward<__half>(a, c, s, state_out, room, st);
}

extern "C" gs_status gs_linear_attn_bwd(const gs_linear_attn* a, const gs_attn_heads* q, const gs_attn_heads* k,
                                        const gs_attn_heads* v, const gs_attn_heads* dout,
                                        const gs_attn_heads* dq, const gs_attn_heads* dk, const gs_attn_heads* dv,
                                        const float* dstate_out, float* dstate, void* workspace, size_t ws_bytes,
                                        void* stream) {
  if (!a || !shape_ok(a) || !aligned_or_none(a) || (!a->group_offsets && a->groups != 1)) return GS_ERR_INVALID_ARG;
  const Call c(a, true);
  Side s[7] = {};
  if (a->tokens > 0 &&
      (!side(&s[0], a, q, a->dim, false, false) || !side(&s[1], a, k, a->dim, true, false) ||
       !side(&s[2], a, v, a->vdim, true, false) || !side(&s[3], a, dout, a->vdim, false, false) ||
       !side(&s[4], a, dq, a->dim, false, true) || !side(&s[5], a, dk, a->dim, true, true) ||
       !side(&s[6], a, dv, a->vdim, true, true)))
    return GS_ERR_INVALID_ARG;
  const Room room(workspace, a, c.slots, true, a->tokens > 0 ? to_copy(s, 4) : 0);
  if (!workspace || !aligned16(workspace) || ws_bytes < room.bytes) return GS_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  if (a->tokens == 0 && !dstate) return GS_OK;
  if (a->tokens == 0) {
    return run_scan(ScanArgs{c.split, a->q_heads, a->dim, a->vdim, c.Dp, c.Ep, a->log_decay,
                             {Scan{dstate_out, dstate, room.grads, 1}, Scan{}}, 1}, st);
  }
  return a->dtype == GS_BF16 ? backward<__nv_bfloat16>(a, c, s, dstate_out, dstate, room, st)
                             : backward<__half>(a, c, s, dstate_out, dstate, room, st);
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
