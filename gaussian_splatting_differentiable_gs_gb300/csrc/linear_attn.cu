// linear_attn.cu -- gs_linear_attn_fwd, _bwd, _step: linear attention with a decay for
// each head.
//
//   S_t = d S_{t-1} + k_t v_t^T,  o_t = scale q_t S_t,  d = e^log_decay
//
// In chunks of 128 tokens (n of them, i and j counted from a chunk's start, S its state
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
// state in registers (fp32) between a segment's chunks.  Where query heads share a key
// head, its gradients leave in fp32 for each of them and a fourth kernel sums these.
//
// Products are on the tensor cores (tcgen05, 128 rows), sums and states fp32.  What is
// rounded to the inputs' type on the way: the decayed products q_i k_j, and the state
// where it is multiplied by a query (not where it is kept); each of the two parts of an
// output is rounded once there and once more as the output.  In fp16 both, and the decayed
// keys, are brought into its range by a power of two for each chunk, from the largest finite
// state, query and key (32640 tokens, 16 heads of 64: with the products' range 103 us
// forward and 249 backward, with the other two alone 102 and 242; products past 65504 were
// infinities then, and those below 2^-14 had fewer bits).  The decayed keys of a
// state's sum are taken as 3 (bf16) or 2 (fp16) terms, exact to fp32's rounding, for the
// states that are handed on, and as 2 terms for the others.
#include <atomic>
#include <type_traits>

#include "activation.cuh"
#include "tensor_core.cuh"

namespace gs {
namespace {

constexpr int kL = 128;  // tokens of a chunk: the rows of a product
constexpr int kV = 64;   // values' channels of a block: wider heads take two blocks
constexpr int kThreads = 256;
constexpr int kBlock = kL * 128;  // bytes of 64 channels of a chunk
constexpr unsigned int kErrTimeout = 1u;
constexpr int64_t kWaitNs = 2000000000;
// What the products of a block are limited to: in the self-test fewer than it waits for.
struct Limits {
  uint32_t products;  // sets of products
  int64_t wait_ns;    // after a block's first wait, its last one gives up
};
// The keys' channels are padded to KD = 64 or 128.

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
  int64_t from, upto;      // only segments that start in these tokens
  Limits limits;
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
  return Span{lo, start, in < 0 || left <= 0 || start < s.from || start >= s.upto ? 0 : (int)(left < s.seg ? left : s.seg)};
}
// The first token of the segment that a token of the groups is in.
__device__ __forceinline__ int64_t segment_start(const Split& s, int64_t token) {
  int lo = 0, hi = s.groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (offset_of(s, mid) <= token) lo = mid;
    else hi = mid - 1;
  }
  const int64_t begin = offset_of(s, lo);
  return begin + (token - begin) / s.seg * s.seg;
}

// Set where a wait for the tensor core ran out (gs_linear_attn_status).
__device__ unsigned int attn_timeouts;

// ---- tcgen05 on one SM ------------------------------------------------------------
// Descriptors of operands in 128-byte swizzled rows (64 channels of a token, the granules
// of 16 bytes exchanged by the token's last three bits).  K-major: the channels are the
// sum's terms, 16 on are 32 bytes.  MN-major: the tokens are the sum's terms, 16 on are
// 2048 bytes; the next 64 channels follow a block later.
template <bool MN>
__device__ __forceinline__ uint64_t operand(uint32_t addr) {
  constexpr uint64_t kLead = MN ? (uint64_t)(kBlock >> 4) : 1, kAtom = (uint64_t)(1024 >> 4);
  return (uint64_t)((addr & 0x3ffff) >> 4) | (kLead << 16) | (kAtom << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
template <typename T>
__device__ __forceinline__ constexpr uint32_t instruction(int m, int n, bool a_mn, bool b_mn) {
  const uint32_t type = std::is_same<T, __half>::value ? 0u : 1u;
  return (1u << 4) | (type << 7) | (type << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
      "r"((uint32_t)add)
      : "memory");
}
// The first operand in TMEM: a row a lane, two terms a column.
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
      "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// What this thread wrote to shared memory is there for the tensor core (after a barrier).
__device__ __forceinline__ void publish() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

struct Control {
  uint64_t done[3];
  uint32_t issued[3];         // 1 + the phase that the last products issued end, or 0
  uint32_t tmem;
  volatile int64_t until;     // when waiting ends; 0: nothing has been waited for
  volatile uint32_t abort;    // a wait gave up
  alignas(16) uint32_t top[4][kThreads / 32];  // the warps' largest magnitudes (floats' bits)
  alignas(16) float decay[64];  // mul d^(31 - i) (fp16: in the scores' range), then zeros
};
static_assert(sizeof(Control) <= 1024, "control");
// Products by one thread; once a wait of its has given up, or the limit is reached, none are
// issued any more.
struct Products {
  Control* c;
  int64_t wait_ns;
  uint32_t left;
  __device__ __forceinline__ Products(Control* control, const Limits& l) : c(control), wait_ns(l.wait_ns), left(l.products) {}
  __device__ __forceinline__ bool issues() {  // (of thread 0)
    if (!left) return false;
    --left;
    return true;
  }
  __device__ __forceinline__ void commit(int which, uint32_t parity) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(&c->done[which]))
                 : "memory");
    c->issued[which] = parity + 1;
  }
  // Waits for products; at most two seconds from the block's first wait on, after which nothing
  // is waited for any more, the results are undefined and the error is on record.
  __device__ __forceinline__ void wait(int which, uint32_t parity) {
    const uint32_t bar = smem_u32(&c->done[which]);
    if (!mbar_try(bar, parity)) {
      int64_t until = c->until;
      if (!until) c->until = until = now_ns() + wait_ns;  // (threads that do so together mean the same)
      while (!mbar_try(bar, parity)) {
        if (c->abort) {
          left = 0;
          break;
        }
        if (now_ns() > until) {
          c->abort = 1;
          atomicOr(&attn_timeouts, kErrTimeout);
        }
      }
    }
    __syncwarp();  // the warp's accesses to TMEM are in step
  }
};
template <int COLUMNS>
__device__ __forceinline__ uint32_t begin(Control* c) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < 3; ++i) mbar_init(smem_u32(&c->done[i]), 1), c->issued[i] = 0;
    c->until = 0;
    c->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x >> 5 == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&c->tmem)),
                 "n"(COLUMNS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  before_sync();
  __syncthreads();
  after_sync();
  return c->tmem;
}
// After giving up, nothing is under way when the block ends that writes its shared memory or
// TMEM: its threads wait for their own copies, one of them, again for two seconds at most, for
// the products that were issued and their arrivals (one at most on each barrier).
template <int COLUMNS>
__device__ __forceinline__ void end(Control* c, const Limits& limits, uint32_t tmem) {
  before_sync();
  __syncthreads();
  after_sync();
  if (c->abort) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (threadIdx.x == 0) {
      const int64_t until = now_ns() + limits.wait_ns;
      for (int i = 0; i < 3; ++i)
        while (c->issued[i] && !mbar_try(smem_u32(&c->done[i]), c->issued[i] - 1) && now_ns() < until) {}
    }
    __syncthreads();
  }
  if (threadIdx.x >> 5 == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(COLUMNS));
}

// 32 columns of the thread's lane; the values are there after loaded().
__device__ __forceinline__ void load32(uint32_t addr, float (&f)[32]) {
  uint32_t(&v)[32] = reinterpret_cast<uint32_t(&)[32]>(f);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(addr)
      : "memory");
}
// 16 lanes x 32 columns: thread t has columns 8 i + 2 (t % 4) and the next of lane t / 4
// in f[4 i], f[4 i + 1], and of lane t / 4 + 8 in the two after.
__device__ __forceinline__ void load16x32(uint32_t addr, float (&f)[16]) {
  uint32_t(&v)[16] = reinterpret_cast<uint32_t(&)[16]>(f);
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(addr)
      : "memory");
}
// Ties loaded values to the wait, so that no use of them moves before it.
template <int N>
__device__ __forceinline__ void loaded(float (&f)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(f[i]));
}
// 32 terms (16 words) of the thread's row.
__device__ __forceinline__ void store16(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// ---- tiles ------------------------------------------------------------------------
// A chunk's tile of W = 64 or 128 channels, in blocks of 64.  A chunk of n < kL tokens has
// them in its last n rows and zeros before them, so that a row's distance to the chunk's
// end is the same in every chunk.  Columns from dim on (a multiple of 8) are zeros.  A
// thread brings one granule of every kRows-th row.
template <int W>
struct Rows {
  static constexpr int kG = W / 8, kRows = kThreads / kG, kCount = kL / kRows;
  int r0, c;
  uint32_t at;  // of the thread's first granule; the next ones are kRows * 128 bytes on
  __device__ __forceinline__ Rows()
      : r0(threadIdx.x / kG), c(threadIdx.x % kG), at(c / 8 * kBlock + r0 * 128 + (((c & 7) ^ (r0 & 7)) << 4)) {}
};
template <typename T, int W>
__device__ __forceinline__ void load_tile(uint32_t tile, const T* from, int64_t stride, int n, int dim) {
  const Rows<W> k;
  const int pad = kL - n;
  const T* p = from + (k.r0 - pad) * stride + k.c * 8;
  uint32_t bytes = k.c * 8 < dim ? 16 : 0;
  int64_t next = k.kRows * stride;
  if (pad == 0) {
    if (!bytes) p = from, next = 0;  // (nothing is read there)
#pragma unroll
    for (int i = 0; i < k.kCount; ++i) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tile + k.at + i * k.kRows * 128), "l"(p),
                   "r"(bytes)
                   : "memory");
      p += next;
    }
  } else {
#pragma unroll 1
    for (int i = 0; i < k.kCount; ++i) {
      const bool there = bytes && k.r0 + i * k.kRows >= pad;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tile + k.at + i * k.kRows * 128),
                   "l"(there ? p : from), "r"(there ? 16 : 0)
                   : "memory");
      p += next;
    }
  }
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last N groups of copies are there.
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint4 get_granule(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void put_granule(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

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
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// The exponent that brings m near 2^13 when it is taken away.
__device__ __forceinline__ int exponent_of(float m) {
  return m > 0.f ? min(max((int)(__float_as_uint(m) >> 23) - 127 - 13, -100), 100) : 0;
}

// The tile's keys, weighted by d^(127 - row + shift) mul, as TERMS terms of T in as many
// tiles of the same layout, `next_term` bytes after one another (the first may be
// the keys' own tile).  Each thread takes the granules that it brought itself.
//
// bf16 in two terms: with the weight w = wh + wl in two, hi = k wh + k wl rounded once and
// lo = (k wh - hi) + k wl, off by 2^-17 of the value; two elements an instruction.
template <typename T, int KD, int TERMS>
__device__ __forceinline__ void weigh(uint32_t keys, uint32_t first_term, uint32_t next_term, float a, int shift,
                                      float mul) {
  const Rows<KD> k;
  float w = mul * power2(a * (float)(kL - 1 - (k.r0 + (k.kCount - 1) * k.kRows) + shift));
  const float next = power2(a * (float)k.kRows);
#pragma unroll
  for (int i = k.kCount - 1; i >= 0; --i) {
    const uint32_t at = k.at + i * k.kRows * 128;
    const uint4 raw = get_granule(keys + at);
    const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t out[TERMS][4];
    if constexpr (!std::is_same<T, __half>::value && TERMS == 2) {
      const __nv_bfloat16 first = __float2bfloat16_rn(w);
      const __nv_bfloat162 wh(first, first), wl = __float2bfloat162_rn(w - __bfloat162float(first));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&in[j]), t = __hmul2(x, wl);
        const __nv_bfloat162 hi = __hfma2(x, wh, t), lo = __hadd2(__hfma2(x, wh, __hneg2(hi)), t);
        out[0][j] = *reinterpret_cast<const uint32_t*>(&hi);
        out[1][j] = *reinterpret_cast<const uint32_t*>(&lo);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 x = mul2(unpack<T>(in[j]), both(w));
#pragma unroll
        for (int t = 0; t < TERMS; ++t) {
          out[t][j] = pair_word<T>(x.x, x.y);
          if (t + 1 < TERMS) x = fma2(unpack<T>(out[t][j]), both(-1.f), x);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < TERMS; ++t)
      put_granule(first_term + t * next_term + at, make_uint4(out[t][0], out[t][1], out[t][2], out[t][3]));
    w *= next;
  }
}
// Magnitudes compare as whole numbers, so that a warp's largest takes one instruction.
__device__ __forceinline__ uint32_t warp_top(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }
// A block's, by way of shared memory: the warps leave theirs before a barrier.
__device__ __forceinline__ void leave_top(Control* c, int which, float x) {
  if ((threadIdx.x & 31) == 0) c->top[which][threadIdx.x >> 5] = __float_as_uint(x);
}
__device__ __forceinline__ float top_of(const Control* c, int which) {
  const uint4 a = reinterpret_cast<const uint4*>(c->top[which])[0], b = reinterpret_cast<const uint4*>(c->top[which])[1];
  return __uint_as_float(max(max(max(a.x, a.y), max(a.z, a.w)), max(max(b.x, b.y), max(b.z, b.w))));
}
static_assert(kThreads == 256, "eight warps");
// fp16: the largest finite magnitude among the thread's own granules of the keys, in the warp.
// (An infinity must not set the range in which the others are kept; a maximum passes over
// NaN.)
template <int KD>
__device__ __forceinline__ float top_key(uint32_t keys) {
  const Rows<KD> k;
  __half2 most = __float2half2_rn(0.f);
#pragma unroll
  for (int i = 0; i < k.kCount; ++i) {
    const uint4 v = get_granule(keys + k.at + i * k.kRows * 128);
    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) most = __hmax2(most, __habs2(*reinterpret_cast<const __half2*>(&in[j])));
  }
  const float2 two = __half22float2(most);
  uint32_t top = warp_top(__float_as_uint(fmaxf(two.x, two.y)));
  if (top >= 0x7f800000u) {
    float x = 0.f;
#pragma unroll 1
    for (int i = 0; i < k.kCount * 8; ++i) {
      uint16_t v;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(keys + k.at + (i / 8) * k.kRows * 128 + i % 8 * 2) : "memory");
      if ((v & 0x7fffu) < 0x7c00u) x = fmaxf(x, __half2float(__ushort_as_half(v & 0x7fffu)));
    }
    top = warp_top(__float_as_uint(x));
  }
  return __uint_as_float(top);
}

// ---- the state: [KD][64] in the products' layout, half of the columns a half of the warps.
// KD = 64: a warp has 16 rows; 128: twice 16.
template <int KD>
struct State {
  static constexpr int kM = KD / 64;
  float v[kM][16];
  int row0, col0, g, t;
  uint32_t lanes;
  __device__ __forceinline__ State() {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    row0 = (warp & 3) * (KD / 4);
    col0 = (warp >> 2) * 32;
    g = lane >> 2, t = lane & 3;
    lanes = (uint32_t)((warp & 3) * 32) << 16;
  }
  __device__ __forceinline__ int row(int m, int j) const { return row0 + m * 16 + g + (j >> 1 & 1) * 8; }
  __device__ __forceinline__ int col(int j) const { return col0 + (j >> 2) * 8 + 2 * t + (j & 1); }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int j = 0; j < 16; ++j) v[m][j] = 0.f;
  }
  // Entry (row, e0 + col) from src[row * rs + (e0 + col) * cs].
  __device__ __forceinline__ void get(const float* src, int64_t rs, int64_t cs, int e0, int rows, int cols) {
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int r = row(m, j), c = e0 + col(j);
        v[m][j] = src && r < rows && c < cols ? src[r * rs + c * cs] : 0.f;
      }
  }
  __device__ __forceinline__ void put(float* to, int64_t stride) const {
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int j = 0; j < 16; j += 2)
        *reinterpret_cast<float2*>(to + row(m, j) * stride + col(j)) = make_float2(v[m][j], v[m][j + 1]);
  }
  // The largest finite magnitude in the warp.
  __device__ __forceinline__ float top() const {
    constexpr float kMost = 3.402823466e38f;
    float x = 0.f;
    auto in_warp = [&] { x = __uint_as_float(warp_top(__float_as_uint(x))); };
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int j = 0; j < 16; ++j) x = fmaxf(x, fabsf(v[m][j]));
    in_warp();
    if (x > kMost) {
      x = 0.f;
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (fabsf(v[m][j]) <= kMost) x = fmaxf(x, fabsf(v[m][j]));
      in_warp();
    }
    return x;
  }
  // As the products take it: rows of 64 T.
  template <typename T>
  __device__ __forceinline__ void to_tile(uint32_t tile, float scale) const {
#pragma unroll
    for (int m = 0; m < kM; ++m) {
      const uint32_t at = tile + (row0 + m * 16 + g) * 128 + ((col0 / 8 ^ g) << 4) + t * 4;
#pragma unroll
      for (int j = 0; j < 16; j += 2)
        asm volatile("st.shared.b32 [%0], %1;" ::"r"((at ^ (j >> 2 << 4)) + (j >> 1 & 1) * 1024),
                     "r"(pair_word<T>(v[m][j] * scale, v[m][j + 1] * scale))
                     : "memory");
    }
  }
  // v <- decay v + back (what the tensor core summed at `sum`)
  __device__ __forceinline__ void update(uint32_t sum, float decay, float back) {
    float u[kM][16];
#pragma unroll
    for (int m = 0; m < kM; ++m) load16x32(sum + lanes + ((uint32_t)(m * 16) << 16) + col0, u[m]);
#pragma unroll
    for (int m = 0; m < kM; ++m) {
      loaded(u[m]);
#pragma unroll
      for (int j = 0; j < 16; ++j) v[m][j] = v[m][j] * decay + u[m][j] * back;
    }
  }
};
// terms^T values: the products of a state's update, by one thread.
template <typename T, int KD, int TERMS>
__device__ __forceinline__ void mma_state(uint32_t d, uint32_t first_term, uint32_t next_term, uint32_t values) {
  const uint32_t idesc = instruction<T>(KD, kV, true, true);
  const uint64_t b = operand<true>(values);
#pragma unroll
  for (int t = 0; t < TERMS; ++t) {
    const uint64_t a = operand<true>(first_term + t * next_term);
#pragma unroll
    for (int i = 0; i < kL / 16; ++i) mma(d, a + i * (2048 >> 4), b + i * (2048 >> 4), idesc, t > 0 || i > 0);
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

// Up to 64 channels two sets of keys and values, and the terms: loads are two chunks ahead.
// With 128 one set, in which the first term takes the keys' place, so that an SM has two
// blocks (4 groups of 2040 tokens, 8 heads of 128: 16 us; two sets, one block 22).
template <int KD, int TERMS>
constexpr int kPartsSmem = 1024 + (KD == 64 ? 2 * 2 + TERMS : 3 + 2 * (TERMS - 1)) * kBlock;

template <typename T, int KD, int TERMS>
__device__ __forceinline__ void sum_part(const PartsArgs& p, const Part& part, int e0, Control* c, uint32_t tiles,
                                         uint32_t tmem) {
  constexpr bool kHalfType = std::is_same<T, __half>::value;
  constexpr int kSets = KD == 64 ? 2 : 1;
  constexpr uint32_t kTerm = KD / 64 * kBlock, kSet = kTerm + kBlock;
  const uint32_t terms = kSets == 2 ? tiles + 2 * kSet : tiles;
  const int h = blockIdx.y;
  const Span s = span_of(p.split, blockIdx.x);
  const float a = log2_decay(p.log_decay, h);
  const int64_t from = part.back ? s.start + s.n - 1 : s.start;
  const int64_t step = part.back ? -1 : 1;
  const T* k = head_at<T>(part.key, h, p.rep, from);
  const T* v = head_at<T>(part.value, h, p.rep, from) + e0;
  const int chunks = (s.n + kL - 1) / kL;
  // Two sets: a chunk's keys make room when they have been weighed (each thread brings the
  // granules that it weighs), its values when they have been multiplied.
  auto keys_of = [&](int i) { return kSets == 2 ? tiles + (i & 1) * kSet : tiles; };
  auto values_of = [&](int i) { return kSets == 2 ? tiles + (i & 1) * kSet + kTerm : tiles + TERMS * kTerm; };
  auto load_keys = [&](int i) {
    if (i < chunks)
      load_tile<T, KD>(keys_of(i), k + step * i * kL * part.key.token, step * part.key.token, min(kL, s.n - i * kL),
                       part.key.dim);
    copies_commit();
  };
  auto load_values = [&](int i) {
    if (i < chunks)
      load_tile<T, kV>(values_of(i), v + step * i * kL * part.value.token, step * part.value.token,
                       min(kL, s.n - i * kL), part.value.dim - e0);
    copies_commit();
  };
  Products products(c, p.split.limits);
  State<KD> st;
  st.zero();
#pragma unroll
  for (int i = 0; i < kSets; ++i) {
    load_keys(i);
    load_values(i);
  }
  for (int i = 0; i < chunks; ++i) {
    const uint32_t keys = keys_of(i);
    copies_wait<2 * (kSets - 1)>();
    float mul = part.mul, back = 1.f;
    if constexpr (kHalfType) {
      leave_top(c, i & 1, top_key<KD>(keys));
      __syncthreads();
      const int e = exponent_of(top_of(c, i & 1) * fabsf(part.mul) * power2(a * (float)part.shift));
      mul *= power_of_two(-e);
      back = power_of_two(e);
    }
    weigh<T, KD, TERMS>(keys, terms, kTerm, a, part.shift, mul);
    publish();
    before_sync();
    __syncthreads();
    if (threadIdx.x == 0 && products.issues()) {
      after_sync();
      mma_state<T, KD, TERMS>(tmem, terms, kTerm, values_of(i));
      products.commit(0, i & 1);
    }
    if (kSets == 2) load_keys(i + kSets);
    products.wait(0, i & 1);
    after_sync();
    if (kSets == 1) load_keys(i + kSets);
    load_values(i + kSets);
    st.update(tmem, power2(a * (float)min(kL, s.n - i * kL)), back);
  }
  if (s.n) st.put(part.to + ((int64_t)blockIdx.x * p.heads + h) * p.Dp * p.Ep + e0, p.Ep);
}

// TERMS: the most that a part's keys are taken as.  Bound by the loads of rows of 128 bytes:
// 32640 tokens, 16 heads of 64, bf16, 14 chunks a segment: 33 us for 134 MB (2 terms 27);
// with neither the weighing nor the products 28, without one of them 29.  Halves of a chunk
// in turn, one weighed while the other is multiplied, gained nothing (35).
template <typename T, int KD, int TERMS>
__global__ void __launch_bounds__(kThreads, 2) attn_parts_kernel(const __grid_constant__ PartsArgs p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Control* c = (Control*)smem;
  const uint32_t tmem = begin<64>(c);
  launch_dependents();
  wait_for_previous();
  const int blocks = p.Ep / kV, e0 = blockIdx.z % blocks * kV;
  const Part& part = p.part[blockIdx.z / blocks];
  if (TERMS == 2 || !part.exact) sum_part<T, KD, 2>(p, part, e0, c, smem_u32(smem) + 1024, tmem);
  else sum_part<T, KD, TERMS>(p, part, e0, c, smem_u32(smem) + 1024, tmem);
  end<64>(c, p.split.limits, tmem);
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

// VEC neighbouring elements of the state in a row a thread, AHEAD segments' loads under
// way.
constexpr int kScanThreads = 256;
template <int VEC, int AHEAD>
__global__ void __launch_bounds__(kScanThreads) attn_scan_kernel(const __grid_constant__ ScanArgs p) {
  launch_dependents();
  wait_for_previous();
  const Scan& k = p.scan[blockIdx.z];
  const int across = (p.E + VEC - 1) / VEC, per = (p.D * across + kScanThreads - 1) / kScanThreads;
  const int h = blockIdx.y, g = blockIdx.x / per, i = blockIdx.x % per * kScanThreads + threadIdx.x;
  if (i >= p.D * across) return;
  const int row = i / across, col = i % across * VEC, size = p.Dp * p.Ep;
  const float a = log2_decay(p.log_decay, h);
  const uint32_t begin = (uint32_t)offset_of(p.split, g), end = (uint32_t)offset_of(p.split, g + 1);
  const uint32_t seg = p.split.seg;
  const int64_t first = begin / seg + g;
  const int slots = end > begin ? (end - begin + seg - 1) / seg : 0;
  const int tail = (int)(end - begin - (slots - 1) * seg);
  const int64_t mat = ((int64_t)g * p.heads + h) * p.D * p.E + row * p.E + col;
  Pack<float, VEC> s;
#pragma unroll
  for (int x = 0; x < VEC; ++x) s.v[x] = k.edge && col + x < p.E ? k.edge[mat + x] : 0.f;
  const float full = power2(a * (float)p.split.seg), rest = power2(a * (float)tail);
  const int last = slots - 1;
  const int64_t stride = (k.back ? -1 : 1) * (int64_t)p.heads * size;
  float* at = k.parts + ((first + (k.back ? last : 0)) * p.heads + h) * size + row * p.Ep + col;
  for (int b = 0; b < slots; b += AHEAD) {
    Pack<float, VEC> u[AHEAD];  // (a part's columns go on to a whole vector)
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
      if (b + j < slots) u[j] = load_pack<float, VEC>(at + stride * (b + j));
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      if (b + j >= slots) break;
      store_pack<float, VEC>(at + stride * (b + j), s);
      const float d = (k.back ? b + j == 0 : b + j == last) ? rest : full;
#pragma unroll
      for (int x = 0; x < VEC; ++x) s.v[x] = s.v[x] * d + u[j].v[x];
    }
  }
  if (k.last)
#pragma unroll
    for (int x = 0; x < VEC; ++x)
      if (col + x < p.E) k.last[mat + x] = s.v[x];
}

// ---- outputs -----------------------------------------------------------------
// TMEM: the products of queries and keys; the decayed ones as the next product's operand;
// queries times the state; in the first one's place then the decayed ones times the values
// and the state's update.
constexpr uint32_t kScores = 0, kDecayed = 128, kOuter = 192, kInner = 0, kUpdate = 64;

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

// scores = queries keys^T, outer = queries state (TRANSPOSED: state^T, of 64 x 64), by one
// thread.
template <typename T, int KD, bool TRANSPOSED>
__device__ __forceinline__ void mma_scores(uint32_t tmem, uint32_t queries, uint32_t keys, uint32_t state) {
  const uint64_t q = operand<false>(queries), k = operand<false>(keys), s = operand<!TRANSPOSED>(state);
  const uint32_t scores = instruction<T>(kL, kL, false, false), outer = instruction<T>(kL, kV, false, !TRANSPOSED);
#pragma unroll
  for (int i = 0; i < KD / 16; ++i) {
    const uint64_t at = (i / 4 * kBlock + i % 4 * 32) >> 4;
    mma(tmem + kScores, q + at, k + at, scores, i > 0);
  }
#pragma unroll
  for (int i = 0; i < KD / 16; ++i)
    mma(tmem + kOuter, q + ((i / 4 * kBlock + i % 4 * 32) >> 4), s + i * (TRANSPOSED ? 32 >> 4 : 2048 >> 4), outer, i > 0);
}
// inner = decayed values
template <typename T>
__device__ __forceinline__ void mma_inner(uint32_t tmem, uint32_t values) {
  const uint64_t v = operand<true>(values);
  const uint32_t inner = instruction<T>(kL, kV, false, true);
#pragma unroll
  for (int i = 0; i < kL / 16; ++i) mma_tmem(tmem + kInner, tmem + kDecayed + 8 * i, v + i * (2048 >> 4), inner, i > 0);
}

// The scores' decay and mask: a thread has a row, and of its four blocks of 32 columns
// every second one.  Row and column are l and x in their blocks: below the diagonal
// d^(32 (row block - column block) + l - 31) d^(31 - x), on it d^(l - x) where x <= l.
template <typename T>
__device__ __forceinline__ void decay_scores(uint32_t tmem, const Control* c, float a) {
  const int warp = threadIdx.x >> 5, l = threadIdx.x & 31, rb = warp & 3;
  const uint32_t lanes = tmem + ((uint32_t)(rb * 32) << 16);
#pragma unroll 1
  for (int b = warp >> 2; b < 4; b += 2) {
    uint32_t o[16];
    if (b > rb) {
#pragma unroll
      for (int j = 0; j < 16; ++j) o[j] = 0;
    } else {
      float s[32];
      load32(lanes + kScores + 32 * b, s);
      if (b < rb) {
        const float2 f = both(power2(a * (float)(32 * (rb - b) + l - 31)));
        loaded(s);
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 d = *reinterpret_cast<const float4*>(c->decay + j);
          const float2 x = mul2(mul2(make_float2(s[j], s[j + 1]), make_float2(d.x, d.y)), f);
          const float2 y = mul2(mul2(make_float2(s[j + 2], s[j + 3]), make_float2(d.z, d.w)), f);
          o[j / 2] = pair_word<T>(x.x, x.y);
          o[j / 2 + 1] = pair_word<T>(y.x, y.y);
        }
      } else {
        const float* d = c->decay + 31 - l;
        loaded(s);
#pragma unroll
        for (int j = 0; j < 32; j += 2)  // (what the mask takes out may be a NaN)
          o[j / 2] = pair_word<T>(s[j] * d[j], s[j + 1] * d[j + 1]) & (j < l ? 0xffffffffu : j == l ? 0xffffu : 0u);
      }
    }
    store16(lanes + kDecayed + 16 * b, o);
  }
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

struct Output {
  void* p;              // of the chunk's first token and the block's first channel
  int64_t stride;       // between the chunk's tokens
  int32_t dim, wide;    // channels from there on; whole granules on 16-byte boundaries
};
struct Whole {  // outputs in fp32, or NULL
  float* p;             // as Output::p
  int64_t stride;
};
// back inner (fp16, else inner) + f outer of half a row: to memory in fp32, or as 32 T.
template <typename T>
__device__ __forceinline__ void get_outputs(uint32_t tmem, float back, float f, const Whole& whole, int pad,
                                            uint32_t (&w)[16]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = warp >> 2, row = (warp & 3) * 32 + lane;
  const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16) + half * 32;
  float x[32], y[32];
  load32(lanes + kInner, x);
  load32(lanes + kOuter, y);
  loaded(x);
  loaded(y);
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    float2 u = make_float2(x[j], x[j + 1]);
    if (std::is_same<T, __half>::value) u = mul2(u, both(back));
    const float2 v = fma2(make_float2(y[j], y[j + 1]), both(f), u);
    x[j] = v.x, x[j + 1] = v.y;
  }
  if (whole.p) {
    float4* to = reinterpret_cast<float4*>(whole.p + (row - pad) * whole.stride + half * 32);
    if (row >= pad)
#pragma unroll
      for (int j = 0; j < 8; ++j) to[j] = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
    return;
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) w[j] = pair_word<T>(x[2 * j], x[2 * j + 1]);
}
// These to memory, by way of `room` (a tile whose rows of the warp nothing uses); the rows
// from pad on are there.  A warp stores its 32 rows' halves.
template <typename T>
__device__ __forceinline__ void put_outputs(uint32_t room, const uint32_t (&w)[16], const Output& out, int pad) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, half = warp >> 2, row = (warp & 3) * 32 + lane;
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j)
    put_granule(room + row * 128 + (((half * 4 + j) ^ (row & 7)) << 4),
                make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]));
  __syncwarp();
  if (out.wide) {
    // (rows r and r + 4 together: their granules lie in different banks)
    const int g = half * 4 + (lane & 3), r0 = (warp & 3) * 32 + (lane >> 3) + (lane & 4);
    T* to = (T*)out.p + (r0 - pad) * out.stride + g * 8;
    if (g * 8 < out.dim)
#pragma unroll
      for (int i = 0; i < 4; ++i, to += 8 * out.stride) {
        const int r = r0 + i * 8;
        if (r >= pad) *reinterpret_cast<uint4*>(to) = get_granule(room + r * 128 + ((g ^ (r & 7)) << 4));
      }
  } else {
    const int col = half * 32 + lane;
    if (col < out.dim)
      for (int r = max((warp & 3) * 32, pad); r < (warp & 3) * 32 + 32; ++r) {
        uint16_t v;
        asm volatile("ld.shared.u16 %0, [%1];"
                     : "=h"(v)
                     : "r"(room + r * 128 + (((col >> 3) ^ (r & 7)) << 4) + (col & 7) * 2)
                     : "memory");
        reinterpret_cast<uint16_t*>(out.p)[(r - pad) * out.stride + col] = v;
      }
  }
  __syncwarp();
}

// fp16: powers of two that keep the state, the weighted keys and the decayed scores in range,
// from the block's largest ones; nothing for bf16.  A score is a sum of `channels` products,
// and none is beyond that many times the largest query and key.
struct Fit {
  float state = 1.f, state_back = 1.f, key = 1.f, key_back = 1.f, score = 1.f, score_back = 1.f;
};
__device__ __forceinline__ void fit_scores(Fit& f, float top_query, float top_key, float channels) {
  const int e = exponent_of(top_query * top_key * channels);
  f.score = power_of_two(-e), f.score_back = power_of_two(e);
}
// Control::decay, which is read after a barrier.
__device__ __forceinline__ void leave_decay(Control* c, float mul, float a) {
  if (threadIdx.x < 32) c->decay[threadIdx.x] = mul * power2(a * (float)(31 - (int)threadIdx.x));
}
// keys: those that are weighted; score_weight: what the scores are multiplied by, times their
// channels.  Takes a barrier.
template <typename T, int KD>
__device__ __forceinline__ Fit fit_of(Control* c, const State<KD>& st, uint32_t keys, float top_weight, uint32_t queries,
                                      float score_weight) {
  Fit f;
  if constexpr (std::is_same<T, __half>::value) {
    leave_top(c, 0, st.top());
    leave_top(c, 1, top_key<KD>(keys));
    leave_top(c, 2, top_key<KD>(queries));
    __syncthreads();
    const float key = top_of(c, 1);
    const int e = exponent_of(top_of(c, 0)), ke = exponent_of(key * fabsf(top_weight));
    f.state = power_of_two(-e), f.state_back = power_of_two(e);
    f.key = power_of_two(-ke), f.key_back = power_of_two(ke);
    fit_scores(f, top_of(c, 2), key, fabsf(score_weight));
  }
  return f;
}

struct OutArgs {
  Split split;
  int32_t heads, rep;    // query heads
  Side query, key, value, out;
  const float* log_decay;
  int32_t K, V, Kp, Vp;  // keys' and values' channels, and rounded up to 64 or 128
  const float* states;   // [slots][heads][Kp][Vp], NULL: no group has more than one segment
  const float* edge;     // [groups][heads][..] or NULL (zeros)
  int32_t transposed;    // states are stored [values' channels][keys' channels] (and [Vp][Kp])
  int32_t back, shift;
  float mul_inner, mul_state, mul_key;
  float* whole;          // [tokens from split.from][heads][Vp]: instead of out, in fp32
};
template <int KD>
constexpr int kOutSets = KD == 64 ? 2 : 1;
template <int KD>
constexpr int kOutSmem = 1024 + kOutSets<KD> * (2 * (KD / 64) + 1) * kBlock + KD * 128 + (KD == 64 ? 0 : kBlock);

// One pass over a segment's queries, keys and values.  32640 tokens, 16 heads of 64, bf16,
// forward: 58 us for 273 MB, 4.7 TB/s; no part of the work bounds it alone: taken out by
// itself, the stores of the outputs are worth 8 us, the decay, the weighing and the state's
// products 4 or 5 each.  Shared memory is busy for three quarters of a chunk's time.
// WHOLE: in fp32, instead.
template <typename T, int KD, bool WHOLE>
__device__ __forceinline__ void form_outputs(const OutArgs& p, int slot, int h, int e0, Control* c, uint32_t tiles,
                                             uint32_t tmem) {
  constexpr uint32_t kKeys = KD / 64 * kBlock;
  // The weighted keys' terms take the places of the keys and of the queries when these have
  // been multiplied.  Up to 64 channels there is room for two sets of tiles in turn, so that
  // a chunk comes while the one before is worked on, whose outputs leave through its keys'
  // tile while the next one's scores are formed; with 128 one set, and a tile for the
  // outputs, leave room for two blocks an SM instead.
  constexpr bool kHalfType = std::is_same<T, __half>::value;
  constexpr uint32_t kSets = kOutSets<KD>, kSet = 2 * kKeys + kBlock;  // queries, keys, values
  const uint32_t state = tiles + kSets * kSet;
  const Span s = span_of(p.split, slot);
  const int64_t from = p.back ? s.start + s.n - 1 : s.start, step = p.back ? -1 : 1;
  const int chunks = (s.n + kL - 1) / kL;
  const int row = ((int)threadIdx.x >> 5 & 3) * 32 + ((int)threadIdx.x & 31);
  uint32_t phase = 0, update_phase = 0;
  if (!s.n) return;
  Products products(c, p.split.limits);

  const float a = log2_decay(p.log_decay, h);
  const T* q = head_at<T>(p.query, h, p.rep, from);
  const T* k = head_at<T>(p.key, h, p.rep, from);
  const T* v = head_at<T>(p.value, h, p.rep, from) + e0;
  auto load_keys = [&](int i) {
    load_tile<T, KD>(tiles + i % kSets * kSet + kKeys, k + step * i * kL * p.key.token, step * p.key.token,
                     min(kL, s.n - i * kL), p.key.dim);
    copies_commit();
  };
  auto load_others = [&](int i) {
    const int n = min(kL, s.n - i * kL);
    const int64_t at = step * i * kL;
    const uint32_t to = tiles + i % kSets * kSet;
    load_tile<T, KD>(to, q + at * p.query.token, step * p.query.token, n, p.query.dim);
    load_tile<T, kV>(to + 2 * kKeys, v + at * p.value.token, step * p.value.token, n, p.value.dim - e0);
    copies_commit();
  };
  load_keys(0);
  load_others(0);
  if (threadIdx.x < 32) c->decay[32 + threadIdx.x] = 0.f;
  if (!kHalfType) leave_decay(c, p.mul_inner, a);
  State<KD> st;
  const Stored src = stored(p.states, p.edge, p.Kp, p.Vp, p.K, p.V, p.transposed, (int64_t)slot * p.heads + h,
                            (int64_t)s.group * p.heads + h);
  st.get(src.p, src.rs, src.cs, e0, p.K, p.V);
  const float top_weight = p.mul_key * power2(a * (float)p.shift);

  auto room = [&](int i) { return kSets == 2 ? tiles + (i & 1) * kSet + kKeys : state + KD * 128; };
  auto put = [&](int i, const uint32_t(&w)[16], int pad) {
    const int64_t tok = from + step * i * kL;
    put_outputs<T>(room(i), w, Output{(T*)p.out.p + (int64_t)h * p.out.head + tok * p.out.token + e0,
                                      step * p.out.token, p.out.dim - e0, p.out.wide}, pad);
  };
  uint32_t w[16];
  for (int i = 0; i < chunks; ++i, phase ^= 1) {
    const int n = min(kL, s.n - i * kL), pad = kL - n;
    const uint32_t queries = tiles + i % kSets * kSet, keys = queries + kKeys, values = keys + kKeys;
    const bool more = i + 1 < chunks;
    copies_wait<0>();
    const Fit fit = fit_of<T, KD>(c, st, keys, top_weight, queries, p.mul_inner * (float)p.K);
    if (kHalfType) leave_decay(c, p.mul_inner * fit.score, a);
    st.template to_tile<T>(state, fit.state);
    publish();
    before_sync();
    __syncthreads();
    if (threadIdx.x == 0 && products.issues()) {
      after_sync();
      mma_scores<T, KD, false>(tmem, queries, keys, state);
      products.commit(0, phase);
    }
    if (more && kSets == 2) load_others(i + 1);
    if (i > 0 && !WHOLE) put(i - 1, w, 0);
    products.wait(0, phase);
    after_sync();
    if (more) weigh<T, KD, 2>(keys, keys, queries - keys, a, p.shift, p.mul_key * fit.key);
    decay_scores<T>(tmem, c, a);
    publish();
    before_sync();
    __syncthreads();
    if (threadIdx.x == 0 && products.issues()) {
      after_sync();
      mma_inner<T>(tmem, values);
      products.commit(1, phase);
      if (more) {
        mma_state<T, KD, 2>(tmem + kUpdate, keys, queries - keys, values);
        products.commit(2, update_phase);
      }
    }
    if (more && kSets == 2) load_keys(i + 1);
    products.wait(1, phase);
    after_sync();
    const int64_t tok = from + step * i * kL;
    const Whole whole{WHOLE ? p.whole + ((tok - p.split.from) * p.heads + h) * p.Vp + e0 : nullptr,
                      step * p.heads * p.Vp};
    // (rows before the chunk's first token are not there)
    get_outputs<T>(tmem, fit.score_back, p.mul_state * fit.state_back * power2(a * (float)max(row + 1 - p.shift - pad, 0)),
                   whole, pad, w);
    if (more) {
      products.wait(2, update_phase);
      update_phase ^= 1;
      after_sync();
      if (kSets == 1) {
        load_keys(i + 1);
        load_others(i + 1);
      }
      st.update(tmem + kUpdate, power2(a * (float)n), fit.key_back);
    }
  }
  if (!WHOLE) put(chunks - 1, w, kL - (s.n - (chunks - 1) * kL));
}

template <typename T, int KD>
__global__ void __launch_bounds__(kThreads, 2) attn_out_kernel(const __grid_constant__ OutArgs p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Control* c = (Control*)smem;
  const uint32_t tmem = begin<256>(c);
  launch_dependents();
  wait_for_previous();
  form_outputs<T, KD, false>(p, blockIdx.x, blockIdx.y, blockIdx.z * kV, c, smem_u32(smem) + 1024, tmem);
  end<256>(c, p.split.limits, tmem);
}

// ---- the gradients of keys and values together -----------------------------------
// Heads of up to 64 channels: both go through the tokens backwards with the same state R
// [dim][vdim] (the gradient of the state), which is read as it lies for dv and transposed
// for dk, and updated once.
struct KvArgs {
  Split split;
  int32_t heads, rep;
  Side q, k, v, g, dk, dv;
  int32_t D, E;
  const float* log_decay;
  const float* states;  // [slots][heads][64][64], NULL: no group has more than one segment
  const float* edge;    // [groups][heads][dim][vdim] or NULL (zeros)
  float scale;
  float* whole[2];      // [tokens from split.from][heads][64]: instead of dk and dv, in fp32
};
constexpr int kKvSmem = 1024 + 6 * kBlock + 64 * 128;  // keys and queries twice, values, douts; the state

template <typename T, bool WHOLE>
__device__ __forceinline__ void form_kv(const KvArgs& p, int slot, int h, Control* c, uint32_t tiles, uint32_t tmem) {
  constexpr bool kHalfType = std::is_same<T, __half>::value;
  // Keys and queries in two pairs of tiles in turn: the next chunk's come while this one's
  // last products are formed, its values and douts while its first scores are.  The weighted
  // queries' terms take the places of keys and values when these have been multiplied.  dv
  // and dk leave through a keys' tile that is not in use while the next scores are formed.
  const uint32_t pairs = tiles, values = pairs + 4 * kBlock, douts = values + kBlock, state = douts + kBlock;
  const Span s = span_of(p.split, slot);
  const int64_t from = s.start + s.n - 1;
  const int chunks = (s.n + kL - 1) / kL;
  const int row = ((int)threadIdx.x >> 5 & 3) * 32 + ((int)threadIdx.x & 31);
  uint32_t update_phase = 0;
  if (!s.n) return;
  Products products(c, p.split.limits);

  const float a = log2_decay(p.log_decay, h);
  auto load_keys = [&](int i) {
    load_tile<T, 64>(pairs + (i & 1) * 2 * kBlock, head_at<T>(p.k, h, p.rep, from - (int64_t)i * kL), -p.k.token,
                     min(kL, s.n - i * kL), p.k.dim);
    copies_commit();
  };
  auto load_queries = [&](int i) {
    load_tile<T, 64>(pairs + (i & 1) * 2 * kBlock + kBlock, head_at<T>(p.q, h, p.rep, from - (int64_t)i * kL),
                     -p.q.token, min(kL, s.n - i * kL), p.q.dim);
    copies_commit();
  };
  auto load_others = [&](int i) {
    const int n = min(kL, s.n - i * kL);
    const int64_t at = from - (int64_t)i * kL;
    load_tile<T, 64>(douts, head_at<T>(p.g, h, p.rep, at), -p.g.token, n, p.g.dim);
    load_tile<T, 64>(values, head_at<T>(p.v, h, p.rep, at), -p.v.token, n, p.v.dim);
    copies_commit();
  };
  load_queries(0);
  load_keys(0);
  load_others(0);
  if (threadIdx.x < 32) c->decay[32 + threadIdx.x] = 0.f;
  if (!kHalfType) leave_decay(c, p.scale, a);
  State<64> st;
  const Stored src = stored(p.states, p.edge, 64, 64, p.D, p.E, 0, (int64_t)slot * p.heads + h,
                            (int64_t)s.group * p.heads + h);
  st.get(src.p, src.rs, src.cs, 0, p.D, p.E);
  const float top_weight = p.scale * power2(a);

  auto put = [&](int i, const uint32_t(&w)[16], const Side& side, uint32_t room, int pad) {
    put_outputs<T>(room, w, Output{head_at<T>(side, h, p.rep, from - (int64_t)i * kL), -side.token, side.dim, side.wide},
                   pad);
  };
  uint32_t w[16];
  for (int i = 0; i < chunks; ++i) {
    const int n = min(kL, s.n - i * kL), pad = kL - n;
    const bool more = i + 1 < chunks;
    const uint32_t keys = pairs + (i & 1) * 2 * kBlock, queries = keys + kBlock, other = pairs + (~i & 1) * 2 * kBlock;
    copies_wait<1>();  // (values and douts may be on their way)
    Fit fit = fit_of<T, 64>(c, st, queries, top_weight, keys, p.scale * (float)p.D);
    if (kHalfType) leave_decay(c, p.scale * fit.score, a);
    st.template to_tile<T>(state, fit.state);
    publish();
    before_sync();
    __syncthreads();
    const float f = fit.state_back * power2(a * (float)max(row - pad, 0));
    const int64_t at = ((from - p.split.from - (int64_t)i * kL) * p.heads + h) * 64;
#pragma unroll
    for (int ph = 0; ph < 2; ++ph) {  // dv, dk: the first two barriers are used twice a chunk
      if (threadIdx.x == 0 && products.issues()) {
        after_sync();
        if (ph == 0) mma_scores<T, 64, false>(tmem, keys, queries, state);
        else mma_scores<T, 64, true>(tmem, values, douts, state);
        products.commit(0, ph);
      }
      if (ph == 0) {
        if (more) load_queries(i + 1);
        else copies_commit();
      }
      if (!WHOLE && (ph || i > 0)) put(ph ? i : i - 1, w, ph ? p.dv : p.dk, other, ph ? pad : 0);
      products.wait(0, ph);
      after_sync();
      if (ph == 1 && more) weigh<T, 64, 2>(queries, keys, values - keys, a, 1, p.scale * fit.key);
      decay_scores<T>(tmem, c, a);
      if (ph == 0) copies_wait<1>();  // they are there, the next queries may be on their way
      if (ph == 0 && kHalfType) leave_top(c, 0, top_key<64>(values)), leave_top(c, 1, top_key<64>(douts));
      publish();
      before_sync();
      __syncthreads();
      if (threadIdx.x == 0 && products.issues()) {
        after_sync();
        mma_inner<T>(tmem, ph ? queries : douts);
        products.commit(1, ph);
        if (ph == 1 && more) {
          mma_state<T, 64, 2>(tmem + kUpdate, keys, values - keys, douts);
          products.commit(2, update_phase);
        }
      }
      if (ph == 1 && more) load_keys(i + 1);
      products.wait(1, ph);
      after_sync();
      get_outputs<T>(tmem, fit.score_back, f, Whole{WHOLE ? p.whole[1 - ph] + at : nullptr, -(int64_t)p.heads * 64}, pad, w);
      if (ph == 0) {
        if (kHalfType) {
          fit_scores(fit, top_of(c, 0), top_of(c, 1), fabsf(p.scale) * (float)p.E);
          leave_decay(c, p.scale * fit.score, a);
        }
        before_sync();
        __syncthreads();  // the sums in TMEM have been read
      } else if (more) {
        products.wait(2, update_phase);
        update_phase ^= 1;
        after_sync();
        load_others(i + 1);
        st.update(tmem + kUpdate, power2(a * (float)n), fit.key_back);
      }
    }
  }
  if (!WHOLE) put(chunks - 1, w, p.dk, pairs + (~chunks & 1) * 2 * kBlock, kL - (s.n - (chunks - 1) * kL));
}

// ---- all gradients in one launch ------------------------------------------------------
// Two or three kinds of blocks, the ones that take longest first, so that few are left alone
// at the end (5003 tokens in 7 groups, heads of 72 and 41: 91 us in three launches, 51 in
// one).  A segment's blocks next to one another read a quarter less from memory (32640
// tokens, 16 heads of 64, bf16: 351 MB, as it is 486) and take longer all the same, 195 us
// instead of 160: the long ones at the end.  ED, EE: dim and vdim, padded.  SHARED: key
// heads are; dk and dv then leave in fp32, for the join.
struct GradArgs {
  int32_t slot0, slots, heads;
  int32_t first, second;  // where the blocks of a kind end
  OutArgs dq, dk, dv;
  KvArgs both;            // dk and dv of heads of up to 64 channels
};
template <int ED, int EE>
constexpr int kGradSmem = ED == 64 && EE == 64 ? (kKvSmem > kOutSmem<64> ? kKvSmem : kOutSmem<64>)
                                               : (kOutSmem<64> > kOutSmem<128> ? kOutSmem<64> : kOutSmem<128>);

template <typename T, int ED, int EE, bool SHARED>
__global__ void __launch_bounds__(kThreads, 2) attn_grad_kernel(const __grid_constant__ GradArgs p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Control* c = (Control*)smem;
  const uint32_t tmem = begin<256>(c), tiles = smem_u32(smem) + 1024;
  launch_dependents();
  wait_for_previous();
  const int kind = (int)blockIdx.x < p.first ? 0 : (int)blockIdx.x < p.second ? 1 : 2;
  const int b = blockIdx.x - (kind == 0 ? 0 : kind == 1 ? p.first : p.second);
  const int at = b / p.slots, slot = p.slot0 + b % p.slots, h = at % p.heads, e0 = at / p.heads * kV;
  if (kind == 0) {
    if constexpr (ED == 64 && EE == 64) form_kv<T, SHARED>(p.both, slot, h, c, tiles, tmem);
    else form_outputs<T, EE, SHARED>(p.dk, slot, h, e0, c, tiles, tmem);
  } else if (kind == 1) {
    if constexpr (ED != 64 || EE != 64) form_outputs<T, ED, SHARED>(p.dv, slot, h, e0, c, tiles, tmem);
  } else {
    form_outputs<T, EE, false>(p.dq, slot, h, e0, c, tiles, tmem);
  }
  end<256>(c, p.dq.split.limits, tmem);
}

// ---- gradients of shared heads: the sums over their query heads, in their order ----------
struct JoinArgs {
  Split split;
  int32_t heads, rep;     // key heads
  const float* whole[2];  // [tokens from split.from][query heads][padded]
  int32_t padded[2];
  Side to[2];
};
// Four channels of a token's head a thread.  Bound by the bytes.  (A block that goes through
// a key head's query heads itself, its sums in memory between them, needs no such kernel,
// but takes longer: 32640 tokens, 16 heads of 64 over 4, 543 us, in this way 306.)
template <typename T>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ JoinArgs p) {
  launch_dependents();
  wait_for_previous();
  const int w = blockIdx.y;
  const Side& to = p.to[w];
  const int fours = (to.dim + 3) / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, r = i / fours, token = p.split.from + r / p.heads;
  const int c = (int)(i % fours) * 4, h = (int)(r % p.heads);
  if (token < offset_of(p.split, 0) || token >= offset_of(p.split, p.split.groups)) return;
  // a segment at an end of the range belongs to the one that it starts in
  if (token >= p.split.upto || (p.split.from && token < p.split.from + p.split.seg)) {
    const int64_t start = segment_start(p.split, token);
    if (start < p.split.from || start >= p.split.upto) return;
  }
  const float* from = p.whole[w] + r * p.rep * p.padded[w] + c;
  float4 v = *reinterpret_cast<const float4*>(from);
  for (int j = 1; j < p.rep; ++j) {
    const float4 u = *reinterpret_cast<const float4*>(from + j * p.padded[w]);
    v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
  }
  T* out = (T*)to.p + token * to.token + h * to.head + c;
  const uint32_t lo = pair_word<T>(v.x, v.y), hi = pair_word<T>(v.z, v.w);
  if (to.wide) {
    *reinterpret_cast<uint2*>(out) = make_uint2(lo, hi);
  } else {
    const uint16_t e[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c + j < to.dim) reinterpret_cast<uint16_t*>(out)[j] = e[j];
  }
}

// ---- rows that start anywhere, copied to padded rows --------------------------------
struct RowsArgs {
  Side from[4];
  void* to[4];        // [tokens][heads][dim rounded up to 8]
  int32_t heads[4];
  Split split;
};
template <typename W>
__global__ void __launch_bounds__(256) attn_rows_kernel(const __grid_constant__ RowsArgs p) {
  launch_dependents();
  wait_for_previous();
  const Side& s = p.from[blockIdx.y];
  const int heads = p.heads[blockIdx.y], granules = (s.dim + 7) / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, r = i / granules, token = r / heads;
  const int c = (int)(i % granules) * 8, h = (int)(r % heads);
  if (token < offset_of(p.split, 0) || token >= offset_of(p.split, p.split.groups)) return;
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
// in one pass.  Bound by the state's bytes: 256 tokens, 16 heads of 64, bf16, 136 MB in 22.9
// us, 5.9 TB/s; one token 2.3 us, of the call's 7 to 8.
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

// Backward with shared key heads: the gradients of keys and values wait in fp32, one for each
// query head, for their sum.  That is as much as two states for each 64 tokens, so they are
// formed in ranges of tokens for which there is room.  A range's segments start in it; where
// groups start anywhere, the last ones reach beyond it by less than a segment.  (32640 tokens,
// 16 heads of 64 over 4, bf16: in one range 304 us, in two 316, in four 345; 8160 tokens: 93,
// 107 and 133; 2000 tokens, 16 over 2: 39, 58 and 85.)
size_t two_states(const gs_linear_attn* a, int64_t seg) {  // for each seg tokens, and each group's rest
  return sizeof(float) * 2 * (a->tokens / seg + a->groups) * a->q_heads * padded_dim(a->dim) * padded_dim(a->vdim);
}
// Tokens that there is room for in so many bytes.
int64_t room_for(const gs_linear_attn* a, size_t bytes) {
  const int64_t n = (int64_t)(bytes / (sizeof(float) * a->q_heads * (padded_dim(a->dim) + padded_dim(a->vdim))));
  return n < a->tokens ? n : a->tokens;
}
// Tokens of a range, a segment at least, all of about the same length (0: there is no room).
int64_t range_of(const gs_linear_attn* a, bool anywhere, int64_t seg, int64_t room) {
  if (room >= a->tokens) return a->tokens;
  const int64_t most = anywhere ? room - seg : room / seg * seg;
  if (most < seg) return 0;
  const int64_t even = div_up(a->tokens, div_up(a->tokens, most));
  return anywhere ? even : div_up(even, seg) * seg;
}
// The bytes that states and ranges should do with: two states of the wider head for each 64
// tokens and each group, and two more.
size_t modest(const gs_linear_attn* a) {
  gs_linear_attn square = *a;
  square.dim = square.vdim = a->dim > a->vdim ? a->dim : a->vdim;
  square.groups = a->groups + 1;
  return two_states(&square, 64);
}
// How many ranges that makes.
int64_t modest_ranges(const gs_linear_attn* a, int64_t seg) {
  const size_t all = modest(a), states = two_states(a, seg);
  const int64_t range = range_of(a, a->groups > 1, seg, room_for(a, all > states ? all - states : 0));
  return range ? div_up(a->tokens, range) : a->tokens ? INT64_MAX : 1;
}

// Tokens of a segment.  A chunk of the outputs or of the queries' gradients costs two units
// of time, of the states' sums one, of the keys' and values' gradients four; each segment
// costs one chunk more for its start and its state.  With two blocks an SM, blocks of one
// kind run in waves; of several kinds about as long as their work takes and half of the
// longest.  The sums' and the scan's start costs six; where a group is one segment and its
// last state is not wanted, there are neither.  The groups' lengths are on the device: they
// are taken as equal, and a lone segment as long as two of them.  (Backward, 32640 tokens, 16
// heads of 64: segments of 7 chunks, as chosen, 231 us, of 15 232; 8160 tokens, 16 and 4
// heads of 64: of 4, as chosen, 94, of 2 104, of 7 111.)
int32_t segment_tokens(const gs_linear_attn* a, bool backward, bool states) {
  const int64_t chunks = div_up(div_up(a->tokens, a->groups), kL);
  const int64_t longest = a->groups > 1 ? 2 * chunks : chunks;
  const int64_t resident = (int64_t)device_sms() * 2;
  const int64_t tiles = padded_dim(a->vdim) / kV, key_tiles = padded_dim(a->dim) / kV;
  const bool shared = backward && a->q_heads > a->k_heads;
  int best = 16;
  int64_t cost = INT64_MAX;
  for (int m = 1; m <= 16; ++m) {
    if (shared && modest_ranges(a, m * kL) > 4) continue;
    const bool alone = longest <= m;
    const int64_t n = alone ? longest : m, segments = a->groups * (alone ? 1 : div_up(chunks, m));
    const int64_t sums = segments * a->q_heads * tiles * (backward ? 2 : 1);
    int64_t c = 0;
    if (!alone || states) c += div_up(sums, resident) * (n + 1) + 6;
    if (backward) {
      const int64_t q = 2 * (n + 1), kv = 4 * (n + 1);
      const int64_t spread = div_up(segments * a->q_heads * key_tiles * (q + tiles * kv), resident) + kv / 2;
      c += spread > kv ? spread : kv;
    } else {
      c += 2 * div_up(sums, resident) * (n + 1);
    }
    if (c < cost) cost = c, best = m;
  }
  // Few tokens in groups, whose gradients would take several ranges, are a segment a group: no
  // sums, no scan, one range.  (262 tokens in 2 groups, 32 heads of 32 over 8: 31 us, in segments
  // of a chunk 70, or 45 with more room; 700 tokens, 8 heads of 64 over 4: 41, 64 and 44; launched and
  // waited for.)
  if (shared && a->groups > 1 && a->tokens <= 6 * kL && modest_ranges(a, best * kL) > 1) best = (int)div_up(a->tokens, kL);
  return best * kL;
}

struct Room {
  float *states, *grads, *whole[2];
  void* rows[4];
  size_t bytes;
  // copied: the inputs (q, k, v, dout) whose rows have to be copied, a bit each; joined: tokens
  // whose gradients of keys and values wait for their sum over the query heads
  Room(void* ws, const gs_linear_attn* a, int64_t slots, bool backward, int copied, int64_t joined) {
    char* base = (char*)ws;
    size_t at = 0;
    auto take = [&](size_t n) {
      char* p = base + at;
      at += (n + 255) / 256 * 256;
      return (float*)p;
    };
    const size_t d = padded_dim(a->dim), e = padded_dim(a->vdim);
    const size_t one = sizeof(float) * slots * a->q_heads * d * e;
    const size_t heads = sizeof(float) * joined * a->q_heads;
    states = take(one);
    grads = take(backward ? one : 0);
    whole[0] = take(heads * d);
    whole[1] = take(heads * e);
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

// No two elements of the heads in one place.
bool apart(const gs_linear_attn* a, int64_t token, int64_t head, int32_t heads, int32_t dim) {
  const int64_t t = token < 0 ? -token : token, e = head < 0 ? -head : head;
  const bool many = a->tokens > 1;
  if ((heads > 1 && e < dim) || (many && t < dim)) return false;
  return heads < 2 || !many || t >= e * (heads - 1) + dim || e >= t * (a->tokens - 1) + dim;
}
bool side(Side* s, const gs_linear_attn* a, const gs_attn_heads* h, int32_t dim, bool of_key, bool output) {
  if (!h->p || !aligned_to(h->p, 2)) return false;
  constexpr int64_t kMost = (int64_t)1 << 40;
  if (h->token >= kMost || h->token <= -kMost || h->head >= kMost || h->head <= -kMost) return false;
  const int32_t heads = of_key ? a->k_heads : a->q_heads;
  if (output && !apart(a, h->token, h->head, heads, dim)) return false;
  *s = Side{h->p, h->token, h->head, dim, of_key ? 1 : 0,
            dim % 8 == 0 && aligned16(h->p) && (a->tokens < 2 || h->token % 8 == 0) && (heads < 2 || h->head % 8 == 0)
                ? 1 : 0};
  return true;
}

// Outputs at an input's address, or at one another's: other blocks would still read there.
bool in_place(const Side* s, int inputs, int all) {
  for (int o = inputs; o < all; ++o)
    for (int i = 0; i < o; ++i)
      if (s[i].p == s[o].p) return true;
  return false;
}
// A single token's output at an input's address is its block's own, if both have the same
// heads: read before it is written.
bool own_place(const gs_linear_attn* a, const Side& in, const Side& out) {
  if (in.p != out.p) return true;
  return (!in.of_key || a->q_heads == a->k_heads) && (a->tokens < 2 || in.token == out.token) &&
         (a->q_heads < 2 || in.head == out.head) &&
         apart(a, in.token, in.head, a->q_heads, in.dim > out.dim ? in.dim : out.dim);
}

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
gs_status copy_rows(const gs_linear_attn* a, const Split& split, Side* s, int n, const Room& room, cudaStream_t st) {
  RowsArgs p{};
  p.split = split;
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
gs_status run_parts_of(const PartsArgs& p, int64_t slots, int parts, cudaStream_t st) {
  constexpr int kTerms = std::is_same<T, __half>::value ? 2 : 3;
  static std::atomic<uint64_t> known{0};
  if (!allow_smem(attn_parts_kernel<T, KD, kTerms>, known, kPartsSmem<KD, kTerms>)) {
    (void)cudaGetLastError();
    return GS_ERR_CUDA;
  }
  GS_CUDA(launch_overlapped(attn_parts_kernel<T, KD, kTerms>, dim3((unsigned)slots, p.heads, parts * (p.Ep / kV)),
                            dim3(kThreads), kPartsSmem<KD, kTerms>, st, p));
  return GS_OK;
}
// A thread has one element while those are fewer than the threads that the machine holds:
// the loads' latency counts, and 40 of them under way hide it (one group, 19 segments of 16
// heads of 64: 6 us, with 16 loads 9, with 8 13; with four elements a thread 29).  With
// more elements the instructions count, and a thread has four (4 groups, 5 segments each, 8
// heads of 128: 11 us, with one 16).
gs_status run_scan(const ScanArgs& p, cudaStream_t st) {
  const bool vec = (int64_t)p.split.groups * p.heads * p.D * p.E * p.scans > (int64_t)device_sms() * 2048;
  const int64_t blocks = p.split.groups * div_up(p.D * div_up(p.E, vec ? 4 : 1), kScanThreads);
  if (blocks > INT32_MAX) return GS_ERR_INVALID_ARG;
  const dim3 grid((unsigned)blocks, p.heads, p.scans);
  GS_CUDA(vec ? launch_overlapped(attn_scan_kernel<4, 8>, grid, dim3(kScanThreads), 0, st, p)
              : launch_overlapped(attn_scan_kernel<1, 40>, grid, dim3(kScanThreads), 0, st, p));
  return GS_OK;
}

template <typename T, int KD>
gs_status run_out_of(const OutArgs& p, int64_t slots, cudaStream_t st) {
  static std::atomic<uint64_t> known{0};
  if (!allow_smem(attn_out_kernel<T, KD>, known, kOutSmem<KD>)) {
    (void)cudaGetLastError();
    return GS_ERR_CUDA;
  }
  GS_CUDA(launch_overlapped(attn_out_kernel<T, KD>, dim3((unsigned)slots, p.heads, p.Vp / kV), dim3(kThreads),
                            kOutSmem<KD>, st, p));
  return GS_OK;
}
template <typename T, int ED, int EE, bool SHARED>
gs_status run_grad_of(const GradArgs& p, int64_t blocks, cudaStream_t st) {
  static std::atomic<uint64_t> known{0};
  if (!allow_smem(attn_grad_kernel<T, ED, EE, SHARED>, known, kGradSmem<ED, EE>)) {
    (void)cudaGetLastError();
    return GS_ERR_CUDA;
  }
  GS_CUDA(launch_overlapped(attn_grad_kernel<T, ED, EE, SHARED>, dim3((unsigned)blocks), dim3(kThreads), kGradSmem<ED, EE>, st,
                            p));
  return GS_OK;
}

struct Call {
  Split split;
  int64_t slots;
  int Dp, Ep, rep;
  // chunks: of a segment; 0: as many as is best
  Call(const gs_linear_attn* a, bool backward, bool states, int32_t chunks = 0, Limits limits = {UINT32_MAX, kWaitNs}) {
    split = Split{a->tokens, a->group_offsets, a->groups, chunks ? chunks * kL : segment_tokens(a, backward, states), 0,
                  a->tokens, limits};
    slots = a->tokens / split.seg + a->groups;
    Dp = padded_dim(a->dim);
    Ep = padded_dim(a->vdim);
    rep = a->q_heads / a->k_heads;
  }
};

template <typename T, bool SHARED>
gs_status run_grad_of(const GradArgs& p, const Call& c, int64_t blocks, cudaStream_t st) {
  if (c.Dp == 64)
    return c.Ep == 64 ? run_grad_of<T, 64, 64, SHARED>(p, blocks, st) : run_grad_of<T, 64, 128, SHARED>(p, blocks, st);
  return c.Ep == 64 ? run_grad_of<T, 128, 64, SHARED>(p, blocks, st) : run_grad_of<T, 128, 128, SHARED>(p, blocks, st);
}

// The states at the segments' starts (and, with two parts, the gradients at their ends).
template <typename T>
gs_status states_of(const gs_linear_attn* a, const Call& c, const Part (&part)[2], const Scan (&scan)[2], int n,
                    cudaStream_t st) {
  const PartsArgs p{c.split, a->q_heads, c.rep, c.Dp, c.Ep, a->log_decay, {part[0], part[1]}};
  const gs_status r = c.Dp == 64 ? run_parts_of<T, 64>(p, c.slots, n, st) : run_parts_of<T, 128>(p, c.slots, n, st);
  if (r != GS_OK) return r;
  return run_scan(ScanArgs{c.split, a->q_heads, a->dim, a->vdim, c.Dp, c.Ep, a->log_decay, {scan[0], scan[1]}, n}, st);
}

template <typename T>
gs_status forward(const gs_linear_attn* a, const Call& c, Side (&s)[4], float* state_out, const Room& room,
                  cudaStream_t st) {
  const bool scan = a->tokens > c.split.seg || state_out;
  const gs_status copied = copy_rows(a, c.split, s, 3, room, st);
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
  return c.Dp == 64 ? run_out_of<T, 64>(o, c.slots, st) : run_out_of<T, 128>(o, c.slots, st);
}

template <typename T>
gs_status backward(const gs_linear_attn* a, const Call& c, Side (&s)[7], const float* dstate_out,
                   float* dstate, const Room& room, int64_t range, cudaStream_t st) {
  // the largest launches
  const bool small = c.Dp == 64 && c.Ep == 64;
  auto slots_of = [&](int64_t from, int64_t upto) { return (upto - 1) / c.split.seg + a->groups - from / c.split.seg; };
  const int64_t kinds = (small ? 1 : c.Dp / kV + c.Ep / kV) + c.Dp / kV;
  const int64_t fours = a->k_heads * div_up(a->dim > a->vdim ? a->dim : a->vdim, 4);
  if (slots_of(0, a->tokens) * a->q_heads * kinds > INT32_MAX || div_up((range + c.split.seg) * fours, 256) > INT32_MAX)
    return GS_ERR_INVALID_ARG;
  const gs_status copied = copy_rows(a, c.split, s, 4, room, st);
  if (copied != GS_OK) return copied;
  const Side &q = s[0], &k = s[1], &v = s[2], &g = s[3];
  const bool scan = a->tokens > c.split.seg || dstate;
  if (scan) {
    const gs_status r =
        states_of<T>(a, c, {Part{k, v, 1.f, 0, 0, 0, room.states}, Part{q, g, a->scale, 1, 1, dstate != nullptr, room.grads}},
                     {Scan{a->state, nullptr, room.states, 0}, Scan{dstate_out, dstate, room.grads, 1}}, 2, st);
    if (r != GS_OK) return r;
  }
  for (int64_t from = 0; from < a->tokens; from += range) {
    OutArgs o{};
    o.split = c.split;
    o.split.from = from;
    o.split.upto = from + range < a->tokens ? from + range : a->tokens;
    o.heads = a->q_heads;
    o.rep = c.rep;
    o.log_decay = a->log_decay;
    o.mul_inner = a->scale;
    OutArgs dq = o;
    dq.query = g, dq.key = v, dq.value = k, dq.out = s[4];
    dq.K = a->vdim, dq.V = a->dim, dq.Kp = c.Ep, dq.Vp = c.Dp;
    dq.states = scan ? room.states : nullptr;
    dq.edge = a->state;
    dq.transposed = 1;
    dq.mul_state = a->scale;
    dq.mul_key = 1.f;
    o.back = o.shift = 1;
    o.mul_state = 1.f;
    o.mul_key = a->scale;
    o.states = scan ? room.grads : nullptr;
    o.edge = dstate_out;
    OutArgs dk = o, dv = o;
    dk.query = v, dk.key = g, dk.value = q, dk.out = s[5];
    dk.K = a->vdim, dk.V = a->dim, dk.Kp = c.Ep, dk.Vp = c.Dp;
    dk.transposed = 1;
    float* const whole[2] = {c.rep > 1 ? room.whole[0] : nullptr, c.rep > 1 ? room.whole[1] : nullptr};
    dk.whole = whole[0];
    dv.query = k, dv.key = q, dv.value = g, dv.out = s[6];
    dv.K = a->dim, dv.V = a->vdim, dv.Kp = c.Dp, dv.Vp = c.Ep;
    dv.whole = whole[1];

    const int64_t slots = slots_of(from, o.split.upto), blocks_a_tile = slots * a->q_heads;
    const int64_t first = blocks_a_tile * (small ? 1 : c.Dp / kV);
    const int64_t second = first + (small ? 0 : blocks_a_tile * (c.Ep / kV));
    const GradArgs p{(int32_t)(from / c.split.seg), (int32_t)slots, a->q_heads, (int32_t)first, (int32_t)second, dq, dk, dv,
                     KvArgs{o.split, a->q_heads, c.rep, q, k, v, g, s[5], s[6], a->dim, a->vdim, a->log_decay, o.states,
                            o.edge, a->scale, {whole[0], whole[1]}}};
    const int64_t blocks = blocks_a_tile * kinds;
    const gs_status r = c.rep > 1 ? run_grad_of<T, true>(p, c, blocks, st) : run_grad_of<T, false>(p, c, blocks, st);
    if (r != GS_OK) return r;
    if (c.rep == 1) continue;
    const int64_t reach = o.split.upto + (a->group_offsets ? c.split.seg : 0);
    const int64_t joins = div_up(((reach < a->tokens ? reach : a->tokens) - from) * fours, 256);
    GS_CUDA(launch_overlapped(attn_join_kernel<T>, dim3((unsigned)joins, 2), dim3(256), 0, st,
                              JoinArgs{o.split, a->k_heads, c.rep, {whole[0], whole[1]}, {c.Dp, c.Ep}, {s[5], s[6]}}));
  }
  return GS_OK;
}

bool chunked_ok(const gs_linear_attn* a, const gs_attn_heads* heads) {
  return a && heads && shape_ok(a) && aligned_or_none(a) && (a->group_offsets || a->groups == 1);
}

gs_status forward(const gs_linear_attn* a, const Call& c, const gs_attn_heads* heads, float* state_out, void* workspace,
                  size_t ws_bytes, cudaStream_t st) {
  Side s[4] = {};
  if (a->tokens > 0 && (!side(&s[0], a, &heads[0], a->dim, false, false) || !side(&s[1], a, &heads[1], a->dim, true, false) ||
                        !side(&s[2], a, &heads[2], a->vdim, true, false) || !side(&s[3], a, &heads[3], a->vdim, false, true) ||
                        in_place(s, 3, 4)))
    return GS_ERR_INVALID_ARG;
  const Room room(workspace, a, c.slots, false, a->tokens > 0 ? to_copy(s, 3) : 0, 0);
  if (!workspace || !aligned16(workspace) || ws_bytes < room.bytes) return GS_ERR_INVALID_ARG;
  if (a->tokens == 0 && !state_out) return GS_OK;
  if (a->tokens == 0) {
    return run_scan(ScanArgs{c.split, a->q_heads, a->dim, a->vdim, c.Dp, c.Ep, a->log_decay,
                             {Scan{a->state, state_out, room.states, 0}, Scan{}}, 1}, st);
  }
  return a->dtype == GS_BF16 ? forward<__nv_bfloat16>(a, c, s, state_out, room, st)
                             : forward<__half>(a, c, s, state_out, room, st);
}

gs_status backward(const gs_linear_attn* a, const Call& c, const gs_attn_heads* heads, const float* dstate_out,
                   float* dstate, void* workspace, size_t ws_bytes, cudaStream_t st) {
  Side s[7] = {};
  if (a->tokens > 0 &&
      (!side(&s[0], a, &heads[0], a->dim, false, false) || !side(&s[1], a, &heads[1], a->dim, true, false) ||
       !side(&s[2], a, &heads[2], a->vdim, true, false) || !side(&s[3], a, &heads[3], a->vdim, false, false) ||
       !side(&s[4], a, &heads[4], a->dim, false, true) || !side(&s[5], a, &heads[5], a->dim, true, true) ||
       !side(&s[6], a, &heads[6], a->vdim, true, true) || in_place(s, 4, 7)))
    return GS_ERR_INVALID_ARG;
  const int copied = a->tokens > 0 ? to_copy(s, 4) : 0;
  const size_t others = Room(nullptr, a, c.slots, true, copied, 0).bytes;
  const int64_t joined = c.rep > 1 ? room_for(a, ws_bytes > others ? ws_bytes - others : 0) : 0;
  const int64_t range = c.rep > 1 ? range_of(a, a->group_offsets != nullptr, c.split.seg, joined) : a->tokens;
  const Room room(workspace, a, c.slots, true, copied, joined);
  if (!workspace || !aligned16(workspace) || ws_bytes < room.bytes || (a->tokens > 0 && range == 0)) return GS_ERR_INVALID_ARG;
  if (a->tokens == 0 && !dstate) return GS_OK;
  if (a->tokens == 0) {
    return run_scan(ScanArgs{c.split, a->q_heads, a->dim, a->vdim, c.Dp, c.Ep, a->log_decay,
                             {Scan{dstate_out, dstate, room.grads, 1}, Scan{}}, 1}, st);
  }
  return a->dtype == GS_BF16 ? backward<__nv_bfloat16>(a, c, s, dstate_out, dstate, room, range, st)
                             : backward<__half>(a, c, s, dstate_out, dstate, room, range, st);
}

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" size_t gs_linear_attn_workspace_bytes(const gs_linear_attn* a, int32_t backward) {
  if (!a || !shape_ok(a)) return 0;
  size_t most = 0;
  for (int states = 0; states < 2; ++states) {
    const Call c(a, backward != 0, states != 0);
    size_t n = Room(nullptr, a, c.slots, backward != 0, backward ? 15 : 7, 0).bytes;
    if (backward && c.rep > 1) {
      // as few ranges as a modest room allows, four at most, and one of up to 4096 tokens
      const int64_t left = room_for(a, modest(a) > n ? modest(a) - n : 0);
      const int64_t quarter = div_up(a->tokens, 4) + 2 * c.split.seg, least = quarter > 4096 ? quarter : 4096;
      const int64_t joined = left > least ? left : least;
      n = Room(nullptr, a, c.slots, true, 15, joined < a->tokens ? joined : a->tokens).bytes;
    }
    if (n > most) most = n;
  }
  return most;
}

extern "C" gs_status gs_linear_attn_fwd(const gs_linear_attn* a, const gs_attn_heads* heads, float* state_out,
                                        void* workspace, size_t ws_bytes, void* stream) {
  if (!chunked_ok(a, heads)) return GS_ERR_INVALID_ARG;
  return forward(a, Call(a, false, state_out != nullptr), heads, state_out, workspace, ws_bytes, (cudaStream_t)stream);
}

extern "C" gs_status gs_linear_attn_bwd(const gs_linear_attn* a, const gs_attn_heads* heads,
                                        const float* dstate_out, float* dstate, void* workspace, size_t ws_bytes,
                                        void* stream) {
  if (!chunked_ok(a, heads)) return GS_ERR_INVALID_ARG;
  return backward(a, Call(a, true, dstate != nullptr), heads, dstate_out, dstate, workspace, ws_bytes,
                  (cudaStream_t)stream);
}

extern "C" int32_t gs_selftest_linear_attn_chunks(const gs_linear_attn* a, int32_t backward, int32_t states) {
  return a && shape_ok(a) ? Call(a, backward != 0, states != 0).split.seg / kL : 0;
}

extern "C" gs_status gs_selftest_linear_attn(const gs_linear_attn* a, const gs_attn_heads* heads, int32_t backward_pass,
                                             const float* dstate_out, float* state_out, void* workspace, size_t ws_bytes,
                                             int32_t chunks, int32_t products, void* stream) {
  if (!chunked_ok(a, heads) || chunks < 0 || chunks > 16) return GS_ERR_INVALID_ARG;
  const Limits limits = products < 0 ? Limits{UINT32_MAX, kWaitNs} : Limits{(uint32_t)products, 20000000};
  const Call c(a, backward_pass != 0, state_out != nullptr, chunks, limits);
  const gs_status s = backward_pass ? backward(a, c, heads, dstate_out, state_out, workspace, ws_bytes, (cudaStream_t)stream)
                                    : forward(a, c, heads, state_out, workspace, ws_bytes, (cudaStream_t)stream);
  return s != GS_OK ? s : gs_linear_attn_status(stream);
}

extern "C" gs_status gs_linear_attn_status(void* stream) {
  unsigned int found = 0;
  const unsigned int none = 0;
  cudaStream_t st = (cudaStream_t)stream;
  GS_CUDA(cudaMemcpyFromSymbolAsync(&found, attn_timeouts, sizeof(found), 0, cudaMemcpyDeviceToHost, st));
  GS_CUDA(cudaStreamSynchronize(st));
  if (!found) return GS_OK;
  GS_CUDA(cudaMemcpyToSymbolAsync(attn_timeouts, &none, sizeof(none), 0, cudaMemcpyHostToDevice, st));
  GS_CUDA(cudaStreamSynchronize(st));
  return GS_ERR_TIMEOUT;
}

extern "C" gs_status gs_linear_attn_step(const gs_linear_attn* a, const gs_attn_heads* heads, float* state,
                                         void* stream) {
  if (!a || !heads || !shape_ok(a) || !aligned_or_none(a)) return GS_ERR_INVALID_ARG;
  if (a->tokens == 0) return GS_OK;
  StepArgs p{};
  if (!state || !aligned_to(state, 4) || !side(&p.q, a, &heads[0], a->dim, false, false) ||
      !side(&p.k, a, &heads[1], a->dim, true, false) || !side(&p.v, a, &heads[2], a->vdim, true, false) ||
      !side(&p.out, a, &heads[3], a->vdim, false, true) || !own_place(a, p.q, p.out) || !own_place(a, p.k, p.out) ||
      !own_place(a, p.v, p.out))
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
