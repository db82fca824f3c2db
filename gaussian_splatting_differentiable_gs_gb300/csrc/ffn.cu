// ffn.cu -- gs_ffn_fwd, gs_ffn_bwd: the gated feed-forward block's two projections,
// activation and product in one kernel, and its backward pass from the input alone.
//
//   [gate | up] = x W^T,  h = act(gate) * up,  W = [Wg; Wu]  (2 hidden x channels)
//   dgate = dh up act'(gate), dup = dh act(gate)
//   dx = dgate Wg + dup Wu,  dW = [dgate | dup]^T x
//
// Four products on one tensor-core kernel, which differ in how their operands lie and in
// what is done with a finished tile:
//   forward    tokens x 128 hidden channels, gate and up side by side: the first CTA of a
//              pair brings the tile's rows of Wg, the second those of Wu, so that every
//              TMEM lane (a token) holds both and h is formed on the way out.  Neither
//              gate nor up is ever in memory.
//   recompute  the same product again in the backward pass; on the way out dgate and dup
//              are formed from dh, rounded to the inputs' type (they are operands of the
//              next two products, and as far off there as any 16-bit gradient) and put
//              into the workspace.  Nothing but x is kept between the two directions.
//   dx         [dgate | dup] times W, W as it lies (its channels contiguous: "MN-major")
//   dW         x^T times [dgate | dup] over the tokens, both as they lie
//
// A pair of CTAs (cluster of two, tcgen05 cta_group::2) works on 256 x 256 results: each
// CTA holds 128 rows of the first operand and half of the second's columns in six stages
// of 64 steps (TMA, 128-byte swizzle), and 128 x 256 fp32 sums in TMEM, twice, so that
// eight warps write one tile while the next one's products run.  Sums are fp32; the
// tensor core cuts, not rounds, its sum at every product, so that a sum's error grows with
// its length.  dW, whose sums are as long as there are tokens and which may be asked for in
// fp32, is therefore summed in runs of 32 steps, added up in registers with rounding: 32640
// tokens are off by 2.1e-6 of the result's norm, 2.6e-6 where all terms are positive; in one
// run 3.7e-5 and 1.7e-4, in the same time.  (The other sums are as long as there are
// channels or hidden ones, and their results have 16 bits.)
//
// Rows that do not start on 16-byte boundaries (TMA's rule) are first copied to padded
// rows in the workspace.
#include <type_traits>

#include "activation.cuh"
#include "tensor_core.cuh"

namespace gs {
namespace {

constexpr int kTile = 256;                 // rows and columns of a pair's tile
constexpr int kHalf = 128;                 // a CTA's rows, and its columns of the second operand
constexpr int kStep = 64;                  // terms of the sums per stage
constexpr int kOperand = kHalf * kStep * 2;  // bytes of a CTA's half of an operand
constexpr int kStage = 2 * kOperand;
constexpr int kStages = 6;
constexpr int kSums = 2;                   // sums in TMEM: 2 x 256 columns
template <int MODE>
constexpr int kRun = MODE == 3 ? 32 : 0;   // steps of a run that the tensor core sums alone; 0: all of a tile
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr int kRowsOut = 32 * 128;         // a warp's room for 32 rows of 128 bytes
constexpr int kCtrlBytes = 1024;
constexpr int kSmem = kStages * kStage + kEpiWarps * kRowsOut + kCtrlBytes + 1024;  // + alignment
static_assert(kSmem <= 227 * 1024, "shared memory");
constexpr int kMaxClusters = 96;
constexpr size_t kPartialFloats = (size_t)kHalf * kTile;  // one CTA's half tile
constexpr unsigned int kErrTimeout = 1u;
constexpr int64_t kWaitNs = 2000000000;

enum { kFwd, kRecompute, kDx, kDw };

struct Job {
  int64_t rows, cols;          // valid rows and columns of the result
  int32_t tiles_n;             // tiles side by side; the tiles of a row of tiles follow each other
  int32_t steps, part_steps;   // of a tile; of the first of the two parts of the sum (kDx)
  int32_t clusters, waves;     // whole tiles per cluster
  int64_t rem_steps, quota;    // the remaining tiles' steps, and a cluster's share of them
  void* out;                   // result [rows][out_stride]; kDw: [column][out_stride], row contiguous
  int64_t out_stride;
  int32_t out_wide;            // rows of out start on 16-byte boundaries
  const void* dh;              // kRecompute
  int64_t dh_stride;           // (rows on 16-byte boundaries)
  int32_t hidden, hidden_ld;   // hidden, padded: columns of dgate in the workspace
  int32_t accumulate;
  uint32_t load_steps;  // steps whose operands are brought: all, but in the self-test
  int64_t wait_ns;      // after which a wait gives up
};

// A cluster's steps one by one: its whole tiles, then its share of the remaining tiles'
// steps, RUN steps (0: all of a tile) a sum.
template <int RUN>
struct Walk {
  const Job& p;
  int cluster, wave = 0;
  int64_t at, stop;
  int tile = 0, step = -1, left = 0, in_run = 0;
  int slot = -1;  // place of the partial sum of a tile that several clusters share, or -1
  bool begins = false;  // a sum
  __device__ __forceinline__ Walk(const Job& job, int cl) : p(job), cluster(cl) {
    at = (int64_t)cl * p.quota;
    stop = min(at + p.quota, p.rem_steps);
  }
  __device__ __forceinline__ bool next() {
    begins = false;
    if (--left >= 0) {
      ++step;
      if (RUN && ++in_run == RUN) in_run = 0, begins = true;
      return true;
    }
    return segment();
  }
  __device__ __forceinline__ bool ends() const { return left == 0 || (RUN && in_run == RUN - 1); }
  // Of the segment that has just begun.
  __device__ __forceinline__ int runs() const { return RUN ? left / (RUN ? RUN : 1) + 1 : 1; }
  // The next segment: the steps of one tile that this cluster sums.
  __device__ __forceinline__ bool segment() {
    begins = true;
    in_run = 0;
    if (wave < p.waves) {
      slot = -1;
      tile = wave++ * p.clusters + cluster;
      step = 0;
      left = p.steps - 1;
      return true;
    }
    if (at >= stop) return false;
    const int i = (int)(at / p.steps);
    const int64_t upto = min(stop, (int64_t)(i + 1) * p.steps);
    const int n = (int)(upto - at);
    slot = n == p.steps ? -1 : at == (int64_t)cluster * p.quota ? 0 : 1;
    tile = p.waves * p.clusters + i;
    step = (int)(at - (int64_t)i * p.steps);
    left = n - 1;
    at = upto;
    return true;
  }
};

struct Control {
  uint64_t full[kStages], empty[kStages];        // operands of both CTAs (full: the first's)
  uint64_t sum_full[kSums], sum_empty[kSums];    // (sum_empty: the first's)
  uint32_t tmem;
  uint32_t loads, products, sums;   // when a role ends: what it asked for
  volatile uint32_t abort;          // a wait of the pair gave up
};
static_assert(sizeof(Control) <= kCtrlBytes, "control");

// Waits for a barrier's phase, at most p.wait_ns; false (and the status word set) when
// that ran out or another wait of the pair gave up.
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, Control* c, const Job& p,
                                          unsigned int* status) {
  const int64_t t0 = now_ns();
  while (true) {
    if (mbar_try(bar, parity)) return true;
    if (c->abort) return false;
    if (now_ns() - t0 > p.wait_ns) {
      store_pair(&c->abort, 0, 1);
      store_pair(&c->abort, 1, 1);
      atomicOr(status, kErrTimeout);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, Control* c, const Job& p,
                                     unsigned int* status) {
  if (mbar_try(bar, parity)) return true;
  return wait_slow(bar, parity, c, p, status);
}

// After giving up: one thread of each CTA waits, at most p.wait_ns in all, until nothing
// of the pair is under way that writes shared memory or TMEM: copies, products, and the
// arrivals at their end.  Every role of both CTAs has ended, so what was asked for is known.
__device__ __forceinline__ void drain(Control* c, const Job& p, uint32_t rank) {
  const int64_t until = now_ns() + p.wait_ns;
  auto last = [&](uint64_t* ring, uint32_t places, uint32_t n) {  // the phases that the last n ended
    for (uint32_t i = n < places ? 0 : n - places; i < n; ++i)
      while (!mbar_try(smem_u32(&ring[i % places]), i / places & 1) && now_ns() < until) {}
  };
  last(c->empty, kStages, load_pair(&c->products, 0));
  last(c->sum_full, kSums, load_pair(&c->sums, 0));
  if (rank) return;
  // Both CTAs' copies end at the first one's barriers; where only one of the two asked for
  // its half of a step, the other half is made up for.
  const uint32_t own = c->loads, other = load_pair(&c->loads, 1), steps = max(own, other);
  for (uint32_t i = steps < kStages ? 0 : steps - kStages; i < steps; ++i) {
    const uint32_t bar = smem_u32(&c->full[i % kStages]);
    if (i >= own) mbar_expect(bar, kStage);
    if (i >= other)
      asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(in_cta0(bar)),
                   "r"((uint32_t)kStage)
                   : "memory");
  }
  last(c->full, kStages, steps);
}

__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// Shared-memory descriptors of operands in 128-byte swizzled rows.  K-major: a row is 64
// terms of the sum, eight rows an atom of 1024 bytes; 16 terms on are 32 bytes.  MN-major:
// a row is 64 rows (columns) of the result at one term, eight terms an atom, the next 64
// rows follow after kStep terms; 16 terms on are two atoms.
template <bool MN>
__device__ __forceinline__ uint64_t operand(uint32_t addr) {
  constexpr uint64_t kLead = MN ? (uint64_t)(kStep * 128 >> 4) : 1, kAtom = (uint64_t)(1024 >> 4);
  return (uint64_t)((addr & 0x3ffff) >> 4) | (kLead << 16) | (kAtom << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)2 << 61);
}
template <bool MN>
constexpr uint64_t kNext16 = MN ? 2048 >> 4 : 32 >> 4;

// Instruction descriptor: fp32 sums, 16-bit operands, 256 x 256.
template <typename T, bool A_MN, bool B_MN>
constexpr uint32_t instruction() {
  constexpr uint32_t type = sizeof(T) == 2 && !std::is_same<T, __half>::value ? 1u : 0u;
  return (1u << 4) | (type << 7) | (type << 10) | ((A_MN ? 1u : 0u) << 15) |
         ((B_MN ? 1u : 0u) << 16) | ((uint32_t)(kTile >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b),
      "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// 32 columns of the warp's lanes; the values are there after tmem_wait.
__device__ __forceinline__ void tmem_load32(uint32_t addr, float (&f)[32]) {
  uint32_t(&v)[32] = reinterpret_cast<uint32_t(&)[32]>(f);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]),
        "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]),
        "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t addr, float (&f)[16]) {
  uint32_t(&v)[16] = reinterpret_cast<uint32_t(&)[16]>(f);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(addr)
      : "memory");
}
// Ties the loaded values to the wait, so that no use of them moves before it.
template <int N>
__device__ __forceinline__ void tmem_wait(float (&f)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(f[i]));
}

// ---- 32 rows of 64 16-bit elements between a warp's room in shared memory and rows of a
// matrix.  Granule g (16 bytes) of row r lies at r * 128 + ((g ^ r % 8) * 16), so that
// neither a thread with a row of its own nor eight threads of a row meet in a bank.
__device__ __forceinline__ uint32_t granule_at(int r, int g) { return r * 128 + ((g ^ (r & 7)) << 4); }

template <typename T>
__device__ __forceinline__ void rows_out(const uint8_t* room, T* to, int64_t stride, int rows, int cols,
                                         bool wide, int lane) {
  if (wide) {
    const int g = lane & 7;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = i * 4 + (lane >> 3);
      if (r >= rows || g * 8 >= cols) continue;
      const uint4 v = *reinterpret_cast<const uint4*>(room + granule_at(r, g));
      T* p = to + r * stride + g * 8;
      if (g * 8 + 8 <= cols) {
        *reinterpret_cast<uint4*>(p) = v;
      } else {
        const Pack<T, 8> e = *reinterpret_cast<const Pack<T, 8>*>(&v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (g * 8 + j < cols) p[j] = e.v[j];
      }
    }
  } else {
    for (int r = 0; r < rows; ++r)
#pragma unroll
      for (int c = lane; c < 64; c += 32)
        if (c < cols) to[r * stride + c] = *reinterpret_cast<const T*>(room + granule_at(r, c >> 3) + (c & 7) * 2);
  }
}
// Rows on 16-byte boundaries; zeros where the matrix has nothing (from granules that
// hold any of it).
template <typename T>
__device__ __forceinline__ void rows_in(uint8_t* room, const T* from, int64_t stride, int rows, int cols, int lane) {
  const int g = lane & 7;
  uint4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = i * 4 + (lane >> 3);
    v[i] = make_uint4(0, 0, 0, 0);
    if (r >= rows || g * 8 >= cols) continue;
    const T* p = from + r * stride + g * 8;
    if (g * 8 + 8 <= cols) {
      v[i] = *reinterpret_cast<const uint4*>(p);
    } else {
      Pack<T, 8> e;
#pragma unroll
      for (int j = 0; j < 8; ++j) e.v[j] = g * 8 + j < cols ? p[j] : from_f32<T>(0.f);
      v[i] = *reinterpret_cast<const uint4*>(&e);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    *reinterpret_cast<uint4*>(room + granule_at(i * 4 + (lane >> 3), g)) = v[i];
}
// Words 16 c .. 16 c + 15 (32 elements) of the thread's own row.
__device__ __forceinline__ void own_row_put(uint8_t* room, int lane, int c, const uint32_t* w) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint4*>(room + granule_at(lane, 4 * c + i)) =
        make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}
__device__ __forceinline__ void own_row_get(const uint8_t* room, int lane, int c, uint32_t* w) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 v = *reinterpret_cast<const uint4*>(room + granule_at(lane, 4 * c + i));
    w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
  }
}
template <typename T>
__device__ __forceinline__ float2 two_of(uint32_t w) {
  const Pack<T, 2> e = *reinterpret_cast<const Pack<T, 2>*>(&w);
  return make_float2(to_f32(e.v[0]), to_f32(e.v[1]));
}

// mma.sync, 16 x 8 x 16.
template <typename T>
__device__ __forceinline__ void mma_rows(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <typename TO>
__device__ __forceinline__ void put_dw(TO* p, float v, int accumulate) {
  *p = from_f32<TO>(accumulate ? v + to_f32(*p) : v);
}
// Row of dw that column n of [dgate | dup] belongs to, or -1 (padding).
__device__ __forceinline__ int64_t dw_row(const Job& p, int64_t n) {
  const int64_t part = n >= p.hidden_ld ? 1 : 0, f = n - part * p.hidden_ld;
  return f < p.hidden ? part * p.hidden + f : -1;
}

// MODE: see above.  TO: the type of dw (else T).
//
// Bound by the tensor cores, and in long loops by the power that they may take.  32640 tokens
// x 1024 channels x 2816 hidden, bf16, 188.3 GFLOP each: forward 195 us (tensor cores 96 % of
// the cycles; 220 in long loops), dx 208 (95 %; 416 MB read), dW 212 (93 %; 653 MB read),
// recompute 240 (81 %: its tiles' way out, dh in and dgate and dup out by way of shared
// memory, takes longer than the next tile's products).  5003 x 997 x 1361, fp16: 34, 30 and 28 us, half of them
// start, end and the shares of 80 tiles among 76 pairs.
template <typename T, typename TO, int MODE, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ffn_kernel(const __grid_constant__ Job p, const __grid_constant__ CUtensorMap a_map,
               const __grid_constant__ CUtensorMap b_map, float* partial, unsigned int* status) {
  constexpr bool kAMn = MODE == kDw, kBMn = MODE == kDw || MODE == kDx;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
  uint8_t* rooms = smem + kStages * kStage;
  Control* c = (Control*)(rooms + kEpiWarps * kRowsOut);
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int cluster = blockIdx.x >> 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&c->full[i]), 1);
      mbar_init(smem_u32(&c->empty[i]), 1);
    }
    for (int i = 0; i < kSums; ++i) {
      mbar_init(smem_u32(&c->sum_full[i]), 1);
      mbar_init(smem_u32(&c->sum_empty[i]), 2 * kEpiWarps);
    }
    c->loads = c->products = c->sums = 0;
    c->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(&c->tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = c->tmem;
  launch_dependents();
  wait_for_previous();

  if (warp == 0) {
    // ---- operands by TMA: this CTA's rows of the first, its half of the second ----
    const bool issues = elect_one();
    const uint32_t bars = in_cta0(smem_u32(&c->full[0]));
    Walk<kRun<MODE>> w(p, cluster);
    uint32_t st = 0, phase = 0, it = 0;
    int m = 0, n = 0;
    while (it < p.load_steps && w.next()) {
      if (w.begins) {
        m = w.tile / p.tiles_n * kTile + (int)rank * kHalf;
        n = w.tile % p.tiles_n * (MODE == kFwd || MODE == kRecompute ? kHalf : kTile);
      }
      if (!wait(smem_u32(&c->empty[st]), phase ^ 1, c, p, status)) break;
      if (issues) {
        if (rank == 0) mbar_expect(smem_u32(&c->full[st]), 2 * kStage);
        const uint32_t a = smem_u32(smem) + st * kStage, b = a + kOperand, bar = bars + st * 8;
        if (MODE == kFwd || MODE == kRecompute) {
          tma_load(a, &a_map, w.step * kStep, m, bar);
          tma_load3(b, &b_map, w.step * kStep, n, (int)rank, bar);
        } else if (MODE == kDx) {
          const int part = w.step >= p.part_steps, k = (w.step - part * p.part_steps) * kStep;
          const int col = n + (int)rank * kHalf;
          tma_load3(a, &a_map, k, m, part, bar);
          tma_load3(b, &b_map, col, k, part, bar);
          tma_load3(b + kOperand / 2, &b_map, col + 64, k, part, bar);
        } else {
          const int col = n + (int)rank * kHalf, t = w.step * kStep;
          tma_load(a, &a_map, m, t, bar);
          tma_load(a + kOperand / 2, &a_map, m + 64, t, bar);
          tma_load(b, &b_map, col, t, bar);
          tma_load(b + kOperand / 2, &b_map, col + 64, t, bar);
        }
      }
      ++it;
      if (++st == kStages) st = 0, phase ^= 1;
    }
    if (issues) c->loads = it;
    // the last products release the last stages: every arrival is in before this CTA ends
    for (uint32_t i = it < kStages ? 0 : it - kStages; i < it; ++i)
      if (!wait(smem_u32(&c->empty[i % kStages]), (i / kStages) & 1, c, p, status)) break;
  } else if (warp == 1) {
    // ---- products: the whole warp walks the steps, so that what it computes stays in
    // uniform registers; one elected lane issues.
    if (rank == 0) {
      constexpr uint32_t idesc = instruction<T, kAMn, kBMn>();
      const bool issues = elect_one();
      const uint64_t a_first = operand<kAMn>(smem_u32(smem));
      const uint64_t b_first = operand<kBMn>(smem_u32(smem) + kOperand);
      Walk<kRun<MODE>> w(p, cluster);
      uint32_t st = 0, phase = 0, it = 0, sums = 0;
      while (w.next()) {
        const uint32_t sum = sums % kSums;
        if (w.begins && !wait(smem_u32(&c->sum_empty[sum]), (sums / kSums & 1) ^ 1, c, p, status)) break;
        if (!wait(smem_u32(&c->full[st]), phase, c, p, status)) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if (issues) {
          const uint64_t a = a_first + st * (kStage >> 4), b = b_first + st * (kStage >> 4);
#pragma unroll
          for (int i = 0; i < kStep / 16; ++i)
            mma(tmem + sum * kTile, a + i * kNext16<kAMn>, b + i * kNext16<kBMn>, idesc,
                !w.begins || i > 0);
          mma_commit(smem_u32(&c->empty[st]));
          if (w.ends()) mma_commit(smem_u32(&c->sum_full[sum]));
        }
        ++it;
        sums += w.ends();
        if (++st == kStages) st = 0, phase ^= 1;
      }
      if (issues) c->products = it, c->sums = sums;
    }
  } else {
    // ---- finished tiles ------------------------------------------------------
    const int quarter = warp & 3;              // the TMEM lanes this warp may read
    const int half = (warp - 2) / 4;           // of the columns
    uint8_t* room = rooms + (warp - 2) * kRowsOut;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t empty = in_cta0(smem_u32(&c->sum_empty[0]));
    Walk<kRun<MODE>> w(p, cluster);
    uint32_t sums = 0, sum = 0, from = 0;
    auto next_sum = [&] {
      sum = sums % kSums;
      from = lanes + sum * kTile;
      if (!__all_sync(0xffffffffu, wait(smem_u32(&c->sum_full[sum]), sums++ / kSums & 1, c, p, status))) return false;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      return true;
    };
    auto release = [&] {  // the sum is in registers
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive_pair(empty + sum * 8);
    };
    while (w.segment()) {
      const int64_t row0 = (int64_t)(w.tile / p.tiles_n) * kTile + (int)rank * kHalf + quarter * 32;
      const int rows = (int)max((int64_t)0, min((int64_t)32, p.rows - row0));
      const int tn = w.tile % p.tiles_n;
      if (MODE == kRecompute) {
        const int col0 = tn * kHalf + half * 64, cols = (int)min((int64_t)64, p.cols - col0);
        rows_in<T>(room, (const T*)p.dh + row0 * p.dh_stride + col0, p.dh_stride, rows, cols, lane);
        __syncwarp();
      }
      if (!next_sum()) break;
      if (MODE == kFwd || MODE == kRecompute) {
        const int col0 = tn * kHalf + half * 64, cols = (int)min((int64_t)64, p.cols - col0);
        uint32_t dg[32];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float gate[32], up[32];
          tmem_load32(from + half * 64 + b * 32, gate);
          tmem_load32(from + kHalf + half * 64 + b * 32, up);
          tmem_wait(gate);
          tmem_wait(up);
          if (b == 1) release();
          uint32_t o[16];
          if (MODE == kFwd) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float2 f = act_value<T, ACT>(make_float2(gate[2 * j], gate[2 * j + 1]));
              o[j] = pair_word<T>(f.x * up[2 * j], f.y * up[2 * j + 1]);
            }
          } else {
            own_row_get(room, lane, b, o);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float2 f, df;
              act_both<T, ACT>(make_float2(gate[2 * j], gate[2 * j + 1]), f, df);
              const float2 d = two_of<T>(o[j]);
              dg[b * 16 + j] = pair_word<T>(d.x * up[2 * j] * df.x, d.y * up[2 * j + 1] * df.y);
              o[j] = pair_word<T>(d.x * f.x, d.y * f.y);
            }
          }
          own_row_put(room, lane, b, o);
        }
        __syncwarp();
        T* to = (T*)p.out + row0 * p.out_stride + col0;
        if (MODE == kFwd) {
          rows_out<T>(room, to, p.out_stride, rows, cols, p.out_wide, lane);
        } else {
          rows_out<T>(room, to + p.hidden_ld, p.out_stride, rows, cols, true, lane);
          __syncwarp();
          own_row_put(room, lane, 0, dg);
          own_row_put(room, lane, 1, dg + 16);
          __syncwarp();
          rows_out<T>(room, to, p.out_stride, rows, cols, true, lane);
        }
        __syncwarp();
      } else if (MODE == kDx && w.slot >= 0) {
        float* to = partial + ((size_t)(cluster * 2 + w.slot) * 2 + rank) * kPartialFloats +
                    half * kHalf * kHalf + (quarter * 32 + lane) * 4;
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
          float v[32];
          tmem_load32(from + half * kHalf + b * 32, v);
          tmem_wait(v);
          if (b == 3) release();
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4*>(to + (b * 32 + j) * kHalf) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
      } else if (MODE == kDx) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t col0 = (int64_t)tn * kTile + half * kHalf + h * 64;
          const int cols = (int)max((int64_t)0, min((int64_t)64, p.cols - col0));
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            float v[32];
            uint32_t o[16];
            tmem_load32(from + half * kHalf + h * 64 + b * 32, v);
            tmem_wait(v);
            if (h == 1 && b == 1) release();
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = pair_word<T>(v[2 * j], v[2 * j + 1]);
            own_row_put(room, lane, b, o);
          }
          __syncwarp();
          rows_out<T>(room, (T*)p.out + row0 * p.out_stride + col0, p.out_stride, rows, cols, p.out_wide, lane);
          __syncwarp();
        }
      } else {
        float v[kHalf];  // the sums of the runs so far
#pragma unroll
        for (int j = 0; j < kHalf; ++j) v[j] = 0.f;
        bool there = true;
        int runs = w.runs();
#pragma unroll 1
        do {
#pragma unroll
          for (int b = 0; b < kHalf / 16; ++b) {
            float u[16];
            tmem_load16(from + half * kHalf + b * 16, u);
            tmem_wait(u);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[b * 16 + j] += u[j];
          }
          release();
        } while (--runs && (there = next_sum()));
        if (!there) break;
        const int64_t ch = row0 + lane;
        if (w.slot < 0) {
#pragma unroll
          for (int b = 0; b < kHalf; b += 64) {  // (64 columns are all dgate's, or all dup's)
            const int64_t n = (int64_t)tn * kTile + half * kHalf + b, part = n >= p.hidden_ld ? 1 : 0;
            const int64_t f = n - part * p.hidden_ld;
            const int left = lane < rows ? (int)max((int64_t)0, min((int64_t)64, p.hidden - f)) : 0;
            TO* to = (TO*)p.out + (part * p.hidden + f) * p.out_stride + ch;
#pragma unroll
            for (int j = 0; j < 64; ++j, to += p.out_stride)
              if (j < left) put_dw<TO>(to, v[b + j], p.accumulate);
          }
        } else {
          float* to = partial + ((size_t)(cluster * 2 + w.slot) * 2 + rank) * kPartialFloats +
                      half * kHalf * kHalf + quarter * 32 + lane;
#pragma unroll
          for (int j = 0; j < kHalf; ++j) to[j * kHalf] = v[j];
        }
      }
    }
  }

  // Every role of both CTAs is done, or gave up: then both know.
  __syncthreads();
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  cluster_sync();
  if (c->abort) {
    if (threadIdx.x == 0) drain(c, p, rank);
    __syncthreads();
    __syncwarp();
    cluster_sync();  // neither CTA ends while the other looks at it
  }
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// Joins the partial sums of the tiles that several clusters share, in the clusters' order.
// dW's lie column by column, 128 channels each: a warp takes a column of a CTA's half tile,
// a thread four channels.  dx's lie by fours of columns, 128 rows each: a warp takes 32
// rows, a thread eight columns of one.
template <typename TO, bool DX>
__device__ __forceinline__ void join_partials(const Job& p, const float* partial, int block) {
  constexpr int kLines = DX ? kHalf : kTile, kPerHalf = kLines / 4, kPer = DX ? 8 : 4;
  const int tile = block / (2 * kPerHalf), rank = block / kPerHalf % 2;
  const int line = block % kPerHalf * 4 + (int)(threadIdx.x >> 5), lane = threadIdx.x % 32;
  // the thread's row and column of the half tile
  const int mi = DX ? line % 4 * 32 + lane : lane * 4, ni = DX ? line / 4 * 8 : line;
  const int64_t first = (int64_t)tile * p.steps, last = first + p.steps - 1;
  const int lo = (int)(first / p.quota), hi = (int)(last / p.quota);
  if (lo == hi) return;  // summed by one cluster, and written by it
  const int id = p.waves * p.clusters + tile;
  const int64_t m = (int64_t)(id / p.tiles_n) * kTile + rank * kHalf + mi;
  const int64_t n = (int64_t)(id % p.tiles_n) * kTile + ni;
  const int64_t row = DX ? m : n < p.cols ? dw_row(p, n) : -1;
  if (row < 0 || m >= p.rows || n >= p.cols) return;
  // a cluster's first segment is in its slot 0, its second in slot 1
  const int two = (int64_t)lo * p.quota / p.steps == tile ? 0 : 1;
  const float4* from = reinterpret_cast<const float4*>(partial + ((size_t)lo * 4 + rank) * kPartialFloats +
                                                       (size_t)ni * kHalf + (DX ? mi * 4 : mi));
  const size_t next = kPartialFloats;  // float4s from one cluster's slot 0 to the next one's
  float4 v[kPer / 4];
#pragma unroll
  for (int q = 0; q < kPer / 4; ++q) v[q] = from[(two ? kPartialFloats / 2 : 0) + q * kHalf];
#pragma unroll 4
  for (int i = 1; i <= hi - lo; ++i)
#pragma unroll
    for (int q = 0; q < kPer / 4; ++q) {
      const float4 u = from[i * next + q * kHalf];
      v[q].x += u.x, v[q].y += u.y, v[q].z += u.z, v[q].w += u.w;
    }
  Pack<TO, kPer> r;
  TO* to = (TO*)p.out + row * p.out_stride + (DX ? n : m);
  const int64_t left = DX ? p.cols - n : p.rows - m;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const float x = (&v[j / 4].x)[j % 4];
    r.v[j] = from_f32<TO>(p.accumulate && j < left ? x + to_f32(to[j]) : x);
  }
  if (p.out_wide && left >= kPer) {
    store_pack<TO, kPer>(to, r);
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (j < left) to[j] = r.v[j];
  }
}
// Both in one launch: dx's blocks, then dW's.
struct Joins {
  Job dx, dw;
  int32_t dx_blocks;
  const float *dx_partial, *dw_partial;
};
template <typename T, typename TO>
__global__ void __launch_bounds__(128) ffn_join_kernel(const __grid_constant__ Joins p) {
  launch_dependents();
  wait_for_previous();
  if ((int)blockIdx.x < p.dx_blocks) join_partials<T, true>(p.dx, p.dx_partial, blockIdx.x);
  else join_partials<TO, false>(p.dw, p.dw_partial, blockIdx.x - p.dx_blocks);
}

// Rows that start anywhere, copied to padded rows that TMA can read (`granules` of eight
// elements each); the padding is zeros.
struct Copies {
  int count;
  struct {
    const void* from;
    void* to;
    int64_t rows, stride, to_stride;
    int32_t cols, granules;
  } c[3];
};
template <typename W>
__global__ void __launch_bounds__(256) ffn_rows_kernel(const __grid_constant__ Copies p) {
  launch_dependents();
  wait_for_previous();
  const auto& k = p.c[blockIdx.y];
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, r = i / k.granules;
  const int c = (int)(i % k.granules) * 8;
  if (r >= k.rows) return;
  const W* from = (const W*)k.from + r * k.stride;
  Pack<W, 8> v;
#pragma unroll
  for (int j = 0; j < 8; ++j) v.v[j] = c + j < k.cols ? from[c + j] : W(0);
  store_pack<W, 8>((W*)k.to + r * k.to_stride + c, v);
}

// ---- few tokens -----------------------------------------------------------------
// Up to 8 NT tokens: the weights' bytes bound the call, so each is read once, straight
// from memory into the operands' registers (mma.sync).  A block has 8 hidden channels:
// the first operand's 16 rows are their 8 rows of Wg and 8 of Wu, so that a thread holds
// gate and up of the same channel and token; its warps share out the channels of x.  A
// thread takes 16 bytes of a row at a time: the sum's terms in another order than the
// instruction's, the same one in both operands.  (1024 x 2816 bf16,
// one token: 3.7 us, 3.1 TB/s.)
constexpr int kFewWarps = 8;
constexpr int kFewRows = 8;

template <typename T, bool WIDE>
__device__ __forceinline__ uint4 eight_of(const T* row, int k, int channels) {
  if (WIDE && k + 8 <= channels) return *reinterpret_cast<const uint4*>(row + k);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (k + j < channels) w[j / 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(row + k + j) << (j % 2 * 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

struct Few {
  int32_t tokens, channels, hidden;
  const void *x, *w;
  int64_t x_stride, w_stride;
  void* h;
  int64_t h_stride;
};

template <typename T, int ACT, int NT, bool WIDE>
__global__ void __launch_bounds__(32 * kFewWarps) ffn_few_kernel(const __grid_constant__ Few p) {
  launch_dependents();
  wait_for_previous();
  __shared__ float sums[kFewWarps][NT * 4][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int f = blockIdx.x * kFewRows + g;
  const T* gate = (const T*)p.w + (int64_t)min(f, p.hidden - 1) * p.w_stride;
  const T* up = gate + (int64_t)p.hidden * p.w_stride;
  float c[NT][4] = {};
  constexpr int kAhead = NT > 2 ? 2 : 4;  // blocks of 32 channels under way
  for (int b = warp; b * 32 < p.channels; b += kFewWarps * kAhead) {
    uint4 a0[kAhead], a1[kAhead], x[kAhead][NT];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = (b + i * kFewWarps) * 32 + t * 8;
      a0[i] = a1[i] = make_uint4(0, 0, 0, 0);
      if (k < p.channels) {
        a0[i] = eight_of<T, WIDE>(gate, k, p.channels);
        a1[i] = eight_of<T, WIDE>(up, k, p.channels);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        x[i][n] = make_uint4(0, 0, 0, 0);
        if (k < p.channels && n * 8 + g < p.tokens)
          x[i][n] = eight_of<T, WIDE>((const T*)p.x + (n * 8 + g) * p.x_stride, k, p.channels);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma_rows<T>(c[n], a0[i].x, a1[i].x, a0[i].y, a1[i].y, x[i][n].x, x[i][n].y);
        mma_rows<T>(c[n], a0[i].z, a1[i].z, a0[i].w, a1[i].w, x[i][n].z, x[i][n].w);
      }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) sums[warp][n * 4 + j][lane] = c[n][j];
  __syncthreads();
  if (warp >= NT) return;
  float v[4];  // gate of tokens 2t, 2t + 1, up of the same
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[j] = sums[0][warp * 4 + j][lane];
#pragma unroll
    for (int i = 1; i < kFewWarps; ++i) v[j] += sums[i][warp * 4 + j][lane];
  }
  const float2 a = act_value<T, ACT>(make_float2(v[0], v[1]));
  const int token = warp * 8 + 2 * t;
  T* to = (T*)p.h + token * p.h_stride + f;
  if (f < p.hidden && token < p.tokens) to[0] = from_f32<T>(a.x * v[2]);
  if (f < p.hidden && token + 1 < p.tokens) to[p.h_stride] = from_f32<T>(a.y * v[3]);
}

// ---- host ------------------------------------------------------------------
template <typename T>
const void* kernel_of(int mode, int act, bool f32) {
  switch (mode) {
    case kFwd:
      return act == GS_ACT_SILU ? (const void*)ffn_kernel<T, T, kFwd, GS_ACT_SILU>
                                : (const void*)ffn_kernel<T, T, kFwd, GS_ACT_GELU>;
    case kRecompute:
      return act == GS_ACT_SILU ? (const void*)ffn_kernel<T, T, kRecompute, GS_ACT_SILU>
                                : (const void*)ffn_kernel<T, T, kRecompute, GS_ACT_GELU>;
    case kDx:
      return (const void*)ffn_kernel<T, T, kDx, 0>;
    default:
      return f32 ? (const void*)ffn_kernel<T, float, kDw, 0> : (const void*)ffn_kernel<T, T, kDw, 0>;
  }
}
template <typename T>
bool allow_smem() {
  for (int mode = kFwd; mode <= kDw; ++mode)
    for (int v = 0; v < 2; ++v)
      if (cudaFuncSetAttribute(kernel_of<T>(mode, v, v != 0), cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kSmem) != cudaSuccess)
        return false;
  return true;
}

// Clusters of two that run at once on the current device (0: none), looked up once per
// device, with the kernels' shared memory limits.
int resident_clusters() {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  int n = known[dev].load(std::memory_order_acquire);
  if (n) return n;
  if (!allow_smem<__nv_bfloat16>() || !allow_smem<__half>()) return 0;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, kernel_of<__half>(kRecompute, GS_ACT_GELU, false), &cfg) !=
          cudaSuccess ||
      n < 1)
    return 0;
  if (n > kMaxClusters) n = kMaxClusters;
  known[dev].store(n, std::memory_order_release);
  return n;
}

// A tensor map of 16-bit elements: `dims` and boxes innermost first, strides in elements
// between the entries of the outer axes.
bool make_map(CUtensorMap* map, int32_t dtype, const void* p, int rank, const int64_t* dims,
              const int64_t* strides, const int* box) {
  const EncodeFn encode = encode_fn();
  if (!encode) return false;
  cuuint64_t d[3], s[2];
  cuuint32_t b[3], unit[3] = {1, 1, 1};
  for (int i = 0; i < rank; ++i) d[i] = (cuuint64_t)dims[i], b[i] = (cuuint32_t)box[i];
  for (int i = 0; i + 1 < rank; ++i) s[i] = (cuuint64_t)strides[i] * 2;
  return encode(map, dtype == GS_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                (cuuint32_t)rank, const_cast<void*>(p), d, s, b, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int64_t kMaxTokens = ((int64_t)1 << 31) - 2 * kTile;
constexpr int32_t kMaxWidth = 1 << 20;
// Rows in the workspace: whole lines of 128 bytes, as a row of a tile is.  (Tensors whose
// rows start elsewhere in a line cost L2 a half more: 5000 x 1000 x 1360 as they lie forward
// 27 us, 4864 x 1024 x 1408, the same number of tiles, 18.5.)
int64_t padded(int64_t n) { return div_up(n, 64) * 64; }
bool shape_ok(int64_t tokens, int32_t channels, int32_t hidden) {
  return tokens >= 0 && tokens <= kMaxTokens && channels >= 1 && channels <= kMaxWidth && hidden >= 1 &&
         hidden <= kMaxWidth && div_up(tokens, kTile) * div_up(hidden, kHalf) < ((int64_t)1 << 31) &&
         div_up(tokens, kTile) * div_up(channels, kTile) < ((int64_t)1 << 31);
}
// Element alignment, a stride that TMA can count, outputs whose rows do not overlap.
bool matrix_ok(const void* p, int64_t rows, int64_t cols, int64_t stride, int elem, bool output) {
  constexpr int64_t kMost = (int64_t)1 << 38;
  return p && aligned_to(p, elem) && stride < kMost && stride > -kMost &&
         (!output || rows < 2 || stride >= cols);
}

constexpr size_t kHeader = 256;
constexpr size_t kPartialBytes = sizeof(float) * kPartialFloats * 4 * kMaxClusters;

struct Room {  // the workspace's parts
  char *x, *w, *grads;
  float *partial, *dw_partial;  // of dx, of dW
  unsigned int* status;
  size_t bytes;
  Room(void* ws, int64_t tokens, int32_t channels, int32_t hidden, bool backward) {
    char* base = (char*)ws;
    size_t at = kHeader;
    status = (unsigned int*)(base + kWsStatusOffset);
    auto take = [&](size_t n) {
      char* p = base + at;
      at += (n + 255) / 256 * 256;
      return p;
    };
    x = take((size_t)tokens * padded(channels) * 2);
    w = take((size_t)2 * hidden * padded(channels) * 2);
    grads = take(backward ? (size_t)tokens * 2 * padded(hidden) * 2 : 0);
    partial = (float*)take(backward ? kPartialBytes : 0);
    dw_partial = (float*)take(backward ? kPartialBytes : 0);
    bytes = at;
  }
};

// The matrix itself, or (then to be copied) its copy in padded rows, as TMA reads it.
struct Rows {
  const void* p;
  int64_t stride;
};
bool readable(const void* p, int64_t rows, int64_t cols, int64_t stride) {
  return aligned16(p) && (rows < 2 || (stride % 8 == 0 && stride >= cols));
}
void copy_rows(Copies* c, const void* from, int64_t rows, int32_t cols, int64_t stride, void* to, int64_t to_stride) {
  auto& k = c->c[c->count++];
  k.from = from, k.to = to;
  k.rows = rows, k.stride = stride, k.to_stride = to_stride;
  k.cols = cols, k.granules = (int32_t)(padded(cols) / 8);
}
Rows rows_of(Copies* c, const void* p, int64_t rows, int32_t cols, int64_t stride, void* room) {
  const int64_t ld = padded(cols);
  if (readable(p, rows, cols, stride)) return Rows{p, rows < 2 ? ld : stride};
  copy_rows(c, p, rows, cols, stride, room, ld);
  return Rows{room, ld};
}
gs_status run_copies(const Copies& c, cudaStream_t st) {
  int64_t most = 0;
  for (int i = 0; i < c.count; ++i)
    if (c.c[i].rows * c.c[i].granules > most) most = c.c[i].rows * c.c[i].granules;
  if (!most) return GS_OK;
  const int64_t blocks = div_up(most, 256);
  if (blocks > INT32_MAX) return GS_ERR_INVALID_ARG;
  GS_CUDA(launch_overlapped(ffn_rows_kernel<uint16_t>, dim3((unsigned)blocks, c.count), dim3(256), 0, st, c));
  return GS_OK;
}

// Deals out the tiles: whole ones to each cluster in turn, and the rest whole, or (SPLIT)
// in equal shares of their steps.
void deal(Job* p, int64_t tiles, int clusters, bool split) {
  p->clusters = clusters;
  p->waves = (int)(tiles / clusters);
  const int64_t rem = tiles - (int64_t)p->waves * clusters;
  p->rem_steps = rem * p->steps;
  p->quota = p->steps;
  // A share is worth its partial sum from 8 steps on; the join takes as long as 12 steps
  // and one more for every third tile (32640 x 5632 x 1024, dx: its 56 remaining tiles
  // of 88 steps whole 206 us, in shares 205 and 10 for the join).
  const int64_t share = div_up(p->rem_steps, clusters), quota = share > 8 ? share : 8;
  if (split && rem && quota + 12 + rem / 3 < p->steps) p->quota = quota;
}

gs_status launch(const void* kernel, const Job& p, const CUtensorMap& a, const CUtensorMap& b, float* partial,
                 unsigned int* status, cudaStream_t st) {
  const int used = p.waves ? p.clusters : (int)div_up(p.rem_steps, p.quota);
  auto* k = reinterpret_cast<void (*)(Job, CUtensorMap, CUtensorMap, float*, unsigned int*)>(
      const_cast<void*>(kernel));
  GS_CUDA(launch_overlapped(k, dim3(2 * used), dim3(kThreads), kSmem, st, p, a, b, partial, status));
  return GS_OK;
}

// Blocks that join a product's shared tiles (0: there are none).
int64_t join_blocks(const Job& p, int64_t tiles, bool dx) {
  const int64_t rem = tiles - (int64_t)p.waves * p.clusters;
  return !rem || p.quota % p.steps == 0 ? 0 : rem * 2 * (dx ? kHalf / 4 : kTile / 4);
}
const void* pick(int32_t dtype, int mode, int act, bool f32 = false) {
  return dtype == GS_BF16 ? kernel_of<__nv_bfloat16>(mode, act, f32) : kernel_of<__half>(mode, act, f32);
}

struct Args {
  int64_t tokens;
  int32_t channels, hidden, dtype, act;
  const void *x, *w;
  int64_t x_stride, w_stride;
};
bool args_ok(const Args& a) {
  return shape_ok(a.tokens, a.channels, a.hidden) && (a.dtype == GS_BF16 || a.dtype == GS_F16) &&
         (a.act == GS_ACT_SILU || a.act == GS_ACT_GELU) &&
         (a.tokens == 0 || (matrix_ok(a.x, a.tokens, a.channels, a.x_stride, 2, false) &&
                            matrix_ok(a.w, 2 * (int64_t)a.hidden, a.channels, a.w_stride, 2, false) &&
                            a.w_stride * a.hidden < ((int64_t)1 << 38)));
}

// The forward's product, or (dh) the backward's: x times W.
gs_status project(const Args& a, const Rows& x, const Rows& w, const Job& job, int mode, int clusters,
                  const Room& room, cudaStream_t st) {
  CUtensorMap am, bm;
  const int64_t ad[2] = {a.channels, a.tokens}, as[1] = {x.stride};
  const int64_t bd[3] = {a.channels, a.hidden, 2}, bs[2] = {w.stride, w.stride * a.hidden};
  const int ab[2] = {kStep, kHalf}, bb[3] = {kStep, kHalf, 1};
  if (!make_map(&am, a.dtype, x.p, 2, ad, as, ab) || !make_map(&bm, a.dtype, w.p, 3, bd, bs, bb))
    return GS_ERR_CUDA;
  Job p = job;
  p.rows = a.tokens;
  p.cols = a.hidden;
  p.tiles_n = (int)div_up(a.hidden, kHalf);
  p.steps = p.part_steps = (int)div_up(a.channels, kStep);
  deal(&p, div_up(a.tokens, kTile) * p.tiles_n, clusters, false);
  return launch(pick(a.dtype, mode, a.act), p, am, bm, room.partial, room.status, st);
}

template <typename T, int ACT, int NT>
gs_status few_of(const Few& p, bool wide, cudaStream_t st) {
  const dim3 grid((unsigned)div_up(p.hidden, kFewRows)), block(32 * kFewWarps);
  GS_CUDA(wide ? launch_overlapped(ffn_few_kernel<T, ACT, NT, true>, grid, block, 0, st, p)
               : launch_overlapped(ffn_few_kernel<T, ACT, NT, false>, grid, block, 0, st, p));
  return GS_OK;
}
template <typename T, int ACT>
gs_status few_of(const Few& p, bool wide, cudaStream_t st) {
  return p.tokens <= 8 ? few_of<T, ACT, 1>(p, wide, st) : p.tokens <= 16 ? few_of<T, ACT, 2>(p, wide, st)
                                                                         : few_of<T, ACT, 4>(p, wide, st);
}
// (1024 x 2816, 16 and 32 tokens: 5.7 and 7.9 us, on the tensor cores' tiles 8.9;
// 2048 x 5632: 14.4 and 19.7, 14.0.  Rows that start anywhere, which the tiles have copied
// first: 1023 x 2815, 15.2 and 14.6, 16.4; 2047 x 5631, 16 tokens 42, on the tiles 40.)
bool few(const Args& a) {
  return a.tokens <= 16 || (a.tokens <= 32 && (int64_t)a.channels * a.hidden <= (1 << 22));
}
gs_status few_tokens(const Args& a, void* h, int64_t h_stride, cudaStream_t st) {
  const Few p{(int32_t)a.tokens, a.channels, a.hidden, a.x, a.w, a.x_stride, a.w_stride, h, h_stride};
  const bool wide = rows_aligned(a.x, a.tokens < 2 ? 0 : a.x_stride, 2, 16) && rows_aligned(a.w, a.w_stride, 2, 16);
  if (a.dtype == GS_BF16)
    return a.act == GS_ACT_SILU ? few_of<__nv_bfloat16, GS_ACT_SILU>(p, wide, st)
                                : few_of<__nv_bfloat16, GS_ACT_GELU>(p, wide, st);
  return a.act == GS_ACT_SILU ? few_of<__half, GS_ACT_SILU>(p, wide, st) : few_of<__half, GS_ACT_GELU>(p, wide, st);
}

gs_status forward(const Args& a, void* h, int64_t h_stride, void* workspace, size_t ws_bytes,
                  uint32_t load_steps, int64_t wait_ns, cudaStream_t st) {
  if (!args_ok(a)) return GS_ERR_INVALID_ARG;
  const Room room(workspace, a.tokens, a.channels, a.hidden, false);
  if (!workspace || !aligned16(workspace) || ws_bytes < room.bytes) return GS_ERR_INVALID_ARG;
  if (a.tokens == 0) return GS_OK;
  // (an output at the address of an input that is still read while it is written)
  if (!matrix_ok(h, a.tokens, a.hidden, h_stride, 2, true) || h == a.x || h == a.w) return GS_ERR_INVALID_ARG;
  if (few(a) && load_steps == UINT32_MAX) return few_tokens(a, h, h_stride, st);
  const int clusters = resident_clusters();
  if (!clusters) {
    (void)cudaGetLastError();
    return GS_ERR_CUDA;
  }
  Copies copies{};
  const Rows x = rows_of(&copies, a.x, a.tokens, a.channels, a.x_stride, room.x);
  const Rows w = rows_of(&copies, a.w, 2 * (int64_t)a.hidden, a.channels, a.w_stride, room.w);
  const gs_status s = run_copies(copies, st);
  if (s != GS_OK) return s;
  Job p{};
  p.out = h;
  p.out_stride = h_stride;
  p.out_wide = rows_aligned(h, a.tokens < 2 ? 0 : h_stride, 2, 16);
  p.load_steps = load_steps;
  p.wait_ns = wait_ns;
  return project(a, x, w, p, kFwd, clusters, room, st);
}

gs_status backward(const Args& a, const void* dh, int64_t dh_stride, void* dx, int64_t dx_stride, void* dw,
                   int64_t dw_stride, int32_t dw_dtype, int32_t accumulate, void* workspace,
                   size_t ws_bytes, cudaStream_t st) {
  if (!args_ok(a) || (dw && dw_dtype != a.dtype && dw_dtype != GS_F32)) return GS_ERR_INVALID_ARG;
  const Room room(workspace, a.tokens, a.channels, a.hidden, true);
  if (!workspace || !aligned16(workspace) || ws_bytes < room.bytes) return GS_ERR_INVALID_ARG;
  const int64_t rows = 2 * (int64_t)a.hidden;
  if (dw && !matrix_ok(dw, rows, a.channels, dw_stride, dtype_size(dw_dtype), true))
    return GS_ERR_INVALID_ARG;
  if (a.tokens == 0) {
    if (dw && !accumulate) {
      const size_t e = dtype_size(dw_dtype);
      GS_CUDA(cudaMemset2DAsync(dw, dw_stride * e, 0, a.channels * e, rows, st));
    }
    return GS_OK;
  }
  if (!matrix_ok(dh, a.tokens, a.hidden, dh_stride, 2, false) ||
      (dx && (!matrix_ok(dx, a.tokens, a.channels, dx_stride, 2, true) || dx == a.x || dx == a.w || dx == dw)) ||
      (dw && dw == a.x))
    return GS_ERR_INVALID_ARG;
  if (!dx && !dw) return GS_OK;
  const int clusters = resident_clusters();
  if (!clusters) {
    (void)cudaGetLastError();
    return GS_ERR_CUDA;
  }
  Copies copies{};
  const Rows x = rows_of(&copies, a.x, a.tokens, a.channels, a.x_stride, room.x);
  const Rows w = rows_of(&copies, a.w, rows, a.channels, a.w_stride, room.w);
  // odd rows of dh are copied to where dup will be: a warp reads its block of dh before it
  // writes that of dup
  const int64_t ld = padded(a.hidden);
  const bool dh_wide = rows_aligned(dh, a.tokens < 2 ? 0 : dh_stride, 2, 16);
  uint16_t* dh_room = (uint16_t*)room.grads + ld;
  if (!dh_wide) copy_rows(&copies, dh, a.tokens, a.hidden, dh_stride, dh_room, 2 * ld);
  gs_status s = run_copies(copies, st);
  if (s != GS_OK) return s;

  Job p{};
  p.hidden = a.hidden;
  p.hidden_ld = (int)ld;
  p.load_steps = UINT32_MAX;
  p.wait_ns = kWaitNs;
  {
    Job q = p;
    q.out = room.grads;
    q.out_stride = 2 * ld;
    q.dh = dh_wide ? dh : dh_room;
    q.dh_stride = dh_wide ? dh_stride : 2 * ld;
    s = project(a, x, w, q, kRecompute, clusters, room, st);
    if (s != GS_OK) return s;
  }
  Joins joins{};
  int64_t blocks = 0;
  CUtensorMap am, bm;
  if (dx) {
    Job q = p;
    q.rows = a.tokens;
    q.cols = a.channels;
    q.out = dx;
    q.out_stride = dx_stride;
    q.out_wide = rows_aligned(dx, a.tokens < 2 ? 0 : dx_stride, 2, 16);
    q.tiles_n = (int)div_up(a.channels, kTile);
    q.part_steps = (int)div_up(a.hidden, kStep);
    q.steps = 2 * q.part_steps;
    const int64_t tiles = div_up(a.tokens, kTile) * q.tiles_n;
    deal(&q, tiles, clusters, true);
    const int64_t ad[3] = {a.hidden, a.tokens, 2}, as[2] = {2 * ld, ld};
    const int64_t bd[3] = {a.channels, a.hidden, 2}, bs[2] = {w.stride, w.stride * a.hidden};
    const int ab[3] = {kStep, kHalf, 1}, bb[3] = {64, kStep, 1};
    if (!make_map(&am, a.dtype, room.grads, 3, ad, as, ab) || !make_map(&bm, a.dtype, w.p, 3, bd, bs, bb))
      return GS_ERR_CUDA;
    s = launch(pick(a.dtype, kDx, 0), q, am, bm, room.partial, room.status, st);
    if (s != GS_OK) return s;
    joins.dx = q;
    joins.dx_blocks = (int32_t)join_blocks(q, tiles, true);
  }
  if (dw) {
    Job q = p;
    q.rows = a.channels;
    q.cols = 2 * ld;
    q.out = dw;
    q.out_stride = dw_stride;
    q.out_wide = rows_aligned(dw, dw_stride, dtype_size(dw_dtype), 16);
    q.accumulate = accumulate != 0;
    q.tiles_n = (int)div_up(2 * ld, kTile);
    q.steps = q.part_steps = (int)div_up(a.tokens, kStep);
    const int64_t tiles = div_up(a.channels, kTile) * q.tiles_n;
    deal(&q, tiles, clusters, true);
    const int64_t ad[2] = {a.channels, a.tokens}, as[1] = {x.stride};
    const int64_t bd[2] = {2 * ld, a.tokens}, bs[1] = {2 * ld};
    const int box[2] = {64, kStep};
    if (!make_map(&am, a.dtype, x.p, 2, ad, as, box) || !make_map(&bm, a.dtype, room.grads, 2, bd, bs, box))
      return GS_ERR_CUDA;
    const bool f32 = dw_dtype == GS_F32;
    s = launch(pick(a.dtype, kDw, 0, f32), q, am, bm, room.dw_partial, room.status, st);
    if (s != GS_OK) return s;
    joins.dw = q;
    blocks = join_blocks(q, tiles, false);
  }
  if (blocks += joins.dx_blocks) {
    joins.dx_partial = room.partial, joins.dw_partial = room.dw_partial;
    const dim3 grid((unsigned)blocks), block(128);
    if (a.dtype == GS_BF16)
      GS_CUDA(dw && dw_dtype == GS_F32
                  ? launch_overlapped(ffn_join_kernel<__nv_bfloat16, float>, grid, block, 0, st, joins)
                  : launch_overlapped(ffn_join_kernel<__nv_bfloat16, __nv_bfloat16>, grid, block, 0, st, joins));
    else
      GS_CUDA(dw && dw_dtype == GS_F32 ? launch_overlapped(ffn_join_kernel<__half, float>, grid, block, 0, st, joins)
                                       : launch_overlapped(ffn_join_kernel<__half, __half>, grid, block, 0, st, joins));
  }
  return GS_OK;
}

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" size_t gs_ffn_workspace_bytes(int64_t tokens, int32_t channels, int32_t hidden, int32_t backward) {
  if (!shape_ok(tokens, channels, hidden)) return 0;
  return Room(nullptr, tokens, channels, hidden, backward != 0).bytes;
}

extern "C" gs_status gs_ffn_fwd(int64_t tokens, int32_t channels, int32_t hidden, int32_t dtype, int32_t act,
                                const void* x, int64_t x_stride, const void* w, int64_t w_stride, void* h,
                                int64_t h_stride, void* workspace, size_t ws_bytes, void* stream) {
  return forward(Args{tokens, channels, hidden, dtype, act, x, w, x_stride, w_stride}, h, h_stride, workspace,
                 ws_bytes, UINT32_MAX, kWaitNs, (cudaStream_t)stream);
}

extern "C" gs_status gs_ffn_bwd(int64_t tokens, int32_t channels, int32_t hidden, int32_t dtype, int32_t act,
                                const void* x, int64_t x_stride, const void* w, int64_t w_stride,
                                const void* dh, int64_t dh_stride, void* dx, int64_t dx_stride, void* dw,
                                int64_t dw_stride, int32_t dw_dtype, int32_t accumulate, void* workspace,
                                size_t ws_bytes, void* stream) {
  return backward(Args{tokens, channels, hidden, dtype, act, x, w, x_stride, w_stride}, dh, dh_stride, dx,
                  dx_stride, dw, dw_stride, dw_dtype, accumulate, workspace, ws_bytes, (cudaStream_t)stream);
}

extern "C" gs_status gs_selftest_ffn_timeout(int64_t tokens, int32_t channels, int32_t hidden, const void* x,
                                             const void* w, void* h, void* workspace, size_t ws_bytes,
                                             int32_t steps, void* stream) {
  // The operands stop after `steps` steps of a pair, so that the products, and with them
  // every other role, wait for what never comes: 100 ms.
  if (steps < 0) return GS_ERR_INVALID_ARG;
  const gs_status s = forward(Args{tokens, channels, hidden, GS_BF16, GS_ACT_SILU, x, w, channels, channels}, h,
                              hidden, workspace, ws_bytes, (uint32_t)steps, 100000000, (cudaStream_t)stream);
  return s != GS_OK ? s : gs_workspace_status(workspace, stream);
}
