// wgrad.cu -- gs_act8_wgrad: the weight gradient of a linear layer from the
// 8-bit checkpoint of its input, on the tensor cores.
//
//   dw[n][c] = sum_t dy[t][n] * q[t][c] * 2^(e[t][c / 32] - 127)
//
// The product is D (channels x columns of dy) = X8^T dY, summed over tokens.  A
// pair of CTAs (a cluster of two) works on 256 channels x BN columns with
// tcgen05.mma over both SMs: each CTA holds 128 channels of X8 and half of the
// columns.  dy is read as it lies ("MN-major": 64 neighbouring columns of one
// token are one 128-byte row of a swizzled tile).  X8 goes to TMEM: an operand
// there has a channel per lane and a pair of tokens per column, and it neither
// has to be written to nor read from shared memory, which would otherwise be the
// bound: per step of 64 tokens an SM would move 80 KB or more through it (dy in
// and out, the bytes in and out, X8 in and out), 640 cycles at 128 bytes each,
// against 570 of the tensor cores.
//
// Warps of a CTA: one brings dy in by TMA, one the checkpoint's bytes (TMA), one
// its exponents, eight turn the bytes into bf16 (exact: at most 8 significant
// bits times a power of two) on the way from shared memory to TMEM, one (of the
// pair's first CTA) issues the products, eight add finished runs of products
// from TMEM to their registers and write the result.  The decoding warps touch
// shared memory and TMEM only: a cluster-wide release or a fence in a thread
// with global loads in flight waits for those loads.
//
// dy enters whole in every type: bf16 by TMA as it lies in memory where its
// rows allow it; otherwise as 1 (bf16), 2 (fp16) or 3 (fp32) bf16 terms whose
// sum is the value (8 bits of the significand each), which a first kernel
// writes to the workspace, and the product runs over the terms.
//
// Work: tiles of 256 channels x BN columns.  As many whole tiles as divide
// evenly over the clusters are summed by one cluster each; the token steps of
// the remaining tiles are dealt out evenly, and the partial sums of a tile
// that several clusters share are joined in a fixed order by a second kernel.
#include <atomic>

#include "tensor_core.cuh"

namespace gs {
namespace {

constexpr int kBM = 256;          // channels of a tile (two CTAs of 128)
constexpr int kBN = 256;          // most columns of a tile
constexpr int kBT = 64;           // tokens of a step
constexpr int kStages = 8;        // of operands: dy in shared memory, X8 in TMEM
constexpr int kRaw = 6;           // of checkpoint bytes
constexpr int kAColumns = kBT / 2;          // TMEM columns of a CTA's half of X8
constexpr int kBBytes = kBN / 2 * kBT * 2;  // a CTA's half of dy
static_assert(kBN + kStages * kAColumns <= 512, "TMEM");
constexpr int kRawBytes = 128 * kBT;        // a CTA's 128 channels
constexpr int kExpBytes = 2 * 4 * kBT;      // and their steps as bf16, [4 groups][tokens]
constexpr int kBatch = 8, kBatches = 4;  // exponents: steps of a batch, batches of the ring
constexpr int kCtrlBytes = 1024;
constexpr int kSmem =
    kStages * kBBytes + kRaw * kRawBytes + kBatches * kBatch * kExpBytes + kCtrlBytes + 1024;  // + alignment
constexpr int kDecodeWarps = 8, kTeamWarps = 4, kTeams = kDecodeWarps / kTeamWarps;
static_assert(kTeamWarps == 4, "a team's warps are the four quarters of TMEM's lanes");
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (4 + kEpiWarps + kDecodeWarps);
// Registers a thread: the launch gives every thread kLaunchRegs, the roles
// then share those out (61,440 a CTA).
constexpr int kLaunchRegs = 96, kCtrlRegs = 48, kEpiRegs = 176, kDecodeRegs = 40;
static_assert(128 * kCtrlRegs + 32 * kEpiWarps * kEpiRegs + 32 * kDecodeWarps * kDecodeRegs <=
                  kThreads * kLaunchRegs,
              "a role would wait for registers that the launch does not have");
// Steps that the tensor core sums on its own.  Its fp32 sum is cut, not rounded,
// after every product of 16 tokens, so its error grows with the length: 32640
// tokens in one run are off by 1.7e-5 of the result's norm (an fp32 product on
// the fp32 units: 8.8e-7); in runs of 32 steps, added up in registers with
// rounding, by 4.7e-7.
constexpr int kChunk = 32;
static_assert(kTeams <= kStages && kTeams <= kRaw, "rings");
constexpr int kMaxClusters = 128;
constexpr size_t kPartialFloats = (size_t)128 * kBN;  // one CTA's half tile
constexpr unsigned int kErrTimeout = 1u;
constexpr int64_t kWaitNs = 2000000000;

struct Plan {
  int64_t tokens;
  int32_t rows, channels;      // dw's shape
  int32_t bn;                  // columns of a tile
  int32_t tiles_m;             // channel tiles
  int32_t terms;               // bf16 terms of dy
  int64_t term_rows;           // rows of the tensor map between terms
  int32_t token_steps, steps;  // steps over the tokens; of a whole tile
  int32_t clusters, waves;     // whole tiles per cluster
  int32_t rem_tiles;           // tiles dealt out in steps
  int64_t rem_steps, quota;    // their steps, and a cluster's share
  int64_t dws;
  int32_t accumulate;
  uint32_t exp_steps;  // steps whose exponents are brought: all, but in the self-test
  int64_t wait_ns;     // after which a wait gives up
};

// A cluster's steps one by one: its whole tiles, then its share of the dealt-out
// steps.  Within a tile the steps run over blocks of kChunk token steps, all of
// them for one term of dy after the other, so that a run of products that the
// tensor core sums on its own has terms of one size.  Every role goes through
// this once per step, on the latency of its own instructions: divisions are done
// once per segment (the steps of one tile).
struct Walk {
  const Plan& p;
  int cluster, wave, left;
  int64_t at, stop;
  int ch0, n0;            // the tile's first channel and column
  int slot;               // place of the segment's partial sum, or -1: the whole tile
  int ts, term;           // the step's tokens (from 64 ts on) and term of dy
  int block, block_end;   // the block of token steps it is in
  __device__ __forceinline__ Walk(const Plan& plan, int cl)
      : p(plan), cluster(cl), wave(0), left(0), ch0(0), n0(0), slot(-1), ts(0), term(0), block(0),
        block_end(0) {
    at = (int64_t)cl * p.quota;
    stop = min(at + p.quota, p.rem_steps);
  }
  __device__ __forceinline__ void begin(int tile, int first, int steps) {
    n0 = tile / p.tiles_m * p.bn;
    ch0 = tile % p.tiles_m * kBM;
    block = first / (kChunk * p.terms) * kChunk;
    block_end = min(block + kChunk, p.token_steps);
    const int in = first - block * p.terms, size = block_end - block;
    term = in / size;
    ts = block + in - term * size;
    left = steps - 1;
  }
  __device__ __forceinline__ bool next() {
    if (--left >= 0) {
      if (++ts == block_end) {
        if (++term == p.terms) {
          term = 0;
          block = block_end;
          block_end = min(block + kChunk, p.token_steps);
        }
        ts = block;
      }
      return true;
    }
    if (wave < p.waves) {
      slot = -1;
      begin(wave++ * p.clusters + cluster, 0, p.steps);
      return true;
    }
    if (at >= stop) return false;
    const int i = (int)(at / p.steps);
    const int64_t upto = min(stop, (int64_t)(i + 1) * p.steps);
    const int n = (int)(upto - at);
    slot = n == p.steps ? -1 : at == (int64_t)cluster * p.quota ? 0 : 1;
    begin(p.waves * p.clusters + i, (int)(at - (int64_t)i * p.steps), n);
    at = upto;
    return true;
  }
  __device__ __forceinline__ bool segment_ends() const { return left == 0; }
  __device__ __forceinline__ bool run_ends() const { return left == 0 || ts + 1 == block_end; }
};

__device__ __forceinline__ int64_t cluster_steps(const Plan& p, int cluster) {
  const int64_t at = (int64_t)cluster * p.quota;
  const int64_t dealt = min(at + p.quota, p.rem_steps) - at;
  return (int64_t)p.waves * p.steps + (dealt > 0 ? dealt : 0);
}

struct Control {
  uint64_t raw_full[kRaw], raw_empty[kRaw];      // bytes of a step
  uint64_t exp_full[kBatches], exp_empty[kBatches];
  uint64_t full[kStages], empty[kStages];        // both operands of both CTAs (the first's)
  uint64_t acc_full, acc_empty;
  uint32_t tmem;
  // when a role ends: steps whose copies and products it asked for, runs, steps decoded
  uint32_t dy_steps, raw_steps, products, runs, decoded[kDecodeWarps];
  volatile uint32_t abort;                       // a wait of the pair gave up
};

// Waits for a barrier's phase, at most p.wait_ns; false (and the status word set) when
// that ran out or another wait of the pair gave up.
__device__ __forceinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity, Control* c,
                                               const Plan& p, unsigned int* status) {
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
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, Control* c, const Plan& p,
                                          unsigned int* status) {
  if (mbar_try(bar, parity)) return true;
  return mbar_wait_slow(bar, parity, c, p, status);
}

// After giving up: one thread of each CTA waits, at most p.wait_ns in all, until nothing
// of the pair is under way that writes shared memory or TMEM: copies of bytes and of dy,
// products, and the arrivals at their end.  Every role of both CTAs has ended, so the
// steps that were asked for are known.
__device__ __forceinline__ void drain(Control* c, const Plan& p, uint32_t rank) {
  const int64_t until = now_ns() + p.wait_ns;
  auto wait = [&](uint64_t* ring, int places, uint32_t step) {  // the phase that `step` ends
    while (!mbar_try(smem_u32(&ring[step % places]), step / places & 1) && now_ns() < until) {}
  };
  auto last = [&](uint64_t* ring, int places, uint32_t steps) {
    for (uint32_t i = steps < places ? 0 : steps - places; i < steps; ++i) wait(ring, places, i);
  };
  last(c->raw_full, kRaw, c->raw_steps);
  last(c->empty, kStages, load_pair(&c->products, 0));
  if (const uint32_t runs = load_pair(&c->runs, 0)) wait(&c->acc_full, 1, runs - 1);
  if (rank) return;
  // dy's copies of both CTAs end at the first one's barriers, at whose steps what else was
  // to arrive is made up for: X8 of decoding warps that gave up, and dy's other half where
  // only one CTA asked for its own.
  const uint32_t own = c->dy_steps, other = load_pair(&c->dy_steps, 1), steps = max(own, other);
  const uint32_t half = (uint32_t)(p.bn / 2 * kBT * 2);
  for (uint32_t i = steps < kStages ? 0 : steps - kStages; i < steps; ++i) {
    const uint32_t bar = smem_u32(&c->full[i % kStages]);
    uint32_t missing = 0;
    for (uint32_t w = i % kTeams * kTeamWarps, n = 0; n < kTeamWarps; ++w, ++n)
      missing += (c->decoded[w] <= i) + (load_pair(&c->decoded[w], 1) <= i);
    if (i >= own) mbar_expect(bar, half);
    if (i >= other)
      asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(in_cta0(bar)),
                   "r"(half)
                   : "memory");
    if (missing)
      asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(missing) : "memory");
  }
  last(c->full, kStages, steps);
}

// Shared-memory descriptor of an MN-major operand in 128-byte swizzled rows:
// 64 channels are a row, 8 tokens an atom of 1024 bytes (stride between atoms
// along the tokens), and the next 64 channels follow after kBT rows.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
  constexpr uint64_t kMn = (uint64_t)(kBT * 128 >> 4), kTok = (uint64_t)(1024 >> 4);
  return (uint64_t)((addr & 0x3ffff) >> 4) | (kMn << 16) | (kTok << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)2 << 61);
}
// Instruction descriptor: fp32 accumulator, bf16 operands, the second MN-major.
__device__ __forceinline__ uint32_t instr_desc(int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(kBM >> 4) << 24);
}
// First operand in TMEM (each CTA's own), second in shared memory.
__device__ __forceinline__ void mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d), "r"(a), "l"(b),
      "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
// 32 columns of the warp's lanes, added to acc.
__device__ __forceinline__ void tmem_add32(uint32_t addr, float* acc) {
  uint32_t v[32];
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
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) acc[i] += __uint_as_float(v[i]);
}
// 16 lanes x 8 columns: thread t gives columns 2 (t % 4) and the next of lane
// t / 4, then of lane t / 4 + 8.
__device__ __forceinline__ void tmem_store16x8(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                               uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x1.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

__device__ __forceinline__ uint32_t load_shared(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint2 load_shared2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

template <typename TO>
__device__ __forceinline__ void put_dw(TO* p, float v, int accumulate) {
  *p = from_f32<TO>(accumulate ? v + to_f32(*p) : v);
}

// Two bytes of the checkpoint (the low bytes of the halves) to two bf16 values
// times two steps.  A byte b = 128 s + m (two's complement: the value is m - 128 s)
// sits in the significand of 128 + m; taking 128 (s = 0) or 256 (s = 1), whose
// bf16 patterns differ by that very bit, from it leaves the value.  Exact, but for
// 64 steps of 2^122, which are bf16's infinity: taking the largest number in their
// place, as the other readers do, cost 3 % of the kernel (32640 x 5632 x 1024: 287 us
// in place of 278, with marked batches of exponents and a second path for those).
__device__ __forceinline__ uint32_t decode2(uint32_t bytes, uint32_t steps) {
  const uint32_t m = (bytes & 0x007f007fu) | 0x43004300u;
  const uint32_t c = (bytes & 0x00800080u) | 0x43004300u;
  const __nv_bfloat162 v = __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162*>(&m),
                                           *reinterpret_cast<const __nv_bfloat162*>(&c)),
                                   *reinterpret_cast<const __nv_bfloat162*>(&steps));
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <typename TO>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    wgrad_kernel(const __grid_constant__ Plan p, const __grid_constant__ CUtensorMap dy_map,
                 const __grid_constant__ CUtensorMap q_map, const uint8_t* e,
                 int64_t es, TO* dw, float* partial, unsigned int* status) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
  uint8_t* raw_q = smem + kStages * kBBytes;
  uint8_t* raw_e = raw_q + kRaw * kRawBytes;
  Control* c = (Control*)(raw_e + kBatches * kBatch * kExpBytes);
  // (the same in every lane, and known to be)
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int cluster = blockIdx.x >> 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&c->full[i]), 1 + 2 * kTeamWarps);  // dy's bytes; both CTAs' X8
      mbar_init(smem_u32(&c->empty[i]), 1);
    }
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(smem_u32(&c->raw_full[i]), 1);
      mbar_init(smem_u32(&c->raw_empty[i]), kTeamWarps);
    }
    for (int i = 0; i < kBatches; ++i) {
      mbar_init(smem_u32(&c->exp_full[i]), 1);
      mbar_init(smem_u32(&c->exp_empty[i]), kBatch * kTeamWarps);
    }
    mbar_init(smem_u32(&c->acc_full), 1);
    mbar_init(smem_u32(&c->acc_empty), 2 * kEpiWarps);
    c->dy_steps = c->raw_steps = c->products = c->runs = 0;
    c->abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) {
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
  wait_for_previous();  // dy's terms, and all before, are there

  if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCtrlRegs));
  if (warp == 0) {
    // ---- dy by TMA: this CTA's half of the tile's columns ------------------
    const bool issues = elect_one();
    const int half = p.bn / 2;
    const uint32_t bars = in_cta0(smem_u32(&c->full[0])), bytes = (uint32_t)(half * kBT * 2 * 2);
    const uint32_t total = (uint32_t)cluster_steps(p, cluster);
    Walk w(p, cluster);
    uint32_t st = 0, phase = 0, it = 0;
    for (; it < total; ++it) {
      w.next();
      if (!mbar_wait(smem_u32(&c->empty[st]), phase ^ 1, c, p, status)) break;
      if (issues) {
        if (rank == 0) mbar_expect(smem_u32(&c->full[st]), bytes);
        const uint32_t dst = smem_u32(smem) + st * kBBytes;
        const int x = w.n0 + (int)rank * half, y = w.term * (int)p.term_rows + w.ts * kBT;
        tma_load(dst, &dy_map, x, y, bars + st * 8);
        if (half == 128) tma_load(dst + kBT * 128, &dy_map, x + 64, y, bars + st * 8);
      }
      if (++st == kStages) st = 0, phase ^= 1;
    }
    if (issues) c->dy_steps = it;
    // the last products release the last stages: every arrival is in before this CTA ends
    for (uint32_t i = total < kStages ? 0 : total - kStages; i < total; ++i)
      if (!mbar_wait(smem_u32(&c->empty[i % kStages]), (i / kStages) & 1, c, p, status)) break;
  } else if (warp == 1) {
    // ---- products ----------------------------------------------------------
    // The whole warp walks the steps, so that what it computes stays in uniform
    // registers, as the product's operands have to be; one elected lane issues.
    if (rank == 0) {
      const uint32_t idesc = instr_desc(p.bn);
      const bool issues = elect_one();
      const uint64_t b_first = smem_desc(smem_u32(smem));
      const int64_t total = cluster_steps(p, cluster);
      Walk w(p, cluster);
      uint32_t st = 0, phase = 0, acc_phase = 1, runs = 0;
      bool begins = true;  // a run of products
      int64_t it = 0;
      for (; it < total; ++it) {
        w.next();
        if (begins) {
          if (!mbar_wait(smem_u32(&c->acc_empty), acc_phase, c, p, status)) break;
          acc_phase ^= 1;
        }
        if (!mbar_wait(smem_u32(&c->full[st]), phase, c, p, status)) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t a = tmem + kBN + st * kAColumns;
        const uint64_t b = b_first + st * (kBBytes >> 4);
        const bool ends = w.run_ends();
        if (issues) {
#pragma unroll
          for (int i = 0; i < kBT / 16; ++i)  // 16 tokens: 8 columns, and two atoms of 1024 bytes
            mma(tmem, a + 8 * i, b + (i * 2048 >> 4), idesc, !begins || i > 0);
          mma_commit(smem_u32(&c->empty[st]));
          if (ends) mma_commit(smem_u32(&c->acc_full));
        }
        begins = ends;
        runs += ends;
        if (++st == kStages) st = 0, phase ^= 1;
      }
      if (issues) c->products = (uint32_t)it, c->runs = runs;
    }
  } else if (warp == 3) {
    // ---- the checkpoint's bytes by TMA -------------------------------------
    const bool issues = elect_one();
    Walk w(p, cluster);
    uint32_t rs = 0, phase = 0, steps = 0;
    while (w.next()) {
      if (!mbar_wait(smem_u32(&c->raw_empty[rs]), phase ^ 1, c, p, status)) break;
      if (issues) {
        const uint32_t bar = smem_u32(&c->raw_full[rs]);
        mbar_expect(bar, kRawBytes);
        tma_load_own(smem_u32(raw_q) + rs * kRawBytes, &q_map, w.ch0 + (int)rank * 128, w.ts * kBT,
                     bar);
      }
      ++steps;
      if (++rs == kRaw) rs = 0, phase ^= 1;
    }
    if (issues) c->raw_steps = steps;
  } else if (warp == 2) {
    // ---- and its exponents, kBatch steps at a time ---------------------------
    // Exponent rows start anywhere, so they come by plain loads; the arrival
    // that hands a batch on waits for those loads, once for kBatch steps.
    Walk w(p, cluster);
    const int groups = (p.channels + GS_ACT8_GROUP - 1) / GS_ACT8_GROUP;
    const bool words = ((es | (int64_t)(uintptr_t)e) & 3) == 0;
    const uint32_t total = min((uint32_t)cluster_steps(p, cluster), p.exp_steps);
    for (uint32_t it0 = 0; it0 < total; it0 += kBatch) {
      uint32_t x[kBatch][2];  // four groups of tokens 2 lane and 2 lane + 1
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        x[i][0] = x[i][1] = 0x01010101u;
        if (!w.next()) continue;
        const int g = w.ch0 / GS_ACT8_GROUP + (int)rank * 4;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t t = (int64_t)w.ts * kBT + 2 * lane + h;
          if (t >= p.tokens) continue;
          const uint8_t* src = e + t * es + g;
          if (words && g + 4 <= groups) {
            x[i][h] = *reinterpret_cast<const uint32_t*>(src);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (g + j < groups)
                x[i][h] = (x[i][h] & ~(0xffu << 8 * j)) | (uint32_t)src[j] << 8 * j;
          }
        }
      }
      const uint32_t n = it0 / kBatch, bs = n % kBatches;
      if (!__all_sync(0xffffffffu,
                      mbar_wait(smem_u32(&c->exp_empty[bs]), ((n / kBatches) & 1) ^ 1, c, p, status)))
        break;
      uint32_t* to = reinterpret_cast<uint32_t*>(raw_e + bs * kBatch * kExpBytes) + lane;
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)  // 2^(e - 127) in bf16, of two tokens; 255: infinity
          to[i * 128 + j * 32] =
              __byte_perm(x[i][0] >> 8 * j, x[i][1] >> 8 * j, 0x5410) << 7 & 0x7f807f80u;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&c->exp_full[bs]));
    }
  } else if (warp < 4 + kEpiWarps) {
    // ---- chunks of the sum from TMEM into registers, then to memory ----------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpiRegs));
    const int quarter = warp & 3;  // the TMEM lanes this warp may read
    const int cols = p.bn / 2, c0 = (warp - 4) / 4 * cols;
    // the lane's channel: see the decoding warps
    const int row = quarter * 32 + 4 * (lane & 7) + (lane >> 3);
    uint32_t phase = 0;
    float acc[kBN / 2];
#pragma unroll
    for (int j = 0; j < kBN / 2; ++j) acc[j] = 0.f;
    Walk w(p, cluster);
    while (w.next()) {
      if (!w.run_ends()) continue;
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&c->acc_full), phase, c, p, status))) break;
      phase ^= 1;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t from = tmem + c0 + ((uint32_t)(quarter * 32) << 16);
#pragma unroll
      for (int j = 0; j < kBN / 2; j += 32)
        if (j < cols) tmem_add32(from + j, acc + j);
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive_pair(in_cta0(smem_u32(&c->acc_empty)));
      if (!w.segment_ends()) continue;
      const int n0 = w.n0 + c0, ch = w.ch0 + (int)rank * 128 + row;
      if (w.slot < 0) {
        TO* to = dw + (int64_t)n0 * p.dws + ch;
#pragma unroll
        for (int j = 0; j < kBN / 2; ++j, to += p.dws)
          if (ch < p.channels && j < cols && n0 + j < p.rows) put_dw<TO>(to, acc[j], p.accumulate);
      } else {
        float* to = partial + ((size_t)(cluster * 2 + w.slot) * 2 + rank) * kPartialFloats +
                    c0 * 128 + row;
#pragma unroll
        for (int j = 0; j < kBN / 2; ++j)
          if (j < cols) to[j * 128] = acc[j];
      }
#pragma unroll
      for (int j = 0; j < kBN / 2; ++j) acc[j] = 0.f;
    }
  } else {
    // ---- bytes to bf16 -------------------------------------------------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kDecodeRegs));
    // kTeams teams of warps take the steps in turn: a step's waits and loads then
    // overlap with the next one's (three or four teams, with fewer registers each,
    // gain nothing: 32640 x 5632 x 1024 in 249 and 252 us, with two 248).
    //
    // A warp has a quarter of TMEM's lanes: 32 channels, one group.  Thread t takes
    // the word of channels 4 (t / 4) .. + 3 of tokens 4 (t % 4) .. + 3 of every 16,
    // and gives lanes t / 4 + 8 i the pairs of channel i of the four: lane r of the
    // quarter holds channel 4 (r % 8) + r / 8.  The threads of the upper two token
    // groups read their tokens in the order 2, 3, 0, 1: with the bytes' 16-byte
    // chunks swizzled by the token, the warp's words then lie in 32 banks.
    const int team = (warp - 4 - kEpiWarps) / kTeamWarps;
    const int quarter = warp & 3, word = lane >> 2, grp = lane & 3;
    const bool swap = grp >= 2;
    const uint32_t lanes = tmem + kBN + ((uint32_t)(quarter * 32) << 16);
    uint32_t from[4];  // the four tokens' words of a stage; the next 16 tokens are 2048 bytes on
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = grp * 4 + (swap ? i ^ 2 : i);
      from[i] = smem_u32(raw_q) + t * 128 + (((quarter * 2 + (word >> 2)) ^ (t & 7)) << 4) +
                (word & 3) * 4;
    }
    const uint32_t steps = smem_u32(raw_e) + quarter * (2 * kBT) + grp * 8;
    const uint32_t full = in_cta0(smem_u32(&c->full[0]));
    const uint32_t total = (uint32_t)cluster_steps(p, cluster);
    uint32_t st = team, st_phase = 0, rs = team, rs_phase = 0, slot = team, slot_phase = 0;
    uint32_t it = team;
    for (; it < total; it += kTeams) {
      if (!__all_sync(0xffffffffu,
                      mbar_wait(smem_u32(&c->exp_full[slot / kBatch]), slot_phase, c, p, status) &&
                          mbar_wait(smem_u32(&c->raw_full[rs]), rs_phase, c, p, status) &&
                          mbar_wait(smem_u32(&c->empty[st]), st_phase ^ 1, c, p, status)))
        break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      const uint32_t bytes = rs * kRawBytes, step_at = steps + slot * kExpBytes;
      const uint32_t to = lanes + st * kAColumns;
#pragma unroll
      for (int b = 0; b < kBT / 16; ++b) {  // 16 tokens: 8 columns
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = load_shared(from[i] + bytes + b * 2048);
        const uint2 s = load_shared2(step_at + b * 32);
        const uint32_t w0 = swap ? w[2] : w[0], w1 = swap ? w[3] : w[1];
        const uint32_t w2 = swap ? w[0] : w[2], w3 = swap ? w[1] : w[3];
        tmem_store16x8(to + b * 8, decode2(__byte_perm(w0, w1, 0x0400), s.x),
                       decode2(__byte_perm(w2, w3, 0x0400), s.y),
                       decode2(__byte_perm(w0, w1, 0x0501), s.x),
                       decode2(__byte_perm(w2, w3, 0x0501), s.y));
        tmem_store16x8(to + b * 8 + (16u << 16), decode2(__byte_perm(w0, w1, 0x0602), s.x),
                       decode2(__byte_perm(w2, w3, 0x0602), s.y),
                       decode2(__byte_perm(w0, w1, 0x0703), s.x),
                       decode2(__byte_perm(w2, w3, 0x0703), s.y));
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_pair(full + st * 8);
        mbar_arrive(smem_u32(&c->raw_empty[rs]));
        mbar_arrive(smem_u32(&c->exp_empty[slot / kBatch]));
      }
      if ((st += kTeams) >= kStages) st -= kStages, st_phase ^= 1;
      if ((rs += kTeams) >= kRaw) rs -= kRaw, rs_phase ^= 1;
      if ((slot += kTeams) >= kBatch * kBatches) slot -= kBatch * kBatches, slot_phase ^= 1;
    }
    if (lane == 0) c->decoded[warp - 4 - kEpiWarps] = it;
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
  if (warp == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// Joins the partial sums of the tiles that several clusters share: a warp takes
// one column of a CTA's half tile, a thread four channels.
template <typename TO>
__global__ void __launch_bounds__(128) wgrad_join_kernel(const __grid_constant__ Plan p,
                                                         const float* partial,
                                                         TO* dw) {
  launch_dependents();
  wait_for_previous();
  const int per_half = p.bn / 4;
  const int tile = blockIdx.x / (2 * per_half), rank = blockIdx.x / per_half % 2;
  const int col = blockIdx.x % per_half * 4 + (int)(threadIdx.x >> 5), in = threadIdx.x % 32 * 4;
  const int64_t first = (int64_t)tile * p.steps, last = first + p.steps - 1;
  const int lo = (int)(first / p.quota), hi = (int)(last / p.quota);
  if (lo == hi) return;  // summed by one cluster, and written by it
  const int id = p.waves * p.clusters + tile;
  const int n = id / p.tiles_m * p.bn + col;
  const int ch = id % p.tiles_m * kBM + rank * 128 + in;
  if (n >= p.rows || ch >= p.channels) return;
  // a cluster's first segment is in its slot 0, its second in slot 1
  const int two = (int64_t)lo * p.quota / p.steps == tile ? 0 : 1;
  const float4* from = reinterpret_cast<const float4*>(
      partial + ((size_t)lo * 4 + rank) * kPartialFloats + (size_t)col * 128 + in);
  const size_t next = kPartialFloats;  // float4s from one cluster's slot 0 to the next one's
  float4 v = from[two ? kPartialFloats / 2 : 0];
#pragma unroll 8
  for (int i = 1; i <= hi - lo; ++i) {
    const float4 u = from[i * next];
    v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
  }
  const float r[4] = {v.x, v.y, v.z, v.w};
  TO* to = dw + (int64_t)n * p.dws + ch;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (ch + j < p.channels) put_dw<TO>(to + j, r[j], p.accumulate);
}

// dy [tokens][rows] as `terms` bf16 matrices [padded tokens][ld], the next
// 8 bits of the significand in each (cut, not rounded: the rest is exact).
template <typename T>
__global__ void __launch_bounds__(256) wgrad_terms_kernel(int64_t tokens, int64_t padded, int rows,
                                                          int ld, int terms, const T* dy,
                                                          int64_t dys, __nv_bfloat16* out) {
  launch_dependents();
  wait_for_previous();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t t = i / (ld / 2);
  const int n = (int)(i % (ld / 2)) * 2;
  if (t >= padded) return;
  float v[2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
    v[j] = t < tokens && n + j < rows ? to_f32(dy[t * dys + n + j]) : 0.f;
  for (int k = 0; k < terms; ++k) {
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t bits = __float_as_uint(v[j]);
      uint32_t top = bits & 0xffff0000u;
      if ((bits & 0x7fffffffu) > 0x7f800000u) top |= 0x00400000u;  // a NaN stays one
      const bool finite = (bits & 0x7f800000u) != 0x7f800000u;
      v[j] = finite ? v[j] - __uint_as_float(top) : 0.f;
      w |= j ? top : top >> 16;
    }
    *reinterpret_cast<uint32_t*>(out + (k * padded + t) * ld + n) = w;
  }
}

int64_t padded_tokens(int64_t tokens) { return div_up(tokens, kBT) * kBT; }
int padded_rows(int rows) { return (int)div_up(rows, 8) * 8; }
int terms_of(int32_t dtype) { return dtype == GS_BF16 ? 1 : dtype == GS_F16 ? 2 : 3; }

// Clusters of two that run at once on the current device (0: none).  Looked up
// once per device, with the kernels' shared memory limits.
int resident_clusters() {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  int n = known[dev].load(std::memory_order_acquire);
  if (n) return n;
  for (const void* f : {(const void*)wgrad_kernel<float>, (const void*)wgrad_kernel<__nv_bfloat16>}) {
    cudaFuncAttributes a;
    if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess ||
        cudaFuncGetAttributes(&a, f) != cudaSuccess || a.numRegs != kLaunchRegs)
      return 0;  // (the build checks the registers that the roles share out)
  }
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
  if (cudaOccupancyMaxActiveClusters(&n, wgrad_kernel<float>, &cfg) != cudaSuccess || n < 1) return 0;
  if (n > kMaxClusters) n = kMaxClusters;
  known[dev].store(n, std::memory_order_release);
  return n;
}

// dy's terms one after the other have to fit a tensor map's 32-bit coordinates, with the
// rows that the last step reads beyond them.
bool shape_ok(int64_t tokens, int32_t rows, int32_t channels, int32_t dtype) {
  return tokens >= 0 && tokens < ((int64_t)1 << 31) && rows >= 1 && channels >= 1 &&
         dtype_ok(dtype) && terms_of(dtype) * padded_tokens(tokens) <= ((int64_t)1 << 31) - kBT;
}

constexpr size_t kHeader = 256;
size_t partial_bytes() { return sizeof(float) * kPartialFloats * 4 * kMaxClusters; }

}  // namespace
}  // namespace gs

using namespace gs;

extern "C" size_t gs_act8_wgrad_workspace_bytes(int64_t tokens, int32_t rows, int32_t channels,
                                                int32_t dtype) {
  if (!shape_ok(tokens, rows, channels, dtype)) return 0;
  return kHeader + partial_bytes() +
         sizeof(__nv_bfloat16) * terms_of(dtype) * padded_tokens(tokens) * padded_rows(rows);
}

namespace {

// exp_steps, wait_ns: see Plan.
gs_status weight_gradient(int64_t tokens, int32_t rows, int32_t channels, int32_t dtype,
                          const void* dy, int64_t dy_stride, const int8_t* q, int64_t q_stride,
                          const uint8_t* e, int64_t e_stride, void* dw, int64_t dw_stride,
                          int32_t out_dtype, int32_t accumulate, void* workspace, size_t ws_bytes,
                          uint32_t exp_steps, int64_t wait_ns, void* stream) {
  if (!shape_ok(tokens, rows, channels, dtype) ||
      (out_dtype != GS_F32 && out_dtype != GS_BF16) || !dw ||
      !aligned_to(dw, dtype_size(out_dtype)) || !workspace || !aligned16(workspace) ||
      ws_bytes < gs_act8_wgrad_workspace_bytes(tokens, rows, channels, dtype))
    return GS_ERR_INVALID_ARG;
  if (tokens > 0 && (!dy || !aligned_to(dy, dtype_size(dtype)) ||
                     !ckpt_ok(tokens, channels, q, q_stride, e, e_stride)))
    return GS_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  const size_t out_elem = dtype_size(out_dtype);
  if (tokens == 0) {
    if (!accumulate)
      GS_CUDA(cudaMemset2DAsync(dw, dw_stride * out_elem, 0, channels * out_elem, rows, st));
    return GS_OK;
  }
  const EncodeFn encode = encode_fn();
  const int clusters = resident_clusters();
  if (!encode || !clusters) {
    (void)cudaGetLastError();
    return GS_ERR_CUDA;
  }

  Plan p{};
  p.tokens = tokens;
  p.rows = rows;
  p.channels = channels;
  p.bn = rows > 128 ? 256 : 128;
  p.dws = dw_stride;
  p.accumulate = accumulate != 0;
  p.exp_steps = exp_steps;
  p.wait_ns = wait_ns;
  float* partial = (float*)((char*)workspace + kHeader);

  // dy as the tensor map reads it
  const bool direct =
      dtype == GS_BF16 && rows_aligned(dy, dy_stride, 2, 16) && dy_stride >= rows;
  const void* src = dy;
  int64_t height = tokens, stride = dy_stride;
  p.terms = 1;
  p.term_rows = 0;
  if (!direct) {
    p.terms = terms_of(dtype);
    p.term_rows = padded_tokens(tokens);
    const int ld = padded_rows(rows);
    __nv_bfloat16* out = (__nv_bfloat16*)((char*)partial + partial_bytes());
    const unsigned blocks = (unsigned)div_up(p.term_rows * (ld / 2), 256);
    if (dtype == GS_BF16)
      GS_CUDA(launch_overlapped(wgrad_terms_kernel<__nv_bfloat16>, blocks, 256, 0, st, tokens,
                                p.term_rows, rows, ld, 1, (const __nv_bfloat16*)dy, dy_stride, out));
    else if (dtype == GS_F16)
      GS_CUDA(launch_overlapped(wgrad_terms_kernel<__half>, blocks, 256, 0, st, tokens, p.term_rows,
                                rows, ld, 2, (const __half*)dy, dy_stride, out));
    else
      GS_CUDA(launch_overlapped(wgrad_terms_kernel<float>, blocks, 256, 0, st, tokens, p.term_rows,
                                rows, ld, 3, (const float*)dy, dy_stride, out));
    src = out;
    height = p.terms * p.term_rows;
    stride = ld;
  }
  CUtensorMap map;
  const cuuint64_t dims[2] = {(cuuint64_t)rows, (cuuint64_t)height};
  const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
  const cuuint32_t box[2] = {64, kBT}, unit[2] = {1, 1};
  if (encode(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(src), dims, strides, box,
             unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return GS_ERR_CUDA;

  CUtensorMap qmap;
  const cuuint64_t qdims[2] = {(cuuint64_t)div_up(channels, GS_ACT8_GROUP) * GS_ACT8_GROUP,
                               (cuuint64_t)tokens};
  const cuuint64_t qstrides[1] = {(cuuint64_t)q_stride};
  const cuuint32_t qbox[2] = {128, kBT};
  if (encode(&qmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(q), qdims, qstrides, qbox,
             unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return GS_ERR_CUDA;

  p.tiles_m = (int)div_up(channels, kBM);
  const int64_t tiles = p.tiles_m * div_up(rows, p.bn);
  p.token_steps = (int)div_up(tokens, kBT);
  p.steps = p.token_steps * p.terms;
  p.clusters = clusters;
  p.waves = (int)(tiles / clusters);
  p.rem_tiles = (int)(tiles - (int64_t)p.waves * clusters);
  p.rem_steps = (int64_t)p.rem_tiles * p.steps;
  // A share of the dealt-out steps is worth its partial sum from kMinSteps on.
  constexpr int64_t kMinSteps = 8;
  p.quota = div_up(p.rem_steps, clusters);
  if (p.quota < kMinSteps) p.quota = kMinSteps < p.steps ? kMinSteps : p.steps;
  const int used = p.waves ? clusters : (int)div_up(p.rem_steps, p.quota);
  unsigned int* status = (unsigned int*)((char*)workspace + kWsStatusOffset);
  if (out_dtype == GS_F32)
    GS_CUDA(launch_overlapped(wgrad_kernel<float>, 2 * used, kThreads, kSmem, st, p, map, qmap, e,
                              e_stride, (float*)dw, partial, status));
  else
    GS_CUDA(launch_overlapped(wgrad_kernel<__nv_bfloat16>, 2 * used, kThreads, kSmem, st, p, map,
                              qmap, e, e_stride, (__nv_bfloat16*)dw, partial, status));
  if (p.rem_tiles && p.quota % p.steps != 0) {
    const unsigned blocks = (unsigned)(p.rem_tiles * 2 * (p.bn / 4));
    if (out_dtype == GS_F32)
      GS_CUDA(launch_overlapped(wgrad_join_kernel<float>, blocks, 128, 0, st, p, partial, (float*)dw));
    else
      GS_CUDA(launch_overlapped(wgrad_join_kernel<__nv_bfloat16>, blocks, 128, 0, st, p, partial,
                                (__nv_bfloat16*)dw));
  }
  return GS_OK;
}

}  // namespace

extern "C" gs_status gs_act8_wgrad(int64_t tokens, int32_t rows, int32_t channels, int32_t dtype,
                                   const void* dy, int64_t dy_stride, const int8_t* q,
                                   int64_t q_stride, const uint8_t* e, int64_t e_stride, void* dw,
                                   int64_t dw_stride, int32_t out_dtype, int32_t accumulate,
                                   void* workspace, size_t ws_bytes, void* stream) {
  return weight_gradient(tokens, rows, channels, dtype, dy, dy_stride, q, q_stride, e, e_stride, dw,
                         dw_stride, out_dtype, accumulate, workspace, ws_bytes, UINT32_MAX, kWaitNs,
                         stream);
}

extern "C" gs_status gs_selftest_wgrad_timeout(int64_t tokens, int32_t rows, int32_t channels,
                                               const void* dy, const int8_t* q, const uint8_t* e,
                                               void* dw, void* workspace, size_t ws_bytes,
                                               int32_t steps, void* stream) {
  // The exponents stop after `steps` steps of 64 tokens (a multiple of kBatch), so that the
  // decoding warps, and with them every other role, wait for what never comes: 100 ms.
  if (steps < 0) return GS_ERR_INVALID_ARG;
  const int64_t ld = div_up(channels, GS_ACT8_GROUP) * GS_ACT8_GROUP;
  const gs_status s = weight_gradient(tokens, rows, channels, GS_BF16, dy, rows, q, ld, e,
                                      ld / GS_ACT8_GROUP, dw, channels, GS_F32, 0, workspace,
                                      ws_bytes, (uint32_t)steps, 100000000, stream);
  return s != GS_OK ? s : gs_workspace_status(workspace, stream);
}
