// gemm_fp8.cu — products of 8-bit floating-point operands with one fp32 scale per block of 128
// along the reduction, on the 5th-generation tensor cores, persistent.
//
//   matmul  y[r, n]     = sum_b as[b, r] ws[n / 128, b] sum_{k in block b} a[r, k] w[e, n, k]
//           for the rows r of expert e (offsets[e] <= r < offsets[e + 1]), or of one matrix
//   wgrad   dw[e, n, k] = sum_{b of e} dys[b, n] xs[b, k] sum_{r in block b} dy[n, r] x[k, r]
//           with expert e's rows padded to whole blocks of 128
//
// The scales are arbitrary fp32 numbers, which the tensor cores' own block scaling (powers of
// two per 32) does not take.  So the tensor cores compute one block of 128 at a time into one of
// several TMEM buffers, and the epilogue warps add buffer x scales to fp32 accumulators in
// registers while the next block's MMAs run.  Adding a 128 x 256 block takes 128 x 256 fused
// multiply-adds on the CUDA cores (128 a cycle) beside 128 x 256 x 128 on the tensor cores
// (8192 a cycle): half the time, as packed pairs a quarter of the issue slots.
//
// The weights' rows are the MMA's 128 lanes and the tokens its columns ("lane" and "column"
// operand below): the column count of an MMA is any multiple of 16, so an expert with 40 rows
// costs 48 columns, not a 128-row tile; one token costs 16.  A weight's 128 x 128 block is
// exactly a tile's lanes, so its scale is one number per block and is folded into the columns'
// scales; in wgrad every lane has a scale of its own.
//
// Roles of a CTA: warp 0 lane 0 TMA producer; warp 1 lane 0 MMA issuer (warp 1 owns the TMEM);
// warp 2 stages the column scales of each block in shared memory; warps 4.. epilogue, warp w on
// TMEM lanes 32 (w % 4) .. (and column half (w - 4) / 4 with eight of them).
//
// kSplit: few tiles (a few tokens).  A cluster of S CTAs computes one tile, each a range of the
// blocks; the others leave their accumulators in the first one's shared memory, which adds them
// in rank order.
#include "../../include/latent_moe.h"
#include "internal.h"
#include "ptx.cuh"

namespace lmoe {
namespace {

enum Fp8Mode : int { kMatmul = 0, kWgrad = 1, kSplit = 2 };
constexpr int kMaxGroups = 1024;
constexpr int kMaxSplit = 8;

struct Fp8Args {
  long long rows;        // matmul: rows of a and y; wgrad: columns of dy and x (a multiple of 128)
  int lanes, cols;       // extents of the lane operand and (wgrad) of the column operand
  int num_kb;            // matmul: blocks of the reduction
  int E;
  const int32_t* offsets;   // [E + 1], or nullptr: one group of all rows
  const float* ps;       // scales of the lane operand
  const float* qs;       // scales of the column operand, [block][ldq]
  long long ldq;
  void* out;
  int out_f32, accumulate;
  unsigned fmt_p, fmt_q;   // 0 e4m3, 1 e5m2
  unsigned* status;      // error word or nullptr
  long long budget;
  int splits;            // kSplit: CTAs per tile (the cluster size)
};

template <int BN, int MODE>
struct Fp8Cfg {
  static constexpr int kEpiWarps = BN == 256 ? 8 : 4;
  static constexpr int kCols = BN * 4 / kEpiWarps;   // accumulator columns of one thread
  static constexpr int kThreads = 128 + 32 * kEpiWarps;
  static constexpr int kPBytes = 128 * 128;
  static constexpr int kQBytes = BN * 128;
  static constexpr int kStageBytes = kPBytes + kQBytes;
  static constexpr int kBox = BN < 64 ? BN : 64;      // rows of one column-operand box
  static constexpr int kSlots = 8;                    // staged scale blocks
  static constexpr int kBufs = BN == 256 ? 2 : 8;     // TMEM buffers
  static constexpr uint32_t kTmemCols = BN * kBufs;
  static constexpr int kMaxS = BN == 16 ? kMaxSplit : 4;
  static constexpr int kRedBytes = MODE == kSplit ? (kMaxS - 1) * BN * 128 * 4 : 0;
  static constexpr int kTableBytes = 3 * (kMaxGroups + 4) * 4;
  static constexpr int kFixed = kRedBytes + kSlots * BN * 4 + kTableBytes + 512 + 1024;
  static constexpr int kStagesFit = (227 * 1024 - kFixed) / kStageBytes;
  static constexpr int kStages = kStagesFit > 11 ? 11 : kStagesFit;
  static constexpr int kSmemBytes = kFixed + kStages * kStageBytes;
  static_assert(kStages >= 3, "pipeline depth");
  static_assert((2 * kStages + 2 * kBufs + 2 * kSlots + 1) * 8 + 8 <= 512, "barriers");
  static_assert(MODE == kMatmul || BN != 256 || MODE == kWgrad, "split tiles are narrow");
};

// Instruction descriptor of kind::f8f6f4: D fp32 ([4,6) = 1), formats at [7,10) and [10,13),
// both operands K-major, N >> 3 at [17,23), M >> 4 at [24,29).
LMOE_DEV uint32_t idesc_f8(uint32_t fa, uint32_t fb, int n) {
  return (1u << 4) | (fa << 7) | (fb << 10) | (static_cast<uint32_t>(n >> 3) << 17) | ((128u >> 4) << 24);
}
LMOE_DEV void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
LMOE_DEV void tma_load_3d_hint(void* dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1, int c2,
                               uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
      : "memory");
}
// 16 consecutive columns of the warp's 32 lanes
LMOE_DEV void tmem_ld_16cols(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// Waits for the warp's TMEM reads; r passes through, so that no use of it moves ahead of the wait.
LMOE_DEV void tmem_ld_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
// packed pairs of fp32
LMOE_DEV uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
LMOE_DEV void unpack2(uint64_t v, float& lo, float& hi) {
  uint32_t a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
  lo = __uint_as_float(a);
  hi = __uint_as_float(b);
}
LMOE_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
LMOE_DEV uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// Registers of a warpgroup (all four of its warps).  256-column tiles: the epilogue's two
// warpgroups hold 128 accumulators a thread; 4 x 32 x 72 + 8 x 32 x 216 = 384 x 168, what the
// block was launched with.
template <int N>
LMOE_DEV void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
LMOE_DEV void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
LMOE_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
LMOE_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
LMOE_DEV uint32_t cluster_map(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
LMOE_DEV void cluster_store(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// The tiles of a launch, the same walk for every role.  Tables in shared memory, per group e:
// start[e] its first column tile (matmul) or first block (wgrad), lo/hi its rows (matmul).
struct Fp8Walk {
  const int *start, *lo, *hi;
  int E, lane_tiles, col_tiles, total;
};
struct Fp8Tile {
  int e, p0, q0, ncols, kb0, kb1;
  long long out;   // element offset of (first column, first lane)
};

template <int BN, int MODE>
LMOE_DEV Fp8Tile tile_at(const Fp8Walk& w, const Fp8Args& a, int id, int rank) {
  Fp8Tile t;
  int lt, ct;
  if (MODE == kWgrad) {
    const int per = w.lane_tiles * w.col_tiles;
    t.e = id / per;
    grouped_tile(id - t.e * per, w.col_tiles, w.lane_tiles, kRasterGroup, ct, lt);
    t.p0 = lt * 128;
    t.q0 = ct * BN;
    t.ncols = min(BN, a.cols - t.q0);
    t.kb0 = w.start[t.e];
    t.kb1 = w.start[t.e + 1];
    t.out = (static_cast<long long>(t.e) * a.cols + t.q0) * a.lanes + t.p0;
  } else {
    int l = 0, h = w.E;   // the last e with start[e] * lane_tiles <= id
    const int s = id / w.lane_tiles;
    while (h - l > 1) {
      const int m = (l + h) >> 1;
      if (w.start[m] <= s) l = m;
      else h = m;
    }
    t.e = l;
    grouped_tile(id - w.start[l] * w.lane_tiles, w.start[l + 1] - w.start[l], w.lane_tiles, kRasterGroup, ct, lt);
    t.p0 = lt * 128;
    t.q0 = w.lo[l] + ct * BN;
    t.ncols = min(BN, w.hi[l] - t.q0);
    t.kb0 = 0;
    t.kb1 = a.num_kb;
    if (MODE == kSplit) {
      t.kb0 = static_cast<int>(static_cast<long long>(a.num_kb) * rank / a.splits);
      t.kb1 = static_cast<int>(static_cast<long long>(a.num_kb) * (rank + 1) / a.splits);
    }
    t.out = static_cast<long long>(t.q0) * a.lanes + t.p0;
  }
  return t;
}

template <int BN, int MODE>
__global__ void __launch_bounds__(Fp8Cfg<BN, MODE>::kThreads, 1)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                    const Fp8Args args) {
  using C = Fp8Cfg<BN, MODE>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  float* red = reinterpret_cast<float*>(smem + C::kStages * C::kStageBytes);
  float* sc = red + C::kRedBytes / 4;                       // [kSlots][BN]
  int* start = reinterpret_cast<int*>(sc + C::kSlots * BN);   // [E + 1], then lo, hi
  int* lo = start + kMaxGroups + 4;
  int* hi = lo + kMaxGroups + 4;
  uint64_t* full = reinterpret_cast<uint64_t*>(hi + kMaxGroups + 4);
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;
  uint64_t* acc_empty = acc_full + C::kBufs;
  uint64_t* sfull = acc_empty + C::kBufs;
  uint64_t* sempty = sfull + C::kSlots;
  uint64_t* mma_done = sempty + C::kSlots;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], C::kEpiWarps);
    }
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&sfull[s], 1);
      mbar_init(&sempty[s], C::kEpiWarps);
    }
    mbar_init(mma_done, 1);
    fence_mbar_init();
    prefetch_tmap(&tmP);
    prefetch_tmap(&tmQ);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  griddep_enter();

  // the groups: offsets are clamped into the rows there are, so that no table sends a load or a
  // store out of range
  Fp8Walk walk;
  walk.start = start;
  walk.lo = lo;
  walk.hi = hi;
  walk.E = args.E;
  walk.lane_tiles = (args.lanes + 127) / 128;
  walk.col_tiles = MODE == kWgrad ? (args.cols + BN - 1) / BN : 0;
  constexpr int kUnit = MODE == kWgrad ? 128 : BN;   // rows of one unit of start[]
  for (int e = threadIdx.x; e < args.E; e += C::kThreads) {
    int l = 0, h = static_cast<int>(args.rows);
    if (args.offsets != nullptr) {
      const int cap = static_cast<int>(args.rows);
      l = min(max(args.offsets[e], 0), cap);
      h = min(max(args.offsets[e + 1], l), cap);
    }
    lo[e] = l;
    hi[e] = h;
  }
  __syncthreads();
  if (warp == 0) {   // exclusive prefix sum of the groups' units, a run of groups per lane
    const int per = (args.E + 31) / 32, e0 = min(lane * per, args.E), e1 = min(e0 + per, args.E);
    const int cap = MODE == kWgrad ? static_cast<int>(args.rows / 128) : 0x7fffffff;
    int sum = 0;
    for (int e = e0; e < e1; ++e) sum += (hi[e] - lo[e] + kUnit - 1) / kUnit;
    int run = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(~0u, run, d);
      if (lane >= d) run += up;
    }
    const int tot = __shfl_sync(~0u, run, 31);
    run -= sum;
    for (int e = e0; e < e1; ++e) {
      start[e] = min(run, cap);
      run += (hi[e] - lo[e] + kUnit - 1) / kUnit;
    }
    if (lane == 0) start[args.E] = min(tot, cap);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  walk.total = (MODE == kWgrad ? args.E * walk.col_tiles : start[args.E]) * walk.lane_tiles;
  const int S = MODE == kSplit ? args.splits : 1;
  const int rank = MODE == kSplit ? static_cast<int>(blockIdx.x % S) : 0;
  const int id0 = static_cast<int>(blockIdx.x) / S, step = static_cast<int>(gridDim.x) / S;
  const long long budget = args.budget;
  if (MODE == kSplit) cluster_arrive();   // every CTA of the cluster has started (waited for below)

  if (warp < 4) {
  if constexpr (BN == 256) regs_dec<72>();
  if (warp == 0) {
    if (lane == 0) {
      // ---- TMA producer
      // (narrow tiles: few rows, each weight is read about once)
      const uint64_t pol_p = BN == 256 ? policy_evict_normal() : policy_evict_first();
      const uint64_t pol_q = policy_evict_normal();
      int it = 0;
      bool ok = true;
      for (int id = id0; ok && id < walk.total; id += step) {
        const Fp8Tile t = tile_at<BN, MODE>(walk, args, id, rank);
        const int boxes = (t.ncols + C::kBox - 1) / C::kBox;
        const uint32_t tx = C::kPBytes + boxes * C::kBox * 128;
        for (int kb = t.kb0; kb < t.kb1; ++kb, ++it) {
          const int s = it % C::kStages;
          if (!mbar_wait(&empty[s], ((it / C::kStages) & 1) ^ 1, budget)) {
            if (args.status) atomicOr(args.status, kErrWaitProducer);
            ok = false;
            break;
          }
          uint8_t* sp = smem + s * C::kStageBytes;
          mbar_arrive_expect_tx(&full[s], tx);
          if (MODE == kWgrad) tma_load_2d_hint(sp, &tmP, &full[s], kb * 128, t.p0, pol_p);
          else tma_load_3d_hint(sp, &tmP, &full[s], kb * 128, t.p0, t.e, pol_p);
          for (int b = 0; b < boxes; ++b)
            tma_load_2d_hint(sp + C::kPBytes + b * C::kBox * 128, &tmQ, &full[s], kb * 128, t.q0 + b * C::kBox,
                             pol_q);
        }
      }
      // every copy of this thread lands before the CTA leaves
      for (int j = max(0, it - C::kStages); j < it; ++j)
        if (!mbar_wait(&full[j % C::kStages], (j / C::kStages) & 1, kDrainBudget))
          if (args.status) atomicOr(args.status, kErrDrain);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ---- MMA issuer: one block of 128 into one TMEM buffer
      int it = 0;
      bool ok = true;
      for (int id = id0; ok && id < walk.total; id += step) {
        const Fp8Tile t = tile_at<BN, MODE>(walk, args, id, rank);
        const uint32_t idesc = idesc_f8(args.fmt_p, args.fmt_q, (t.ncols + 15) / 16 * 16);
        for (int kb = t.kb0; kb < t.kb1; ++kb, ++it) {
          const int s = it % C::kStages, buf = it % C::kBufs;
          if (!mbar_wait(&acc_empty[buf], ((it / C::kBufs) & 1) ^ 1, budget) ||
              !mbar_wait(&full[s], (it / C::kStages) & 1, budget)) {
            if (args.status) atomicOr(args.status, kErrWaitMma);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t p0 = smem_u32(smem + s * C::kStageBytes);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f8(tmem + buf * BN, sw128_kmajor_desc(p0 + kk * 32), sw128_kmajor_desc(p0 + C::kPBytes + kk * 32),
                   idesc, kk > 0);
          mma_commit(&empty[s]);
          mma_commit(&acc_full[buf]);
        }
      }
      mma_commit(mma_done);
    }
  } else if (warp == 2) {
    // ---- column scales (times the lane block's scale where there is one), four blocks' loads
    // in flight at a time
    constexpr int kPer = (BN + 31) / 32, kBatch = 4;
    int it = 0;
    bool ok = true;
    for (int id = id0; ok && id < walk.total; id += step) {
      const Fp8Tile t = tile_at<BN, MODE>(walk, args, id, rank);
      const float* q = args.qs + t.q0 + lane;
      const float* p = MODE == kWgrad ? nullptr
                                      : args.ps + (static_cast<long long>(t.e) * walk.lane_tiles + t.p0 / 128) *
                                                      args.num_kb;
      for (int kb = t.kb0; ok && kb < t.kb1; kb += kBatch) {
        float v[kBatch][kPer], u[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const bool in = kb + j < t.kb1;
          u[j] = MODE == kWgrad ? 1.f : (in ? p[kb + j] : 0.f);
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            v[j][i] = in && lane + 32 * i < t.ncols ? q[(kb + j) * args.ldq + 32 * i] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          if (!ok || kb + j >= t.kb1) break;
          const int s = it % C::kSlots;
          if (!mbar_wait(&sempty[s], ((it / C::kSlots) & 1) ^ 1, budget)) {
            if (args.status) atomicOr(args.status, kErrWaitProducer);
            ok = false;
            break;
          }
#pragma unroll
          for (int i = 0; i < kPer; ++i)
            if (lane + 32 * i < BN) sc[s * BN + lane + 32 * i] = v[j][i] * u[j];
          __syncwarp();
          if (lane == 0) mbar_arrive(&sfull[s]);
          ++it;
        }
      }
    }
  }
  } else {
    // ---- epilogue
    if constexpr (BN == 256) regs_inc<216>();
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const int r = quad * 32 + lane, c0 = half * C::kCols;
    const uint32_t tq = tmem + (static_cast<uint32_t>(quad * 32) << 16) + c0;
    constexpr int kCh = 16;   // columns of one TMEM read (two are held: 32 registers beside the accumulators)
    constexpr int kN = C::kCols / kCh;
    int it = 0;
    bool ok = true;
    for (int id = id0; ok && id < walk.total; id += step) {
      const Fp8Tile t = tile_at<BN, MODE>(walk, args, id, rank);
      const bool lane_ok = t.p0 + r < args.lanes;
      uint64_t acc[C::kCols / 2];
#pragma unroll
      for (int i = 0; i < C::kCols / 2; ++i) acc[i] = 0;
      const float* ps = MODE == kWgrad ? args.ps + t.p0 + r : nullptr;
      float sp_next = (MODE == kWgrad && lane_ok && t.kb0 < t.kb1) ? ps[static_cast<long long>(t.kb0) * args.lanes] : 0.f;
      for (int kb = t.kb0; kb < t.kb1; ++kb, ++it) {
        const float sp = sp_next;
        if (MODE == kWgrad && lane_ok && kb + 1 < t.kb1) sp_next = ps[static_cast<long long>(kb + 1) * args.lanes];
        const int buf = it % C::kBufs, s = it % C::kSlots;
        if (!mbar_wait(&sfull[s], (it / C::kSlots) & 1, budget) ||
            !mbar_wait(&acc_full[buf], (it / C::kBufs) & 1, budget)) {
          if (args.status) atomicOr(args.status, kErrWaitEpilogue);
          ok = false;
          break;
        }
        tc_fence_after();
        const float* scs = sc + s * BN + c0;
        const uint64_t sp2 = pack2(__float_as_uint(sp), __float_as_uint(sp));
        uint32_t v[2][kCh];
        tmem_ld_16cols(tq + buf * BN, v[0]);

        tmem_ld_wait(v[0]);
#pragma unroll
        for (int ch = 0; ch < kN; ++ch) {
          if (ch + 1 < kN) {
            tmem_ld_16cols(tq + buf * BN + (ch + 1) * kCh, v[(ch + 1) & 1]);
          } else {   // every column of the buffer has been read
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[buf]);
          }
#pragma unroll
          for (int i = 0; i < kCh; i += 4) {
            const ulonglong2 s2 = *reinterpret_cast<const ulonglong2*>(scs + ch * kCh + i);
            uint64_t a = pack2(v[ch & 1][i], v[ch & 1][i + 1]), b = pack2(v[ch & 1][i + 2], v[ch & 1][i + 3]);
            if (MODE == kWgrad) {
              a = mul2(a, sp2);
              b = mul2(b, sp2);
            }
            const int q = (ch * kCh + i) / 2;
            acc[q] = fma2(a, s2.x, acc[q]);
            acc[q + 1] = fma2(b, s2.y, acc[q + 1]);
          }
          if (ch + 1 < kN) tmem_ld_wait(v[(ch + 1) & 1]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sempty[s]);
      }
      if (MODE == kSplit) {
        // one tile per cluster: the accumulators of ranks 1.. go to rank 0 (below)
        if (rank > 0) {
          cluster_wait();
          const uint32_t dst = cluster_map(smem_u32(red + (rank - 1) * BN * 128 + c0 * 128 + r), 0);
#pragma unroll
          for (int i = 0; i < C::kCols / 2; ++i) {
            float x, y;
            unpack2(acc[i], x, y);
            cluster_store(dst + (2 * i) * 512, x);
            cluster_store(dst + (2 * i + 1) * 512, y);
          }
          cluster_arrive();
          cluster_wait();
        } else {
          cluster_wait();
          cluster_arrive();
          cluster_wait();
          for (int q = 1; q < S; ++q) {
            const float* src = red + (q - 1) * BN * 128 + c0 * 128 + r;
#pragma unroll
            for (int i = 0; i < C::kCols / 2; ++i) {
              float x, y;
              unpack2(acc[i], x, y);
              x += src[(2 * i) * 128];
              y += src[(2 * i + 1) * 128];
              acc[i] = pack2(__float_as_uint(x), __float_as_uint(y));
            }
          }
        }
      }
      const bool adds_nothing = args.accumulate && t.kb0 == t.kb1;
      if (ok && lane_ok && rank == 0 && !adds_nothing) {
        const int n = min(C::kCols, t.ncols - c0);
        const long long base = t.out + static_cast<long long>(c0) * args.lanes + r;
        if (args.out_f32) {
          float* o = static_cast<float*>(args.out) + base;
#pragma unroll
          for (int i = 0; i < C::kCols / 2; ++i) {
            float x, y;
            unpack2(acc[i], x, y);
            if (2 * i < n) *o = args.accumulate ? *o + x : x;
            o += args.lanes;
            if (2 * i + 1 < n) *o = args.accumulate ? *o + y : y;
            o += args.lanes;
          }
        } else {
          __nv_bfloat16* o = static_cast<__nv_bfloat16*>(args.out) + base;
#pragma unroll
          for (int i = 0; i < C::kCols / 2; ++i) {
            float x, y;
            unpack2(acc[i], x, y);
            if (2 * i < n) *o = __float2bfloat16_rn(args.accumulate ? __bfloat162float(*o) + x : x);
            o += args.lanes;
            if (2 * i + 1 < n) *o = __float2bfloat16_rn(args.accumulate ? __bfloat162float(*o) + y : y);
            o += args.lanes;
          }
        }
      }
    }
  }
  if (MODE == kSplit) {
    // the cluster barriers count every thread; warps (and CTAs) without a tile pass them here
    const bool passed = warp >= 4 && id0 < walk.total;
    __syncwarp();
    if (!passed) {
      cluster_wait();
      cluster_arrive();
      cluster_wait();
    }
  }
  // ---- teardown: all MMAs of this CTA have completed before the columns are released
  if (warp == 1 && lane == 0)
    if (!mbar_wait(mma_done, 0, kDrainBudget))
      if (args.status) atomicOr(args.status, kErrDrain);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int BN, int MODE>
cudaError_t launch_one(const CUtensorMap& p, const CUtensorMap& q, const Fp8Args& a, long long tiles,
                       cudaStream_t s) {
  using C = Fp8Cfg<BN, MODE>;
  auto kern = gemm_fp8_kernel<BN, MODE>;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), C::kSmemBytes);
  if (e != cudaSuccess) return e;
  if (MODE == kSplit)
    return launch_pdl_cluster(kern, dim3(static_cast<unsigned>(tiles * a.splits)), dim3(C::kThreads), C::kSmemBytes,
                              s, a.splits, p, q, a);
  const long long sms = sm_count();
  return launch_pdl(kern, dim3(static_cast<unsigned>(tiles < sms ? tiles : sms)), dim3(C::kThreads), C::kSmemBytes,
                    s, p, q, a);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
constexpr int kSms = 152;

}  // namespace
}  // namespace lmoe

using namespace lmoe;

extern "C" lmoe_status lmoe_matmul_fp8(const lmoe_fp8_matmul* c, const uint8_t* a, const float* a_scales,
                                       const uint8_t* w, const float* w_scales, const int32_t* offsets, void* out,
                                       uint32_t* status, cudaStream_t stream) {
  if (c == nullptr || c->rows < 0 || c->N <= 0 || c->K <= 0 || c->n_experts <= 0) return LMOE_ERR_ARG;
  if (c->a_format > LMOE_FP8_E5M2 || c->b_format > LMOE_FP8_E5M2) return LMOE_ERR_ARG;
  if (c->accumulate) return LMOE_ERR_ARG;
  if (offsets == nullptr && c->n_experts != 1) return LMOE_ERR_ARG;
  if (c->out_dtype != LMOE_F32 && c->out_dtype != LMOE_BF16) return LMOE_ERR_UNSUPPORTED;
  if (c->n_experts > kMaxGroups || c->K % 16 || c->K > (1 << 20) || c->N > (1 << 20) || c->rows > (1LL << 24))
    return LMOE_ERR_UNSUPPORTED;
  const long long wt = (c->N + 127) / 128;
  if ((c->rows / 16 + c->n_experts) * wt > 0x7fffffffLL) return LMOE_ERR_UNSUPPORTED;
  if (c->rows == 0) return LMOE_OK;
  if (a == nullptr || a_scales == nullptr || w == nullptr || w_scales == nullptr || out == nullptr)
    return LMOE_ERR_ARG;
  if (!aligned(a, 16) || !aligned(w, 16) || !aligned(a_scales, 4) || !aligned(w_scales, 4) || !aligned(offsets, 4) ||
      !aligned(status, 4) || !aligned(out, c->out_dtype == LMOE_F32 ? 4 : 2))
    return LMOE_ERR_ALIGN;

  Fp8Args g = {};
  g.rows = c->rows;
  g.lanes = c->N;
  g.num_kb = (c->K + 127) / 128;
  g.E = c->n_experts;
  g.offsets = offsets;
  g.ps = w_scales;
  g.qs = a_scales;
  g.ldq = c->rows;
  g.out = out;
  g.out_f32 = c->out_dtype == LMOE_F32;
  g.fmt_p = c->b_format;
  g.fmt_q = c->a_format;
  g.status = status;
  g.budget = kDefaultWaitBudget;
  // Column tile: the widest that the rows of an expert fill.  Up to 16 rows in all: 16.  Then by
  // the mean rows of an expert.
  const long long live = c->n_experts < c->rows ? c->n_experts : c->rows;
  const int bn = c->rows <= 16 ? 16 : (c->rows <= 64 || c->rows / c->n_experts < 48) ? 64 : 256;
  const long long tiles = ((c->rows + bn - 1) / bn + (live - 1)) * wt;   // at most
  const unsigned long long K = c->K, N = c->N;
  CUtensorMap tp, tq;
  const unsigned long long pd[3] = {K, N, static_cast<unsigned long long>(c->n_experts)}, pst[2] = {K, K * N};
  const unsigned pbox[3] = {128, 128, 1};
  const unsigned long long qd[2] = {K, static_cast<unsigned long long>(c->rows)}, qst[1] = {K};
  const unsigned qbox[2] = {128, static_cast<unsigned>(bn < 64 ? bn : 64)};
  if (!encode_u8_swizzled(&tp, w, 3, pd, pst, pbox) || !encode_u8_swizzled(&tq, a, 2, qd, qst, qbox))
    return LMOE_ERR_CUDA;
  // Few tiles: split the reduction among the CTAs of a cluster, at least four blocks each.
  int split = 1;
  if (bn < 256)
    while (split < (bn == 16 ? 8 : 4) && tiles * split * 2 <= kSms && g.num_kb / (split * 2) >= 4) split *= 2;
  g.splits = split;
  cudaError_t e;
  if (split > 1) e = bn == 16 ? launch_one<16, kSplit>(tp, tq, g, tiles, stream) : launch_one<64, kSplit>(tp, tq, g, tiles, stream);
  else if (bn == 16) e = launch_one<16, kMatmul>(tp, tq, g, tiles, stream);
  else if (bn == 64) e = launch_one<64, kMatmul>(tp, tq, g, tiles, stream);
  else e = launch_one<256, kMatmul>(tp, tq, g, tiles, stream);
  return e == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}

extern "C" lmoe_status lmoe_matmul_fp8_wgrad(const lmoe_fp8_matmul* c, const uint8_t* dy_t, const float* dy_scales,
                                             const uint8_t* x_t, const float* x_scales, const int32_t* offsets,
                                             void* dw, uint32_t* status, cudaStream_t stream) {
  if (c == nullptr || c->rows < 0 || c->rows % 128 || c->N <= 0 || c->K <= 0 || c->n_experts <= 0) return LMOE_ERR_ARG;
  if (c->a_format > LMOE_FP8_E5M2 || c->b_format > LMOE_FP8_E5M2) return LMOE_ERR_ARG;
  if (offsets == nullptr && c->n_experts != 1) return LMOE_ERR_ARG;
  if (c->out_dtype != LMOE_F32 && c->out_dtype != LMOE_BF16) return LMOE_ERR_UNSUPPORTED;
  if (c->n_experts > kMaxGroups || c->K > (1 << 20) || c->N > (1 << 20) || c->rows > (1LL << 24))
    return LMOE_ERR_UNSUPPORTED;
  const long long lt = (c->K + 127) / 128, ct = (c->N + 255) / 256, tiles = lt * ct * c->n_experts;
  if (tiles > 0x7fffffffLL) return LMOE_ERR_UNSUPPORTED;
  const int ob = c->out_dtype == LMOE_F32 ? 4 : 2;
  if (dw == nullptr) return LMOE_ERR_ARG;
  if (!aligned(dw, ob)) return LMOE_ERR_ALIGN;
  if (c->rows == 0) {
    if (c->accumulate) return LMOE_OK;
    const size_t bytes = static_cast<size_t>(c->n_experts) * c->N * c->K * ob;
    return cudaMemsetAsync(dw, 0, bytes, stream) == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
  }
  if (dy_t == nullptr || dy_scales == nullptr || x_t == nullptr || x_scales == nullptr) return LMOE_ERR_ARG;
  if (!aligned(dy_t, 16) || !aligned(x_t, 16) || !aligned(dy_scales, 4) || !aligned(x_scales, 4) ||
      !aligned(offsets, 4) || !aligned(status, 4))
    return LMOE_ERR_ALIGN;

  Fp8Args g = {};
  g.rows = c->rows;
  g.lanes = c->K;
  g.cols = c->N;
  g.E = c->n_experts;
  g.offsets = offsets;
  g.ps = x_scales;
  g.qs = dy_scales;
  g.ldq = c->N;
  g.out = dw;
  g.out_f32 = c->out_dtype == LMOE_F32;
  g.accumulate = c->accumulate;
  g.fmt_p = c->b_format;
  g.fmt_q = c->a_format;
  g.status = status;
  g.budget = kDefaultWaitBudget;
  g.splits = 1;
  const unsigned long long R = static_cast<unsigned long long>(c->rows);
  CUtensorMap tp, tq;
  const unsigned long long pd[2] = {R, static_cast<unsigned long long>(c->K)};
  const unsigned long long qd[2] = {R, static_cast<unsigned long long>(c->N)}, st[1] = {R};
  const unsigned pbox[2] = {128, 128}, qbox[2] = {128, 64};
  if (!encode_u8_swizzled(&tp, x_t, 2, pd, st, pbox) || !encode_u8_swizzled(&tq, dy_t, 2, qd, st, qbox))
    return LMOE_ERR_CUDA;
  return launch_one<256, kWgrad>(tp, tq, g, tiles, stream) == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}
