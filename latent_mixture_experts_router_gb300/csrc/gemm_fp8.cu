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
// (8192 a cycle): half the time.
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
  int out_vec;           // bf16: 16-byte stores fit the output's base and rows
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
  static constexpr int kStageCols = 16;               // columns of one pass of the bf16 store
  static constexpr int kOutBytes = kEpiWarps * kStageCols * 64;
  static constexpr int kTableBytes = 3 * (kMaxGroups + 4) * 4;
  static constexpr int kFixed = kRedBytes + kSlots * BN * 4 + kOutBytes + kTableBytes + 512 + 1024;
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
// 16 lanes x 8 N columns: thread l gets, per 8 columns, columns 2 (l % 4), + 1 of lanes l / 4
// (registers 0, 1) and l / 4 + 8 (registers 2, 3).
LMOE_DEV void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
LMOE_DEV void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
// d += (value read from TMEM) * s, and (value) *= s: volatile, so that the compiler keeps them
// behind the wait for the read that the value comes from.
LMOE_DEV void fma_acc(float& d, uint32_t v, float s) {
  asm volatile("fma.rn.f32 %0, %1, %2, %0;" : "+f"(d) : "r"(v), "f"(s));
}
LMOE_DEV void scale_in_place(uint32_t& v, float s) { asm volatile("mul.rn.f32 %0, %0, %1;" : "+r"(v) : "f"(s)); }
// Stores four 8 x 8 matrices of 16-bit values transposed: thread l names the 16-byte row l % 8
// of matrix l / 8; matrix m's elements (row t / 4, columns 2 (t % 4), + 1) are thread t's r[m].
LMOE_DEV void stmatrix_x4_trans(uint32_t saddr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
// Registers of a warpgroup (all four of its warps).  256-column tiles: the epilogue's two
// warpgroups hold 128 accumulators a thread; 4 x 32 x 56 + 8 x 32 x 224 = 384 x 168, what the
// block was launched with.
template <int N>
LMOE_DEV void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
LMOE_DEV void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
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
  uint8_t* stage_out = reinterpret_cast<uint8_t*>(red) + C::kRedBytes;
  float* sc = reinterpret_cast<float*>(stage_out + C::kOutBytes);   // [kSlots][BN]
  int* start = reinterpret_cast<int*>(sc + C::kSlots * BN);         // [E + 1], then lo, hi
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
  if constexpr (BN == 256) regs_dec<56>();
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
    // ---- column scales (times the lane block's scale where there is one), the loads of
    // several blocks in flight at a time
    constexpr int kPer = (BN + 31) / 32, kBatch = BN == 256 ? 2 : 4;
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
    // ---- epilogue.  A TMEM read in the 16 x 256-bit shape gives a thread two columns of four
    // lanes per 8 columns, so that it needs two of their scales, not eight: with a lane's whole
    // row per thread every scale goes to every thread, and returning those from shared memory
    // (128 bytes a cycle) takes twice the MMAs' time.
    if constexpr (BN == 256) regs_inc<224>();
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const int r = quad * 32 + (lane >> 2);                 // lanes r, + 8, + 16, + 24 of the tile
    const int c0 = half * C::kCols, cl = (lane & 3) * 2;   // columns c0 + 8 g + cl, + 1
    const uint32_t tq = tmem + (static_cast<uint32_t>(quad * 32) << 16) + c0;
    constexpr int kChC = C::kCols >= 64 ? 64 : 16;         // columns of one TMEM read
    constexpr int kG = kChC / 8, kN = C::kCols / kChC * 2;
    int it = 0;
    bool ok = true;
    for (int id = id0; ok && id < walk.total; id += step) {
      // (the tile is worked out again for the stores: its registers are the accumulators' here)
      int kb, kb1;
      const float* ps = nullptr;   // wgrad: scale of this thread's first lane in the next block
      int left = 0;                // lanes of the operand from there on
      {
        const Fp8Tile t = tile_at<BN, MODE>(walk, args, id, rank);
        kb = t.kb0;
        kb1 = t.kb1;
        if (MODE == kWgrad) {
          ps = args.ps + static_cast<long long>(kb) * args.lanes + t.p0 + r;
          left = args.lanes - t.p0 - r;
        }
      }
      // acc[g][j][u]: column u of group g's pair, lane 8 j + l / 4 of the warp's 32
      float acc[C::kCols / 8][4][2];
#pragma unroll
      for (int i = 0; i < C::kCols; ++i) acc[i >> 3][(i >> 1) & 3][i & 1] = 0.f;
      float sp_next[4] = {};
      if (MODE == kWgrad && kb < kb1) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (8 * j < left) sp_next[j] = ps[8 * j];
      }
      uint32_t v[2][kG * 4];
      // waits for block `i` of the ring and reads its first columns
      const auto begin = [&](int i) {
        const int buf = i % C::kBufs, s = i % C::kSlots;
        if (!mbar_wait(&sfull[s], (i / C::kSlots) & 1, budget) ||
            !mbar_wait(&acc_full[buf], (i / C::kBufs) & 1, budget)) {
          if (args.status) atomicOr(args.status, kErrWaitEpilogue);
          return false;
        }
        tc_fence_after();
        tmem_ld_frag(tq + buf * BN, v[0]);
        return true;
      };
      for (; kb < kb1; ++kb, ++it) {
        ok = begin(it);
        if (!ok) break;
        tmem_ld_wait();
        float sp[4];
        if (MODE == kWgrad) {
          ps += args.lanes;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            sp[j] = sp_next[j];
            if (kb + 1 < kb1 && 8 * j < left) sp_next[j] = ps[8 * j];
          }
        }
        const int s = it % C::kSlots;
        const float* scs = sc + s * BN + c0 + cl;
#pragma unroll
        for (int ch = 0; ch < kN; ++ch) {   // 16 lanes x kChC columns: lane half ch % 2
          const int h = ch & 1, g0 = (ch >> 1) * kG;
          // the next read is under way while these columns are added: of this block, or, every
          // column of its buffer having been read, the first of the next block's
          if (ch + 1 < kN) {
            tmem_ld_frag(tq + (it % C::kBufs) * BN + ((ch + 1) >> 1) * kChC + (((ch + 1) & 1) ? (16u << 16) : 0u),
                         v[(ch + 1) & 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[it % C::kBufs]);
          }
#pragma unroll
          for (int g = 0; g < kG; ++g) {
            const float2 s2 = *reinterpret_cast<const float2*>(scs + (g0 + g) * 8);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t *w = &v[ch & 1][4 * g + 2 * q];
              if (MODE == kWgrad) {
                scale_in_place(w[0], sp[2 * h + q]);
                scale_in_place(w[1], sp[2 * h + q]);
              }
              float(&d)[2] = acc[g0 + g][2 * h + q];
              fma_acc(d[0], w[0], s2.x);
              fma_acc(d[1], w[1], s2.y);
            }
          }
          if (ch + 1 < kN) tmem_ld_wait();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sempty[s]);
      }
      if (MODE == kSplit) {
        // one tile per cluster: the accumulators of ranks 1.. go to rank 0 (element i of thread x
        // at i * 128 + x: threads beside each other, words beside each other)
        const int tid = threadIdx.x - 128;
        if (rank > 0) {
          cluster_wait();
          const uint32_t dst = cluster_map(smem_u32(red + (rank - 1) * BN * 128 + tid), 0);
#pragma unroll
          for (int i = 0; i < C::kCols; ++i) cluster_store(dst + i * 512, acc[i >> 3][(i >> 1) & 3][i & 1]);
          cluster_arrive();
          cluster_wait();
        } else {
          cluster_wait();
          cluster_arrive();
          cluster_wait();
          for (int q = 1; q < S; ++q) {
            const float* src = red + (q - 1) * BN * 128 + tid;
#pragma unroll
            for (int i = 0; i < C::kCols; ++i) acc[i >> 3][(i >> 1) & 3][i & 1] += src[i * 128];
          }
        }
      }
      const Fp8Tile t = tile_at<BN, MODE>(walk, args, id, rank);
      if (!ok || rank != 0 || (args.accumulate && t.kb0 == t.kb1)) continue;
      const int n = min(C::kCols, t.ncols - c0);   // live columns (may be negative)
      if (!args.out_f32 && !args.accumulate) {
        // bf16: 16 columns at a time through this warp's shared memory, transposed there: a store
        // instruction then writes 64 bytes (32 lanes' values) of each of 8 columns (rows of the
        // output).  16-byte chunk i of column c is at place i ^ (c / 2 % 4): no bank conflicts
        // either way.
        uint8_t* so = stage_out + (warp - 4) * C::kStageCols * 64;
        const int left_n = args.lanes - t.p0 - quad * 32 - (lane & 3) * 8;   // of this thread's chunk
        __nv_bfloat16* o = static_cast<__nv_bfloat16*>(args.out) + t.out + quad * 32 + (lane & 3) * 8 +
                           static_cast<long long>(c0 + (lane >> 2)) * args.lanes;
#pragma unroll
        for (int g = 0; g < C::kCols / 8; g += 2) {
          if (8 * g >= n) break;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(acc[g + u][j][0], acc[g + u][j][1]);
            const int c = 8 * u + (lane & 7), chunk = lane >> 3;
            stmatrix_x4_trans(smem_u32(so + c * 64 + ((chunk ^ ((c >> 1) & 3)) << 4)), w);
          }
          __syncwarp();
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int c = 8 * u + (lane >> 2), chunk = lane & 3;
            const uint4 q = *reinterpret_cast<const uint4*>(so + c * 64 + ((chunk ^ ((c >> 1) & 3)) << 4));
            if (8 * g + c < n && left_n > 0) {
              if (args.out_vec) {
                *reinterpret_cast<uint4*>(o) = q;
              } else {
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  if (i < left_n) o[i] = __ushort_as_bfloat16(static_cast<unsigned short>(w[i >> 1] >> (16 * (i & 1))));
              }
            }
            o += 8LL * args.lanes;
          }
          __syncwarp();
        }
      } else {
        // fp32: a store instruction writes 8 lanes' words of 4 columns: whole 32-byte sectors
#pragma unroll
        for (int g = 0; g < C::kCols / 8; ++g)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int c = 8 * g + cl + u;
            if (c >= n) continue;
            const long long base = t.out + static_cast<long long>(c0 + c) * args.lanes + r;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (t.p0 + r + 8 * j >= args.lanes) continue;
              const float val = acc[g][j][u];
              if (args.out_f32) {
                float* o = static_cast<float*>(args.out) + base + 8 * j;
                *o = args.accumulate ? *o + val : val;
              } else {
                __nv_bfloat16* o = static_cast<__nv_bfloat16*>(args.out) + base + 8 * j;
                *o = __float2bfloat16_rn(__bfloat162float(*o) + val);
              }
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
  g.out_vec = aligned(out, 16) && c->N % 8 == 0;
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
  g.out_vec = aligned(dw, 16) && c->K % 8 == 0;
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
