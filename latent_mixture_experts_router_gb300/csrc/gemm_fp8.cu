// gemm_fp8.cu — products of 8-bit floating-point operands with one fp32 scale per block of 128
// along the reduction, on the 5th-generation tensor cores, persistent.
//
//   matmul  y[r, n]     = sum_b as[b, r] ws[n / 128, b] sum_{k in block b} a[r, k] w[e, n, k]
//           for the rows r of expert e (offsets[e] <= r < offsets[e + 1]), or of one matrix
//   wgrad   dw[e, n, k] = sum_{b of e} dys[b, n] xs[b, k] sum_{r in block b} dy[n, r] x[k, r]
//           with expert e's rows padded to whole blocks of 128
//
// The scales are arbitrary fp32 numbers, which the tensor cores' own block scaling (powers of two per 32)
// does not take; scales that are powers of two go the same way.  So the tensor cores compute one block of
// 128 at a time into one of several TMEM buffers, and the epilogue warps add buffer x scales to fp32
// accumulators in registers while the next block's MMAs run.  Adding a 128 x 256 block takes 128 x 256 fused
// multiply-adds on the CUDA cores (128 a cycle) beside 128 x 256 x 128 on the tensor cores (8192 a cycle):
// half the time.
//
// Measured on normally distributed operands, other inputs in each call: 32768 rows over 64 experts of 4096 x 4096
// 592 us (1.86 PFLOP/s; an eighth are ragged tiles; 506 with small codes, which take less power), 2047 x 8192 x
// 4096 to fp32 78.6 us (1.75), 8 rows over 64 experts 24.1 us, weight gradients of 8192 rows over 16
// experts of 4096 x 2048 223 us, of 1000 rows by 4096 x 8192 78.0 us.  Small codes: 8192 x 8192 x 16384 888 us,
// 2560 rows over 64 experts 178.6 us (6.2 TB/s: the weights).  Many rows: bound by the tensor cores' reads of
// operands and the round trip of the two TMEM buffers.  Weight gradients: by the epilogue's arithmetic and
// waits (without MMAs and loads 411 of 454 us at 16384 x 4096 x 4096) and its stores.
//
// Which operand is the MMA's 128 lanes ("lane operand") and which its columns:
//   kRows   rows of a are lanes, rows of w columns (128 x 256 tiles): many rows per expert.  A thread
//           holds one lane, so its scale as ws is one register for 128 columns.
//   kCols   rows of w are lanes, rows of a columns: the column count is any multiple of 16, so an
//           expert with 20 rows costs 32 columns, not a 128-row tile, and one token costs 16.
//   kSplit  kCols where the tiles are few (a few tokens): a cluster of S CTAs computes one tile,
//           each a range of the blocks; the others leave their sums in the first one's shared
//           memory, which adds them in rank order.
//   kWgrad  rows of x_t are lanes, rows of dy_t columns; both have scales of their own.
//
// Roles of a CTA: warp 0 lane 0 TMA producer; lane 0 of warps 1 and 3 MMA issuers (warp 1 owns the TMEM);
// warp 2 stages the scales of each block in shared memory; warps 4.. epilogue, warp w on TMEM lanes
// 32 (w % 4) .. (and column half (w - 4) / 4 with eight of them).  A finished tile passes
// through shared memory on its way out, so that a store instruction writes whole rows (bulk copies of
// single rows, 256 or 512 bytes, take the copy engine about 60 cycles each: 9000 cycles a tile).
#include <mutex>

#include "../../include/latent_moe.h"
#include "internal.h"
#include "ptx.cuh"

namespace lmoe {
namespace {

enum Fp8Mode : int { kCols = 0, kWgrad = 1, kSplit = 2, kRows = 3 };
constexpr int kMaxGroups = 1024;
constexpr int kMaxSplit = 8;

// Division of n < 2^31 by a fixed d, by a multiplication (Granlund and Montgomery 1994): the walk of
// the tiles divides several times for each, and a division takes a thread beside busy ones hundreds
// of cycles.
struct FastDiv {
  unsigned d, mul, shift;
  __host__ static FastDiv of(unsigned d) {
    unsigned shift = 0;
    while ((1ull << shift) < d) ++shift;
    return {d, static_cast<unsigned>(((1ull << 32) * ((1ull << shift) - d)) / d + 1), shift};
  }
  __device__ __forceinline__ int div(int n) const {
    return static_cast<int>((__umulhi(static_cast<unsigned>(n), mul) + static_cast<unsigned>(n)) >> shift);
  }
  __device__ __forceinline__ int mod(int n) const { return n - div(n) * static_cast<int>(d); }
};

struct Fp8Args {
  FastDiv by_others, by_group, by_E;   // tiles across; kRasterGroup rows of them; experts
  long long rows;        // matmul: rows of a and y; wgrad: columns of dy_t and x_t (a multiple of 128)
  int n, k;              // matmul: rows of w; wgrad: rows of dy_t and of x_t
  int num_kb;            // matmul: blocks of the reduction
  int E;
  const int32_t* offsets;   // [E + 1], or nullptr: one group of all rows
  const float* ps;       // scales of the lane operand
  const float* qs;       // scales of the column operand
  void* out;
  int ldo;               // elements of an output row
  int out_f32, accumulate;
  int out_vec;           // output rows start on 16 bytes: 16-byte stores
  unsigned fmt_p, fmt_q;   // 0 e4m3, 1 e5m2
  unsigned* status;      // error word, or nullptr: the device's own (g_status)
  long long budget;
  int cap;               // rows that offsets are clamped to
  int box;               // kCols, kSplit: rows of a that a tile loads
  int splits;            // kSplit: CTAs per tile (the cluster size)
  float far;             // the largest as ws 2^64 (matmul), p s (wgrad) with which no sum times 2^64 leaves fp32's range
};

// What waits that gave up leave for lmoe_fp8_check_status where the caller has no word for it.
__device__ unsigned g_status, g_status_taken;
__global__ void take_status_kernel() {
  griddep_enter();
  g_status_taken = atomicExch(&g_status, 0u);
}

template <int BN, int MODE>
struct Fp8Cfg {
  static constexpr int kEpiWarps = BN == 256 ? 8 : 4;
  static constexpr int kAcc = BN * 4 / kEpiWarps;   // accumulator columns of one thread's warpgroup
  static constexpr int kThreads = 128 + 32 * kEpiWarps;
  // CTAs of an SM, and the registers of the producers' and the epilogue's warpgroups (0: as launched)
  static constexpr int kCtas = MODE == kWgrad ? 2 : 1;
  static constexpr int kDec = BN == 256 ? 56 : MODE == kWgrad ? 40 : 0;
  static constexpr int kInc = BN == 256 ? 224 : MODE == kWgrad ? 216 : 0;
  static constexpr int kPBytes = 128 * 128;
  static constexpr int kQBytes = BN * 128;
  static constexpr int kStageBytes = kPBytes + kQBytes;
  static constexpr int kSlots = 8;                    // staged scale blocks
  static constexpr int kBufs = BN >= 128 ? 2 : 8;     // TMEM buffers
  static constexpr uint32_t kTmemCols = BN * kBufs;
  static constexpr int kMaxS = BN == 16 ? kMaxSplit : 4;
  static constexpr int kRedBytes = MODE == kSplit ? (kMaxS - 1) * BN * 128 * 4 : 0;
  // output staging of a warpgroup: kAcc columns of 128 bf16, or kOutCols of 128 fp32 at a time (kRows:
  // 128 rows of 128 bf16 or of 64 fp32), each with 16 bytes of padding against bank conflicts
  static constexpr int kOutCols = kAcc >= 64 ? kAcc / 2 : kAcc;
  static constexpr int kOutBytes = MODE == kRows ? 128 * 272 : kAcc * 272 > kOutCols * 528 ? kAcc * 272 : kOutCols * 528;
  static constexpr int kTableBytes = (kMaxGroups + 4) * 4 + (MODE == kRows ? 16 * 16 : MODE == kWgrad ? 4 * 48 : 0);
  // floats of one: columns' (lanes') scales, their mark, and (few columns) the scales as they are
  static constexpr int kSlotLd = BN <= 64 ? 2 * BN + 4 : BN + 4;
  static constexpr int kFixed = kRedBytes + kSlots * kSlotLd * 4 + kOutBytes * (kEpiWarps / 4) + kTableBytes + 512 + 1024;
  static constexpr int kStagesFit = ((kCtas == 2 ? 113 : 227) * 1024 - kFixed) / kStageBytes;
  // an odd number of stages, no more than the TMEM buffers, would break the MMA issuers' waits
  static constexpr int kStagesMost = kStagesFit > 11 ? 11 : kStagesFit;
  static constexpr int kStages = kStagesMost % 2 && kStagesMost <= kBufs ? kStagesMost - 1 : kStagesMost;
  static constexpr int kSmemBytes = kFixed + kStages * kStageBytes;
  static_assert(kStages >= 2, "pipeline depth");
  static_assert((kStages % 2 == 0 || kStages > kBufs) && kBufs % 2 == 0, "two MMA issuers");
  static_assert((2 * kStages + 2 * kBufs + 2 * kSlots + 2 * 4 + 1) * 8 + 8 <= 512, "barriers");
  static_assert((BN == 256) == (MODE == kRows) && (BN == 128) == (MODE == kWgrad), "tile widths");
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
LMOE_DEV void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
LMOE_DEV void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
LMOE_DEV void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
// d += (value read from TMEM) * s: volatile, so that the compiler keeps it behind the wait for the
// read that the value comes from.
LMOE_DEV void fma_acc(float& d, uint32_t v, float s) {
  asm volatile("fma.rn.f32 %0, %1, %2, %0;" : "+f"(d) : "r"(v), "f"(s));
}
// the same for two neighbouring columns, and scaled by p as well: d += (v p) s
LMOE_DEV void fma_pair(uint64_t& d, uint32_t v0, uint32_t v1, uint64_t s) {
  asm volatile("{\n\t.reg .b64 t;\n\tmov.b64 t, {%1, %2};\n\tfma.rn.f32x2 %0, t, %3, %0;\n\t}"
               : "+l"(d)
               : "r"(v0), "r"(v1), "l"(s));
}
LMOE_DEV void fma_pair(uint64_t& d, uint32_t v0, uint32_t v1, uint64_t p, uint64_t s) {
  asm volatile(
      "{\n\t.reg .b64 t;\n\tmov.b64 t, {%1, %2};\n\t"
      "mul.rn.f32x2 t, t, %3;\n\t"
      "fma.rn.f32x2 %0, t, %4, %0;\n\t}"
      : "+l"(d)
      : "r"(v0), "r"(v1), "l"(p), "l"(s));
}
LMOE_DEV uint64_t pack2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
LMOE_DEV void unpack2(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }

// Far scales.  A block's sum v is 0 or between 2^-32 and 2^39 in magnitude (the smallest and the largest
// product of two codes, 128 of them), so v as ws may be a normal number where as ws is not: a block of
// zeros has the scale 2^-126, tiny gradients come close to it.
//
// So sums are held lifted, times 2^64, and the factor staged for v is as ws 2^64 (wgrad: p 2^64 and s, one after
// the other): it has all its bits from as ws = 2^-190 on, below which v as ws is less than the smallest
// number.  Up to Fp8Args::far no lifted sum leaves the range at its other end.  A block with a larger
// product has a mark beside its scales: matmul then finds them there as they are, and ws in the mark (wgrad:
// always its largest s).  From a larger product on a sum is held as it is, or lowered by 2^64 if even that is too
// large: a row's sums in kRows, a column's in kCols and kSplit, a lane's in wgrad, so that far scales of one
// do not cost the others' small sums (its own blocks with small products then count down to 2^-111, or
// 2^-47; a lane's columns of wgrad share that).  wgrad multiplying p s first would need no rule for large p,
// but takes 411 us instead of 383 at 16384 x 4096 x 4096.  Sums are brought back when they are stored.
// Measured with it and with as ws as one factor of sums as they are: 32768 rows over 64 experts of 4096 x 4096
// 506 us and 506, 16384 rows by 8192 x 8192 888 and 891, 2560 rows over 64 experts 177.6 and 174.8, 100 rows by 8192 x
// 8192 24.3 and 22.9, 8 rows over 64 experts 28.1 and 27.8.
constexpr float kFarLane = 0x1p24f;   // wgrad: of p, so that v p 2^64 stays below 2^127
constexpr float kLift = 0x1p64f, kFloatMax = 3.402823466e38f;
// what a sum is held times, as the exponent field of a power of two: 2^64, 1, 2^-64
enum Held : unsigned { kLifted = 127 + 64, kAsIs = 127, kLowered = 127 - 64 };
LMOE_DEV float held_times(unsigned h) { return __uint_as_float(h << 23); }
LMOE_DEV float held_back(unsigned h) { return __uint_as_float((254 - h) << 23); }
// lowers h to `to` and returns what its sums are multiplied by
LMOE_DEV float held_lower(unsigned& h, unsigned to) {
  if (to >= h) return 1.f;
  const float f = h - to == 64 ? 0x1p-64f : 0x1p-128f;
  h = to;
  return f;
}
LMOE_DEV bool finite(float v) { return fabsf(v) <= kFloatMax; }
// matmul: as ws of a marked block in the unit h of its sums, which may be lowered for it: f is what they are
// multiplied by.  Each multiple of 2 goes where it does not leave the range before the product does.
LMOE_DEV float marked_product(float a, float b, unsigned& h, float far, float& f) {
  const float p = fabsf(a) < 1.f ? (a * kLift) * b : a * (b * kLift);
  f = 1.f;
  if (!finite(a) || !finite(b)) return a * b;   // (infinities and NaN are what they are in any unit)
  if (fabsf(p) > far) f = held_lower(h, fabsf(a * b) < 0x1p127f ? kAsIs : kLowered);
  // (lowered, past 2^191: any factor so large brings any v but 0 out of range)
  return h == kLifted ? p : h == kAsIs ? a * b : fminf(fmaxf((a * 0x1p-32f) * (b * 0x1p-32f), -kFloatMax), kFloatMax);
}
LMOE_DEV void scale_pair(uint64_t& d, float x, float y) {
  asm volatile("mul.rn.f32x2 %0, %0, %1;" : "+l"(d) : "l"(pack2(x, y)));
}
// Stores four 8 x 8 matrices of 16-bit values transposed: thread l names the 16-byte row l % 8
// of matrix l / 8; matrix m's elements (row t / 4, columns 2 (t % 4), + 1) are thread t's r[m].
LMOE_DEV void stmatrix_x4_trans(uint32_t saddr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
// Registers of a warpgroup (all four of its warps).  The epilogue's warpgroups hold 128
// accumulators a thread; 4 x 32 x 56 + 8 x 32 x 224 = 384 x 168, or 4 x 32 x 40 + 4 x 32 x 216 = 256 x
// 128, is what the block was launched with.
template <int N>
LMOE_DEV void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
LMOE_DEV void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

LMOE_DEV void named_barrier(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// The same barrier, with whether every thread's `ok` is set.
LMOE_DEV bool named_barrier_all(int id, int threads, bool ok) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %3, 0;\n\t"
      "bar.red.and.pred q, %1, %2, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"(static_cast<int>(ok))
      : "memory");
  return r != 0;
}
// mbar_wait of a whole warp, with one outcome: its lanes' own waits may give up one by one, and TMEM reads,
// votes and warp barriers follow that need all of them.
LMOE_DEV bool warp_wait(uint64_t* bar, uint32_t parity, long long budget) {
  return __all_sync(~0u, mbar_wait(bar, parity, budget));
}
// Rows of group e, clamped into the rows there are, so that no offsets send a load or a store out
// of range.
LMOE_DEV void group_rows(const Fp8Args& a, int e, int& lo, int& hi) {
  const int cap = a.cap;
  lo = 0;
  hi = cap;
  if (a.offsets != nullptr) {
    lo = min(max(a.offsets[e], 0), cap);
    hi = min(max(a.offsets[e + 1], lo), cap);
  }
}

// The tiles of a launch, the same walk for every role.  start[e] (shared memory): the first row
// tile of group e (matmul) or its first block (wgrad).
struct Fp8Walk {
  const int* start;
  int E, others, total;   // others: tiles across, per row tile; wgrad: lane tiles
  int cols;               // wgrad: column tiles
};
struct Fp8Tile {
  int e, p0, q0, ncols, lanes, kb0, kb1;   // lanes, ncols: live ones
  int skip;        // kCols, kSplit: columns before the first live one (of another expert, not stored)
  long long out;   // kRows: element offset of (first lane, first column), else of (column, lane)
};

// kRows: what the epilogue needs of a tile for its stores, left in shared memory by the scale warp,
// which is at most kSlots blocks (and so tiles) ahead
struct Fp8Info {
  long long out;
  int lanes, ncols;
};
constexpr int kInfos = 16;
// kWgrad: whole tiles by the same way, in a ring with barriers of its own (a tile may have no
// block).  Working one out takes an epilogue thread 1500 cycles, six divisions beside the others'
// arithmetic.
constexpr int kTileRing = 4;

// grouped_tile (ptx.cuh) without its divisions: tile i of `rows` x by_others.d tiles
__constant__ unsigned g_ceil_recip[kRasterGroup] = {   // ceil(2^32 / d): exact quotients below 2^28
    0, 0, 0x80000000u, 0x55555556u, 0x40000000u, 0x33333334u, 0x2aaaaaabu, 0x24924925u,
    0x20000000u, 0x1c71c71du, 0x1999999au, 0x1745d175u, 0x15555556u, 0x13b13b14u, 0x12492493u, 0x11111112u};
LMOE_DEV void raster(const Fp8Args& a, int i, int rows, int& row, int& other) {
  const int g = a.by_group.div(i), first = g * kRasterGroup, gm = min(kRasterGroup, rows - first);
  const int local = i - g * static_cast<int>(a.by_group.d);
  other = gm == kRasterGroup ? local / kRasterGroup
          : gm == 1          ? local
                             : static_cast<int>(__umulhi(static_cast<unsigned>(local), g_ceil_recip[gm]));
  row = first + local - other * gm;
}

template <int BN, int MODE>
LMOE_DEV Fp8Tile tile_at(const Fp8Walk& w, const Fp8Args& a, int id, int rank) {
  Fp8Tile t;
  int ot, rt;
  if (MODE == kWgrad) {
    // The experts take turns, tile by tile, in an order that shifts: CTAs side by side then have tiles
    // of more and of fewer blocks, and some store while others compute (all at once, the stores of
    // a wave of tiles fill L2 and wait for memory).
    const int i = a.by_E.div(id);
    t.e = a.by_E.mod(id - i * w.E + i + a.by_E.div(i));
    raster(a, i, w.cols, rt, ot);
    t.p0 = ot * 128;
    t.q0 = rt * BN;
    t.ncols = min(BN, a.n - t.q0);
    t.skip = 0;
    t.lanes = a.k - t.p0;
    t.kb0 = w.start[t.e];
    t.kb1 = w.start[t.e + 1];
    t.out = (static_cast<long long>(t.e) * a.n + t.q0) * a.ldo + t.p0;
    return t;
  }
  int l = 0, h = w.E, lo, hi;   // the last e with start[e] * others <= id
  const int s = a.by_others.div(id);
  while (h - l > 1) {
    const int m = (l + h) >> 1;
    if (w.start[m] <= s) l = m;
    else h = m;
  }
  t.e = l;
  raster(a, id - w.start[l] * w.others, w.start[l + 1] - w.start[l], rt, ot);
  group_rows(a, l, lo, hi);
  t.kb0 = 0;
  t.kb1 = a.num_kb;
  if (MODE == kRows) {
    t.p0 = lo + rt * 128;
    t.q0 = ot * BN;
    t.skip = 0;
    t.lanes = hi - t.p0;
    t.ncols = min(BN, a.n - t.q0);
    t.out = static_cast<long long>(t.p0) * a.ldo + t.q0;
  } else {
    // No row behind the last is asked for: a box that reaches past the end, filled with zeros
    // there, costs the copy engine far more than rows do (20 rows of 8 experts, 4096 x 4096: 61 us, so 26).  A
    // tile near the end starts earlier instead and skips the columns before its own.
    t.p0 = ot * 128;
    const int q0 = lo + rt * BN;
    t.q0 = min(q0, static_cast<int>(a.rows) - a.box);
    t.skip = q0 - t.q0;
    t.lanes = a.n - t.p0;
    t.ncols = t.skip + min(BN, hi - q0);   // <= box
    t.out = static_cast<long long>(t.q0) * a.ldo + t.p0;
    if (MODE == kSplit) {
      t.kb0 = static_cast<int>(static_cast<long long>(a.num_kb) * rank / a.splits);
      t.kb1 = static_cast<int>(static_cast<long long>(a.num_kb) * (rank + 1) / a.splits);
    }
  }
  return t;
}

// Row tiles of `unit` rows that any split of `rows` among E experts takes at most (rows > 0).
__host__ __device__ constexpr int most_tiles(int rows, int E, int unit) {
  return (rows + unit - 1) / unit + (E < rows ? E : rows) - 1;
}

// What an epilogue thread needs to wait for the blocks of its tile.
template <int BN, int MODE>
struct Fp8Ring {
  using C = Fp8Cfg<BN, MODE>;
  uint64_t *acc_full, *acc_empty, *sempty;
  unsigned* status;
  long long budget;
  // the block's products are in their buffer, and its scales staged (the MMA issuer waits for them)
  LMOE_DEV bool wait(int it) const {
    const bool ok = warp_wait(&acc_full[it % C::kBufs], (it / C::kBufs) & 1, budget);
    if (!ok) atomicOr(status, kErrWaitEpilogue);
    tc_fence_after();
    return ok;
  }
  // the warp has read the TMEM buffer / the scales / both
  LMOE_DEV void buffer_read(int it, int lane) const {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&acc_empty[it % C::kBufs]);
  }
  LMOE_DEV void scales_read(int it, int lane) const {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sempty[it % C::kSlots]);
  }
  LMOE_DEV void both_read(int it, int lane) const {
    buffer_read(it, lane);
    if (lane == 0) mbar_arrive(&sempty[it % C::kSlots]);
  }
};

// ---- epilogue of kRows: a thread owns lane (row) r and 128 columns
template <int BN>
LMOE_DEV void epilogue_rows(const Fp8Args& args, const Fp8Walk& walk, const Fp8Ring<BN, kRows>& ring, const float* sc,
                            const Fp8Info* infos, uint8_t* stage_out, uint32_t tmem, int id0, int step) {
  using C = Fp8Cfg<BN, kRows>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = warp & 3, half = (warp - 4) >> 2, r = quad * 32 + lane;
  const uint32_t tq = tmem + (static_cast<uint32_t>(quad * 32) << 16) + half * 128;
  uint8_t* mine = stage_out + half * C::kOutBytes + quad * 32 * 272;
  int it = 0;
  bool ok = true;
  int tile = 0;
  for (int id = id0; ok && id < walk.total; id += step, ++tile) {
    float acc[128];
#pragma unroll
    for (int i = 0; i < 128; ++i) acc[i] = 0.f;
    unsigned held = kLifted;   // this thread's sums
    for (int kb = 0; kb < args.num_kb; ++kb, ++it) {
      ok = ring.wait(it);
      if (!ok) break;
      const uint32_t tb = tq + (it % C::kBufs) * BN;
      uint32_t v[2][32];
      tmem_ld_32cols(tb, v[0]);
      float s = sc[(it % C::kSlots) * C::kSlotLd + half * 128 + r];
      const float2 ws = *reinterpret_cast<const float2*>(sc + (it % C::kSlots) * C::kSlotLd + BN);   // the mark
      tmem_ld_wait();
      if (ws.x != 0.f || ws.y != 0.f) {   // (the same for the CTA)
        float f;
        s = marked_product(s, half ? ws.y : ws.x, held, args.far, f);
#pragma unroll
        for (int i = 0; i < 128; ++i) acc[i] *= f;
      } else {
        s *= held_times(held) * 0x1p-64f;
      }
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) {
        if (ch < 3) tmem_ld_32cols(tb + (ch + 1) * 32, v[(ch + 1) & 1]);
        else ring.both_read(it, lane);
#pragma unroll
        for (int i = 0; i < 32; ++i) fma_acc(acc[ch * 32 + i], v[ch & 1][i], s);
        if (ch < 3) tmem_ld_wait();
      }
    }
    const float back = held_back(held);
    const Fp8Info t = infos[tile % kInfos];   // written before the tile's first scales
    const int n = min(128, t.ncols - half * 128);   // live columns (may be negative)
    if (ok && n > 0) {   // (the same for the warp)
      // the warp's 32 rows through its own shared memory, 256 bytes of each at a time: a thread
      // writes its row, a store instruction takes two rows
      const long long base = t.out + static_cast<long long>(quad * 32) * args.ldo + half * 128;
      const int rows = min(32, t.lanes - quad * 32);
      const int es = args.out_f32 ? 4 : 2, rounds = args.out_f32 ? 2 : 1;
#pragma unroll
      for (int round = 0; round < 2; ++round) {
        if (round >= rounds) break;
        if (args.out_f32) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float* a = acc + round * 64 + 4 * i;
            *reinterpret_cast<float4*>(mine + lane * 272 + 16 * i) =
                make_float4(a[0] * back, a[1] * back, a[2] * back, a[3] * back);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float* a = acc + 8 * i;
            *reinterpret_cast<uint4*>(mine + lane * 272 + 16 * i) =
                make_uint4(pack_bf16x2(a[0] * back, a[1] * back), pack_bf16x2(a[2] * back, a[3] * back),
                           pack_bf16x2(a[4] * back, a[5] * back), pack_bf16x2(a[6] * back, a[7] * back));
          }
        }
        __syncwarp();
        const int bytes = (n - round * 64) * es;   // of a row, from here on (may be negative)
        uint8_t* o = static_cast<uint8_t*>(args.out) + (base + round * 64) * es;
        if (args.out_vec) {
          o += static_cast<long long>(lane >> 4) * args.ldo * es + (lane & 15) * 16;
          const bool in = (lane & 15) * 16 < bytes;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int row = 2 * i + (lane >> 4);
            const uint4 q = *reinterpret_cast<const uint4*>(mine + row * 272 + (lane & 15) * 16);
            if (in && row < rows) *reinterpret_cast<uint4*>(o) = q;
            o += 2LL * args.ldo * es;
          }
        } else {
          for (int row = 0; row < rows; ++row, o += static_cast<long long>(args.ldo) * es)
            for (int i = lane; i < min(bytes, 256) / es; i += 32) {
              if (args.out_f32) reinterpret_cast<float*>(o)[i] = reinterpret_cast<const float*>(mine + row * 272)[i];
              else reinterpret_cast<__nv_bfloat16*>(o)[i] = reinterpret_cast<const __nv_bfloat16*>(mine + row * 272)[i];
            }
        }
        __syncwarp();
      }
    }
    __syncwarp();
  }
}

// ---- epilogue of the other modes.  A TMEM read in the 16 x 256-bit shape gives a thread two
// columns of four lanes per 8 columns, so that it needs two of their scales, not eight.
template <int BN, int MODE>
LMOE_DEV void epilogue_cols(const Fp8Args& args, const Fp8Walk& walk, const Fp8Ring<BN, MODE>& ring, const float* sc,
                            float* red, uint8_t* stage_out, uint32_t tmem, int id0, int step, int rank,
                            const Fp8Tile* tiles, uint64_t* tfull, uint64_t* tempty) {
  using C = Fp8Cfg<BN, MODE>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = warp & 3, half = (warp - 4) >> 2;
  const int tid = threadIdx.x & 127;                    // within the warpgroup
  const int r = quad * 32 + (lane >> 2);                // lanes r, + 8, + 16, + 24 of the tile
  const int c0 = half * C::kAcc, cl = (lane & 3) * 2;   // columns c0 + 8 g + cl, + 1
  const uint32_t tq = tmem + (static_cast<uint32_t>(quad * 32) << 16) + c0;
  // columns of one TMEM read: as many as the registers hold (64 columns in reads of 64: 20.8 us for 128
  // rows by 8192 x 8192, in reads of 32 21.4; a weight gradient's 128 sums leave room for 32)
  constexpr int kChC = C::kAcc == 64 ? 64 : C::kAcc > 64 ? 32 : 16;
  constexpr int kG = kChC / 8, kN = C::kAcc / kChC * 2;
  uint8_t* so = stage_out + half * C::kOutBytes;
  int it = 0;
  bool ok = true;
  Fp8Tile t = {};
  int tile = 0;
  const auto fetch = [&](int id) {   // the next tile (of the ring: this warp's turn with it ends here)
    if constexpr (MODE == kWgrad) {
      if (ok) {
        const int i = tile % kTileRing;
        ok = warp_wait(&tfull[i], (tile / kTileRing) & 1, ring.budget);
        ++tile;
        if (ok) {
          t = tiles[i];
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[i]);
          return;
        }
        atomicOr(ring.status, kErrWaitEpilogue);
      }
    }
    // (wgrad: also once a wait has given up, so that all warps know the same tiles and meet at the same barriers)
    t = tile_at<BN, MODE>(walk, args, id, rank);
  };
  if (id0 < walk.total) fetch(id0);
  float sp_next[4] = {};   // wgrad: scales of this thread's four lanes in the next block
  const auto lane_scales = [&](const Fp8Tile& u, int kb) {
    const float* ps = args.ps + static_cast<long long>(kb) * args.k + u.p0 + r;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (r + 8 * j < u.lanes) sp_next[j] = ps[8 * j];
  };
  if (MODE == kWgrad && ok && id0 < walk.total && t.kb0 < t.kb1) lane_scales(t, t.kb0);
  for (int id = id0; id < walk.total; id += step) {
    // acc[g][j]: the column pair of group g, lane 8 j + l / 4 of the warp's 32
    uint64_t acc[C::kAcc / 8][4];
#pragma unroll
    for (int i = 0; i < C::kAcc / 2; ++i) acc[i >> 2][i & 3] = 0;
    // what the sums are held times, a byte each: wgrad four lanes, the others a column pair's two beside the next's
    unsigned held[MODE == kWgrad ? 1 : (C::kAcc / 8 + 1) / 2];
#pragma unroll
    for (unsigned& h : held) h = kLifted * 0x01010101u;
    bool lowered = false;   // any of them (not wgrad; the same for the warp)
    for (int kb = t.kb0; ok && kb < t.kb1; ++kb, ++it) {
      ok = ring.wait(it);
      if (!ok) break;
      const uint32_t tb = tq + (it % C::kBufs) * BN;
      uint32_t v[2][kG * 4];
      tmem_ld_frag(tb, v[0]);
      uint64_t sp[4], s2[kG];
      const float mark = sc[(it % C::kSlots) * C::kSlotLd + BN];
      if (MODE == kWgrad) {
        float top = 0.f;   // (infinities and NaN are what they are in any unit)
#pragma unroll
        for (int j = 0; j < 4; ++j) top = fmaxf(top, finite(sp_next[j]) ? fabsf(sp_next[j]) : 0.f);
        if (top * mark > args.far || top > kFarLane) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float p = finite(sp_next[j]) ? fabsf(sp_next[j]) : 0.f;
            if (!(p * mark > args.far || p > kFarLane)) continue;
            unsigned h = held[0] >> (8 * j) & 0xff;
            const float f = held_lower(h, p * mark < 0x1p127f && p < 0x1p88f ? kAsIs : kLowered);
            held[0] = (held[0] & ~(0xffu << (8 * j))) | h << (8 * j);
#pragma unroll
            for (int g = 0; g < C::kAcc / 8; ++g) scale_pair(acc[g][j], f, f);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = sp_next[j] * held_times(held[0] >> (8 * j) & 0xff);
          sp[j] = pack2(p, p);
        }
        __syncwarp();   // (the TMEM reads are the whole warp's)
        if (kb + 1 < t.kb1) lane_scales(t, kb + 1);
      }
      const float* scs = sc + (it % C::kSlots) * C::kSlotLd + c0 + cl;
      const auto far_columns = [&] {   // scales of a marked block, or to sums that are not lifted any more
        lowered = true;
#pragma unroll
        for (int g = 0; g < C::kAcc / 8; ++g) {
          float x[2], f[2] = {1.f, 1.f};
          unpack2(s2[g % kG], x[0], x[1]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int at = 8 * (2 * (g & 1) + i);
            unsigned h = held[g / 2] >> at & 0xff;
            if (mark != 0.f) x[i] = marked_product(scs[8 * g + i + BN + 4], mark, h, args.far, f[i]);
            else x[i] *= held_times(h) * 0x1p-64f;
            held[g / 2] = (held[g / 2] & ~(0xffu << at)) | h << at;
          }
          s2[g % kG] = pack2(x[0], x[1]);
#pragma unroll
          for (int j = 0; j < 4; ++j) scale_pair(acc[g][j], f[0], f[1]);
        }
      };
      static_assert(MODE == kWgrad || kN == 2, "all columns' scales at once");
      tmem_ld_wait();
#pragma unroll
      for (int ch = 0; ch < kN; ++ch) {   // 16 lanes x kChC columns: lane half ch % 2
        const int h = ch & 1, g0 = (ch >> 1) * kG;
        if (ch + 1 < kN)
          tmem_ld_frag(tb + ((ch + 1) >> 1) * kChC + (((ch + 1) & 1) ? (16u << 16) : 0u), v[(ch + 1) & 1]);
        else
          ring.buffer_read(it, lane);
        if (h == 0) {
#pragma unroll
          for (int g = 0; g < kG; ++g) s2[g] = *reinterpret_cast<const uint64_t*>(scs + (g0 + g) * 8);
          if (MODE != kWgrad && (mark != 0.f || lowered)) far_columns();   // (the same for the warp)
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int g = 0; g < kG; ++g) {
            const uint32_t* w = &v[ch & 1][4 * g + 2 * q];
            if (MODE == kWgrad) fma_pair(acc[g0 + g][2 * h + q], w[0], w[1], sp[2 * h + q], s2[g]);
            else fma_pair(acc[g0 + g][2 * h + q], w[0], w[1], s2[g]);
          }
        if (ch + 1 < kN) tmem_ld_wait();
      }
      ring.scales_read(it, lane);
    }
    float even = 0x1p-64f;   // what is left to be taken out of all sums, as they are stored (wgrad: a lane's own)
    if (MODE != kWgrad && (MODE == kSplit || lowered)) {   // (the CTAs of a cluster may hold theirs otherwise)
      even = 1.f;
#pragma unroll
      for (int g = 0; g < C::kAcc / 8; ++g) {
        const unsigned h = held[g / 2] >> (16 * (g & 1));
#pragma unroll
        for (int j = 0; j < 4; ++j) scale_pair(acc[g][j], held_back(h & 0xff), held_back(h >> 8 & 0xff));
      }
    }
    if (MODE == kSplit) {
      // one tile per cluster: the sums of ranks 1.. go to rank 0 (the i-th four of thread x at
      // i * 128 + x: threads beside each other, fours beside each other)
      if (rank > 0) {
        cluster_wait();
        const uint32_t dst = cluster_map(smem_u32(red + (rank - 1) * BN * 128 + 4 * tid), 0);
#pragma unroll
        for (int i = 0; i < C::kAcc / 4; ++i) {
          float4 q;
          unpack2(acc[i >> 1][2 * (i & 1)], q.x, q.y);
          unpack2(acc[i >> 1][2 * (i & 1) + 1], q.z, q.w);
          cluster_store(dst + i * 2048, q);
        }
        cluster_arrive();
        cluster_wait();
      } else {
        cluster_wait();
        cluster_arrive();
        cluster_wait();
        for (int q = 1; q < args.splits; ++q) {
          const float* src = red + (q - 1) * BN * 128 + 4 * tid;
#pragma unroll
          for (int i = 0; i < C::kAcc / 4; ++i) {
            const float4 o = *reinterpret_cast<const float4*>(src + i * 512);
            uint64_t(&d)[4] = acc[i >> 1];
            float x, y;
            unpack2(d[2 * (i & 1)], x, y);
            d[2 * (i & 1)] = pack2(x + o.x, y + o.y);
            unpack2(d[2 * (i & 1) + 1], x, y);
            d[2 * (i & 1) + 1] = pack2(x + o.z, y + o.w);
          }
        }
      }
    }
    const auto back = [&](int j) { return MODE == kWgrad ? held_back(held[0] >> (8 * j) & 0xff) : even; };
    const int n = min(C::kAcc, t.ncols - c0);   // columns to store: below n (may be negative), from skip on
    const int skip = MODE == kWgrad ? 0 : t.skip;
    const int lanes = min(128, t.lanes);
    const long long base = t.out + static_cast<long long>(c0) * args.ldo;
    const bool store = rank == 0 && n > 0 && !(args.accumulate && t.kb0 == t.kb1);
    // the next tile, and its first scales, before this one is stored
    if (id + step < walk.total) {
      fetch(id + step);
      if (MODE == kWgrad && ok && t.kb0 < t.kb1) lane_scales(t, t.kb0);
    }
    // Below, a wait that gave up in one warp ends the whole warpgroup at its next barrier, so that
    // none of its warps stays at one.
    if (!store) continue;   // (the same for the warpgroup)
    const bool f32 = args.out_f32 || args.accumulate;   // (a bf16 sum is rounded once, after the addition)
    if (!f32) {
      // all columns, transposed on the way: column c is 256 bytes at so + 272 c
#pragma unroll
      for (int g = 0; g < C::kAcc / 8; ++g) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x, y;
          unpack2(acc[g][j], x, y);
          w[j] = pack_bf16x2(x * back(j), y * back(j));
        }
        stmatrix_x4_trans(smem_u32(so + (8 * g + (lane & 7)) * 272 + (quad * 4 + (lane >> 3)) * 16), w);
      }
      if (!named_barrier_all(1 + half, 128, ok)) break;
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(args.out) + base;
      if (args.out_vec) {
        // two columns to a store instruction, kBatch loads under way together
        constexpr int kBatch = C::kAcc / 8 < 8 ? C::kAcc / 8 : 8;
        const int part = (lane & 15) * 8, c0v = quad * 2 + (lane >> 4);
        o += static_cast<long long>(c0v) * args.ldo + part;
#pragma unroll
        for (int b = 0; b < C::kAcc / 8; b += kBatch) {
          uint4 q[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
            q[i] = *reinterpret_cast<const uint4*>(so + (c0v + 8 * (b + i)) * 272 + part * 2);
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
            if (part < lanes && c0v + 8 * (b + i) >= skip && c0v + 8 * (b + i) < n)
              *reinterpret_cast<uint4*>(o + 8LL * (b + i) * args.ldo) = q[i];
        }
      } else if (tid < lanes) {
        for (int c = skip; c < n; ++c)
          o[static_cast<long long>(c) * args.ldo + tid] = *reinterpret_cast<const __nv_bfloat16*>(so + c * 272 + tid * 2);
      }
      named_barrier(1 + half, 128);   // (it is written again)
    } else {
      // kOutCols columns at a time: column c is 512 bytes at so + 528 c
#pragma unroll
      for (int round = 0; round < C::kAcc / C::kOutCols; ++round) {
        const int here = min(C::kOutCols, n - round * C::kOutCols), from = skip - round * C::kOutCols;
        if (here <= 0) break;   // (the same for the warpgroup)
#pragma unroll
        for (int g = 0; g < C::kOutCols / 8; ++g)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float x, y;
            unpack2(acc[round * (C::kOutCols / 8) + g][j], x, y);
            float* o = reinterpret_cast<float*>(so + (8 * g + cl) * 528 + (r + 8 * j) * 4);
            o[0] = x * back(j);
            o[132] = y * back(j);
          }
        ok = named_barrier_all(1 + half, 128, ok);
        if (!ok) break;
        const long long o = base + static_cast<long long>(round * C::kOutCols) * args.ldo;
        if (args.out_vec && args.out_f32) {
          // a column to a store instruction, kBatch columns' loads under way together
          constexpr int kBatch = C::kOutCols / 4 < 8 ? C::kOutCols / 4 : 8;
          const int part = lane * 4;
          float* d = static_cast<float*>(args.out) + o + static_cast<long long>(quad) * args.ldo + part;
#pragma unroll
          for (int b = 0; b < C::kOutCols / 4; b += kBatch) {
            float4 q[kBatch], old[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              q[i] = *reinterpret_cast<const float4*>(so + (quad + 4 * (b + i)) * 528 + part * 4);
              old[i] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (args.accumulate && part < lanes && quad + 4 * (b + i) < here)
                old[i] = *reinterpret_cast<const float4*>(d + 4LL * (b + i) * args.ldo);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              if (args.accumulate)
                q[i] = make_float4(old[i].x + q[i].x, old[i].y + q[i].y, old[i].z + q[i].z, old[i].w + q[i].w);
              if (part < lanes && quad + 4 * (b + i) >= from && quad + 4 * (b + i) < here)
                *reinterpret_cast<float4*>(d + 4LL * (b + i) * args.ldo) = q[i];
            }
          }
        } else if (tid < lanes) {
          for (int c = max(from, 0); c < here; ++c) {
            float v = *reinterpret_cast<const float*>(so + c * 528 + tid * 4);
            const long long at = o + static_cast<long long>(c) * args.ldo + tid;
            if (args.out_f32) {
              float* d = static_cast<float*>(args.out) + at;
              *d = args.accumulate ? *d + v : v;
            } else {
              __nv_bfloat16* d = static_cast<__nv_bfloat16*>(args.out) + at;
              *d = __float2bfloat16_rn(__bfloat162float(*d) + v);
            }
          }
        }
        named_barrier(1 + half, 128);   // (it is written again)
      }
      if (!ok) break;
    }
    __syncwarp();
  }
}

template <int BN, int MODE>
__global__ void __launch_bounds__(Fp8Cfg<BN, MODE>::kThreads, Fp8Cfg<BN, MODE>::kCtas)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                    const Fp8Args args) {
  using C = Fp8Cfg<BN, MODE>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  float* red = reinterpret_cast<float*>(smem + C::kStages * C::kStageBytes);
  uint8_t* stage_out = reinterpret_cast<uint8_t*>(red) + C::kRedBytes;
  float* sc = reinterpret_cast<float*>(stage_out + C::kOutBytes * (C::kEpiWarps / 4));   // [kSlots][kSlotLd]
  int* start = reinterpret_cast<int*>(sc + C::kSlots * C::kSlotLd);                      // [E + 1]
  Fp8Info* infos = reinterpret_cast<Fp8Info*>(start + kMaxGroups + 4);                   // [kInfos] (kRows)
  Fp8Tile* tiles = reinterpret_cast<Fp8Tile*>(start + kMaxGroups + 4);                   // [kTileRing] (kWgrad)
  uint64_t* full = MODE == kWgrad ? reinterpret_cast<uint64_t*>(tiles + kTileRing)
                                  : reinterpret_cast<uint64_t*>(infos + (MODE == kRows ? kInfos : 0));
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;
  uint64_t* acc_empty = acc_full + C::kBufs;
  uint64_t* sfull = acc_empty + C::kBufs;
  uint64_t* sempty = sfull + C::kSlots;
  uint64_t* tfull = sempty + C::kSlots;   // [kTileRing] (kWgrad)
  uint64_t* tempty = tfull + kTileRing;
  uint64_t* mma_done = tempty + kTileRing;
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
    for (int i = 0; i < kTileRing; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], C::kEpiWarps);
    }
    mbar_init(mma_done, 2);
    fence_mbar_init();
    prefetch_tmap(&tmP);
    prefetch_tmap(&tmQ);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  griddep_enter();

  // start[]: exclusive prefix sum of the groups' units (row tiles, or blocks)
  constexpr int kUnit = MODE == kWgrad || MODE == kRows ? 128 : BN;
  for (int e = threadIdx.x; e < args.E; e += C::kThreads) {
    int lo, hi;
    group_rows(args, e, lo, hi);
    start[e] = (hi - lo + kUnit - 1) / kUnit;
  }
  __syncthreads();
  if (warp == 0) {   // a run of groups per lane
    const int per = (args.E + 31) / 32, e0 = min(lane * per, args.E), e1 = min(e0 + per, args.E);
    // no more units than the launch has room for, whatever the offsets say (kSplit: one tile to a cluster)
    const int rows = static_cast<int>(args.rows);
    const int cap = MODE == kWgrad ? rows / 128 : most_tiles(rows, args.E, kUnit);
    int sum = 0;
    for (int e = e0; e < e1; ++e) sum += start[e];
    int run = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(~0u, run, d);
      if (lane >= d) run += up;
    }
    const int tot = __shfl_sync(~0u, run, 31);
    run -= sum;
    for (int e = e0; e < e1; ++e) {
      const int c = start[e];
      start[e] = min(run, cap);
      run += c;
    }
    if (lane == 0) start[args.E] = min(tot, cap);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Fp8Walk walk;
  walk.start = start;
  walk.E = args.E;
  walk.others = MODE == kWgrad ? (args.k + 127) / 128 : MODE == kRows ? (args.n + BN - 1) / BN : (args.n + 127) / 128;
  walk.cols = (args.n + BN - 1) / BN;
  walk.total = (MODE == kWgrad ? args.E * walk.cols : start[args.E]) * walk.others;
  const int S = MODE == kSplit ? args.splits : 1;   // CTAs of a cluster
  const int rank = static_cast<int>(blockIdx.x % S);
  const int id0 = static_cast<int>(blockIdx.x) / S, step = static_cast<int>(gridDim.x) / S;
  const long long budget = args.budget;
  unsigned* const status = args.status != nullptr ? args.status : &g_status;
  if (MODE == kSplit) cluster_arrive();   // every CTA of the cluster has started (waited for below)

  if (warp < 4) {
    if constexpr (C::kDec > 0) regs_dec<C::kDec>();
    if (warp == 0 && lane == 0) {
      // ---- TMA producer.  Tiles of few rows read each weight about once: those leave L2 first (8 rows over 64
      // experts of 4096 x 4096 28.6 us, otherwise 33.4; 512 rows, 256 of them one expert's, whose 16 tiles
      // side by side read the same weights, 193 and 200).  The weight gradient reads its lane operand
      // again in every column of tiles (32768 rows over 64 experts of 4096 x 2048 811 us, leaving first 908).
      const uint64_t pol_p = MODE == kCols || MODE == kSplit ? policy_evict_first() : policy_evict_normal();
      const uint64_t pol_q = policy_evict_normal();
      const uint32_t tx = C::kPBytes + (MODE == kCols || MODE == kSplit ? args.box : BN) * 128;
      int it = 0;
      bool ok = true;
      for (int id = id0; ok && id < walk.total; id += step) {
        const Fp8Tile t = tile_at<BN, MODE>(walk, args, id, rank);
        for (int kb = t.kb0; kb < t.kb1; ++kb, ++it) {
          const int s = it % C::kStages;
          if (!mbar_wait(&empty[s], ((it / C::kStages) & 1) ^ 1, budget)) {
            atomicOr(status, kErrWaitProducer);
            ok = false;
            break;
          }
          uint8_t* sp = smem + s * C::kStageBytes;
          mbar_arrive_expect_tx(&full[s], tx);
          if (MODE == kRows) {
            tma_load_2d_hint(sp, &tmP, &full[s], kb * 128, t.p0, pol_p);
            tma_load_3d_hint(sp + C::kPBytes, &tmQ, &full[s], kb * 128, t.q0, t.e, pol_q);
          } else {
            if (MODE == kWgrad) tma_load_2d_hint(sp, &tmP, &full[s], kb * 128, t.p0, pol_p);
            else tma_load_3d_hint(sp, &tmP, &full[s], kb * 128, t.p0, t.e, pol_p);
            tma_load_2d_hint(sp + C::kPBytes, &tmQ, &full[s], kb * 128, t.q0, pol_q);
          }
        }
      }
      // every copy of this thread lands before the CTA leaves
      for (int j = max(0, it - C::kStages); j < it; ++j)
        if (!mbar_wait(&full[j % C::kStages], (j / C::kStages) & 1, kDrainBudget))
          atomicOr(status, kErrDrain);
    } else if ((warp == 1 || warp == 3) && lane == 0) {
      // ---- MMA issuers: one block of 128 into one TMEM buffer, warp 1 the even blocks of the ring,
      // warp 3 the odd ones.  Issuing a block's MMAs and commits holds a thread for most of the time
      // they take, and its waits and arithmetic for the next one take 400 cycles more, in which the
      // tensor cores would run dry; so the other thread does its own meanwhile.
      const int mine = warp >> 1;
      int it = 0;
      bool ok = true;
      for (int id = id0; ok && id < walk.total; id += step) {
        // (kRows: all 256 columns, whatever the tile: those past the weight's rows are zeros, and
        // working a tile out here would hold up its first MMAs)
        int ncols = BN, blocks = args.num_kb;
        if (MODE != kRows) {
          const Fp8Tile t = tile_at<BN, MODE>(walk, args, id, rank);
          ncols = t.ncols;
          blocks = t.kb1 - t.kb0;
        }
        const uint32_t idesc = idesc_f8(args.fmt_p, args.fmt_q, (ncols + 15) / 16 * 16);
        const int end = it + blocks;
        for (it += (it ^ mine) & 1; it < end; it += 2) {
          const int s = it % C::kStages, buf = it % C::kBufs, slot = it % C::kSlots;
          // The buffer first: a stage's barrier may be waited for only once its previous use is over (a
          // wait for the phase after next returns at once).  With three stages that use was the other
          // warp's; but this buffer's release means that every block up to it - kBufs has been read.
          if (!mbar_wait(&sfull[slot], (it / C::kSlots) & 1, budget) ||
              !mbar_wait(&acc_empty[buf], ((it / C::kBufs) & 1) ^ 1, budget) ||
              !mbar_wait(&full[s], (it / C::kStages) & 1, budget)) {
            atomicOr(status, kErrWaitMma);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t p0 = smem_u32(smem + s * C::kStageBytes);
          const uint64_t pd = sw128_kmajor_desc(p0), qd = sw128_kmajor_desc(p0 + C::kPBytes);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)   // 32 bytes on: 2 in the descriptors' 16-byte addresses
            mma_f8(tmem + buf * BN, pd + 2 * kk, qd + 2 * kk, idesc, kk > 0);
          mma_commit(&acc_full[buf]);
          mma_commit(&empty[s]);
        }
        it = end;
      }
      mma_commit(mma_done);
    } else if (warp == 2) {
      // ---- scales, the loads of several blocks in flight at a time.  kRows: as[row] ws[half] for
      // the 128 lanes of each column half; kCols, kSplit: as ws of each column; wgrad: of each column
      constexpr int kPer = (BN + 31) / 32, kOwn = MODE == kRows ? 4 : kPer, kBatch = BN >= 128 ? 2 : 4;
      int it = 0, tile = 0;
      bool ok = true;
      for (int id = id0; ok && id < walk.total; id += step) {
        const Fp8Tile t = tile_at<BN, MODE>(walk, args, id, rank);
        const float* q = MODE == kRows ? args.ps + t.p0 + lane : args.qs + t.q0 + lane;
        const long long ldq = MODE == kWgrad ? args.n : args.rows;
        const int live = MODE == kRows ? t.lanes : t.ncols;
        const int nb = (args.n + 127) / 128;   // the weight's 128 x 128 blocks
        const int b0 = MODE == kRows ? t.q0 / 128 : t.p0 / 128;
        const float* w = (MODE == kRows ? args.qs : args.ps) + (static_cast<long long>(t.e) * nb + b0) * args.num_kb;
        const bool two = MODE == kRows && b0 + 1 < nb;
        bool told = false;
        if (MODE == kWgrad) {
          if (!warp_wait(&tempty[tile % kTileRing], ((tile / kTileRing) & 1) ^ 1, budget)) {
            atomicOr(status, kErrWaitProducer);
            break;
          }
          if (lane == 0) {
            tiles[tile % kTileRing] = t;
            mbar_arrive(&tfull[tile % kTileRing]);
          }
          ++tile;
        }
        for (int kb = t.kb0; ok && kb < t.kb1; kb += kBatch) {
          float v[kBatch][kPer], u[kBatch][2];
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const bool in = kb + j < t.kb1;
            u[j][0] = MODE == kWgrad ? 1.f : (in ? w[kb + j] : 0.f);
            u[j][1] = two && in ? w[args.num_kb + kb + j] : u[j][0];
#pragma unroll
            for (int i = 0; i < kOwn; ++i)
              v[j][i] = in && lane + 32 * i < live ? q[(kb + j) * ldq + 32 * i] : 0.f;
#pragma unroll
            for (int i = kOwn; i < kPer; ++i) v[j][i] = v[j][i - kOwn];
          }
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            if (!ok || kb + j >= t.kb1) break;
            const int s = it % C::kSlots;
            if (!warp_wait(&sempty[s], ((it / C::kSlots) & 1) ^ 1, budget)) {
              atomicOr(status, kErrWaitProducer);
              ok = false;
              break;
            }
            if (MODE == kRows && !told) {   // (here, and not before the slot is free: see Fp8Info)
              if (lane == 0) infos[tile % kInfos] = {t.out, t.lanes, t.ncols};
              told = true;
              ++tile;
            }
            float* at = sc + s * C::kSlotLd;
            if (MODE == kWgrad) {
#pragma unroll
              for (int i = 0; i < kPer; ++i)
                if (lane + 32 * i < BN) at[lane + 32 * i] = v[j][i];
              float top = 0.f;
#pragma unroll
              for (int i = 0; i < kPer; ++i) top = fmaxf(top, finite(v[j][i]) ? fabsf(v[j][i]) : 0.f);
              top = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(top)));
              if (lane == 0) at[BN] = top;
            } else if (MODE == kRows) {
              const float b0 = u[j][0] * kLift, b1 = u[j][1] * kLift;
              float top = fabsf(v[j][0]);   // this lane's largest scale (a NaN is left out, and staged as it is)
#pragma unroll
              for (int i = 0; i < kPer; ++i) {
                if (i > 0 && i < kOwn) top = fmaxf(top, fabsf(v[j][i]));
                if (lane + 32 * i < BN) at[lane + 32 * i] = v[j][i] * (i / 4 & 1 ? b1 : b0);
              }
              // (a zero of ws: the mark stays zero, and so do the products)
              const bool near = __all_sync(~0u, top * fmaxf(fabsf(b0), fabsf(b1)) <= args.far);
              const bool far = !near && (u[j][0] != 0.f || u[j][1] != 0.f);
              if (far) {
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                  if (lane + 32 * i < BN) at[lane + 32 * i] = v[j][i];
              }
              if (lane == 0)
                *reinterpret_cast<float2*>(at + BN) = far ? make_float2(u[j][0], u[j][1]) : make_float2(0.f, 0.f);
            } else {
              // the mark without a vote, which a small tile's start would wait for (2560 rows over 64 experts of
              // 4096 x 4096: 178.6 us, with a vote as above 183)
              if (lane == 0) at[BN] = 0.f;
              __syncwarp();
              const float b0 = u[j][0] * kLift;
#pragma unroll
              for (int i = 0; i < kPer; ++i)
                if (lane + 32 * i < BN) {
                  at[lane + 32 * i] = v[j][i] * b0;
                  at[BN + 4 + lane + 32 * i] = v[j][i];
                  if (!(fabsf(v[j][i]) * fabsf(b0) <= args.far) && u[j][0] != 0.f) at[BN] = u[j][0];
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sfull[s]);
            ++it;
          }
        }
      }
    }
  } else {
    if constexpr (C::kInc > 0) regs_inc<C::kInc>();
    const Fp8Ring<BN, MODE> ring = {acc_full, acc_empty, sempty, status, budget};
    if constexpr (MODE == kRows) epilogue_rows<BN>(args, walk, ring, sc, infos, stage_out, tmem, id0, step);
    else epilogue_cols<BN, MODE>(args, walk, ring, sc, red, stage_out, tmem, id0, step, rank, tiles, tfull, tempty);
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
      atomicOr(status, kErrDrain);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int BN, int MODE>
cudaError_t launch_one(const CUtensorMap& p, const CUtensorMap& q, Fp8Args a, long long tiles, cudaStream_t s) {
  using C = Fp8Cfg<BN, MODE>;
  const unsigned others = (MODE == kWgrad ? a.k + 127 : MODE == kRows ? a.n + 255 : a.n + 127) / (MODE == kRows ? 256 : 128);
  a.by_others = FastDiv::of(others);
  a.by_group = FastDiv::of(others * kRasterGroup);
  a.by_E = FastDiv::of(a.E);
  auto kern = gemm_fp8_kernel<BN, MODE>;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), C::kSmemBytes);
  if (e != cudaSuccess) return e;
  if (MODE == kSplit)
    return launch_pdl_cluster(kern, dim3(static_cast<unsigned>(tiles * a.splits)), dim3(C::kThreads), C::kSmemBytes,
                              s, a.splits, p, q, a);
  const long long sms = static_cast<long long>(C::kCtas) * sm_count();
  return launch_pdl(kern, dim3(static_cast<unsigned>(tiles < sms ? tiles : sms)), dim3(C::kThreads), C::kSmemBytes,
                    s, p, q, a);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool known(lmoe_fp8_format f) { return f == LMOE_FP8_E4M3 || f == LMOE_FP8_E5M2; }
// the largest sum of a block's 128 products of codes
double largest_sum(const lmoe_fp8_matmul& c) {
  const auto largest = [](lmoe_fp8_format f) { return f == LMOE_FP8_E5M2 ? 57344.0 : 448.0; };
  return 128.0 * largest(c.a_format) * largest(c.b_format);
}
constexpr int kSms = 152;
constexpr int kRowsMin = 55, kRowsMinOne = 65, kFewRows = 8;

}  // namespace
}  // namespace lmoe

using namespace lmoe;

extern "C" lmoe_status lmoe_matmul_fp8(const lmoe_fp8_matmul* c, const uint8_t* a, const float* a_scales,
                                       const uint8_t* w, const float* w_scales, const int32_t* offsets, void* out,
                                       uint32_t* status, cudaStream_t stream) {
  if (c == nullptr || c->rows < 0 || c->N <= 0 || c->K <= 0 || c->n_experts <= 0) return LMOE_ERR_ARG;
  if (c->wait_budget_cycles < 0) return LMOE_ERR_ARG;
  if (!known(c->a_format) || !known(c->b_format)) return LMOE_ERR_ARG;
  if (c->accumulate || c->unpadded_rows != 0) return LMOE_ERR_ARG;
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
  g.n = c->N;
  g.k = c->K;
  g.num_kb = (c->K + 127) / 128;
  g.E = c->n_experts;
  g.offsets = offsets;
  g.out = out;
  g.ldo = c->N;
  g.out_f32 = c->out_dtype == LMOE_F32;
  g.out_vec = aligned(out, 16) && c->N % (g.out_f32 ? 4 : 8) == 0;
  g.status = status;
  g.budget = c->wait_budget_cycles > 0 ? c->wait_budget_cycles : kDefaultWaitBudget;
  g.splits = 1;
  g.cap = static_cast<int>(c->rows);
  g.far = static_cast<float>(0x1p126 / (g.num_kb * largest_sum(*c)));
  // Up to 16 rows in all, or up to kFewRows for an expert on average: 16-column tiles.  Measured
  // against 64 columns, 4096 x 4096: 1 row 6.8 us and 9.1, 8 and 24 rows of 64 experts 24.3, 45.5 and 26.0, 48.5, 480 rows
  // of them 155 and 161; beyond the limit 800 and 1024 rows 164, 172 and 163, 163, 20 rows of 2 experts 18 and 12.
  // (The average says nothing of the split, which is known to the device alone: 512 rows of 64 experts even 168 and
  // 172, with 64, 128, 256, 448 rows of one of them 172, 182, 190, 210 and 172, 171, 175, 185.)
  // Then rows as lanes, unless an expert has fewer than kRowsMin rows on average (one matrix:
  // kRowsMinOne) or those tiles would leave three quarters of the SMs idle: then 64 rows at a time,
  // four of whose tiles cover one of the others.  Measured, rows as lanes against 64 at a time:
  //   64 experts of 4096 x 4096 with 44, 52, 58, 64, 96 rows   183, 196, 194, 189, 202 us and 176, 192, 197, 207, 264
  //   one matrix of 8192 x 16384 with 64 and 100 rows          41, 41 and 23, 40
  //   256 rows by 4096 x 4096, 128 and 512 by 8192 x 8192      18.4, 31.6, 38 and 12.6, 21.9, 75
  const long long live = c->n_experts < c->rows ? c->n_experts : c->rows;
  const int R = static_cast<int>(c->rows);
  const long long row_tiles = 1LL * most_tiles(R, c->n_experts, 128) * ((c->N + 255) / 256);
  const bool rows = c->rows / live >= (c->n_experts == 1 ? kRowsMinOne : kRowsMin) && row_tiles * 4 > kSms;
  const int bn = rows ? 256 : c->rows <= 16 || c->rows / live <= kFewRows ? 16 : 64;
  const unsigned long long K = c->K, N = c->N;
  const unsigned long long wd[3] = {K, N, static_cast<unsigned long long>(c->n_experts)}, wst[2] = {K, K * N};
  const unsigned long long ad[2] = {K, static_cast<unsigned long long>(c->rows)}, ast[1] = {K};
  const unsigned wbox[3] = {128, rows ? 256u : 128u, 1};
  g.box = static_cast<int>(c->rows < bn ? c->rows : bn);
  const unsigned abox[2] = {128, rows ? 128u : static_cast<unsigned>(g.box)};
  CUtensorMap tw, ta;
  if (!encode_u8_swizzled(&tw, w, 3, wd, wst, wbox) || !encode_u8_swizzled(&ta, a, 2, ad, ast, abox))
    return LMOE_ERR_CUDA;
  cudaError_t e;
  if (rows) {
    g.ps = a_scales;
    g.qs = w_scales;
    g.fmt_p = c->a_format;
    g.fmt_q = c->b_format;
    e = launch_one<256, kRows>(ta, tw, g, row_tiles, stream);
  } else {
    g.ps = w_scales;
    g.qs = a_scales;
    g.fmt_p = c->b_format;
    g.fmt_q = c->a_format;
    const long long tiles = most_tiles(R, c->n_experts, bn) * wt;
    // Few tiles: split the reduction among the CTAs of a cluster, at least four blocks each (1 and 64
    // rows by 4096 x 4096: 7.4 and 9.5 us, one CTA a tile 10.9 and 12.1; 16 by 8192 x 8192 12.2 and 17.9).
    while (g.splits < (bn == 16 ? 8 : 4) && tiles * g.splits * 2 <= kSms && g.num_kb / (g.splits * 2) >= 4) g.splits *= 2;
    if (g.splits > 1) e = bn == 16 ? launch_one<16, kSplit>(tw, ta, g, tiles, stream) : launch_one<64, kSplit>(tw, ta, g, tiles, stream);
    else e = bn == 16 ? launch_one<16, kCols>(tw, ta, g, tiles, stream) : launch_one<64, kCols>(tw, ta, g, tiles, stream);
  }
  return e == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}

extern "C" lmoe_status lmoe_matmul_fp8_wgrad(const lmoe_fp8_matmul* c, const uint8_t* dy_t, const float* dy_scales,
                                             const uint8_t* x_t, const float* x_scales, const int32_t* offsets,
                                             void* dw, uint32_t* status, cudaStream_t stream) {
  if (c == nullptr || c->rows < 0 || c->rows % 128 || c->N <= 0 || c->K <= 0 || c->n_experts <= 0) return LMOE_ERR_ARG;
  if (c->wait_budget_cycles < 0) return LMOE_ERR_ARG;
  if (!known(c->a_format) || !known(c->b_format)) return LMOE_ERR_ARG;
  if (offsets == nullptr && c->n_experts != 1) return LMOE_ERR_ARG;
  if (c->unpadded_rows < 0 || (c->unpadded_rows > 0 && lmoe_fp8_padded_rows(c->unpadded_rows, c->n_experts) != c->rows))
    return LMOE_ERR_ARG;
  if (c->out_dtype != LMOE_F32 && c->out_dtype != LMOE_BF16) return LMOE_ERR_UNSUPPORTED;
  if (c->n_experts > kMaxGroups || c->K > (1 << 20) || c->N > (1 << 20) || c->rows > (1LL << 24))
    return LMOE_ERR_UNSUPPORTED;
  const long long lt = (c->K + 127) / 128, ct = (c->N + 127) / 128, tiles = lt * ct * c->n_experts;
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
  g.n = c->N;
  g.k = c->K;
  g.E = c->n_experts;
  g.offsets = offsets;
  g.ps = x_scales;
  g.qs = dy_scales;
  g.out = dw;
  g.ldo = c->K;
  g.out_f32 = c->out_dtype == LMOE_F32;
  g.out_vec = aligned(dw, 16) && c->K % (g.out_f32 ? 4 : 8) == 0;
  g.accumulate = c->accumulate;
  g.fmt_p = c->b_format;
  g.fmt_q = c->a_format;
  g.status = status;
  g.budget = c->wait_budget_cycles > 0 ? c->wait_budget_cycles : kDefaultWaitBudget;
  g.splits = 1;
  g.cap = static_cast<int>(c->unpadded_rows > 0 ? c->unpadded_rows : c->rows);
  g.far = static_cast<float>(0x1p62 / (c->rows / 128 * largest_sum(*c)));
  const unsigned long long R = static_cast<unsigned long long>(c->rows);
  CUtensorMap tp, tq;
  const unsigned long long pd[2] = {R, static_cast<unsigned long long>(c->K)};
  const unsigned long long qd[2] = {R, static_cast<unsigned long long>(c->N)}, st[1] = {R};
  const unsigned box[2] = {128, 128};
  if (!encode_u8_swizzled(&tp, x_t, 2, pd, st, box) || !encode_u8_swizzled(&tq, dy_t, 2, qd, st, box))
    return LMOE_ERR_CUDA;
  return launch_one<128, kWgrad>(tp, tq, g, tiles, stream) == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}

extern "C" lmoe_status lmoe_fp8_check_status(cudaStream_t stream, uint32_t* detail) {
  static std::mutex mu;   // (one landing place for the word)
  std::lock_guard<std::mutex> lock(mu);
  uint32_t word = 0;
  if (launch_pdl(take_status_kernel, dim3(1), dim3(1), 0, stream) != cudaSuccess ||
      cudaMemcpyFromSymbolAsync(&word, g_status_taken, 4, 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
      cudaStreamSynchronize(stream) != cudaSuccess)
    return LMOE_ERR_CUDA;
  if (detail != nullptr) *detail = word;
  return word == 0 ? LMOE_OK : LMOE_ERR_TIMEOUT;
}

extern "C" lmoe_status lmoe_fp8_wait_selftest(long long budget_cycles, cudaStream_t stream) {
  const long long b = budget_cycles < 1 ? 1 : budget_cycles > kDefaultWaitBudget ? kDefaultWaitBudget : budget_cycles;
  void* word = nullptr;
  if (cudaGetSymbolAddress(&word, g_status) != cudaSuccess) return LMOE_ERR_CUDA;
  return launch_wait_selftest(b, static_cast<unsigned*>(word), stream) == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}
