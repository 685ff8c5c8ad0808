// gemm_bf16.cu — products of bf16 rows sorted by expert with their expert's weights, and what a
// gated feed-forward block makes of them, forward and backward, on the 5th-generation tensor
// cores, persistent.  For the rows r of expert e (offsets[e] <= r < offsets[e + 1]), or of one matrix:
//
//   kGated      g = x Wg^T, u = x Wu^T, h = silu(g) u         (g and u stored too if asked for)
//   kGatedGrad  dh = dy Wd; dg = dh u s (1 + g (1 - s)), du = dh g s, s = sigmoid(g)
//   kProduct    out = a W^T (+ a2 W2^T)
//   kProductT   out = a W (+ a2 W2), W [k, n]
//   kWgrad      dw[e] (+)= dy^T x over e's rows (and dw2 from dy2)
//
// Operands are bf16, sums fp32 in tensor memory, each result rounded once where it is stored.  The lane
// operand (a, or dy transposed) gives an MMA its rows, the column operand (the weights, or x) its
// columns.  An operand whose reduction is its rows' own dimension lies in shared memory as boxes of 64 of
// them (128 bytes, swizzled) by its rows; the weights of kGatedGrad and kProductT and both operands of
// kWgrad are reduced along their other dimension and lie there as boxes of 64 columns by 64 of the reduction,
// which the tensor cores read as they are (MN-major), so nothing is transposed in memory.
//
// An expert's rows rarely fill kWgrad's last block of 64.  What lies behind them is another expert's (maybe
// infinities or NaN, which a product with zero would keep), so a warp clears those rows of both operands in
// shared memory before the tensor cores read them, up to the next 16; steps of 16 behind that are left out.
//
// Tiles (UNIT rows, see rows_product for which where and what was measured):
//   256   a pair of CTAs (cta_group::2), 256 x 256 sums: each CTA loads 128 rows of the lane operand and half of the
//         column operand's tile, 32 KB for 128 x 256 x 64 products, which shared memory can take in in the time of the MMAs
//         (a single CTA's 128 x 128 tiles take in twice as much: 32768 uneven rows over 64 experts of 4096 x 4096, gate and
//         up 2568 us, by pairs 2010 with all else as it was).  kGated: columns are 64 of gate, the same 64 of up, and so on.  An
//         expert's last tile, if it has no more than 128 rows, goes by MMAs of half the height (612 and 412 rows in turn: 1600 us
//         without, so 1440 to 1480).
//   128   one CTA, 128 x 128 sums: fewer rows per expert, or too few tiles of 256.
//   32    the same with loads of up to 32 rows: a few tokens.  Bound by the stream of weights.
// Few tiles with a long reduction are shared by a cluster of up to 8 CTAs.
//
// Roles of a CTA: one thread of warp 0 loads the lane operand, one of warp 3 the column operand (one thread for both: weight
// gradients 267 us, so 245), one of warp 1 issues MMAs (in a pair the first CTA's, for both), warp 2 clears kWgrad's
// rows, warps 4.. are the epilogue, warp w on TMEM lanes 32 (w % 4) ..  Two accumulator buffers: a tile is stored while
// the next one is computed.  A warp's 32 rows of 128 bytes (kGatedGrad: 64, and gate and up come in the same way) pass
// through its own shared memory and leave by tensor stores; where they are not all the tile's, by stores of whole segments.
//
// Measured (other inputs in each call, power-limited at 1.6 to 1.7 GHz where it is tensor-bound): 32768 uneven rows over 64 experts
// of 4096 x 4096, g and u stored, 1790 to 1900 us (even experts, the same inputs: 1270); the gradient of 16384 over 32 475 us (even, the
// same 384); dx of 16384 over 32, two pairs, 925 us (650); 16384 x 8192 x 8192 1120 to 1220 us a call (1.8 to 1.96 PFLOP/s), 1315 back
// to back (1.67); two weight gradients of 8192 rows over 16 to fp32 520 us (4.5 TB/s); one token on 8 of 64 experts, gate and up, 73
// to 81 us, 1024 rows over 64 experts 323 us (6.8 TB/s).  Tensor pipe busy 88 to 95 % (gradient 80, weight gradient 56
// beside 62 % of HBM's nominal rate) at 512 rows per expert.
#include <mutex>

#include "../../include/latent_moe.h"
#include "groups.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace lmoe {
namespace {

enum Bf16Mode : int { kGated = 0, kGatedGrad = 1, kProduct = 2, kProductT = 3, kWgrad = 4 };
constexpr int kRaster = 8;       // row tiles that take turns before the next column of tiles
// Tensor memory's fp32 sums are cut, not rounded, at each addition, in proportion to their number: 4096 products in a row leave
// 4.4e-6 of the result (2-norm), and products of one sign, which are all cut in one direction, 6e-9 each.  For fp32 results a
// sum in TMEM ends after kChunk blocks of 64, and the epilogue adds those in registers (7e-7, of one sign 1.3e-6.  Sums of 8
// blocks: 5e-7, but experts of about 512 rows then take two: their weight gradients 246 us instead of 239).  bf16 results, whose
// rounding is 1.7e-3 (2-norm), go the same way from kLong blocks on, where the cuts are 1e-4 (of 2^20 products they were 3.9e-3).
constexpr int kChunk = 12, kLong = 256;
// Budget of the waits for a CTA's own copies and MMAs at its end: they take microseconds.  (In a pair whose second CTA gave
// up, the first one waits that long for copies that never started.)  A pair with a producer that gave up stays kLast more.
constexpr long long kDrain = 20000000, kLast = 2000000;

struct Bf16Args {
  FastDiv by_others, by_group;   // tiles across; kRaster rows of them
  FastDiv by_tiles;              // kWgrad: tiles of an expert
  long long rows;                // rows of a (kWgrad: of dy and x)
  int n, k;                      // out is [rows, n], reduced over k (kWgrad: dw is [n, k])
  int num_kb;                    // blocks of 64 of k (0: kWgrad)
  int pairs;                     // pairs of operands that are summed (kWgrad: weights)
  int E;
  const int32_t* offsets;        // [E + 1], or nullptr: one group of all rows
  int box;                       // rows of a that a load brings (tiles of few rows)
  int splits;                    // CTAs (a cluster) that share a tile's reduction
  const __nv_bfloat16 *gate, *up;   // kGatedGrad
  void *out, *out2, *out3;       // h, gate, up; dgate, dup; out; dw, dw2
  int out_f32, accumulate;
  int whole;                     // whole groups of 32 rows leave by tensor stores
  unsigned* status;              // error word, or nullptr: the device's own (g_status)
  long long budget;
};

// What waits that gave up leave for lmoe_bf16_check_status where the caller has no word for it.
__device__ unsigned g_status, g_status_taken;
__global__ void take_status_kernel() {
  griddep_enter();
  g_status_taken = atomicExch(&g_status, 0u);
}

// UNIT: rows of a tile; 256: a pair of CTAs, 128 rows and half of the column operand's tile each.
// CHUNKED: sums of kChunk blocks, added in registers: fp32 results, and bf16 ones of more than kLong blocks.
template <int MODE, int UNIT, bool CHUNKED>
struct Bf16Cfg {
  static constexpr bool kPair = UNIT == 256;
  static constexpr bool kLanesMn = MODE == kWgrad;
  static constexpr bool kColsMn = MODE == kWgrad || MODE == kGatedGrad || MODE == kProductT;
  static constexpr int kLanes = kPair ? 128 : UNIT;               // that a CTA loads
  static constexpr int kBN = kPair ? 256 : 128;                   // accumulator columns
  static constexpr int kOutCols = MODE == kGated ? kBN / 2 : kBN;  // columns of a tile
  static constexpr int kEpiWarps = kPair && CHUNKED ? 8 : 4;
  // few rows: the one warp that has them leaves the sums in shared memory (in two buffers by turns), and all four finish them
  static constexpr bool kFlat = UNIT == 32;
  static constexpr int kLdFlat = 132;                             // floats of a row of 128 sums
  static constexpr int kThreads = 128 + 32 * kEpiWarps;
  static constexpr int kABytes = kLanes * 128, kBBytes = 128 * 128, kStageBytes = kABytes + kBBytes;
  // a warp's 32 rows of 128 bytes on their way out (kGatedGrad: of 64 bytes, and in, of gate and of up)
  static constexpr int kRow = MODE == kGatedGrad ? 64 : 128;
  static constexpr int kWarpBytes = 32 * kRow * (MODE == kGatedGrad ? 3 : 1);
  static constexpr int kStagingBytes = kFlat ? 2 * 32 * kLdFlat * 4 : kEpiWarps * kWarpBytes;
  // off[], and start[] (not kWgrad).  A chunked kWgrad has room for a stage more than with all offsets: from kOffsets experts
  // on they are read where they are (read there always, 16 experts' weight gradients to bf16 took 195 us, so 181).
  static constexpr int kOffsets = CHUNKED && MODE == kWgrad ? 320 : kMaxGroups + 4;
  static constexpr int kTableBytes = kOffsets * 4 * (MODE == kWgrad ? 1 : 2);
  static constexpr int kFixed = kStagingBytes + kTableBytes + 512 + 1024;
  static constexpr int kFit = (227 * 1024 - kFixed) / kStageBytes;
  static constexpr int kStages = kFit > 12 ? 12 : kFit;
  static constexpr int kSmemBytes = kFixed + kStages * kStageBytes;
  static constexpr uint32_t kTmemCols = 2 * kBN;
  // A pair's last tile of an expert, with no more than 128 rows: an MMA of 128 rows (64 of each CTA) takes half the time.
  // Its sums lie with their first 128 columns in lanes 0..63 and the others in lanes 64..127.
  static constexpr bool kShort = kPair && MODE != kWgrad;
  static constexpr int kChunkBlocks = CHUNKED ? kChunk : kLong;   // (kLong: all of it, no reduction is longer)
  static_assert((3 * kStages + 2 * 2 + 1 + 4) * 8 + 2 * 4 <= 512, "barriers, tmem_slot, gave_up");
  // the MMA reads 128 lanes, the tile's rows and whatever lies behind them in the stage
  static_assert(kStageBytes >= 128 * 128, "lane operand");
  // sums of a tile shared by a cluster of up to 8: of each row 128, and 4 or 8 floats of padding for each CTA
  static_assert(kPair || kStages * kStageBytes >= kLanes * (128 + 8 * 8) * 4, "partial sums");
};

// Shared-memory descriptor of an MN-major operand tile with 128-byte swizzle: boxes of 64 columns (128 bytes) by 64
// of the reduction, the next 64 columns 8192 bytes on (leading offset), the next 8 of the reduction 1024
// (stride offset).  16 of the reduction are 2048 bytes.
LMOE_DEV uint64_t sw128_mnmajor_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(8192 >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// ---- pairs of CTAs (cta_group::2): both hold their halves of the operands at the same place, the first one's thread
// issues for both, and barriers that it waits for are the first one's.
LMOE_DEV void tmem_alloc_pair(uint32_t* slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
LMOE_DEV void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
LMOE_DEV void mma_bf16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on this barrier of both CTAs.
LMOE_DEV void mma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
// ---- loads into this CTA's shared memory (addresses, not pointers: a producer thread's own instructions are what
// bounds it).  In a pair they are counted by the barrier at cluster address `bar`.
template <bool PAIR>
LMOE_DEV void load_2d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, uint64_t policy) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        ".L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "l"(policy)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "l"(policy)
        : "memory");
}
template <bool PAIR>
LMOE_DEV void load_3d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2, uint64_t policy) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
        : "memory");
}
LMOE_DEV void arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
LMOE_DEV bool wait_at(uint32_t bar, uint32_t parity, long long budget) {   // mbar_wait
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait_sleep(bar, parity, kWaitSleepNs)) {
    if (clock64() - t0 > budget) return false;
  }
  return true;
}
// One thread of a converged warp.  (As the condition of what issues copies and MMAs: the compiler knows then that one
// thread runs it, and needs no loops over the warp for their uniform operands; with lane == 0 16384 x 8192 x 8192 took
// 1264 us, so 1162.)
LMOE_DEV bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// A place in the ring of stages.
template <int STAGES>
struct RingAt {
  uint32_t s = 0, phase = 0;
  LMOE_DEV void next() {
    if (++s == STAGES) {
      s = 0;
      phase ^= 1;
    }
  }
};

// (Of CTA scope: what it orders are TMEM reads and shared memory that this CTA's own tensor cores read.  A release at cluster
// scope would wait for the epilogue's global stores, an acquire cost the MMA issuer several hundred cycles a block:
// weight gradients of 8192 rows, 16 experts, 509 us instead of 267.)
LMOE_DEV void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
LMOE_DEV void set_at(uint32_t addr) { asm volatile("st.shared::cluster.u32 [%0], 1;" ::"r"(addr) : "memory"); }
// Registers of a warpgroup: 4 x 32 x 56 + 8 x 32 x 224 = 384 x 168, what the block was launched with.
template <int N>
LMOE_DEV void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
LMOE_DEV void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

LMOE_DEV void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 1 / (1 + exp(-g)), for g below 0 exp(g) / (1 + exp(g)): exp(-g) is infinity from g = -88.7 on, where the result is still
// 3e-39, and beside an up of 1e38 or so far from nothing.
LMOE_DEV float sigmoid(float g) {
  const float t = __expf(-fabsf(g));
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.f + t));
  return g < 0.f ? t * r : r;
}

// A tile as one CTA sees it.
struct Bf16Tile {
  int e, p0, q0;      // first lane (row of a; kWgrad: row of dw), first column
  int skip, live;     // lanes [skip, live) are the tile's
  int kb0, kb1;       // blocks of the reduction, of
  int blocks;         // so many
  int r0, rows;       // kWgrad: the expert's rows
  int second;         // kWgrad: of dw2
  bool brief;         // a short tile
};

LMOE_DEV int clamp_to(int v, int lo, int hi) { return min(max(v, lo), hi); }

// Offset i, clamped into the rows there are, so that no offsets send a load or a store out of range.
LMOE_DEV int offset_of(const Bf16Args& a, int i) {
  const int cap = static_cast<int>(a.rows);
  return a.offsets != nullptr ? clamp_to(__ldg(a.offsets + i), 0, cap) : i * cap;
}
// off: offsets (if they fit); start[e]: first row tile of group e (not kWgrad)
struct Bf16Walk {
  const int *off, *start;
  int total;
};

template <int MODE, int UNIT, bool CHUNKED>
LMOE_DEV Bf16Tile tile_at(const Bf16Walk& w, const Bf16Args& a, int id, int rank) {
  using C = Bf16Cfg<MODE, UNIT, CHUNKED>;
  Bf16Tile t = {};
  int i, rows;   // tile i of `rows` row tiles by by_others.d
  if (MODE == kWgrad) {
    t.e = a.by_tiles.div(id);
    i = id - t.e * static_cast<int>(a.by_tiles.d);
    rows = (a.n + UNIT - 1) / UNIT;
    const int one = rows * static_cast<int>(a.by_others.d);
    t.second = i >= one;
    if (t.second) i -= one;
  } else {
    int l = 0, h = a.E;   // the last e with start[e] * others <= id
    const int s = a.by_others.div(id);
    while (h - l > 1) {
      const int m = (l + h) >> 1;
      if (w.start[m] <= s) l = m;
      else h = m;
    }
    t.e = l;
    i = id - w.start[l] * static_cast<int>(a.by_others.d);
    rows = w.start[l + 1] - w.start[l];
  }
  const int g = a.by_group.div(i), first = g * kRaster, gm = min(kRaster, rows - first);
  const int local = i - g * static_cast<int>(a.by_group.d), other = local / gm;
  const int rt = first + local - other * gm;
  const bool near = C::kOffsets > kMaxGroups || a.E < C::kOffsets;
  const int lo = near ? w.off[t.e] : offset_of(a, t.e);
  const int hi = max(near ? w.off[t.e + 1] : offset_of(a, t.e + 1), lo);
  t.q0 = other * C::kOutCols;
  if (MODE == kWgrad) {
    t.p0 = rt * UNIT + (C::kPair ? rank * 128 : 0);
    t.live = min(a.n - t.p0, C::kLanes);
    t.r0 = lo;
    t.rows = hi - lo;
    t.blocks = (hi - lo + kBK - 1) / kBK;
  } else if (C::kPair) {
    const int p0 = lo + rt * UNIT;
    t.brief = C::kShort && hi - p0 <= 128;
    const int mine = t.brief ? 64 : 128;   // rows of this CTA
    t.p0 = p0 + rank * mine;
    t.live = min(hi - t.p0, mine);
    t.blocks = a.num_kb * a.pairs;
  } else {
    // Tiles of few rows: no row behind the last is asked for (a box filled with zeros past the end costs the
    // copy engine more than rows); a tile near the end starts earlier and skips the lanes before its own.
    const int p0 = lo + rt * UNIT;
    t.p0 = min(p0, static_cast<int>(a.rows) - a.box);
    t.skip = p0 - t.p0;
    t.live = t.skip + min(UNIT, hi - p0);
    t.blocks = a.num_kb * a.pairs;
  }
  t.kb1 = t.blocks;
  if (!C::kPair && a.splits > 1) {
    t.kb0 = static_cast<int>(static_cast<long long>(t.blocks) * rank / a.splits);
    t.kb1 = static_cast<int>(static_cast<long long>(t.blocks) * (rank + 1) / a.splits);
  }
  return t;
}

// ---- epilogue
LMOE_DEV float4 load4_bf16(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u));
}
LMOE_DEV float4 load4(const void* p, long long at, bool f32) {
  if (f32) return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
  return load4_bf16(static_cast<const __nv_bfloat16*>(p) + at);
}
LMOE_DEV void store4(void* out, long long at, float4 v, bool f32) {
  if (f32)
    *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = v;
  else
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at) =
        make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}
LMOE_DEV void gated_grad(float dh, float g, float u, float& dg, float& du) {
  const float s = sigmoid(g);
  dg = dh * (u * (s * (1.f + g * (1.f - s))));   // (dh u may leave fp32's range before the rest takes it back)
  du = dh * (g * s);
}
LMOE_DEV float silu_mul(float g, float u) { return g * sigmoid(g) * u; }
// Four sums v of out's element `at` (kGated: of gate and up) to where they belong (tiles shared by a cluster).
template <int MODE>
LMOE_DEV void finish4(const Bf16Args& a, void* out, long long at, float4 v, float4 v2) {
  if (MODE == kGated) {
    store4(a.out, at, make_float4(silu_mul(v.x, v2.x), silu_mul(v.y, v2.y), silu_mul(v.z, v2.z), silu_mul(v.w, v2.w)), false);
    if (a.out2 != nullptr) {
      store4(a.out2, at, v, false);
      store4(a.out3, at, v2, false);
    }
  } else if (MODE == kGatedGrad) {
    const float4 g = load4_bf16(a.gate + at), u = load4_bf16(a.up + at);
    float4 dg, du;
    gated_grad(v.x, g.x, u.x, dg.x, du.x);
    gated_grad(v.y, g.y, u.y, dg.y, du.y);
    gated_grad(v.z, g.z, u.z, dg.z, du.z);
    gated_grad(v.w, g.w, u.w, dg.w, du.w);
    store4(a.out, at, dg, false);
    store4(a.out2, at, du, false);
  } else {
    if (MODE == kWgrad && a.accumulate) {
      const float4 o = load4(out, at, a.out_f32);
      v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
    }
    store4(out, at, v, a.out_f32);
  }
}

// Finishes rows [skip, live) of a tile from the sums of `parts` CTAs: four columns of a row to a thread, of 4 << shift from
// column col0 on; row r of CTA q's sums is at red + (q rows + r) ld (kGated: up's behind gate's).
struct Bf16Sums {
  const float* red;
  int parts, rows, ld, shift, col0;
};
template <int MODE>
LMOE_DEV void finish_sums(const Bf16Args& a, const Bf16Sums& s, const Bf16Tile& t) {
  const int width = MODE == kWgrad ? a.k : a.n;
  void* out = MODE == kWgrad && t.second ? a.out2 : a.out;
  const long long row0 = (MODE == kWgrad ? static_cast<long long>(t.e) * a.n : 0) + t.p0;
  for (int i = threadIdx.x & 127; i < (t.live - t.skip) << s.shift; i += 128) {
    const int r = t.skip + (i >> s.shift), c = (i & ((1 << s.shift) - 1)) * 4, col = s.col0 + c;
    if (col >= width) continue;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f), v2 = v;
    for (int q = 0; q < s.parts; ++q) {
      const float* src = s.red + (q * s.rows + r) * s.ld + c;
      const float4 o = *reinterpret_cast<const float4*>(src);
      v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
      if (MODE == kGated) {
        const float4 p = *reinterpret_cast<const float4*>(src + (4 << s.shift));
        v2 = make_float4(v2.x + p.x, v2.y + p.y, v2.z + p.z, v2.w + p.w);
      }
    }
    finish4<MODE>(a, out, (row0 + r) * width + col, v, v2);
  }
}

// A warp's 32 rows of ROW bytes (128, or 64) in shared memory, one to a thread: their 16-byte parts swizzled as the tensor
// copies have them (part j of row r at j ^ (r % 8), or j ^ (r / 2 % 4)), which is free of bank conflicts by rows and by
// columns.
template <int ROW>
LMOE_DEV uint4* part_of(uint8_t* st, int r, int j) {
  return reinterpret_cast<uint4*>(st + r * ROW + ((j ^ (ROW == 128 ? r & 7 : r >> 1 & 3)) << 4));
}
template <int ROW>
LMOE_DEV void put_row(uint8_t* st, int lane, const uint32_t* w) {
#pragma unroll
  for (int j = 0; j < ROW / 16; ++j) *part_of<ROW>(st, lane, j) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
}
template <int ROW>
LMOE_DEV void get_row(uint8_t* st, int lane, uint32_t (&w)[ROW / 4]) {
#pragma unroll
  for (int j = 0; j < ROW / 16; ++j) {
    const uint4 q = *part_of<ROW>(st, lane, j);
    w[4 * j] = q.x;
    w[4 * j + 1] = q.y;
    w[4 * j + 2] = q.z;
    w[4 * j + 3] = q.w;
  }
}
template <bool THREE>
LMOE_DEV void tensor_store(const CUtensorMap* m, const void* src, int c0, int c1, int c2) {
  if constexpr (THREE)
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
  else
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(m)),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1)
                 : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// What an epilogue warp writes: rows [from, to) of 32 from row `row` of out (ld bytes each) on, `limit` bytes of each.
struct Bf16Rows {
  uint8_t* st;
  int lane, from, to;
  bool whole;        // by tensor stores
  long long row, ld;
  int limit;
  int r0, e;         // kWgrad: the first row of expert e's matrix
};
// The staged rows have been read (by whichever way the last ones left): they may be written again.
LMOE_DEV void staging_free() {
  if (elect_one()) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
}
// ROW bytes of each row, from byte `col` on, one row to a thread.
template <int MODE, int ROW>
LMOE_DEV void emit(const Bf16Rows& o, const CUtensorMap* m, void* out, int col, const uint32_t* w) {
  staging_free();
  put_row<ROW>(o.st, o.lane, w);
  if (o.whole) {
    fence_async_shared();
    __syncwarp();
    if (elect_one()) tensor_store<MODE == kWgrad>(m, o.st, col, MODE == kWgrad ? o.r0 : static_cast<int>(o.row), o.e);
  } else {
    __syncwarp();
    constexpr int kParts = ROW / 16, kAtOnce = 32 / kParts;   // rows to a store instruction
    const int j = o.lane % kParts, r0 = o.lane / kParts;
    uint8_t* p = static_cast<uint8_t*>(out) + (o.row + r0) * o.ld + col + j * 16;
#pragma unroll
    for (int i = 0; i < kParts; ++i, p += kAtOnce * o.ld) {
      const int r = kAtOnce * i + r0;
      const uint4 q = *part_of<ROW>(o.st, r, j);
      if (r >= o.from && r < o.to && col + j * 16 < o.limit) *reinterpret_cast<uint4*>(p) = q;
    }
  }
}
// 32 columns of sums, added to what the rows hold.
LMOE_DEV void emit_added(const Bf16Rows& o, void* out, int width, int col, bool f32, const uint32_t* w) {
  __syncwarp();
  put_row<128>(o.st, o.lane, w);
  __syncwarp();
  const int j = o.lane & 7, c = col + j * 4;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 4 * i + (o.lane >> 3);
    const float4 q = *reinterpret_cast<const float4*>(part_of<128>(o.st, r, j));
    if (r >= o.from && r < o.to && c < width) {
      const long long at = (o.row + r) * width + c;
      const float4 p = load4(out, at, f32);
      store4(out, at, make_float4(q.x + p.x, q.y + p.y, q.z + p.z, q.w + p.w), f32);
    }
  }
}

// Where an epilogue warp waits for sums, and gives their buffers back.
struct Bf16Ring {
  uint64_t* acc_full;
  uint32_t acc_empty;   // cluster address where the MMA issuer's barriers are (its own CTA's)
  unsigned* status;
  long long budget;
  LMOE_DEV bool wait(int tc) const {
    const bool ok = warp_wait(&acc_full[tc & 1], (tc >> 1) & 1, budget);
    if (!ok) atomicOr(status, kErrWaitEpilogue);
    tc_fence_after();
    return ok;
  }
  LMOE_DEV void release(int tc, int lane) const {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_cluster(acc_empty + (tc & 1) * 8);
  }
};
// The sums of a tile over all its chunks, `cols` (128 or 64) columns of this thread's lane from column c0 on, in registers;
// false if a wait gave up.
template <int BN>
LMOE_DEV bool gather_sums(const Bf16Ring& ring, uint32_t tmem, int c0, int cols, int chunks, int& tc, int lane, int quad,
                          float (&acc)[128]) {
  for (int ch = 0; ch < chunks; ++ch, ++tc) {
    if (!ring.wait(tc)) return false;
    const uint32_t tq = tmem + (tc & 1) * BN + c0 + (static_cast<uint32_t>(quad * 32) << 16);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c * 32 >= cols) break;
      uint32_t v[32];
      tmem_ld_32cols(tq + c * 32, v);
      tmem_ld_wait();
      if (ch == 0) {
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[c * 32 + i] = __uint_as_float(v[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) acc[c * 32 + i] += __uint_as_float(v[i]);
      }
    }
    ring.release(tc, lane);
  }
  return true;
}

// 64 columns of bf16 from two reads of 32.
LMOE_DEV void pack32(const uint32_t (&v)[32], uint32_t* w) {
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
}

struct Bf16Maps {
  const CUtensorMap *out, *out2, *out3, *gate, *up;
};

template <int MODE, int UNIT, bool CHUNKED>
LMOE_DEV void epilogue(const Bf16Args& args, const Bf16Walk& walk, const Bf16Ring& ring, const Bf16Maps& maps,
                       uint8_t* staging, uint64_t* landed, uint32_t tmem, int id0, int step, int rank) {
  using C = Bf16Cfg<MODE, UNIT, CHUNKED>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = warp & 3, half = (warp - 4) >> 2;
  constexpr int kCols = C::kOutCols * 4 / C::kEpiWarps;   // of this warp
  const int es = CHUNKED && args.out_f32 ? 4 : 2;
  const int width = MODE == kWgrad ? args.k : args.n;
  uint8_t* st = staging + (warp - 4) * C::kWarpBytes;
  uint8_t* in = st + 32 * C::kRow;   // kGatedGrad: gate's rows, and up's behind them
  uint64_t* mine = landed + (warp - 4);
  int tc = 0, loads = 0;
  for (int id = id0; id < walk.total; id += step) {
    const Bf16Tile t = tile_at<MODE, UNIT, CHUNKED>(walk, args, id, rank);
    const int blocks = t.kb1 - t.kb0;   // (kWgrad: an expert without rows has none, and gets zeros)
    // (short tiles: 64 rows, whose other columns are two quadrants on)
    const int rows0 = C::kShort && t.brief ? (quad & 1) * 32 : quad * 32;
    const int cols = C::kShort && t.brief ? kCols / 2 : kCols;
    const int q0 = t.q0 + half * cols + (C::kShort && t.brief ? (quad >> 1) * (C::kOutCols / 2) : 0);
    Bf16Rows o;
    o.st = st;
    o.lane = lane;
    o.from = max(t.skip - rows0, 0);
    o.to = min(t.live - rows0, 32);
    o.row = (MODE == kWgrad ? static_cast<long long>(t.e) * args.n : 0) + t.p0 + rows0;
    o.ld = static_cast<long long>(width) * es;
    o.limit = width * es;
    o.r0 = t.p0 + rows0;
    o.e = t.e;
    // (kWgrad's tensors end with an expert's rows; elsewhere the rows behind may be another expert's)
    o.whole = args.whole && (MODE == kWgrad || (o.from == 0 && o.to == 32));
    void* out = MODE == kWgrad && t.second ? args.out2 : args.out;
    const CUtensorMap* map = MODE == kWgrad && t.second ? maps.out2 : maps.out;
    const bool any = o.from < o.to && q0 < width;   // (the same for the warp)
    if (blocks == 0) {
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) w[i] = 0;
      if (any && !args.accumulate)
        for (int c = 0; c < kCols && q0 + c < width; c += C::kRow / es) emit<MODE, C::kRow>(o, map, out, (q0 + c) * es, w);
      continue;
    }
    if constexpr (CHUNKED) {
      constexpr bool kTwo = MODE == kGated || MODE == kGatedGrad;   // (another product beside each sum)
      static_assert(!kTwo || !C::kPair, "a warp has 64 columns of gate and the same of up");
      float acc[128];
      const int chunks = (blocks + C::kChunkBlocks - 1) / C::kChunkBlocks;
      if (!gather_sums<C::kBN>(ring, tmem, half * cols, kTwo ? 128 : cols, chunks, tc, lane, quad, acc)) break;
      if (!any) continue;
      const uint32_t* w = reinterpret_cast<const uint32_t*>(acc);
      if constexpr (kTwo) {   // (a row to a thread: a few us behind so long a reduction)
        if (lane >= o.from && lane < o.to) {
#pragma unroll
          for (int c = 0; c < kCols; c += 4) {
            constexpr int kUp = MODE == kGated ? 64 : 0;
            if (q0 + c < width)
              finish4<MODE>(args, out, (o.row + lane) * width + q0 + c, make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]),
                            make_float4(acc[c + kUp], acc[c + kUp + 1], acc[c + kUp + 2], acc[c + kUp + 3]));
          }
        }
      } else if (args.out_f32 || (MODE == kWgrad && args.accumulate)) {
#pragma unroll
        for (int c = 0; c < kCols; c += 32) {
          if (c >= cols || q0 + c >= width) break;
          if (MODE == kWgrad && args.accumulate) emit_added(o, out, width, q0 + c, args.out_f32, w + c);
          else emit<MODE, C::kRow>(o, map, out, (q0 + c) * 4, w + c);
        }
      } else {
#pragma unroll
        for (int c = 0; c < kCols; c += 64) {
          if (c >= cols || q0 + c >= width) break;
          uint32_t h[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) h[i] = pack_bf16x2(acc[c + 2 * i], acc[c + 2 * i + 1]);
          emit<MODE, C::kRow>(o, map, out, (q0 + c) * 2, h);
        }
      }
    } else {
      const auto load_gate = [&](int c) {   // 32 columns of gate and up
        if constexpr (MODE == kGatedGrad) {
          __syncwarp();
          if (elect_one()) {
            const uint32_t bar = smem_u32(mine);
            arrive_expect_tx(bar, 4096);
            load_2d<false>(smem_u32(in), maps.gate, bar, (q0 + c) * 2, o.r0, policy_evict_normal());
            load_2d<false>(smem_u32(in + 2048), maps.up, bar, (q0 + c) * 2, o.r0, policy_evict_normal());
          }
          __syncwarp();
        }
      };
      if (any) load_gate(0);
      bool ok = ring.wait(tc);
      if (any && ok) {
        const uint32_t tq = tmem + (tc & 1) * C::kBN + half * cols + (static_cast<uint32_t>(quad * 32) << 16);
        const int end = min(cols, width - q0);
        constexpr int kStep = C::kRow / 2;
#pragma unroll 1
        for (int c = 0; c < end; c += kStep) {
          const bool last = c + kStep >= end;
          uint32_t v[2][32];
          if constexpr (MODE == kGated) {
            uint32_t h[32], g[32], u[32];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              // (64 columns of gate, then the same of up)
              tmem_ld_32cols(tq + 2 * c + b * 32, v[0]);
              tmem_ld_32cols(tq + 2 * c + 64 + b * 32, v[1]);
              tmem_ld_wait();
              if (b == 1 && last) ring.release(tc, lane);   // (all of it has been read)
              pack32(v[0], g + b * 16);
              pack32(v[1], u + b * 16);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                v[0][i] = __float_as_uint(silu_mul(__uint_as_float(v[0][i]), __uint_as_float(v[1][i])));
              pack32(v[0], h + b * 16);
            }
            emit<MODE, C::kRow>(o, maps.out, args.out, (q0 + c) * 2, h);
            if (args.out2 != nullptr) {
              emit<MODE, C::kRow>(o, maps.out2, args.out2, (q0 + c) * 2, g);
              emit<MODE, C::kRow>(o, maps.out3, args.out3, (q0 + c) * 2, u);
            }
          } else if constexpr (MODE == kGatedGrad) {
            tmem_ld_32cols(tq + c, v[0]);
            tmem_ld_wait();
            if (last) ring.release(tc, lane);
            ok = warp_wait(mine, loads & 1, ring.budget);
            if (!ok) {
              atomicOr(ring.status, kErrWaitEpilogue);
              break;
            }
            ++loads;
            uint32_t g[16], u[16], w[16];
            get_row<64>(in, lane, g);
            get_row<64>(in + 2048, lane, u);
            // (the reads are done, not only issued, before the next rows may land on them: where the tensor cores fill
            // shared memory's bandwidth they were overtaken)
            fence_async_shared();
            if (!last) load_gate(c + 32);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float dg[2], du[2];
#pragma unroll
              for (int b = 0; b < 2; ++b) {
                const uint32_t gi = b ? g[i] & 0xffff0000u : g[i] << 16, ui = b ? u[i] & 0xffff0000u : u[i] << 16;
                gated_grad(__uint_as_float(v[0][2 * i + b]), __uint_as_float(gi), __uint_as_float(ui), dg[b], du[b]);
              }
              w[i] = pack_bf16x2(dg[0], dg[1]);
              u[i] = pack_bf16x2(du[0], du[1]);
            }
            emit<MODE, C::kRow>(o, maps.out, args.out, (q0 + c) * 2, w);
            emit<MODE, C::kRow>(o, maps.out2, args.out2, (q0 + c) * 2, u);
          } else {
            tmem_ld_32cols(tq + c, v[0]);
            tmem_ld_32cols(tq + c + 32, v[1]);
            tmem_ld_wait();
            if (last) ring.release(tc, lane);
            if (MODE == kWgrad && args.accumulate) {
              emit_added(o, out, width, q0 + c, false, v[0]);
              if (q0 + c + 32 < width) emit_added(o, out, width, q0 + c + 32, false, v[1]);
            } else {
              uint32_t w[32];
              pack32(v[0], w);
              pack32(v[1], w + 16);
              emit<MODE, C::kRow>(o, map, out, (q0 + c) * 2, w);
            }
          }
        }
      } else if (ok) {
        ring.release(tc, lane);
      }
      if (!ok) {
        if (MODE == kGatedGrad && any) warp_wait(mine, loads & 1, kDrain);   // (what was asked for lands here)
        break;
      }
      ++tc;
    }
  }
  // what this warp stored is there before the CTA leaves
  if (elect_one()) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  __syncwarp();
}

// Epilogue of tiles of few rows.  What a tile takes here is what bounds short reductions: a warp's own way (rows by tensor or
// segment stores, gate and up of 32 columns at a time) took 5.8 us a tile for kGatedGrad.
template <int MODE, int UNIT, bool CHUNKED>
LMOE_DEV void epilogue_flat(const Bf16Args& args, const Bf16Walk& walk, const Bf16Ring& ring, float* sums, uint32_t tmem, int id0,
                            int step) {
  using C = Bf16Cfg<MODE, UNIT, CHUNKED>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kShift = C::kOutCols == 128 ? 5 : 4;   // fours of columns
  int tc = 0, turn = 0;
  for (int id = id0; id < walk.total; id += step, turn ^= 1) {
    const Bf16Tile t = tile_at<MODE, UNIT, CHUNKED>(walk, args, id, 0);
    float* buf = sums + turn * 32 * C::kLdFlat;
    bool ok = true;
    if (warp == 4) {
      float acc[128];
      const int chunks = (t.blocks + C::kChunkBlocks - 1) / C::kChunkBlocks;
      ok = gather_sums<C::kBN>(ring, tmem, 0, 128, chunks, tc, lane, 0, acc);
      if (ok && lane >= t.skip && lane < t.live) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          *reinterpret_cast<float4*>(buf + lane * C::kLdFlat + 4 * i) =
              make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
      }
    }
    // (a buffer is written again after the next tile's barrier, which all reach when they are done with it)
    if (!named_barrier_all(1, 128, ok)) break;
    finish_sums<MODE>(args, {buf, 1, 32, C::kLdFlat, kShift, t.q0}, t);
  }
}

template <int MODE, int UNIT, bool CHUNKED>
__global__ void __launch_bounds__(Bf16Cfg<MODE, UNIT, CHUNKED>::kThreads, 1)
    gemm_bf16_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA2,
                     const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmB2,
                     const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CUtensorMap tmO2,
                     const __grid_constant__ CUtensorMap tmO3, const __grid_constant__ CUtensorMap tmGate,
                     const __grid_constant__ CUtensorMap tmUp, const Bf16Args args) {
  using C = Bf16Cfg<MODE, UNIT, CHUNKED>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* staging = smem + C::kStages * C::kStageBytes;
  int* off = reinterpret_cast<int*>(staging + C::kStagingBytes);   // [E + 1]
  int* start = off + C::kOffsets;                                  // [E + 1] (not kWgrad)
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + C::kStagingBytes + C::kTableBytes);
  uint64_t* empty = full + C::kStages;
  uint64_t* tail = empty + C::kStages;       // kWgrad: a block with rows to be cleared has landed
  uint64_t* acc_full = tail + C::kStages;    // [2]
  uint64_t* acc_empty = acc_full + 2;        // [2]
  uint64_t* mma_done = acc_empty + 2;
  uint64_t* landed = mma_done + 1;           // [4] kGatedGrad: a warp's rows of gate and up
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(landed + 4);
  uint32_t* gave_up = tmem_slot + 1;         // whether a producer of either CTA of a pair did

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], C::kPair && MODE == kWgrad ? 2 : 1);
      mbar_init(&empty[s], 1);
      mbar_init(&tail[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], C::kFlat ? 1 : C::kEpiWarps * (C::kPair ? 2 : 1));
    }
    mbar_init(mma_done, 1);
    for (int i = 0; i < 4; ++i) mbar_init(&landed[i], 1);
    *gave_up = 0;
    fence_mbar_init();
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
    if (args.pairs > 1) prefetch_tmap(&tmA2);
    if (MODE == kGated || (MODE != kWgrad && args.pairs > 1)) prefetch_tmap(&tmB2);
  }
  if (warp == 1) {
    if (C::kPair) {
      tmem_alloc_pair(tmem_slot, C::kTmemCols);
    } else {
      tmem_alloc(tmem_slot, C::kTmemCols);
      tmem_relinquish();
    }
  }
  griddep_enter();

  if (C::kOffsets > kMaxGroups || args.E < C::kOffsets)
    for (int e = threadIdx.x; e <= args.E; e += C::kThreads) off[e] = offset_of(args, e);
  __syncthreads();
  if (MODE != kWgrad && warp == 0) {   // start[]: exclusive prefix sum of the row tiles, a run of groups per lane
    const int per = (args.E + 31) / 32, e0 = min(lane * per, args.E), e1 = min(e0 + per, args.E);
    // no more than the launch has room for, whatever the offsets say
    const int most = most_tiles(static_cast<int>(args.rows), args.E, UNIT);
    int sum = 0;
    for (int e = e0; e < e1; ++e) sum += (max(off[e + 1] - off[e], 0) + UNIT - 1) / UNIT;
    int run = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(~0u, run, d);
      if (lane >= d) run += up;
    }
    const int tot = __shfl_sync(~0u, run, 31);
    run -= sum;
    for (int e = e0; e < e1; ++e) {
      start[e] = min(run, most);
      run += (max(off[e + 1] - off[e], 0) + UNIT - 1) / UNIT;
    }
    if (lane == 0) start[args.E] = min(tot, most);
  }
  tc_fence_before();
  __syncthreads();
  if (C::kPair) cluster_sync();   // both CTAs' barriers are there
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Bf16Walk walk;
  walk.off = off;
  walk.start = start;
  walk.total = MODE == kWgrad ? args.E * static_cast<int>(args.by_tiles.d)
                              : start[args.E] * static_cast<int>(args.by_others.d);
  const int S = C::kPair ? 2 : args.splits;   // CTAs of a cluster
  const int rank = static_cast<int>(blockIdx.x % S);
  const int id0 = static_cast<int>(blockIdx.x) / S, step = static_cast<int>(gridDim.x) / S;
  const long long budget = args.budget;
  unsigned* const status = args.status != nullptr ? args.status : &g_status;

  const Bf16Ring ring = {acc_full, C::kPair ? cluster_map(smem_u32(acc_empty), 0) : smem_u32(acc_empty), status, budget};
  if (warp < 4) {
    if constexpr (C::kPair && CHUNKED) regs_dec<56>();
    const uint32_t stages = smem_u32(smem), full0 = smem_u32(full), empty0 = smem_u32(empty), tail0 = smem_u32(tail);
    const uint32_t lead0 = C::kPair ? cluster_map(full0, 0) : full0;   // the barriers that the MMA issuer waits for
    if ((warp == 0 || warp == 3) && elect_one()) {
      // ---- TMA producers, warp 0 of the lane operand, warp 3 of the column operand
      const bool lanes = warp == 0;
      const uint64_t pol = policy_evict_normal();
      const uint32_t tx = (MODE == kWgrad || C::kPair ? C::kABytes : args.box * 128) + C::kBBytes;
      RingAt<C::kStages> at;
      int issued = 0;
      uint32_t cleared = 0, phases = 0;   // stages whose last block went by its tail barrier; those barriers' parities
      bool ok = true;
      for (int id = id0; ok && id < walk.total; id += step) {
        const Bf16Tile t = tile_at<MODE, UNIT, CHUNKED>(walk, args, id, rank);
        // the column operand's part of this CTA
        const int qb = t.q0 + (C::kPair ? rank * (C::kOutCols / 2) : 0);
        const CUtensorMap* map = lanes ? (MODE == kWgrad && t.second ? &tmA2 : &tmA) : &tmB;
        int k0 = (MODE == kWgrad ? t.r0 : 0) + t.kb0 * kBK;   // of the reduction
        for (int kb = t.kb0; kb < t.kb1; ++kb, k0 += kBK) {
          if (MODE != kGated && MODE != kWgrad && kb == args.num_kb) {   // on to the second pair
            map = lanes ? &tmA2 : &tmB2;
            k0 = 0;
          } else if (MODE != kGated && MODE != kWgrad && kb == t.kb0 && kb > args.num_kb) {
            map = lanes ? &tmA2 : &tmB2;
            k0 = (kb - args.num_kb) * kBK;
          }
          const uint32_t s = at.s;
          if (!wait_at(empty0 + s * 8, at.phase ^ 1, budget)) {
            atomicOr(status, kErrWaitProducer);
            ok = false;
            break;
          }
          const bool fix = MODE == kWgrad && kb + 1 == t.blocks && t.rows % 16 != 0;   // cleared before it is full
          const uint32_t bar = fix ? tail0 + s * 8 : lead0 + s * 8;
          const uint32_t dst = stages + s * C::kStageBytes + (lanes ? 0 : C::kABytes);
          if (MODE == kWgrad) {
            cleared = (cleared & ~(1u << s)) | (fix ? 1u << s : 0u);
            phases ^= fix ? 1u << s : 0u;
          }
          if (lanes) {
            if (fix || !C::kPair) arrive_expect_tx(fix ? bar : full0 + s * 8, tx);
            else if (rank == 0) arrive_expect_tx(full0 + s * 8, 2 * (t.brief ? tx - 8192 : tx));
            else if (MODE == kWgrad) mbar_arrive_cluster(bar);
          }
          // (the maps' innermost coordinates are bytes)
          if (MODE == kWgrad) {
            const int c = (lanes ? t.p0 : qb) * 2;
            if (fix) {
              load_2d<false>(dst, map, bar, c, k0, pol);
              load_2d<false>(dst + 8192, map, bar, c + 128, k0, pol);
            } else {
              load_2d<C::kPair>(dst, map, bar, c, k0, pol);
              load_2d<C::kPair>(dst + 8192, map, bar, c + 128, k0, pol);
            }
          } else if (lanes) {
            load_2d<C::kPair>(dst, map, bar, k0 * 2, t.p0, pol);   // (a pair's: 64 rows at a time)
            if (C::kPair && !t.brief) load_2d<C::kPair>(dst + 8192, map, bar, k0 * 2, t.p0 + 64, pol);
          } else if (C::kColsMn) {
            load_3d<C::kPair>(dst, map, bar, qb * 2, k0, t.e, pol);
            load_3d<C::kPair>(dst + 8192, map, bar, qb * 2 + 128, k0, t.e, pol);
          } else {   // (kGated: 64 rows of gate and the same of up)
            load_3d<C::kPair>(dst, map, bar, k0 * 2, qb, t.e, pol);
            if (MODE == kGated) load_3d<C::kPair>(dst + 8192, &tmB2, bar, k0 * 2, qb, t.e, pol);
          }
          at.next();
          ++issued;
        }
      }
      // Every copy lands before the CTA leaves.  A pair's are counted by the first CTA, and neither leaves before the other; once
      // any of a pair's producers gave up, the others may have copies that the first CTA does not count (see the teardown).
      if (C::kPair && !ok) {
        set_at(cluster_map(smem_u32(gave_up), 0));
        set_at(cluster_map(smem_u32(gave_up), 1));
      }
      for (int j = max(0, issued - C::kStages); j < issued; ++j) {
        const int s = j % C::kStages;
        const bool tail_bar = MODE == kWgrad && (cleared >> s & 1);
        if (C::kPair && rank != 0 && !tail_bar) continue;
        const bool landed = tail_bar ? wait_at(tail0 + s * 8, (phases >> s & 1) ^ 1, kDrain)
                                     : wait_at(full0 + s * 8, (j / C::kStages) & 1, kDrain);
        if (!landed) {
          atomicOr(status, kErrDrain);
          break;
        }
      }
    } else if (warp == 1 && (!C::kPair || rank == 0) && elect_one()) {
      // ---- MMA issuer
      constexpr uint32_t kMajor = (C::kLanesMn ? 1u << 15 : 0u) | (C::kColsMn ? 1u << 16 : 0u);
      constexpr uint32_t kWhole = idesc_bf16_f32(C::kPair ? 256 : 128, C::kBN) | kMajor;
      constexpr uint32_t kBrief = idesc_bf16_f32(128, C::kBN) | kMajor;
      constexpr int kStepA = C::kLanesMn ? 128 : 2, kStepB = C::kColsMn ? 128 : 2;   // 16 on, in 16-byte addresses
      const uint64_t ad0 = C::kLanesMn ? sw128_mnmajor_desc(stages) : sw128_kmajor_desc(stages);
      const uint64_t bd0 = C::kColsMn ? sw128_mnmajor_desc(stages + C::kABytes) : sw128_kmajor_desc(stages + C::kABytes);
      const auto commit = [](uint64_t* bar) {
        if (C::kPair) mma_commit_pair(bar);
        else mma_commit(bar);
      };
      uint32_t idesc = kWhole;
      const auto mma = [&](uint32_t acc, uint64_t a, uint64_t b, bool add) {
        if (C::kPair) mma_bf16_pair(acc, a, b, idesc, add);
        else mma_bf16(acc, a, b, idesc, add);
      };
      RingAt<C::kStages> at;
      int tc = 0;
      bool ok = true;
      for (int id = id0; ok && id < walk.total; id += step) {
        const Bf16Tile t = tile_at<MODE, UNIT, CHUNKED>(walk, args, id, rank);
        if (C::kShort) idesc = t.brief ? kBrief : kWhole;
        for (int c0 = t.kb0; ok && c0 < t.kb1; c0 += C::kChunkBlocks, ++tc) {
          const int buf = tc & 1, c1 = min(t.kb1 - c0, C::kChunkBlocks) + c0;
          if (!mbar_wait(&acc_empty[buf], ((tc >> 1) & 1) ^ 1, budget)) {
            atomicOr(status, kErrWaitMma);
            ok = false;
            break;
          }
          const uint32_t acc = tmem + buf * C::kBN;
          for (int kb = c0; kb < c1; ++kb) {
            if (!wait_at(full0 + at.s * 8, at.phase, budget)) {
              atomicOr(status, kErrWaitMma);
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t ad = ad0 + at.s * (C::kStageBytes / 16), bd = bd0 + at.s * (C::kStageBytes / 16);
            mma(acc, ad, bd, kb > c0);
            // of the reduction, 64 in all but its last blocks
            const int left = MODE == kWgrad ? t.rows - kb * kBK : args.k - (kb >= args.num_kb ? kb - args.num_kb : kb) * kBK;
            if (left >= kBK) {
#pragma unroll
              for (int kk = 1; kk < kBK / 16; ++kk) mma(acc, ad + kStepA * kk, bd + kStepB * kk, true);
            } else {
              for (int kk = 1; kk * 16 < left; ++kk) mma(acc, ad + kStepA * kk, bd + kStepB * kk, true);
            }
            commit(&empty[at.s]);
            at.next();
          }
          commit(&acc_full[buf]);
        }
      }
      commit(mma_done);
    } else if (MODE == kWgrad && warp == 2) {
      // ---- rows behind an expert's last, cleared in both operands
      int it = 0;
      uint32_t phases = 0;
      for (int id = id0; id < walk.total; id += step) {
        const Bf16Tile t = tile_at<MODE, UNIT, CHUNKED>(walk, args, id, rank);
        it += t.kb1 - t.kb0;
        if (t.rows % 16 == 0 || t.kb0 == t.kb1 || t.kb1 != t.blocks) continue;
        const int s = (it - 1) % C::kStages;
        if (!warp_wait(&tail[s], phases >> s & 1, budget)) {
          atomicOr(status, kErrWaitProducer);
          break;
        }
        phases ^= 1u << s;
        const int r = (t.rows - 1) % kBK + 1, end = (r + 15) / 16 * 16;   // rows [r, end) of each of the four boxes
        uint8_t* at = smem + s * C::kStageBytes;
        for (int i = lane; i < (end - r) * 32; i += 32) {
          const int box = i >> 3 & 3, k = r + (i >> 5);
          *reinterpret_cast<uint4*>(at + box * 8192 + k * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(C::kPair ? cluster_map(smem_u32(&full[s]), 0) : smem_u32(&full[s]));
      }
    }
  } else {
    if constexpr (C::kPair && CHUNKED) regs_inc<224>();
    if (C::kPair || S == 1) {
      if constexpr (C::kFlat) {
        epilogue_flat<MODE, UNIT, CHUNKED>(args, walk, ring, reinterpret_cast<float*>(staging), tmem, id0, step);
      } else {
        const Bf16Maps maps = {&tmO, &tmO2, &tmO3, &tmGate, &tmUp};
        epilogue<MODE, UNIT, CHUNKED>(args, walk, ring, maps, staging, landed, tmem, id0, step, rank);
      }
    }
  }

  if constexpr (!C::kPair) {
    if (S > 1) {
      // One tile per cluster, each CTA with a part of the reduction.  CTA q finishes the q-th part of the columns: every CTA's
      // sums of those go to its stages (free once its own MMAs are done), and it adds them in rank order.  All threads
      // pass the cluster barriers, whatever their role.
      const bool mine = warp >= 4 && id0 < walk.total;
      const int row = (warp & 3) * 32 + lane, rows = MODE == kWgrad ? 128 : args.box;
      constexpr int kParts = C::kOutCols / 4;   // fours of columns of the result
      const int shift = __ffs(kParts) - __ffs(S), part = 4 << shift;   // columns of a CTA
      const int width = (MODE == kGated ? 2 * part : part) + 4;          // floats of a row of sums
      Bf16Tile t = {};
      float acc[128];
      if (mine) {
        t = tile_at<MODE, UNIT, CHUNKED>(walk, args, id0, rank);
        int tc = 0;
        const int n = t.kb1 - t.kb0, chunks = (n + C::kChunkBlocks - 1) / C::kChunkBlocks;
        const bool ok = C::kFlat && warp != 4 ? true : gather_sums<C::kBN>(ring, tmem, 0, 128, chunks, tc, lane, warp & 3, acc);
        if (!ok || chunks == 0) {
#pragma unroll
          for (int i = 0; i < 128; ++i) acc[i] = 0.f;
        }
      }
      cluster_sync();
      if (mine && row < rows) {
        const uint32_t at = smem_u32(smem) + (rank * rows + row) * width * 4;
#pragma unroll
        for (int i = 0; i < 32; ++i) {   // (kGated: 16 of gate, 16 of up)
          const int p = i % kParts, c = (p & ((1 << shift) - 1)) * 4 + (i < kParts ? 0 : part);
          cluster_store(cluster_map(at, p >> shift) + c * 4,
                        make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]));
        }
      }
      cluster_sync();
      if (mine && !(MODE == kWgrad && args.accumulate && t.blocks == 0))
        finish_sums<MODE>(args, {reinterpret_cast<const float*>(smem), S, rows, width, shift, t.q0 + rank * part}, t);
    }
  }
  // ---- teardown: all MMAs of this CTA have completed before the columns are released.  (A pair's second CTA, whose warp 1 has had
  // nothing to do so far, waits once the first one is done: the arrival here is then under way.)
  const bool issuer = !C::kPair || rank == 0;
  if (issuer && warp == 1 && lane == 0)
    if (!mbar_wait(mma_done, 0, kDrain)) atomicOr(status, kErrDrain);
  tc_fence_before();
  if (C::kPair) cluster_sync();
  else __syncthreads();
  // (no producer of either CTA issues any more: what was not counted lands within this millisecond, in both CTAs' memory and on
  // the first one's barriers)
  if (C::kPair && warp == 3 && lane == 0 && *gave_up != 0)
    for (const long long t0 = clock64(); clock64() - t0 < kLast;) __nanosleep(1000);
  if (!issuer && warp == 1) {
    if (!warp_wait(mma_done, 0, kDrain) && lane == 0) atomicOr(status, kErrDrain);
  }
  if (warp == 1) {
    tc_fence_after();
    if (C::kPair) tmem_dealloc_pair(tmem, C::kTmemCols);
    else tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int MODE, int UNIT, bool CHUNKED>
cudaError_t launch_one(const CUtensorMap (&m)[9], Bf16Args a, cudaStream_t s) {
  using C = Bf16Cfg<MODE, UNIT, CHUNKED>;
  const unsigned others = ((MODE == kWgrad ? a.k : a.n) + C::kOutCols - 1) / C::kOutCols;
  const long long row_tiles = MODE == kWgrad ? (a.n + UNIT - 1) / UNIT : most_tiles(static_cast<int>(a.rows), a.E, UNIT);
  a.by_others = FastDiv::of(others);
  a.by_group = FastDiv::of(others * kRaster);
  a.by_tiles = FastDiv::of(static_cast<unsigned>(MODE == kWgrad ? row_tiles * others * a.pairs : 1));
  const long long tiles = row_tiles * others * (MODE == kWgrad ? 1LL * a.E * a.pairs : 1);
  auto kern = gemm_bf16_kernel<MODE, UNIT, CHUNKED>;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), C::kSmemBytes);
  if (e != cudaSuccess) return e;
  if (a.splits > 1)
    return launch_pdl_cluster(kern, dim3(static_cast<unsigned>(tiles * a.splits)), dim3(C::kThreads), C::kSmemBytes, s,
                              a.splits, m[0], m[1], m[2], m[3], m[4], m[5], m[6], m[7], m[8], a);
  const long long sms = sm_count();
  if (C::kPair)
    return launch_pdl_cluster(kern, dim3(static_cast<unsigned>(tiles < sms / 2 ? tiles : sms / 2) * 2), dim3(C::kThreads),
                              C::kSmemBytes, s, 2, m[0], m[1], m[2], m[3], m[4], m[5], m[6], m[7], m[8], a);
  return launch_pdl(kern, dim3(static_cast<unsigned>(tiles < sms ? tiles : sms)), dim3(C::kThreads), C::kSmemBytes, s,
                    m[0], m[1], m[2], m[3], m[4], m[5], m[6], m[7], m[8], a);
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
constexpr int kSms = 152;
constexpr int kFewRows = 16, kFewTiles = 8, kPairRows = 96, kPairTiles = 46;

// [rows, cols] bf16, boxes of 64 columns (half: 32) by `high` rows; and [E, rows, cols]
bool map_rows(CUtensorMap* m, const void* p, long long rows, int cols, int high, bool half = false) {
  const unsigned long long d[2] = {2ull * cols, static_cast<unsigned long long>(rows)}, st[1] = {2ull * cols};
  const unsigned box[2] = {half ? 64u : 128u, static_cast<unsigned>(high)};
  return encode_u8_swizzled(m, p, 2, d, st, box, half);
}
bool map_weights(CUtensorMap* m, const void* p, int E, int rows, int cols, int high) {
  const unsigned long long d[3] = {2ull * cols, static_cast<unsigned long long>(rows), static_cast<unsigned long long>(E)};
  const unsigned long long st[2] = {2ull * cols, 2ull * cols * rows};
  const unsigned box[3] = {128, static_cast<unsigned>(high), 1};
  return encode_u8_swizzled(m, p, 3, d, st, box);
}

// What all four entry points check of a shape.
lmoe_status check_shape(const lmoe_bf16_matmul* c, const int32_t* offsets) {
  if (c == nullptr || c->rows < 0 || c->N <= 0 || c->K <= 0 || c->n_experts <= 0 || c->wait_budget_cycles < 0)
    return LMOE_ERR_ARG;
  if (offsets == nullptr && c->n_experts != 1) return LMOE_ERR_ARG;
  if (c->out_dtype != LMOE_F32 && c->out_dtype != LMOE_BF16) return LMOE_ERR_UNSUPPORTED;
  if (c->n_experts > kMaxGroups || c->K % 8 || c->N % 8 || c->K > (1 << 20) || c->N > (1 << 20) || c->rows > (1LL << 24))
    return LMOE_ERR_UNSUPPORTED;
  if ((c->rows / 128 + c->n_experts) * ((c->N + 63) / 64) > 0x7fffffffLL) return LMOE_ERR_UNSUPPORTED;   // tiles of the narrowest
  return LMOE_OK;
}
// A matrix in memory, or the offsets: where it begins, and its bytes.
struct Span {
  const void* p;
  long long n;
};
// Whether no result (the first `results`) shares memory with another one or with an operand.
template <int N>
bool apart(const Span (&m)[N], int results) {
  for (int i = 0; i < results; ++i)
    for (int j = i + 1; j < N; ++j) {
      if (m[i].p == nullptr || m[j].p == nullptr) continue;
      const uintptr_t a = reinterpret_cast<uintptr_t>(m[i].p), b = reinterpret_cast<uintptr_t>(m[j].p);
      if (a < b + m[j].n && b < a + m[i].n) return false;
    }
  return true;
}
Bf16Args args_of(const lmoe_bf16_matmul* c, const int32_t* offsets, uint32_t* status) {
  Bf16Args g = {};
  g.rows = c->rows;
  g.n = c->N;
  g.k = c->K;
  g.num_kb = (c->K + kBK - 1) / kBK;
  g.pairs = 1;
  g.E = c->n_experts;
  g.offsets = offsets;
  g.splits = 1;
  g.out_f32 = c->out_dtype == LMOE_F32;
  g.status = status;
  g.budget = c->wait_budget_cycles > 0 ? c->wait_budget_cycles : kDefaultWaitBudget;
  return g;
}

// Clusters of s such CTAs (one to an SM) that run side by side: fewer than the SMs' number divided by s, since a cluster keeps
// to one GPC and those have any number of SMs (clusters of 8: 16 of them took 27 us for what 14 do in 16).
int most_clusters(int s) {
  static std::mutex mu;
  static int known[9] = {};
  std::lock_guard<std::mutex> lock(mu);
  if (known[s] == 0) {
    using C = Bf16Cfg<kProduct, 32, false>;
    auto kern = gemm_bf16_kernel<kProduct, 32, false>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(s);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(s);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (allow_smem(reinterpret_cast<const void*>(kern), C::kSmemBytes) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = kSms / s;
    }
    known[s] = n;
  }
  return known[s];
}
// CTAs (a cluster) for each of few tiles: as long as all clusters run side by side, and with at least four blocks of the
// reduction to a CTA.  Fewer than `from` blocks are not shared: the sums' way to the CTAs that finish them takes 2 to 3 us.
int splits_for(long long tiles, long long blocks, int from) {
  int s = 1;
  while (s < 8 && blocks >= from && tiles * s * 2 <= kSms && blocks / (s * 2) >= 4 && tiles <= most_clusters(s * 2)) s *= 2;
  return s;
}
// Cycles, about, of tiles of 256 rows (in a pair a block of 64 takes 600, or 430 if none of them has more than 128 rows) and of 128
// (575, shared by s CTAs), by their waves over the SMs; a pair takes 3000 longer to start and end, a cluster 5000.  (2811 rows of
// 1000 x 8184: 60 us by pairs, 115 by tiles of 128 rows; 32 of 8192 x 1024 12.8 and 8.5.)
long long pair_cycles(long long tiles, long long blocks, bool brief) {
  return (tiles + kSms / 2 - 1) / (kSms / 2) * blocks * (brief ? 430 : 600) + 3000;
}
long long one_cycles(long long tiles, long long blocks, int s) {
  return (tiles * s + kSms - 1) / kSms * blocks * 575 / s + (s > 1 ? 5000 : 0);
}
// One of the modes that take rows of a: which tile, and the launch.  A pair is (a, w).
//
// Tiles of 32 rows up to kFewRows rows per expert on average, or where kFewTiles tiles of 128 rows or fewer would leave most
// SMs idle; of 256 rows from kPairTiles of them and kPairRows rows per expert on, or for fewer rows where the weights' rows are
// no multiple of 128 bytes (a box then takes two lines for each of its rows, and the pair takes fewer boxes in); else of
// 128.  One matrix, whose tiles are known: of 256 or 128 rows by the cycles they take.  Measured in us, 32 / 128 / 256 rows each:
//   64 experts of 4096 x 4096, even splits     8 rows   318 / 326 / 333      64 rows    382 / 337 / 343
//                                              16       320 / 328 / 335      128        779 / 345 / 353
//                                              32       325 / 330 / 338      160        920 / 483 / 376
//   uneven splits, by the average              16       322 / 330 / 335      64         464 / 345 / 346
//                                              32       333 / 333 / 339      96         666 / 370 / 354
//   20 experts of 6768 x 7800, uneven          20       381 / 531 / 401      80         897 / 598 / 428
//   one matrix of 4096 x 4096                  128      17 / 17 / 18         512        50 / 22 / 25
//                                              256      28 / 19 / 24         1024       83 / 37 / 26
//   one of 1024 x 4096                         128      11 / 16 / 17         1024       28 / 19 / 24
// A cluster shares the reduction where tiles are few, from 24 blocks on for 32 rows, 48 for 128 and for weight gradients, 8 for
// kGatedGrad (whose tiles a cluster finishes with more threads).  Shared and not: one row of 4096 x 4096 10.0 and 19 us, 16
// rows of 2048 x 2048 8.5 and 10.7, of 1024 x 1024 8.4 and 8.1; 100 rows of 2048 x 4096 13.2 and 15.4, of 2048 x 2048 11.8 and 11.0;
// kGatedGrad 16 rows of 1024 x 1024 9.4 and 13.8; weight gradients of 256 x 256 over 32768, 8000, 4000, 2000 rows 24.5, 15.4, 13.8,
// 11.9 and (a pair's tile) 142, 22, 16.9, 11.4.
template <int MODE, bool CHUNKED>
lmoe_status rows_product(Bf16Args g, const void* a, const void* w, const void* a2, const void* w2, cudaStream_t stream) {
  const int R = static_cast<int>(g.rows), live = g.E < R ? g.E : R;
  const auto tiles_of = [&](int unit) {
    const int across = (MODE == kGated ? 64 : 128) * (unit == 256 ? 2 : 1);
    return 1LL * most_tiles(R, g.E, unit) * ((g.n + across - 1) / across);
  };
  const bool few = R / live <= kFewRows || tiles_of(128) <= kFewTiles;
  constexpr bool mn = MODE == kGatedGrad || MODE == kProductT;
  const int wr = mn ? g.k : g.n, wc = mn ? g.n : g.k;   // a weight's rows and columns
  const long long blocks = g.num_kb * g.pairs;
  const int from = MODE == kGatedGrad ? 8 : few ? 24 : 48, shared = splits_for(tiles_of(few ? 32 : 128), blocks, from);
  // (gate's and up's sums of more than one chunk: a warp of one CTA has the same columns of both in registers, a pair's has not)
  constexpr bool single = CHUNKED && (MODE == kGated || MODE == kGatedGrad);
  const bool pair = single     ? false
                    : g.E == 1 ? pair_cycles(tiles_of(256), blocks, R <= 128) < one_cycles(tiles_of(128), blocks, shared)
                               : tiles_of(256) >= kPairTiles && (wc % 64 != 0 || R / live >= kPairRows);
  const int unit = few ? 32 : pair ? 256 : 128;
  g.box = R < unit ? R : unit;
  if (unit < 256) g.splits = shared;
  const int high = mn || MODE == kGated ? 64 : 128;
  const int rows = unit == 256 ? 64 : g.box;
  CUtensorMap m[9];
  if (!map_rows(&m[0], a, R, g.k, rows) || !map_weights(&m[2], w, g.E, wr, wc, high)) return LMOE_ERR_CUDA;
  for (int i = 1; i < 9; ++i)   // (some are not used)
    if (i != 2) m[i] = m[i == 3 ? 2 : 0];
  g.whole = unit > 32 && g.splits == 1;
  if (g.whole) {
    const int es = g.out_f32 ? 2 : 1;   // (in 16-bit columns)
    constexpr bool half = MODE == kGatedGrad;
    if (!map_rows(&m[4], g.out, R, g.n * es, 32, half) || (g.out2 != nullptr && !map_rows(&m[5], g.out2, R, g.n * es, 32, half)) ||
        (g.out3 != nullptr && !map_rows(&m[6], g.out3, R, g.n * es, 32)))
      return LMOE_ERR_CUDA;
  }
  if (MODE == kGatedGrad && unit > 32 && (!map_rows(&m[7], g.gate, R, g.n, 32, true) || !map_rows(&m[8], g.up, R, g.n, 32, true)))
    return LMOE_ERR_CUDA;
  if ((a2 != nullptr && !map_rows(&m[1], a2, R, g.k, rows)) || (w2 != nullptr && !map_weights(&m[3], w2, g.E, wr, wc, high)))
    return LMOE_ERR_CUDA;
  cudaError_t e = cudaErrorInvalidValue;
  if (unit == 32) {
    e = launch_one<MODE, 32, CHUNKED>(m, g, stream);
  } else if (unit == 128) {
    e = launch_one<MODE, 128, CHUNKED>(m, g, stream);
  } else if constexpr (!single) {
    e = launch_one<MODE, 256, CHUNKED>(m, g, stream);
  }
  return e == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}

}  // namespace
}  // namespace lmoe

using namespace lmoe;

extern "C" lmoe_status lmoe_gated_ffn(const lmoe_bf16_matmul* c, const void* x, const void* w_gate, const void* w_up,
                                      const int32_t* offsets, void* h, void* gate, void* up, uint32_t* status,
                                      cudaStream_t stream) {
  const lmoe_status st = check_shape(c, offsets);
  if (st != LMOE_OK) return st;
  if (c->transposed || c->accumulate || (gate == nullptr) != (up == nullptr)) return LMOE_ERR_ARG;
  if (c->out_dtype != LMOE_BF16) return LMOE_ERR_UNSUPPORTED;
  if (c->rows == 0) return LMOE_OK;
  if (x == nullptr || w_gate == nullptr || w_up == nullptr || h == nullptr) return LMOE_ERR_ARG;
  if (!aligned(x, 16) || !aligned(w_gate, 16) || !aligned(w_up, 16) || !aligned(h, 16) || !aligned(gate, 16) ||
      !aligned(up, 16) || !aligned(offsets, 4) || !aligned(status, 4))
    return LMOE_ERR_ALIGN;
  const long long rn = 2LL * c->rows * c->N, w = 2LL * c->n_experts * c->N * c->K, o = 4LL * (c->n_experts + 1);
  if (!apart<8>({{h, rn}, {gate, rn}, {up, rn}, {x, 2LL * c->rows * c->K}, {w_gate, w}, {w_up, w}, {offsets, o}, {status, 4}}, 3))
    return LMOE_ERR_ARG;
  Bf16Args g = args_of(c, offsets, status);
  g.out = h;
  g.out2 = gate;
  g.out3 = up;
  return g.num_kb > kLong ? rows_product<kGated, true>(g, x, w_gate, nullptr, w_up, stream)
                          : rows_product<kGated, false>(g, x, w_gate, nullptr, w_up, stream);
}

extern "C" lmoe_status lmoe_gated_ffn_grad(const lmoe_bf16_matmul* c, const void* dy, const void* w_down,
                                           const void* gate, const void* up, const int32_t* offsets, void* dgate,
                                           void* dup, uint32_t* status, cudaStream_t stream) {
  const lmoe_status st = check_shape(c, offsets);
  if (st != LMOE_OK) return st;
  if (c->transposed || c->accumulate) return LMOE_ERR_ARG;
  if (c->out_dtype != LMOE_BF16) return LMOE_ERR_UNSUPPORTED;
  if (c->rows == 0) return LMOE_OK;
  if (dy == nullptr || w_down == nullptr || gate == nullptr || up == nullptr || dgate == nullptr || dup == nullptr)
    return LMOE_ERR_ARG;
  if (!aligned(dy, 16) || !aligned(w_down, 16) || !aligned(gate, 16) || !aligned(up, 16) || !aligned(dgate, 16) ||
      !aligned(dup, 16) || !aligned(offsets, 4) || !aligned(status, 4))
    return LMOE_ERR_ALIGN;
  const long long rn = 2LL * c->rows * c->N, w = 2LL * c->n_experts * c->N * c->K, o = 4LL * (c->n_experts + 1);
  const void* g_in = gate == dgate ? nullptr : gate;   // (in place)
  const void* u_in = up == dup ? nullptr : up;
  if (!apart<8>({{dgate, rn}, {dup, rn}, {g_in, rn}, {u_in, rn}, {dy, 2LL * c->rows * c->K}, {w_down, w}, {offsets, o}, {status, 4}}, 2))
    return LMOE_ERR_ARG;
  Bf16Args g = args_of(c, offsets, status);
  g.gate = static_cast<const __nv_bfloat16*>(gate);
  g.up = static_cast<const __nv_bfloat16*>(up);
  g.out = dgate;
  g.out2 = dup;
  return g.num_kb > kLong ? rows_product<kGatedGrad, true>(g, dy, w_down, nullptr, nullptr, stream)
                          : rows_product<kGatedGrad, false>(g, dy, w_down, nullptr, nullptr, stream);
}

extern "C" lmoe_status lmoe_matmul_bf16(const lmoe_bf16_matmul* c, const void* a, const void* w, const void* a2,
                                        const void* w2, const int32_t* offsets, void* out, uint32_t* status,
                                        cudaStream_t stream) {
  const lmoe_status st = check_shape(c, offsets);
  if (st != LMOE_OK) return st;
  if (c->accumulate) return LMOE_ERR_ARG;
  if (c->rows == 0) return LMOE_OK;   // (an empty tensor's address may be null)
  if ((a2 == nullptr) != (w2 == nullptr)) return LMOE_ERR_ARG;
  if (a == nullptr || w == nullptr || out == nullptr) return LMOE_ERR_ARG;
  if (!aligned(a, 16) || !aligned(w, 16) || !aligned(a2, 16) || !aligned(w2, 16) || !aligned(out, 16) ||
      !aligned(offsets, 4) || !aligned(status, 4))
    return LMOE_ERR_ALIGN;
  const long long rk = 2LL * c->rows * c->K, wb = 2LL * c->n_experts * c->N * c->K, o = 4LL * (c->n_experts + 1);
  const long long rn = (c->out_dtype == LMOE_F32 ? 4LL : 2LL) * c->rows * c->N;
  if (!apart<7>({{out, rn}, {a, rk}, {a2, rk}, {w, wb}, {w2, wb}, {offsets, o}, {status, 4}}, 1)) return LMOE_ERR_ARG;
  Bf16Args g = args_of(c, offsets, status);
  g.pairs = a2 != nullptr ? 2 : 1;
  g.out = out;
  const bool chunked = g.out_f32 || g.num_kb * g.pairs > kLong;
  if (c->transposed)
    return chunked ? rows_product<kProductT, true>(g, a, w, a2, w2, stream)
                   : rows_product<kProductT, false>(g, a, w, a2, w2, stream);
  return chunked ? rows_product<kProduct, true>(g, a, w, a2, w2, stream)
                 : rows_product<kProduct, false>(g, a, w, a2, w2, stream);
}

extern "C" lmoe_status lmoe_matmul_bf16_wgrad(const lmoe_bf16_matmul* c, const void* dy, const void* x,
                                              const void* dy2, const int32_t* offsets, void* dw, void* dw2,
                                              uint32_t* status, cudaStream_t stream) {
  const lmoe_status st = check_shape(c, offsets);
  if (st != LMOE_OK) return st;
  if (c->transposed || dw == nullptr) return LMOE_ERR_ARG;
  if (c->rows > 0 && (dy == nullptr || x == nullptr || (dy2 == nullptr) != (dw2 == nullptr))) return LMOE_ERR_ARG;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(dy2, 16) || !aligned(dw, 16) || !aligned(dw2, 16) ||
      !aligned(offsets, 4) || !aligned(status, 4))
    return LMOE_ERR_ALIGN;
  if (c->rows == 0) {
    if (c->accumulate) return LMOE_OK;
    const size_t bytes = static_cast<size_t>(c->n_experts) * c->N * c->K * (c->out_dtype == LMOE_F32 ? 4 : 2);
    if (cudaMemsetAsync(dw, 0, bytes, stream) != cudaSuccess) return LMOE_ERR_CUDA;
    if (dw2 != nullptr && cudaMemsetAsync(dw2, 0, bytes, stream) != cudaSuccess) return LMOE_ERR_CUDA;
    return LMOE_OK;
  }
  Bf16Args g = args_of(c, offsets, status);
  g.num_kb = 0;
  g.pairs = dy2 != nullptr ? 2 : 1;
  g.out = dw;
  g.out2 = dw2;
  g.accumulate = c->accumulate != 0;
  const long long tiles = 1LL * ((c->N + 127) / 128) * ((c->K + 127) / 128) * c->n_experts * g.pairs;
  if (tiles > 0x7fffffffLL) return LMOE_ERR_UNSUPPORTED;
  const long long rn = 2LL * c->rows * c->N, o = 4LL * (c->n_experts + 1);
  const long long wb = (g.out_f32 ? 4LL : 2LL) * c->n_experts * c->N * c->K;
  if (!apart<7>({{dw, wb}, {dw2, wb}, {dy, rn}, {dy2, rn}, {x, 2LL * c->rows * c->K}, {offsets, o}, {status, 4}}, 2)) return LMOE_ERR_ARG;
  CUtensorMap m[9];
  const int es = g.out_f32 ? 2 : 1;   // (in 16-bit columns)
  const long long wide = 1LL * ((c->N + 255) / 256) * ((c->K + 255) / 256) * c->n_experts * g.pairs;
  const long long blocks = c->rows / c->n_experts / kBK + 1;
  const int shared = splits_for(tiles, blocks, 48);
  // (a tile's store takes as long as some 8 blocks; an expert of one row, 4096 x 4096: 21.0 us by pairs, 28.8 without this)
  const long long least = blocks > 8 ? blocks : 8;
  const bool pair = pair_cycles(wide, least, false) < one_cycles(tiles, least, shared);
  if (!pair) g.splits = shared;
  g.whole = !g.accumulate && g.splits == 1;
  if (!map_rows(&m[0], dy, c->rows, c->N, kBK) || !map_rows(&m[2], x, c->rows, c->K, kBK) ||
      !map_weights(&m[4], dw, g.E, g.n, g.k * es, 32))
    return LMOE_ERR_CUDA;
  for (int i = 1; i < 9; ++i)   // (some are not used)
    if (i != 2 && i != 4) m[i] = m[0];
  if (dw2 != nullptr && !map_weights(&m[5], dw2, g.E, g.n, g.k * es, 32)) return LMOE_ERR_CUDA;
  if (dy2 != nullptr && !map_rows(&m[1], dy2, c->rows, c->N, kBK)) return LMOE_ERR_CUDA;
  const bool chunked = g.out_f32 || c->rows > 1LL * kLong * kBK;   // (one expert may have all rows)
  const cudaError_t e = chunked ? (pair ? launch_one<kWgrad, 256, true>(m, g, stream) : launch_one<kWgrad, 128, true>(m, g, stream))
                                : (pair ? launch_one<kWgrad, 256, false>(m, g, stream) : launch_one<kWgrad, 128, false>(m, g, stream));
  return e == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}

extern "C" lmoe_status lmoe_bf16_check_status(cudaStream_t stream, uint32_t* detail) {
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

extern "C" lmoe_status lmoe_bf16_wait_selftest(long long budget_cycles, cudaStream_t stream) {
  const long long b = budget_cycles < 1 ? 1 : budget_cycles > kDefaultWaitBudget ? kDefaultWaitBudget : budget_cycles;
  void* word = nullptr;
  if (cudaGetSymbolAddress(&word, g_status) != cudaSuccess) return LMOE_ERR_CUDA;
  return launch_wait_selftest(b, static_cast<unsigned*>(word), stream) == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}
