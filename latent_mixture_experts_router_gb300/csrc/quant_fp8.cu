// quant_fp8.cu — 8-bit floating-point quantisation with one fp32 scale per block of 128, in the
// three layouts the 8-bit products read (gemm_fp8.cu).
//
// Rule, every rounding in fp32 and in this order (M the format's largest value: e4m3 448,
// e5m2 57344):
//   s = max(amax / M, 2^-126)       (with pow2: rounded up to a power of two)
//   code = nearest-even(v * (1 / s)), saturating
// The floor keeps 1 / s finite for a block of zeros.  amax is taken on the magnitudes' bit
// patterns, whose order puts infinity and NaN on top, so a block that holds one gets a scale that
// is not finite instead of hiding it.
//
// rows:   [rows, K], a block is 128 of a row; scales [K/128][rows]; rows gathered by index
// weight: [G][N, K], a block is 128 x 128; scales [N/128][K/128]; the transpose on request
// cols:   [rows, K], a block is 128 rows of one column; codes transposed, [K][padded rows], each
//         expert's rows padded to whole blocks; scales [blocks][K]
// All three read and write each element once; the memory traffic bounds them.  Measured: 16384 x 8192
// bf16 rows 59.9 us (6.7 TB/s), 4096 x 4096 gathered to 8 rows each 43.1 us (issue slots: each row is
// converted eight times); 8 x 4096 x 4096 bf16 weights, both orientations, 81.7 us (6.6 TB/s); columns of 16384 x
// 4096 bf16 41.3 us (4.9 TB/s, issue slots at 65 %).
#include <algorithm>

#include "../../include/latent_moe.h"
#include "internal.h"
#include "ptx.cuh"

namespace lmoe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxGroups = 1024;

struct Fmt {
  float largest;
  int pow2;
};
// four codes, a's in the low byte
template <bool E5M2>
LMOE_DEV uint32_t cvt4(float a, float b, float c, float d) {
  uint32_t r;
  if constexpr (E5M2)
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e5m2x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e5m2x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}" : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
  else
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}" : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
// four codes of v * s, the products two to an instruction: the conversions' issue slots are what the
// gathered rows wait for (4096 x 4096 bf16 to 8 rows each, the same inputs in each call: 40.3 us, one product an instruction 41.4;
// weights 80.9 and 81.6; columns the same, fp32 ones 62.2 and 61.4: those keep single products)
template <bool E5M2>
LMOE_DEV uint32_t cvt4_scaled(float a, float b, float c, float d, float s) {
  const auto mul = [&](float& x, float& y) {
    asm("{\n\t.reg .b64 v, w;\n\tmov.b64 v, {%0, %1};\n\tmov.b64 w, {%2, %2};\n\t"
        "mul.rn.f32x2 v, v, w;\n\tmov.b64 {%0, %1}, v;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(s));
  };
  mul(a, b);
  mul(c, d);
  return cvt4<E5M2>(a, b, c, d);
}
LMOE_DEV float scale_of(uint32_t amax_bits, const Fmt& f) {
  float s = __fdiv_rn(__uint_as_float(amax_bits), f.largest);
  if (s < 1.17549435e-38f) s = 1.17549435e-38f;
  if (f.pow2) {
    const uint32_t b = __float_as_uint(s);
    if (b < 0x7f800000u) s = __uint_as_float((b + 0x7fffffu) & 0x7f800000u);
  }
  return s;
}
LMOE_DEV uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// the larger magnitudes of two pairs of bf16 (of any sign: masked when the last is found), NaN if
// either is
LMOE_DEV uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// 16 or 8 bytes, with ALL or zeros where `on` is not set (a predicated load: no branch around it)
template <bool ALL>
LMOE_DEV uint4 load16(const void* p, bool on) {
  if constexpr (ALL) return *static_cast<const uint4*>(p);
  uint4 q;
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
               "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
               "@p ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
               : "=&r"(q.x), "=&r"(q.y), "=&r"(q.z), "=&r"(q.w) : "l"(p), "r"(static_cast<int>(on)));
  return q;
}
template <bool ALL>
LMOE_DEV uint2 load8(const void* p, bool on) {
  if constexpr (ALL) return *static_cast<const uint2*>(p);
  uint2 q;
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
               "@p ld.global.v2.b32 {%0, %1}, [%2];\n\t}"
               : "=&r"(q.x), "=&r"(q.y) : "l"(p), "r"(static_cast<int>(on)));
  return q;
}
constexpr uint32_t kMag = 0x7fffffffu;   // an fp32's magnitude
LMOE_DEV float lo16(uint32_t w) { return __uint_as_float(w << 16); }
LMOE_DEV float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// N consecutive elements of a row, as loaded, and their magnitudes.  Magnitudes are compared as
// bit patterns: 32 bits for fp32, 16 for bf16 (two to a word).
template <typename T, int N>
struct Raw;
template <int N>
struct Raw<float, N> {
  uint32_t w[N];
  template <bool VEC, bool ALL = false>
  LMOE_DEV void load(const float* p, bool on = true) {   // zeros where `on` is not set
#pragma unroll
    for (int j = 0; j < N / 4; ++j) {
      if constexpr (VEC) {
        const uint4 q = load16<ALL>(p + 4 * j, on);
        w[4 * j] = q.x, w[4 * j + 1] = q.y, w[4 * j + 2] = q.z, w[4 * j + 3] = q.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[4 * j + i] = on ? __float_as_uint(p[4 * j + i]) : 0u;
      }
    }
  }
  LMOE_DEV float get(int i) const { return __uint_as_float(w[i]); }
};
template <int N>
struct Raw<__nv_bfloat16, N> {
  uint32_t w[N / 2];
  template <bool VEC, bool ALL = false>
  LMOE_DEV void load(const __nv_bfloat16* p, bool on = true) {
    if constexpr (VEC && N == 8) {
      const uint4 q = load16<ALL>(p, on);
      w[0] = q.x, w[1] = q.y, w[2] = q.z, w[3] = q.w;
    } else if constexpr (VEC) {
      const uint2 q = load8<ALL>(p, on);
      w[0] = q.x, w[1] = q.y;
    } else {
      const unsigned short* u = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
      for (int j = 0; j < N / 2; ++j) w[j] = on ? u[2 * j] | (static_cast<uint32_t>(u[2 * j + 1]) << 16) : 0u;
    }
  }
  LMOE_DEV float get(int i) const { return i & 1 ? hi16(w[i >> 1]) : lo16(w[i >> 1]); }
};

// ------------------------------------------------------------------ rows
// Half a warp reads 128 elements of a row (8 per lane), of all its rows before it works on any; a
// warp takes 16 (fp32: 8) rows of one block of columns, warps beside each other the next blocks
// of the same rows.  The maxima of a half's rows are reduced together: each step of the butterfly
// halves the rows a lane carries, so that eight rows cost five shuffles and a lane ends up with
// one row, whose scale it alone works out; the reciprocals are then handed round.
struct RowsArgs {
  const void* src;
  long long ld, src_rows, rows;
  const int32_t* index;
  int K, kb;
  unsigned chunks;   // ceil(kb / kb_warps)
  int kb_warps;
  Fmt f;
  uint8_t* codes;
  float* scales;
};
template <typename T>
constexpr int kHalfRows = sizeof(T) == 2 ? 8 : 4;   // rows of half a warp
template <typename T, bool VEC, bool E5M2>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 5 : 4) rows_kernel(const RowsArgs a) {
  griddep_enter();
  constexpr int R = kHalfRows<T>;
  const int lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
  // the CTA's warps: kb_warps blocks of columns (a power of two) x the rest in rows
  const int warp = threadIdx.x >> 5;
  const int kb = (blockIdx.x % a.chunks) * a.kb_warps + (warp & (a.kb_warps - 1));
  const long long w0 = static_cast<long long>(blockIdx.x / a.chunks) * (kThreads / 32 / a.kb_warps) + warp / a.kb_warps;
  const long long r0 = w0 * (2 * R) + half * R;   // this half's first row
  if (r0 - half * R >= a.rows || kb >= a.kb) return;
  const int c = kb * 128 + l * 8;
  const bool in_k = c < a.K;   // K is a multiple of 16
  int mine = -1;               // lane j < R of a half: source row of row r0 + j (at most 2^24)
  if (l < R && r0 + l < a.rows) {
    mine = a.index != nullptr ? a.index[r0 + l] : static_cast<int>(r0) + l;
    if (mine < 0 || mine >= a.src_rows) mine = -1;
  }
  const T* src = static_cast<const T*>(a.src) + c;
  const bool whole = __all_sync(~0u, in_k && (l >= R || mine >= 0));   // nothing to leave out
  Raw<T, 8> v[R];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int q = __shfl_sync(~0u, mine, half * 16 + j);
    if (whole) v[j].template load<VEC, true>(src + q * a.ld);
    else v[j].template load<VEC>(src + q * a.ld, q >= 0 && in_k);
  }
  uint32_t m[4];   // bf16: rows i (low half) and i + 4 (high half); fp32: row i
  const auto mx = [](uint32_t x, uint32_t y) { return sizeof(T) == 2 ? max_u16x2(x, y) : max(x, y); };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      uint32_t p[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t* w = v[i + 4 * h].w;
        p[h] = max_abs_bf16x2(max_abs_bf16x2(w[0], w[1]), max_abs_bf16x2(w[2], w[3]));
      }
      // row i's two halves in the low halves of two words, row i + 4's in the high ones
      m[i] = max_u16x2(__byte_perm(p[0], p[1], 0x5410) & 0x7fff7fffu, __byte_perm(p[0], p[1], 0x7632) & 0x7fff7fffu);
    } else {
      m[i] = 0u;
#pragma unroll
      for (int e = 0; e < 8; ++e) m[i] = max(m[i], v[i].w[e] & kMag);
    }
  }
  {   // lane l keeps row (l >> 3 & 1) * 2 + (l >> 2 & 1)
    const bool b3 = l & 8, b2 = l & 4;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t other = __shfl_xor_sync(~0u, b3 ? m[i] : m[i + 2], 8);
      m[i] = mx(b3 ? m[i + 2] : m[i], other);
    }
    const uint32_t other = __shfl_xor_sync(~0u, b2 ? m[0] : m[1], 4);
    m[0] = mx(b2 ? m[1] : m[0], other);
    m[0] = mx(m[0], __shfl_xor_sync(~0u, m[0], 2));
    m[0] = mx(m[0], __shfl_xor_sync(~0u, m[0], 1));
  }
  // bf16: the even lanes work out the low half's row, the odd ones the high half's
  const int row = ((l >> 3) & 1) * 2 + ((l >> 2) & 1) + (sizeof(T) == 2 ? 4 * (l & 1) : 0);
  const uint32_t bits = sizeof(T) == 2 ? (l & 1 ? m[0] & 0xffff0000u : m[0] << 16) : m[0];
  const float s = scale_of(bits, a.f), inv = __frcp_rn(s);
  if ((l & 2) == 0 && (sizeof(T) == 2 || (l & 1) == 0) && r0 + row < a.rows)
    a.scales[static_cast<long long>(kb) * a.rows + r0 + row] = s;
  uint8_t* dst = a.codes + r0 * a.K + c;
#pragma unroll
  for (int j = 0; j < R; ++j, dst += a.K) {
    const float rj = __shfl_sync(~0u, inv, half * 16 + ((j >> 1) & 1) * 8 + (j & 1) * 4 + (j >> 2));
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = cvt4_scaled<E5M2>(v[j].get(4 * i), v[j].get(4 * i + 1), v[j].get(4 * i + 2), v[j].get(4 * i + 3), rj);
    if (r0 + j < a.rows && in_k) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
  }
}

// ------------------------------------------------------------------ 128 x 128 tiles
// Warp w holds rows 16 w .. 16 w + 15 of a tile, lane l columns 4 l .. 4 l + 3: a row's loads and
// stores are whole lines, and a thread's 16 rows of one column are 16 bytes of the transpose.
// Those pass through shared memory, chunk w of column c at place w ^ ((c / 4) % 8), which keeps
// both the writes (32 columns apart by 128 bytes) and the reads free of bank conflicts.
// Magnitudes of a thread's four columns over its rows: two words of packed 16-bit patterns for
// bf16, four words for fp32.
template <typename T>
struct ColMax;
template <>
struct ColMax<float> {
  uint4 m;
  LMOE_DEV void add(const Raw<float, 4>& v) {
    m = make_uint4(max(m.x, v.w[0] & kMag), max(m.y, v.w[1] & kMag), max(m.z, v.w[2] & kMag), max(m.w, v.w[3] & kMag));
  }
  LMOE_DEV void add(const ColMax& o) {
    m = make_uint4(max(m.x, o.m.x), max(m.y, o.m.y), max(m.z, o.m.z), max(m.w, o.m.w));
  }
  LMOE_DEV uint32_t bits(int j) const { return j == 0 ? m.x : j == 1 ? m.y : j == 2 ? m.z : m.w; }
};
template <>
struct ColMax<__nv_bfloat16> {
  uint2 m;
  LMOE_DEV void add(const Raw<__nv_bfloat16, 4>& v) {
    m = make_uint2(max_u16x2(m.x, v.w[0] & 0x7fff7fffu), max_u16x2(m.y, v.w[1] & 0x7fff7fffu));
  }
  LMOE_DEV void add(const ColMax& o) { m = make_uint2(max_u16x2(m.x, o.m.x), max_u16x2(m.y, o.m.y)); }
  LMOE_DEV uint32_t bits(int j) const {
    const uint32_t w = j < 2 ? m.x : m.y;
    return j & 1 ? w & 0xffff0000u : w << 16;
  }
};
// CTAs an SM holds: bf16 rows take half the registers.  (bf16, 8 x 4096 x 4096 weights: 3 CTAs 85 us,
// 4 87; columns of 16384 x 4096: 4 CTAs 41 us, 3 44)
template <typename T>
constexpr int kWeightCtas = sizeof(T) == 2 ? 3 : 2;
template <typename T>
constexpr int kColsCtas = sizeof(T) == 2 ? 4 : 2;

// writes the transposed tile from shared memory: column c's 128 bytes to dst + c * ld
LMOE_DEV void store_transposed(const uint8_t* tile, uint8_t* dst, long long ld, int ncols, int nbytes) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunk = lane & 7;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = warp * 16 + i * 4 + (lane >> 3);
    const uint4 q = *reinterpret_cast<const uint4*>(tile + c * 128 + ((chunk ^ ((c >> 2) & 7)) << 4));
    if (c < ncols && chunk * 16 < nbytes) *reinterpret_cast<uint4*>(dst + c * ld + chunk * 16) = q;
  }
}

struct WeightArgs {
  const void* src;   // [G][N, K]
  int N, K, nb, kb;
  Fmt f;
  uint8_t *codes, *codes_t;
  float *scales, *scales_t;
};
template <typename T, bool VEC, bool E5M2>
__global__ void __launch_bounds__(kThreads, kWeightCtas<T>) weight_kernel(const WeightArgs a) {
  __shared__ __align__(16) uint8_t tile[128 * 128];
  __shared__ uint32_t wmax[kThreads / 32];
  griddep_enter();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kb = blockIdx.x % a.kb;
  const long long gn = blockIdx.x / a.kb;
  const long long g = gn / a.nb;
  const int nb = static_cast<int>(gn % a.nb);
  const int n0 = nb * 128 + warp * 16, k0 = kb * 128 + lane * 4;
  const T* src = static_cast<const T*>(a.src) + (g * a.N + n0) * a.K + k0;
  Raw<T, 4> v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    v[i].template load<VEC>(src + static_cast<long long>(i) * a.K, n0 + i < a.N && k0 < a.K);
  }
  ColMax<T> cm{};
#pragma unroll
  for (int i = 0; i < 16; ++i) cm.add(v[i]);
  uint32_t m = __reduce_max_sync(~0u, max(max(cm.bits(0), cm.bits(1)), max(cm.bits(2), cm.bits(3))));
  if (lane == 0) wmax[warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) m = max(m, wmax[w]);
  const float s = scale_of(m, a.f), inv = __frcp_rn(s);
  if (threadIdx.x == 0) {
    a.scales[(g * a.nb + nb) * a.kb + kb] = s;
    if (a.scales_t != nullptr) a.scales_t[(g * a.kb + kb) * a.nb + nb] = s;
  }
  uint32_t tr[4][4];   // tr[j][q]: column j, rows 4 q .. 4 q + 3
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t w[4];   // four rows of four columns
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Raw<T, 4>& x = v[4 * q + i];
      w[i] = cvt4_scaled<E5M2>(x.get(0), x.get(1), x.get(2), x.get(3), inv);
      if (n0 + 4 * q + i < a.N && k0 < a.K)
        *reinterpret_cast<uint32_t*>(a.codes + (g * a.N + n0 + 4 * q + i) * a.K + k0) = w[i];
    }
    const uint32_t lo = __byte_perm(w[0], w[1], 0x5140), lo2 = __byte_perm(w[2], w[3], 0x5140);   // columns 0, 1
    const uint32_t up = __byte_perm(w[0], w[1], 0x7362), up2 = __byte_perm(w[2], w[3], 0x7362);   // columns 2, 3
    tr[0][q] = __byte_perm(lo, lo2, 0x5410);
    tr[1][q] = __byte_perm(lo, lo2, 0x7632);
    tr[2][q] = __byte_perm(up, up2, 0x5410);
    tr[3][q] = __byte_perm(up, up2, 0x7632);
  }
  if (a.codes_t == nullptr) return;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4*>(tile + (lane * 4 + j) * 128 + ((warp ^ (lane & 7)) << 4)) =
        make_uint4(tr[j][0], tr[j][1], tr[j][2], tr[j][3]);
  __syncthreads();
  store_transposed(tile, a.codes_t + (g * a.K + kb * 128) * a.N + nb * 128, a.N, a.K - kb * 128, a.N - nb * 128);
}

struct ColsArgs {
  const void* src;
  long long ld, src_rows, rows, padded;   // rows: routed rows; padded: columns of codes_t
  const int32_t* index;
  const int32_t* offsets;
  int E, K, kb;
  Fmt f;
  uint8_t* codes;
  float* scales;
};
template <typename T, bool VEC, bool E5M2>
__global__ void __launch_bounds__(kThreads, kColsCtas<T>) cols_kernel(const ColsArgs a) {
  __shared__ __align__(16) uint8_t tile[128 * 128];
  __shared__ ColMax<T> cmax[kThreads / 32][32];
  __shared__ int start[kMaxGroups + 1], lo[kMaxGroups], hi[kMaxGroups];
  griddep_enter();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cap = static_cast<int>(a.rows);
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    int l = 0, h = cap;
    if (a.offsets != nullptr) {   // clamped: no table reads or writes out of range
      l = min(max(a.offsets[e], 0), cap);
      h = min(max(a.offsets[e + 1], l), cap);
    }
    lo[e] = l;
    hi[e] = h;
  }
  __syncthreads();
  if (warp == 0) {   // first block of each expert
    const int per = (a.E + 31) / 32, e0 = min(lane * per, a.E), e1 = min(e0 + per, a.E);
    int sum = 0;
    for (int e = e0; e < e1; ++e) sum += (hi[e] - lo[e] + 127) / 128;
    int run = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int up = __shfl_up_sync(~0u, run, d);
      if (lane >= d) run += up;
    }
    const int tot = __shfl_sync(~0u, run, 31), most = static_cast<int>(a.padded / 128);
    run -= sum;
    for (int e = e0; e < e1; ++e) {
      start[e] = min(run, most);
      run += (hi[e] - lo[e] + 127) / 128;
    }
    if (lane == 0) start[a.E] = min(tot, most);
  }
  __syncthreads();
  const long long units = static_cast<long long>(start[a.E]) * a.kb;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int blk = static_cast<int>(u / a.kb), kb = static_cast<int>(u % a.kb);
    int l = 0, h = a.E;
    while (h - l > 1) {
      const int mid = (l + h) >> 1;
      if (start[mid] <= blk) l = mid;
      else h = mid;
    }
    const int r0 = lo[l] + (blk - start[l]) * 128 + warp * 16, k0 = kb * 128 + lane * 4;
    const int rend = hi[l];
    int mine = -1;   // lane i < 16: source row of row r0 + i
    if (lane < 16 && r0 + lane < rend) {
      mine = a.index != nullptr ? a.index[r0 + lane] : r0 + lane;
      if (mine < 0 || mine >= a.src_rows) mine = -1;
    }
    const T* src = static_cast<const T*>(a.src) + k0;
    Raw<T, 4> v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int q = __shfl_sync(~0u, mine, i);
      v[i].template load<VEC>(src + q * a.ld, q >= 0 && k0 < a.K);
    }
    ColMax<T> m{};
#pragma unroll
    for (int i = 0; i < 16; ++i) m.add(v[i]);
    cmax[warp][lane] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m.add(cmax[w][lane]);
    float inv[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float s = scale_of(m.bits(j), a.f);
      inv[j] = __frcp_rn(s);
      if (warp == 0 && k0 + j < a.K) a.scales[static_cast<long long>(blk) * a.K + k0 + j] = s;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        w[q] = cvt4<E5M2>(v[4 * q].get(j) * inv[j], v[4 * q + 1].get(j) * inv[j], v[4 * q + 2].get(j) * inv[j],
                          v[4 * q + 3].get(j) * inv[j]);
      *reinterpret_cast<uint4*>(tile + (lane * 4 + j) * 128 + ((warp ^ (lane & 7)) << 4)) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
    __syncthreads();
    store_transposed(tile, a.codes + static_cast<long long>(kb) * 128 * a.padded + blk * 128LL, a.padded,
                     a.K - kb * 128, 128);
    __syncthreads();   // the tile and the maxima are written again
  }
}

bool on(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
int cdiv(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }
bool dtype_ok(lmoe_dtype d) { return d == LMOE_F32 || d == LMOE_BF16; }
Fmt fmt_of(lmoe_fp8_format f, int pow2) { return Fmt{f == LMOE_FP8_E5M2 ? 57344.f : 448.f, pow2 != 0}; }

// f(T, VEC, E5M2) for the source's type and alignment and the codes' format
template <typename F>
cudaError_t by_source(lmoe_dtype d, bool vec, lmoe_fp8_format fmt, F f) {
  const auto with = [&](auto t, auto v) {
    return fmt == LMOE_FP8_E5M2 ? f(t, v, std::true_type{}) : f(t, v, std::false_type{});
  };
  if (d == LMOE_F32) return vec ? with(float{}, std::true_type{}) : with(float{}, std::false_type{});
  return vec ? with(__nv_bfloat16{}, std::true_type{}) : with(__nv_bfloat16{}, std::false_type{});
}

}  // namespace
}  // namespace lmoe

using namespace lmoe;

extern "C" long long lmoe_fp8_padded_rows(long long rows, int n_experts) {
  if (rows <= 0 || n_experts <= 0) return 0;
  return (rows + 127 * std::min<long long>(n_experts, rows)) / 128 * 128;
}

extern "C" lmoe_status lmoe_quantize_fp8_rows(const void* src, lmoe_dtype src_dtype, long long ld_src,
                                              const int32_t* row_index, long long src_rows, long long rows, int K,
                                              lmoe_fp8_format format, int pow2_scales, uint8_t* codes, float* scales,
                                              cudaStream_t stream) {
  if (rows < 0 || src_rows < 0 || K <= 0 || ld_src < K || (format != LMOE_FP8_E4M3 && format != LMOE_FP8_E5M2))
    return LMOE_ERR_ARG;
  if (row_index == nullptr && src_rows < rows) return LMOE_ERR_ARG;
  if (!dtype_ok(src_dtype) || K % 16 || K > (1 << 20) || rows > (1LL << 24)) return LMOE_ERR_UNSUPPORTED;
  if (rows == 0) return LMOE_OK;
  if ((src == nullptr && src_rows > 0) || codes == nullptr || scales == nullptr) return LMOE_ERR_ARG;
  const int es = src_dtype == LMOE_F32 ? 4 : 2;
  if (!on(src, es) || !on(codes, 16) || !on(scales, 4) || !on(row_index, 4)) return LMOE_ERR_ALIGN;
  const int kb = cdiv(K, 128);
  int kb_warps = 1;
  while (kb_warps < kb && kb_warps < kThreads / 32) kb_warps *= 2;
  const RowsArgs a = {src,      ld_src, src_rows, rows, row_index, K, kb, static_cast<unsigned>(cdiv(kb, kb_warps)),
                      kb_warps, fmt_of(format, pow2_scales), codes, scales};
  const int cta_rows = 2 * (es == 2 ? kHalfRows<__nv_bfloat16> : kHalfRows<float>) * (kThreads / 32 / kb_warps);
  const long long ctas = (rows + cta_rows - 1) / cta_rows * a.chunks;
  if (ctas > 0x7fffffffLL) return LMOE_ERR_UNSUPPORTED;
  const cudaError_t e = by_source(src_dtype, on(src, 16) && ld_src * es % 16 == 0, format, [&](auto t, auto v, auto f) {
    return launch_pdl(rows_kernel<decltype(t), decltype(v)::value, decltype(f)::value>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, stream, a);
  });
  return e == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}

extern "C" lmoe_status lmoe_quantize_fp8_weight(const void* src, lmoe_dtype src_dtype, int n_experts, int N, int K,
                                                lmoe_fp8_format format, int pow2_scales, uint8_t* codes,
                                                float* scales, uint8_t* codes_t, float* scales_t,
                                                cudaStream_t stream) {
  if (n_experts < 0 || N <= 0 || K <= 0 || (format != LMOE_FP8_E4M3 && format != LMOE_FP8_E5M2)) return LMOE_ERR_ARG;
  if ((codes_t == nullptr) != (scales_t == nullptr)) return LMOE_ERR_ARG;
  if (!dtype_ok(src_dtype) || K % 16 || (codes_t != nullptr && N % 16) || K > (1 << 20) || N > (1 << 20))
    return LMOE_ERR_UNSUPPORTED;
  if (n_experts == 0) return LMOE_OK;
  if (src == nullptr || codes == nullptr || scales == nullptr) return LMOE_ERR_ARG;
  const int es = src_dtype == LMOE_F32 ? 4 : 2;
  if (!on(src, es) || !on(codes, 16) || !on(codes_t, 16) || !on(scales, 4) || !on(scales_t, 4)) return LMOE_ERR_ALIGN;
  const WeightArgs a = {src, N, K, cdiv(N, 128), cdiv(K, 128), fmt_of(format, pow2_scales), codes, codes_t, scales, scales_t};
  const long long ctas = static_cast<long long>(n_experts) * a.nb * a.kb;
  if (ctas > 0x7fffffffLL) return LMOE_ERR_UNSUPPORTED;
  const cudaError_t e = by_source(src_dtype, on(src, 4 * es), format, [&](auto t, auto v, auto f) {
    return launch_pdl(weight_kernel<decltype(t), decltype(v)::value, decltype(f)::value>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, stream, a);
  });
  return e == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}

extern "C" lmoe_status lmoe_quantize_fp8_cols(const void* src, lmoe_dtype src_dtype, long long ld_src,
                                              const int32_t* row_index, long long src_rows, long long rows, int K,
                                              const int32_t* offsets, int n_experts, long long padded_rows,
                                              lmoe_fp8_format format, int pow2_scales, uint8_t* codes_t,
                                              float* scales_t, cudaStream_t stream) {
  if (rows < 0 || src_rows < 0 || K <= 0 || ld_src < K || n_experts <= 0 ||
      (format != LMOE_FP8_E4M3 && format != LMOE_FP8_E5M2))
    return LMOE_ERR_ARG;
  if (row_index == nullptr && src_rows < rows) return LMOE_ERR_ARG;
  if ((offsets == nullptr && n_experts != 1) || padded_rows != lmoe_fp8_padded_rows(rows, n_experts)) return LMOE_ERR_ARG;
  if (!dtype_ok(src_dtype) || K % 16 || K > (1 << 20) || rows > (1LL << 24) || n_experts > kMaxGroups)
    return LMOE_ERR_UNSUPPORTED;
  if (rows == 0) return LMOE_OK;
  if ((src == nullptr && src_rows > 0) || codes_t == nullptr || scales_t == nullptr) return LMOE_ERR_ARG;
  const int es = src_dtype == LMOE_F32 ? 4 : 2;
  if (!on(src, es) || !on(codes_t, 16) || !on(scales_t, 4) || !on(row_index, 4) || !on(offsets, 4)) return LMOE_ERR_ALIGN;
  const ColsArgs a = {src,     ld_src,    src_rows, rows, padded_rows, row_index, offsets,
                      n_experts, K, cdiv(K, 128), fmt_of(format, pow2_scales), codes_t, scales_t};
  const long long units = padded_rows / 128 * a.kb;
  const int grid = static_cast<int>(std::min<long long>(units, (es == 2 ? kColsCtas<__nv_bfloat16> : kColsCtas<float>) * sm_count()));
  const cudaError_t e = by_source(src_dtype, on(src, 4 * es) && ld_src % 4 == 0, format, [&](auto t, auto v, auto f) {
    return launch_pdl(cols_kernel<decltype(t), decltype(v)::value, decltype(f)::value>, dim3(grid), dim3(kThreads), 0, stream, a);
  });
  return e == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}
