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
// All three read and write each element once; the memory traffic bounds them.
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
  int e5m2, pow2;
};
// two codes, a's in the low byte
LMOE_DEV uint32_t cvt2(float a, float b, int e5m2) {
  uint16_t r;
  if (e5m2) asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  else asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
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
LMOE_DEV uint32_t mag(float v) { return __float_as_uint(v) & 0x7fffffffu; }
LMOE_DEV float lo16(uint32_t w) { return __uint_as_float(w << 16); }
LMOE_DEV float hi16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// N consecutive elements as fp32
template <bool VEC, int N>
LMOE_DEV void load_n(const float* p, float (&v)[N]) {
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < N / 4; ++j) {
      const float4 q = reinterpret_cast<const float4*>(p)[j];
      v[4 * j] = q.x, v[4 * j + 1] = q.y, v[4 * j + 2] = q.z, v[4 * j + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = p[j];
  }
}
template <bool VEC, int N>
LMOE_DEV void load_n(const __nv_bfloat16* p, float (&v)[N]) {
  if constexpr (VEC && N == 8) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    v[0] = lo16(q.x), v[1] = hi16(q.x), v[2] = lo16(q.y), v[3] = hi16(q.y);
    v[4] = lo16(q.z), v[5] = hi16(q.z), v[6] = lo16(q.w), v[7] = hi16(q.w);
  } else if constexpr (VEC) {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    v[0] = lo16(q.x), v[1] = hi16(q.x), v[2] = lo16(q.y), v[3] = hi16(q.y);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = __bfloat162float(p[j]);
  }
}

// ------------------------------------------------------------------ rows
// A warp takes 8 rows of one block of columns: half a warp reads a row's 128 elements (8 per
// lane), four rows each in flight at once, and the eight scales are one 32-byte sector of
// scales[kb].  Warps beside each other take the next blocks of the same rows.
struct RowsArgs {
  const void* src;
  long long ld, src_rows, rows;
  const int32_t* index;
  int K, kb;
  Fmt f;
  uint8_t* codes;
  float* scales;
};
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) rows_kernel(const RowsArgs a) {
  griddep_enter();
  const int lane = threadIdx.x & 31, half = lane >> 4, l16 = lane & 15;
  const long long unit = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const long long r0 = unit / a.kb * 8;
  const int kb = static_cast<int>(unit % a.kb);
  if (r0 >= a.rows) return;
  const int c = kb * 128 + l16 * 8;
  const bool in_k = c < a.K;   // K is a multiple of 16
  float v[4][8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const long long r = r0 + 2 * j + half;
    long long q = r;
    bool ok = in_k && r < a.rows;
    if (ok && a.index != nullptr) {
      q = a.index[r];
      ok = q >= 0 && q < a.src_rows;
    }
    if (ok) {
      load_n<VEC>(static_cast<const T*>(a.src) + q * a.ld + c, v[j]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = 0.f;
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const long long r = r0 + 2 * j + half;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, mag(v[j][i]));
#pragma unroll
    for (int d = 8; d; d >>= 1) m = max(m, __shfl_xor_sync(~0u, m, d));
    const float s = scale_of(m, a.f), inv = __frcp_rn(s);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = cvt2(v[j][2 * i] * inv, v[j][2 * i + 1] * inv, a.f.e5m2);
    if (r < a.rows) {
      if (in_k) *reinterpret_cast<uint2*>(a.codes + r * a.K + c) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
      if (l16 == 0) a.scales[static_cast<long long>(kb) * a.rows + r] = s;
    }
  }
}

// ------------------------------------------------------------------ 128 x 128 tiles
// Warp w holds rows 16 w .. 16 w + 15 of a tile, lane l columns 4 l .. 4 l + 3: a row's loads and
// stores are whole lines, and a thread's 16 rows of one column are 16 bytes of the transpose.
// Those pass through shared memory, chunk w of column c at place w ^ ((c / 4) % 8), which keeps
// both the writes (32 columns apart by 128 bytes) and the reads free of bank conflicts.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  float4 q;
  LMOE_DEV void zero() { q = make_float4(0.f, 0.f, 0.f, 0.f); }
  template <bool VEC>
  LMOE_DEV void load(const float* p) {
    if constexpr (VEC) q = *reinterpret_cast<const float4*>(p);
    else q = make_float4(p[0], p[1], p[2], p[3]);
  }
  LMOE_DEV float get(int i) const { return i == 0 ? q.x : i == 1 ? q.y : i == 2 ? q.z : q.w; }
};
template <>
struct Raw<__nv_bfloat16> {
  uint2 q;
  LMOE_DEV void zero() { q = make_uint2(0u, 0u); }
  template <bool VEC>
  LMOE_DEV void load(const __nv_bfloat16* p) {
    if constexpr (VEC) {
      q = *reinterpret_cast<const uint2*>(p);
    } else {
      const unsigned short* u = reinterpret_cast<const unsigned short*>(p);
      q = make_uint2(u[0] | (static_cast<uint32_t>(u[1]) << 16), u[2] | (static_cast<uint32_t>(u[3]) << 16));
    }
  }
  LMOE_DEV float get(int i) const { return i == 0 ? lo16(q.x) : i == 1 ? hi16(q.x) : i == 2 ? lo16(q.y) : hi16(q.y); }
};

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
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) weight_kernel(const WeightArgs a) {
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
  Raw<T> v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (n0 + i < a.N && k0 < a.K) v[i].template load<VEC>(src + static_cast<long long>(i) * a.K);
    else v[i].zero();
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max(m, mag(v[i].get(j)));
  m = __reduce_max_sync(~0u, m);
  if (lane == 0) wmax[warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) m = max(m, wmax[w]);
  const float s = scale_of(m, a.f), inv = __frcp_rn(s);
  if (threadIdx.x == 0) {
    a.scales[(g * a.nb + nb) * a.kb + kb] = s;
    if (a.scales_t != nullptr) a.scales_t[(g * a.kb + kb) * a.nb + nb] = s;
  }
  uint32_t tr[4][4];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t w01 = cvt2(v[i].get(0) * inv, v[i].get(1) * inv, a.f.e5m2);
    const uint32_t w23 = cvt2(v[i].get(2) * inv, v[i].get(3) * inv, a.f.e5m2);
    if (n0 + i < a.N && k0 < a.K)
      *reinterpret_cast<uint32_t*>(a.codes + (g * a.N + n0 + i) * a.K + k0) = w01 | (w23 << 16);
    const uint32_t b[4] = {w01 & 0xffu, w01 >> 8, w23 & 0xffu, w23 >> 8};
#pragma unroll
    for (int j = 0; j < 4; ++j) tr[j][i >> 2] = (i & 3) == 0 ? b[j] : tr[j][i >> 2] | (b[j] << (8 * (i & 3)));
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
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) cols_kernel(const ColsArgs a) {
  __shared__ __align__(16) uint8_t tile[128 * 128];
  __shared__ __align__(16) uint32_t cmax[kThreads / 32][128];
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
    long long mine = -1;   // lane i < 16: source row of row r0 + i
    if (lane < 16 && r0 + lane < rend) {
      mine = a.index != nullptr ? a.index[r0 + lane] : r0 + lane;
      if (mine < 0 || mine >= a.src_rows) mine = -1;
    }
    Raw<T> v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const long long q = __shfl_sync(~0u, mine, i);
      if (q >= 0 && k0 < a.K) v[i].template load<VEC>(static_cast<const T*>(a.src) + q * a.ld + k0);
      else v[i].zero();
    }
    uint4 m = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      m.x = max(m.x, mag(v[i].get(0)));
      m.y = max(m.y, mag(v[i].get(1)));
      m.z = max(m.z, mag(v[i].get(2)));
      m.w = max(m.w, mag(v[i].get(3)));
    }
    *reinterpret_cast<uint4*>(&cmax[warp][lane * 4]) = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const uint4 o = *reinterpret_cast<const uint4*>(&cmax[w][lane * 4]);
      m = make_uint4(max(m.x, o.x), max(m.y, o.y), max(m.z, o.z), max(m.w, o.w));
    }
    const uint32_t mm[4] = {m.x, m.y, m.z, m.w};
    float inv[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float s = scale_of(mm[j], a.f);
      inv[j] = __frcp_rn(s);
      if (warp == 0 && k0 + j < a.K) a.scales[static_cast<long long>(blk) * a.K + k0 + j] = s;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        w[q] = cvt2(v[4 * q].get(j) * inv[j], v[4 * q + 1].get(j) * inv[j], a.f.e5m2) |
               (cvt2(v[4 * q + 2].get(j) * inv[j], v[4 * q + 3].get(j) * inv[j], a.f.e5m2) << 16);
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
Fmt fmt_of(lmoe_fp8_format f, int pow2) { return Fmt{f == LMOE_FP8_E5M2 ? 57344.f : 448.f, f == LMOE_FP8_E5M2, pow2 != 0}; }

// f(T, VEC) for the source's type and alignment
template <typename F>
cudaError_t by_source(lmoe_dtype d, bool vec, F f) {
  if (d == LMOE_F32) return vec ? f(float{}, std::true_type{}) : f(float{}, std::false_type{});
  return vec ? f(__nv_bfloat16{}, std::true_type{}) : f(__nv_bfloat16{}, std::false_type{});
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
  const RowsArgs a = {src, ld_src, src_rows, rows, row_index, K, kb, fmt_of(format, pow2_scales), codes, scales};
  const long long ctas = ((rows + 7) / 8 * kb + kThreads / 32 - 1) / (kThreads / 32);
  if (ctas > 0x7fffffffLL) return LMOE_ERR_UNSUPPORTED;
  const cudaError_t e = by_source(src_dtype, on(src, 16) && ld_src * es % 16 == 0, [&](auto t, auto v) {
    return launch_pdl(rows_kernel<decltype(t), decltype(v)::value>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, stream, a);
  });
  return e == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}

extern "C" lmoe_status lmoe_quantize_fp8_weight(const void* src, lmoe_dtype src_dtype, int n_experts, int N, int K,
                                                lmoe_fp8_format format, int pow2_scales, uint8_t* codes,
                                                float* scales, uint8_t* codes_t, float* scales_t,
                                                cudaStream_t stream) {
  if (n_experts < 0 || N <= 0 || K <= 0 || (format != LMOE_FP8_E4M3 && format != LMOE_FP8_E5M2)) return LMOE_ERR_ARG;
  if ((codes_t == nullptr) != (scales_t == nullptr)) return LMOE_ERR_ARG;
  if (!dtype_ok(src_dtype) || K % 16 || (codes_t != nullptr && N % 16) || K > (1 << 20) || N > (1 << 20) ||
      n_experts > kMaxGroups)
    return LMOE_ERR_UNSUPPORTED;
  if (n_experts == 0) return LMOE_OK;
  if (src == nullptr || codes == nullptr || scales == nullptr) return LMOE_ERR_ARG;
  const int es = src_dtype == LMOE_F32 ? 4 : 2;
  if (!on(src, es) || !on(codes, 16) || !on(codes_t, 16) || !on(scales, 4) || !on(scales_t, 4)) return LMOE_ERR_ALIGN;
  const WeightArgs a = {src, N, K, cdiv(N, 128), cdiv(K, 128), fmt_of(format, pow2_scales), codes, codes_t, scales, scales_t};
  const long long ctas = static_cast<long long>(n_experts) * a.nb * a.kb;
  if (ctas > 0x7fffffffLL) return LMOE_ERR_UNSUPPORTED;
  const cudaError_t e = by_source(src_dtype, on(src, 4 * es), [&](auto t, auto v) {
    return launch_pdl(weight_kernel<decltype(t), decltype(v)::value>, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, stream, a);
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
  const int grid = static_cast<int>(std::min<long long>(units, 2LL * sm_count()));
  const cudaError_t e = by_source(src_dtype, on(src, 4 * es) && ld_src % 4 == 0, [&](auto t, auto v) {
    return launch_pdl(cols_kernel<decltype(t), decltype(v)::value>, dim3(grid), dim3(kThreads), 0, stream, a);
  });
  return e == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}
