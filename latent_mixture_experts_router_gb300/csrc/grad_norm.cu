// grad_norm.cu — the norm over many gradient tensors, and the gradients scaled to a largest norm.
//
//   norm = sqrt(sum over all tensors of g^2),   out = g min(1, max_norm / (norm + 1e-6))
//
// Memory-bound: everything is read once for the norm, and read and written once for the clip.  The tensors'
// addresses and sizes travel as kernel parameters (up to kMany to a launch), so a call allocates and copies nothing
// and can be captured.  A tensor is cut into chunks of kChunk bytes; a CTA takes chunks blockIdx.x, + gridDim.x, ...
// of all tensors.  Each CTA leaves one fp64 partial sum in the workspace; they are added in index order by one
// CTA (the norm alone), or by each CTA of the clip, which saves that launch.  No atomics: the same bits every time.
//
// A thread sums its 8 x 16 bytes of a chunk in fp32 and adds that to an fp64 sum.  Squares leave fp32's range for
// elements beyond 2^+-63: a sum that is not between 2^-80 and 2^100 (and not of zeros alone) is taken again
// in fp64, from memory once more; terms that an accepted sum loses below 2^-126 are 2^-40 of it.
#include "../../include/latent_moe.h"
#include "internal.h"
#include "ptx.cuh"

#include <algorithm>
#include <utility>
#include <vector>

namespace lmoe {
namespace {

constexpr int kFew = 32, kSome = 256, kMany = 1024;   // tensors of a launch (its parameters: 1, 7 or 28 KB)
constexpr int kNormThreads = 256, kUnroll = 8;
constexpr int kVecs = kNormThreads * kUnroll;   // 16-byte vectors of a chunk
constexpr int kNormCtas = 152 * 8;          // of a launch, at most

// n: elements * 2 + (1 if fp32); first: index of the tensor's first chunk
template <int CAP>
struct GradTable {
  const void* src[CAP];
  long long n[CAP];
  int first[CAP + 1];
  int count;
};
template <int CAP>
struct ClipTable {
  GradTable<CAP> t;
  void* dst[CAP];
};

template <int CAP>
LMOE_DEV int tensor_of(const GradTable<CAP>& t, int chunk) {
  int l = 0, h = t.count;
  while (h - l > 1) {
    const int m = (l + h) >> 1;
    if (t.first[m] <= chunk) l = m;
    else h = m;
  }
  return l;
}
// elements before the first 16-byte boundary
template <typename T>
__host__ __device__ inline long long head_of(const void* p, long long n) {
  const long long h = static_cast<long long>((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T);
  return h < n ? h : n;
}
template <typename T>
__host__ __device__ inline int chunks_of(const void* p, long long n) {
  const long long v = (n - head_of<T>(p, n)) / static_cast<long long>(16 / sizeof(T));
  const long long c = (v + kVecs - 1) / kVecs;
  return static_cast<int>(c < 1 ? 1 : c);
}

LMOE_DEV void halves(uint32_t w, float& lo, float& hi) {
  lo = __uint_as_float(w << 16);
  hi = __uint_as_float(w & 0xffff0000u);
}
template <typename T>
LMOE_DEV void unpack(const uint4& q, float (&v)[16 / sizeof(T)]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(w[i]);
    else halves(w[i], v[2 * i], v[2 * i + 1]);
  }
}
LMOE_DEV float value(float v) { return v; }
LMOE_DEV float value(__nv_bfloat16 v) { return __bfloat162float(v); }

// This thread's part of the sum of squares of a chunk.
template <typename T>
LMOE_DEV double chunk_squares(const T* p, long long n, int chunk, bool last) {
  constexpr int V = 16 / sizeof(T);
  const long long head = head_of<T>(p, n), vecs = (n - head) / V;
  const uint4* body = reinterpret_cast<const uint4*>(p + head);
  const long long v0 = static_cast<long long>(chunk) * kVecs + threadIdx.x;
  uint4 q[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const long long at = v0 + i * kNormThreads;
    q[i] = at < vecs ? __ldg(body + at) : make_uint4(0, 0, 0, 0);
  }
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    float v[V];
    unpack<T>(q[i], v);
    any |= q[i].x | q[i].y | q[i].z | q[i].w;
#pragma unroll
    for (int j = 0; j < V; ++j) s[j & 3] = fmaf(v[j], v[j], s[j & 3]);
  }
  const float sum = (s[0] + s[1]) + (s[2] + s[3]);
  double d = sum;
  if (!(sum >= 0x1p-80f && sum <= 0x1p100f) && any != 0) {
    d = 0.0;
#pragma unroll 1
    for (int i = 0; i < kUnroll; ++i) {
      float v[V];
      const long long at = v0 + i * kNormThreads;
      unpack<T>(at < vecs ? __ldg(body + at) : make_uint4(0, 0, 0, 0), v);
      for (int j = 0; j < V; ++j) d += static_cast<double>(v[j]) * v[j];
    }
  }
  if (chunk == 0 && static_cast<long long>(threadIdx.x) < head) {
    const double v = value(p[threadIdx.x]);
    d += v * v;
  }
  const long long rest = head + vecs * V;
  if (last && threadIdx.x < n - rest) {
    const double v = value(p[rest + threadIdx.x]);
    d += v * v;
  }
  return d;
}

// Sum over the CTA, in thread 0; a fixed tree.
LMOE_DEV double cta_sum(double d) {
  __shared__ double part[kNormThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_down_sync(~0u, d, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = d;
  __syncthreads();
  double t = 0.0;
  if (threadIdx.x == 0)
    for (int i = 0; i < kNormThreads / 32; ++i) t += part[i];
  return t;
}

template <int CAP>
__global__ void __launch_bounds__(kNormThreads) squares_kernel(const __grid_constant__ GradTable<CAP> t, double* partial) {
  griddep_enter();
  double d = 0.0;
  for (int c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
    const int i = tensor_of(t, c), chunk = c - t.first[i];
    const bool last = c + 1 == t.first[i + 1];
    const long long n = t.n[i] >> 1;
    if (t.n[i] & 1) d += chunk_squares(static_cast<const float*>(t.src[i]), n, chunk, last);
    else d += chunk_squares(static_cast<const __nv_bfloat16*>(t.src[i]), n, chunk, last);
  }
  const double s = cta_sum(d);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// The norm from the partial sums, in thread 0.
LMOE_DEV float norm_of(const double* partial, int partials) {
  double d = 0.0;
  for (int i = threadIdx.x; i < partials; i += kNormThreads) d += partial[i];
  return static_cast<float>(sqrt(cta_sum(d)));
}
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const double* partial, int partials, float* norm) {
  griddep_enter();
  const float v = norm_of(partial, partials);
  if (threadIdx.x == 0) *norm = v;
}

template <typename T>
LMOE_DEV T scaled(T v, float f);
template <>
LMOE_DEV float scaled(float v, float f) { return v * f; }
template <>
LMOE_DEV __nv_bfloat16 scaled(__nv_bfloat16 v, float f) { return __float2bfloat16_rn(__bfloat162float(v) * f); }

template <typename T>
LMOE_DEV void clip_chunk(const T* p, T* o, long long n, int chunk, bool last, float f) {
  constexpr int V = 16 / sizeof(T);
  const long long head = head_of<T>(p, n), vecs = (n - head) / V, rest = head + vecs * V;
  const long long v0 = static_cast<long long>(chunk) * kVecs + threadIdx.x;
  const uint4* body = reinterpret_cast<const uint4*>(p + head);
  const bool along = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) == 0;
  uint4 q[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const long long at = v0 + i * kNormThreads;
    if (at < vecs) q[i] = body[at];
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const long long at = v0 + i * kNormThreads;
    if (at >= vecs) break;
    float v[V];
    unpack<T>(q[i], v);
    if (along) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) w[j] = __float_as_uint(v[j] * f);
        else w[j] = pack_bf16x2(v[2 * j] * f, v[2 * j + 1] * f);
      }
      reinterpret_cast<uint4*>(o + head)[at] = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if constexpr (sizeof(T) == 4) o[head + at * V + j] = v[j] * f;
        else o[head + at * V + j] = __float2bfloat16_rn(v[j] * f);
      }
    }
  }
  if (chunk == 0 && static_cast<long long>(threadIdx.x) < head) o[threadIdx.x] = scaled(p[threadIdx.x], f);
  if (last && threadIdx.x < n - rest) o[rest + threadIdx.x] = scaled(p[rest + threadIdx.x], f);
}

// partial != nullptr: the norm is taken from there, and stored.  Chunks in falling order: the last ones
// that the norm read are still in L2.
template <int CAP>
__global__ void __launch_bounds__(kNormThreads)
    clip_kernel(const __grid_constant__ ClipTable<CAP> c, const double* partial, int partials, float* norm, float max_norm) {
  __shared__ float s_norm;
  griddep_enter();
  float v;
  if (partial != nullptr) {
    v = norm_of(partial, partials);
    if (threadIdx.x == 0) s_norm = v;
    __syncthreads();
    v = s_norm;
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = v;
  } else {
    v = *norm;
  }
  const float r = max_norm / (v + 1e-6f), f = r >= 1.f ? 1.f : r;   // (NaN stays NaN)
  const GradTable<CAP>& t = c.t;
  const int total = t.first[t.count];
  for (int k = blockIdx.x; k < total; k += gridDim.x) {
    const int at = total - 1 - k, i = tensor_of(t, at), chunk = at - t.first[i];
    if (f == 1.f && c.dst[i] == t.src[i]) continue;   // nothing to change
    const bool last = at + 1 == t.first[i + 1];
    const long long n = t.n[i] >> 1;
    if (t.n[i] & 1) clip_chunk(static_cast<const float*>(t.src[i]), static_cast<float*>(c.dst[i]), n, chunk, last, f);
    else clip_chunk(static_cast<const __nv_bfloat16*>(t.src[i]), static_cast<__nv_bfloat16*>(c.dst[i]), n, chunk, last, f);
  }
}

// ---- host
struct Grads {
  const void* const* src;
  void* const* dst;
  const long long* sizes;
  const int* dtypes;
  int count;
};
// Fills the table with tensors from `at` on; returns where it stopped (full, or past 2^30 chunks).
template <int CAP>
int fill(GradTable<CAP>& t, void** dst, const Grads& g, int at) {
  t.count = 0;
  t.first[0] = 0;
  for (; at < g.count && t.count < CAP; ++at) {
    if (g.sizes[at] == 0) continue;
    const bool f32 = g.dtypes[at] == LMOE_F32;
    const int c = f32 ? chunks_of<float>(g.src[at], g.sizes[at]) : chunks_of<__nv_bfloat16>(g.src[at], g.sizes[at]);
    if (t.count > 0 && t.first[t.count] > (1 << 30) - c) break;
    t.src[t.count] = g.src[at];
    if (dst != nullptr) dst[t.count] = g.dst[at];
    t.n[t.count] = g.sizes[at] * 2 + (f32 ? 1 : 0);
    t.first[t.count + 1] = t.first[t.count] + c;
    ++t.count;
  }
  return at;
}
unsigned ctas_of(int chunks) { return static_cast<unsigned>(chunks < kNormCtas ? chunks : kNormCtas); }

template <int CAP>
cudaError_t launch_squares(const Grads& g, double* partial, int& partials, cudaStream_t s) {
  GradTable<CAP> t;
  for (int at = 0; at < g.count;) {
    at = fill(t, nullptr, g, at);
    if (t.count == 0) break;
    const unsigned grid = ctas_of(t.first[t.count]);
    const cudaError_t e = launch_pdl(squares_kernel<CAP>, dim3(grid), dim3(kNormThreads), 0, s, t, partial + partials);
    if (e != cudaSuccess) return e;
    partials += static_cast<int>(grid);
  }
  return cudaSuccess;
}
template <int CAP>
cudaError_t launch_clip(const Grads& g, const double* partial, int partials, float* norm, float max_norm, cudaStream_t s) {
  ClipTable<CAP> c;
  for (int at = 0; at < g.count;) {
    at = fill(c.t, c.dst, g, at);
    if (c.t.count == 0) break;
    const cudaError_t e = launch_pdl(clip_kernel<CAP>, dim3(ctas_of(c.t.first[c.t.count])), dim3(kNormThreads), 0, s, c,
                                     partial, partials, norm, max_norm);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// (the smaller the table, the shorter the launch: 200 tensors' norm and clip took the host 12.7 us with tables for 1024)
cudaError_t squares(const Grads& g, double* partial, int& partials, cudaStream_t s) {
  return g.count <= kFew    ? launch_squares<kFew>(g, partial, partials, s)
         : g.count <= kSome ? launch_squares<kSome>(g, partial, partials, s)
                            : launch_squares<kMany>(g, partial, partials, s);
}
cudaError_t clip(const Grads& g, const double* partial, int partials, float* norm, float max_norm, cudaStream_t s) {
  return g.count <= kFew    ? launch_clip<kFew>(g, partial, partials, norm, max_norm, s)
         : g.count <= kSome ? launch_clip<kSome>(g, partial, partials, norm, max_norm, s)
                            : launch_clip<kMany>(g, partial, partials, norm, max_norm, s);
}

size_t workspace_of(int count) { return static_cast<size_t>((count + kMany - 1) / kMany + 1) * kNormCtas * sizeof(double); }

lmoe_status check_grads(const Grads& g) {
  if (g.count < 0 || (g.count > 0 && (g.src == nullptr || g.sizes == nullptr || g.dtypes == nullptr))) return LMOE_ERR_ARG;
  if (g.count > (1 << 20)) return LMOE_ERR_UNSUPPORTED;
  for (int i = 0; i < g.count; ++i) {
    if (g.sizes[i] < 0 || (g.sizes[i] > 0 && g.src[i] == nullptr)) return LMOE_ERR_ARG;
    if (g.dtypes[i] != LMOE_F32 && g.dtypes[i] != LMOE_BF16) return LMOE_ERR_UNSUPPORTED;
    if (g.sizes[i] > (1LL << 40)) return LMOE_ERR_UNSUPPORTED;
  }
  for (int i = 0; i < g.count; ++i)
    if (g.sizes[i] > 0 && (reinterpret_cast<uintptr_t>(g.src[i]) & (g.dtypes[i] == LMOE_F32 ? 3 : 1))) return LMOE_ERR_ALIGN;
  return LMOE_OK;
}
// A tensor that is written may not share memory with another one that is read or written.
lmoe_status check_outputs(const Grads& g) {
  if (g.count > 0 && g.dst == nullptr) return LMOE_ERR_ARG;
  struct Range {
    uintptr_t lo, hi;
    int i;
    bool write;
  };
  std::vector<Range> r;
  try {
    r.reserve(2 * static_cast<size_t>(g.count));
  } catch (...) {
    return LMOE_ERR_ARG;
  }
  bool sorted = true;
  for (int i = 0; i < g.count; ++i) {
    if (g.sizes[i] == 0) continue;
    if (g.dst[i] == nullptr) return LMOE_ERR_ARG;
    const size_t es = g.dtypes[i] == LMOE_F32 ? 4 : 2;
    const uintptr_t d = reinterpret_cast<uintptr_t>(g.dst[i]), p = reinterpret_cast<uintptr_t>(g.src[i]);
    if (d & (es - 1)) return LMOE_ERR_ALIGN;
    sorted = sorted && (r.empty() || r.back().lo <= d);
    r.push_back({d, d + g.sizes[i] * es, i, true});
    if (p != d) {
      sorted = sorted && r.back().lo <= p;
      r.push_back({p, p + g.sizes[i] * es, i, false});
    }
  }
  if (!sorted) std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  // the furthest end so far of what is read, and of what is written
  uintptr_t read = 0, written = 0;
  for (const Range& x : r) {
    if (x.lo < written || (x.write && x.lo < read)) return LMOE_ERR_ARG;
    (x.write ? written : read) = std::max(x.write ? written : read, x.hi);
  }
  return LMOE_OK;
}

// The norm and the workspace (bytes: 0, none) may share memory with each other or with a tensor no more than tensors may: CTAs write
// them while others read or write those.  (A norm that is only read, lmoe_grad_clip's, may lie in a tensor that is.)
lmoe_status check_own(const Grads& g, const float* norm, const void* workspace, size_t bytes) {
  const auto meet = [](const void* a, size_t n, const void* b, size_t m) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + m && y < x + n;
  };
  if (meet(norm, 4, workspace, bytes)) return LMOE_ERR_ARG;
  for (int i = 0; i < g.count; ++i) {
    const size_t n = static_cast<size_t>(g.sizes[i]) * (g.dtypes[i] == LMOE_F32 ? 4 : 2);
    if (n == 0) continue;
    if (bytes != 0 && (meet(g.src[i], n, norm, 4) || meet(g.src[i], n, workspace, bytes))) return LMOE_ERR_ARG;
    if (g.dst != nullptr && (meet(g.dst[i], n, norm, 4) || meet(g.dst[i], n, workspace, bytes))) return LMOE_ERR_ARG;
  }
  return LMOE_OK;
}

}  // namespace
}  // namespace lmoe

using namespace lmoe;

extern "C" lmoe_status lmoe_grad_norm_workspace_size(int count, size_t* bytes) {
  if (count < 0 || bytes == nullptr) return LMOE_ERR_ARG;
  if (count > (1 << 20)) return LMOE_ERR_UNSUPPORTED;
  *bytes = workspace_of(count);
  return LMOE_OK;
}

static lmoe_status check_norm(const Grads& g, const float* norm, const void* workspace, size_t workspace_bytes) {
  const lmoe_status st = check_grads(g);
  if (st != LMOE_OK) return st;
  if (norm == nullptr) return LMOE_ERR_ARG;
  if (workspace == nullptr || workspace_bytes < workspace_of(g.count)) return LMOE_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 7) || (reinterpret_cast<uintptr_t>(norm) & 3)) return LMOE_ERR_ALIGN;
  return LMOE_OK;
}

extern "C" lmoe_status lmoe_grad_norm(const void* const* grads, const long long* sizes, const int* dtypes, int count,
                                      float* norm, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const Grads g = {grads, nullptr, sizes, dtypes, count};
  lmoe_status st = check_norm(g, norm, workspace, workspace_bytes);
  if (st == LMOE_OK) st = check_own(g, norm, workspace, workspace_of(count));
  if (st != LMOE_OK) return st;
  double* partial = static_cast<double*>(workspace);
  int partials = 0;
  cudaError_t e = squares(g, partial, partials, stream);
  if (e == cudaSuccess) e = launch_pdl(norm_kernel, dim3(1), dim3(kNormThreads), 0, stream, partial, partials, norm);
  return e == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}

extern "C" lmoe_status lmoe_grad_clip(const void* const* grads, void* const* out, const long long* sizes,
                                      const int* dtypes, int count, const float* norm, float max_norm,
                                      cudaStream_t stream) {
  const Grads g = {grads, out, sizes, dtypes, count};
  lmoe_status st = check_grads(g);
  if (st != LMOE_OK) return st;
  if (norm == nullptr || !(max_norm >= 0.f)) return LMOE_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(norm) & 3) return LMOE_ERR_ALIGN;
  st = check_outputs(g);
  if (st == LMOE_OK) st = check_own(g, norm, nullptr, 0);
  if (st != LMOE_OK) return st;
  float* nm = const_cast<float*>(norm);
  const cudaError_t e = clip(g, nullptr, 0, nm, max_norm, stream);
  return e == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}

extern "C" lmoe_status lmoe_clip_grad_norm(const void* const* grads, void* const* out, const long long* sizes,
                                           const int* dtypes, int count, float* norm, float max_norm, void* workspace,
                                           size_t workspace_bytes, cudaStream_t stream) {
  const Grads g = {grads, out, sizes, dtypes, count};
  lmoe_status st = check_norm(g, norm, workspace, workspace_bytes);
  if (st != LMOE_OK) return st;
  if (!(max_norm >= 0.f)) return LMOE_ERR_ARG;
  st = check_outputs(g);
  if (st == LMOE_OK) st = check_own(g, norm, workspace, workspace_of(count));
  if (st != LMOE_OK) return st;
  double* partial = static_cast<double*>(workspace);
  int partials = 0;
  cudaError_t e = squares(g, partial, partials, stream);
  if (e != cudaSuccess) return LMOE_ERR_CUDA;
  if (partials == 0)   // no tensors: the norm is 0
    e = launch_pdl(norm_kernel, dim3(1), dim3(kNormThreads), 0, stream, partial, 0, norm);
  else
    e = clip(g, partial, partials, norm, max_norm, stream);
  return e == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}
