// router_train.cu — what trains the router: its balance loss and z loss with the per-expert
// counts, and the gradient of its logits.
//
// Row t holds E logits l (plus the router bias), p = softmax(l), lse = log sum exp(l).  A row is
// live when the mask keeps it and at least one of its logits is above -inf; n live rows, f_e =
// counts_e / (k n) with counts_e the slots of live rows that name expert e, P_e = mean of p_e:
//   balance = E sum_e f_e P_e,   z = mean lse^2
//   dlogits_e = p_e (gb E / n (f_e - sum_j f_j p_j) + gz 2 / n lse)
//             + sum over the row's slots j of expert e: w_j (gw_j - sum_i w_i gw_i),
//   w = softmax of the row's selected logits over its slots (the routing weights).
// (f is a count: no gradient flows through it.)
//
// Both read each logit once; the memory traffic bounds them.  A warp takes a row at a time, V
// values per lane in registers, and loads its next row before it works on the present one.  exp
// is one FMA and ex2: exp2(l log2e - m log2e), exact in m's part (it cancels in p).
#include <algorithm>

#include "../../include/latent_moe.h"
#include "internal.h"
#include "ptx.cuh"

namespace lmoe {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr float kLog2e = 1.4426950408889634f;

LMOE_DEV float to_f32(float v) { return v; }
LMOE_DEV float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
LMOE_DEV void store_as(float* p, float v) { *p = v; }
LMOE_DEV void store_as(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
// larger of two, NaN if either is
LMOE_DEV float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
LMOE_DEV float warp_max_nan(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = max_nan(v, __shfl_xor_sync(~0u, v, d));
  return v;
}
LMOE_DEV float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
  return v;
}

// Value i of a lane is element col<VEC>(lane, i) of the row: four neighbours at a time where the
// rows allow 4-element loads, else every 32nd.
template <bool VEC>
LMOE_DEV int col(int lane, int i) {
  return VEC ? (i >> 2) * 128 + lane * 4 + (i & 3) : lane + 32 * i;
}

template <typename T, int V, bool VEC>
LMOE_DEV void load_row(const T* row, int E, int lane, float (&v)[V]) {
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < V / 4; ++j) {
      const int e = col<true>(lane, 4 * j);
      if (e < E) {
        if constexpr (sizeof(T) == 4) {
          const float4 q = *reinterpret_cast<const float4*>(row + e);
          v[4 * j] = q.x, v[4 * j + 1] = q.y, v[4 * j + 2] = q.z, v[4 * j + 3] = q.w;
        } else {
          const uint2 q = *reinterpret_cast<const uint2*>(row + e);
          v[4 * j] = __uint_as_float(q.x << 16), v[4 * j + 1] = __uint_as_float(q.x & 0xffff0000u);
          v[4 * j + 2] = __uint_as_float(q.y << 16), v[4 * j + 3] = __uint_as_float(q.y & 0xffff0000u);
        }
      } else {
        v[4 * j] = v[4 * j + 1] = v[4 * j + 2] = v[4 * j + 3] = -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = col<false>(lane, i);
      v[i] = e < E ? to_f32(row[e]) : -INFINITY;
    }
  }
}
template <int V, bool VEC>
LMOE_DEV void add_bias(const float* bias, int E, int lane, float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = col<VEC>(lane, i);
    if (e < E) v[i] += bias[e];
  }
}
// v becomes exp(l - max); returns their sum over the row.  m: the row's maximum.
template <int V>
LMOE_DEV float exp_row(float (&v)[V], float m) {
  const float c = m * kLog2e;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    v[i] = exp2f(fmaf(v[i], kLog2e, -c));
    s += v[i];
  }
  return warp_sum(s);
}
template <int V>
LMOE_DEV float row_max(const float (&v)[V]) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < V; ++i) m = max_nan(m, v[i]);
  return warp_max_nan(m);
}

struct LossArgs {
  const void* logits;
  long long ld;
  const float* bias;
  const uint8_t* mask;
  const int32_t* idx;
  int T, E, k;
  int32_t* counts;      // [E + 1], the last the live rows
  float* mean;          // [E]
  float* losses;        // [2]
  float* part_p;        // [grid][E]
  int32_t* part_c;      // [grid][E]
  float* part_z;        // [grid]
  int32_t* part_n;      // [grid]
  int grid;
};

// Sum over a CTA of kThreads, in warp order.
LMOE_DEV double block_sum(double v, double* sm) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0;
  for (int w = 0; w < kWarps; ++w) s += sm[w];
  return s;
}

// The results from the column sums of p and the counts: expert e = threadIdx.x, + kThreads, ..
// through `at(e, p, c)`.
template <typename F>
LMOE_DEV void finish(const LossArgs& a, int n, double zsum, F at, double* sm) {
  const double inv = n > 0 ? 1.0 / n : 0.0;
  double dot = 0;
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    double p;
    int c;
    at(e, p, c);
    a.mean[e] = static_cast<float>(p * inv);
    a.counts[e] = c;
    dot += p * c;
  }
  dot = block_sum(dot, sm);
  if (threadIdx.x == 0) {
    a.counts[a.E] = n;
    a.losses[0] = static_cast<float>(dot * inv * inv * a.E / a.k);
    a.losses[1] = static_cast<float>(zsum * inv);
  }
}

template <typename T, int V, bool VEC>
__global__ void __launch_bounds__(kThreads) losses_kernel(const LossArgs a) {
  extern __shared__ float sm_p[];   // [kWarps][E], then int hist[E]
  int* hist = reinterpret_cast<int*>(sm_p + kWarps * a.E);
  __shared__ float sm_z[kWarps];
  __shared__ int sm_n[kWarps];
  __shared__ double sm_d[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < a.E; e += kThreads) hist[e] = 0;
  griddep_enter();
  __syncthreads();
  const T* logits = static_cast<const T*>(a.logits);
  const int step = gridDim.x * kWarps;
  float acc[V], next[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  float z = 0.f;
  int n = 0;
  int t = blockIdx.x * kWarps + warp;
  bool live = t < a.T && (a.mask == nullptr || a.mask[t] != 0);
  int id = -1;
  if (live) {
    load_row<T, V, VEC>(logits + t * a.ld, a.E, lane, next);
    if (lane < a.k) id = a.idx[static_cast<long long>(t) * a.k + lane];
  }
  while (t < a.T) {
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = next[i];
    const bool here = live;
    const int slot = id;
    t += step;
    live = t < a.T && (a.mask == nullptr || a.mask[t] != 0);
    if (live) {
      load_row<T, V, VEC>(logits + t * a.ld, a.E, lane, next);
      if (lane < a.k) id = a.idx[static_cast<long long>(t) * a.k + lane];
    }
    if (!here) continue;
    if (a.bias != nullptr) add_bias<V, VEC>(a.bias, a.E, lane, v);
    const float m = row_max(v);
    if (m == -INFINITY) continue;
    const float s = exp_row(v, m);
    const float r = 1.f / s;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = fmaf(v[i], r, acc[i]);
    const float lse = m + logf(s);
    z = fmaf(lse, lse, z);
    ++n;
    if (lane < a.k && slot >= 0 && slot < a.E) atomicAdd(&hist[slot], 1);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = col<VEC>(lane, i);
    if (e < a.E) sm_p[warp * a.E + e] = acc[i];
  }
  if (lane == 0) {
    sm_z[warp] = z;
    sm_n[warp] = n;
  }
  __syncthreads();
  int nb = 0;
  float zb = 0.f;
  for (int w = 0; w < kWarps; ++w) {
    nb += sm_n[w];
    zb += sm_z[w];
  }
  const auto column = [&](int e) {
    float p = 0.f;
    for (int w = 0; w < kWarps; ++w) p += sm_p[w * a.E + e];
    return p;
  };
  if (a.grid == 1) {
    finish(a, nb, zb, [&](int e, double& p, int& c) { p = column(e), c = hist[e]; }, sm_d);
    return;
  }
  const long long o = static_cast<long long>(blockIdx.x) * a.E;
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    a.part_p[o + e] = column(e);
    a.part_c[o + e] = hist[e];
  }
  if (threadIdx.x == 0) {
    a.part_z[blockIdx.x] = zb;
    a.part_n[blockIdx.x] = nb;
  }
}

// Sums the CTAs' partials in order.  Each of kThreads / W groups of W threads takes every
// (kThreads / W)-th CTA, W the experts rounded up to a power of two.
__global__ void __launch_bounds__(kThreads) losses_finish_kernel(const LossArgs a) {
  __shared__ double sm_p[kThreads];
  __shared__ int sm_c[kThreads];
  __shared__ double sm_d[kWarps];
  griddep_enter();
  int n = 0;
  double z = 0;
  for (int g = threadIdx.x; g < a.grid; g += kThreads) {
    n += a.part_n[g];
    z += a.part_z[g];
  }
  const int nb = static_cast<int>(block_sum(n, sm_d));
  z = block_sum(z, sm_d);
  int W = 32;
  while (W < a.E && W < kThreads) W *= 2;
  const int groups = kThreads / W, grp = threadIdx.x / W, e0 = threadIdx.x % W;
  if (groups == 1) {
    finish(a, nb, z,
           [&](int e, double& p, int& c) {
             p = 0, c = 0;
#pragma unroll 8
             for (int g = 0; g < a.grid; ++g) {
               p += a.part_p[static_cast<long long>(g) * a.E + e];
               c += a.part_c[static_cast<long long>(g) * a.E + e];
             }
           },
           sm_d);
    return;
  }
  double p = 0;
  int c = 0;
  if (e0 < a.E) {
#pragma unroll 8
    for (int g = grp; g < a.grid; g += groups) {
      p += a.part_p[static_cast<long long>(g) * a.E + e0];
      c += a.part_c[static_cast<long long>(g) * a.E + e0];
    }
  }
  sm_p[threadIdx.x] = p;
  sm_c[threadIdx.x] = c;
  __syncthreads();
  finish(a, nb, z,
         [&](int e, double& pp, int& cc) {
           pp = 0, cc = 0;
           for (int g = 0; g < groups; ++g) {
             pp += sm_p[g * W + e];
             cc += sm_c[g * W + e];
           }
         },
         sm_d);
}

struct GradArgs {
  const void* logits;
  long long ld;
  const float* bias;
  const uint8_t* mask;
  const int32_t* idx;
  const float* gw;          // [T, k] or nullptr
  const int32_t* counts;    // [E + 1] } or both nullptr
  const float* gl;          // [2]     }
  int T, E, k;
  void* out;
  long long ldo;
};

template <typename T, int V, bool VEC>
__global__ void __launch_bounds__(kThreads) grad_kernel(const GradArgs a) {
  extern __shared__ float sm_row[];   // [kWarps][E]: one row while its slots' terms are added
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* row = sm_row + warp * a.E;
  griddep_enter();
  const T* logits = static_cast<const T*>(a.logits);
  T* out = static_cast<T*>(a.out);
  const int step = gridDim.x * kWarps;
  float f[V], next[V], cb = 0.f, cz = 0.f;
  if (a.gl != nullptr) {
    const int n = max(a.counts[a.E], 1);
    const float inv = 1.f / n;
    cb = a.gl[0] * a.E * inv;
    cz = a.gl[1] * 2.f * inv;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = col<VEC>(lane, i);
      f[i] = e < a.E ? a.counts[e] * inv / a.k : 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = 0.f;
  }
  int t = blockIdx.x * kWarps + warp;
  bool live = t < a.T && (a.mask == nullptr || a.mask[t] != 0);
  if (live) load_row<T, V, VEC>(logits + t * a.ld, a.E, lane, next);
  while (t < a.T) {
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = next[i];
    const int here = t;
    bool on = live;
    // the row's slots: their logits are read before the row is written (it may be written in place)
    int id = -1;
    float sel = -INFINITY, gw = 0.f;
    if (on && a.gw != nullptr && lane < a.k) {
      id = a.idx[static_cast<long long>(here) * a.k + lane];
      if (id >= 0 && id < a.E) {
        sel = to_f32(logits[here * a.ld + id]) + (a.bias != nullptr ? a.bias[id] : 0.f);
        gw = a.gw[static_cast<long long>(here) * a.k + lane];
      } else {
        id = -1;
      }
    }
    t += step;
    live = t < a.T && (a.mask == nullptr || a.mask[t] != 0);
    if (live) load_row<T, V, VEC>(logits + t * a.ld, a.E, lane, next);
    float m = -INFINITY;
    if (on) {
      if (a.bias != nullptr) add_bias<V, VEC>(a.bias, a.E, lane, v);
      m = row_max(v);
      on = m != -INFINITY;
    }
    if (on) {
      const float s = exp_row(v, m), r = 1.f / s;
      const float lz = cz * (m + logf(s));
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[i] *= r;
        dot = fmaf(v[i], f[i], dot);
      }
      dot = warp_sum(dot);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] *= fmaf(cb, f[i] - dot, lz);
      if (a.gw != nullptr) {
        const float sm = warp_max_nan(sel);
        // (no slot with a finite logit: the weights are undefined and give no gradient)
        float w = sm == -INFINITY ? 0.f : exp2f((sel - sm) * kLog2e);
        const float ws = warp_sum(w);
        w = ws == 0.f ? 0.f : w / ws;
        const float g = warp_sum(w == 0.f ? 0.f : w * gw);
        float d = w == 0.f ? 0.f : w * (gw - g);
        // an expert named by several slots of the row: its first slot adds them all, in order
        const unsigned same = __match_any_sync(~0u, id);
        const bool first = id >= 0 && lane == __ffs(same) - 1;
        if (__any_sync(~0u, id >= 0 && __popc(same) > 1)) {
          float tot = 0.f;
          for (int j = 0; j < a.k; ++j) {
            const float dj = __shfl_sync(~0u, d, j);
            if ((same >> j) & 1u) tot += dj;
          }
          d = tot;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e = col<VEC>(lane, i);
          if (e < a.E) row[e] = v[i];
        }
        __syncwarp();
        if (first) row[id] += d;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e = col<VEC>(lane, i);
          if (e < a.E) v[i] = row[e];
        }
        __syncwarp();
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = 0.f;
    }
    T* o = out + here * a.ldo;
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < V / 4; ++j) {
        const int e = col<true>(lane, 4 * j);
        if (e < a.E) {
          if constexpr (sizeof(T) == 4)
            *reinterpret_cast<float4*>(o + e) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          else
            *reinterpret_cast<uint2*>(o + e) =
                make_uint2(pack_bf16x2(v[4 * j], v[4 * j + 1]), pack_bf16x2(v[4 * j + 2], v[4 * j + 3]));
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = col<false>(lane, i);
        if (e < a.E) store_as(o + e, v[i]);
      }
    }
  }
}

// Calls f with (T, V, VEC) of the smallest V that holds E.
template <typename F>
cudaError_t by_shape(bool f32, int E, bool vec, F f) {
  const auto with_v = [&](auto v) {
    if (f32) return vec ? f(float{}, v, std::true_type{}) : f(float{}, v, std::false_type{});
    return vec ? f(__nv_bfloat16{}, v, std::true_type{}) : f(__nv_bfloat16{}, v, std::false_type{});
  };
  if (E <= 128) return with_v(std::integral_constant<int, 4>{});
  if (E <= 256) return with_v(std::integral_constant<int, 8>{});
  if (E <= 512) return with_v(std::integral_constant<int, 16>{});
  return with_v(std::integral_constant<int, 32>{});
}

// rows of 4-element loads: base, row length and the count of elements allow them
bool rows_vec(const void* p, long long ld, int E, int es) {
  return E % 4 == 0 && ld % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (4 * es) == 0;
}
constexpr int kMaxGrid = 152;   // CTAs of the losses kernel: the partials a workspace holds
int losses_grid(int T) { return std::max(1, std::min(kMaxGrid, (T + 4 * kWarps - 1) / (4 * kWarps))); }

lmoe_status check_rows(const void* logits, lmoe_dtype dt, long long ld, const float* bias, const int32_t* idx, int T,
                       int E, int k) {
  if (T < 0 || T > (1 << 20) || E < 1 || k < 1 || k > 16 || k > E || ld < E) return LMOE_ERR_ARG;
  if (E > 1024 || (dt != LMOE_F32 && dt != LMOE_BF16)) return LMOE_ERR_UNSUPPORTED;
  if (T > 0 && logits == nullptr) return LMOE_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(logits) % (dt == LMOE_F32 ? 4 : 2) || reinterpret_cast<uintptr_t>(bias) % 4 ||
      reinterpret_cast<uintptr_t>(idx) % 4)
    return LMOE_ERR_ALIGN;
  return LMOE_OK;
}

}  // namespace
}  // namespace lmoe

using namespace lmoe;

extern "C" lmoe_status lmoe_router_losses_workspace_size(int T, int E, size_t* bytes) {
  if (bytes == nullptr || T < 0 || T > (1 << 20) || E < 1) return LMOE_ERR_ARG;
  if (E > 1024) return LMOE_ERR_UNSUPPORTED;
  *bytes = static_cast<size_t>(losses_grid(T)) * (2 * E + 2) * 4;
  return LMOE_OK;
}

extern "C" lmoe_status lmoe_router_losses(const void* logits, lmoe_dtype logits_dtype, long long ld_logits,
                                          const float* router_bias, const uint8_t* row_mask, const int32_t* topk_idx,
                                          int T, int E, int k, int32_t* counts, float* mean_probs, float* losses,
                                          void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const lmoe_status st = check_rows(logits, logits_dtype, ld_logits, router_bias, topk_idx, T, E, k);
  if (st != LMOE_OK) return st;
  if (counts == nullptr || mean_probs == nullptr || losses == nullptr || (T > 0 && topk_idx == nullptr))
    return LMOE_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(counts) % 4 || reinterpret_cast<uintptr_t>(mean_probs) % 4 ||
      reinterpret_cast<uintptr_t>(losses) % 4 || reinterpret_cast<uintptr_t>(workspace) % 4)
    return LMOE_ERR_ALIGN;
  LossArgs a = {logits, ld_logits, router_bias, row_mask, topk_idx, T, E, k, counts, mean_probs, losses};
  a.grid = losses_grid(T);
  const size_t need = static_cast<size_t>(a.grid) * (2 * E + 2) * 4;
  if (workspace == nullptr || workspace_bytes < need) return LMOE_ERR_WORKSPACE;
  a.part_p = static_cast<float*>(workspace);
  a.part_c = reinterpret_cast<int32_t*>(a.part_p + static_cast<size_t>(a.grid) * E);
  a.part_z = reinterpret_cast<float*>(a.part_c + static_cast<size_t>(a.grid) * E);
  a.part_n = reinterpret_cast<int32_t*>(a.part_z + a.grid);
  const size_t smem = static_cast<size_t>(kWarps + 1) * E * 4;
  const bool f32 = logits_dtype == LMOE_F32;
  cudaError_t e = by_shape(f32, E, rows_vec(logits, ld_logits, E, f32 ? 4 : 2), [&](auto t, auto v, auto vec) {
    auto kern = losses_kernel<decltype(t), decltype(v)::value, decltype(vec)::value>;
    const cudaError_t r = allow_smem(reinterpret_cast<const void*>(kern), static_cast<int>(smem));
    return r != cudaSuccess ? r : launch_pdl(kern, dim3(a.grid), dim3(kThreads), smem, stream, a);
  });
  if (e == cudaSuccess && a.grid > 1) e = launch_pdl(losses_finish_kernel, dim3(1), dim3(kThreads), 0, stream, a);
  return e == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}

extern "C" lmoe_status lmoe_router_grad(const void* logits, lmoe_dtype logits_dtype, long long ld_logits,
                                        const float* router_bias, const uint8_t* row_mask, const int32_t* topk_idx,
                                        const float* topk_w_grad, const int32_t* counts, const float* loss_grads,
                                        int T, int E, int k, void* dlogits, long long ld_dlogits,
                                        cudaStream_t stream) {
  const lmoe_status st = check_rows(logits, logits_dtype, ld_logits, router_bias, topk_idx, T, E, k);
  if (st != LMOE_OK) return st;
  if (ld_dlogits < E || (loss_grads == nullptr && topk_w_grad == nullptr)) return LMOE_ERR_ARG;
  if (logits == dlogits && ld_logits != ld_dlogits) return LMOE_ERR_ARG;
  if (loss_grads != nullptr && counts == nullptr) return LMOE_ERR_ARG;
  if (T == 0) return LMOE_OK;
  if (dlogits == nullptr || (topk_w_grad != nullptr && topk_idx == nullptr)) return LMOE_ERR_ARG;
  const bool f32 = logits_dtype == LMOE_F32;
  const int es = f32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(dlogits) % es || reinterpret_cast<uintptr_t>(topk_w_grad) % 4 ||
      reinterpret_cast<uintptr_t>(counts) % 4 || reinterpret_cast<uintptr_t>(loss_grads) % 4)
    return LMOE_ERR_ALIGN;
  const GradArgs a = {logits, ld_logits, router_bias, row_mask, topk_idx, topk_w_grad, counts, loss_grads,
                      T,      E,         k,           dlogits,  ld_dlogits};
  const size_t smem = static_cast<size_t>(kWarps) * E * 4;
  const bool vec = rows_vec(logits, ld_logits, E, es) && rows_vec(dlogits, ld_dlogits, E, es);
  const int grid = std::max(1, std::min(4 * sm_count(), (T + kWarps - 1) / kWarps));
  const cudaError_t e = by_shape(f32, E, vec, [&](auto t, auto v, auto vc) {
    auto kern = grad_kernel<decltype(t), decltype(v)::value, decltype(vc)::value>;
    const cudaError_t r = allow_smem(reinterpret_cast<const void*>(kern), static_cast<int>(smem));
    return r != cudaSuccess ? r : launch_pdl(kern, dim3(grid), dim3(kThreads), smem, stream, a);
  });
  return e == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}
