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
// Both read each logit once; the memory traffic bounds them.  G lanes take a row, V values each in
// registers (G V >= E), so a warp has 32 / G rows under way, and loads its next ones before it
// works on the present ones.  exp(l - m) is exp2((l - m) log2e): the difference first, so that a row
// of the type's lowest value, whose product with log2e overflows, still gets its probabilities.
// Sums are held in fp32: against 64 bits the losses of 16384 x 256 are off by 5.8e-8 of themselves, half a step of fp32
// (sums in 64 bits, rounded once, by 3.5e-8).
// The column sums of p stay in registers over a warp's rows, are added over the CTA's warps and,
// through the cluster's shared memory, over eight CTAs, always in the same order; one cluster
// finishes by itself, several leave a row of sums each for a second kernel.
//
// Measured, launched from a graph: losses of 64 x 16 2.8 us, of 16384 x 256 fp32 11.2 us (2.5 us of memory
// traffic; two launches, each a trip to memory and the reductions behind it); gradient of 512 x 256
// 3.7 us, of 16384 x 256 bf16 10.4 us (2.6 us of traffic; a row's chain of load, reductions and store).
#include <algorithm>

#include "../../include/latent_moe.h"
#include "internal.h"
#include "ptx.cuh"

namespace lmoe {
namespace {

constexpr int kLossWarps = 16, kGradWarps = 8;
constexpr int kLossThreads = kLossWarps * 32, kGradThreads = kGradWarps * 32;
constexpr int kCluster = 8;
constexpr int kMaxClusters = 36;   // two CTAs on 144 of 152 SMs: what fits inside the units' borders
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
// over a group of G lanes
template <int G>
LMOE_DEV float group_max_nan(float v) {
#pragma unroll
  for (int d = G / 2; d; d >>= 1) v = max_nan(v, __shfl_xor_sync(~0u, v, d));
  return v;
}
template <int G>
LMOE_DEV float group_sum(float v) {
#pragma unroll
  for (int d = G / 2; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
  return v;
}

// Value i of lane l of a group is element col(l, i) of the row: four neighbours at a time where
// the rows allow 4-element loads, else every G-th.
template <int G, bool VEC>
LMOE_DEV int col(int l, int i) {
  return VEC ? (i >> 2) * (4 * G) + l * 4 + (i & 3) : l + G * i;
}

template <typename T, int G, int V, bool VEC>
LMOE_DEV void load_row(const T* row, int E, int l, float (&v)[V]) {
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < V / 4; ++j) {
      const int e = col<G, true>(l, 4 * j);
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
      const int e = col<G, false>(l, i);
      v[i] = e < E ? to_f32(row[e]) : -INFINITY;
    }
  }
}
template <int G, int V, bool VEC>
LMOE_DEV void add_bias(const float* bias, int E, int l, float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = col<G, VEC>(l, i);
    if (e < E) v[i] += bias[e];
  }
}
// v becomes exp(l - max); returns their sum over the row.  m: the row's maximum, not -inf.
template <int G, int V>
LMOE_DEV float exp_row(float (&v)[V], float m) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    v[i] = exp2f((v[i] - m) * kLog2e);
    s += v[i];
  }
  return group_sum<G>(s);
}
template <int G, int V>
LMOE_DEV float row_max(const float (&v)[V]) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < V; ++i) m = max_nan(m, v[i]);
  return group_max_nan<G>(m);
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
  float* part_p;        // [clusters][E]
  int32_t* part_c;      // [clusters][E]
  float* part_z;        // [clusters]
  int32_t* part_n;      // [clusters]
  int cluster, clusters;
};

// Sum over a CTA of kLossThreads, in warp order, in every thread.
LMOE_DEV float block_sum(float v, float* sm) {
  v = group_sum<32>(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int w = 0; w < kLossWarps; ++w) s += sm[w];
  return s;
}

template <typename T, int G, int V, bool VEC>
__global__ void __launch_bounds__(kLossThreads, V <= 16 ? 2 : 1) losses_kernel(const LossArgs a) {
  constexpr int kRows = 32 / G, kSlots = G < 16 ? 16 / G : 1;
  extern __shared__ float sm_p[];   // [kLossWarps][E], whose first row becomes the CTA's sums; hist [E]
  int* hist = reinterpret_cast<int*>(sm_p + kLossWarps * a.E);
  __shared__ float sm_z[kLossWarps];
  __shared__ int sm_n[kLossWarps];
  __shared__ float sm_d[kLossWarps];
  __shared__ float cta_z, cta_dot;
  __shared__ int cta_n;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane / G, l = lane % G;
  for (int e = threadIdx.x; e < a.E; e += kLossThreads) hist[e] = 0;
  griddep_enter();
  __syncthreads();
  const T* logits = static_cast<const T*>(a.logits);
  const int step = gridDim.x * kLossWarps * kRows;
  float acc[V], next[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  float z = 0.f;
  int n = 0, ids[kSlots];
  int t = (blockIdx.x * kLossWarps + warp) * kRows + g;
  bool live;
#pragma unroll
  for (int i = 0; i < V; ++i) next[i] = -INFINITY;
  // row t, if there is one: loaded beside its mask, not after it
  const auto fetch = [&] {
    live = t < a.T;
    if (live) {
      load_row<T, G, V, VEC>(logits + t * a.ld, a.E, l, next);
#pragma unroll
      for (int s = 0; s < kSlots; ++s)
        ids[s] = l + G * s < a.k ? a.idx[static_cast<long long>(t) * a.k + l + G * s] : -1;
      if (a.mask != nullptr) live = a.mask[t] != 0;
    }
  };
  fetch();
  while (t - g < a.T) {   // (the same for the warp)
    float v[V];
    int slot[kSlots];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = next[i];
#pragma unroll
    for (int s = 0; s < kSlots; ++s) slot[s] = ids[s];
    const bool here = live;
    t += step;
    fetch();
    if (a.bias != nullptr) add_bias<G, V, VEC>(a.bias, a.E, l, v);
    float m = row_max<G>(v);
    const bool on = here && m != -INFINITY;
    m = on ? m : 0.f;
    const float s = exp_row<G>(v, m);
    const float r = 1.f / s;
    if (on) {   // (a row that is not live may hold anything)
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = fmaf(v[i], r, acc[i]);
      const float lse = m + logf(s);
      z = fmaf(lse, lse, z);
      ++n;
#pragma unroll
      for (int q = 0; q < kSlots; ++q)
        if (slot[q] >= 0 && slot[q] < a.E) atomicAdd(&hist[slot[q]], 1);
    }
  }
  // the CTA's sums: groups of a warp, then warps
#pragma unroll
  for (int d = G; d < 32; d <<= 1) {
    z += __shfl_xor_sync(~0u, z, d);
    n += __shfl_xor_sync(~0u, n, d);
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] += __shfl_xor_sync(~0u, acc[i], d);
  }
  if (g == 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = col<G, VEC>(l, i);
      if (e < a.E) sm_p[warp * a.E + e] = acc[i];
    }
  }
  if (lane == 0) {
    sm_z[warp] = z;
    sm_n[warp] = n;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kLossThreads) {
    float p = 0.f;
    for (int w = 0; w < kLossWarps; ++w) p += sm_p[w * a.E + e];
    sm_p[e] = p;   // (column e is this thread's alone)
  }
  if (threadIdx.x == 0) {
    float zz = 0.f;
    int nn = 0;
    for (int w = 0; w < kLossWarps; ++w) {
      zz += sm_z[w];
      nn += sm_n[w];
    }
    cta_z = zz;
    cta_n = nn;
  }
  // the cluster's: each CTA adds its share of the columns over all of them
  cluster_sync();
  const int rank = blockIdx.x % a.cluster, cl = blockIdx.x / a.cluster;
  const int share = (a.E + a.cluster - 1) / a.cluster, e0 = rank * share, e1 = min(e0 + share, a.E);
  float zz = 0.f, dot = 0.f;
  int nn = 0;
  for (int q = 0; q < a.cluster; ++q) {
    zz += __uint_as_float(cluster_load(cluster_map(smem_u32(&cta_z), q)));
    nn += static_cast<int>(cluster_load(cluster_map(smem_u32(&cta_n), q)));
  }
  const float inv = nn > 0 ? 1.f / nn : 0.f;
  for (int e = e0 + threadIdx.x; e < e1; e += kLossThreads) {
    float p = 0.f;
    int c = 0;
    for (int q = 0; q < a.cluster; ++q) {
      p += __uint_as_float(cluster_load(cluster_map(smem_u32(sm_p + e), q)));
      c += static_cast<int>(cluster_load(cluster_map(smem_u32(hist + e), q)));
    }
    if (a.clusters == 1) {
      a.mean[e] = p * inv;
      a.counts[e] = c;
      dot = fmaf(p * inv, c * inv, dot);
    } else {
      a.part_p[static_cast<long long>(cl) * a.E + e] = p;
      a.part_c[static_cast<long long>(cl) * a.E + e] = c;
    }
  }
  if (a.clusters == 1) {
    dot = block_sum(dot, sm_d);
    if (threadIdx.x == 0) cta_dot = dot;
  }
  cluster_sync();
  if (rank == 0 && threadIdx.x == 0) {
    if (a.clusters == 1) {
      float d = 0.f;
      for (int q = 0; q < a.cluster; ++q) d += __uint_as_float(cluster_load(cluster_map(smem_u32(&cta_dot), q)));
      a.counts[a.E] = nn;
      a.losses[0] = d * a.E / a.k;
      a.losses[1] = zz * inv;
    } else {
      a.part_z[cl] = zz;
      a.part_n[cl] = nn;
    }
  }
  cluster_sync();   // no CTA leaves while another reads its shared memory
}

// Adds the clusters' sums, in order: groups of threads, one to an expert each, take every
// groups-th cluster, whose loads are then under way together.
constexpr int kFinishThreads = 1024;
__global__ void __launch_bounds__(kFinishThreads) losses_finish_kernel(const LossArgs a) {
  __shared__ float sm_p[kFinishThreads];
  __shared__ int sm_c[kFinishThreads];
  __shared__ float sm_d[kFinishThreads / 32];
  griddep_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int W = 32;
  while (W < a.E) W *= 2;   // E <= 1024
  const int groups = kFinishThreads / W, grp = threadIdx.x / W, e = threadIdx.x % W;
  constexpr int kPerLane = (kMaxClusters + 31) / 32, kBatch = 12;
  float p = 0.f, z = 0.f, n = 0.f;   // (counts of rows are exact in fp32: at most 2^20)
  int c = 0;
  // every load of a thread under way before the first sum
  float zs[kPerLane], ps[kBatch];
  int ns[kPerLane], cs[kBatch];
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const bool in = lane + 32 * i < a.clusters;
    ns[i] = in ? a.part_n[lane + 32 * i] : 0;
    zs[i] = in ? a.part_z[lane + 32 * i] : 0.f;
  }
  for (int q0 = grp; q0 < a.clusters; q0 += groups * kBatch) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int q = q0 + i * groups;
      const bool in = q < a.clusters && e < a.E;
      ps[i] = in ? a.part_p[q * a.E + e] : 0.f;
      cs[i] = in ? a.part_c[q * a.E + e] : 0;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      p += ps[i];
      c += cs[i];
    }
  }
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    n += static_cast<float>(ns[i]);
    z += zs[i];
  }
  n = group_sum<32>(n);
  z = group_sum<32>(z);
  const float inv = n > 0.f ? 1.f / n : 0.f;
  sm_p[threadIdx.x] = p;
  sm_c[threadIdx.x] = c;
  __syncthreads();
  float dot = 0.f;
  if (threadIdx.x < a.E) {
    for (int g = 1; g < groups; ++g) {
      p += sm_p[g * W + e];
      c += sm_c[g * W + e];
    }
    a.mean[e] = p * inv;
    a.counts[e] = c;
    dot = p * inv * (c * inv);
  }
  dot = group_sum<32>(dot);
  if (lane == 0) sm_d[warp] = dot;
  __syncthreads();
  if (warp == 0) {
    dot = group_sum<32>(sm_d[lane]);
    if (lane == 0) {
      a.counts[a.E] = static_cast<int>(n);
      a.losses[0] = dot * a.E / a.k;
      a.losses[1] = z * inv;
    }
  }
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

template <typename T, int G, int V, bool VEC>
__global__ void __launch_bounds__(kGradThreads, V <= 16 ? 4 : 2) grad_kernel(const GradArgs a) {
  constexpr int kRows = 32 / G, kSlots = G < 16 ? 16 / G : 1;
  extern __shared__ float sm_row[];   // [rows of the CTA][E]: a row while its slots' terms are added
  __shared__ int sm_id[G < 16 ? kGradWarps * kRows : 1][16];
  __shared__ float sm_g[G < 16 ? kGradWarps * kRows : 1][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane / G, l = lane % G;
  const int local = warp * kRows + g;
  float* sm_f = sm_row + kGradWarps * kRows * a.E;   // [E] shares of the slots
  float* row = sm_row + local * a.E;
  griddep_enter();
  const T* logits = static_cast<const T*>(a.logits);
  T* out = static_cast<T*>(a.out);
  // one row per group: more CTAs hide the latencies better than rows loaded ahead, whose registers
  // they need (16384 x 256 bf16: 10.3 us, loaded ahead 11.6)
  const int t = (blockIdx.x * kGradWarps + warp) * kRows + g;
  float v[V], gw[kSlots], sel[kSlots];
  int id[kSlots];
  bool on = t < a.T;
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = -INFINITY;
#pragma unroll
  for (int s = 0; s < kSlots; ++s) {
    id[s] = -1;
    gw[s] = 0.f;
  }
  if (on) {   // the row beside its mask and its slots, not after them
    load_row<T, G, V, VEC>(logits + t * a.ld, a.E, l, v);
    if (a.gw != nullptr) {
#pragma unroll
      for (int s = 0; s < kSlots; ++s)
        if (l + G * s < a.k) {
          id[s] = a.idx[static_cast<long long>(t) * a.k + l + G * s];
          gw[s] = a.gw[static_cast<long long>(t) * a.k + l + G * s];
        }
    }
    if (a.mask != nullptr) on = a.mask[t] != 0;
  }
  float cb = 0.f, cz = 0.f;
  if (a.gl != nullptr) {
    const float inv = 1.f / max(a.counts[a.E], 1);
    cb = a.gl[0] * a.E * inv;
    cz = a.gl[1] * 2.f * inv;
    const float fk = inv / a.k;
    for (int e = threadIdx.x; e < a.E; e += kGradThreads) sm_f[e] = a.counts[e] * fk;
    __syncthreads();
  }
  {
    // the slots' logits are read before the row is written (it may be written in place)
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      if (id[s] < 0 || id[s] >= a.E) {
        id[s] = -1;
        gw[s] = 0.f;
      }
      sel[s] = id[s] < 0 ? -INFINITY
                         : to_f32(logits[t * a.ld + id[s]]) + (a.bias != nullptr ? a.bias[id[s]] : 0.f);
    }
    if (a.bias != nullptr) add_bias<G, V, VEC>(a.bias, a.E, l, v);
    // The row's reductions in two rounds, the maxima and the sums, those of a round side by side (a
    // round is a chain of shuffles).  sum f p = (sum f exp) / (sum exp), and so for the weights.
    float m = v[0], sm = sel[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = max_nan(m, v[i]);
#pragma unroll
    for (int q = 1; q < kSlots; ++q) sm = max_nan(sm, sel[q]);
#pragma unroll
    for (int d = G / 2; d; d >>= 1) {
      m = max_nan(m, __shfl_xor_sync(~0u, m, d));
      sm = max_nan(sm, __shfl_xor_sync(~0u, sm, d));
    }
    on = on && m != -INFINITY;
    m = on ? m : 0.f;
    const bool none = sm == -INFINITY;   // no slot with a logit above -inf: no weights, no gradient
    float s = 0.f, sf = 0.f, ws = 0.f, wg = 0.f, w[kSlots];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = col<G, VEC>(l, i);
      v[i] = exp2f((v[i] - m) * kLog2e);
      s += v[i];
      if (a.gl != nullptr && e < a.E) sf = fmaf(v[i], sm_f[e], sf);
    }
#pragma unroll
    for (int q = 0; q < kSlots; ++q) {
      w[q] = none ? 0.f : exp2f((sel[q] - sm) * kLog2e);
      ws += w[q];
      wg = fmaf(w[q], gw[q], wg);
    }
#pragma unroll
    for (int d = G / 2; d; d >>= 1) {
      s += __shfl_xor_sync(~0u, s, d);
      sf += __shfl_xor_sync(~0u, sf, d);
      ws += __shfl_xor_sync(~0u, ws, d);
      wg += __shfl_xor_sync(~0u, wg, d);
    }
    if (on && a.gl != nullptr) {
      const float r = 1.f / s, lz = cz * (m + logf(s)), dot = sf * r;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = col<G, VEC>(l, i);
        if (e < a.E) v[i] *= r * fmaf(cb, sm_f[e] - dot, lz);
      }
    } else {   // (a row that is not live may hold anything)
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = 0.f;
    }
    if (a.gw != nullptr) {
      const float wr = none ? 0.f : 1.f / ws;
      wg *= wr;
      float d[kSlots];
#pragma unroll
      for (int q = 0; q < kSlots; ++q) d[q] = on && id[q] >= 0 ? w[q] * wr * (gw[q] - wg) : 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = col<G, VEC>(l, i);
        if (e < a.E) row[e] = v[i];
      }
      // an expert named by several slots of the row: its first slot adds them all, in order
      if constexpr (G >= 16) {
        const unsigned same = __match_any_sync(~0u, (g << 16) | (id[0] & 0xffff));
        const bool first = id[0] >= 0 && lane == __ffs(same) - 1;
        if (__any_sync(~0u, id[0] >= 0 && __popc(same) > 1)) {
          float tot = 0.f;
          for (int j = 0; j < a.k; ++j) {
            const float dj = __shfl_sync(~0u, d[0], g * G + j);
            if ((same >> (g * G + j)) & 1u) tot += dj;
          }
          d[0] = tot;
        }
        __syncwarp();
        if (first) row[id[0]] += d[0];
      } else {
#pragma unroll
        for (int q = 0; q < kSlots; ++q)
          if (l + G * q < 16) {
            sm_id[local][l + G * q] = id[q];
            sm_g[local][l + G * q] = d[q];
          }
        __syncwarp();
#pragma unroll
        for (int q = 0; q < kSlots; ++q) {
          bool first = id[q] >= 0;
          float tot = 0.f;
          for (int j = 0; j < a.k; ++j) {
            if (sm_id[local][j] != id[q]) continue;
            if (j < l + G * q) first = false;
            tot += sm_g[local][j];
          }
          if (first) row[id[q]] += tot;
        }
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = col<G, VEC>(l, i);
        if (e < a.E) v[i] = row[e];
      }
      __syncwarp();
    }
    if (t >= a.T) return;
    T* o = out + t * a.ldo;
    if constexpr (VEC) {
#pragma unroll
      for (int j = 0; j < V / 4; ++j) {
        const int e = col<G, true>(l, 4 * j);
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
        const int e = col<G, false>(l, i);
        if (e < a.E) store_as(o + e, v[i]);
      }
    }
  }
}

// Calls f with (T, G, V, VEC) for E experts.
template <int V>
using Int = std::integral_constant<int, V>;
template <typename F>
cudaError_t by_shape(bool f32, int E, bool vec, F f) {
  const auto with = [&](auto g, auto v) {
    if (f32) return vec ? f(float{}, g, v, std::true_type{}) : f(float{}, g, v, std::false_type{});
    return vec ? f(__nv_bfloat16{}, g, v, std::true_type{}) : f(__nv_bfloat16{}, g, v, std::false_type{});
  };
  if (E <= 16) return with(Int<4>{}, Int<4>{});
  if (E <= 64) return with(Int<8>{}, Int<8>{});
  if (E <= 128) return with(Int<8>{}, Int<16>{});
  if (E <= 256) return with(Int<16>{}, Int<16>{});
  if (E <= 512) return with(Int<32>{}, Int<16>{});
  return with(Int<32>{}, Int<32>{});
}
// rows of a warp at a time
int warp_rows(int E) { return E <= 16 ? 8 : E <= 128 ? 4 : E <= 256 ? 2 : 1; }

// rows of 4-element loads: base, row length and the count of elements allow them
bool rows_vec(const void* p, long long ld, int E, int es) {
  return E % 4 == 0 && ld % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (4 * es) == 0;
}
// CTAs of the losses kernel, in clusters of one or eight: one CTA while each warp takes up to four
// turns of rows, then clusters of two turns, as many as the SMs hold.
struct LossGrid {
  int cluster, clusters;
};
LossGrid losses_grid(int T, int E) {
  const int turn = kLossWarps * warp_rows(E);   // rows of a CTA at a time
  if (T <= 4 * turn) return {1, 1};
  const int want = (T + 2 * turn * kCluster - 1) / (2 * turn * kCluster);
  return {kCluster, std::min(want, E <= 512 ? kMaxClusters : kMaxClusters / 2)};
}

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
  *bytes = static_cast<size_t>(losses_grid(T, E).clusters) * (2 * E + 2) * 4;
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
  const LossGrid lg = losses_grid(T, E);
  a.cluster = lg.cluster;
  a.clusters = lg.clusters;
  const size_t need = static_cast<size_t>(lg.clusters) * (2 * E + 2) * 4;
  if (workspace == nullptr || workspace_bytes < need) return LMOE_ERR_WORKSPACE;
  a.part_p = static_cast<float*>(workspace);
  a.part_c = reinterpret_cast<int32_t*>(a.part_p + static_cast<size_t>(lg.clusters) * E);
  a.part_z = reinterpret_cast<float*>(a.part_c + static_cast<size_t>(lg.clusters) * E);
  a.part_n = reinterpret_cast<int32_t*>(a.part_z + lg.clusters);
  const size_t smem = static_cast<size_t>(kLossWarps + 1) * E * 4;
  const bool f32 = logits_dtype == LMOE_F32;
  cudaError_t e = by_shape(f32, E, rows_vec(logits, ld_logits, E, f32 ? 4 : 2), [&](auto t, auto g, auto v, auto vec) {
    auto kern = losses_kernel<decltype(t), decltype(g)::value, decltype(v)::value, decltype(vec)::value>;
    const cudaError_t r = allow_smem(reinterpret_cast<const void*>(kern), static_cast<int>(smem));
    return r != cudaSuccess ? r
                            : launch_pdl_cluster(kern, dim3(lg.cluster * lg.clusters), dim3(kLossThreads), smem,
                                                 stream, lg.cluster, a);
  });
  if (e == cudaSuccess && lg.clusters > 1)
    e = launch_pdl(losses_finish_kernel, dim3(1), dim3(kFinishThreads), 0, stream, a);
  return e == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}

extern "C" lmoe_status lmoe_router_grad(const void* logits, lmoe_dtype logits_dtype, long long ld_logits,
                                        const float* router_bias, const uint8_t* row_mask, const int32_t* topk_idx,
                                        const float* topk_w_grad, const int32_t* counts, const float* loss_grads,
                                        int T, int E, int k, void* dlogits, long long ld_dlogits,
                                        cudaStream_t stream) {
  const lmoe_status st = check_rows(logits, logits_dtype, ld_logits, router_bias, topk_idx, T, E, k);
  if (st != LMOE_OK) return st;
  if (ld_dlogits < E) return LMOE_ERR_ARG;
  if (logits == dlogits && ld_logits != ld_dlogits) return LMOE_ERR_ARG;
  if (loss_grads != nullptr && counts == nullptr) return LMOE_ERR_ARG;
  if (T == 0) return LMOE_OK;   // (an empty tensor's pointer may be NULL)
  if (loss_grads == nullptr && topk_w_grad == nullptr) return LMOE_ERR_ARG;
  if (dlogits == nullptr || (topk_w_grad != nullptr && topk_idx == nullptr)) return LMOE_ERR_ARG;
  const bool f32 = logits_dtype == LMOE_F32;
  const int es = f32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(dlogits) % es || reinterpret_cast<uintptr_t>(topk_w_grad) % 4 ||
      reinterpret_cast<uintptr_t>(counts) % 4 || reinterpret_cast<uintptr_t>(loss_grads) % 4)
    return LMOE_ERR_ALIGN;
  const GradArgs a = {logits, ld_logits, router_bias, row_mask, topk_idx, topk_w_grad, counts, loss_grads,
                      T,      E,         k,           dlogits,  ld_dlogits};
  const int turn = kGradWarps * warp_rows(E);   // rows of a CTA at a time
  const size_t smem = static_cast<size_t>(turn + 1) * E * 4;
  const bool vec = rows_vec(logits, ld_logits, E, es) && rows_vec(dlogits, ld_dlogits, E, es);
  const int grid = (T + turn - 1) / turn;
  const cudaError_t e = by_shape(f32, E, vec, [&](auto t, auto g, auto v, auto vc) {
    auto kern = grad_kernel<decltype(t), decltype(g)::value, decltype(v)::value, decltype(vc)::value>;
    const cudaError_t r = allow_smem(reinterpret_cast<const void*>(kern), static_cast<int>(smem));
    return r != cudaSuccess ? r : launch_pdl(kern, dim3(grid), dim3(kGradThreads), smem, stream, a);
  });
  return e == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}
