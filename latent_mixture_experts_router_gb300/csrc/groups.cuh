// groups.cuh — rows sorted by expert, as the grouped products walk them.
#pragma once
#include "internal.h"
#include "ptx.cuh"

namespace lmoe {

constexpr int kMaxGroups = 1024;

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

// Row tiles of `unit` rows that any split of `rows` among E experts takes at most (rows > 0).
__host__ __device__ constexpr int most_tiles(int rows, int E, int unit) {
  return (rows + unit - 1) / unit + (E < rows ? E : rows) - 1;
}

// mbar_wait of a whole warp, with one outcome: its lanes' own waits may give up one by one, and TMEM reads,
// votes and warp barriers follow that need all of them.
LMOE_DEV bool warp_wait(uint64_t* bar, uint32_t parity, long long budget) {
  return __all_sync(~0u, mbar_wait(bar, parity, budget));
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

LMOE_DEV void tma_load_3d_hint(void* dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1, int c2,
                               uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
      : "memory");
}

}  // namespace lmoe
