// Head rows of q, k and v: element loads and stores in fp32 or bf16 (one
// rounding, to nearest even, NaN stays NaN), cache row offsets.
#pragma once

#include "common.h"
#include "launch.h"

namespace moe {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__bf16 x) { return static_cast<float>(x); }
template <class T>
__device__ __forceinline__ T from_f32(float x) { return static_cast<T>(x); }   // bf16: v_cvt_pk_bf16_f32

// What an E4M3 row of magnitude amax is multiplied by. Below 448 / 2^128 the quotient would be infinite, and the row's
// zeros NaN; the largest finite number leaves its values off by less than 2^-119.
__device__ __forceinline__ float row_factor(float amax) {
  return amax > 0.0f ? fminf(kE4M3Max / amax, 0x1.fffffep127f) : 0.0f;
}

// Row (in rows of D elements) of a cache slot's head; -1 if the slot is not in the cache.
__device__ __forceinline__ long long slot_row(const Cache& c, int slot, int head) {
  if (slot < 0) return -1;
  const int page = slot / c.page_size, r = slot % c.page_size;
  if (page >= c.n_pages) return -1;
  return (static_cast<long long>(page) * c.heads + head) * c.page_size + r;
}

}  // namespace moe
