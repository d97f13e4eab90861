// Attention over the paged cache for sequences that share a prefix:
//   out_r = sum_j exp(s_rj - m) v_j / sum_j exp(s_rj - m),  s_rj = scale q_r . k_j,
// j over the prefix and the row's own tokens, with the running maximum m and
// the sums in fp32 (one pass over the keys).
#include "heads.h"

namespace moe {

template <class C>
__device__ __forceinline__ float cache_f32(const C* p, long long i) {
  if constexpr (sizeof(C) == 1) return e4m3_to_f32(p[i]);
  else return to_f32(p[i]);
}

constexpr int kKeys = 256;   // keys of a step: one per thread

// One block per query row (b, i, h). A step scores 256 keys (a thread per key), takes the block's maximum,
// then a thread per channel adds the weighted values.
template <class T, class C>
__global__ __launch_bounds__(256) void attend_kernel(AttendArgs a) {
  __shared__ float qs[256], ps[kKeys], red[8];
  __shared__ long long rows[kKeys];
  const int tid = threadIdx.x, D = a.c.D, Hq = a.q.heads, G = Hq / a.c.heads;
  const int h = blockIdx.x % Hq, t = blockIdx.x / Hq, b = t / a.S, i = t % a.S, hk = h / G;
  const T* q = static_cast<const T*>(a.q.in) + t * a.q.in_t + h * a.q.in_h;
  if (tid < D) qs[tid] = to_f32(q[tid]) * a.scale;
  int n = 0;
  if (a.table_pages > 0) {
    n = clampi(a.lens[b], 0, static_cast<int>(min(static_cast<long long>(a.table_pages) * a.c.page_size, 0x7fffffffLL)));
    n = max(0, n - a.S + 1 + i);
  }
  const long long total = static_cast<long long>(a.P) + n;
  float m = -INFINITY, l = 0.0f, o = 0.0f;
  __syncthreads();
  for (long long j0 = 0; j0 < total; j0 += kKeys) {
    const long long j = j0 + tid;
    float s = -INFINITY;
    long long row = -1;
    if (j < total) {
      const bool pre = j < a.P;
      const int jj = static_cast<int>(pre ? j : j - a.P);
      const int page = pre ? a.prefix_pages[jj / a.c.page_size]
                           : a.page_table[static_cast<long long>(b) * a.table_pages + jj / a.c.page_size];
      if (page >= 0 && page < a.c.n_pages)
        row = (static_cast<long long>(page) * a.c.heads + hk) * a.c.page_size + jj % a.c.page_size;
    }
    if (row >= 0) {
      const C* k = static_cast<const C*>(a.c.k) + row * D;
      s = 0.0f;
      for (int c = 0; c < D; ++c) s = fmaf(qs[c], cache_f32(k, c), s);
      if constexpr (sizeof(C) == 1) s *= a.c.k_scale[row];
    }
    rows[tid] = row;
    float w = wave_max(s);
    if ((tid & 63) == 0) red[tid >> 6] = w;
    __syncthreads();
    const float mn = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
    const float keep = mn == -INFINITY ? 1.0f : __expf(m - mn);
    float p = row >= 0 ? __expf(s - mn) : 0.0f;
    float sum = p;
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d, kWave);
    if ((tid & 63) == 0) red[4 + (tid >> 6)] = sum;
    if constexpr (sizeof(C) == 1) p *= row >= 0 ? a.c.v_scale[row] : 0.0f;
    ps[tid] = p;
    __syncthreads();
    l = l * keep + (red[4] + red[5] + red[6] + red[7]);
    m = mn;
    if (tid < D) {
      o *= keep;
      for (int e = 0; e < kKeys; ++e)
        if (rows[e] >= 0) o = fmaf(ps[e], cache_f32(static_cast<const C*>(a.c.v) + rows[e] * D, tid), o);
    }
    __syncthreads();
  }
  if (tid < D) {
    T* out = static_cast<T*>(a.q.out) + t * a.q.out_t + h * a.q.out_h;
    out[tid] = from_f32<T>(m == -INFINITY ? 0.0f : o / l);
  }
  if (a.lse && tid == 0) a.lse[static_cast<long long>(t) * Hq + h] = m == -INFINITY ? -INFINITY : m + logf(l);
}

size_t attend_ws_bytes(const Cache&, int, int, int, int, int) { return 256; }

hipError_t launch_attend(const AttendArgs& a, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.B) * a.S * a.q.heads), block(256);
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, block, 0, st, a);
    return hipGetLastError();
  };
  if (a.act == MOE_F32) return go(attend_kernel<float, float>);
  return a.c.dtype == MOE_BF16 ? go(attend_kernel<__bf16, __bf16>) : go(attend_kernel<__bf16, uint8_t>);
}

}  // namespace moe
