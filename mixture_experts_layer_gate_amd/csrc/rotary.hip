// Rotary positions (forward and gradient), their table, and the append of
// rotated keys and values to the paged cache.
//
// A pair (a, b) of channels turns by the angle of its token's position:
// (a c - b s, b c + a s). The gradient is the transposed rotation, s -> -s.
#include "heads.h"

namespace moe {

__global__ void rope_table_kernel(int half, long long n, double log_base_step, double factor, double orig_len, double slow,
                                  double fast, double amplitude, bool parts, float* __restrict__ table) {
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long e = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; e < n; e += stride) {
    const long long p = e / half;
    const int i = static_cast<int>(e - p * half);
    double theta = exp(-i * log_base_step);
    if (parts) {
      const double turns = orig_len * theta / 6.283185307179586476925;
      const double g = fmin(fmax((turns - slow) / (fast - slow), 0.0), 1.0);
      theta *= g + (1.0 - g) / factor;
    } else {
      theta /= factor;
    }
    double s, c;
    sincos(static_cast<double>(p) * theta, &s, &c);
    table[2 * e] = static_cast<float>(amplitude * c);
    table[2 * e + 1] = static_cast<float>(amplitude * s);
  }
}

hipError_t launch_rope_table(int R, int n_positions, double base, double factor, double orig_len, double slow,
                             double fast, double amplitude, bool parts, float* table, hipStream_t st) {
  const int half = R / 2;
  const long long n = static_cast<long long>(n_positions) * half;
  const long long blocks = (n + 255) / 256;
  const int grid = static_cast<int>(blocks < 65536 ? blocks : 65536);
  hipLaunchKernelGGL(rope_table_kernel, dim3(grid), dim3(256), 0, st, half, n, 2.0 * log(base) / R, factor, orig_len,
                     slow, fast, amplitude, parts, table);
  return hipGetLastError();
}

// The two channels of pair i.
__device__ __forceinline__ void pair_channels(const moe_rope& r, int i, int& a, int& b) {
  if (r.layout == MOE_ROPE_HALF) { a = i; b = i + r.rot_dim / 2; }
  else { a = 2 * i; b = 2 * i + 1; }
}

// One wave per (token, head); a lane takes every 64th pair, then every 64th channel after the rotated ones.
template <class T>
__device__ void rotate_row(const moe_rope& r, int D, const T* x, T* y, const float* cs, float sign) {
  const int lane = threadIdx.x & 63, half = r.rot_dim / 2;
  for (int i = lane; i < half; i += 64) {
    int a, b;
    pair_channels(r, i, a, b);
    const float c = cs[2 * i], s = sign * cs[2 * i + 1];
    const float xa = to_f32(x[a]), xb = to_f32(x[b]);
    y[a] = from_f32<T>(xa * c - xb * s);
    y[b] = from_f32<T>(xb * c + xa * s);
  }
  for (int c = r.rot_dim + lane; c < D; c += 64) y[c] = x[c];
}

template <class T>
__global__ __launch_bounds__(256) void rotary_kernel(moe_rope r, int n_tok, int D, Rows q, Rows k,
                                                     const int32_t* __restrict__ positions, float sign) {
  const int heads = q.heads + k.heads;
  const long long n = static_cast<long long>(n_tok) * heads;
  for (long long w = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 6); w < n; w += 4LL * gridDim.x) {
    const int t = static_cast<int>(w / heads);
    int h = static_cast<int>(w - static_cast<long long>(t) * heads);
    const int p = positions[t];
    if (p < 0 || p >= r.n_positions) continue;
    const bool is_q = h < q.heads;
    const Rows& m = is_q ? q : k;
    if (!is_q) h -= q.heads;
    rotate_row<T>(r, D, static_cast<const T*>(m.in) + t * m.in_t + h * m.in_h,
                  static_cast<T*>(m.out) + t * m.out_t + h * m.out_h, r.table + static_cast<long long>(p) * r.rot_dim,
                  sign);
  }
}

static int wave_blocks(long long waves) {
  const long long b = (waves + 3) / 4, cap = static_cast<long long>(device_cu_count()) * 32;
  return static_cast<int>(b < cap ? b : cap);
}

hipError_t launch_rotary(const moe_rope& rope, moe_dtype act, int T, int D, const Rows& q, const Rows& k,
                         const int32_t* positions, float sign, hipStream_t st) {
  const dim3 grid(wave_blocks(static_cast<long long>(T) * (q.heads + k.heads))), block(256);
  if (act == MOE_BF16)
    hipLaunchKernelGGL(rotary_kernel<__bf16>, grid, block, 0, st, rope, T, D, q, k, positions, sign);
  else
    hipLaunchKernelGGL(rotary_kernel<float>, grid, block, 0, st, rope, T, D, q, k, positions, sign);
  return hipGetLastError();
}

// Channel c of the row after the rotation, in fp32.
template <class T>
__device__ float rotated(const moe_rope& r, const T* x, const float* cs, int c) {
  if (c >= r.rot_dim) return to_f32(x[c]);
  const int half = r.rot_dim / 2;
  const bool first = r.layout == MOE_ROPE_HALF ? c < half : (c & 1) == 0;
  const int i = r.layout == MOE_ROPE_HALF ? (first ? c : c - half) : c >> 1;
  int a, b;
  pair_channels(r, i, a, b);
  const float co = cs[2 * i], s = cs[2 * i + 1], xa = to_f32(x[a]), xb = to_f32(x[b]);
  return first ? xa * co - xb * s : xb * co + xa * s;
}

// One wave per (token, head of q, k or v).
template <class T, class C>
__global__ __launch_bounds__(256) void kv_append_kernel(Cache ca, moe_rope r, int n_tok, Rows k, Rows v, Rows q,
                                                        const int32_t* __restrict__ positions,
                                                        const int32_t* __restrict__ slots) {
  const int heads = q.heads + k.heads + v.heads, D = ca.D, lane = threadIdx.x & 63;
  const long long n = static_cast<long long>(n_tok) * heads;
  for (long long w = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 6); w < n; w += 4LL * gridDim.x) {
    const int t = static_cast<int>(w / heads);
    int h = static_cast<int>(w - static_cast<long long>(t) * heads);
    const float* cs = nullptr;
    if (r.rot_dim > 0) {
      const int p = positions[t];
      if (p < 0 || p >= r.n_positions) continue;
      cs = r.table + static_cast<long long>(p) * r.rot_dim;
    }
    if (h < q.heads) {
      rotate_row<T>(r, D, static_cast<const T*>(q.in) + t * q.in_t + h * q.in_h,
                    static_cast<T*>(q.out) + t * q.out_t + h * q.out_h, cs, 1.0f);
      continue;
    }
    h -= q.heads;
    const bool is_k = h < k.heads;
    if (!is_k) h -= k.heads;
    const long long row = slot_row(ca, slots[t], h);
    if (row < 0) continue;
    const Rows& m = is_k ? k : v;
    moe_rope rr = r;
    if (!is_k) rr.rot_dim = 0;
    const T* x = static_cast<const T*>(m.in) + t * m.in_t + h * m.in_h;
    C* y = static_cast<C*>(is_k ? ca.k : ca.v) + row * D;
    if constexpr (sizeof(C) == 1) {
      float amax = 0.0f;
      for (int c = lane; c < D; c += 64) amax = fmaxf(amax, fabsf(rotated<T>(rr, x, cs, c)));
      amax = wave_max(amax);
      const float inv = amax > 0.0f ? kE4M3Max / amax : 0.0f;
      for (int c = lane; c < D; c += 64) y[c] = static_cast<C>(f32_to_e4m3(rotated<T>(rr, x, cs, c) * inv));
      if (lane == 0) (is_k ? ca.k_scale : ca.v_scale)[row] = amax > 0.0f ? amax / kE4M3Max : 1.0f;
    } else {
      for (int c = lane; c < D; c += 64) y[c] = from_f32<C>(rotated<T>(rr, x, cs, c));
    }
  }
}

hipError_t launch_kv_append(const Cache& c, const moe_rope& rope, moe_dtype act, int T, const Rows& k, const Rows& v,
                            const Rows& q, const int32_t* positions, const int32_t* slots, hipStream_t st) {
  const dim3 grid(wave_blocks(static_cast<long long>(T) * (q.heads + k.heads + v.heads))), block(256);
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, block, 0, st, c, rope, T, k, v, q, positions, slots);
    return hipGetLastError();
  };
  if (act == MOE_BF16)
    return c.dtype == MOE_BF16 ? go(kv_append_kernel<__bf16, __bf16>) : go(kv_append_kernel<__bf16, uint8_t>);
  return c.dtype == MOE_F32 ? go(kv_append_kernel<float, float>) : go(kv_append_kernel<float, uint8_t>);
}

}  // namespace moe
