// Rotary positions (forward and gradient), their table, and the append of
// rotated keys and values to the paged cache.
//
// A pair (a, b) of channels turns by the angle of its token's position:
// (a c - b s, b c + a s). The gradient is the transposed rotation, s -> -s.
// All of it is bound by HBM: every channel is read once and written once, beside 4 R bytes of table a token.
//
// Two forms. Rows: a power of two of lanes takes a head row, each lane two 16-byte pieces of it (the two
// halves of its pairs, or neighbours), so a row is one load and one store per piece, and the q, k and v rows
// of all tokens are one flat range over the grid. It needs 16-byte aligned rows and pairs that fill whole
// pieces. Scalar: a wave per row, two elements a lane at a time, for every other stride, alignment and size.
// Rows against scalar: 8192 tokens of 64 heads of 128 (64 rotated) 58 us (4.7 TB/s) against 200; the gradient of 16384 of
// 20 heads 36 against 93; fp32, 4093 of 24 heads of 80, 13 against 30.
//
// The rotation is in fp32 and rounded once, to the output's type; an E4M3 row is scaled from the unrounded fp32 row.
#include <initializer_list>

#include "heads.h"

namespace moe {

// cos and sin of p theta_i in fp64, rounded once: at positions past 2^17 an fp32 angle would be off by 2^-8. Made once
// for a model, bound by the fp64 sine and cosine.
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

// ---------------------------------------------------------------- 16-byte pieces

template <class T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);     // channels of a piece
  float x[N];
  __device__ __forceinline__ void load(const T* p) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        x[i] = __uint_as_float(w[i]);
      }
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    union {
      T t[N];
      uint4 u;
    } y;
#pragma unroll
    for (int i = 0; i < N; ++i) y.t[i] = from_f32<T>(x[i]);
    *reinterpret_cast<uint4*>(p) = y.u;
  }
  __device__ __forceinline__ void store_e4m3(uint8_t* p, float inv) const {
    uint32_t w[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      w[i] = f32x4_to_e4m3(x[4 * i] * inv, x[4 * i + 1] * inv, x[4 * i + 2] * inv, x[4 * i + 3] * inv);
    if constexpr (N == 8) *reinterpret_cast<uint2*>(p) = uint2{w[0], w[1]};
    else *reinterpret_cast<uint32_t*>(p) = w[0];
  }
};

// Lane j of a row's 2^lg lanes takes pieces c0 and c1 (-1: none). Half layout: the two halves of pairs N j ..,
// then the channels after them; interleaved: pieces 2j and 2j + 1.
struct RowsPlan {
  int lg;              // log2 of the lanes of a row
  uint32_t magic;      // ceil(2^32 / rows of a token); 0 for one row
  int rows;            // head rows of a token
};
template <class T>
__device__ __forceinline__ void row_pieces(const moe_rope& r, int D, int j, int& c0, int& c1, bool& turn0, bool& turn1) {
  constexpr int N = Vec<T>::N;
  const int pieces = D / N;
  if (r.layout == MOE_ROPE_HALF) {
    const int half = r.rot_dim / 2 / N;
    if (j < half) { c0 = j; c1 = j + half; turn0 = turn1 = true; return; }
    c0 = 2 * half + 2 * (j - half);
    turn0 = turn1 = false;
  } else {
    c0 = 2 * j;
    turn0 = c0 * N < r.rot_dim;
    turn1 = (c0 + 1) * N < r.rot_dim;
  }
  c1 = c0 + 1 < pieces ? c0 + 1 : -1;
  if (c0 >= pieces) c0 = -1;
}

// Turns the lane's two pieces in place; cs: the position's table row.
template <class T>
__device__ __forceinline__ void turn_pieces(const moe_rope& r, const float* cs, float sign, int c0, int c1, bool turn0,
                                            bool turn1, Vec<T>& x, Vec<T>& y) {
  constexpr int N = Vec<T>::N;
  if (r.layout == MOE_ROPE_HALF) {
    if (!turn0) return;
    const float4* t = reinterpret_cast<const float4*>(cs + 2 * N * c0);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float4 w = t[i];      // (c, s) of two pairs
      const float a0 = x.x[2 * i], b0 = y.x[2 * i], a1 = x.x[2 * i + 1], b1 = y.x[2 * i + 1];
      x.x[2 * i] = a0 * w.x - b0 * (sign * w.y);
      y.x[2 * i] = b0 * w.x + a0 * (sign * w.y);
      x.x[2 * i + 1] = a1 * w.z - b1 * (sign * w.w);
      y.x[2 * i + 1] = b1 * w.z + a1 * (sign * w.w);
    }
    return;
  }
  auto one = [&](Vec<T>& v, int c) {
    const float4* t = reinterpret_cast<const float4*>(cs + N * c);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 w = t[i];
      const float a0 = v.x[4 * i], b0 = v.x[4 * i + 1], a1 = v.x[4 * i + 2], b1 = v.x[4 * i + 3];
      v.x[4 * i] = a0 * w.x - b0 * (sign * w.y);
      v.x[4 * i + 1] = b0 * w.x + a0 * (sign * w.y);
      v.x[4 * i + 2] = a1 * w.z - b1 * (sign * w.w);
      v.x[4 * i + 3] = b1 * w.z + a1 * (sign * w.w);
    }
  };
  if (turn0) one(x, c0);
  if (turn1 && c1 >= 0) one(y, c1);
}

// Token and row of this thread's group: the block's first row by a division, the thread's from there.
__device__ __forceinline__ bool thread_row(const RowsPlan& pl, int n_tok, int& t, int& h) {
  const uint32_t per_block = 256u >> pl.lg;
  const uint32_t first = blockIdx.x * per_block, t0 = first / pl.rows;
  const uint32_t n = first - t0 * pl.rows + (threadIdx.x >> pl.lg), dt = pl.magic ? __umulhi(n, pl.magic) : n;
  t = t0 + dt;
  h = n - dt * pl.rows;
  return t < n_tok;
}

template <class T>
__global__ __launch_bounds__(256) void rotary_rows_kernel(moe_rope r, RowsPlan pl, int n_tok, int D, Rows q, Rows k,
                                                          const int32_t* __restrict__ positions, float sign) {
  constexpr int N = Vec<T>::N;
  int t, h, c0, c1;
  bool turn0, turn1;
  if (!thread_row(pl, n_tok, t, h)) return;
  const int p = positions[t];
  if (p < 0 || p >= r.n_positions) return;
  row_pieces<T>(r, D, threadIdx.x & ((1 << pl.lg) - 1), c0, c1, turn0, turn1);
  if (c0 < 0) return;
  const bool is_q = h < q.heads;
  const Rows& m = is_q ? q : k;
  if (!is_q) h -= q.heads;
  const T* in = static_cast<const T*>(m.in) + t * m.in_t + h * m.in_h;
  T* out = static_cast<T*>(m.out) + t * m.out_t + h * m.out_h;
  Vec<T> x, y;
  x.load(in + c0 * N);
  if (c1 >= 0) y.load(in + c1 * N);
  turn_pieces<T>(r, r.table + static_cast<long long>(p) * r.rot_dim, sign, c0, c1, turn0, turn1, x, y);
  x.store(out + c0 * N);
  if (c1 >= 0) y.store(out + c1 * N);
}

// C: the cache's element. Rows of a token: q, then k, then v. 12289 tokens of 8 + 8 heads of 128: 25 us against 102 in
// the scalar form (4.3 TB/s); 8191 tokens to E4M3, whose row's largest magnitude takes a butterfly over its lanes, 15
// against 83 (3.4 TB/s); 256 tokens with 56 query heads 5 us, of 10 between calls (the host's part).
template <class T, class C>
__global__ __launch_bounds__(256) void append_rows_kernel(Cache ca, moe_rope r, RowsPlan pl, int n_tok, Rows k, Rows v, Rows q,
                                                          const int32_t* __restrict__ positions,
                                                          const int32_t* __restrict__ slots) {
  constexpr int N = Vec<T>::N;
  const int D = ca.D;
  int t, h, c0, c1;
  bool turn0, turn1;
  if (!thread_row(pl, n_tok, t, h)) return;       // whole groups of lanes leave
  const float* cs = nullptr;
  if (r.rot_dim > 0) {
    const int p = positions[t];
    if (p < 0 || p >= r.n_positions) return;
    cs = r.table + static_cast<long long>(p) * r.rot_dim;
  }
  const bool is_q = h < q.heads, is_k = !is_q && h < q.heads + k.heads;
  const Rows& m = is_q ? q : is_k ? k : v;
  h -= is_q ? 0 : is_k ? q.heads : q.heads + k.heads;
  const long long row = is_q ? 0 : slot_row(ca, slots[t], h);
  if (row < 0) return;
  row_pieces<T>(r, D, threadIdx.x & ((1 << pl.lg) - 1), c0, c1, turn0, turn1);
  const T* in = static_cast<const T*>(m.in) + t * m.in_t + h * m.in_h;
  Vec<T> x, y;
#pragma unroll
  for (int i = 0; i < N; ++i) x.x[i] = y.x[i] = 0.0f;
  if (c0 >= 0) x.load(in + c0 * N);
  if (c1 >= 0) y.load(in + c1 * N);
  if (c0 >= 0 && (is_q || is_k)) turn_pieces<T>(r, cs, 1.0f, c0, c1, turn0, turn1, x, y);
  if (sizeof(C) == 1 && !is_q) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) amax = fmaxf(amax, fmaxf(fabsf(x.x[i]), fabsf(y.x[i])));
    for (int o = 1; o < (1 << pl.lg); o <<= 1) amax = fmaxf(amax, __shfl_xor(amax, o, kWave));
    const float inv = row_factor(amax);
    uint8_t* out = static_cast<uint8_t*>(is_k ? ca.k : ca.v) + row * D;
    if (c0 >= 0) x.store_e4m3(out + c0 * N, inv);
    if (c1 >= 0) y.store_e4m3(out + c1 * N, inv);
    if (c0 == 0) (is_k ? ca.k_scale : ca.v_scale)[row] = amax > 0.0f ? amax / kE4M3Max : 1.0f;
    return;
  }
  T* out = is_q ? static_cast<T*>(m.out) + t * m.out_t + h * m.out_h : static_cast<T*>(is_k ? ca.k : ca.v) + row * D;
  if (c0 >= 0) x.store(out + c0 * N);
  if (c1 >= 0) y.store(out + c1 * N);
}

// Whether the rows form takes this call, and its plan.
static bool rows_plan(const moe_rope& r, int es, int T, int D, int rows, std::initializer_list<const Rows*> all, RowsPlan& pl) {
  const int N = 16 / es;
  if (D % N || (r.layout == MOE_ROPE_HALF ? r.rot_dim / 2 % N : r.rot_dim % N)) return false;
  if (r.rot_dim > 0 && reinterpret_cast<uintptr_t>(r.table) % 16) return false;
  for (const Rows* m : all) {
    if (m->heads == 0) continue;
    const uintptr_t a = reinterpret_cast<uintptr_t>(m->in) | reinterpret_cast<uintptr_t>(m->out);
    if (a % 16 || m->in_t % N || m->in_h % N || m->out_t % N || m->out_h % N) return false;
  }
  const int half = r.layout == MOE_ROPE_HALF ? r.rot_dim / 2 / N : 0;
  const int lanes = half + (D / N - 2 * half + 1) / 2;
  if (lanes > 64) return false;
  pl.lg = 0;
  while ((1 << pl.lg) < lanes) ++pl.lg;
  pl.rows = rows;
  pl.magic = rows > 1 ? static_cast<uint32_t>(((1ull << 32) + rows - 1) / rows) : 0;
  // n = at most rows + 255 times the magic number is exact for n * rows < 2^32; a launch has fewer than 2^32 threads
  const long long all_rows = static_cast<long long>(T) * rows;
  return rows <= 32768 && all_rows < (1LL << 31) && (all_rows << pl.lg) <= (1LL << 32) - 256;
}

hipError_t launch_rotary(const moe_rope& rope, moe_dtype act, int T, int D, const Rows& q, const Rows& k,
                         const int32_t* positions, float sign, hipStream_t st) {
  RowsPlan pl;
  const int rows = q.heads + k.heads;
  if (rows_plan(rope, act == MOE_BF16 ? 2 : 4, T, D, rows, {&q, &k}, pl)) {
    const dim3 grid(static_cast<unsigned>((static_cast<long long>(T) * rows + (256 >> pl.lg) - 1) / (256 >> pl.lg)));
    if (act == MOE_BF16)
      hipLaunchKernelGGL(rotary_rows_kernel<__bf16>, grid, dim3(256), 0, st, rope, pl, T, D, q, k, positions, sign);
    else
      hipLaunchKernelGGL(rotary_rows_kernel<float>, grid, dim3(256), 0, st, rope, pl, T, D, q, k, positions, sign);
    return hipGetLastError();
  }
  const dim3 grid(wave_blocks(static_cast<long long>(T) * rows)), block(256);
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
      const float inv = row_factor(amax);
      for (int c = lane; c < D; c += 64) y[c] = static_cast<C>(f32_to_e4m3(rotated<T>(rr, x, cs, c) * inv));
      if (lane == 0) (is_k ? ca.k_scale : ca.v_scale)[row] = amax > 0.0f ? amax / kE4M3Max : 1.0f;
    } else {
      for (int c = lane; c < D; c += 64) y[c] = from_f32<C>(rotated<T>(rr, x, cs, c));
    }
  }
}

hipError_t launch_kv_append(const Cache& c, const moe_rope& rope, moe_dtype act, int T, const Rows& k, const Rows& v,
                            const Rows& q, const int32_t* positions, const int32_t* slots, hipStream_t st) {
  const int rows = q.heads + k.heads + v.heads;
  const bool e4m3 = c.dtype == MOE_F8E4M3, bf16 = act == MOE_BF16;
  RowsPlan pl;
  if ((reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v)) % 16 == 0 &&
      rows_plan(rope, bf16 ? 2 : 4, T, c.D, rows, {&q, &k, &v}, pl)) {
    const dim3 grid(static_cast<unsigned>((static_cast<long long>(T) * rows + (256 >> pl.lg) - 1) / (256 >> pl.lg)));
    auto go = [&](auto kern) {
      hipLaunchKernelGGL(kern, grid, dim3(256), 0, st, c, rope, pl, T, k, v, q, positions, slots);
      return hipGetLastError();
    };
    if (bf16) return e4m3 ? go(append_rows_kernel<__bf16, uint8_t>) : go(append_rows_kernel<__bf16, __bf16>);
    return e4m3 ? go(append_rows_kernel<float, uint8_t>) : go(append_rows_kernel<float, float>);
  }
  const dim3 grid(wave_blocks(static_cast<long long>(T) * rows)), block(256);
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, grid, block, 0, st, c, rope, T, k, v, q, positions, slots);
    return hipGetLastError();
  };
  if (bf16) return e4m3 ? go(kv_append_kernel<__bf16, uint8_t>) : go(kv_append_kernel<__bf16, __bf16>);
  return e4m3 ? go(kv_append_kernel<float, uint8_t>) : go(kv_append_kernel<float, float>);
}

}  // namespace moe
