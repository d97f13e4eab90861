// Layer norm of rows and its gradient:
//   y = (x - mean) rstd w + b,   rstd = 1 / sqrt(mean((x - mean)^2) + eps),
//   dx = rstd (g - mean(g) - xhat mean(g xhat)) + d_residual,   g = dy w,  xhat = (x - mean) rstd,
//   dw = sum over rows of dy xhat,   db = sum over rows of dy.
//
// Bound by HBM: 8192 rows of 7168 bf16 channels take 44 us (5.3 TB/s), the gradient with a residual 98 us (4.8 TB/s); in fp32 91
// us, the gradient 136. Rows that lie on no 16 bytes are read an element at a time: 4093 fp32 rows of 1001 channels take 17 us in
// the gradient (2.9 TB/s, and 4 us of them the second launch), 2236 rows of 5263 in bf16 35 us (1.3 TB/s) and 140 in the gradient,
// in fp32 35 and 103: past 2048 such channels a thread has 32 pieces, of which the gradient spills 116 (fp32) or 170 (bf16)
// registers. The gradient of 4096 rows of 16384 fp32 channels, which spills 43, takes 247 us (3.3 TB/s).
//
// A row is read once and stays in the registers of the 16, 64, 256 or 512 threads that share it (the fewest that hold it in four
// pieces each; up to 32 numbers in the longest rows), so its mean comes before the sum of squares about it, and neither is a
// difference of large sums. The mean of d fp32 numbers is off by some of its last bits; the mean of (x - mean), which is exact for
// numbers near it, corrects that in y and in the variance.
//
// A block takes rows in steps of the grid, with w and b (and the column sums of the gradient) in registers: read
// from L2 for every row they would be four times the bytes of a bf16 row. The column sums of the blocks are joined by a second
// launch, in a fixed order.
#include <algorithm>

#include "heads.h"

namespace moe {
namespace {

template <class T_, int V_, int TPR_, int N_>
struct NormCfg {
  using T = T_;
  static constexpr int V = V_;        // elements of a piece (16 bytes, or one element)
  static constexpr int TPR = TPR_;    // threads of a row
  static constexpr int N = N_;        // pieces of a thread
  static constexpr int NT = TPR < 256 ? 256 : TPR;
  static constexpr int RPB = NT / TPR;
  // The gradient's next row is on its way while one is worked on, where 512 registers a wave allow that.
  static constexpr bool AHEAD = NT <= 256;
};

template <class T, int V>
__device__ __forceinline__ void load_piece(const T* p, float (&x)[V]) {
  if constexpr (V == 1) {
    x[0] = to_f32(*p);
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        x[i] = __uint_as_float(w[i]);
      } else {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  }
}
template <class T, int V>
__device__ __forceinline__ void store_piece(T* p, const float (&x)[V]) {
  if constexpr (V == 1) {
    *p = from_f32<T>(x[0]);
  } else {
    union {
      T e[V];
      uint4 u;
    } y;
#pragma unroll
    for (int i = 0; i < V; ++i) y.e[i] = from_f32<T>(x[i]);
    *reinterpret_cast<uint4*>(p) = y.u;
  }
}
template <int V>
__device__ __forceinline__ void load_vector(const float* p, float (&x)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += V < 4 ? 1 : 4) {
    if constexpr (V == 1) {
      x[0] = p[0];
    } else {
      const f32x4 y = *reinterpret_cast<const f32x4*>(p + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[i + e] = y[e];
    }
  }
}

// Sums of two numbers over the threads of a row. `at`: LDS for this call alone until the next barrier but one.
template <class C>
__device__ __forceinline__ float2 row_sums(float a, float b, float2* at) {
#pragma unroll
  for (int o = (C::TPR < 64 ? C::TPR : 64) / 2; o > 0; o >>= 1) {
    a += __shfl_xor(a, o, kWave);
    b += __shfl_xor(b, o, kWave);
  }
  if constexpr (C::TPR > 64) {
    constexpr int W = C::TPR / 64;
    if ((threadIdx.x & 63) == 0) at[threadIdx.x >> 6] = float2{a, b};
    __syncthreads();
    a = b = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2 x = at[w];
      a += x.x;
      b += x.y;
    }
  }
  return float2{a, b};
}

// A row's pieces as they lie in memory (fp32 copies would take twice the registers while they are on their way).
template <class C>
struct RawRow {
  typedef typename std::conditional<C::V == 1, typename C::T, uint4>::type P;
  P p[C::N];
  __device__ __forceinline__ void load(const typename C::T* row, int pieces, int t) {
#pragma unroll
    for (int n = 0; n < C::N; ++n) {
      const int c = n * C::TPR + t;
      if (c < pieces) p[n] = *reinterpret_cast<const P*>(row + static_cast<long long>(c) * C::V);
    }
  }
  __device__ __forceinline__ void get(int n, float (&x)[C::V]) const {
    load_piece<typename C::T, C::V>(reinterpret_cast<const typename C::T*>(&p[n]), x);
  }
};

}  // namespace

template <class C>
__global__ __launch_bounds__(C::NT) void norm_kernel(NormArgs a) {
  using T = typename C::T;
  constexpr int V = C::V, N = C::N;
  __shared__ float2 sums[2][2][8];
  const int t = threadIdx.x % C::TPR, pieces = a.d / V;
  const float inv = 1.0f / a.d;
  float w[N][V], b[N][V];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int c = n * C::TPR + t;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      w[n][e] = 1.0f;
      b[n][e] = 0.0f;
    }
    if (c < pieces) {
      if (a.weight) load_vector<V>(a.weight + c * V, w[n]);
      if (a.bias) load_vector<V>(a.bias + c * V, b[n]);
    }
  }
  const long long step = static_cast<long long>(gridDim.x) * C::RPB;
  long long r = static_cast<long long>(blockIdx.x) * C::RPB + threadIdx.x / C::TPR;
  RawRow<C> next;
  if (r < a.rows) next.load(static_cast<const T*>(a.x) + r * a.x_stride, pieces, t);
  // the waves of a row agree on r: with more than one wave a block has one row
  for (int k = 0; r < a.rows; r += step, k ^= 1) {
    const RawRow<C> raw = next;
    if (r + step < a.rows) next.load(static_cast<const T*>(a.x) + (r + step) * a.x_stride, pieces, t);
    float x[N][V], sum = 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if (n * C::TPR + t < pieces) {
        raw.get(n, x[n]);
#pragma unroll
        for (int e = 0; e < V; ++e) sum += x[n][e];
      }
    }
    const float mean = row_sums<C>(sum, 0.0f, sums[k][0]).x * inv;
    float off = 0.0f, sq = 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (n * C::TPR + t < pieces) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          x[n][e] -= mean;
          off += x[n][e];
          sq = fmaf(x[n][e], x[n][e], sq);
        }
      }
    const float2 s = row_sums<C>(off, sq, sums[k][1]);
    const float fix = s.x * inv, square = s.y * inv - fix * fix, var = square < 0.0f ? 0.0f : square;
    const float rstd = 1.0f / sqrtf(var + a.eps);
    if (t == 0) {
      if (a.mean) a.mean[r] = mean + fix;
      if (a.rstd) a.rstd[r] = rstd;
    }
    T* y = static_cast<T*>(a.y) + r * a.y_stride;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int c = n * C::TPR + t;
      if (c >= pieces) continue;
      float o[V];
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = fmaf((x[n][e] - fix) * rstd, w[n][e], b[n][e]);
      store_piece<T, V>(y + static_cast<long long>(c) * V, o);
    }
  }
}

// sums: [blocks][2][d], or the results themselves if there is one block.
template <class C>
__global__ __launch_bounds__(C::NT) void norm_backward_kernel(NormBackwardArgs a, float* dw_part, float* db_part,
                                                              long long part_stride) {
  using T = typename C::T;
  constexpr int V = C::V, N = C::N;
  __shared__ float2 sums[2][8];
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int t = threadIdx.x % C::TPR, pieces = a.d / V;
  const float inv = 1.0f / a.d;
  float w[N][V], dw[N][V], db[N][V];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int c = n * C::TPR + t;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      w[n][e] = 1.0f;
      dw[n][e] = db[n][e] = 0.0f;
    }
    if (a.weight && c < pieces) load_vector<V>(a.weight + c * V, w[n]);
  }
  const long long step = static_cast<long long>(gridDim.x) * C::RPB;
  long long r = static_cast<long long>(blockIdx.x) * C::RPB + threadIdx.x / C::TPR;
  RawRow<C> nx, ny, nr;
  float nmean = 0.0f, nrstd = 0.0f;
  auto load = [&](long long row) {
    nx.load(static_cast<const T*>(a.x) + row * a.x_stride, pieces, t);
    ny.load(static_cast<const T*>(a.dy) + row * a.dy_stride, pieces, t);
    if (a.d_residual) nr.load(static_cast<const T*>(a.d_residual) + row * a.dr_stride, pieces, t);
    nmean = a.mean[row];
    nrstd = a.rstd[row];
  };
  if (C::AHEAD && r < a.rows) load(r);
  for (int k = 0; r < a.rows; r += step, k ^= 1) {
    if (!C::AHEAD) load(r);
    const RawRow<C> rx = nx, ry = ny, rr = nr;
    const float mean = nmean, rstd = nrstd;
    if (C::AHEAD && r + step < a.rows) load(r + step);
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (n * C::TPR + t < pieces) {
        float x[V], y[V];
        rx.get(n, x);
        ry.get(n, y);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float h = (x[e] - mean) * rstd, g = y[e] * w[n][e];
          dw[n][e] = fmaf(y[e], h, dw[n][e]);
          db[n][e] += y[e];
          s0 += g;
          s1 = fmaf(g, h, s1);
        }
      }
    const float2 s = row_sums<C>(s0, s1, sums[k]);
    const float m0 = s.x * inv, m1 = s.y * inv;
    T* dx = static_cast<T*>(a.dx) + r * a.dx_stride;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int c = n * C::TPR + t;
      if (c >= pieces) continue;
      float x[V], y[V], z[V], o[V];
      rx.get(n, x);
      ry.get(n, y);
      if (a.d_residual) rr.get(n, z);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float h = (x[e] - mean) * rstd;
        o[e] = rstd * (fmaf(y[e], w[n][e], -m0) - h * m1);
        if (a.d_residual) o[e] += z[e];
      }
      store_piece<T, V>(dx + static_cast<long long>(c) * V, o);
    }
  }
  if (!dw_part && !db_part) return;
  if constexpr (C::RPB > 1) {      // the rows of a wave, then the block's waves one after the other
    constexpr int W = C::NT / 64;
    if constexpr (C::TPR < 64) {
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < V; ++e)
#pragma unroll
          for (int o = C::TPR; o < 64; o <<= 1) {
            dw[n][e] += __shfl_xor(dw[n][e], o, kWave);
            db[n][e] += __shfl_xor(db[n][e], o, kWave);
          }
    }
    float* const both = reinterpret_cast<float*>(lds);
#pragma unroll 1
    for (int q = 0; q < W; ++q) {
      __syncthreads();
      if (threadIdx.x / 64 != q || (threadIdx.x & 63) >= C::TPR) continue;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int c = n * C::TPR + t;
        if (c >= pieces) continue;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float* p = both + 2 * (c * V + e);
          if (q > 0) {
            dw[n][e] += p[0];
            db[n][e] += p[1];
          }
          p[0] = dw[n][e];
          p[1] = db[n][e];
        }
      }
    }
    if (threadIdx.x / 64 != W - 1 || (threadIdx.x & 63) >= C::TPR) return;
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int c = n * C::TPR + t;
    if (c >= pieces) continue;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const long long at = blockIdx.x * part_stride + c * V + e;
      if (dw_part) dw_part[at] = dw[n][e];
      if (db_part) db_part[at] = db[n][e];
    }
  }
}

// out[c] = sum over parts of part[p][c], in order within 16 interleaved runs, then over the runs.
__global__ __launch_bounds__(1024) void norm_join_kernel(const float* dw_part, const float* db_part, int parts, int d,
                                                         float* dw, float* db) {
  __shared__ float run[16][64];
  const int c = blockIdx.x * 64 + (threadIdx.x & 63), s = threadIdx.x >> 6;
  const float* in = blockIdx.y ? db_part : dw_part;
  float* out = blockIdx.y ? db : dw;
  if (!out) return;
  float sum = 0.0f;
  if (c < d) {
#pragma unroll 4
    for (int p = s; p < parts; p += 16) sum += in[static_cast<long long>(p) * 2 * d + c];
  }
  run[s][threadIdx.x & 63] = sum;
  __syncthreads();
  if (s || c >= d) return;
  sum = 0.0f;
#pragma unroll
  for (int q = 0; q < 16; ++q) sum += run[q][threadIdx.x];
  out[c] = sum;
}

namespace {

// wide: every row and vector on 16 bytes, d in whole pieces.
template <class F>
auto with_norm(moe_dtype act, int d, bool wide, F f) {
  auto by_size = [&](auto zero, auto width) {
    using T = decltype(zero);
    constexpr int V = decltype(width)::value;
    if (d <= 16 * 4 * V) return f(NormCfg<T, V, 16, 4>{});
    if (d <= 64 * 4 * V) return f(NormCfg<T, V, 64, 4>{});
    if (d <= 256 * 4 * V) return f(NormCfg<T, V, 256, 4>{});
    if constexpr (V < 8) {
      if (d > 512 * 4 * V) return f(NormCfg<T, V, 512, 32 / V>{});
    }
    return f(NormCfg<T, V, 512, 4>{});
  };
  using W1 = std::integral_constant<int, 1>;
  if (act == MOE_F32) return wide ? by_size(0.0f, std::integral_constant<int, 4>{}) : by_size(0.0f, W1{});
  return wide ? by_size(__bf16{}, std::integral_constant<int, 8>{}) : by_size(__bf16{}, W1{});
}

bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

// Blocks of the gradient, each of which leaves column sums: one for each CU (8192 rows of 7168 bf16 channels: 100 us, with two 113,
// which write and join twice the sums; 32768 of 2048: 108 and 119). Rows read an element at a time have too little on their way for
// that and take two (4093 rows of 1001 fp32 channels: 22 us with one, 18 with two).
constexpr int kNormParts = 256;

template <class C>
static int norm_parts(long long rows) {
  return static_cast<int>(std::min<long long>((rows + C::RPB - 1) / C::RPB, C::V == 1 ? 2 * kNormParts : kNormParts));
}

size_t norm_backward_ws_bytes(long long rows, int d) {
  return static_cast<size_t>(std::min<long long>(rows, 2 * kNormParts)) * 2 * d * sizeof(float);
}

hipError_t launch_norm(const NormArgs& a, moe_dtype act, hipStream_t st) {
  const int es = act == MOE_F32 ? 4 : 2;
  const bool wide = a.d * es % 16 == 0 && on16(a.x) && on16(a.y) && on16(a.weight) && on16(a.bias) &&
                    a.x_stride * es % 16 == 0 && a.y_stride * es % 16 == 0;
  return with_norm(act, a.d, wide, [&](auto cfg) {
    using C = decltype(cfg);
    // two blocks for each CU (8192 rows of 7168 bf16 channels: 46 us; with one 65, with four 53, with eight 50: each reads w and
    // b), or four that read an element at a time (4093 rows of 1001 fp32 channels: 13.2 us with two, 10.5 with four)
    const long long blocks = std::min<long long>((a.rows + C::RPB - 1) / C::RPB, device_cu_count() * (C::V == 1 ? 4LL : 2LL));
    hipLaunchKernelGGL(norm_kernel<C>, dim3(static_cast<unsigned>(blocks)), dim3(C::NT), 0, st, a);
    return hipGetLastError();
  });
}

hipError_t launch_norm_backward(const NormBackwardArgs& a, moe_dtype act, float* ws, hipStream_t st) {
  const int es = act == MOE_F32 ? 4 : 2;
  const bool wide = a.d * es % 16 == 0 && on16(a.x) && on16(a.dy) && on16(a.d_residual) && on16(a.dx) && on16(a.weight) &&
                    a.x_stride * es % 16 == 0 && a.dy_stride * es % 16 == 0 && a.dr_stride * es % 16 == 0 &&
                    a.dx_stride * es % 16 == 0;
  const bool columns = a.dweight || a.dbias;
  int parts = 0;
  if (a.rows > 0) {
    const hipError_t e = with_norm(act, a.d, wide, [&](auto cfg) {
      using C = decltype(cfg);
      parts = norm_parts<C>(a.rows);
      const bool direct = parts == 1 || !columns;
      float* dw = direct ? a.dweight : ws;
      float* db = direct ? a.dbias : ws + a.d;
      const int lds = C::RPB > 1 && columns ? a.d * 8 : 0;
      hipLaunchKernelGGL(norm_backward_kernel<C>, dim3(parts), dim3(C::NT), lds, st, a, dw, db, 2LL * a.d);
      return hipGetLastError();
    });
    if (e != hipSuccess || parts == 1) return e;
  }
  if (!columns) return hipSuccess;
  hipLaunchKernelGGL(norm_join_kernel, dim3((a.d + 63) / 64, 2), dim3(1024), 0, st, ws, ws + a.d, parts, a.d, a.dweight,
                     a.dbias);
  return hipGetLastError();
}

}  // namespace moe
