// Causal attention of packed sequences:
//   o_i = sum_j exp(s_ij - m) v_j / sum_j exp(s_ij - m),  s_ij = scale q_i . k_j,  start(i) <= j <= i,
// in one pass over the keys with a running reference m, sums in fp32.
//
// A block takes 128 rows of one query head, a wave 32 of them; keys and values come to LDS in stages that the waves share, the
// next one on its way while one is worked on. Rows are tiled by their place in the buffer, whatever sequences they belong to: a
// tile's keys begin where its first row's sequence does, so short sequences share tiles.
#include "packed.h"

namespace moe {

namespace {

template <class C>
struct CausalKernel {
  static constexpr int EU = C::F32 ? (C::DP <= 64 ? 2 : 1) : (C::DP <= 128 ? 2 : 1);   // waves of a SIMD
  static constexpr int LDS = 4 * C::STAGE;
};

// A row's reference is moved (and its sums rescaled) when the weights of a half wave's 16 tokens add up to more than this: that
// shows in a sum that is needed anyway, and spares the maximum of every tile. Weights and sums are relative to m, so the result
// does not depend on m; 2^30 tokens weigh at most 2^38, and values up to 2^88 cannot overflow their sums.
constexpr float kHighSum = 0x1p12f;

template <class C>
struct RowSums {
  f32x16 o[C::NB];
  float m, l;      // reference (base 2), this half wave's part of the sum
};

template <class C>
__device__ __forceinline__ void raise(RowSums<C>& st, float m) {
  const float f = m == st.m ? 1.0f : __builtin_amdgcn_exp2f(st.m - m);
  st.m = m;
  st.l *= f;
#pragma unroll
  for (int i = 0; i < C::NB; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) st.o[i][e] *= f;
}

// A tile of 32 keys; whole: every row of the wave sees all of them, else `seen`.
template <class C>
__device__ __forceinline__ void tile_turn(RowSums<C>& st, const Quad (&qf)[C::NF], const char* k, const char* v,
                                          const TileLanes& at, float c, bool whole, uint32_t seen) {
  f32x16 s;
#pragma unroll
  for (int e = 0; e < 16; ++e) s[e] = 0.0f;
  s = tile_products<C>(k, at, qf, s);
  float p[16];
  auto weigh = [&](float m) {
#pragma unroll
    for (int e = 0; e < 16; ++e) p[e] = __builtin_amdgcn_exp2f(fmaf(s[e], c, -m));
    if (!whole) mask_weights(p, seen);
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 16; ++e) sum[e & 3] += p[e];
    return (sum[0] + sum[1]) + (sum[2] + sum[3]);
  };
  float sum = weigh(st.m);
  const bool high = !(halves_max(sum) <= kHighSum);      // NaN too: the reference was -infinity
  if (__any(high)) {
    float m = -INFINITY;
#pragma unroll
    for (int e = 0; e < 16; ++e) m = nan_max(m, whole || ((seen >> lds_token(e)) & 1) ? s[e] * c : -INFINITY);
    m = halves_max(m);
    raise<C>(st, high && m > st.m ? m : st.m);
    const float again = weigh(st.m == -INFINITY ? 0.0f : st.m);
    sum = high ? again : sum;
  }
  st.l += sum;
  Weights<C> w;
#pragma unroll
  for (int e = 0; e < 16; ++e) w.set(e, p[e]);
  add_columns<C>(v, at, w, st.o);
}

// One row over the keys it sees alone, 64 at a time: a lane a key for the scores, a lane a channel for the sums.
template <class C>
__device__ __forceinline__ void row_alone(const PackedArgs& a, int head, int kv, int row, int start) {
  using E = typename C::E;
  constexpr int NC = (C::DP + 63) / 64;
  const int lane = threadIdx.x & 63, D = a.D;
  const float c = a.scale * kLog2e;
  const E* q = static_cast<const E*>(a.q.in) + row * a.q.in_t + head * a.q.in_h;
  const E* k = static_cast<const E*>(a.k.in) + kv * a.k.in_h;
  const E* v = static_cast<const E*>(a.v.in) + kv * a.v.in_h;
  float m = -INFINITY, l = 0.0f, o[NC] = {};
#pragma unroll 1
  for (int j = start; j <= row; j += 64) {
    const int n = min(64, row + 1 - j);
    const float s = lane < n ? row_dot<E>(q, k + (j + lane) * a.k.in_t, D) * c : -INFINITY;
    float mj = s;
#pragma unroll
    for (int w = 32; w > 0; w >>= 1) mj = nan_max(mj, __shfl_xor(mj, w, kWave));
    const float mn = nan_max(m, mj), f = mn == m ? 1.0f : __builtin_amdgcn_exp2f(m - mn);
    m = mn;
    const float p = lane < n ? __builtin_amdgcn_exp2f(s - (m == -INFINITY ? 0.0f : m)) : 0.0f;
    l = l * f + p;
#pragma unroll
    for (int i = 0; i < NC; ++i) o[i] *= f;
    add_rows_alone<C, NC>(v + j * a.v.in_t, a.v.in_t, n, D, p, o);
  }
#pragma unroll
  for (int w = 32; w > 0; w >>= 1) l += __shfl_xor(l, w, kWave);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  E* out = static_cast<E*>(a.q.out) + row * a.q.out_t + head * a.q.out_h;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int ch = 64 * i + lane;
    if (ch < D) out[ch] = from_f32<E>(l == 0.0f ? 0.0f : o[i] * inv);
  }
  if (a.lse_out && lane == 0)
    a.lse_out[static_cast<long long>(row) * a.q.heads + head] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2;
}

}  // namespace

template <class C>
__global__ __launch_bounds__(C::NT, CausalKernel<C>::EU) void causal_kernel(PackedArgs a, PackedGrid grid) {
  using E = typename C::E;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  __shared__ int ends[2][C::NW];
  int head, rank;
  if (!grid.item(blockIdx.x, head, rank)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row0 = (grid.tiles - 1 - rank) * C::ROWS + wave * 32, row = row0 + (lane & 31);
  const Span span = find_span(a.seq_start, a.n_seqs, a.T, row0, row);
  const bool live = span.live;
  const WaveSpan ws(live);
  const int lo = ws.last < 0 ? INT_MAX : ws.of_first(span.start), hi = ws.last < 0 ? -1 : row0 + ws.last;
  const int whole_from = ws.of_last(span.start), whole_to = row0 + ws.first;
  int first, last;
  block_range<C>(lo, hi, ends, first, last);
  if (last < 0) return;
  const int kv = head / (a.q.heads / a.k.heads);
  const RowLoader<C> ks(a.k.in, a.k.in_t, a.k.in_h, kv, a.T, a.D, a.direct & 1);
  const RowLoader<C> vs(a.v.in, a.v.in_t, a.v.in_h, kv, a.T, a.D, a.direct & 2);
  const TileLanes lanes;
  // two waves' tiles fit beside the first stage, or four
  constexpr bool BESIDE = C::NS == 2;
  auto stage0 = [&] {
    ks.issue(lds, first);
    vs.issue(lds + C::STAGE, first);
  };
  if (BESIDE) stage0();
  char* const own = lds + (BESIDE ? 2 * C::STAGE : 0) + wave * C::TILE;
  Quad qf[C::NF];
  {
    const E* q = static_cast<const E*>(a.q.in) + head * a.q.in_h;
    if constexpr (BESIDE) {
      WaveRows<C> rows;
      rows.load(q, a.q.in_t, row0, a.T, a.D, a.wide & 1);
      rows.give(own, lanes, a.D, live, qf);
    } else {
      WaveRows<C>::bring(own, q, a.q.in_t, row0, a.T, a.D, a.wide & 1);
      WaveRows<C>::pick(own, lanes, live, qf);
    }
  }
  if (!BESIDE) {
    __syncthreads();
    stage0();
  }
  const float c = a.scale * kLog2e;
  RowSums<C> st;
  clear_sums(st.o);
  st.m = -INFINITY;
  st.l = 0.0f;
  int at = 0;
  for (int j = first; j <= last; j += C::KT, at ^= 1) {
    stage_barrier();
    const char* k = lds + at * 2 * C::STAGE;
    if (j + C::KT <= last) {
      char* next = lds + (at ^ 1) * 2 * C::STAGE;
      ks.issue(next, j + C::KT);
      vs.issue(next + C::STAGE, j + C::KT);
    }
#pragma unroll
    for (int t = 0; t < C::NS; ++t) {
      const int jt = j + 32 * t;
      if (jt > hi || jt + 31 < lo) continue;
      const char *kt = k + t * C::TILE, *vt = kt + C::STAGE;
      tile_turn<C>(st, qf, kt, vt, lanes, c, jt >= whole_from && jt + 31 <= whole_to,
                   tokens_below(row + 1, jt) & ~tokens_below(span.start, jt));
    }
  }
  const float l = halves_sum(st.l);
  if (live && a.lse_out && lane < 32)
    a.lse_out[static_cast<long long>(row) * a.q.heads + head] = l == 0.0f ? -INFINITY : (st.m + __builtin_amdgcn_logf(l)) * kLn2;
  __syncthreads();      // the stages are read
  store_rows<C>(lds + wave * C::TILE, static_cast<E*>(a.q.out) + head * a.q.out_h, a.q.out_t, row0, a.D, st.o,
                l == 0.0f ? 0.0f : 1.0f / l, ws.b, a.wide & 2);
  uint32_t again = tokens_not_finite(st.o, live) ;
#pragma unroll 1
  while (again) {
    const int t = __builtin_ctz(again);
    again &= again - 1;
    row_alone<C>(a, head, kv, row0 + t, __builtin_amdgcn_readlane(span.start, t));
  }
}

hipError_t launch_causal(const PackedArgs& args, moe_dtype act, hipStream_t st) {
  return with_packed_cfg(act, args.D, [&](auto cfg) {
    using C = decltype(cfg);
    PackedArgs a = args;
    a.direct = loads_direct(a.k.in, a.k.in_t, a.k.in_h, C::ES) | loads_direct(a.v.in, a.v.in_t, a.v.in_h, C::ES) << 1;
    a.wide = aligned16(a.q.in, a.q.in_t, a.q.in_h, C::ES) | aligned16(a.q.out, a.q.out_t, a.q.out_h, C::ES) << 1;
    constexpr int LDS = CausalKernel<C>::LDS;
    static const hipError_t allowed = hipFuncSetAttribute(reinterpret_cast<const void*>(causal_kernel<C>),
                                                          hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
    if (allowed != hipSuccess) return allowed;
    const PackedGrid grid = PackedGrid::of(a.q.heads, (a.T + C::ROWS - 1) / C::ROWS);
    hipLaunchKernelGGL(causal_kernel<C>, dim3(grid.blocks), dim3(C::NT), LDS, st, a, grid);
    return hipGetLastError();
  });
}

}  // namespace moe
