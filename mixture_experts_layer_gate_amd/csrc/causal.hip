// Causal attention of packed sequences:
//   o_i = sum_j exp(s_ij - m) v_j / sum_j exp(s_ij - m),  s_ij = scale q_i . k_j,  start(i) <= j <= i,
// in one pass over the keys with a running reference m, sums in fp32.
//
// A block takes 128 rows of one query head, a wave 32 of them; keys and values come to LDS in stages that the waves share, the
// next one on its way while one is worked on. Rows are tiled by their place in the buffer, whatever sequences they belong to: a
// tile's keys begin where its first row's sequence does, so short sequences share tiles. Few rows: 32 of them to a block, whose
// waves share out the keys.
//
// Bound by the matrix units beside the vector instructions of the softmax, which two waves a SIMD overlap: 8192 tokens of 56
// heads of 128 channels on 8 take 1035 us in bf16, 929 TFLOP/s (4 D operations for each pair) with the units 0.42 busy; 12
// sequences of up to 4000 tokens, 24833 in all, of 16 heads on 4 take 387 us, 688 TFLOP/s: masked tiles, and the last blocks
// alone. With 64 channels a score's vector work is twice as much beside its products: 6 sequences of 2975 to 5950 tokens of 10
// heads take 271 us, 580 TFLOP/s.
// Queries, and not keys, stay in registers, beside the sums that belong to them: 32 rows' queries and sums take 32 + 64 of a
// lane's registers in bf16 with 128 channels.
#include "packed.h"

namespace moe {

namespace {

template <class C>
struct CausalKernel {
  static constexpr int EU = C::F32 ? (C::DP <= 64 ? 2 : 1) : (C::DP <= 64 ? 4 : 2);   // waves of a SIMD
  static constexpr int LDS = 4 * C::STAGE;
  using Split = SplitCfg<C>;
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

// One row over the keys it sees alone, 64 at a time: a lane a key for the scores, a lane a channel for the sums. Its result is
// stored here first: it may lie where q does.
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

// SPLIT: a block takes 32 rows, its waves every fourth tile of their keys.
template <class C, bool SPLIT>
__global__ __launch_bounds__(C::NT, SPLIT ? 1 : CausalKernel<C>::EU) void causal_kernel(PackedArgs a, PackedGrid grid) {
  using E = typename C::E;
  using S = typename CausalKernel<C>::Split;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  __shared__ int ends[2][C::NW];
  int head, rank;
  if (!grid.item(blockIdx.x, head, rank)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tile = grid.tiles - 1 - rank, row0 = SPLIT ? tile * 32 : tile * C::ROWS + wave * 32, row = row0 + (lane & 31);
  EarlyRows<C> q;
  q.begin(static_cast<const E*>(a.q.in) + head * a.q.in_h, a.q.in_t, row0, a.T, a.D, a.wide & 1);
  const int end = packed_end(a.seq_start, a.n_seqs, a.T);
  const Span span = find_span(a.seq_start, a.n_seqs, a.T, end, row0, row);
  const bool live = span.live;
  const WaveSpan ws(live);
  const int lo = ws.last < 0 ? INT_MAX : ws.of_first(span.start), hi = ws.last < 0 ? -1 : row0 + ws.last;
  const int whole_from = ws.of_last(span.start), whole_to = row0 + ws.first;
  int first = lo, last = hi;
  if (!SPLIT) block_range<C>(lo, hi, ends, first, last);
  if (last < 0) return;
  const int kv = head / (a.q.heads / a.k.heads);
  const RowLoader<C> ks(a.k.in, a.k.in_t, a.k.in_h, kv, end, a.D, a.direct & 1);
  const RowLoader<C> vs(a.v.in, a.v.in_t, a.v.in_h, kv, end, a.D, a.direct & 2);
  const TileLanes lanes;
  Quad qf[C::NF];
  const float c = a.scale * kLog2e;
  RowSums<C> st;
  clear_sums(st.o);
  st.m = -INFINITY;
  st.l = 0.0f;
  auto turn = [&](const char* k, const char* v, int j) {
    tile_turn<C>(st, qf, k, v, lanes, c, j >= whole_from && j + 31 <= whole_to,
                 tokens_below(row + 1, j) & ~tokens_below(span.start, j));
  };
  if constexpr (SPLIT) {
    char* const own = lds + wave * S::OWN;
    auto issue = [&](char* to, int j) {
      ks.issue_tile(to, j);
      vs.issue_tile(to + C::TILE, j);
    };
    const int j = first + 32 * wave;
    if (S::SLOTS == 2 && j <= last) issue(own, j);
    char* const other = own + (S::SLOTS - 1) * S::SLOT;
    q.end(other, lanes, live, qf);
    wave_tiles<C, S>(own, j, last, (a.direct & 3) == 3, issue, [&](const char* at, int i) { turn(at, at + C::TILE, i); });
    // the four waves' sums, relative to the largest of their references
    __shared__ float2 ml[4][32];
    __shared__ uint32_t bad[4];
    const float l = halves_sum(st.l);
    if (lane < 32) ml[wave][lane] = float2{st.m, l};
    if (lane == 0) bad[wave] = 0;
    __syncthreads();
    float m = -INFINITY, total = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) m = nan_max(m, ml[w][lane & 31].x);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float2 x = ml[w][lane & 31];
      total += x.x == -INFINITY ? x.y : x.y * __builtin_amdgcn_exp2f(x.x - m);      // the former: 0, or NaN
    }
    if (live && a.lse_out && wave == 0 && lane < 32)
      a.lse_out[static_cast<long long>(row) * a.q.heads + head] =
          total == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(total)) * kLn2;
    const float inv = total == 0.0f ? 0.0f : 1.0f / total;
    // a row that sees a NaN score is NaN throughout, and right as it is
    join_waves<S::OWN>(lds, st.o, st.m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(st.m - m), live && total == total, bad,
                       [&](int i, const f32x16 (&x)[1]) {
                         const uint32_t done = ws.b & ~(bad[0] | bad[1] | bad[2] | bad[3]);
                         store_rows<C>(lds + wave * C::TILE, static_cast<E*>(a.q.out) + head * a.q.out_h, a.q.out_t, row0, a.D, x,
                                       inv, done, a.wide & 2, i);
                       });
    stage_barrier();
    uint32_t again = bad[0] | bad[1] | bad[2] | bad[3];
#pragma unroll 1
    for (; again; again &= again - 1) {
      const int t = __builtin_ctz(again);
      if ((t & 3) == wave) row_alone<C>(a, head, kv, row0 + t, __builtin_amdgcn_readlane(span.start, t));
    }
  } else {
    // two waves' tiles fit beside the first stage, or four
    constexpr bool BESIDE = C::NS == 2;
    auto issue = [&](char* to, int j) {
      ks.issue(to, j);
      vs.issue(to + C::STAGE, j);
    };
    if (BESIDE) issue(lds, first);
    char* const own = lds + (BESIDE ? 2 * C::STAGE : 0) + wave * C::TILE;
    q.end(own, lanes, live, qf);
    if (!BESIDE) {
      __syncthreads();
      issue(lds, first);
    }
    int at = 0;
    for (int j = first; j <= last; j += C::KT, at ^= 1) {
      stage_barrier();
      const char* k = lds + at * 2 * C::STAGE;
      if (j + C::KT <= last) issue(lds + (at ^ 1) * 2 * C::STAGE, j + C::KT);
#pragma unroll
      for (int t = 0; t < C::NS; ++t)
        if (j + 32 * t <= hi && j + 32 * t + 31 >= lo) turn(k + t * C::TILE, k + t * C::TILE + C::STAGE, j + 32 * t);
    }
    const float l = halves_sum(st.l);
    if (live && a.lse_out && lane < 32)
      a.lse_out[static_cast<long long>(row) * a.q.heads + head] =
          l == 0.0f ? -INFINITY : (st.m + __builtin_amdgcn_logf(l)) * kLn2;
    // a row that sees a NaN score is NaN throughout, and right as it is
    uint32_t again = tokens_not_finite(st.o, live && l == l);
    __syncthreads();      // the stages are read
    store_rows<C>(lds + wave * C::TILE, static_cast<E*>(a.q.out) + head * a.q.out_h, a.q.out_t, row0, a.D, st.o,
                  l == 0.0f ? 0.0f : 1.0f / l, ws.b & ~again, a.wide & 2);
#pragma unroll 1
    for (; again; again &= again - 1) {
      const int t = __builtin_ctz(again);
      row_alone<C>(a, head, kv, row0 + t, __builtin_amdgcn_readlane(span.start, t));
    }
  }
}

hipError_t launch_causal(const PackedArgs& args, moe_dtype act, hipStream_t st) {
  return with_packed_cfg(act, args.D, [&](auto cfg) {
    using C = decltype(cfg);
    using S = typename CausalKernel<C>::Split;
    PackedArgs a = args;
    a.direct = loads_direct(a.k.in, a.k.in_t, a.k.in_h, C::ES) | loads_direct(a.v.in, a.v.in_t, a.v.in_h, C::ES) << 1;
    a.wide = aligned16(a.q.in, a.q.in_t, a.q.in_h, C::ES) | aligned16(a.q.out, a.q.out_t, a.q.out_h, C::ES) << 1;
    auto go = [&](auto split) {
      constexpr bool SPLIT = decltype(split)::value;
      constexpr int LDS = SPLIT ? 4 * S::OWN : CausalKernel<C>::LDS, ROWS = SPLIT ? 32 : C::ROWS;
      static const hipError_t allowed = hipFuncSetAttribute(reinterpret_cast<const void*>(causal_kernel<C, SPLIT>),
                                                            hipFuncAttributeMaxDynamicSharedMemorySize, LDS);
      if (allowed != hipSuccess) return allowed;
      const PackedGrid grid = PackedGrid::of(a.q.heads, (a.T + ROWS - 1) / ROWS);
      hipLaunchKernelGGL((causal_kernel<C, SPLIT>), dim3(grid.blocks), dim3(C::NT), LDS, st, a, grid);
      return hipGetLastError();
    };
    if constexpr (S::FITS) {
      if (split_rows(a.T, a.n_seqs, a.q.heads, a.D, C::F32)) return go(std::true_type{});
    }
    return go(std::false_type{});
  });
}

}  // namespace moe
