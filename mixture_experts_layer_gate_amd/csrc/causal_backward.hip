// The gradient of causal attention of packed sequences. With p_ij = exp(s_ij - lse_i) and g = d_out,
//   delta_i = g_i . o_i,   t_ij = p_ij (g_i . v_j - delta_i),
//   dq_i = scale sum_j t_ij k_j,   dk_j = scale sum_i t_ij q_i,   dv_j = sum_i p_ij g_i,
// the latter two over the query heads of the group as well. p and t are computed again from q, k, v and lse, in fp32, and
// rounded to bf16 for the products that sum them (with bf16 inputs), as their operand has to be.
//
// Two launches, each with a fixed order of its sums (no atomics): the first takes rows of queries, as the forward pass does,
// and leaves dq, and lse and delta by heads for the second; that takes rows of keys. Both compute s and g.v again: seven products
// of tiles for the five that the formulas hold, against a dq that would have to be summed through memory.
//
// Bound by the matrix units for long sequences: 8192 tokens of 16 heads on 4 of 128 channels in bf16 take 382 + 511 us and 23 for
// the join of the heads' parts (units 0.56 and 0.51 busy), 753 TFLOP/s counting five products. Short ones wait for their rows: 300
// sequences of up to 120 tokens, 32 heads on 8 of 64 channels, 107 + 100 us for 375 MB that no call can do without (73 us). fp32,
// five sequences of up to 1000 tokens, 12 heads of 80 channels: 107 + 140 us, one wave a SIMD (units 0.44 and 0.47 busy). Past 128
// channels fp32 keys keep sums in scratch memory (256 bytes a lane with 192, 1040 with 256): 443 tokens of 40 heads of 256, 709 us.
#include "packed.h"

namespace moe {

namespace {

template <class C>
struct BackwardKernel {
  static constexpr int EU_Q = C::F32 ? 1 : (C::DP <= 128 ? 2 : 1);
  // bf16 keys of 96 to 192 channels: eight waves whose V comes from LDS for every product, so that two fit a SIMD (gradient of 1788
  // tokens of 84 heads of 192: 570 -> 505 us; heads of 64 fit with V in registers, and lose by it: 577 -> 612 us)
  static constexpr bool V_LDS = !C::F32 && C::DP >= 96 && C::DP <= 192;
  static constexpr int NW_K = V_LDS ? 8 : 4;
  // up to 64 channels three waves fit (gradient of 300 sequences of up to 120 tokens, 32 heads of 64: 215 -> 198 us)
  static constexpr int EU_K = V_LDS ? 2 : (!C::F32 && C::DP <= 64) ? 3 : 1;
  static constexpr int LDS_Q = 4 * C::STAGE;
  static constexpr int STATS = 2 * 64 * 4;                    // lse and -delta of a stage's queries
  static constexpr int LDS_K = 2 * (2 * C::STAGE + STATS) + (V_LDS ? NW_K * C::TILE : 0);
  // Past 128 channels K, V, dK and dV of a wave's keys together pass the registers: dv and dk are taken one after the other; with
  // fp32 past 192 channels dk in two halves of its channels.
  static constexpr int PASSES = C::DP <= 128 ? 1 : C::F32 && C::DP > 192 ? 3 : 2;
};
// What a pass over the queries sums: dv or not, and NK blocks of 32 channels of dk from K0 on.
template <bool DV_, int K0_, int NK_>
struct KeySums {
  static constexpr bool DV = DV_;
  static constexpr int K0 = K0_, NK = NK_;
};

__device__ __forceinline__ float exp_base2(float s, float c, float lse2) { return __builtin_amdgcn_exp2f(fmaf(s, c, -lse2)); }

// dq of one row over the keys it sees alone.
template <class C>
__device__ __forceinline__ void dq_alone(const PackedArgs& a, int head, int kv, int row, int start, float lse2, float delta) {
  using E = typename C::E;
  constexpr int NC = (C::DP + 63) / 64;
  const int lane = threadIdx.x & 63, D = a.D;
  const float c = a.scale * kLog2e;
  const E* q = static_cast<const E*>(a.q.in) + row * a.q.in_t + head * a.q.in_h;
  const E* g = static_cast<const E*>(a.d_out) + row * a.do_t + head * a.do_h;
  const E* k = static_cast<const E*>(a.k.in) + kv * a.k.in_h;
  const E* v = static_cast<const E*>(a.v.in) + kv * a.v.in_h;
  float o[NC] = {};
#pragma unroll 1
  for (int j = start; j <= row; j += 64) {
    const int n = min(64, row + 1 - j);
    float t = 0.0f;
    if (lane < n) {
      const float p = exp_base2(row_dot<E>(q, k + (j + lane) * a.k.in_t, D), c, lse2);
      t = p * (row_dot<E>(g, v + (j + lane) * a.v.in_t, D) - delta);
    }
    add_rows_alone<C, NC>(k + j * a.k.in_t, a.k.in_t, n, D, t, o);
  }
  E* out = static_cast<E*>(a.q.out) + row * a.q.out_t + head * a.q.out_h;
#pragma unroll
  for (int i = 0; i < NC; ++i)
    if (64 * i + lane < D) out[64 * i + lane] = from_f32<E>(o[i] * a.scale);
}

}  // namespace

// SPLIT: a block takes 32 rows, its waves every fourth tile of their keys.
template <class C, bool SPLIT>
__global__ __launch_bounds__(C::NT, SPLIT ? 1 : BackwardKernel<C>::EU_Q) void causal_dq_kernel(PackedArgs a, PackedGrid grid) {
  using E = typename C::E;
  using S = SplitCfg<C>;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  __shared__ int ends[2][C::NW];
  int head, rank;
  if (!grid.item(blockIdx.x, head, rank)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tile = grid.tiles - 1 - rank, row0 = SPLIT ? tile * 32 : tile * C::ROWS + wave * 32, row = row0 + (lane & 31);
  EarlyRows<C> g, o, q;
  g.begin(static_cast<const E*>(a.d_out) + head * a.do_h, a.do_t, row0, a.T, a.D, a.wide & 2);
  o.begin(static_cast<const E*>(a.o) + head * a.o_h, a.o_t, row0, a.T, a.D, a.wide & 4);
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
  // two waves' tiles fit beside the first stage, or four
  constexpr bool BESIDE = SPLIT ? S::SLOTS == 2 : C::NS == 2;
  auto issue = [&](char* to, int j) {
    if constexpr (SPLIT) {
      ks.issue_tile(to, j);
      vs.issue_tile(to + C::TILE, j);
    } else {
      ks.issue(to, j);
      vs.issue(to + C::STAGE, j);
    }
  };
  char *const mine = lds + wave * S::OWN, *own = SPLIT ? mine + (S::SLOTS - 1) * S::SLOT
                                                       : lds + (BESIDE ? 2 * C::STAGE : 0) + wave * C::TILE;
  const int begin = SPLIT ? first + 32 * wave : first;
  if (BESIDE && begin <= last) issue(SPLIT ? mine : lds, begin);
  Quad qf[C::NF], gf[C::NF];
  float delta = 0.0f;
  g.end(own, lanes, live, gf);
  o.end(own, lanes, live, qf);
#pragma unroll
  for (int s = 0; s < C::NF; ++s) {
    if constexpr (C::F32) {
      const f32x4 x = __builtin_bit_cast(f32x4, gf[s].u), y = __builtin_bit_cast(f32x4, qf[s].u);
      delta += (x[0] * y[0] + x[1] * y[1]) + (x[2] * y[2] + x[3] * y[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) delta = fmaf(to_f32(gf[s].h[e]), to_f32(qf[s].h[e]), delta);
    }
  }
  q.end(own, lanes, live, qf);
  delta = halves_sum(delta);
  // rows that saw nothing but scores of -infinity have lse -infinity, and weights of 0
  float lse2 = live ? a.lse[static_cast<long long>(row) * a.q.heads + head] * kLog2e : 0.0f;
  if (lse2 == -INFINITY) lse2 = INFINITY;
  if (live && lane < 32 && (!SPLIT || wave == 0)) {
    float* stats = a.ws + static_cast<long long>(head) * 2 * a.T + row;
    stats[0] = lse2;
    stats[a.T] = -delta;
  }
  // sums that may hold what the row does not see; with lse or delta NaN every channel is NaN, and right as it is
  const bool check = live && lse2 == lse2 && delta == delta;
  const float c = a.scale * kLog2e;
  f32x16 sums[C::NB], minus_delta, zero;
  clear_sums(sums);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    minus_delta[e] = -delta;
    zero[e] = 0.0f;
  }
  auto turn = [&](const char* k, const char* v, int j) {
    const f32x16 s = tile_products<C>(k, lanes, qf, zero), dp = tile_products<C>(v, lanes, gf, minus_delta);
    float x[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = exp_base2(s[e], c, lse2);
    const bool whole = j >= whole_from && j + 31 <= whole_to;
    if (!whole) mask_weights(x, tokens_below(row + 1, j) & ~tokens_below(span.start, j));
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] *= dp[e];
    add_weighted<C>(k, lanes, x, !whole, sums);
  };
  E* const out = static_cast<E*>(a.q.out) + head * a.q.out_h;
  uint32_t again = 0;
  if constexpr (SPLIT) {
    __shared__ uint32_t bad[4];
    if (lane == 0) bad[wave] = 0;
    wave_tiles<C, S>(mine, begin, last, (a.direct & 3) == 3, issue, [&](const char* at, int j) { turn(at, at + C::TILE, j); });
    __syncthreads();
    join_waves<S::OWN>(lds, sums, 1.0f, check, bad, [&](int i, const f32x16 (&x)[1]) {
      store_rows<C>(lds + wave * C::TILE, out, a.q.out_t, row0, a.D, x, a.scale, ws.b, a.wide & 8, i);
    });
    stage_barrier();
    again = (bad[0] | bad[1] | bad[2] | bad[3]) & (0x11111111u << wave);
  } else {
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
    __syncthreads();      // the stages are read
    store_rows<C>(lds + wave * C::TILE, out, a.q.out_t, row0, a.D, sums, a.scale, ws.b, a.wide & 8);
    again = tokens_not_finite(sums, check);
  }
#pragma unroll 1
  for (; again; again &= again - 1) {
    const int t = __builtin_ctz(again);
    dq_alone<C>(a, head, kv, row0 + t, __builtin_amdgcn_readlane(span.start, t),
                __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(lse2), t)),
                __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(delta), t)));
  }
}

namespace {

// Where the sums of a part of the heads go: the gradients, or fp32 as the lanes hold them: four channels of
// [part][dk, dv][kv head][tile of 32 keys][channels / 8][lane].
struct KeyOut {
  int parts;
  float* sums;      // null: one part, written as the result
  int tiles;
};
template <class C>
__device__ __forceinline__ float* part_sums(const PackedArgs& a, const KeyOut& out, int part, int which, int kv, int key0) {
  return out.sums + ((static_cast<long long>(part * 2 + which) * a.k.heads + kv) * out.tiles + (key0 >> 5)) * (32 * C::DP);
}
template <int N>
__device__ __forceinline__ void put_part(float* to, const f32x16 (&s)[N], float f, int B0) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      *reinterpret_cast<f32x4*>(to + (((B0 + i) * 4 + g) * 64 + lane) * 4) =
          f32x4{s[i][4 * g] * f, s[i][4 * g + 1] * f, s[i][4 * g + 2] * f, s[i][4 * g + 3] * f};
}
// Channel c of key t of a part's tile.
__device__ __forceinline__ int part_place(int t, int c) { return ((c / 8) * 64 + ((c / 4) & 1) * 32 + t) * 4 + (c & 3); }

// dk and dv of one key over the queries that see it alone, of the heads h0 .. h1 - 1. The last ones come first, and the sums end
// where all are NaN: a NaN in a sequence is mostly in all that comes after it.
template <class C>
__device__ __forceinline__ void key_alone(const PackedArgs& a, int h0, int h1, int kv, int key, int end,
                                          float (&dk)[(C::DP + 63) / 64], float (&dv)[(C::DP + 63) / 64]) {
  using E = typename C::E;
  constexpr int NC = (C::DP + 63) / 64;
  const int lane = threadIdx.x & 63, D = a.D;
  const float c = a.scale * kLog2e;
  const E* k = static_cast<const E*>(a.k.in) + key * a.k.in_t + kv * a.k.in_h;
  const E* v = static_cast<const E*>(a.v.in) + key * a.v.in_t + kv * a.v.in_h;
#pragma unroll
  for (int i = 0; i < NC; ++i) dk[i] = dv[i] = 0.0f;
#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
    const E* q = static_cast<const E*>(a.q.in) + h * a.q.in_h;
    const E* g = static_cast<const E*>(a.d_out) + h * a.do_h;
    const float* stats = a.ws + static_cast<long long>(h) * 2 * a.T;
#pragma unroll 1
    for (int i = key + (end - 1 - key) / 64 * 64; i >= key; i -= 64) {
      const int n = min(64, end - i), row = i + lane;
      float p = 0.0f, t = 0.0f;
      if (lane < n) {
        p = exp_base2(row_dot<E>(q + row * a.q.in_t, k, D), c, stats[row]);
        t = p * (row_dot<E>(g + row * a.do_t, v, D) + stats[a.T + row]);
      }
      add_rows_alone<C, NC>(q + i * a.q.in_t, a.q.in_t, n, D, t, dk);
      add_rows_alone<C, NC>(g + i * a.do_t, a.do_t, n, D, p, dv);
      bool none = true;
#pragma unroll
      for (int x = 0; x < NC; ++x) none = none && (64 * x + lane >= D || (dk[x] != dk[x] && dv[x] != dv[x]));
      if (__all(none)) return;
    }
  }
}

// The sums of one wave's keys, or, SPLIT, of the block's 32 keys, of whose queries (of all heads) the waves take every fourth
// tile.
template <class C, class S, bool SPLIT>
__device__ __forceinline__ void key_pass(const PackedArgs& a, const KeyOut& out, int part, int kv, int h0, int h1, int key0,
                                         const Span& span, int first, int last, int end, char* lds, const EarlyRows<C>& k,
                                         const EarlyRows<C>& v) {
  using E = typename C::E;
  constexpr int SLOT = 2 * C::STAGE + BackwardKernel<C>::STATS;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), key = key0 + (lane & 31);
  const bool live = span.live;
  const WaveSpan ws(live);
  const int lo = ws.last < 0 ? INT_MAX : key0 + ws.first, hi = ws.last < 0 ? -1 : ws.of_last(span.end) - 1;      // queries
  const int whole_from = key0 + ws.last, whole_to = ws.of_first(span.end) - 1;
  using Z = SplitCfg<C, BackwardKernel<C>::STATS>;
  // A stage of queries from row i on: q, d_out, and 64 of lse (base 2) and -delta each.
  auto issue = [&](char* st, int h, int i) {
    const RowLoader<C> qs(a.q.in, a.q.in_t, a.q.in_h, h, end, a.D, a.direct & 1);
    const RowLoader<C> gs(a.d_out, a.do_t, a.do_h, h, end, a.D, a.direct & 2);
    constexpr int TOKENS = SPLIT ? C::TILE : C::STAGE;
    if constexpr (SPLIT) {
      qs.issue_tile(st, i);
      gs.issue_tile(st + TOKENS, i);
    } else {
      qs.issue(st, i);
      gs.issue(st + TOKENS, i);
    }
    auto stats = [&](int which) {
      const float* x = a.ws + (static_cast<long long>(h) * 2 + which) * a.T + i;
      const auto rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(x), static_cast<short>(0),
                                                        4 * min(64, end - i), 0x00020000);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_any_t*)(st + 2 * TOKENS + which * 256), 4, lane * 4, 0, 0, 0);
    };
    if (SPLIT) {
      stats(0);
      stats(1);
    } else if (wave < 2) {
      stats(wave);
    }
  };
  constexpr bool DV = S::DV, DK = S::NK > 0, V_LDS = !SPLIT && BackwardKernel<C>::V_LDS;
  const TileLanes lanes;
  // SPLIT: the wave's work is the tiles wave, wave + 4, .. of h0 .. h1 - 1, first .. last
  const int per_head = (last - first) / 32 + 1, count = per_head * (h1 - h0);
  char* const mine = lds + wave * Z::OWN;
  auto issue_item = [&](char* to, int n) { issue(to, h0 + n / per_head, first + n % per_head * 32); };
  // a tile of the wave's own, where V goes that is kept in LDS; else beside the first stage if that leaves room for all waves
  constexpr bool BESIDE = SPLIT ? Z::SLOTS == 2 : V_LDS || C::NS == 2;
  char* const own = SPLIT ? mine + (Z::SLOTS - 1) * Z::SLOT
                          : lds + (V_LDS ? 2 * SLOT : BESIDE ? SLOT : 0) + wave * C::TILE;
  if (BESIDE) {
    if (!SPLIT) issue(lds, h0, first);
    else if (wave < count) issue_item(mine, wave);
  }
  Quad kf[C::NF], vf[DK && !V_LDS ? C::NF : 1];
  k.end(own, lanes, live, kf);
  if constexpr (DK && !V_LDS) v.end(own, lanes, live, vf);
  if constexpr (DK && V_LDS) v.keep(own);
  if (!BESIDE && !SPLIT) {
    __syncthreads();
    issue(lds, h0, first);
  }
  const float c = a.scale * kLog2e;
  f32x16 dk[DK ? S::NK : 1], dv[DV ? C::NB : 1], zero;
  clear_sums(dk);
  clear_sums(dv);
#pragma unroll
  for (int e = 0; e < 16; ++e) zero[e] = 0.0f;
  const int hb4 = 4 * ((lane >> 5) & 1);
  auto tile = [&](const char* qt, const char* gt, const float* stats, bool whole, uint32_t seen) {
    const f32x16 s = tile_products<C>(qt, lanes, kf, zero);
    float x[16];
#pragma unroll
    for (int e = 0; e < 16; e += 4) {
      const f32x4 lse2 = *reinterpret_cast<const f32x4*>(stats + 2 * e + hb4);
#pragma unroll
      for (int z = 0; z < 4; ++z) x[e + z] = exp_base2(s[e + z], c, lse2[z]);
    }
    if (!whole) mask_weights(x, seen);
    if constexpr (DV) {
      Weights<C> w;
#pragma unroll
      for (int e = 0; e < 16; ++e) w.set(e, x[e]);
      add_columns<C>(gt, lanes, w, dv);
    }
    if constexpr (DK) {
      f32x16 dp;
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const f32x4 y = *reinterpret_cast<const f32x4*>(stats + 64 + 2 * e + hb4);
#pragma unroll
        for (int z = 0; z < 4; ++z) dp[e + z] = y[z];
      }
      if constexpr (V_LDS) dp = tile_products<C>(gt, lanes, own, dp);
      else dp = tile_products<C>(gt, lanes, vf, dp);
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] *= dp[e];
      add_weighted<C, S::K0>(qt, lanes, x, !whole, dk);
    }
  };
  auto turn = [&](const char* qt, const char* gt, const float* stats, int it) {
    const bool whole = it >= whole_from && it + 31 <= whole_to;
    tile(qt, gt, stats, whole, tokens_below(span.live ? span.end : 0, it) & ~tokens_below(key, it));
  };
  const bool parts = out.sums != nullptr;
  uint32_t again = 0;
  if constexpr (SPLIT) {
    __shared__ uint32_t bad[4];
    if (lane == 0) bad[wave] = 0;
    wave_tiles<C, Z, 4, 1>(mine, wave, count - 1, (a.direct & 3) == 3, issue_item, [&](const char* at, int n) {
      turn(at, at + C::TILE, reinterpret_cast<const float*>(at + 2 * C::TILE), first + n % per_head * 32);
    });
    __syncthreads();
    auto finish = [&](const auto& sums, int b0, int which, const Rows& r, float f) {
      join_waves<Z::OWN>(lds, sums, 1.0f, live, bad, [&](int i, const f32x16 (&x)[1]) {
        if (parts) put_part(part_sums<C>(a, out, part, which, kv, key0), x, f, b0 + i);
        else store_rows<C>(lds + wave * C::TILE, static_cast<E*>(r.out) + kv * r.out_h, r.out_t, key0, a.D, x, f, ws.b,
                           a.wide & (which ? 8 : 4), b0 + i);
      });
      __syncthreads();
    };
    if constexpr (DK) finish(dk, S::K0, 0, a.k, a.scale);
    if constexpr (DV) finish(dv, 0, 1, a.v, 1.0f);
    stage_barrier();
    again = (bad[0] | bad[1] | bad[2] | bad[3]) & (0x11111111u << wave);
  } else {
    int h = h0, i = first;
    for (int n = 0; h < h1; ++n) {
      stage_barrier();
      const int now = i;
      i += C::KT;
      if (i > last) {
        i = first;
        ++h;
      }
      if (h < h1) issue(lds + (~n & 1) * SLOT, h, i);
      const char* q = lds + (n & 1) * SLOT;
#pragma unroll
      for (int t = 0; t < C::NS; ++t)
        if (now + 32 * t <= hi && now + 32 * t + 31 >= lo)
          turn(q + t * C::TILE, q + t * C::TILE + C::STAGE, reinterpret_cast<const float*>(q + 2 * C::STAGE) + 32 * t,
               now + 32 * t);
    }
    if constexpr (DK) again |= tokens_not_finite(dk, live);
    if constexpr (DV) again |= tokens_not_finite(dv, live);
    if (parts) {
      if (ws.last >= 0) {
        if constexpr (DK) put_part(part_sums<C>(a, out, part, 0, kv, key0), dk, a.scale, S::K0);
        if constexpr (DV) put_part(part_sums<C>(a, out, part, 1, kv, key0), dv, 1.0f, 0);
      }
    } else {
      __syncthreads();      // the stages are read
      char* const tile = lds + wave * C::TILE;
      if constexpr (DK)
        store_rows<C>(tile, static_cast<E*>(a.k.out) + kv * a.k.out_h, a.k.out_t, key0, a.D, dk, a.scale, ws.b, a.wide & 4, S::K0);
      if constexpr (DV)
        store_rows<C>(tile, static_cast<E*>(a.v.out) + kv * a.v.out_h, a.v.out_t, key0, a.D, dv, 1.0f, ws.b, a.wide & 8);
    }
  }
#pragma unroll 1
  while (again) {
    const int t = __builtin_ctz(again), x = key0 + t;
    again &= again - 1;
    constexpr int NC = (C::DP + 63) / 64;
    float k1[NC], v1[NC];
    key_alone<C>(a, h0, h1, kv, x, __builtin_amdgcn_readlane(span.end, t), k1, v1);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int ch = 64 * i + lane;
      if (ch >= a.D) continue;
      if (parts) {
        if constexpr (DK) part_sums<C>(a, out, part, 0, kv, key0)[part_place(t, ch)] = k1[i] * a.scale;
        if constexpr (DV) part_sums<C>(a, out, part, 1, kv, key0)[part_place(t, ch)] = v1[i];
      } else {
        if constexpr (DK) static_cast<E*>(a.k.out)[x * a.k.out_t + kv * a.k.out_h + ch] = from_f32<E>(k1[i] * a.scale);
        if constexpr (DV) static_cast<E*>(a.v.out)[x * a.v.out_t + kv * a.v.out_h + ch] = from_f32<E>(v1[i]);
      }
    }
  }
}

}  // namespace

// C: with NW_K waves, or four if SPLIT.
template <class C, bool SPLIT>
__global__ __launch_bounds__(C::NT, SPLIT ? 1 : BackwardKernel<C>::EU_K) void causal_dkv_kernel(PackedArgs a, PackedGrid grid,
                                                                                               KeyOut out) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  __shared__ int ends[2][C::NW];
  int item, rank;
  if (!grid.item(blockIdx.x, item, rank)) return;
  const int kv = item / out.parts, part = item % out.parts, G = a.q.heads / a.k.heads;
  const int h0 = kv * G + part * G / out.parts, h1 = kv * G + (part + 1) * G / out.parts;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int key0 = SPLIT ? rank * 32 : rank * C::ROWS + wave * 32, key = key0 + (lane & 31);
  using E = typename C::E;
  EarlyRows<C> k, v;
  auto load = [&] {
    k.begin(static_cast<const E*>(a.k.in) + kv * a.k.in_h, a.k.in_t, key0, a.T, a.D, a.wide & 1);
    v.begin(static_cast<const E*>(a.v.in) + kv * a.v.in_h, a.v.in_t, key0, a.T, a.D, a.wide & 2);
  };
  load();
  const int end = packed_end(a.seq_start, a.n_seqs, a.T);
  const Span span = find_span(a.seq_start, a.n_seqs, a.T, end, key0, key);
  const WaveSpan ws(span.live);
  int first = ws.last < 0 ? INT_MAX : key0 + ws.first, last = ws.last < 0 ? -1 : ws.of_last(span.end) - 1;
  if (!SPLIT) block_range<C>(first, last, ends, first, last);
  last = min(last, end - 1);      // as it is, but for entries out of order: stages begin below `end`
  if (last < first) return;
  constexpr int PASSES = BackwardKernel<C>::PASSES, NB = C::NB;
  if constexpr (PASSES == 1) {
    key_pass<C, KeySums<true, 0, NB>, SPLIT>(a, out, part, kv, h0, h1, key0, span, first, last, end, lds, k, v);
  } else {
    key_pass<C, KeySums<true, 0, 0>, SPLIT>(a, out, part, kv, h0, h1, key0, span, first, last, end, lds, k, v);
    stage_barrier();
    load();
    key_pass<C, KeySums<false, 0, PASSES == 2 ? NB : NB / 2>, SPLIT>(a, out, part, kv, h0, h1, key0, span, first, last, end, lds, k,
                                                                     v);
    if constexpr (PASSES == 3) {
      stage_barrier();
      load();
      key_pass<C, KeySums<false, NB / 2, NB / 2>, SPLIT>(a, out, part, kv, h0, h1, key0, span, first, last, end, lds, k, v);
    }
  }
}

// The parts' sums, in order, as the gradients; a wave takes a tile of 32 keys.
template <class C>
__global__ __launch_bounds__(C::NT) void causal_join_kernel(PackedArgs a, KeyOut out) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  using E = typename C::E;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kv = blockIdx.y >> 1, which = blockIdx.y & 1, key0 = (blockIdx.x * C::NW + wave) * 32;
  const int from = max(a.seq_start[0], 0), to = min(a.seq_start[a.n_seqs], a.T);
  const uint32_t live = tokens_below(to, key0) & ~tokens_below(from, key0);
  if (!live) return;
  f32x16 s[C::NB];
  clear_sums(s);
  for (int p = 0; p < out.parts; ++p) {
    const float* x = part_sums<C>(a, out, p, which, kv, key0);
#pragma unroll
    for (int i = 0; i < C::NB; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 y = *reinterpret_cast<const f32x4*>(x + ((i * 4 + g) * 64 + lane) * 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][4 * g + e] += y[e];
      }
  }
  const Rows& r = which ? a.v : a.k;
  store_rows<C>(lds + wave * C::TILE, static_cast<E*>(r.out) + kv * r.out_h, r.out_t, key0, a.D, s, 1.0f, live,
                a.wide & (which ? 8 : 4));
}

// Parts of a group's heads that blocks of their own take: while there are fewer than four blocks of 128 keys for each CU; with
// blocks of 32 keys, while a wave has more than eight tiles of queries.
static int key_parts(int T, int q_heads, int kv_heads, bool split) {
  const int group = q_heads / kv_heads;
  const long long blocks = static_cast<long long>((T + 127) / 128) * kv_heads;
  int p = 1;
  if (split)
    while (p < group && blocks * 4 * p < 2 * device_cu_count() && static_cast<long long>(T) * group > 1024LL * p) ++p;
  else
    while (p < group && blocks * p < 4 * device_cu_count()) ++p;
  return p;
}

static size_t stats_floats(int T, int q_heads) { return (static_cast<size_t>(q_heads) * 2 * T + 3) / 4 * 4; }

size_t causal_backward_ws_bytes(int T, int D, int q_heads, int kv_heads) {
  const int parts = std::max(key_parts(T, q_heads, kv_heads, false), key_parts(T, q_heads, kv_heads, true));
  const int DP = D <= 64 ? 64 : D <= 96 ? 96 : D <= 128 ? 128 : D <= 192 ? 192 : 256;
  const size_t tiles = (static_cast<size_t>(T) + 31) / 32;
  return 4 * (stats_floats(T, q_heads) + (parts > 1 ? static_cast<size_t>(parts) * 2 * kv_heads * tiles * 32 * DP : 0));
}

template <class K>
static hipError_t allow_lds(K kernel, int bytes) {
  return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

hipError_t launch_causal_backward(const PackedArgs& args, moe_dtype act, hipStream_t st) {
  return with_packed_cfg(act, args.D, [&](auto cfg) {
    using C = decltype(cfg);
    using B = BackwardKernel<C>;
    using SQ = SplitCfg<C>;
    using SK = SplitCfg<C, B::STATS>;
    constexpr int ES = C::ES;
    PackedArgs a = args;
    a.direct = loads_direct(a.k.in, a.k.in_t, a.k.in_h, ES) | loads_direct(a.v.in, a.v.in_t, a.v.in_h, ES) << 1;
    a.wide = aligned16(a.q.in, a.q.in_t, a.q.in_h, ES) | aligned16(a.d_out, a.do_t, a.do_h, ES) << 1 |
             aligned16(a.o, a.o_t, a.o_h, ES) << 2 | aligned16(a.q.out, a.q.out_t, a.q.out_h, ES) << 3;
    auto queries = [&](auto split) {
      constexpr bool SPLIT = decltype(split)::value;
      constexpr int LDS = SPLIT ? 4 * SQ::OWN : B::LDS_Q, ROWS = SPLIT ? 32 : C::ROWS;
      static const hipError_t allowed = allow_lds(causal_dq_kernel<C, SPLIT>, LDS);
      if (allowed != hipSuccess) return allowed;
      const PackedGrid grid = PackedGrid::of(a.q.heads, (a.T + ROWS - 1) / ROWS);
      hipLaunchKernelGGL((causal_dq_kernel<C, SPLIT>), dim3(grid.blocks), dim3(C::NT), LDS, st, a, grid);
      return hipGetLastError();
    };
    KeyOut out{1, nullptr, (a.T + 31) / 32};
    auto keys = [&](auto split) {
      constexpr bool SPLIT = decltype(split)::value;
      using CK = typename C::template with_waves<SPLIT ? 4 : B::NW_K>;
      constexpr int LDS = SPLIT ? 4 * SK::OWN : B::LDS_K, ROWS = SPLIT ? 32 : CK::ROWS;
      static const hipError_t allowed = allow_lds(causal_dkv_kernel<CK, SPLIT>, LDS);
      if (allowed != hipSuccess) return allowed;
      out.parts = key_parts(a.T, a.q.heads, a.k.heads, SPLIT);
      if (out.parts > 1) out.sums = a.ws + stats_floats(a.T, a.q.heads);
      const PackedGrid grid = PackedGrid::of(a.k.heads * out.parts, (a.T + ROWS - 1) / ROWS);
      hipLaunchKernelGGL((causal_dkv_kernel<CK, SPLIT>), dim3(grid.blocks), dim3(CK::NT), LDS, st, a, grid, out);
      return hipGetLastError();
    };
    auto either = [&](auto fits, bool split, auto launch) {
      if constexpr (decltype(fits)::value) {
        if (split) return launch(std::true_type{});
      }
      return launch(std::false_type{});
    };
    hipError_t e = either(std::bool_constant<SQ::FITS>{}, split_rows(a.T, a.n_seqs, a.q.heads, a.D, C::F32), queries);
    if (e != hipSuccess) return e;
    a.direct = loads_direct(a.q.in, a.q.in_t, a.q.in_h, ES) | loads_direct(a.d_out, a.do_t, a.do_h, ES) << 1;
    a.wide = aligned16(a.k.in, a.k.in_t, a.k.in_h, ES) | aligned16(a.v.in, a.v.in_t, a.v.in_h, ES) << 1 |
             aligned16(a.k.out, a.k.out_t, a.k.out_h, ES) << 2 | aligned16(a.v.out, a.v.out_t, a.v.out_h, ES) << 3;
    e = either(std::bool_constant<SK::FITS>{}, split_rows(a.T, a.n_seqs, a.q.heads, a.D, C::F32), keys);
    if (e != hipSuccess || out.parts == 1) return e;
    hipLaunchKernelGGL(causal_join_kernel<C>, dim3((out.tiles + C::NW - 1) / C::NW, 2 * a.k.heads), dim3(C::NT), C::NW * C::TILE,
                       st, a, out);
    return hipGetLastError();
  });
}

}  // namespace moe
