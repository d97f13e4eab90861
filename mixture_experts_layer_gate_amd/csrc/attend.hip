// Attention over the paged cache for sequences that share a prefix:
//   out_r = sum_j exp(s_rj - m) v_j / sum_j exp(s_rj - m),  s_rj = scale q_r . k_j,
// in one pass over the keys with a running reference m, sums in fp32.
//
// Work. The prefix is one stream of keys per key/value head that every query row of the
// batch reads: its rows are all (token, query head of the group). A sequence's own tokens are a
// stream that only its q_len * group rows read. A block takes an item: a tile of one
// stream's rows and a range of its tokens, and leaves (m, l, sum) per row; a second kernel joins the
// parts of each row. Both kinds of item run in one launch, so that the prefix items, bound by
// the matrix units and the exponentials, share the CUs with the own items, bound by HBM.
//
// Tile. 32 tokens x 32 rows. S^T = K Q^T on 32x32 MFMAs leaves lane l the scores of row l % 32
// for the 16 tokens 8 (v / 4) + 4 (l / 32) + v % 4: the softmax needs one exchange between the two half
// waves, and the weights, rounded to bf16, are the second operand of O^T += V^T P^T as they
// lie, with the contraction order permuted the same way in V^T (whose 4 x 16 pieces come out
// of LDS transposed). fp32 inputs run the same scheme on the 32x32x2 fp32 MFMA.
//
// The reference m is moved (and the sums rescaled) only when a score passes it by 2^8: weights stay
// below 2^8 and every sum is relative to m, so the result does not depend on m.
#include <type_traits>

#include "heads.h"

namespace moe {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

enum { kKindF32 = 0, kKindBf16 = 1, kKindE4M3 = 2 };

template <int KIND_, int DP_>
struct AttendCfg {
  static constexpr int KIND = KIND_, DP = DP_;                 // channels, padded to 64, 128 or 256
  static constexpr int ES = KIND == kKindF32 ? 4 : 2;          // bytes of an element in LDS
  static constexpr int NW = KIND == kKindF32 && DP == 256 ? 2 : 4;   // waves of a block (160 KB of LDS)
  static constexpr int NT = NW * 64;
  // Rows of K are read 16 bytes per lane down 32 rows, rows of V as 4 rows x 32 bytes (transposing reads) or
  // along the row (fp32): a row stride of 16 (32) bytes past a multiple of 128 spreads them over the banks.
  static constexpr int KS = DP * ES + 16, VS = DP * ES + (ES == 2 ? 32 : 16);
  static constexpr int TILE = 32 * (KS + VS) + (KIND == kKindE4M3 ? 256 : 0);   // 32 tokens (and their scales)
  static constexpr int SUB = DP == 256 || KIND == kKindF32 ? 1 : 2;   // 32-token tiles of a shared step
  static constexpr int LDS_SHARED = 2 * SUB * TILE;            // two steps shared by the waves
  static constexpr int LDS_OWN = NW * TILE;                    // one tile per wave
  static constexpr int LDS_MERGE = NW * 32 * (DP + 2) * 4;
  static constexpr int LDS = LDS_SHARED > LDS_OWN ? (LDS_SHARED > LDS_MERGE ? LDS_SHARED : LDS_MERGE)
                                                  : (LDS_OWN > LDS_MERGE ? LDS_OWN : LDS_MERGE);
  static constexpr int BLOCKS = LDS <= 80 * 1024 ? 2 : 1;      // per CU
  static constexpr int CE = KIND == kKindF32 ? 4 : 8;          // elements of a piece (16 LDS bytes)
  static constexpr int CPR = DP / CE;                          // pieces of a row
  static constexpr int NF = DP / 16 * (KIND == kKindF32 ? 2 : 1);   // 16-byte fragments of a lane's K or Q row half
  static_assert(LDS <= 160 * 1024, "LDS");
};

// The split of one call, decided on the host.
struct AttendPlan {
  int pre_rows, own_rows;        // rows of a stream
  int pre_shared, own_shared;    // 1: the waves of a block share the key tiles and have 32 rows each
  int pre_tiles, own_tiles;      // row tiles
  int pre_parts, own_parts;      // ranges of tokens
  int pre_chunk;                 // tokens of a prefix part (multiple of 64)
  int pre_groups, own_groups;    // groups of 8 blocks
  int pre_first;                 // 1: prefix groups first; 0: in proportion
};

__device__ __forceinline__ int own_len(const AttendArgs& a, int b) {
  if (a.table_pages <= 0) return 0;
  const long long cap = static_cast<long long>(a.table_pages) * a.c.page_size;
  return clampi(a.lens[b], 0, static_cast<int>(cap));
}
// Tokens of an own part: the n tokens in own_parts equal ranges of whole 32s.
__device__ __forceinline__ int own_chunk(const AttendPlan& p, int n) {
  return ((n + p.own_parts - 1) / p.own_parts + 31) & ~31;
}

// Token and query head of a stream's row.
__device__ __forceinline__ void row_token(const AttendArgs& a, int G, int b, int r, int& t, int& h) {
  t = r / G;
  h = r - t * G;
  if (b >= 0) t += b * a.S;
}

union Piece {
  uint4 u;
  float f[4];
  bf16x8 h;
};

__device__ __forceinline__ bf16x8 e4m3x8_to_bf16(uint2 c) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.x, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.x, 1.0f, true);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.y, 1.0f, false);
  const bf16x2 e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.y, 1.0f, true);
  return bf16x8{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}

// NaN if either is one: such a row's result is NaN whatever the reference. (One instruction, unlike fmaxf.)
__device__ __forceinline__ float row_max(float x, float y) { return __builtin_elementwise_maximum(x, y); }
__device__ __forceinline__ float half_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return row_max(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

template <class C>
struct AttendState {
  f32x16 o[C::DP / 32];   // O^T: channel 32 i + 8 (v / 4) + 4 (lane / 32) + v % 4 of row lane % 32
  float m, l;             // reference (base 2) and this half wave's part of the sum
};

// The lane's Q fragments: its row's channels in the order the K fragments have them, negated if neg.
template <class C>
__device__ __forceinline__ void load_q(const AttendArgs& a, const void* row, bool live, bool wide, bool neg,
                                       Piece (&qf)[C::NF]) {
  const int hb = (threadIdx.x >> 5) & 1, D = a.c.D;
#pragma unroll
  for (int s = 0; s < C::NF; ++s) {
    const int d0 = (2 * s + hb) * C::CE;
    Piece p;
    p.u = uint4{0, 0, 0, 0};
    if (live && d0 < D) {
      if constexpr (C::KIND == kKindF32) {
        const float* x = static_cast<const float*>(row) + d0;
        if (wide) p.u = *reinterpret_cast<const uint4*>(x);
        else {
#pragma unroll
          for (int e = 0; e < 4; ++e) p.f[e] = x[e];
        }
        if (neg) {
#pragma unroll
          for (int e = 0; e < 4; ++e) p.f[e] = -p.f[e];
        }
      } else {
        const __bf16* x = static_cast<const __bf16*>(row) + d0;
        if (wide) p.u = *reinterpret_cast<const uint4*>(x);
        else {
#pragma unroll
          for (int e = 0; e < 8; ++e) p.h[e] = x[e];
        }
        if (neg) p.u = uint4{p.u.x ^ 0x80008000u, p.u.y ^ 0x80008000u, p.u.z ^ 0x80008000u, p.u.w ^ 0x80008000u};
      }
    }
    qf[s] = p;
  }
}


// Pieces of K and V of 32 * NSUB tokens on their way from the cache to LDS, in registers; TH threads take part.
// Piece q of thread i is piece e % CPR of token e / CPR, e = q TH + i.
template <class C, int NSUB, int TH>
struct Staged {
  static constexpr int N = 32 * NSUB * C::CPR / TH;
  static constexpr bool Q8 = C::KIND == kKindE4M3;
  typedef typename std::conditional<Q8, uint2, uint4>::type Raw;
  Raw k[N], v[N];
  float ks, vs;
  uint32_t mask[NSUB];   // tokens that exist

  // page: page of token base + lane (first 32 * NSUB lanes), -1 where there is no such token. Missing tokens read
  // page 0, which exists, and are cleared by store.
  __device__ __forceinline__ void load(const AttendArgs& a, int hk, int base, int page, int i) {
    const uint64_t b = __ballot(page >= 0);
#pragma unroll
    for (int s = 0; s < NSUB; ++s) mask[s] = static_cast<uint32_t>(b >> (32 * s));
    page = page < 0 ? 0 : page;
    const uint32_t ps = a.c.page_size, row_bytes = a.c.D * (Q8 ? 1 : C::ES), page_bytes = a.c.heads * ps * row_bytes;
    const int c = (i % C::CPR) * C::CE;
    const uint32_t in_page = hk * ps * row_bytes + (c < a.c.D ? c : 0) * (Q8 ? 1 : C::ES);
#pragma unroll
    for (int q = 0; q < N; ++q) {
      const int tok = q * (TH / C::CPR) + i / C::CPR;
      const uint64_t off = static_cast<uint64_t>(static_cast<uint32_t>(__shfl(page, tok, 64))) * page_bytes +
                           (in_page + ((base + tok) & (ps - 1)) * row_bytes);
      k[q] = *reinterpret_cast<const Raw*>(static_cast<const char*>(a.c.k) + off);
      v[q] = *reinterpret_cast<const Raw*>(static_cast<const char*>(a.c.v) + off);
    }
    if constexpr (Q8) {
      const uint64_t row = static_cast<uint64_t>(static_cast<uint32_t>(page)) * (a.c.heads * ps) +
                           (hk * ps + ((base + (threadIdx.x & 63)) & (ps - 1)));
      ks = a.c.k_scale[row];
      vs = a.c.v_scale[row];
    }
  }

  template <bool WHOLE>
  __device__ __forceinline__ void put(char* lds, int D, int i) const {
    const int p = i % C::CPR;
#pragma unroll
    for (int q = 0; q < N; ++q) {
      constexpr int PER = TH / C::CPR;      // tokens of one q: all in one 32-token tile
      const int sub = q * PER / 32, tok = q * PER % 32 + i / C::CPR;
      char* t = lds + sub * C::TILE + tok * C::KS + p * 16;
      Piece x, y;
      if constexpr (Q8) {
        x.h = e4m3x8_to_bf16(k[q]);
        y.h = e4m3x8_to_bf16(v[q]);
      } else {
        x.u = k[q];
        y.u = v[q];
      }
      if constexpr (!WHOLE) {
        const uint32_t on = p * C::CE < D && ((mask[sub] >> tok) & 1) ? 0xFFFFFFFFu : 0u;
        x.u = uint4{x.u.x & on, x.u.y & on, x.u.z & on, x.u.w & on};
        y.u = uint4{y.u.x & on, y.u.y & on, y.u.z & on, y.u.w & on};
      }
      *reinterpret_cast<uint4*>(t) = x.u;
      *reinterpret_cast<uint4*>(t + 32 * C::KS + tok * (C::VS - C::KS)) = y.u;
    }
  }
  __device__ __forceinline__ void store(char* lds, int D, int i) const {
    bool whole = D == C::DP;
#pragma unroll
    for (int s = 0; s < NSUB; ++s) whole = whole && mask[s] == 0xFFFFFFFFu;
    if (whole) put<true>(lds, D, i);
    else put<false>(lds, D, i);
    if constexpr (Q8) {
      const int lane = threadIdx.x & 63;
      if (i < 32 * NSUB) {
        float* sc = reinterpret_cast<float*>(lds + (lane >> 5) * C::TILE + 32 * (C::KS + C::VS));
        sc[lane & 31] = ks;
        sc[32 + (lane & 31)] = vs;
      }
    }
  }
};

// V^T fragment of 16 tokens (step ks) and 32 channels (block db): element e of a lane is channel lane % 32 of
// token 16 ks + 8 (e / 4) + 4 (lane / 32) + e % 4.
template <class C>
__device__ __forceinline__ bf16x8 v_fragment(const char* v, int ks, int db) {
  const int lane = threadIdx.x & 63;
  const int row = 16 * ks + 4 * (lane >> 5) + ((lane >> 2) & 3), col = db * 32 + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
  const char* p = v + row * C::VS + col * 2;
  union {
    s16x4 h[2];
    bf16x8 f;
  } u;
  u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p));
  u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 8 * C::VS));
  return u.f;
}

// acc += V^T P^T over the tile's 32 tokens for channel block db (fp32); tokens outside `keep` count as zero if CUT.
template <class C, bool CUT>
__device__ __forceinline__ f32x16 weighted_values_f32(const char* v, const float (&p)[16], int db, uint32_t keep,
                                                      f32x16 acc) {
  const int lane = threadIdx.x & 63, hb = lane >> 5;
  float x[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int tok = 8 * (e >> 2) + 4 * hb + (e & 3);
    x[e] = *reinterpret_cast<const float*>(v + tok * C::VS + (db * 32 + (lane & 31)) * 4);
    if (CUT && !((keep >> tok) & 1)) x[e] = 0.0f;
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int e = 0; e < 16; ++e) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(x[e], p[e], acc, 0, 0, 0);
  return acc;
}

// Tokens of the tile whose V row holds an infinity or a NaN.
template <class C>
__device__ __forceinline__ uint32_t not_finite(const char* v) {
  const int lane = threadIdx.x & 63;
  constexpr int PER = 64 / C::CPR;      // rows that the wave looks at together
  constexpr uint64_t ROW = C::CPR == 64 ? ~0ull : (1ull << (C::CPR & 63)) - 1;
  uint32_t found = 0;
#pragma unroll 1
  for (int r = 0; r < 32; r += PER) {
    const uint4 x = *reinterpret_cast<const uint4*>(v + (r + lane / C::CPR) * C::VS + (lane % C::CPR) * 16);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      bad |= (w[i] & 0x7F800000u) == 0x7F800000u;
      if constexpr (C::KIND != kKindF32) bad |= (w[i] & 0x7F80u) == 0x7F80u;
    }
    const uint64_t b = __ballot(bad);
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if ((b >> (j * C::CPR)) & ROW) found |= 1u << (r + j);
  }
  return found;
}

// J tiles: scores, running reference, weights, sums. ALL: every row sees their tokens; else (one tile) seen: the
// tokens that the lane's row sees, and the tokens `apart` stay out of the matrix product and are added only to the
// rows that see them (a weight of 0 times a NaN is a NaN). c >= 0: scale * log2(e), its sign folded into Q.
template <class C, int J, bool ALL>
__device__ __forceinline__ void tile_step(AttendState<C>& st, const Piece (&qf)[C::NF], const char* lds, float c,
                                          uint32_t seen = 0, uint32_t apart = 0) {
  static_assert(ALL || J == 1, "partial sight goes tile by tile");
  const int lane = threadIdx.x & 63, hb = lane >> 5;
  f32x16 s[J];
  const char* kp = lds + (lane & 31) * C::KS + hb * 16;
  constexpr int KB = C::NF < 8 ? C::NF : 8;      // K fragments of a tile read together
#pragma unroll
  for (int i = 0; i < C::NF; i += KB) {
    Piece k[J][KB];
#pragma unroll
    for (int j = 0; j < KB; ++j)
#pragma unroll
      for (int t = 0; t < J; ++t) k[t][j].u = *reinterpret_cast<const uint4*>(kp + t * C::TILE + (i + j) * 32);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < KB; ++j)
#pragma unroll
      for (int t = 0; t < J; ++t) {
        if (i + j == 0)
#pragma unroll
          for (int e = 0; e < 16; ++e) s[t][e] = 0.0f;
        if constexpr (C::KIND == kKindF32) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[t] = __builtin_amdgcn_mfma_f32_32x32x2f32(k[t][j].f[e], qf[i + j].f[e], s[t], 0, 0, 0);
        } else {
          s[t] = mfma_32x32x16_bf16(k[t][j].h, qf[i + j].h, s[t]);
        }
      }
  }
  // the first V fragments come from LDS while the weights are computed
  const char* v = lds + 32 * C::KS;
  constexpr int VB = C::KIND == kKindF32 ? 0 : C::DP / 32 < 4 ? C::DP / 32 : 4;
  bf16x8 vf[VB > 0 ? VB : 1][2];
#pragma unroll
  for (int i = 0; i < VB; ++i)
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) vf[i][ks] = v_fragment<C>(v, ks, i);
  __builtin_amdgcn_sched_barrier(0);
  const float* sc = reinterpret_cast<const float*>(lds + 32 * (C::KS + C::VS));
  if constexpr (C::KIND == kKindE4M3) {
#pragma unroll
    for (int t = 0; t < J; ++t)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(sc + t * (C::TILE / 4) + 8 * g + 4 * hb);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][4 * g + e] *= x[e];
      }
  }
  auto sees = [&](int e) { return ((seen >> (8 * (e >> 2) + 4 * hb + (e & 3))) & 1) != 0; };
  if constexpr (!ALL) {
#pragma unroll
    for (int e = 0; e < 16; ++e) s[0][e] = sees(e) ? s[0][e] : -INFINITY;
  }
  float mq[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    mq[e] = s[0][e];
#pragma unroll
    for (int t = 0; t < J; ++t)
#pragma unroll
      for (int g = t == 0; g < 4; ++g) mq[e] = row_max(mq[e], s[t][4 * g + e]);
  }
  const float mx = half_max(row_max(row_max(mq[0], mq[1]), row_max(mq[2], mq[3])));
  const float m2 = mx == -INFINITY ? -INFINITY : mx * c;
  if (__any(m2 > st.m + 8.0f)) {
    const float mn = m2 > st.m + 8.0f ? m2 : st.m;      // by the row's own scores alone
    const float f = mn == st.m ? 1.0f : __builtin_amdgcn_exp2f(st.m - mn);
    st.m = mn;
    st.l *= f;
#pragma unroll
    for (int i = 0; i < C::DP / 32; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) st.o[i][e] *= f;
  }
  const float mr = st.m == -INFINITY ? 0.0f : st.m;
#pragma unroll
  for (int t = 0; t < J; ++t) {
    float p[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      p[e] = __builtin_amdgcn_exp2f(fmaf(s[t][e], c, -mr));
      if constexpr (!ALL) p[e] = sees(e) ? p[e] : 0.0f;
    }
    st.l += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7])) +
            (((p[8] + p[9]) + (p[10] + p[11])) + ((p[12] + p[13]) + (p[14] + p[15])));
    if constexpr (C::KIND == kKindE4M3) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(sc + t * (C::TILE / 4) + 32 + 8 * g + 4 * hb);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[4 * g + e] *= x[e];
          if (!ALL && !sees(4 * g + e)) p[4 * g + e] = 0.0f;   // its scale may be NaN
        }
      }
    }
    bf16x8 pb[2];
    if constexpr (C::KIND != kKindF32) {
#pragma unroll
      for (int e = 0; e < 16; ++e) pb[e >> 3][e & 7] = static_cast<__bf16>(p[e]);
    }
    const char* vt = v + t * C::TILE;
#pragma unroll
    for (int i = 0; i < C::DP / 32; ++i) {
      if constexpr (C::KIND == kKindF32) {
        st.o[i] = weighted_values_f32<C, !ALL>(vt, p, i, ~apart, st.o[i]);
      } else {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          bf16x8 x = t == 0 && i < VB ? vf[i < VB ? i : 0][ks] : v_fragment<C>(vt, ks, i);
          if constexpr (!ALL) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if ((apart >> (16 * ks + 8 * (e >> 2) + 4 * hb + (e & 3))) & 1) x[e] = static_cast<__bf16>(0.0f);
          }
          st.o[i] = mfma_32x32x16_bf16(x, pb[ks], st.o[i]);
        }
      }
    }
    if constexpr (!ALL) {
#pragma unroll 1
      while (apart) {
        const int tok = __builtin_ctz(apart), at = 4 * (tok >> 3) + (tok & 3);
        apart &= apart - 1;
        float w = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e) w = e == at ? p[e] : w;
        w = __shfl(w, (lane & 31) + 32 * ((tok >> 2) & 1), 64);
        if (!((seen >> tok) & 1)) continue;
        const char* row = v + tok * C::VS + 4 * hb * C::ES;
#pragma unroll
        for (int i = 0; i < C::DP / 32; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const char* x = row + (32 * i + 8 * (e >> 2) + (e & 3)) * C::ES;
            const float y = C::KIND == kKindF32 ? *reinterpret_cast<const float*>(x)
                                                : static_cast<float>(*reinterpret_cast<const __bf16*>(x));
            st.o[i][e] = fmaf(w, y, st.o[i][e]);
          }
      }
    }
  }
}

// Tokens of a 32-token tile from `base` that lie below lim.
__device__ __forceinline__ uint32_t below(int lim, int base) {
  const int n = lim - base;
  return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
}

// Four consecutive channels of one row.
template <int KIND>
__device__ __forceinline__ void store4(void* row, int c, f32x4 x, bool wide) {
  if constexpr (KIND == kKindF32) {
    float* p = static_cast<float*>(row) + c;
    if (wide) *reinterpret_cast<f32x4*>(p) = x;
    else {
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = x[e];
    }
  } else {
    union {
      __bf16 h[4];
      uint2 u;
    } y;
#pragma unroll
    for (int e = 0; e < 4; ++e) y.h[e] = static_cast<__bf16>(x[e]);
    __bf16* p = static_cast<__bf16*>(row) + c;
    if (wide) *reinterpret_cast<uint2*>(p) = y.u;
    else {
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = y.h[e];
    }
  }
}

struct AttendOut {
  float* o;     // [parts][rows][D], or null: the only part, written as the result
  float2* ml;   // [parts][rows]
  bool q_wide, out_wide;
};

template <int KIND>
__device__ __forceinline__ void finish_row4(const AttendArgs& a, int t, int h, int c, f32x4 x, float l, bool wide) {
  char* row = static_cast<char*>(a.q.out) + (t * a.q.out_t + h * a.q.out_h) * (KIND == kKindF32 ? 4 : 2);
  const float r = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = l == 0.0f ? 0.0f : x[e] * r;
  store4<KIND>(row, c, x, wide);
}
__device__ __forceinline__ float row_lse(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.69314718055994530942f;
}

template <class C>
__global__ __launch_bounds__(C::NT, C::BLOCKS) void attend_kernel(AttendArgs a, AttendPlan pl, AttendOut out) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, D = a.c.D, hkv = a.c.heads, Hq = a.q.heads, G = Hq / hkv;
  // ---- the item. Groups of 8 blocks (one per XCD) are prefix or own; the row tiles of a prefix range follow each
  // other on one XCD, whose L2 holds the range.
  const int grp = blockIdx.x >> 3, x8 = blockIdx.x & 7;
  const long long total = pl.pre_groups + pl.own_groups;
  const int pre_before = pl.pre_first ? min(grp, pl.pre_groups)
                                      : static_cast<int>(static_cast<long long>(grp) * pl.pre_groups / total);
  const bool own = pl.pre_first ? grp >= pl.pre_groups
                                : static_cast<int>(static_cast<long long>(grp + 1) * pl.pre_groups / total) == pre_before;
  const int g = own ? grp - pre_before : pre_before;
  const int tiles = own ? pl.own_tiles : pl.pre_tiles, pair = (g / tiles) * 8 + x8, tile = g % tiles;
  const int hk = pair % hkv, rest = pair / hkv;
  const int parts = own ? pl.own_parts : pl.pre_parts;
  const int part = rest % parts, b = own ? rest / parts : -1;
  if (own ? b >= a.B : rest >= parts) return;
  const bool shared = own ? pl.own_shared : pl.pre_shared;
  const int rows = own ? pl.own_rows : pl.pre_rows, row0 = tile * (shared ? 32 * C::NW : 32);
  const int n = own ? own_len(a, b) : a.P;
  const int chunk = own ? own_chunk(pl, n) : pl.pre_chunk;
  const long long first = static_cast<long long>(part) * chunk;
  if (first >= n && (out.o || part > 0)) return;
  const int j0 = static_cast<int>(first < n ? first : n);
  int j1 = n - j0 < chunk ? n : j0 + chunk;
  const int cut = own ? n - a.S + 1 : n;       // tokens below it are seen by every row
  if (own) {                                   // the tile's last row sees the most
    const int last = min(row0 + (shared ? 32 * C::NW : 32), rows) - 1;
    j1 = max(j0, min(j1, cut + last / G));
  }
  // ---- the lane's row
  const int r = row0 + (shared ? wave * 32 : 0) + (lane & 31);
  const bool live = r < rows;
  int t = 0, h = 0;
  if (live) row_token(a, G, b, r, t, h);
  const int lim = !live ? (own ? cut : n) : own ? cut + (t - b * a.S) : n;
  h += hk * G;
  const float cs = a.scale * 1.44269504088896340736f, c = fabsf(cs);
  Piece qf[C::NF];
  load_q<C>(a, static_cast<const char*>(a.q.in) + (t * a.q.in_t + h * a.q.in_h) * (C::KIND == kKindF32 ? 4 : 2), live,
            out.q_wide, cs < 0.0f, qf);
  AttendState<C> st;
  st.m = -INFINITY;
  st.l = 0.0f;
#pragma unroll
  for (int i = 0; i < C::DP / 32; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) st.o[i][e] = 0.0f;

  const int32_t* pages = own ? a.page_table + static_cast<long long>(b) * a.table_pages : a.prefix_pages;
  const int shift = 31 - __builtin_clz(a.c.page_size);
  // Table entry of token j, read ahead (of the last token for those past it); and the page of token j, -1 if there is
  // none. Apart, so that nothing waits for the entry while key loads are in flight.
  auto entry = [&](int j) { return pages[max(min(j, j1 - 1), 0) >> shift]; };
  auto page_of = [&](int e, int j) { return j < j1 && e >= 0 && e < a.c.n_pages ? e : -1; };
  // A tile that not every row sees whole: past the end, past `cut`, or with a page that is not in the cache.
  auto some_step = [&](const char* tl, int base, uint32_t exist) {
    const uint32_t apart = not_finite<C>(tl + 32 * C::KS) & ~below(cut, base);
    tile_step<C, 1, false>(st, qf, tl, c, exist & below(lim, base), apart);
  };
  const int whole = max(min(cut, j1) - j0, 0);      // tokens from j0 on that every row sees
  if (shared) {
    constexpr int STEP = 32 * C::SUB;
    const int steps = whole / STEP;
    int i = 0;
    auto token = [&](int i) { return lane < STEP ? min(j0 + i * STEP, j1) + lane : j1; };
    if (steps > 0) {
      Staged<C, C::SUB, C::NT> sg;
      auto all_there = [&] {
        uint32_t m = sg.mask[0];
#pragma unroll
        for (int s = 1; s < C::SUB; ++s) m &= sg.mask[s];
        return m == 0xFFFFFFFFu;
      };
      const int e0 = entry(token(0)), e1 = entry(token(1));
      int next_page = entry(token(2));
      sg.load(a, hk, j0, page_of(e0, token(0)), tid);
      bool here = all_there();
      sg.store(lds, D, tid);
      sg.load(a, hk, j0 + STEP, page_of(e1, token(1)), tid);
      __syncthreads();
#pragma unroll 1
      for (; i < steps && here; ++i) {
        // the other buffer was last read before the barrier that ended step i - 1
        int id = tid;       // opaque, so that the addresses are computed here and not kept in registers over the loop
        asm volatile("" : "+v"(id));
        here = all_there();
        int ahead = entry(token(i + 3));
        if (i + 1 < steps) {
          sg.store(lds + ((i + 1) & 1) * C::SUB * C::TILE, D, id);
          sg.load(a, hk, j0 + (i + 2) * STEP, page_of(next_page, token(i + 2)), id);
        }
        const char* tl = lds + (i & 1) * C::SUB * C::TILE;
        tile_step<C, C::SUB, true>(st, qf, tl, c);
        asm volatile("" : "+v"(ahead));      // waits for the entry here, with the key loads after it in flight
        next_page = ahead;
        __syncthreads();
      }
    }
    for (int j = j0 + i * STEP; j < j1; j += 32) {
      Staged<C, 1, C::NT> sg;
      const int tok = lane < 32 ? j + lane : j1;
      sg.load(a, hk, j, page_of(entry(tok), tok), tid);
      sg.store(lds, D, tid);
      __syncthreads();
      some_step(lds, j, sg.mask[0]);
      __syncthreads();
    }
  } else {
    // each wave takes every NW-th tile into an LDS tile of its own
    char* tl = lds + wave * C::TILE;
    const int tiles32 = (j1 - j0 + 31) >> 5, wholes = whole >> 5;
    auto token = [&](int i) { return lane < 32 ? min(j0 + i * 32, j1) + lane : j1; };
    Staged<C, 1, 64> sg;
    int next_page = 0, ahead = 0, i = wave;
    if (i < tiles32) {
      const int e = entry(token(i));
      next_page = entry(token(i + C::NW));
      sg.load(a, hk, j0 + i * 32, page_of(e, token(i)), lane);
    }
    auto turn = [&] {       // the tile in registers goes to LDS, the next one's loads are issued
      int ln = lane;        // opaque, so that the addresses are computed here and not kept in registers over the loop
      asm volatile("" : "+v"(ln));
      __builtin_amdgcn_wave_barrier();
      ahead = entry(token(i + 2 * C::NW));
      sg.store(tl, D, ln);
      __builtin_amdgcn_wave_barrier();
      if (i + C::NW < tiles32) sg.load(a, hk, j0 + (i + C::NW) * 32, page_of(next_page, token(i + C::NW)), ln);
    };
    auto settle = [&] {
      asm volatile("" : "+v"(ahead));      // waits for the entry here, with the key loads after it in flight
      next_page = ahead;
    };
#pragma unroll 1
    for (; i < wholes && sg.mask[0] == 0xFFFFFFFFu; i += C::NW) {
      turn();
      tile_step<C, 1, true>(st, qf, tl, c);
      settle();
    }
#pragma unroll 1
    for (; i < tiles32; i += C::NW) {
      const uint32_t exist = sg.mask[0];
      turn();
      if (exist) some_step(tl, j0 + i * 32, exist);
      settle();
    }
  }
  st.l = half_sum(st.l);

  const long long n_rows = static_cast<long long>(a.B) * a.S * Hq;
  const int hb = lane >> 5;
  if (shared) {
    if (!live) return;
    const long long row = static_cast<long long>(t) * Hq + h;
    if (out.o) {
      const long long at = static_cast<long long>(own ? pl.pre_parts + part : part) * n_rows + row;
      if (hb == 0) out.ml[at] = float2{st.m, st.l};
#pragma unroll
      for (int i = 0; i < C::DP / 32; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int ch = 32 * i + 8 * e + 4 * hb;
          if (ch < D)
            *reinterpret_cast<f32x4*>(out.o + at * D + ch) =
                f32x4{st.o[i][4 * e], st.o[i][4 * e + 1], st.o[i][4 * e + 2], st.o[i][4 * e + 3]};
        }
    } else {
      if (hb == 0 && a.lse) a.lse[row] = row_lse(st.m, st.l);
#pragma unroll
      for (int i = 0; i < C::DP / 32; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int ch = 32 * i + 8 * e + 4 * hb;
          if (ch < D)
            finish_row4<C::KIND>(a, t, h, ch,
                                 f32x4{st.o[i][4 * e], st.o[i][4 * e + 1], st.o[i][4 * e + 2], st.o[i][4 * e + 3]},
                                 st.l, out.out_wide);
        }
    }
    return;
  }
  // ---- join the waves' sums over their tiles
  __syncthreads();
  float* mo = reinterpret_cast<float*>(lds);                    // [NW][32][DP], then m and l [NW][32]
  float* mm = mo + C::NW * 32 * C::DP;
  if (hb == 0) {
    mm[wave * 32 + lane] = st.m;
    mm[(C::NW + wave) * 32 + lane] = st.l;
  }
#pragma unroll
  for (int i = 0; i < C::DP / 32; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<f32x4*>(mo + (wave * 32 + (lane & 31)) * C::DP + 32 * i + 8 * e + 4 * hb) =
          f32x4{st.o[i][4 * e], st.o[i][4 * e + 1], st.o[i][4 * e + 2], st.o[i][4 * e + 3]};
  __syncthreads();
  const int here = min(32, rows - row0), quads = D / 4;
  for (int e = tid; e < here * quads; e += C::NT) {
    const int rr = e / quads, ch = (e - rr * quads) * 4;
    float m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int w = 0; w < C::NW; ++w) m = fmaxf(m, mm[w * 32 + rr]);
    f32x4 x = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < C::NW; ++w) {
      const float lw = mm[(C::NW + w) * 32 + rr];
      const float f = lw == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(mm[w * 32 + rr] - m);
      l += f * lw;
      const f32x4 y = *reinterpret_cast<const f32x4*>(mo + (w * 32 + rr) * C::DP + ch);
#pragma unroll
      for (int q = 0; q < 4; ++q) x[q] += lw == 0.0f ? 0.0f : f * y[q];
    }
    int tt, hh;
    row_token(a, G, b, row0 + rr, tt, hh);
    hh += hk * G;
    const long long row = static_cast<long long>(tt) * Hq + hh;
    if (out.o) {
      const long long at = static_cast<long long>(own ? pl.pre_parts + part : part) * n_rows + row;
      if (ch == 0) out.ml[at] = float2{m, l};
      *reinterpret_cast<f32x4*>(out.o + at * D + ch) = x;
    } else {
      if (ch == 0 && a.lse) a.lse[row] = row_lse(m, l);
      finish_row4<C::KIND>(a, tt, hh, ch, x, l, out.out_wide);
    }
  }
}

// out_r = sum_parts 2^(m_i - M) o_i / sum_parts 2^(m_i - M) l_i. LPR lanes per row, four channels each; with many
// parts a block takes one row, its 256 / LPR lane groups every 256 / LPR-th part, and the groups' sums meet in LDS.
template <int KIND, int LPR, bool MANY>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a, AttendPlan pl, AttendOut out) {
  constexpr int GROUPS = MANY ? 256 / LPR : 1;
  __shared__ f32x4 sx[MANY ? 256 : 1];
  __shared__ float sl[MANY ? GROUPS : 1];
  const int Hq = a.q.heads, D = a.c.D, grp = MANY ? threadIdx.x / LPR : 0;
  const long long n_rows = static_cast<long long>(a.B) * a.S * Hq;
  const long long row = MANY ? blockIdx.x : (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) / LPR;
  if (row >= n_rows) return;
  const int ch = (threadIdx.x % LPR) * 4, t = static_cast<int>(row / Hq), h = static_cast<int>(row - static_cast<long long>(t) * Hq);
  int parts = pl.pre_parts;
  if (pl.own_parts > 0) {
    const int n = own_len(a, t / a.S), chunk = own_chunk(pl, n);
    if (n > 0) parts += (n + chunk - 1) / chunk;
  }
  float m = -INFINITY, l = 0.0f;
#pragma unroll 4
  for (int i = 0; i < parts; ++i) m = fmaxf(m, out.ml[i * n_rows + row].x);
  f32x4 x = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int i = grp; i < parts; i += GROUPS) {
    const float2 ml = out.ml[i * n_rows + row];
    f32x4 y = x;
    if (ch < D) y = *reinterpret_cast<const f32x4*>(out.o + (i * n_rows + row) * D + ch);
    const float f = ml.y == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(ml.x - m);
    l += ml.y == 0.0f ? 0.0f : f * ml.y;
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] += ml.y == 0.0f ? 0.0f : f * y[q];      // a part without tokens left y unset
  }
  if constexpr (MANY) {
    sx[threadIdx.x] = x;
    if (threadIdx.x % LPR == 0) sl[grp] = l;
    __syncthreads();
    if (grp) return;
#pragma unroll
    for (int g = 1; g < GROUPS; ++g) {
      const f32x4 y = sx[g * LPR + threadIdx.x];
#pragma unroll
      for (int q = 0; q < 4; ++q) x[q] += y[q];
      l += sl[g];
    }
  }
  if (ch < D) finish_row4<KIND>(a, t, h, ch, x, l, out.out_wide);
  if (ch == 0 && a.lse) a.lse[row] = row_lse(m, l);
}

// The split. A stream whose rows fit one 32-row tile is read by each wave on its own (more loads in flight);
// with more rows the waves share the tiles and take 32 rows each.
// The prefix items should last as long as the call and leave the own items, bound by HBM, the slots that these
// need to keep pace: the prefix gets the share of the block slots that its time has of the sum of both
// (matrix rate against read rate), as one item a slot, first in the grid. Where there are more prefix items
// than slots, the two kinds alternate. Own ranges are cut until their items fill the slots several times
// over; no range is below kMinTokens, so that a part's sums (4 D bytes a row) stay small beside its keys.
constexpr int kMinTokens = 256;

template <class C>
static AttendPlan attend_plan(const Cache& c, int B, int S, int Hq, int P, int table_pages) {
  AttendPlan p{};
  const int G = Hq / c.heads;
  const long long slots = static_cast<long long>(device_cu_count()) * C::BLOCKS;
  const long long own_max = static_cast<long long>(table_pages) * c.page_size;
  auto cdivl = [](long long x, long long y) { return (x + y - 1) / y; };
  auto parts_of = [&](long long base, long long tokens, long long want) {
    long long n = cdivl(want, base);
    const long long most = cdivl(tokens, kMinTokens);
    n = n < most ? n : most;
    return static_cast<int>(n < 1 ? 1 : n > 256 ? 256 : n);
  };
  if (P > 0) {
    p.pre_rows = B * S * G;
    p.pre_shared = p.pre_rows > 32;
    p.pre_tiles = static_cast<int>(cdivl(p.pre_rows, p.pre_shared ? 32 * C::NW : 32));
    const double flop_us = C::KIND == kKindF32 ? 1e8 : 6e8, byte_us = 5e6;     // rates reached, per microsecond
    const double row_bytes = 2.0 * c.D * (C::KIND == kKindF32 ? 4 : C::KIND == kKindBf16 ? 2 : 1);
    double pre = 4.0 * C::DP * p.pre_tiles * (p.pre_shared ? 32 * C::NW : 32) * P / flop_us;
    if (!p.pre_shared) pre = row_bytes * P / byte_us;
    const double own = row_bytes * B * (own_max / 2) / byte_us;
    const long long base = static_cast<long long>(p.pre_tiles) * c.heads;
    const double share = static_cast<double>(slots) * pre / (pre + own) / base;
    p.pre_parts = parts_of(base, P, base * (share < 1 ? 1 : static_cast<long long>(share)));
    p.pre_chunk = static_cast<int>(cdivl(cdivl(P, p.pre_parts), 64) * 64);
    p.pre_parts = static_cast<int>(cdivl(P, p.pre_chunk));
    p.pre_groups = static_cast<int>(cdivl(static_cast<long long>(p.pre_parts) * c.heads, 8) * p.pre_tiles);
    p.pre_first = 8LL * p.pre_groups <= slots;
  }
  if (own_max > 0) {
    p.own_rows = S * G;
    p.own_shared = p.own_rows > 32;
    p.own_tiles = static_cast<int>(cdivl(p.own_rows, p.own_shared ? 32 * C::NW : 32));
    const long long pairs = static_cast<long long>(B) * c.heads;
    p.own_parts = parts_of(pairs * p.own_tiles, own_max, 4 * slots);
    p.own_groups = static_cast<int>(cdivl(pairs * p.own_parts, 8) * p.own_tiles);
  }
  return p;
}

template <class F>
static auto with_cfg(moe_dtype cache, int D, F f) {
  auto by_dim = [&](auto kind) {
    constexpr int K = decltype(kind)::value;
    if (D <= 64) return f(AttendCfg<K, 64>{});
    if (D <= 128) return f(AttendCfg<K, 128>{});
    return f(AttendCfg<K, 256>{});
  };
  if (cache == MOE_F32) return by_dim(std::integral_constant<int, kKindF32>{});
  if (cache == MOE_BF16) return by_dim(std::integral_constant<int, kKindBf16>{});
  return by_dim(std::integral_constant<int, kKindE4M3>{});
}

static size_t parts_bytes(const AttendPlan& p, long long rows, int D) {
  const int parts = p.pre_parts + p.own_parts;
  return parts > 1 ? static_cast<size_t>(parts) * rows * (4 * D + 8) : 0;
}

size_t attend_ws_bytes(const Cache& c, int B, int S, int Hq, int P, int table_pages) {
  if (B == 0 || S == 0) return 256;
  return with_cfg(c.dtype, c.D, [&](auto cfg) {
    return 256 + parts_bytes(attend_plan<decltype(cfg)>(c, B, S, Hq, P, table_pages), static_cast<long long>(B) * S * Hq, c.D);
  });
}

template <class K>
static hipError_t allow_lds(K kern, int bytes) {
  return hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

hipError_t launch_attend(const AttendArgs& a, hipStream_t st) {
  return with_cfg(a.c.dtype, a.c.D, [&](auto cfg) {
    using C = decltype(cfg);
    AttendPlan p = attend_plan<C>(a.c, a.B, a.S, a.q.heads, a.P, a.table_pages);
    const long long rows = static_cast<long long>(a.B) * a.S * a.q.heads;
    const bool direct = p.pre_parts + p.own_parts <= 1;
    if (p.pre_groups + p.own_groups == 0) {       // no prefix and no own pages: every row sees nothing
      p.own_rows = a.S * (a.q.heads / a.c.heads);
      p.own_shared = 1;
      p.own_tiles = cdiv(p.own_rows, 32 * C::NW);
      p.own_parts = 1;
      p.own_groups = cdiv(a.B * a.c.heads, 8) * p.own_tiles;
    }
    const uintptr_t ob = reinterpret_cast<uintptr_t>(a.q.out), qb = reinterpret_cast<uintptr_t>(a.q.in);
    const int es = C::KIND == kKindF32 ? 4 : 2;
    AttendOut out{};
    out.q_wide = qb % 16 == 0 && a.q.in_t * es % 16 == 0 && a.q.in_h * es % 16 == 0;
    out.out_wide = ob % (4 * es) == 0 && a.q.out_t % 4 == 0 && a.q.out_h % 4 == 0;
    if (!direct) {
      out.o = static_cast<float*>(a.ws);
      out.ml = reinterpret_cast<float2*>(out.o + static_cast<long long>(p.pre_parts + p.own_parts) * rows * a.c.D);
    }
    static const hipError_t allowed = allow_lds(attend_kernel<C>, C::LDS);
    if (allowed != hipSuccess) return allowed;
    hipLaunchKernelGGL(attend_kernel<C>, dim3(8u * (p.pre_groups + p.own_groups)), dim3(C::NT), C::LDS, st, a, p, out);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || direct) return e;
    constexpr int LPR = C::DP / 4;
    if (p.pre_parts + p.own_parts > 256 / LPR)
      hipLaunchKernelGGL((attend_join_kernel<C::KIND, LPR, true>), dim3(static_cast<unsigned>(rows)), dim3(256), 0, st, a, p,
                         out);
    else
      hipLaunchKernelGGL((attend_join_kernel<C::KIND, LPR, false>), dim3(static_cast<unsigned>((rows * LPR + 255) / 256)),
                         dim3(256), 0, st, a, p, out);
    return hipGetLastError();
  });
}

}  // namespace moe
