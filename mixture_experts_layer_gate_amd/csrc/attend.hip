// Attention over the paged cache for sequences that share a prefix:
//   out_r = sum_j exp(s_rj - m) v_j / sum_j exp(s_rj - m),  s_rj = scale q_r . k_j,
// in one pass over the keys with a running reference m, sums in fp32.
//
// Bound by HBM for a sequence's own tokens (4.6 to 5.9 TB/s from 4000 tokens up) and by the matrix units
// and exponentials for a prefix that many rows share (620 to 640 TFLOP/s on 131071 tokens with 256 rows a head).
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
// A row's reference m is moved (and its sums rescaled) only when a score passes it by 8 (base 2), or, in the loop
// over shared tiles, when the weights of a half wave's 16 tokens add up to more than 2^12. Weights and sums are relative
// to m, so the result does not depend on m while both stay finite. Rounding the weights (of E4M3 values, times their
// scales) to bf16 for the second product, as its operand has to be, costs half a bf16 unit of each, as the values' own
// rounding did; their sum is taken in fp32 before it. Relative error against 64 bits, beside that of fp32 weights: on some
// thousand tokens 0.0017 and 0.0017 (bf16), 0.0018 and 0.0017 (E4M3); on up to 64 tokens 0.0018 and 0.0016, 0.0023 and 0.0017.
#include <type_traits>

#include "heads.h"

namespace moe {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// E4M3 codes come in pieces of 16, or of 8 where head_dim is no multiple of 16.
enum { kKindF32 = 0, kKindBf16 = 1, kKindE4M3 = 2, kKindE4M3Narrow = 3 };

template <int KIND_, int DP_>
struct AttendCfg {
  static constexpr int KIND = KIND_, DP = DP_;                 // channels, padded to 64, 128 or 256
  static constexpr bool Q8 = KIND >= kKindE4M3;
  static constexpr int ES = KIND == kKindF32 ? 4 : 2;          // bytes of an element in LDS
  static constexpr int NW = 2, NT = NW * 64;                   // waves of a block
  static constexpr int RW = KIND == kKindF32 || DP == 256 ? 1 : 2;   // row tiles of a wave on shared key tiles
  static constexpr int ROWS = NW * RW * 32;                    // rows of a block there
  // Rows of K are read 16 bytes per lane down 32 rows, rows of V as 4 rows x 32 bytes (transposing reads) or
  // along the row (fp32): a row stride of 16 (64) bytes past a multiple of 128 spreads them over the banks.
  static constexpr int KS = DP * ES + 16, VS = DP * ES + (ES == 2 ? 64 : 16);
  static constexpr int TILE = 32 * (KS + VS) + (Q8 ? 256 : 0);   // 32 tokens (and their scales)
  static constexpr int RING = KIND != kKindF32 && DP <= 128 ? 4 : 2;   // slots of the shared tiles
  static constexpr int LDS_MERGE = NW * 32 * (DP + 2) * 4;
  static constexpr int LDS_TILES = (RING > NW ? RING : NW) * TILE;
  static constexpr int LDS = LDS_TILES > LDS_MERGE ? LDS_TILES : LDS_MERGE;
  static constexpr int LDS_ALONE = NW * TILE > LDS_MERGE ? NW * TILE : LDS_MERGE;
  // Blocks of a CU, waves of a SIMD (512, 256 or 168 registers each), with shared tiles in the call or without: without,
  // two waves a SIMD fit with 128 channels of 16- or 8-bit tokens, three with 64; fp32 has two with 64 either way, and one
  // from 128 up, as have the others from 256 up (8-bit tokens, 64 sequences of up to 4000: 93 -> 83 us, of 64 channels
  // 66 -> 47 us; 243 sequences of up to 23 tokens: 18 -> 12 us).
  static constexpr int blocks(bool shared) {
    const int bytes = shared ? LDS : LDS_ALONE;
    return !shared && bytes <= 26 * 1024 ? 6 : bytes <= 40 * 1024 ? 4 : bytes <= 80 * 1024 ? 2 : 1;
  }
  static constexpr int eu_waves(bool shared) { return blocks(shared) * NW >= 12 ? 3 : blocks(shared) * NW >= 8 ? 2 : 1; }
  static constexpr int QE = KIND == kKindF32 ? 4 : 8;          // elements of 16 LDS bytes
  static constexpr int CE = KIND == kKindE4M3 ? 16 : QE;       // elements of a load (a piece)
  static constexpr int CPR = DP / CE;                          // pieces of a row
  static constexpr int NF = DP / 16 * (KIND == kKindF32 ? 2 : 1);   // 16-byte fragments of a lane's K or Q row half
  // Rows of a stream that the waves read on their own. A wave of 256 fp32 channels has no registers for a whole
  // tile on its way: its streams are shared.
  static constexpr int ALONE_ROWS = KIND == kKindF32 && DP == 256 ? 0 : 64;
  static_assert(LDS <= 160 * 1024, "LDS");
};

// The split of one call, decided on the host from sizes alone.
struct AttendPlan {
  int pre_rows, own_rows;        // rows of a stream
  int pre_shared, own_shared;    // 1: the waves of a block share the key tiles and have RW * 32 rows each
  int pre_tiles, own_tiles;      // row tiles
  int pre_parts, own_parts;      // ranges of tokens
  int pre_chunk;                 // tokens of a prefix part (multiple of 64)
  int pre_groups, own_groups;    // groups of 8 blocks
  int own_sorted;                // 1: the longest sequences first
};

__device__ __forceinline__ int own_len(const AttendArgs& a, int b) {
  if (a.table_pages <= 0) return 0;
  const long long cap = static_cast<long long>(a.table_pages) * a.c.page_size;
  return clampi(a.lens[b], 0, static_cast<int>(cap));
}
// The sequence that comes at `rank` when the longest come first (by sixteenths of the longest one's length, in order
// within one), so that the blocks started last have little to do. Every block works it out, from one load.
constexpr int kSortedMost = 128;
__device__ __forceinline__ int longest_first(const AttendArgs& a, int rank) {
  const int lane = threadIdx.x & 63;
  const int n0 = own_len(a, min(lane, a.B - 1)), n1 = own_len(a, min(64 + lane, a.B - 1));
  int most = max(n0, n1);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) most = max(most, __shfl_xor(most, o, kWave));
  const float f = 16.0f / (most + 1.0f);
  const int k0 = lane < a.B ? min(static_cast<int>(n0 * f), 15) : -1;
  const int k1 = 64 + lane < a.B ? min(static_cast<int>(n1 * f), 15) : -1;
  auto nth = [&](uint64_t in, int n) {
    const int before = __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(in >> 32),
                                                 __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(in), 0));
    return __builtin_ctzll(__ballot(before == n && ((in >> lane) & 1)));
  };
#pragma unroll 1
  for (int k = 15; k >= 0; --k) {
    const uint64_t in0 = __ballot(k0 == k), in1 = __ballot(k1 == k);
    const int c0 = __popcll(in0), c1 = __popcll(in1);
    if (rank < c0) return nth(in0, rank);
    if (rank < c0 + c1) return 64 + nth(in1, rank - c0);
    rank -= c0 + c1;
  }
  return 0;      // not reached: rank < B
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

template <class C, int R>
struct AttendState {
  f32x16 o[R][C::DP / 32];   // O^T: channel 32 i + 8 (v / 4) + 4 (lane / 32) + v % 4 of row lane % 32 of tile r
  float m[R], l[R];          // reference (base 2) and this half wave's part of the sum
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.0f;
#pragma unroll
      for (int i = 0; i < C::DP / 32; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[r][i][e] = 0.0f;
    }
  }
};

// The lane's Q fragments: its row's channels in the order the K fragments have them, negated if neg.
template <class C>
__device__ __forceinline__ void load_q(const AttendArgs& a, const void* row, bool live, bool wide, bool neg,
                                       Piece (&qf)[C::NF]) {
  const int hb = (threadIdx.x >> 5) & 1, D = a.c.D;
#pragma unroll
  for (int s = 0; s < C::NF; ++s) {
    const int d0 = (2 * s + hb) * C::QE;
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

// The page table ahead of a wave: entry base + lane in cur, base + 64 + lane in next. Tiles only go forward, and after
// go() a tile's pages (a power of two of them, or part of one) lie in cur.
struct PageWalk {
  const int32_t* pages;
  int last, base, cur, next;
  __device__ __forceinline__ void start(const int32_t* p, int first_page, int last_page) {
    pages = p;
    last = last_page;
    base = first_page;
    cur = pages[min(base + static_cast<int>(threadIdx.x & 63), last)];
    next = pages[min(base + 64 + static_cast<int>(threadIdx.x & 63), last)];
  }
  __device__ __forceinline__ void go(int page) {
    while (page - base >= 64) {
      base += 64;
      cur = next;
      next = pages[min(base + 64 + static_cast<int>(threadIdx.x & 63), last)];
    }
  }
};

// Pieces of K and V of a tile on their way from the cache to LDS, in registers; TH threads take part.
// Piece q of thread i is piece e % CPR of token e / CPR, e = q TH + i.
template <class C, int TH>
struct Staged {
  static constexpr int N = 32 * C::CPR / TH;
  static constexpr bool Q8 = C::Q8;
  typedef typename std::conditional<C::KIND == kKindE4M3Narrow, uint2, uint4>::type Raw;
  static constexpr int LB = C::CE * C::ES;      // LDS bytes of a piece
  Raw k[N], v[N];
  float ks, vs;
  uint32_t mask;      // tokens that exist

  // A whole tile, piece by piece (n < 2 N: K, then V). `Source`: where its pieces are, in scalar registers.
  struct Source {
    uint64_t off[N];
    bool ok;      // every page is in the cache; else page 0, which exists, is read in its place
  };
  __device__ __forceinline__ static Source source(const AttendArgs& a, int base, int shift, const PageWalk& walk, int i) {
    const uint32_t ps = a.c.page_size, row_bytes = a.c.D * (Q8 ? 1 : C::ES), page_bytes = a.c.heads * ps * row_bytes;
    const uint32_t first = __builtin_amdgcn_readfirstlane(i / C::CPR), n_pages = a.c.n_pages;
    Source s;
    auto page_at = [&](uint32_t tok) {
      const uint32_t p = __builtin_amdgcn_readlane(walk.cur, (tok >> shift) - walk.base);
      return static_cast<uint64_t>(p < n_pages ? p : 0) * page_bytes + (tok & (ps - 1)) * row_bytes;
    };
    // All of the tile's pages, not those of this wave's loads alone: the waves of a block have to agree.
    const uint64_t out = __ballot(static_cast<uint32_t>(walk.cur) >= n_pages) >> ((base >> shift) - walk.base);
    s.ok = (out & (ps >= 32 ? 1ull : (1ull << (32 >> shift)) - 1)) == 0;
    if (ps >= 32) {      // the tile lies in one page
      const uint64_t off = page_at(base) + first * row_bytes;
#pragma unroll
      for (int q = 0; q < N; ++q) s.off[q] = off + q * (TH / C::CPR) * row_bytes;
    } else {             // each load of a wave does
#pragma unroll
      for (int q = 0; q < N; ++q) s.off[q] = page_at(base + q * (TH / C::CPR) + first);
    }
    return s;
  }
  // The lane's part of a piece's address in the cache.
  __device__ __forceinline__ static uint32_t lane_offset(const AttendArgs& a, int hk, int i) {
    const uint32_t row_bytes = a.c.D * (Q8 ? 1 : C::ES);
    const int c = (i % C::CPR) * C::CE;
    return hk * a.c.page_size * row_bytes + (c < a.c.D ? c : 0) * (Q8 ? 1 : C::ES) + (i % 64 / C::CPR) * row_bytes;
  }
  __device__ __forceinline__ void load_piece(const AttendArgs& a, const Source& s, uint32_t lane_off, int n) {
    const char* p = static_cast<const char*>(n < N ? a.c.k : a.c.v) + s.off[n % N];
    (n < N ? k : v)[n % N] = *reinterpret_cast<const Raw*>(p + lane_off);
  }
  __device__ __forceinline__ void load_scales(const AttendArgs& a, int hk, int base, int shift, const PageWalk& walk) {
    if constexpr (Q8) {
      const uint32_t ps = a.c.page_size, tok = base + (threadIdx.x & 31);
      uint32_t page = __shfl(walk.cur, (tok >> shift) - walk.base, 64);
      page = page < static_cast<uint32_t>(a.c.n_pages) ? page : 0;
      const uint64_t row = static_cast<uint64_t>(page) * (a.c.heads * ps) + (hk * ps + (tok & (ps - 1)));
      ks = a.c.k_scale[row];
      vs = a.c.v_scale[row];
    }
  }
  // The thread's places for K and V in an LDS tile.
  __device__ __forceinline__ static uint32_t k_place(int i) { return i / C::CPR * C::KS + i % C::CPR * LB; }
  __device__ __forceinline__ static uint32_t v_place(int i) { return 32 * C::KS + i / C::CPR * C::VS + i % C::CPR * LB; }
  // A piece as LDS holds it, 16 bytes at a time; `on` masks it.
  __device__ __forceinline__ static void write(char* at, Raw x, uint32_t on) {
#pragma unroll
    for (int b = 0; b < LB / 16; ++b) {
      Piece y;
      if constexpr (C::KIND == kKindE4M3) y.h = e4m3x8_to_bf16(b ? uint2{x.z, x.w} : uint2{x.x, x.y});
      else if constexpr (Q8) y.h = e4m3x8_to_bf16(uint2{x.x, x.y});
      else y.u = x;
      *reinterpret_cast<uint4*>(at + 16 * b) = uint4{y.u.x & on, y.u.y & on, y.u.z & on, y.u.w & on};
    }
  }
  __device__ __forceinline__ void store_piece(char* k_at, char* v_at, int n) const {
    write(n < N ? k_at + n * (TH / C::CPR) * C::KS : v_at + (n - N) * (TH / C::CPR) * C::VS, (n < N ? k : v)[n % N],
          0xFFFFFFFFu);
  }
  __device__ __forceinline__ void store_scales(char* tile, int i) const {
    if constexpr (Q8) {
      if (i < 32) {
        float* sc = reinterpret_cast<float*>(tile + 32 * (C::KS + C::VS));
        sc[i] = ks;
        sc[32 + i] = vs;
      }
    }
  }
  // All of a whole tile.
  __device__ __forceinline__ bool load_whole(const AttendArgs& a, int hk, int base, int shift, const PageWalk& walk, int i) {
    const Source s = source(a, base, shift, walk, i);
    const uint32_t off = lane_offset(a, hk, i);
#pragma unroll
    for (int n = 0; n < 2 * N; ++n) load_piece(a, s, off, n);
    load_scales(a, hk, base, shift, walk);
    mask = 0xFFFFFFFFu;
    return s.ok;
  }

  // page: page of token base + lane (first 32 lanes), -1 where there is no such token. Missing tokens read
  // page 0, which exists, and are cleared by store.
  __device__ __forceinline__ void load(const AttendArgs& a, int hk, int base, int page, int i) {
    mask = static_cast<uint32_t>(__ballot(page >= 0));
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
      const int tok = q * (TH / C::CPR) + i / C::CPR;
      char* t = lds + tok * C::KS + p * LB;
      const uint32_t on = WHOLE || (p * C::CE < D && ((mask >> tok) & 1)) ? 0xFFFFFFFFu : 0u;
      write(t, k[q], on);
      write(t + 32 * C::KS + tok * (C::VS - C::KS), v[q], on);
    }
  }
  __device__ __forceinline__ void store(char* lds, int D, int i) const {
    if (D == C::DP && mask == 0xFFFFFFFFu) put<true>(lds, D, i);
    else put<false>(lds, D, i);
    store_scales(lds, i);
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
  constexpr int LP = C::DP / C::QE, PER = 64 / LP;      // rows that the wave looks at together
  constexpr uint64_t ROW = LP == 64 ? ~0ull : (1ull << (LP & 63)) - 1;
  uint32_t found = 0;
#pragma unroll 1
  for (int r = 0; r < 32; r += PER) {
    const uint4 x = *reinterpret_cast<const uint4*>(v + (r + lane / LP) * C::VS + (lane % LP) * 16);
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
      if ((b >> (j * LP)) & ROW) found |= 1u << (r + j);
  }
  return found;
}

// K fragments of a tile: 16 bytes down each of the 32 rows, in the order of Q's.
template <class C>
__device__ __forceinline__ void read_k(const char* lds, Piece (&k)[C::NF]) {
  const int lane = threadIdx.x & 63;
  const char* p = lds + (lane & 31) * C::KS + (lane >> 5) * 16;
#pragma unroll
  for (int i = 0; i < C::NF; ++i) k[i].u = *reinterpret_cast<const uint4*>(p + i * 32);
}

template <class C>
__device__ __forceinline__ f32x16 add_product(const Piece& k, const Piece& q, f32x16 s) {
  if constexpr (C::KIND == kKindF32) {
#pragma unroll
    for (int e = 0; e < 4; ++e) s = __builtin_amdgcn_mfma_f32_32x32x2f32(k.f[e], q.f[e], s, 0, 0, 0);
    return s;
  } else {
    return mfma_32x32x16_bf16(k.h, q.h, s);
  }
}

// Scores of a tile: the lane's 16 of each of R row tiles.
template <int R>
struct Scores {
  f32x16 s[R];
};

// S^T = K Q^T of a tile.
template <class C, int R>
__device__ __forceinline__ void products(const Piece (&k)[C::NF], const Piece (&qf)[R][C::NF], Scores<R>& x) {
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int e = 0; e < 16; ++e) x.s[r][e] = 0.0f;
#pragma unroll
  for (int i = 0; i < C::NF; ++i)
#pragma unroll
    for (int r = 0; r < R; ++r) x.s[r] = add_product<C>(k[i], qf[r][i], x.s[r]);
}

// The keys' scales (E4M3) and the mask of a partial tile.
template <class C, int R, bool ALL>
__device__ __forceinline__ void finish_scores(Scores<R>& x, const char* lds, const uint32_t (&seen)[R]) {
  const int hb = (threadIdx.x >> 5) & 1;
  if constexpr (C::Q8) {
    const float* sc = reinterpret_cast<const float*>(lds + 32 * (C::KS + C::VS));
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const f32x4 y = *reinterpret_cast<const f32x4*>(sc + 8 * g + 4 * hb);
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) x.s[r][4 * g + e] *= y[e];
    }
  }
  if constexpr (!ALL) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < 16; ++e)
        x.s[r][e] = (seen[r] >> (8 * (e >> 2) + 4 * hb + (e & 3))) & 1 ? x.s[r][e] : -INFINITY;
  }
}
// Moves the rows' references to their scores' maxima where these pass them by 2^8 (by each row's own scores alone).
template <class C, int R>
__device__ __forceinline__ void raise_reference(AttendState<C, R>& st, const float (&m2)[R]) {
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float mn = m2[r] > st.m[r] + 8.0f ? m2[r] : st.m[r];
    const float f = mn == st.m[r] ? 1.0f : __builtin_amdgcn_exp2f(st.m[r] - mn);
    st.m[r] = mn;
    st.l[r] *= f;
#pragma unroll
    for (int i = 0; i < C::DP / 32; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) st.o[r][i][e] *= f;
  }
}
template <int R>
__device__ __forceinline__ void row_maxima(const Scores<R>& x, float c, float (&m2)[R]) {
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float mq[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) mq[e] = row_max(row_max(x.s[r][e], x.s[r][4 + e]), row_max(x.s[r][8 + e], x.s[r][12 + e]));
    const float mx = half_max(row_max(row_max(mq[0], mq[1]), row_max(mq[2], mq[3])));
    m2[r] = mx == -INFINITY ? -INFINITY : mx * c;
  }
}

// One tile's scores: running reference, weights, sums. ALL: every row sees its tokens; else seen: the
// tokens that the lane's row sees, and the tokens `apart` stay out of the matrix product and are added only to the
// rows that see them (a weight of 0 times a NaN is a NaN). c >= 0: scale * log2(e), its sign folded into Q.
template <class C, int R, bool ALL>
__device__ __forceinline__ void tile_sums(AttendState<C, R>& st, const Scores<R>& x, const char* lds, float c,
                                          const uint32_t (&seen)[R], uint32_t apart) {
  const int lane = threadIdx.x & 63, hb = lane >> 5;
  const char* v = lds + 32 * C::KS;
  const float* sc = reinterpret_cast<const float*>(lds + 32 * (C::KS + C::VS));
  constexpr int NB = C::DP / 32, VB = C::KIND == kKindF32 ? 0 : NB < 4 ? NB : 4;
  bf16x8 vf[VB > 0 ? VB : 1][2];      // the first V fragments come from LDS while the weights are computed
#pragma unroll
  for (int ks = 0; ks < 2; ++ks)
#pragma unroll
    for (int i = 0; i < VB; ++i) vf[i][ks] = v_fragment<C>(v, ks, i);
  f32x4 vs[4];
  if constexpr (C::Q8) {
#pragma unroll
    for (int g = 0; g < 4; ++g) vs[g] = *reinterpret_cast<const f32x4*>(sc + 32 + 8 * g + 4 * hb);
  }
  float m2[R];
  bool up = false;
  row_maxima<R>(x, c, m2);
#pragma unroll
  for (int r = 0; r < R; ++r) up = up || m2[r] > st.m[r] + 8.0f;
  if (__any(up)) raise_reference<C, R>(st, m2);
  auto sees = [&](int r, int e) { return ((seen[r] >> (8 * (e >> 2) + 4 * hb + (e & 3))) & 1) != 0; };
  float pv[R][16];      // weights times the values' scales
  bf16x8 pb[R][2];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float mr = st.m[r] == -INFINITY ? 0.0f : st.m[r];
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float p = __builtin_amdgcn_exp2f(fmaf(x.s[r][e], c, -mr));
      if constexpr (!ALL) p = sees(r, e) ? p : 0.0f;
      sum[e & 3] += p;
      if constexpr (C::Q8) {
        p *= vs[e >> 2][e & 3];
        if (!ALL && !sees(r, e)) p = 0.0f;      // its scale may be NaN
      }
      pv[r][e] = p;
      if constexpr (C::KIND != kKindF32) pb[r][e >> 3][e & 7] = static_cast<__bf16>(p);
    }
    st.l[r] += (sum[0] + sum[1]) + (sum[2] + sum[3]);
  }
  if constexpr (C::KIND == kKindF32) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < NB; ++i) st.o[r][i] = weighted_values_f32<C, !ALL>(v, pv[r], i, ~apart, st.o[r][i]);
  } else {
#pragma unroll
    for (int n = 0; n < 2 * NB; ++n) {
      const int ks = n / NB, i = n % NB;
      bf16x8 z = i < VB ? vf[i < VB ? i : 0][ks] : v_fragment<C>(v, ks, i);
      if constexpr (!ALL) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if ((apart >> (16 * ks + 8 * (e >> 2) + 4 * hb + (e & 3))) & 1) z[e] = static_cast<__bf16>(0.0f);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) st.o[r][i] = mfma_32x32x16_bf16(z, pb[r][ks], st.o[r][i]);
    }
  }
  if constexpr (!ALL) {
#pragma unroll 1
    while (apart) {
      const int tok = __builtin_ctz(apart), at = 4 * (tok >> 3) + (tok & 3);
      apart &= apart - 1;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float w = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; ++e) w = e == at ? pv[r][e] : w;
        w = __shfl(w, (lane & 31) + 32 * ((tok >> 2) & 1), 64);
        if (!((seen[r] >> tok) & 1)) continue;
        const char* row = v + tok * C::VS + 4 * hb * C::ES;
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const char* z = row + (32 * i + 8 * (e >> 2) + (e & 3)) * C::ES;
            const float val = C::KIND == kKindF32 ? *reinterpret_cast<const float*>(z)
                                                  : static_cast<float>(*reinterpret_cast<const __bf16*>(z));
            st.o[r][i][e] = fmaf(w, val, st.o[r][i][e]);
          }
      }
    }
  }
}

// The sums of a whole tile (at lds) and the scores of the one after it, whose K fragments k holds (and whose scales
// lie at lds1); then k gets those of the second tile after it (at lds2). x: the tile's scores, replaced by the next.
//
// A wave has a SIMD to itself here (its sums, Q and K fragments and two tiles on their way take 450 registers), so
// nothing else fills its gaps and the order is fixed by hand: between two matrix instructions (32 cycles)
// a few of the vector ones that need neither. QK of the next tile runs over the weights of this one; PV
// over the sums and `between` (2 * R * DP / 32 calls: the loads and LDS stores of later tiles). Every LDS read is issued
// a phase before its use.
//
// The reference is not compared with every score: weights above 2^8 that add up to 2^12 or more show in their sum, before
// they are used, and only then are the row's maximum taken, its reference raised and its weights computed again. So
// 2^31 tokens weigh at most 2^39, and values up to 2^88 cannot overflow their sums. (A bound of 2^60 is as fast, and
// overflows with values from 2^68 up.)
constexpr float kHighWeights = 0x1p12f;
template <class C, int R, class F>
__device__ __forceinline__ void turn_sums(AttendState<C, R>& st, Scores<R>& x, const Piece (&qf)[R][C::NF], const char* lds,
                                          float c, Piece (&k)[C::NF], const char* lds1, const char* lds2, F between) {
  const int hb = (threadIdx.x >> 5) & 1;
  const char* v = lds + 32 * C::KS;
  constexpr int NB = C::DP / 32;
  static_assert(C::KIND != kKindF32 && NB <= 4, "bf16 products, at most 128 channels");
  bf16x8 vf[NB][2];
#pragma unroll
  for (int ks = 0; ks < 2; ++ks)
#pragma unroll
    for (int i = 0; i < NB; ++i) vf[i][ks] = v_fragment<C>(v, ks, i);
  f32x4 vs[4];
  if constexpr (C::Q8) {
    const float* sc = reinterpret_cast<const float*>(lds + 32 * (C::KS + C::VS));
#pragma unroll
    for (int g = 0; g < 4; ++g) vs[g] = *reinterpret_cast<const f32x4*>(sc + 32 + 8 * g + 4 * hb);
  }
  __builtin_amdgcn_sched_barrier(0);
  float p[R][16];
  bf16x8 pb[R][2];
  auto weight = [&](int r, int e) {
    p[r][e] = __builtin_amdgcn_exp2f(fmaf(x.s[r][e], c, -st.m[r]));
    float w = p[r][e];
    if constexpr (C::Q8) w *= vs[e >> 2][e & 3];
    pb[r][e >> 3][e & 7] = static_cast<__bf16>(w);
  };
  f32x16 y[R];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int e = 0; e < 16; ++e) y[r][e] = 0.0f;
#pragma unroll
  for (int i = 0; i < C::NF; ++i)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      y[r] = mfma_32x32x16_bf16(k[i].h, qf[r][i].h, y[r]);
#pragma unroll
      for (int e = 16 * i / C::NF; e < 16 * (i + 1) / C::NF; ++e) weight(r, e);
      __builtin_amdgcn_sched_barrier(0);
    }
  read_k<C>(lds2, k);
  float sum[R];
  bool high = false;
  auto add_up = [&](int r) {
    sum[r] = 0.0f;
#pragma unroll
    for (int e = 0; e < 16; e += 4) sum[r] += (p[r][e] + p[r][e + 1]) + (p[r][e + 2] + p[r][e + 3]);
  };
#pragma unroll
  for (int r = 0; r < R; ++r) {
    add_up(r);
    high = high || sum[r] > kHighWeights;
  }
  if (__any(high)) {      // the other rows keep their references, and get the same weights again
    float m2[R];
    bool own[R];
    row_maxima<R>(x, c, m2);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      own[r] = half_max(sum[r]) > kHighWeights;
      m2[r] = own[r] ? m2[r] : st.m[r];
    }
    raise_reference<C, R>(st, m2);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float again = 0.0f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        weight(r, e);
        again += p[r][e];
      }
      sum[r] = own[r] ? again : sum[r];
    }
  }
#pragma unroll
  for (int n = 0; n < 2 * NB; ++n)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      st.o[r][n % NB] = mfma_32x32x16_bf16(vf[n % NB][n / NB], pb[r][n / NB], st.o[r][n % NB]);
      between(n * R + r);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    st.l[r] += sum[r];
    x.s[r] = y[r];
  }
  finish_scores<C, R, true>(x, lds1, {});
}

// A tile from its K fragments to its sums.
template <class C, int R, bool ALL>
__device__ __forceinline__ void tile_step(AttendState<C, R>& st, const Piece (&qf)[R][C::NF], const char* lds, float c,
                                          const uint32_t (&seen)[R], uint32_t apart) {
  Scores<R> x;
  if constexpr (C::NF <= 16) {
    Piece k[C::NF];
    read_k<C>(lds, k);
    __builtin_amdgcn_sched_barrier(0);      // all reads are under way before the first product waits for one
    products<C, R>(k, qf, x);
  } else {      // 8 at a time: the registers hold no more
    const char* p = lds + (threadIdx.x & 31) * C::KS + ((threadIdx.x >> 5) & 1) * 16;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < 16; ++e) x.s[r][e] = 0.0f;
#pragma unroll
    for (int i0 = 0; i0 < C::NF; i0 += 8) {
      Piece k[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) k[i].u = *reinterpret_cast<const uint4*>(p + (i0 + i) * 32);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int r = 0; r < R; ++r) x.s[r] = add_product<C>(k[i], qf[r][i0 + i], x.s[r]);
    }
  }
  finish_scores<C, R, ALL>(x, lds, seen);
  tile_sums<C, R, ALL>(st, x, lds, c, seen, apart);
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

// What a block works on.
struct AttendItem {
  bool own;
  int hk, b, part;              // b < 0: the prefix
  int row0, rows;               // first row of the tile; rows of the stream
  int j0, j1, cut;              // tokens; those below cut are seen by every row of the stream
  const int32_t* pages;
  int shift;
};

// Table entry of token j (of the last token for those past it), and the page of token j, -1 if there is none.
__device__ __forceinline__ int page_of(const AttendArgs& a, const AttendItem& it, int j) {
  const int e = it.pages[max(min(j, it.j1 - 1), 0) >> it.shift];
  return j < it.j1 && e >= 0 && e < a.c.n_pages ? e : -1;
}

// The lane's row of tile r: its Q fragments, its output row (or -1), the end of what it sees.
template <class C>
__device__ __forceinline__ void open_row(const AttendArgs& a, const AttendItem& it, int r, bool q_wide, bool neg,
                                         Piece (&qf)[C::NF], int& t, int& h, int& lim) {
  const int G = a.q.heads / a.c.heads;
  const bool live = r < it.rows;
  t = h = 0;
  if (live) row_token(a, G, it.b, r, t, h);
  lim = live && it.own ? it.cut + (t - it.b * a.S) : it.cut;
  h += it.hk * G;
  load_q<C>(a, static_cast<const char*>(a.q.in) + (t * a.q.in_t + h * a.q.in_h) * (C::KIND == kKindF32 ? 4 : 2), live, q_wide,
            neg, qf);
  if (!live) t = -1;
}

// Four channels of a finished part, or of the result if it is the only one.
template <class C>
__device__ __forceinline__ void put4(const AttendArgs& a, const AttendOut& out, long long at, int t, int h, int ch, f32x4 x,
                                     float l) {
  if (out.o) *reinterpret_cast<f32x4*>(out.o + at * a.c.D + ch) = x;
  else finish_row4<C::KIND>(a, t, h, ch, x, l, out.out_wide);
}
__device__ __forceinline__ void put_sums(const AttendArgs& a, const AttendOut& out, long long at, long long row, float m,
                                         float l) {
  if (out.o) out.ml[at] = float2{m, l};
  else if (a.lse) a.lse[row] = row_lse(m, l);
}

// The waves share the key tiles and take RW * 32 rows each: with 64, a fragment of K or V read from LDS feeds two
// products. 131071 tokens with 256 rows a head: 107 to 111 us (620 to 640 TFLOP/s), of which 30 us are the start, the parts'
// 31 MB and the join. EXACT: D = DP.
//
// Tiles without masks and with the next ones on their way are those that every row of the stream sees: none of the own
// tokens of a prompt's chunk whose queries are all of them (8192 tokens of 56 heads: 3.8 ms, 254 TFLOP/s).
template <class C, bool EXACT>
__device__ __forceinline__ void run_shared(const AttendArgs& a, const AttendOut& out, const AttendItem& it, long long part_rows,
                                           char* lds, float c, bool neg) {
  constexpr int R = C::RW;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, hb = lane >> 5, D = a.c.D;
  const int j0 = it.j0, j1 = it.j1;
  const int whole = max(min(it.cut, j1) - j0, 0) >> 5;      // tiles that every row sees
  int t[R], h[R], lim[R];
  Piece qf[R][C::NF];
  AttendState<C, R> st;
  st.clear();
#pragma unroll
  for (int r = 0; r < R; ++r)
    open_row<C>(a, it, it.row0 + (wave * R + r) * 32 + (lane & 31), out.q_wide, neg, qf[r], t[r], h[r], lim[r]);
  const uint32_t none[R] = {};
  // a load of a wave stays in one page; with smaller pages all tiles go the slow way below
  int stop = a.c.page_size >= 64 / C::CPR ? whole : 0;      // tiles before the first that is not whole
  if (stop > 0) {
    // Past the end the last tile comes again, from the caches. It is the last of all tiles, not of those before `stop`: one
    // found outside the cache moves stop back, and the walk goes only forward.
    const int last = stop - 1;
    Staged<C, C::NT> sg[2];
    PageWalk walk;
    walk.start(it.pages, j0 >> it.shift, (j1 - 1) >> it.shift);
    auto fetch = [&](Staged<C, C::NT>& x, int i) {
      const int n = min(i, last), j = j0 + 32 * n;
      walk.go(j >> it.shift);
      if (!x.load_whole(a, it.hk, j, it.shift, walk, tid)) stop = min(stop, n);
    };
    Scores<R> x;
    Piece k[C::NF];
    if constexpr (C::RING == 4) {
      // While the sums of tile i are taken, the scores of tile i + 1 are computed, the K fragments of tile i + 2 read,
      // tile i + 3 is stored and tiles i + 4, i + 5 are on their way in registers. The slot of tile i + 3 was last
      // read for the sums of tile i - 1, before the barrier that ended its turn.
      using S = Staged<C, C::NT>;
      {
        S s2, s3;      // the first four tiles are on their way together
        fetch(sg[0], 0);
        fetch(sg[1], 1);
        fetch(s2, 2);
        fetch(s3, 3);
        sg[0].store(lds, D, tid);
        fetch(sg[0], 4);
        sg[1].store(lds + C::TILE, D, tid);
        s2.store(lds + 2 * C::TILE, D, tid);
        sg[1] = s3;
      }
#pragma unroll
      for (int r = 0; r < R; ++r)      // only matrix products read Q from here on
#pragma unroll
        for (int n = 0; n < C::NF; ++n) asm volatile("" : "+a"(qf[r][n].h));
      __syncthreads();
      read_k<C>(lds, k);
      products<C, R>(k, qf, x);
      read_k<C>(lds + C::TILE, k);
      finish_scores<C, R, true>(x, lds, none);
      // The first references. Where tile 0 is not there, or leaves a row none, all tiles go the slow way.
      row_maxima<R>(x, c, st.m);
      bool none_yet = stop == 0;
#pragma unroll
      for (int r = 0; r < R; ++r) none_yet = none_yet || st.m[r] == -INFINITY;
      if (__syncthreads_or(none_yet)) {
        stop = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) st.m[r] = -INFINITY;
      }
      const uint32_t lane_part = S::lane_offset(a, it.hk, tid), k_at = S::k_place(tid), v_at = S::v_place(tid);
      auto turn = [&](S& s, int i) {
        auto slot = [&](int n) { return lds + ((i + n) & 3) * C::TILE; };
        uint32_t lane_off = lane_part;      // opaque: scalar base + lane offset in the load itself, not a sum kept per lane
        if constexpr (!C::Q8) asm volatile("" : "+v"(lane_off));
        const int n = min(i + 5, last), j = j0 + 32 * n;
        walk.go(j >> it.shift);
        const typename S::Source src = S::source(a, j, it.shift, walk, tid);
        if (!src.ok) stop = min(stop, n);
        if constexpr (!EXACT) s.store(slot(3), D, tid);
        else s.store_scales(slot(3), tid);
        constexpr int SLOTS = 2 * R * (C::DP / 32), EACH = (2 * S::N + SLOTS / 2 - 1) / (SLOTS / 2);
        turn_sums<C, R>(st, x, qf, slot(0), c, k, slot(1), slot(2), [&](int step) {
#pragma unroll
          for (int e = 0; e < EACH; ++e) {
            const int p = step % (SLOTS / 2) * EACH + e;
            if (p >= 2 * S::N) continue;
            if (step < SLOTS / 2) {
              if constexpr (EXACT) s.store_piece(slot(3) + k_at, slot(3) + v_at, p);
            } else {
              s.load_piece(a, src, lane_off, p);
            }
          }
        });
        s.load_scales(a, it.hk, j, it.shift, walk);
        __builtin_amdgcn_sched_barrier(0);
        __syncthreads();
      };
#pragma unroll 1
      for (int i = 0; i < stop; i += 2) {
        turn(sg[1], i);
        if (i + 1 < stop) turn(sg[0], i + 1);
      }
    } else {
      // Two slots: tile i + 1 is stored beside tile i, and read when every wave is done with that. Two tiles are on
      // their way (one of 256 fp32 channels: two would not fit the registers).
      constexpr int AHEAD = C::KIND == kKindF32 && C::DP == 256 ? 1 : 2;
      fetch(sg[0], 0);
      if constexpr (AHEAD == 2) fetch(sg[1], 1);
      auto turn = [&](Staged<C, C::NT>& s, int i) {
        char* tl = lds + (i & 1) * C::TILE;
        s.store(tl, D, tid);
        fetch(s, i + AHEAD);
        __syncthreads();
        tile_step<C, R, true>(st, qf, tl, c, none, 0);
      };
#pragma unroll 1
      for (int i = 0; i < stop; i += 2) {
        turn(sg[0], i);
        if (i + 1 < stop) turn(sg[AHEAD - 1], i + 1);
      }
      __syncthreads();
    }
  }
  for (int j = j0 + 32 * stop; j < j1; j += 32) {
    Staged<C, C::NT> sg;
    sg.load(a, it.hk, j, lane < 32 ? page_of(a, it, j + lane) : -1, tid);
    sg.store(lds, D, tid);
    __syncthreads();
    uint32_t seen[R];
#pragma unroll
    for (int r = 0; r < R; ++r) seen[r] = sg.mask & below(lim[r], j);
    tile_step<C, R, false>(st, qf, lds, c, seen, not_finite<C>(lds + 32 * C::KS) & ~below(it.cut, j));
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float l = half_sum(st.l[r]);
    if (t[r] < 0) continue;
    const long long row = static_cast<long long>(t[r]) * a.q.heads + h[r], at = part_rows + row;
    if (hb == 0) put_sums(a, out, at, row, st.m[r], l);
#pragma unroll
    for (int i = 0; i < C::DP / 32; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int ch = 32 * i + 8 * e + 4 * hb;
        const f32x16& o = st.o[r][i];
        if (ch < D) put4<C>(a, out, at, t[r], h[r], ch, f32x4{o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]}, l);
      }
  }
}

// A row tile of 32: each wave takes every NW-th tile into an LDS tile of its own, and the waves' sums are joined. Bound
// by HBM: 256 sequences of up to 1024 tokens 116 us (4.67 TB/s), 16 of 32768 tokens 366 us (5.87 TB/s).
template <class C, bool SHARED>
__device__ __forceinline__ void run_alone(const AttendArgs& a, const AttendOut& out, const AttendItem& it, long long part_rows,
                                          char* lds, float c, bool neg) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, hb = lane >> 5, D = a.c.D, Hq = a.q.heads;
  const int j0 = it.j0, j1 = it.j1;
  const int tiles = (j1 - j0 + 31) >> 5;
  int t, h, lim;
  Piece qf[1][C::NF];
  AttendState<C, 1> st;
  st.clear();
  open_row<C>(a, it, it.row0 + (lane & 31), out.q_wide, neg, qf[0], t, h, lim);
  const uint32_t none[1] = {0};
  char* tl = lds + wave * C::TILE;
  int stop = a.c.page_size >= 64 / C::CPR ? max(min(it.cut, j1) - j0, 0) >> 5 : 0, i = wave;
  if (i < stop) {
    // Tiles on their way in registers: one while the next is worked on. Two of 8-bit codes, half the bytes, where a wave
    // has a SIMD to itself (64 sequences of up to 4000 tokens: 95 -> 91 us; of bf16 beside a prefix a second one costs
    // 147 -> 153 us, and with two waves a SIMD the registers hold no second one: 83 -> 118 us).
    constexpr int AHEAD = C::Q8 && C::eu_waves(SHARED) == 1 ? 2 : 1;
    Staged<C, 64> sg[AHEAD];
    const int last = wave + (stop - 1 - wave) / C::NW * C::NW;      // the wave's; comes again past the end
    PageWalk walk;
    walk.start(it.pages, (j0 + 32 * i) >> it.shift, (j1 - 1) >> it.shift);
    auto fetch = [&](Staged<C, 64>& s, int n) {
      n = min(n, last);
      const int j = j0 + 32 * n;
      walk.go(j >> it.shift);
      if (!s.load_whole(a, it.hk, j, it.shift, walk, lane)) stop = min(stop, n);
    };
    auto turn = [&](Staged<C, 64>& s) {
      __builtin_amdgcn_wave_barrier();
      s.store(tl, D, lane);
      __builtin_amdgcn_wave_barrier();
      fetch(s, i + AHEAD * C::NW);
      tile_step<C, 1, true>(st, qf, tl, c, none, 0);
      i += C::NW;
    };
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) fetch(sg[n], i + n * C::NW);
#pragma unroll 1
    while (i < stop) {
      turn(sg[0]);
      if constexpr (AHEAD == 2)
        if (i < stop) turn(sg[1]);
    }
  }
  for (; i < tiles; i += C::NW) {
    Staged<C, 64> sg;
    const int j = j0 + 32 * i;
    sg.load(a, it.hk, j, lane < 32 ? page_of(a, it, j + lane) : -1, lane);
    __builtin_amdgcn_wave_barrier();
    sg.store(tl, D, lane);
    __builtin_amdgcn_wave_barrier();
    const uint32_t seen[1] = {sg.mask & below(lim, j)};
    if (sg.mask) tile_step<C, 1, false>(st, qf, tl, c, seen, not_finite<C>(tl + 32 * C::KS) & ~below(it.cut, j));
  }
  st.l[0] = half_sum(st.l[0]);
  __syncthreads();
  float* mo = reinterpret_cast<float*>(lds);                    // [NW][32][DP], then m and l [NW][32]
  float* mm = mo + C::NW * 32 * C::DP;
  if (hb == 0) {
    mm[wave * 32 + lane] = st.m[0];
    mm[(C::NW + wave) * 32 + lane] = st.l[0];
  }
#pragma unroll
  for (int n = 0; n < C::DP / 32; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<f32x4*>(mo + (wave * 32 + (lane & 31)) * C::DP + 32 * n + 8 * e + 4 * hb) =
          f32x4{st.o[0][n][4 * e], st.o[0][n][4 * e + 1], st.o[0][n][4 * e + 2], st.o[0][n][4 * e + 3]};
  __syncthreads();
  const int here = min(32, it.rows - it.row0), quads = D / 4, G = Hq / a.c.heads;
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
    row_token(a, G, it.b, it.row0 + rr, tt, hh);
    hh += it.hk * G;
    const long long row = static_cast<long long>(tt) * Hq + hh, at = part_rows + row;
    if (ch == 0) put_sums(a, out, at, row, m, l);
    put4<C>(a, out, at, tt, hh, ch, x, l);
  }
}

// SHARED: some stream of the call has more than ALONE_ROWS rows.
template <class C, bool SHARED>
__global__ __launch_bounds__(C::NT, C::eu_waves(SHARED)) void attend_kernel(AttendArgs a, AttendPlan pl, AttendOut out) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int hkv = a.c.heads, G = a.q.heads / hkv;
  // ---- the item. Groups of 8 blocks, one per XCD; the row tiles of a prefix range follow each other on one XCD, whose
  // L2 holds the range.
  const int grp = blockIdx.x >> 3, x8 = blockIdx.x & 7;
  AttendItem it;
  it.own = grp >= pl.pre_groups;
  const int g = it.own ? grp - pl.pre_groups : grp;
  const int tiles = it.own ? pl.own_tiles : pl.pre_tiles, pair = (g / tiles) * 8 + x8, tile = g % tiles;
  const int parts = it.own ? pl.own_parts : pl.pre_parts, rest = pair / hkv;
  it.hk = pair % hkv;
  it.part = rest % parts;
  it.b = it.own ? rest / parts : -1;
  if (it.own ? it.b >= a.B : rest >= parts) return;
  if (it.own && pl.own_sorted) it.b = longest_first(a, it.b);
  const bool shared = SHARED && (it.own ? pl.own_shared : pl.pre_shared);
  it.rows = it.own ? pl.own_rows : pl.pre_rows;
  it.row0 = tile * (shared ? C::ROWS : 32);
  const int n = it.own ? own_len(a, it.b) : a.P;
  const int chunk = it.own ? own_chunk(pl, n) : pl.pre_chunk;
  const long long first = static_cast<long long>(it.part) * chunk;
  if (first >= n && (out.o || it.part > 0)) return;
  it.j0 = static_cast<int>(first < n ? first : n);
  it.j1 = n - it.j0 < chunk ? n : it.j0 + chunk;
  it.cut = it.own ? n - a.S + 1 : n;
  if (it.own) {                                   // the tile's last row sees the most
    const int last = min(it.row0 + (shared ? C::ROWS : 32), it.rows) - 1;
    it.j1 = max(it.j0, min(it.j1, it.cut + last / G));
  }
  it.pages = it.own ? a.page_table + static_cast<long long>(it.b) * a.table_pages : a.prefix_pages;
  it.shift = 31 - __builtin_clz(a.c.page_size);
  const float cs = a.scale * 1.44269504088896340736f;
  const long long part_rows = static_cast<long long>(it.own ? pl.pre_parts + it.part : it.part) * a.B * a.S * a.q.heads;
  if constexpr (SHARED) {
    if (shared && a.c.D == C::DP) return run_shared<C, true>(a, out, it, part_rows, lds, fabsf(cs), cs < 0.0f);
    if (shared) return run_shared<C, false>(a, out, it, part_rows, lds, fabsf(cs), cs < 0.0f);
  }
  if constexpr (C::ALONE_ROWS > 0) run_alone<C, SHARED>(a, out, it, part_rows, lds, fabsf(cs), cs < 0.0f);
}

// out_r = sum_parts 2^(m_i - M) o_i / sum_parts 2^(m_i - M) l_i. LPR lanes per row, four channels each. (1024 rows of
// 64 parts, 35 MB: 11 us; 14336 rows of 2, 15 MB: 9 us; 32 rows: 4 us.) Bound by the
// latency of two dependent loads and the bytes of the parts, so every load that can be is under way at once: with
// few parts a row's lanes hold all of them; with many a block takes one row, a thread per part for (m, l), then each of
// its 256 / LPR lane groups every 256 / LPR-th part, and the groups' sums meet in LDS.
template <int KIND, int LPR, bool MANY>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a, AttendPlan pl, AttendOut out) {
  constexpr int GROUPS = 256 / LPR, FEW = 8;
  const int Hq = a.q.heads, D = a.c.D, tid = threadIdx.x;
  const long long n_rows = static_cast<long long>(a.B) * a.S * Hq;
  const long long row = MANY ? blockIdx.x : (static_cast<long long>(blockIdx.x) * 256 + tid) / LPR;
  if (row >= n_rows) return;
  const int ch = (tid % LPR) * 4, t = static_cast<int>(row / Hq), h = static_cast<int>(row - static_cast<long long>(t) * Hq);
  int parts = pl.pre_parts;
  if (pl.own_parts > 0) {
    const int n = own_len(a, t / a.S), chunk = own_chunk(pl, n);
    if (n > 0) parts += (n + chunk - 1) / chunk;
  }
  f32x4 x = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  float m = -INFINITY, l = 0.0f;
  // a part that saw no token left its sums unset
  auto add = [&](float w, const f32x4& y) {
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] += w == 0.0f ? 0.0f : w * y[q];
  };
  auto sums = [&](int i) { return *reinterpret_cast<const f32x4*>(out.o + (i * n_rows + row) * D + (ch < D ? ch : 0)); };
  if constexpr (MANY) {
    __shared__ float ws[512], red[8];
    __shared__ f32x4 sx[256];
    float2 ml[2];      // at most 512 parts
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      ml[j] = tid + 256 * j < parts ? out.ml[(tid + 256 * j) * n_rows + row] : float2{-INFINITY, 0.0f};
      m = fmaxf(m, ml[j].x);
    }
    m = wave_max(m);
    if ((tid & 63) == 0) red[tid >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float w = ml[j].y == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(ml[j].x - m);
      ws[tid + 256 * j] = w;
      l += w == 0.0f ? 0.0f : w * ml[j].y;
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) l += __shfl_xor(l, o, kWave);
    if ((tid & 63) == 0) red[4 + (tid >> 6)] = l;
    __syncthreads();
    l = (red[4] + red[5]) + (red[6] + red[7]);
    for (int i0 = tid / LPR; i0 < parts; i0 += GROUPS * FEW) {
      f32x4 y[FEW];
#pragma unroll
      for (int j = 0; j < FEW; ++j) y[j] = sums(min(i0 + j * GROUPS, parts - 1));
#pragma unroll
      for (int j = 0; j < FEW; ++j) add(i0 + j * GROUPS < parts ? ws[i0 + j * GROUPS] : 0.0f, y[j]);
    }
    sx[tid] = x;
    __syncthreads();
    if (tid >= LPR) return;
#pragma unroll
    for (int g = 1; g < GROUPS; ++g) {
      const f32x4 y = sx[g * LPR + tid];
#pragma unroll
      for (int q = 0; q < 4; ++q) x[q] += y[q];
    }
  } else if (parts > 0) {
    float2 ml[FEW];
    f32x4 y[FEW];
#pragma unroll
    for (int i = 0; i < FEW; ++i) {
      const int at = min(i, parts - 1);      // past the end: the last part again
      ml[i] = out.ml[at * n_rows + row];
      y[i] = sums(at);
    }
#pragma unroll
    for (int i = 0; i < FEW; ++i) m = i < parts ? fmaxf(m, ml[i].x) : m;
#pragma unroll
    for (int i = 0; i < FEW; ++i) {
      const float w = i >= parts || ml[i].y == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(ml[i].x - m);
      l += w == 0.0f ? 0.0f : w * ml[i].y;
      add(w, y[i]);
    }
  }
  if (ch < D) finish_row4<KIND>(a, t, h, ch, x, l, out.out_wide);
  if (ch == 0 && a.lse) a.lse[row] = row_lse(m, l);
}

// The split.
//
// A stream of at most ALONE_ROWS rows is read by each wave on its own (more loads in flight); its second 32 rows
// read the range again, from L2. With more rows the waves share the tiles. 16 sequences with 4 rows each on
// 16384 / 131071 tokens: 22 / 68 us alone, 24 / 70 us shared; 24 sequences: 30 / 83 us and 26 / 74 us.
//
// Every block slot is taken by a prefix item or an own one. The prefix gets the share of the slots that its time has
// of the sum of both (at the rates that the two kinds reach), as one item a slot, first in the grid, so that it lasts
// as long as the call and leaves the own items, bound by HBM, the slots that these need to keep pace (256 sequences on
// 4100 tokens with up to 1024 of their own: 147 us, and 236 us with the two kinds alternating through the grid). The
// share is rounded to whole parts; with few of them the nearer number is better (8-bit tokens, 120 sequences: 3 parts
// 302 us, 2 parts 372 us), with many the lower one (64 sequences: 5 parts 166 us, 6 parts 171 us). With more row
// tiles than slots the parts are those that fill the last round of blocks (700 sequences: 1445 -> 1068 us).
//
// Each item costs about 10 us of latencies (length, page table, Q, the first keys, its sums), so own ranges are
// cut for one item a slot, or for two beside a prefix, where they even out what the shares above miss (64 sequences of
// 8-bit tokens beside 16397 prefix tokens: 214 us for one, 178 for two, 197 for four; without a prefix, at 512 slots,
// 92, 99, 101 us).
// Two a slot is rounded to the nearer number of parts (100 sequences of up to 3000 tokens on 4100: 129 us, up 142 us), one is
// rounded up (39 fp32 sequences of up to 3439 tokens: 91 us, down 114 us).
// With up to kSortedMost sequences the longest start first, where any item has to wait (178 -> 166 us; 100
// sequences of up to 3000 tokens 151 -> 142 us). Ordering more of them costs each block more than it gives.
// The sequences' own lengths are not known here: they are taken to average half of the table's width. A table far wider than that
// gives the prefix too few slots. 64 sequences of 56 heads with 16 own tokens on 4100: 45 us with room for 64 or 1024
// tokens, 71 for 4096, 124 for 8192 and more; of 16 heads on 131071: 114 us, and 276 with room for 32768.
//
// No range is below kMinTokens, so that a part's sums (4 D bytes a row) stay small beside its keys, or
// a quarter of that where the slots would not be filled (2 sequences on 1000 tokens: 16.8 -> 13.2 us).
constexpr int kMinTokens = 256;

template <class C>
static AttendPlan attend_plan(const Cache& c, int B, int S, int Hq, int P, int table_pages) {
  AttendPlan p{};
  const int G = Hq / c.heads;
  p.pre_rows = P > 0 ? B * S * G : 0;
  p.own_rows = S * G;
  p.pre_shared = p.pre_rows > C::ALONE_ROWS;
  p.own_shared = p.own_rows > C::ALONE_ROWS;
  const long long slots = static_cast<long long>(device_cu_count()) * C::blocks(p.pre_shared || p.own_shared);
  // Prefixes and short ranges are cut for the slots that shared tiles leave, as each part costs its sums: 8 sequences on
  // 131071 tokens 62 us, for all slots 67; 25 sequences of up to 162 tokens 17 us, 26.
  const long long few_slots = static_cast<long long>(device_cu_count()) * C::blocks(true);
  const long long own_max = static_cast<long long>(table_pages) * c.page_size;
  auto cdivl = [](long long x, long long y) { return (x + y - 1) / y; };
  auto parts_of = [&](long long base, long long tokens, long long want) {
    auto least = [](long long x, long long y) { return x < y ? x : y; };
    long long n = least(P > 0 ? (want + base / 2) / base : cdivl(want, base), cdivl(tokens, kMinTokens));
    const long long small = least(least(few_slots, want) / base, cdivl(tokens, kMinTokens / 4));
    n = n < small ? small : n;
    return static_cast<int>(n < 1 ? 1 : n > 256 ? 256 : n);
  };
  if (P > 0) {
    p.pre_tiles = static_cast<int>(cdivl(p.pre_rows, p.pre_shared ? C::ROWS : 32));
    const double flop_us = C::KIND == kKindF32 ? 1e8 : 6e8, byte_us = C::Q8 ? 4e6 : 5e6;     // rates reached, per microsecond
    const double row_bytes = 2.0 * c.D * (C::KIND == kKindF32 ? 4 : C::Q8 ? 1 : 2);
    double pre = 4.0 * C::DP * p.pre_tiles * (p.pre_shared ? C::ROWS : 32) * P / flop_us;
    if (!p.pre_shared) pre = row_bytes * P / byte_us;
    const double own = row_bytes * B * (own_max / 2) / byte_us;
    const long long base = static_cast<long long>(p.pre_tiles) * c.heads;
    const double share = static_cast<double>(few_slots) * pre / (pre + own) / base;
    long long n = share < 1 ? 1 : static_cast<long long>(share + (share < 4 ? 0.5 : 0.0));
    // More row tiles than slots, or almost: the last of few rounds would leave most slots empty.
    auto time = [&](long long m) { return cdivl(m * base, few_slots) * few_slots * pre / (m * base); };
    if (time(n) > 1.5 * (pre + own))
      for (long long m = n + 1; m <= 8; ++m)
        if (time(m) * (1 + 0.01 * m) < time(n) * (1 + 0.01 * n)) n = m;
    p.pre_parts = parts_of(base, P, base * n);
    p.pre_chunk = static_cast<int>(cdivl(cdivl(P, p.pre_parts), 64) * 64);
    p.pre_parts = static_cast<int>(cdivl(P, p.pre_chunk));
    p.pre_groups = static_cast<int>(cdivl(static_cast<long long>(p.pre_parts) * c.heads, 8) * p.pre_tiles);
  }
  if (own_max > 0) {
    p.own_tiles = static_cast<int>(cdivl(p.own_rows, p.own_shared ? C::ROWS : 32));
    const long long pairs = static_cast<long long>(B) * c.heads;
    p.own_parts = parts_of(pairs * p.own_tiles, own_max, P > 0 ? 2 * slots : slots);
    p.own_sorted = B > 1 && B <= kSortedMost && own_max >= 2 * kMinTokens &&
                   pairs * p.own_tiles * p.own_parts + 8LL * p.pre_groups > slots;
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
  if (D % 16 == 0) return by_dim(std::integral_constant<int, kKindE4M3>{});
  return by_dim(std::integral_constant<int, kKindE4M3Narrow>{});
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
      p.own_tiles = cdiv(p.own_rows, C::ROWS);
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
    auto go = [&](auto shared) {
      constexpr bool SHARED = decltype(shared)::value;
      constexpr int LDS = SHARED ? C::LDS : C::LDS_ALONE;
      static const hipError_t allowed = allow_lds(attend_kernel<C, SHARED>, LDS);
      if (allowed != hipSuccess) return allowed;
      hipLaunchKernelGGL((attend_kernel<C, SHARED>), dim3(8u * (p.pre_groups + p.own_groups)), dim3(C::NT), LDS, st, a, p, out);
      return hipGetLastError();
    };
    hipError_t e;
    if constexpr (C::ALONE_ROWS > 0) e = p.pre_shared || p.own_shared ? go(std::true_type{}) : go(std::false_type{});
    else e = go(std::true_type{});
    if (e != hipSuccess || direct) return e;
    constexpr int LPR = C::DP / 4;
    if (p.pre_parts + p.own_parts > 8)
      hipLaunchKernelGGL((attend_join_kernel<C::KIND, LPR, true>), dim3(static_cast<unsigned>(rows)), dim3(256), 0, st, a, p,
                         out);
    else
      hipLaunchKernelGGL((attend_join_kernel<C::KIND, LPR, false>), dim3(static_cast<unsigned>((rows * LPR + 255) / 256)),
                         dim3(256), 0, st, a, p, out);
    return hipGetLastError();
  });
}

}  // namespace moe
