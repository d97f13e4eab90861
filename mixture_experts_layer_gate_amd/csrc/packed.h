// Causal attention of packed sequences: what its forward and backward kernels share. Tokens of all sequences follow each other
// in one buffer; token i of a sequence that starts at s sees the tokens s .. i.
//
// Tiles of 32 tokens x 32 tokens on 32x32 MFMAs. The rows of one operand tile come from LDS (16 bytes of a row per lane), the
// other operand stays in the lane's registers; so a lane has the 16 products of one register-side token (lane % 32) with the
// LDS-side tokens 8 (e / 4) + 4 (lane / 32) + e % 4. Weighted sums over the LDS-side tokens take these, rounded to bf16, as they
// lie, with the contraction order permuted the same way in the other operand, whose 4 x 16 pieces come out of the same LDS rows
// transposed. fp32 runs the same scheme on the 32x32x2 fp32 MFMA.
#pragma once

#include <limits.h>

#include <algorithm>
#include <type_traits>

#include "heads.h"

namespace moe {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) void lds_any_t;

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// A stage in LDS: tiles of 32 tokens, each in groups of 64 bytes of channels: [tile][group][32 tokens][64 bytes]. Piece c (16
// bytes) of a token's group lies at c ^ (token / 4 % 4). So 16 lanes that read one piece of 16 tokens meet all 64 banks, as do the
// transposing reads of 64 bytes of four tokens; a lane's address is one of two, and an offset known at compile time; and a direct
// load to LDS (64 lanes, 1 KB in a row) takes 64 bytes of each of 16 tokens.
template <bool F32_, int DP_, int NW_ = 4>
struct PackedCfg {
  static constexpr bool F32 = F32_;
  static constexpr int DP = DP_;                     // channels, padded to 64, 96, 128, 192 or 256
  static constexpr int ES = F32 ? 4 : 2, QE = 16 / ES;   // bytes of an element, elements of a piece
  static constexpr int NG = DP * ES / 64;            // groups of a token
  static constexpr int NF = NG * 2;                  // pieces of a lane's row half
  static constexpr int NB = DP / 32;                 // blocks of 32 channels
  static constexpr int NW = NW_, NT = NW * 64, ROWS = NW * 32;   // waves of a block, their register-side tokens
  static constexpr int KT = DP * ES <= 256 ? 64 : 32;    // LDS-side tokens of a stage
  static constexpr int NS = KT / 32;
  static constexpr int GROUP = 32 * 64, TILE = NG * GROUP, STAGE = NS * TILE;
  template <int W>
  using with_waves = PackedCfg<F32_, DP_, W>;
  using E = typename std::conditional<F32, float, __bf16>::type;
};

union Quad {      // a 16-byte piece
  uint4 u;
  float f[4];
  bf16x8 h;
};

// A piece whose elements lie anywhere.
template <class C>
__device__ __forceinline__ uint4 load_elements(const typename C::E* p) {
  if constexpr (C::F32) {
    return __builtin_bit_cast(uint4, f32x4{p[0], p[1], p[2], p[3]});
  } else {
    bf16x8 x;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = p[e];
    return __builtin_bit_cast(uint4, x);
  }
}
template <class C>
__device__ __forceinline__ void store_elements(typename C::E* p, uint4 u) {
  if constexpr (C::F32) {
    const f32x4 x = __builtin_bit_cast(f32x4, u);
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = x[e];
  } else {
    const bf16x8 x = __builtin_bit_cast(bf16x8, u);
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = x[e];
  }
}

template <int NB>
__device__ __forceinline__ void clear_sums(f32x16 (&s)[NB]) {
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) s[i][e] = 0.0f;
}

// The operand that a lane's tokens bring to the sums: bf16 fragments of 16 tokens, or fp32 as they are.
template <class C>
struct Weights {
  typename std::conditional<C::F32, float, bf16x8>::type w[C::F32 ? 16 : 2];
  __device__ __forceinline__ void set(int e, float x) {
    if constexpr (C::F32) w[e] = x;
    else w[e >> 3][e & 7] = static_cast<__bf16>(x);
  }
};

// NaN if either is one.
__device__ __forceinline__ float nan_max(float x, float y) { return __builtin_elementwise_maximum(x, y); }
__device__ __forceinline__ float halves_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return nan_max(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float halves_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// Tokens of a 32-token tile from `base` that lie below lim.
__device__ __forceinline__ uint32_t tokens_below(int lim, int base) {
  const int n = lim - base;
  return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
}
__device__ __forceinline__ int lds_token(int e) { return 8 * (e >> 2) + 4 * ((threadIdx.x >> 5) & 1) + (e & 3); }

// ---- sequences

// The last entry of seq_start[0 .. n] that is <= row, -1 if the first is above it: 64 entries at a time.
__device__ __forceinline__ int last_start(const int32_t* seq_start, int n, int row) {
  int at = 0, size = n + 1;
  while (true) {
    const int step = (size + 63) / 64, i = static_cast<int>(threadIdx.x & 63) * step;
    const bool le = i < size && seq_start[at + i] <= row;
    const int count = __popcll(__ballot(le));
    if (count == 0) return -1;      // only on the first turn: later ones start at an entry that is <= row
    at += (count - 1) * step;
    if (step == 1) return at;
    size = min(step, size - (count - 1) * step);
  }
}
// Sequence of the lane's token `row`; `first` is the least row of the wave. Tokens outside all sequences are not live; those from
// `all_end` on are behind the last one.
struct Span {
  int start, end;      // [start, end) in 0 .. T
  bool live;
};
__device__ __forceinline__ Span find_span(const int32_t* seq_start, int n, int T, int all_end, int first, int row) {
  Span s{0, 0, false};
  const int lane = threadIdx.x & 63;
  // the boundaries at .. at + 63, the first of which is above no row of the wave's; up to 64 of them come with one load
  int at = n < 64 ? 0 : max(last_start(seq_start, n, first), 0);
  bool found = row >= all_end;
  while (true) {
    const int b = at + lane <= n ? seq_start[at + lane] : INT_MAX;
    // how many of them are <= row (they ascend)
    int count = 0;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) count += __shfl(b, count + o - 1, kWave) <= row ? o : 0;
    const int last = __shfl(b, 63, kWave);
    count += count == 63 && last <= row ? 1 : 0;
    const int before = __shfl(b, max(count - 1, 0), kWave), after = __shfl(b, min(count, 63), kWave);
    if (!found && count < 64) {
      found = true;
      const int q = at + count - 1;      // sequence
      s.start = max(before, 0);
      s.end = min(after, T);
      s.live = count > 0 && q < n && s.start <= row && row < s.end;
    }
    const uint64_t open = __ballot(!found);
    if (!open || at + 64 > n) return s;
    // from the last boundary on, the start of the sequence behind it, or past empty sequences to that of the first row that is left
    at = max(at + 63, last_start(seq_start, n, __builtin_amdgcn_readlane(row, __builtin_ctzll(open))));
  }
}

// The wave's live tokens lie side by side (row0 + first .. row0 + last; none: last < 0), and starts and ends ascend with them.
struct WaveSpan {
  uint32_t b;
  int first, last;
  __device__ __forceinline__ explicit WaveSpan(bool live) : b(static_cast<uint32_t>(__ballot(live))) {
    first = b ? __builtin_ctz(b) : 0;
    last = b ? 31 - __builtin_clz(b) : -1;
  }
  __device__ __forceinline__ int of_first(int x) const { return __builtin_amdgcn_readlane(x, first); }
  __device__ __forceinline__ int of_last(int x) const { return __builtin_amdgcn_readlane(x, last & 31); }
};
// The least `lo` and the largest `hi` of the block's waves (those without tokens bring INT_MAX and -1). `ends`: LDS.
template <class C>
__device__ __forceinline__ void block_range(int lo, int hi, int (&ends)[2][C::NW], int& first, int& last) {
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) {
    ends[0][wave] = lo;
    ends[1][wave] = hi;
  }
  __syncthreads();
  first = INT_MAX;
  last = -1;
#pragma unroll
  for (int w = 0; w < C::NW; ++w) {
    first = min(first, ends[0][w]);
    last = max(last, ends[1][w]);
  }
  first = __builtin_amdgcn_readfirstlane(first);
  last = __builtin_amdgcn_readfirstlane(last);
}

// Where the sequences end: rows from there on take no part, whatever they and their places in the workspace hold. 0 .. T for any
// entries.
__device__ __forceinline__ int packed_end(const int32_t* seq_start, int n, int T) { return min(max(seq_start[n], 0), T); }

// ---- work of a grid: every (head, tile), heads and tiles spread over the XCDs (blocks go round the eight of them) so that
// the heads of one XCD share its L2, and the tiles with the most work come first.
struct PackedGrid {
  int heads, tiles;
  int share;      // XCDs that share a head
  int per;        // heads of an XCD
  unsigned blocks;
  __host__ static PackedGrid of(int heads, int tiles) {
    int g = 8;
    while (heads % g) g /= 2;
    PackedGrid p{heads, tiles, 8 / g, heads / g, 0};
    p.blocks = 8u * p.per * ((tiles + p.share - 1) / p.share);
    return p;
  }
  // rank 0: the tile that is started first
  __device__ __forceinline__ bool item(unsigned block, int& head, int& rank) const {
    const int x = block & 7, i = block >> 3, groups = 8 / share;
    head = (x % groups) * per + i % per;
    rank = i / per * share + x / groups;
    return rank < tiles;
  }
};

// ---- a head's rows from memory to LDS

constexpr uint32_t kPastAll = 0xFFFFFFF0u;      // an offset past every range: loads zero

template <class C>
struct RowLoader {
  const char* base;
  long long stride;      // bytes
  int end, D;
  bool direct;           // rows on 16 bytes, a stage within 2^31 bytes: loads straight to LDS
  __device__ __forceinline__ RowLoader(const void* p, long long t, long long h, int head, int end_, int D_, bool direct_)
      : base(static_cast<const char*>(p) + head * h * C::ES), stride(t * C::ES), end(end_), D(D_), direct(direct_) {}
  // Rows row0 .. row0 + KT - 1 to `stage`; zeros for those from `end` on and for channels from D on. To be waited for with
  // stage_barrier().
  __device__ __forceinline__ void issue(char* stage, int row0) const {
    bring<C::NW, C::STAGE / 1024>(stage, row0, __builtin_amdgcn_readfirstlane(threadIdx.x >> 6));
  }
  // Rows row0 .. row0 + 31 to a tile, by this wave alone; to be waited for with wave_wait().
  __device__ __forceinline__ void issue_tile(char* tile, int row0) const { bring<1, C::TILE / 1024>(tile, row0, 0); }
  template <int WAVES, int COUNT>
  __device__ __forceinline__ void bring(char* stage, int row0, int wave) const {
    constexpr int LOADS = (COUNT + WAVES - 1) / WAVES;
    const int lane = threadIdx.x & 63;
    const int r = lane >> 2, c = (lane & 3) ^ ((lane >> 4) & 3);
    const int rows = min(COUNT / (2 * C::NG) * 32, end - row0);
    const char* first = base + row0 * stride;
    if (direct) {
      const uint32_t range = rows <= 0 ? 0u : static_cast<uint32_t>((rows - 1) * stride + D * C::ES);
      const auto rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(first), static_cast<short>(0), static_cast<int>(range),
                                                        0x00020000);
      const uint32_t lane_off = r * static_cast<uint32_t>(stride) + c * 16;
#pragma unroll
      for (int n = 0; n < LOADS; ++n) {
        const int q = n * WAVES + wave, half = q & 1, g = (q >> 1) % C::NG, t = (q >> 1) / C::NG;
        if (LOADS * WAVES > COUNT && q >= COUNT) break;
        uint32_t off = lane_off + ((32 * t + 16 * half) * static_cast<uint32_t>(stride) + g * 64);
        if (D != C::DP && g * 64 + c * 16 >= D * C::ES) off = kPastAll;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_any_t*)(stage + q * 1024), 16, off, 0, 0, 0);
      }
    } else {
#pragma unroll 1
      for (int n = 0; n < LOADS; ++n) {
        const int q = n * WAVES + wave, half = q & 1, g = (q >> 1) % C::NG, t = (q >> 1) / C::NG;
        if (q >= COUNT) break;
        const int row = 32 * t + 16 * half + r, at = (g * 64 + c * 16) / C::ES;
        uint4 x = uint4{0, 0, 0, 0};
        if (row < rows && at < D) x = load_elements<C>(reinterpret_cast<const typename C::E*>(first + row * stride) + at);
        *reinterpret_cast<uint4*>(stage + q * 1024 + lane * 16) = x;
      }
    }
  }
};
// Every load and LDS access of the block's waves up to here is done.
__device__ __forceinline__ void stage_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// The wave's own loads are done, but for the newest N (LDS stores of rows that are not loaded directly too).
template <int N>
__device__ __forceinline__ void wave_wait() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// Where there are too few tiles of register-side tokens for the GPU, the four waves of a block share one, each takes every
// fourth tile of the other tokens to LDS of its own, and the sums of the four are joined in LDS.
template <class C, int MORE = 0>
struct SplitCfg {
  static constexpr int SLOT = 2 * C::TILE + MORE;                     // two tensors' tiles, and MORE bytes
  // The next tiles are on their way where two of them leave room for a second block on the CU; else the second block's waves fill
  // the wait (2000 tokens of 16 heads of 128: 59 -> 39 us, gradient 144 -> 122 us).
  static constexpr int SLOTS = 8 * SLOT <= 78 * 1024 ? 2 : 1;
  static constexpr int OWN = SLOTS * SLOT;
  static constexpr bool FITS = 4 * OWN <= 160 * 1024 - 4096;
};
// The wave's items begin, begin + 4 STEP, .. <= last, each brought by issue(LDS, item) and worked on by take(LDS, item). counted:
// every load goes straight to LDS, so that waiting can leave the next item's on their way. The first one is under way if there are
// two slots.
template <class C, class S, int STEP = 128, int EXTRA = 0, class I, class F>
__device__ __forceinline__ void wave_tiles(char* own, int begin, int last, bool counted, I issue, F take) {
  if constexpr (S::SLOTS == 2) {
    int at = 0;
    for (int j = begin; j <= last; j += STEP, at ^= 1) {
      const bool more = j + STEP <= last;
      wave_wait<63>();      // what was in the other slot is read
      if (more) issue(own + (at ^ 1) * S::SLOT, j + STEP);
      if (more && counted) wave_wait<2 * C::TILE / 1024 + 2 * EXTRA>();
      else wave_wait<0>();
      take(own + at * S::SLOT, j);
    }
  } else {
    for (int j = begin; j <= last; j += STEP) {
      wave_wait<0>();
      issue(own, j);
      wave_wait<0>();
      take(own, j);
    }
  }
}
// Tokens of the wave (a bit each) with a sum that is no finite number. Matrix products over masked places multiply
// 0 by what lies there; where that is an infinity or a NaN the sums come out as NaN, and such tokens are done
// again one by one over what they see alone. So finite results never pay for the masked places' contents.
template <int NB>
__device__ __forceinline__ uint32_t tokens_not_finite(const f32x16 (&s)[NB], bool live) {
  float none[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int e = 0; e < 16; ++e) none[e & 3] = fmaf(s[i][e], 0.0f, none[e & 3]);
  const uint64_t b = __ballot(live && (none[0] + none[1]) + (none[2] + none[3]) != 0.0f);
  return static_cast<uint32_t>(b) | static_cast<uint32_t>(b >> 32);
}

// Adds up the four waves' sums by blocks of 32 channels: take(i, sums of block i) for those that are this wave's. Before the first
// of them the tokens of all waves' blocks that are not finite are in bad[0 .. 3] (cleared by the caller).
template <int OWN, int N, class F>
__device__ __forceinline__ void join_waves(char* lds, const f32x16 (&s)[N], float f, bool live, uint32_t (&bad)[4], F take) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  static_assert(N * 4096 <= OWN, "a wave's sums fit its LDS");
  float* own = reinterpret_cast<float*>(lds + wave * OWN) + lane * 4;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      *reinterpret_cast<f32x4*>(own + (i * 4 + g) * 256) =
          f32x4{s[i][4 * g] * f, s[i][4 * g + 1] * f, s[i][4 * g + 2] * f, s[i][4 * g + 3] * f};
  __syncthreads();
  f32x16 x[(N + 3) / 4][1];
#pragma unroll
  for (int n = 0; n < (N + 3) / 4; ++n) {
    const int i = n * 4 + wave;
    if (i >= N) break;
    clear_sums(x[n]);
#pragma unroll
    for (int w = 0; w < 4; ++w)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 y = *reinterpret_cast<const f32x4*>(lds + w * OWN + ((i * 4 + g) * 64 + lane) * 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[n][0][4 * g + e] += y[e];
      }
    const uint32_t b = tokens_not_finite(x[n], live);
    if (lane == 0) bad[wave] |= b;
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < (N + 3) / 4; ++n)
    if (n * 4 + wave < N) take(n * 4 + wave, x[n]);
}

// ---- fragments

// The lane's addresses in a tile.
struct TileLanes {
  uint32_t row[2];      // of a row's pieces 2 s + lane / 32, s even and odd: 16 bytes of token lane % 32
  uint32_t col[2];      // of transposing reads of the tokens 4 (lane / 32) .. + 3, and of those 8 further on
  __device__ __forceinline__ TileLanes() {
    const uint32_t lane = threadIdx.x & 63, r = lane & 31, hb = lane >> 5;
    row[0] = r * 64 + ((hb ^ ((r >> 2) & 3)) << 4);
    row[1] = row[0] ^ 32;
    const uint32_t c = 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1);
    col[0] = (4 * hb + ((lane >> 2) & 3)) * 64 + ((c ^ hb) << 4) + (lane & 1) * 8;
    col[1] = (col[0] ^ 32) + 8 * 64;
  }
};

template <class C>
__device__ __forceinline__ f32x16 add_pieces(const Quad& a, const Quad& b, f32x16 x) {
  if constexpr (C::F32) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x = __builtin_amdgcn_mfma_f32_32x32x2f32(a.f[e], b.f[e], x, 0, 0, 0);
    return x;
  } else {
    return mfma_32x32x16_bf16(a.h, b.h, x);
  }
}

// x + (rows of an LDS tile) . (the lane's row)
template <class C>
__device__ __forceinline__ f32x16 tile_products(const char* tile, const TileLanes& at, const Quad (&f)[C::NF], f32x16 x) {
#pragma unroll
  for (int s = 0; s < C::NF; ++s) {
    Quad a;
    a.u = *reinterpret_cast<const uint4*>(tile + at.row[s & 1] + (s >> 1) * C::GROUP);
    x = add_pieces<C>(a, f[s], x);
    if (C::NF > 8 && s % 8 == 7) __builtin_amdgcn_sched_barrier(0);      // the registers hold no more reads at once
  }
  return x;
}

// x + (rows of an LDS tile) . (the lane's row of another)
template <class C>
__device__ __forceinline__ f32x16 tile_products(const char* tile, const TileLanes& at, const char* own, f32x16 x) {
#pragma unroll
  for (int s = 0; s < C::NF; ++s) {
    Quad a, b;
    a.u = *reinterpret_cast<const uint4*>(tile + at.row[s & 1] + (s >> 1) * C::GROUP);
    b.u = *reinterpret_cast<const uint4*>(own + at.row[s & 1] + (s >> 1) * C::GROUP);
    x = add_pieces<C>(a, b, x);
  }
  return x;
}

// Transposed fragment of tokens 16 ks .. and channels 32 db ..: element e is channel lane % 32 of token
// 16 ks + 8 (e / 4) + 4 (lane / 32) + e % 4.
template <class C>
__device__ __forceinline__ bf16x8 column_fragment(const char* tile, const TileLanes& at, int ks, int db) {
  union {
    s16x4 h[2];
    bf16x8 f;
  } u;
  const char* p = tile + db * C::GROUP + ks * 1024;
  u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + at.col[0]));
  u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + at.col[1]));
  return u.f;
}

// sums[channel] += weights of the 32 LDS tokens times their rows, for the blocks of channels from B0 on
template <class C, int B0 = 0, int N>
__device__ __forceinline__ void add_columns(const char* tile, const TileLanes& at, const Weights<C>& w, f32x16 (&sums)[N]) {
  if constexpr (C::F32) {
    // channel 32 db + lane % 32: group 2 db + lane / 16 % 2
    const int lane = threadIdx.x & 63;
    int hb = lane >> 5;
    asm volatile("" : "+v"(hb));      // addresses are worked out here: kept through the loops, they would take the sums' registers
    const char* p = tile + ((lane >> 4) & 1) * C::GROUP + (lane & 3) * 4 + hb * 256;
#pragma unroll
    for (int db = 0; db < N; ++db) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int c = ((lane >> 2) & 3) ^ ((2 * (e >> 2) + hb) & 3);      // of token 8 (e / 4) + 4 hb + e % 4
        const float x = *reinterpret_cast<const float*>(p + 2 * (B0 + db) * C::GROUP + (8 * (e >> 2) + (e & 3)) * 64 + c * 16);
        sums[db] = __builtin_amdgcn_mfma_f32_32x32x2f32(x, w.w[e], sums[db], 0, 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  } else {
#pragma unroll
    for (int db = 0; db < N; ++db) {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) sums[db] = mfma_32x32x16_bf16(column_fragment<C>(tile, at, ks, B0 + db), w.w[ks], sums[db]);
      if (C::NB > 4) __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// Weights of a tile with tokens that the lane's token does not see.
__device__ __forceinline__ void mask_weights(float (&x)[16], uint32_t seen) {
  const int mine = static_cast<int>(seen >> (4 * ((threadIdx.x >> 5) & 1)));
#pragma unroll
  for (int e = 0; e < 16; ++e)
    x[e] = __uint_as_float(__float_as_uint(x[e]) & __builtin_amdgcn_sbfe(mine, 8 * (e >> 2) + (e & 3), 1));
}

// sums += weights x of the 32 LDS tokens times their rows. fine: what rounding the weights to bf16 leaves is added as well, in
// the same products once more (weights of 16 bits instead of 8).
template <class C, int B0 = 0, int N>
__device__ __forceinline__ void add_weighted(const char* tile, const TileLanes& at, float (&x)[16], bool fine, f32x16 (&sums)[N]) {
  bool more = !C::F32 && fine;
  while (true) {
    Weights<C> w;
#pragma unroll
    for (int e = 0; e < 16; ++e) w.set(e, x[e]);
    add_columns<C, B0>(tile, at, w, sums);
    if (!more) break;
    more = false;
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] -= static_cast<float>(static_cast<__bf16>(x[e]));
  }
}

// ---- a wave's 32 rows between memory and registers, by way of an LDS tile of its own: memory sees whole rows side by side (a
// lane's own pieces would be 32 bytes of each of 32 rows at a time, and the requests to L2, not the bytes, bound short sequences)

template <class C>
struct WaveRows {
  static constexpr int PIECES = C::DP / C::QE, N = 32 * PIECES / 64;      // of a row; of a lane
  // Piece n of the lane: of row n * 64 / PIECES + lane / PIECES and so on.
  __device__ __forceinline__ static int row(int n) { return (n * 64 + (threadIdx.x & 63)) / PIECES; }
  __device__ __forceinline__ static int piece(int n) { return (n * 64 + (threadIdx.x & 63)) % PIECES; }
  __device__ __forceinline__ static uint32_t place(int n) {
    const int r = row(n), c = piece(n);
    return (c >> 2) * C::GROUP + r * 64 + (((c & 3) ^ ((r >> 2) & 3)) << 4);
  }
  uint4 x[N];
  // Rows row0 .. row0 + 31 of a head that lie below T; zeros from D on. stride in elements.
  __device__ __forceinline__ void load(const void* head, long long stride, int row0, int T, int D, bool wide) {
    const typename C::E* const p = static_cast<const typename C::E*>(head);
    auto at = [&](int n) {
      const int c = piece(n) * C::QE;
      return p + min(row0 + row(n), T - 1) * stride + (c < D ? c : 0);
    };
    if (wide) {
#pragma unroll
      for (int n = 0; n < N; ++n) x[n] = *reinterpret_cast<const uint4*>(at(n));
    } else {
#pragma unroll
      for (int n = 0; n < N; ++n) x[n] = load_elements<C>(at(n));
    }
  }
  __device__ __forceinline__ void keep(char* tile, int D) const {
#pragma unroll
    for (int n = 0; n < N; ++n) *reinterpret_cast<uint4*>(tile + place(n)) = piece(n) * C::QE < D ? x[n] : uint4{0, 0, 0, 0};
    __builtin_amdgcn_wave_barrier();
  }
  // The same a few pieces at a time, for rows whose pieces would take too many registers.
  __device__ __forceinline__ static void bring(char* tile, const void* head, long long stride, int row0, int T, int D, bool wide) {
    const typename C::E* const p = static_cast<const typename C::E*>(head);
    constexpr int STEP = N % 4 == 0 ? 4 : 2;
#pragma unroll 1
    for (int n0 = 0; n0 < N; n0 += STEP) {
      uint4 y[STEP];
#pragma unroll
      for (int i = 0; i < STEP; ++i) {
        const int c = piece(n0 + i) * C::QE;
        const typename C::E* at = p + min(row0 + row(n0 + i), T - 1) * stride + (c < D ? c : 0);
        y[i] = wide ? *reinterpret_cast<const uint4*>(at) : load_elements<C>(at);
        if (c >= D) y[i] = uint4{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < STEP; ++i) *reinterpret_cast<uint4*>(tile + place(n0 + i)) = y[i];
    }
    __builtin_amdgcn_wave_barrier();
  }
  // The lane's half of its row (pieces 2 s + lane / 32): zeros from D on and for tokens that are not live.
  __device__ __forceinline__ static void pick(const char* tile, const TileLanes& at, bool live, Quad (&f)[C::NF]) {
#pragma unroll
    for (int s = 0; s < C::NF; ++s) {
      f[s].u = *reinterpret_cast<const uint4*>(tile + at.row[s & 1] + (s >> 1) * C::GROUP);
      if (!live) f[s].u = uint4{0, 0, 0, 0};
    }
    __builtin_amdgcn_wave_barrier();
  }
};

// The lane's half of its row in two steps: begin() sets the loads going, before it is known which tokens there are; end()
// brings them by way of the tile (long fp32 rows, whose pieces would take too many registers, are loaded then).
template <class C>
struct EarlyRows {
  static constexpr bool EARLY = C::TILE <= 16 * 1024;
  WaveRows<C> rows;
  const void* head;
  long long stride;
  int row0, T, D;
  bool wide;
  __device__ __forceinline__ void begin(const void* head_, long long stride_, int row0_, int T_, int D_, bool wide_) {
    head = head_, stride = stride_, row0 = row0_, T = T_, D = D_, wide = wide_;
    if constexpr (EARLY) rows.load(head, stride, row0, T, D, wide);
  }
  __device__ __forceinline__ void keep(char* tile) const {
    if constexpr (EARLY) rows.keep(tile, D);
    else WaveRows<C>::bring(tile, head, stride, row0, T, D, wide);
  }
  __device__ __forceinline__ void end(char* tile, const TileLanes& at, bool live, Quad (&f)[C::NF]) const {
    keep(tile);
    WaveRows<C>::pick(tile, at, live, f);
  }
};

// The sums of the wave's tokens (channel blocks from B0 on), each times its lane's f, to the rows row0 .. of a head; live: a bit
// for each token that has one.
template <class C, int N>
__device__ __forceinline__ void store_rows(char* tile, void* head, long long stride, int row0, int D, const f32x16 (&s)[N], float f,
                                           uint32_t live, bool wide, int B0 = 0) {
  using R = WaveRows<C>;
  const int lane = threadIdx.x & 63, t = lane & 31, hb = lane >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int g = 0; g < 4; ++g) {      // channels 32 (B0 + i) + 8 g + 4 hb .. + 3
      const int c = C::F32 ? 2 * (g & 1) + hb : g;
      char* at = tile + (C::F32 ? 2 * (B0 + i) + (g >> 1) : B0 + i) * C::GROUP + t * 64 + ((c ^ ((t >> 2) & 3)) << 4);
      if constexpr (C::F32) {
        *reinterpret_cast<f32x4*>(at) = f32x4{s[i][4 * g] * f, s[i][4 * g + 1] * f, s[i][4 * g + 2] * f, s[i][4 * g + 3] * f};
      } else {
        union {
          __bf16 h[4];
          uint2 u;
        } y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y.h[e] = static_cast<__bf16>(s[i][4 * g + e] * f);
        *reinterpret_cast<uint2*>(at + 8 * hb) = y.u;
      }
    }
  __builtin_amdgcn_wave_barrier();
  typename C::E* const p = static_cast<typename C::E*>(head);
  auto each = [&](auto put) {
#pragma unroll
    for (int n = 0; n < R::N; ++n) {
      const int r = R::row(n), c = R::piece(n) * C::QE;
      if (!((live >> r) & 1) || c >= D || c < 32 * B0 || c >= 32 * (B0 + N)) continue;
      put(p + (row0 + r) * stride + c, *reinterpret_cast<const uint4*>(tile + R::place(n)));
    }
  };
  if (wide) {
    each([](typename C::E* at, uint4 y) { *reinterpret_cast<uint4*>(at) = y; });
  } else {
    each([](typename C::E* at, uint4 y) { store_elements<C>(at, y); });
  }
  __builtin_amdgcn_wave_barrier();
}

template <class E>
__device__ __forceinline__ float row_dot(const E* a, const E* b, int D) {
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
  for (int c = 0; c < D; c += 4)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = fmaf(to_f32(a[c + e]), to_f32(b[c + e]), s[e]);
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// o[i] += sum over n <= 64 rows of the lane's weight t (of row t) times channel 64 i + lane.
template <class C, int NC>
__device__ __forceinline__ void add_rows_alone(const typename C::E* rows, long long stride, int n, int D, float weight,
                                               float (&o)[NC]) {
  const int lane = threadIdx.x & 63;
#pragma unroll 1
  for (int t = 0; t < n; t += 8) {
    float x[8][NC];
#pragma unroll
    for (int u = 0; u < 8; ++u)
#pragma unroll
      for (int i = 0; i < NC; ++i) x[u][i] = 64 * i + lane < D ? to_f32(rows[min(t + u, n - 1) * stride + 64 * i + lane]) : 0.0f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (t + u >= n) continue;
      const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(weight), t + u));
#pragma unroll
      for (int i = 0; i < NC; ++i) o[i] = fmaf(w, x[u][i], o[i]);
    }
  }
}

__host__ __device__ inline bool aligned16(const void* p, long long t, long long h, int es) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && t * es % 16 == 0 && h * es % 16 == 0;
}
// Rows that RowLoader can load straight to LDS.
inline bool loads_direct(const void* p, long long t, long long h, int es) {
  return aligned16(p, t, h, es) && t >= 0 && t * es < (1LL << 24);
}

// Whether four waves share a tile of 32 tokens: below a number of blocks of 128 tokens for each CU that grows with the mean length
// of the sequences (short ones leave a wave less than a tile of its own), less where one block of shared tiles fills a CU's LDS
// (bf16 past 128 channels), more in fp32, whose products take longer. us without and with, 16 heads on 4, by blocks of 128:
//   bf16, 128 channels, mean 50: forward 14 and 11 (128 blocks), 15 and 18 (240); gradient 58 and 50, 59 and 66
//                       mean 500: 30 and 22 (240), 32 and 40 (480); 104 and 82, 113 and 121
//                       mean 2000: 122 and 106 (480), 101 and 116 (960); 352 and 352, 334 and 411
//   bf16, 256 channels, mean 50: 25 and 25 (128), 28 and 49 (240); mean 500: 58 and 57 (240), 59 and 106 (480); mean 2000: 126 and
//                       98 (240), 243 and 280 (480)
//   fp32, 96 channels, forward, mean 150: 47 and 49 (240), 64 and 97 (480); mean 500: 127 and 123 (480), 219 and 250 (960); mean
//                       2000: 496 and 488 (960), 902 and 1005 (1920)
//                       gradient, mean 150: 151 and 142 (240), 254 and 247 (480); mean 500: 716 and 667 (960), 1631 and 1355
//                       (1920); mean 2000: 1719 and 1571 (960), 3686 and 3068 (1920)
// One rule serves both directions and follows the forward pass. The fp32 gradient gains by sharing beyond it, at all but one of the
// sizes measured from a mean of 150 on (64 channels, mean 2000, 1920 blocks: 2421 without, as the rule has it, and 1853 with), and
// so, by less, does bf16 with 64 channels (mean 2000, 960 blocks: 230 and 215).
inline bool split_rows(int T, int n_seqs, int heads, int D, bool f32) {
  const int length = T / n_seqs, i = length < 256 ? 0 : length < 1000 ? 1 : 2;
  constexpr int quarters[3][3] = {{3, 5, 8}, {2, 4, 4}, {4, 8, 16}};
  return (T + 127LL) / 128 * heads * 4 <= static_cast<long long>(quarters[f32 ? 2 : D > 128][i]) * device_cu_count();
}

template <class F>
auto with_packed_cfg(moe_dtype act, int D, F f) {
  auto by_dim = [&](auto f32) {
    constexpr bool IS32 = decltype(f32)::value;
    if (D <= 64) return f(PackedCfg<IS32, 64>{});
    if (D <= 96) return f(PackedCfg<IS32, 96>{});
    if (D <= 128) return f(PackedCfg<IS32, 128>{});
    if (D <= 192) return f(PackedCfg<IS32, 192>{});
    return f(PackedCfg<IS32, 256>{});
  };
  return act == MOE_F32 ? by_dim(std::true_type{}) : by_dim(std::false_type{});
}

}  // namespace moe
