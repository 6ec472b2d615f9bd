// spax_paged_attention: one new query token per sequence over a paged cache.
//
// Per (sequence, key head) with keys k_j, values v_j and the group's queries q_h, in one pass:
//   s_hj = scale q_h.k_j,  m = running max of s,  p = exp(s - m),
//   l <- l exp(m_old - m) + sum p,   o <- o exp(m_old - m) + sum p v,   out = o / l.
// Pieces of a sequence (m, l, o) join by the same rule.
//
// Bound: the cache's bytes, each read once for up to 16 query heads of a key head (counted: 1.00 to 1.02
// of them come from memory).  Every further 16 ask for them again, at the same time on the same XCD,
// mostly from its L2: 20 and 48 heads on one key head fetch 1.02 and 1.10 of them.  A wave takes a tile
// of 32 keys at a time:
//   * S^T = K Q^T by 16x16x32 matrix instructions, keys as rows and the group's query heads as
//     columns (16 columns are computed whatever the group; the matrix units have the room).
//   * S^T's layout (lane: one head, keys 4g..4g+3 of each half) is already that of the second
//     product's P operand if that product counts the tile's keys in the order {4g+i, 16+4g+i},
//     so probabilities never cross lanes.
//   * O^T = V^T P^T: a lane reads whole pieces of the rows of its 8 keys (16 lanes cover a row),
//     and swaps 2x2 blocks of 16-bit values with byte permutes to get 8 keys of one dim.
//   * p is split into two 16-bit values, p = hi + lo, each multiplied: rounding p to 16 bits
//     would cost as much error again as rounding the result.  hi + lo keeps p to 2^-17 of itself in
//     bf16 and, since fp16 ends at 2^-24, p 2^15 instead of p (Mma::kLift), in fp16 to the larger of
//     2^-22 of itself and 2^-40 of the largest p.  p itself in fp16 lost what was below 2^-25 of one
//     large key while l kept it: 508 keys at e^-18 of it came out an eighth low, 99 in one wave as 0.
//   * Keys go through LDS, values do not: see Wave.  The next tile's loads are in flight through
//     all of a tile's arithmetic.
//
// The work of a call is known only on the device (lens), so the shares are cut there: every key
// head's sequences, laid end to end, are cut into equal shares, one workgroup each and one
// workgroup per compute unit.  Fixed pieces of a longest possible sequence instead left the
// chip to the long ones (48 sequences of 0 to 8192 keys, when it was changed: 94 us to 50).
//
// Measured (one MI355X; plain reads reach 7.2 TB/s): 32 x 32768 keys, 8 heads of 128, e4m3: 323 us,
// 6.7 TB/s.  1 x 32768, fp16: 27.4 us, of which 24 the shares and 4.6 the join where each is timed by
// itself; 18.6 at the read rate.  48 sequences of 0 to 8192, bf16: 41 us, 4.7 TB/s, with the rows
// of a token's heads side by side, 39.5 with each head's rows together.  1 x 509 keys, 32 heads:
// 8.7 us, latency (time stamps of one workgroup: first loads out at 3.0, first tile done at 5.8,
// the second at 7.0, waves joined and stored at 8.6).
#include "layer_ops.h"
#include "mask_core.h"

namespace spax {
namespace {

using namespace elem;

// Keys that a wave takes per step.  64 of the narrower rows were no faster: 32 x 32768 e4m3 325.7 us
// (32: 323.5), 1 x 2000 of dim 64 11.8 (10.8).
constexpr int kTile = 32;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kJoinThreads = 256;
// Waves per workgroup: two per SIMD leave a wave 256 registers, one leaves 512, which the widest
// 16-bit heads need: 8 x 8192 keys of 256 took 30 us with four waves and 55 with eight, which
// spill (before keys went through LDS, where those of eight would not fit).  8-bit heads of 192 and 256
// keep six to eight registers in scratch with eight waves (28 to 36 bytes a lane; 8 x 8192 keys 21.2 and
// 24.3 us); four were not timed for them.  The others lose with four where latency counts (1 x 509
// keys 8.7 to 11.4 us, 256 x 64 18.5 to 19.8) and gain 1 to 2% at best (32 x 32768 e4m3 325 to 321).
constexpr int waves_of(bool narrow, int dim) { return !narrow && dim >= 192 ? 4 : 8; }
constexpr int kMaxShares = 256;
// What a sequence costs besides its keys, in tiles, and the most tiles of a sequence that a wave
// takes by itself, beside other waves, rather than a workgroup together.  48 sequences of 0 to
// 8192 keys: 41.5 us with (4, 4), 43.4 with (2, 4), 40.9 with (6, 6), which loses as much on
// others (300 x 300 keys 30.8 to 31.3); 64 x 100 keys of 32 heads: 23.6 with (4, 4), 39.4 with (2, 2).
constexpr int kSeqCost = 4;
constexpr int kAlone = 4;

struct AttnArgs {
  const void *q, *k, *v;
  void* out;
  float *lse, *part_o, *part_ml;
  const int32_t *lens, *table;
  const float *k_scale, *v_scale;
  int64_t qs, qh, os, oh;
  int64_t k_page, k_head, k_row, v_page, v_head, v_row, table_stride;
  int32_t n_heads, n_kv, group, head_tiles, n_seqs, n_pages, page_shift;
  int32_t max_len, window, shares, lds_waves, k_lds;
  float scale;
};

// kLift: the exponentials are taken of s - m + kLift (base 2), so the largest is 2^kLift, the most
// that fp16 holds with room for its rounding.  It cancels in o / l, and lse takes it off again.
template <class T>
struct Mma;
template <>
struct Mma<f16> {
  static constexpr float kLift = 15.0f, kUnlift = 0x1p-15f;
  typedef f16 v8 __attribute__((ext_vector_type(8)));
  static __device__ inline f32x4 mul(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8, a),
                                                  __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  // two e4m3 values (the low or high half of w) as 16-bit ones, exactly
  template <bool HI>
  static __device__ inline uint32_t widen(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
  }
  typedef f16x2 v2;
};
template <>
struct Mma<bf16> {
  static constexpr float kLift = 0.0f, kUnlift = 1.0f;
  typedef bf16 v8 __attribute__((ext_vector_type(8)));
  static __device__ inline f32x4 mul(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8, a),
                                                   __builtin_bit_cast(v8, b), c, 0, 0, 0);
  }
  template <bool HI>
  static __device__ inline uint32_t widen(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
  }
  typedef bf16x2 v2;
};

// ln of the sum of exponentials whose largest exponent is m (base 2) and whose lifted sum is l.
template <class T>
__device__ inline float lse_of(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + log2f(l * Mma<T>::kUnlift)) * kLn2;
}

// The cache is read once, so its loads are marked as not worth keeping: 1 x 32768 keys 31.0 us
// without, 27.6 with; 48 ragged 45.7 and 41.5; 32 x 32768 e4m3 330 and 325.
__device__ inline u32x4 load16(const void* p) { return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p)); }

// Orders a wave's own LDS accesses between its lanes: what was written before is read after, and
// nothing read before is overwritten.  The wave's LDS accesses run in order, so this is for the
// compiler and costs no instruction.
__device__ inline void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// N dwords at p (aligned to their own size, at most 16 bytes; 3 dwords never occur).
template <int N>
__device__ inline void load_words(const void* p, uint32_t* w) {
  if constexpr (N == 4) {
    const u32x4 x = load16(p);
    w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
  } else if constexpr (N == 2) {
    const u32x2 x = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
    w[0] = x.x; w[1] = x.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// Values of a lane's piece of a V row: 16 lanes cover a block of 16 * n dims.  A head of D dims
// is one or two such blocks, each lane's piece a power of two.
template <int D>
struct VDims {
  static constexpr int n0 = D == 64 || D == 96 ? 4 : 8;
  static constexpr int n1 = D / 16 - n0;
  static constexpr int n = D / 16;
};

template <class T, bool NARROW, int D>
struct Wave {
  static constexpr int KC = D / 32;          // steps of 32 dims
  static constexpr int VN = D / 16;          // a lane's dims of a V row
  static constexpr int EB = NARROW ? 1 : 2;  // bytes per cached value

  u32x4 q[KC];
  f32x4 o[VN];
  float m, l;  // of head lane % 16: the running max (scaled to log2), this lane's part of the sum

  // K rows are loaded whole, 16 bytes a lane, and laid out in LDS (the wave's own, rows padded by
  // 16 bytes against bank conflicts): read straight into the first operand's layout, adjacent
  // lanes ask for different rows, and issuing the loads takes longer than this detour (1 x 509
  // keys 9.4 us to 8.9, 48 ragged 44.1 to 41.5, 32 x 32768 e4m3 335 to 327).
  static constexpr int RB = D * EB;                    // bytes of a row
  static constexpr int kChunks = RB / 16, kRowLds = RB + 16;
  // Which dims a lane holds for which step is free as long as Q's are the same: 16 bytes per
  // read, so a step of 32 dims of a 16-bit row (dims 32 c + 8 g ..), or two steps of an 8-bit row
  // (64 c + 16 g .. for steps 2c and 2c + 1; a last single step by 8 bytes).
  static constexpr int kPairs = NARROW ? KC / 2 : 0;
  static constexpr int KW = NARROW ? kPairs + (KC & 1) : KC;  // reads
  static __device__ inline void read_k(const uint8_t* row, int g, u32x4 k[KW]) {
#pragma unroll
    for (int c = 0; c < (NARROW ? kPairs : KC); ++c)
      k[c] = *reinterpret_cast<const u32x4*>(row + 64 * c + 16 * g);
    if constexpr (NARROW && (KC & 1)) {
      const u32x2 w = *reinterpret_cast<const u32x2*>(row + 64 * kPairs + 8 * g);
      k[kPairs].x = w.x;
      k[kPairs].y = w.y;
    }
  }
  // Step c's operand.
  static __device__ inline u32x4 k_step(const u32x4 k[KW], int c) {
    if constexpr (NARROW) {
      const u32x4 w = k[c / 2];
      const uint32_t x = c % 2 ? w.z : w.x, y = c % 2 ? w.w : w.y;
      u32x4 r;
      r.x = Mma<T>::template widen<false>(x);
      r.y = Mma<T>::template widen<true>(x);
      r.z = Mma<T>::template widen<false>(y);
      r.w = Mma<T>::template widen<true>(y);
      return r;
    } else {
      return k[c];
    }
  }
  // Byte offset in a Q row of step c's eight values.
  static __device__ inline int q_at(int c, int g) {
    if (NARROW && c < 2 * kPairs) return 2 * (64 * (c / 2) + 16 * g + 8 * (c % 2));
    return 2 * (32 * c + 8 * g);
  }
  // A lane's piece of one V row: VN values, packed as stored.
  static constexpr int VW = (VN * EB + 3) / 4 < 1 ? 1 : (VN * EB + 3) / 4;
  static __device__ inline void load_v(const uint8_t* row, int r, uint32_t* w) {
    constexpr int n0 = VDims<D>::n0, n1 = VDims<D>::n1;
    load_words<n0 * EB / 4>(row + n0 * EB * r, w);
    if constexpr (n1 * EB >= 4)
      load_words<n1 * EB / 4>(row + 16 * n0 * EB + n1 * EB * r, w + n0 * EB / 4);
    else if constexpr (n1 * EB == 2)
      w[n0 * EB / 4] = *reinterpret_cast<const uint16_t*>(row + 16 * n0 * EB + n1 * EB * r);
  }
  // Where a piece's rows are.
  struct Source {
    const int32_t* table;
    const uint8_t *k, *v;
    int64_t k_page, k_row, v_page, v_row;
    int page_shift, n_pages, lo, hi;
    float to_log2;
    // The table entry of key tile * kTile + lane % kTile (past the end: of the last key).
    __device__ inline int look_up(int tile, int lane) const {
      const int at = (tile * kTile + (lane & (kTile - 1))) >> page_shift;
      const int end = (hi - 1) >> page_shift;
      return table[at < end ? at : end];
    }
  };
  // A tile's keys and values: two K operands of 16 keys and one V operand.
  static constexpr int KH = kTile / 16, KI = kTile * kChunks / 64;
  struct Tile {
    u32x4 k[KI];  // chunk (64 i + lane) % kChunks of row (64 i + lane) / kChunks
    uint32_t v[8][VW];
    int page;  // of key lane % kTile, or -1 (see place)
    int kb;
    bool whole;
  };

  __device__ inline void begin() {
#pragma unroll
    for (int c = 0; c < KC; ++c) q[c] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int t = 0; t < VN; ++t) o[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    m = -INFINITY;
    l = 0.0f;
  }
  __device__ inline void load_q(const uint8_t* row, int g) {
#pragma unroll
    for (int c = 0; c < KC; ++c) q[c] = *reinterpret_cast<const u32x4*>(row + q_at(c, g));
  }

  static __device__ inline void place(Tile& x, const Source& s, int tile, int entry, int lane) {
    const int kb = tile * kTile, key = kb + (lane & (kTile - 1));
    // -1 where the key's group of four (always on one page) has no key in [lo, hi) or the entry
    // names no page: such rows are read from page 0 and then masked
    const bool ok = (key | 3) >= s.lo && (key & ~3) < s.hi && (uint32_t)entry < (uint32_t)s.n_pages;
    x.page = ok ? entry : -1;
    x.kb = kb;
    x.whole = kb >= s.lo && kb + kTile <= s.hi && __all(ok);
  }
  static __device__ inline void load_keys(Tile& x, const Source& s, int lane) {
    const int row_mask = (1 << s.page_shift) - 1;
#pragma unroll
    for (int i = 0; i < KI; ++i) {
      const int row = (64 * i + lane) / kChunks, chunk = (64 * i + lane) % kChunks;
      const int pg = __shfl(x.page, row);
      const int64_t at = (int64_t)(pg < 0 ? 0 : pg) * s.k_page +
                         (int64_t)((x.kb + row) & row_mask) * s.k_row;
      x.k[i] = load16(s.k + EB * at + 16 * chunk);
    }
  }
  static __device__ inline void load_values(Tile& x, const Source& s, int lane) {
    const int g = lane >> 4, r = lane & 15, row_mask = (1 << s.page_shift) - 1;
#pragma unroll
    for (int h = 0; h < KH; ++h) {
      const int pg = __shfl(x.page, 16 * h + 4 * g);
      const int64_t row = (int64_t)(pg < 0 ? 0 : pg) * s.v_page +
                          (int64_t)((x.kb + 16 * h + 4 * g) & row_mask) * s.v_row;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        load_v(s.v + EB * (row + i * s.v_row), r, x.v[4 * h + i]);
    }
  }

  static __device__ inline void lay_out_keys(const Tile& x, uint8_t* rows, int lane) {
#pragma unroll
    for (int i = 0; i < KI; ++i) {
      const int row = (64 * i + lane) / kChunks, chunk = (64 * i + lane) % kChunks;
      *reinterpret_cast<u32x4*>(rows + row * kRowLds + 16 * chunk) = x.k[i];
    }
  }
  // Scores of the tile's keys in base 2; a lane's are keys 16 h + 4 g + i of its head.
  __device__ inline void score(const uint8_t* rows, const Source& src, int lane, float p[4 * KH]) {
#pragma unroll
    for (int h = 0; h < KH; ++h) {
      u32x4 k[KW];
      read_k(rows + (16 * h + (lane & 15)) * kRowLds, lane >> 4, k);
      f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int c = 0; c < KC; ++c) s = Mma<T>::mul(k_step(k, c), q[c], s);
#pragma unroll
      for (int i = 0; i < 4; ++i) p[4 * h + i] = s[i] * src.to_log2;
    }
  }

  // Masks keys that do not count: their scores and, since 0 * NaN is NaN, their values.
  static __device__ inline void mask_out(Tile& x, const Source& src, int lane, float p[4 * KH]) {
    const int g = lane >> 4;
#pragma unroll
    for (int h = 0; h < KH; ++h) {
      const int pg = __shfl(x.page, 16 * h + 4 * g);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = x.kb + 16 * h + 4 * g + i;
        const uint32_t keep = key >= src.lo && key < src.hi && pg >= 0 ? ~0u : 0u;
        p[4 * h + i] = keep ? p[4 * h + i] : -INFINITY;
#pragma unroll
        for (int y = 0; y < VW; ++y) x.v[4 * h + i][y] &= keep;
      }
    }
  }

  // o * f as this head's result.  A lane has dims (4 g + i) n0 + t of the first block of 16 n0
  // and, after o[n0 - 1], (4 g + i) n1 + t of the second.
  __device__ inline void put(T* out, int g, float f) const {
    constexpr int n0 = VDims<D>::n0, n1 = VDims<D>::n1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x[VN];
#pragma unroll
      for (int t = 0; t < VN; ++t) x[t] = f == 0.0f ? 0.0f : o[t][i] * f;
      store_n<n0>(out + (4 * g + i) * n0, x);
      if constexpr (n1 > 0) store_n<n1>(out + 16 * n0 + (4 * g + i) * n1, x + n0);
    }
  }

  // The softmax step and the product with the tile's values.
  __device__ inline void take(Tile& x, const Source& src, int lane, float p[4 * KH]) {
    if (!x.whole) mask_out(x, src, lane, p);
    float top = p[0];
#pragma unroll
    for (int i = 1; i < 4 * KH; ++i) top = fmaxf(top, p[i]);
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    if (__any(top > m)) {
      const float higher = fmaxf(m, top);
      const float f = higher == m ? 1.0f : __builtin_amdgcn_exp2f(m - higher);
      m = higher;
      l *= f;
#pragma unroll
      for (int t = 0; t < VN; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[t][i] *= f;
    }
    const float base = (m == -INFINITY ? 0.0f : m) - Mma<T>::kLift;
    u32x4 hi2, lo2;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float p0 = __builtin_amdgcn_exp2f(p[i] - base);
      const float p1 = __builtin_amdgcn_exp2f(p[i + 1] - base);
      l += p0 + p1;
      typename Mma<T>::v2 h, rest;
      h.x = (T)p0;
      h.y = (T)p1;
      rest.x = (T)(p0 - (float)h.x);
      rest.y = (T)(p1 - (float)h.y);
      hi2[i / 2] = __builtin_bit_cast(uint32_t, h);
      lo2[i / 2] = __builtin_bit_cast(uint32_t, rest);
    }
    // 8 keys of each dim, pair by pair: byte permutes of two rows' words
#pragma unroll
    for (int t2 = 0; t2 < VN / 2; ++t2) {
      uint32_t y[8];  // dims 2 t2 and 2 t2 + 1 of the 8 keys, 16-bit
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (NARROW)
          y[i] = t2 % 2 ? Mma<T>::template widen<true>(x.v[i][t2 / 2])
                        : Mma<T>::template widen<false>(x.v[i][t2 / 2]);
        else
          y[i] = x.v[i][t2];
      }
      u32x4 even, odd;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        even[i] = __builtin_amdgcn_perm(y[2 * i + 1], y[2 * i], 0x05040100u);
        odd[i] = __builtin_amdgcn_perm(y[2 * i + 1], y[2 * i], 0x07060302u);
      }
      o[2 * t2] = Mma<T>::mul(even, hi2, o[2 * t2]);
      o[2 * t2 + 1] = Mma<T>::mul(odd, hi2, o[2 * t2 + 1]);
      o[2 * t2] = Mma<T>::mul(even, lo2, o[2 * t2]);
      o[2 * t2 + 1] = Mma<T>::mul(odd, lo2, o[2 * t2 + 1]);
    }
  }
};

// The keys [lo, hi) of a sequence that count, and the tiles they lie in.
struct Keys {
  int lo, hi, first, tiles;
};
__device__ inline Keys keys_of(const AttnArgs& a, int n) {
  Keys k;
  k.hi = n < 0 ? 0 : n > a.max_len ? a.max_len : n;
  k.lo = a.window > 0 && k.hi > a.window ? k.hi - a.window : 0;
  k.first = k.lo / kTile;
  k.tiles = (k.hi + kTile - 1) / kTile - k.first;
  return k;
}

// The sequences laid end to end, each as kSeqCost units and then one per tile, cut into a.shares
// equal shares (the units fit 31 bits).  Every wave finds its place by itself: lane l holds
// sequence base + l, and a scan over the lanes gives where each ends.  Past 64 sequences that is a
// chain of loads, one for every 64, in each wave of both launches: 1024 sequences of 32 keys (one key
// head of 64) take 19 us, 4096 take 60, 16384 take 283, a microsecond for every 64.
template <int WAVES>
struct Line {
  int base, len;     // this lane's sequence: base + lane
  int units;         // its kSeqCost + tiles (0 past the last sequence)
  int upto;          // units of the sequences before base + lane + 1
  int last;          // upto of lane 63
  int total, share;  // units in all and per share

  __device__ inline void load(const AttnArgs& a, int lane, int from, int before) {
    base = from;
    const int s = base + lane;
    len = s < a.n_seqs ? a.lens[s] : 0;
    units = s < a.n_seqs ? kSeqCost + keys_of(a, len).tiles : 0;
    upto = before + mask::wave_scan(units);
    last = __builtin_amdgcn_readlane(upto, 63);
  }
  __device__ inline void start(const AttnArgs& a, int lane) {
    load(a, lane, 0, 0);
    total = last;
    if (a.n_seqs > 64) {
      while (base + 64 < a.n_seqs) load(a, lane, base + 64, last);
      total = last;
      load(a, lane, 0, 0);
    }
    share = (int)(((uint32_t)total + (uint32_t)a.shares - 1u) / (uint32_t)a.shares);
  }
  // The lane whose sequence holds unit x < total, at or past the loaded block.
  __device__ inline int find(const AttnArgs& a, int lane, int x) {
    while (x >= last) load(a, lane, base + 64, last);
    return __builtin_ctzll(__ballot(upto > x));
  }
  __device__ inline int share_of(int x) const { return (int)((uint32_t)x / (uint32_t)share); }
  // How many sequences from lane `who` on (at most one per wave) are short and lie in [at, stop).
  __device__ inline int short_run(int who, int at, int stop) const {
    const uint64_t fits = __ballot(units > 0 && units <= kSeqCost + kAlone && upto <= stop &&
                                   upto - units >= at);
    const uint64_t rest = ~(fits >> who);
    const int n = rest ? __builtin_ctzll(rest) : 64;
    return n < WAVES ? n : WAVES;
  }
  // Of the sequence in lane `who`.
  __device__ inline int length(int who) const { return __builtin_amdgcn_readlane(len, who); }
  __device__ inline int end(int who) const { return __builtin_amdgcn_readlane(upto, who); }
  __device__ inline int begin(int who) const {  // of its tiles
    return end(who) - __builtin_amdgcn_readlane(units, who) + kSeqCost;
  }
};

template <class T, bool NARROW, int D>
__global__ __launch_bounds__(64 * waves_of(NARROW, D)) void attention_kernel(AttnArgs a) {
  using W = Wave<T, NARROW, D>;
  constexpr int EB = W::EB, VN = W::VN, kWaves = waves_of(NARROW, D);
  extern __shared__ float lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, r = lane & 15;

  // Work item: a share of the line for one key head (16 of its query heads).  Workgroups go to the
  // 8 XCDs in turn; an XCD gets neighbouring items, so that the heads of a share, whose rows
  // lie side by side in the cache, are read through the same caches and translations.
  const int n_hh = a.n_kv * a.head_tiles;
  const int per_xcd = gridDim.x >> 3;
  const int item = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
  const int share = item / n_hh, hh = item % n_hh;
  if (share >= a.shares) return;
  const int kvh = hh / a.head_tiles, ht = hh % a.head_tiles;
  const int heads = a.group - 16 * ht < 16 ? a.group - 16 * ht : 16;  // of this workgroup
  const int head0 = kvh * a.group + 16 * ht;

  float to_log2 = a.scale * kLog2e, v_mul = 1.0f;
  if constexpr (NARROW) {
    if (a.k_scale) to_log2 *= a.k_scale[kvh];
    if (a.v_scale) v_mul = a.v_scale[kvh];
  }
  const uint8_t* kbase = (const uint8_t*)a.k + (int64_t)EB * kvh * a.k_head;
  const uint8_t* vbase = (const uint8_t*)a.v + (int64_t)EB * kvh * a.v_head;

  uint8_t* k_rows = reinterpret_cast<uint8_t*>(lds) + a.k_lds + wave * (kTile * W::kRowLds);
  Line<kWaves> line;
  line.start(a, lane);
  int at = share * line.share;
  const int stop = at + line.share < line.total ? at + line.share : line.total;
  int who = at < stop ? line.find(a, lane, at) : 0;
  bool again = false;
  while (at < stop) {
    if (who == 64) who = line.find(a, lane, at);
    // Short sequences that lie whole in this share go to one wave each, side by side.
    const int run = line.short_run(who, at, stop);
    const bool alone = run > 1;
    if (alone && wave >= run) {
      at = line.end(who + run - 1);
      who += run;
      continue;
    }
    const int mine = alone ? who + wave : who;
    const int seq = line.base + mine;
    const Keys x = keys_of(a, line.length(mine));
    const int ends = line.end(mine), begins = ends - x.tiles;  // of its tiles
    const bool answers = at <= begins - kSeqCost;              // its first unit is in this share
    const int from = at > begins ? at : begins, to = ends < stop ? ends : stop;
    who += alone ? run : 1;
    at = line.end(who - 1);
    // a sequence of no keys is answered where it begins; otherwise only tiles make a piece
    if (x.tiles == 0 ? !answers : from >= to) continue;
    const int t0 = x.first + from - begins;
    const int t1 = x.tiles ? x.first + to - begins : t0;
    const int step = alone ? 1 : kWaves;

    W w;
    w.begin();
    if (r < heads) w.load_q((const uint8_t*)a.q + 2 * (seq * a.qs + (head0 + r) * a.qh), g);
    const typename W::Source src{a.table + seq * a.table_stride, kbase, vbase, a.k_page, a.k_row,
                                 a.v_page, a.v_row, a.page_shift, a.n_pages, x.lo, x.hi, to_log2};
    int tile = alone ? t0 : t0 + wave;
    if (tile < t1) {
      // The next tile's keys are loaded once this one's are used, its values likewise, so loads
      // are in flight through all of the arithmetic.  Its table entry was loaded ahead of this
      // tile, so it never waits behind one.
      typename W::Tile z;
      W::place(z, src, tile, src.look_up(tile, lane), lane);
      int next = src.look_up(tile + step, lane);
      W::load_keys(z, src, lane);
      W::load_values(z, src, lane);
      for (;;) {
        float p[4 * W::KH];
        wave_lds_order();  // the last tile's rows have been read
        W::lay_out_keys(z, k_rows, lane);
        wave_lds_order();
        tile += step;
        if (tile >= t1) {
          w.score(k_rows, src, lane, p);
          w.take(z, src, lane, p);
          break;
        }
        typename W::Tile after;  // its k and v are z's registers
        W::place(after, src, tile, next, lane);
        next = src.look_up(tile + step, lane);
        W::load_keys(after, src, lane);
        w.score(k_rows, src, lane, p);
        w.take(z, src, lane, p);
        W::load_values(after, src, lane);
        z = after;
      }
    }

    w.l += __shfl_xor(w.l, 16);
    w.l += __shfl_xor(w.l, 32);
    if (alone) {
      if (r < heads) {
        T* out = (T*)a.out + seq * a.os + (head0 + r) * a.oh;
        w.put(out, g, w.l == 0.0f ? 0.0f : v_mul / w.l);
        if (a.lse && g == 0)
          a.lse[(int64_t)seq * a.n_heads + head0 + r] = lse_of<T>(w.m, w.l);
      }
      continue;
    }

    // Join the waves: m and l through LDS, then o of a.lds_waves waves at a time, a block of dims
    // at a time, each wave's scaled to the common maximum before it is stored.
    if (again) __syncthreads();  // the last piece's are still being read
    again = true;
    constexpr int n0 = VDims<D>::n0, n1 = VDims<D>::n1;
    constexpr int kStride = 16 * n0 + 4;  // n1 <= n0
    constexpr int kPer = (16 * 4 * n0 + 64 * kWaves - 1) / (64 * kWaves);  // four-value items per thread
    float* ml = lds;               // [wave][16][2]
    float* ob = lds + kWaves * 32;     // [slot][heads][kStride]
    if (g == 0) {
      ml[(wave * 16 + r) * 2] = w.m;
      ml[(wave * 16 + r) * 2 + 1] = w.l;
    }
    __syncthreads();
    float m_all = -INFINITY;
#pragma unroll
    for (int y = 0; y < kWaves; ++y) m_all = fmaxf(m_all, ml[(y * 16 + r) * 2]);
    const float f_own = __builtin_amdgcn_exp2f(w.m - (m_all == -INFINITY ? 0.0f : m_all));
    // the whole sequence, or the first or a later piece of it
    const bool last = x.tiles == 0 || to - from == x.tiles;
    const int which = from == begins;
#pragma unroll
    for (int block = 0; block < (n1 ? 2 : 1); ++block) {
      const int n = block ? n1 : n0;
      const int t_base = block ? n0 : 0;
      const int items = heads * 4 * n;  // four values of one head each
      f32x4 sum[kPer];
#pragma unroll
      for (int y = 0; y < kPer; ++y) sum[y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      for (int from = 0; from < kWaves; from += a.lds_waves) {
        if (block || from) __syncthreads();
        if (r < heads && wave >= from && wave < from + a.lds_waves) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int t = 0; t < n0; ++t)
              if (t < n)
                ob[((wave - from) * heads + r) * kStride + (4 * g + i) * n + t] =
                    w.o[t_base + t < VN ? t_base + t : 0][i] * f_own;
        }
        __syncthreads();
#pragma unroll
        for (int y = 0; y < kPer; ++y) {
          const int e = threadIdx.x + y * 64 * kWaves;
          if (e < items) {
            const int h = e / (4 * n), d = 4 * (e % (4 * n));
            for (int z = 0; z < a.lds_waves; ++z)
              sum[y] += *reinterpret_cast<const f32x4*>(&ob[(z * heads + h) * kStride + d]);
          }
        }
      }
#pragma unroll
      for (int y = 0; y < kPer; ++y) {
        const int e = threadIdx.x + y * 64 * kWaves;
        if (e >= items) continue;
        const int h = e / (4 * n), dim = (block ? 16 * n0 : 0) + 4 * (e % (4 * n));
        float m = -INFINITY, l = 0.0f;
#pragma unroll
        for (int z = 0; z < kWaves; ++z) m = fmaxf(m, ml[(z * 16 + h) * 2]);
        const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int z = 0; z < kWaves; ++z)
          l += __builtin_amdgcn_exp2f(ml[(z * 16 + h) * 2] - base) * ml[(z * 16 + h) * 2 + 1];
        if (last) {
          const float inv = v_mul / l;
          float out[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) out[i] = l == 0.0f ? 0.0f : sum[y][i] * inv;
          store_n<4>((T*)a.out + seq * a.os + (head0 + h) * a.oh + dim, out);
          if (a.lse && dim == 0)
            a.lse[(int64_t)seq * a.n_heads + head0 + h] = lse_of<T>(m, l);
        } else {
          const int64_t part = 2 * ((int64_t)(head0 + h) * a.shares + share) + which;
          *reinterpret_cast<f32x4*>(a.part_o + part * D + dim) = sum[y];
          if (dim == 0) {
            a.part_ml[2 * part] = m;
            a.part_ml[2 * part + 1] = l;
          }
        }
      }
    }
  }
}

// Joins the pieces of a sequence that was cut: one workgroup per cut and head, of which that of
// the sequence's first cut works.  A launch of its own, 4 us: joined by the last workgroup to
// arrive, through a counter and writes past the L2s, 1 x 32768 took 29.6 us against 28.4, and the
// workspace would have to be kept zeroed.  Heads of 64 keep eight registers in scratch under the
// launch bound.  A share writes at most two pieces of a head: the end of a
// sequence (0) and the beginning of another (1).
template <class T, bool NARROW, int D>
__global__ __launch_bounds__(kJoinThreads, 8) void attention_join_kernel(AttnArgs a) {
  constexpr int kLanes = D / 4;                     // threads per piece
  constexpr int kAtOnce = kJoinThreads / kLanes;    // pieces per round
  constexpr int kFirst = 4;                         // rounds loaded before the weights are known
  __shared__ float lds_o[kAtOnce][D];
  __shared__ float lds_w[kMaxShares];
  const int head = blockIdx.x % a.n_heads, cut = blockIdx.x / a.n_heads + 1;
  const int tid = threadIdx.x, lane = tid & 63;
  Line<waves_of(NARROW, D)> line;
  line.start(a, lane);
  const int x = cut * line.share;
  if (x >= line.total) return;
  const int who = line.find(a, lane, x);
  const int ends = line.end(who), begins = line.begin(who);
  if (x <= begins || line.share_of(begins) != cut - 1) return;
  const int pieces = line.share_of(ends - 1) - cut + 2, seq = line.base + who;

  // piece c of this head: the beginning from the share before the cut, the rest from there on
  const int64_t base = 2 * ((int64_t)head * a.shares + cut - 1);
  const auto place = [&](int c) { return base + (c ? 2 * c : 1); };
  const int part = tid / kLanes, d = 4 * (tid % kLanes);
  // every wave: the common maximum, the weights and their sum, 64 pieces at a time
  const float* ml = a.part_ml;
  const bool has = lane < pieces;
  const float m0 = has ? ml[2 * place(lane)] : -INFINITY;
  const float l0 = has ? ml[2 * place(lane) + 1] : 0.0f;
  const float* p = a.part_o + d;
  f32x4 o[kFirst];
#pragma unroll
  for (int y = 0; y < kFirst; ++y) {
    const int c = part + y * kAtOnce;
    if (part < kAtOnce && c < pieces) o[y] = *reinterpret_cast<const f32x4*>(p + place(c) * D);
  }
  float m = m0;
  for (int c = lane + 64; c < pieces; c += 64) m = fmaxf(m, ml[2 * place(c)]);
#pragma unroll
  for (int z = 32; z > 0; z >>= 1) m = fmaxf(m, __shfl_xor(m, z));
  const float top = m == -INFINITY ? 0.0f : m;
  const float f0 = __builtin_amdgcn_exp2f(m0 - top);
  float l = f0 * l0;
  if (tid < 64) lds_w[lane] = f0;
  for (int c = lane + 64; c < pieces; c += 64) {
    const float f = __builtin_amdgcn_exp2f(ml[2 * place(c)] - top);
    l += f * ml[2 * place(c) + 1];
    if (tid < 64) lds_w[c] = f;
  }
#pragma unroll
  for (int z = 32; z > 0; z >>= 1) l += __shfl_xor(l, z);
  mask::lds_barrier();
  if (part < kAtOnce) {
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int y = 0; y < kFirst; ++y) {
      const int c = part + y * kAtOnce;
      if (c < pieces) sum += o[y] * lds_w[c];
    }
    for (int c = part + kFirst * kAtOnce; c < pieces; c += kAtOnce)
      sum += *reinterpret_cast<const f32x4*>(p + place(c) * D) * lds_w[c];
    *reinterpret_cast<f32x4*>(&lds_o[part][d]) = sum;
  }
  __syncthreads();
  if (tid >= kLanes) return;
  f32x4 total = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int y = 0; y < kAtOnce; ++y) total += *reinterpret_cast<const f32x4*>(&lds_o[y][d]);
  const float inv = (a.v_scale ? a.v_scale[head / a.group] : 1.0f) / l;
  float out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = l == 0.0f ? 0.0f : total[i] * inv;
  store_n<4>((T*)a.out + seq * a.os + head * a.oh + d, out);
  if (a.lse && d == 0)
    a.lse[(int64_t)seq * a.n_heads + head] = lse_of<T>(m, l);
}

template <class T, bool NARROW, int D>
void start(AttnArgs a, hipStream_t s) {
  constexpr int kWaves = waves_of(NARROW, D);
  const int heads = a.group < 16 ? a.group : 16;
  // as many waves' o at a time as fit 60 KB of LDS
  const size_t per = sizeof(float) * (size_t)heads * (16 * VDims<D>::n0 + 4);
  a.lds_waves = kWaves;
  while (a.lds_waves > 1 && a.lds_waves * per > 60 * 1024) a.lds_waves /= 2;
  a.k_lds = (int32_t)(sizeof(float) * kWaves * 32 + a.lds_waves * per);
  const size_t lds = a.k_lds + (size_t)kWaves * kTile * (D * (NARROW ? 1 : 2) + 16);
  const unsigned items = (unsigned)(a.n_kv * a.head_tiles * a.shares);
  const dim3 grid((items + 7) / 8 * 8);
  hipLaunchKernelGGL((attention_kernel<T, NARROW, D>), grid, dim3(64 * kWaves), lds, s, a);
}

template <class T, bool NARROW, int D>
int launch(const AttnArgs& a, hipStream_t s) {
  start<T, NARROW, D>(a, s);
  SPAX_HIP_CHECK(hipGetLastError());
  if (a.shares > 1) {
    hipLaunchKernelGGL((attention_join_kernel<T, NARROW, D>), dim3((unsigned)((a.shares - 1) * a.n_heads)),
                       dim3(kJoinThreads), 0, s, a);
    SPAX_HIP_CHECK(hipGetLastError());
  }
  return SPAX_OK;
}

template <class T, bool NARROW>
int launch_dim(const AttnArgs& a, int dim, hipStream_t s) {
  switch (dim) {
    case 64: return launch<T, NARROW, 64>(a, s);
    case 96: return launch<T, NARROW, 96>(a, s);
    case 128: return launch<T, NARROW, 128>(a, s);
    case 192: return launch<T, NARROW, 192>(a, s);
    default: return launch<T, NARROW, 256>(a, s);
  }
}

}  // namespace

AttentionPlan attention_plan(const spax_attention_args* a) {
  const spax_kv_cache& c = *a->cache;
  AttentionPlan p{};
  const int group = a->n_heads / c.n_kv_heads;
  p.head_tiles = (group + 15) / 16;
  const bool narrow = c.type == SPAX_E4M3;
  const int waves = waves_of(narrow, c.head_dim);
  int64_t tiles = ((int64_t)a->max_len + kTile - 1) / kTile;
  if (a->window > 0) {
    const int64_t w = ((int64_t)a->window + kTile - 1) / kTile + 1;  // a window starts anywhere
    if (w < tiles) tiles = w;
  }
  p.units = c.n_seqs * (tiles + kSeqCost);
  // Joining the pieces is a second launch, as long as about three steps of a wave: up to three steps
  // for each wave of one workgroup are not shared out (1 x 509 keys: 8.7 us whole, 11.8 shared;
  // 1 x 700 of 8 heads 10.5 and 11.9).  Past that one workgroup per compute unit (of 256), as long
  // as each wave has a tile (1 x 2000 keys of one head of 64: 12.3 us, 14.4 whole).
  const int64_t all = c.n_seqs * tiles;
  const int64_t most = all <= 3 * waves ? 1 : (all + waves - 1) / waves;
  int64_t shares = 256 / ((int64_t)c.n_kv_heads * p.head_tiles);
  shares = shares > most ? most : shares;
  p.shares = (int32_t)(shares < 1 ? 1 : shares > kMaxShares ? kMaxShares : shares);
  if (p.shares > 1)
    p.ws_bytes = aligned_size((size_t)a->n_heads * p.shares * 2 * ((size_t)c.head_dim + 2) *
                              sizeof(float));
  return p;
}

int launch_attention(const spax_attention_args* p, void* ws, hipStream_t s) {
  const spax_kv_cache& c = *p->cache;
  const AttentionPlan plan = attention_plan(p);
  AttnArgs a{};
  a.q = p->q; a.k = c.k; a.v = c.v; a.out = p->out; a.lse = p->lse;
  a.lens = p->lens; a.table = c.page_table; a.k_scale = c.k_scale; a.v_scale = c.v_scale;
  a.qs = p->q_seq_stride; a.qh = p->q_head_stride;
  a.os = p->out_seq_stride; a.oh = p->out_head_stride;
  a.k_page = c.k_page_stride; a.k_head = c.k_head_stride; a.k_row = c.k_row_stride;
  a.v_page = c.v_page_stride; a.v_head = c.v_head_stride; a.v_row = c.v_row_stride;
  a.table_stride = c.table_stride;
  a.n_heads = p->n_heads; a.n_kv = c.n_kv_heads; a.group = p->n_heads / c.n_kv_heads;
  a.head_tiles = plan.head_tiles; a.n_seqs = c.n_seqs; a.n_pages = c.n_pages;
  a.page_shift = __builtin_ctz((unsigned)c.page_size);
  a.max_len = p->max_len; a.window = p->window; a.scale = p->scale;
  a.shares = plan.shares;
  a.part_o = (float*)ws;
  a.part_ml = (float*)ws + (size_t)2 * p->n_heads * plan.shares * c.head_dim;
  if (c.type == SPAX_E4M3)
    return p->type == SPAX_F16 ? launch_dim<f16, true>(a, c.head_dim, s)
                               : launch_dim<bf16, true>(a, c.head_dim, s);
  return p->type == SPAX_F16 ? launch_dim<f16, false>(a, c.head_dim, s)
                             : launch_dim<bf16, false>(a, c.head_dim, s);
}

}  // namespace spax
