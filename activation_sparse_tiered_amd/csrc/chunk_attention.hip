// spax_chunk_attention: a chunk of new query tokens per sequence over a paged cache, causal.
//
// A sequence's query rows for one key head, tokens times the group's heads, are laid end to end and
// cut into tiles of 128, so any group fills them.  Per row with keys k_j, values v_j, in one pass:
//   s_j = scale q.k_j,  m = running max of s,  p = exp(s - m),
//   l <- l exp(m_old - m) + sum p,   o <- o exp(m_old - m) + sum p v,   out = o / l.
// Pieces of a tile's keys (m, l, o) join by the same rule.
//
// A workgroup of four waves takes a tile, 32 rows a wave, and walks over its keys, kKeys at a time,
// which pass through LDS once for all four:
//   * S^T = K Q^T by 32x32x16 matrix instructions, keys as rows, query rows as columns.
//   * S^T's layout (lane: one row, keys 8 b + 4 h + i) is that of the second product's P operand if
//     that product counts keys in the order {4 h + i, 8 + 4 h + i} of every 16, so probabilities
//     never cross lanes and a row's maximum and sum are in two lanes.
//   * O^T = V^T P^T: eight keys of one dim come from LDS by transposing reads of four rows.
//   * p enters the product as one 16-bit value, in fp16 lifted by 2^15 (Mma::kLift): splitting it
//     in two, as the attention of single tokens does, would add half of the matrix work again where
//     that is the bound, for an error that is about that of rounding the result.
//   * Masked keys get p = 0, but 0 * inf is NaN: in tiles that some row does not see whole, values
//     that are not finite are taken out of the product and counted apart (see take_values).
#include "attn_core.h"
#include "layer_ops.h"
#include "mask_core.h"

namespace spax {
namespace {

using namespace elem;
using namespace attn;

// Query rows of a tile of so many waves.
constexpr int rows_of(int waves) { return 32 * waves; }

struct ChunkArgs {
  const void *q, *k, *v;
  void* out;
  float *lse, *part_o, *part_ml;
  const int32_t *starts, *lens, *table;
  const float *k_scale, *v_scale;
  int64_t qt, qh, ot, oh;
  int64_t k_page, k_head, k_row, v_page, v_head, v_row, table_stride;
  int32_t n_tokens, n_heads, n_kv, group, n_seqs, n_pages, page_shift;
  int32_t max_len, window, rows, tiles, pieces, least_steps;  // rows: of a tile
  float scale;
};

// A tile of query rows: rows from..to of sequence seq's n_new * group, for one key head.
struct Tile {
  int seq, first, n_new, len;  // first: its first token's row of q
  int from, to;                // from == to: no such tile
  __device__ inline int position(int token) const { return len - n_new + token; }
};

__device__ inline int clamp_to(int x, int most) { return x < 0 ? 0 : x > most ? most : x; }

// The keys [lo, hi) that the token at position p sees.
__device__ inline int lo_of(const ChunkArgs& a, int p) {
  return a.window > 0 && p + 1 > a.window ? p + 1 - a.window : 0;
}
__device__ inline int hi_of(int p) { return p < 0 ? 0 : p + 1; }

// Steps of `keys` keys that hold [lo, hi).
__device__ inline int steps_in(int lo, int hi, int keys) {
  return hi > lo ? (hi + keys - 1) / keys - lo / keys : 0;
}

// Sequence s = base + lane: its first row, new tokens and tiles.
struct Seq {
  int first, n_new, tiles;
};
__device__ inline Seq seq_at(const ChunkArgs& a, int s) {
  Seq q{0, 0, 0};
  if (s < a.n_seqs) {
    q.first = clamp_to(a.starts[s], a.n_tokens);
    const int n = clamp_to(a.starts[s + 1], a.n_tokens) - q.first;
    q.n_new = n < 0 ? 0 : n;
    q.tiles = (q.n_new * a.group + a.rows - 1) / a.rows;
  }
  return q;
}

// Tile `index` of all sequences' tiles laid end to end.  Lane l holds sequence base + l; past 64
// sequences that is a chain of loads, one for every 64.
__device__ inline Tile find_tile(const ChunkArgs& a, int index, int lane) {
  int before = 0;
  for (int base = 0; base < a.n_seqs; base += 64) {
    const Seq q = seq_at(a, base + lane);
    const int upto = before + mask::wave_scan(q.tiles);
    const int last = __builtin_amdgcn_readlane(upto, 63);
    if (index < last) {
      const int who = __builtin_ctzll(__ballot(upto > index));
      Tile t;
      t.seq = base + who;
      t.first = __builtin_amdgcn_readlane(q.first, who);
      t.n_new = __builtin_amdgcn_readlane(q.n_new, who);
      t.len = __builtin_amdgcn_readfirstlane(clamp_to(a.lens[t.seq], a.max_len));
      const int begins =
          __builtin_amdgcn_readlane(upto, who) - __builtin_amdgcn_readlane(q.tiles, who);
      t.from = (index - begins) * a.rows;
      const int rows = t.n_new * a.group;
      t.to = t.from + a.rows < rows ? t.from + a.rows : rows;
      return t;
    }
    before = last;
  }
  return Tile{0, 0, 0, 0, 0, 0};
}

// How many steps of a tile's keys make a piece: an equal share of all tiles' steps for each of kShares
// workgroups, but no fewer than the plan has room for.  Every wave of both launches finds the same
// number, in integers, from at most kCounted sequences; with more the plan's own stands.
constexpr int kShares = 512, kCounted = 256;
__device__ inline int piece_steps(const ChunkArgs& a, int keys, int lane) {
  if (a.pieces == 1 || a.n_seqs > kCounted) return a.least_steps;
  int mine = 0;
  for (int base = 0; base < a.n_seqs; base += 64) {
    const int s = base + lane;
    const Seq q = seq_at(a, s);
    if (q.n_new == 0) continue;
    const int len = clamp_to(a.lens[s], a.max_len), p = len - q.n_new;
    // of the first token and of the last
    const int some = steps_in(lo_of(a, p), hi_of(p), keys);
    const int more = steps_in(lo_of(a, len - 1), hi_of(len - 1), keys);
    const int64_t units = (int64_t)q.tiles * ((some + more + 1) / 2);
    constexpr int kMost = 1 << 22;  // kCounted of them stay below 2^31
    mine += units < kMost ? (int)units : kMost;
  }
#pragma unroll
  for (int z = 32; z > 0; z >>= 1) mine += __shfl_xor(mine, z);
  mine = __builtin_amdgcn_readfirstlane(mine);
  const int64_t share = ((int64_t)mine * a.n_kv + kShares - 1) / kShares;
  return share > a.least_steps ? (int)share : a.least_steps;
}

// A tile of up to kWholeSteps steps stays whole: its pieces' way through memory and the second launch take
// longer than the steps they save (1 x 509 tokens of 32 heads, nine steps: 25 us whole, 36 in
// two).  Longer ones are cut down to kLeastSteps (1 x 5 over 8192: 24.2 us with six, 21.7 with four,
// 21.0 with three, of which more join).
constexpr int kWholeSteps = 12, kLeastSteps = 4;

// The tile's keys [lo, hi), the steps of one piece of them, and how many pieces there are.
struct Piece {
  int lo, hi, first, count, pieces;
};
__device__ inline Piece piece_of(const ChunkArgs& a, const Tile& t, int piece, int per, int keys) {
  Piece p;
  p.hi = hi_of(t.position((t.to - 1) / a.group));
  p.lo = lo_of(a, t.position(t.from / a.group));
  const int all = steps_in(p.lo, p.hi, keys);
  if (all <= kWholeSteps) per = kWholeSteps;
  p.pieces = (all + per - 1) / per;
  const int from = piece * per < all ? piece * per : all;
  p.first = p.lo / keys + from;
  p.count = from + per < all ? per : all - from;
  return p;
}

// How a step's keys and values lie in LDS: rows of D 16-bit values, in 16-byte pieces whose places
// within a row are turned by the row, so that the 16 rows of a pass over K (one piece each) lie on
// different banks, and the four rows of a transposing read of V (four pieces each) do.
template <class T, bool NARROW, int D>
struct Shape {
  static constexpr int kKeys = D >= 192 ? 32 : 64;     // per step
  static constexpr int EB = NARROW ? 1 : 2;
  static constexpr int kPieces = D / 8;                // of a row in LDS
  static constexpr int kRow = 2 * D;
  static constexpr int kBuffer = kKeys * kRow;         // of keys, or of values
  static constexpr int kBlocks = kKeys / 32, kSteps = kKeys / 16;
  // Where piece c of a row is.
  static __device__ inline int k_place(int row, int c) {
    if constexpr (D == 64) return c ^ ((row >> 1) & 7);
    if constexpr (D == 128 || D == 256) return c ^ (row & 15);
    return turned(c + (D == 96 ? (row >> 2) & 3 : (row >> 1) & 7));
  }
  static __device__ inline int v_place(int row, int c) {
    if constexpr (D == 64) return c ^ ((row & 2) << 1);
    if constexpr (D == 128 || D == 256) return c ^ ((row & 3) << 2);
    return D == 96 ? c : turned(c + 4 * ((row >> 1) & 1));
  }
  // Which piece is there.
  static __device__ inline int k_piece(int row, int at) {
    if constexpr (D == 64 || D == 128 || D == 256) return k_place(row, at);
    return turned(at + kPieces - (D == 96 ? (row >> 2) & 3 : (row >> 1) & 7));
  }
  static __device__ inline int v_piece(int row, int at) {
    if constexpr (D == 64 || D == 128 || D == 256) return v_place(row, at);
    return D == 96 ? at : turned(at + kPieces - 4 * ((row >> 1) & 1));
  }
  static __device__ inline int turned(int c) { return c >= kPieces ? c - kPieces : c; }
};

// 16 bytes a lane from memory to LDS, lane after lane from `to` (uniform) on.  By hand, since the
// compiler lets every later LDS access wait for such a load; wait_loads() does before a barrier.
__device__ inline void load_lds(const void* from, const void* to) {
  const uint32_t at = __builtin_amdgcn_readfirstlane(
      (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t*)to);
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(at), "v"(from)
               : "memory");
}
__device__ inline void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" : : : "memory"); }

// Brings a step's keys and values into LDS.  16-bit rows go there straight from memory, 8-bit ones
// through registers, where they are widened once for all four waves.
template <class T, bool NARROW, int D, int W>
struct Loader {
  using S = Shape<T, NARROW, D>;
  static constexpr int kThreads = 64 * W;
  const int32_t* table;  // of the sequence
  int page_shift, n_pages, lo, hi;  // the tile's keys

  // The table entry of key `key0 + lane` (past the end: of the last key).
  __device__ inline int look_up(int key0, int lane) const {
    const int at = key0 + (lane & (S::kKeys - 1));
    return table[(at < hi ? at : hi - 1) >> page_shift];
  }
  // That entry as the key's page, or -1 where it names no page or no row of the tile sees a key of
  // its group of four (which lie on one page).
  __device__ inline int page_of(int entry, int key0, int lane) const {
    const int key = key0 + (lane & (S::kKeys - 1));
    return (key | 3) >= lo && (key & ~3) < hi && (uint32_t)entry < (uint32_t)n_pages ? entry : -1;
  }
  // 16-byte pieces of a step's cached keys, and a thread's share of them
  static constexpr int kCached = D * S::EB / 16;
  static constexpr int kItems = S::kKeys * kCached;
  static constexpr int kLoads = (kItems + kThreads - 1) / kThreads;
  // Where 64 pieces of an access are whole rows, these lie in kGroups groups of four keys (or in part of
  // one), each on one page, whose addresses are found once for the wave; a lane adds its row's place in
  // the group.  Otherwise (dims 96 and 192) each lane works out its own.
  static constexpr bool kWhole = 64 % kCached == 0;
  static constexpr int kRowsAtOnce = kWhole ? 64 / kCached : 1;
  static constexpr int kGroups = kRowsAtOnce > 4 ? kRowsAtOnce / 4 : 1;
  struct Side {  // keys or values
    const uint8_t* base;  // of the key head
    int64_t page, row, lane;
    u32x4 x[NARROW ? kLoads : 1];
  };
  Side k, v;
  __device__ inline void start(int lane) {
    const int at = kWhole ? lane / kCached % 4 : 0;
    k.lane = S::EB * at * k.row;
    v.lane = S::EB * at * v.row;
  }
  // (an unseen key: any row, masked later)
  __device__ inline const uint8_t* row_at(const Side& y, int page, int key) const {
    const int64_t p = page < 0 ? 0 : page, in = key & ((1 << page_shift) - 1);
    return y.base + S::EB * (p * y.page + in * y.row);
  }
  template <bool VALUES>
  __device__ inline void load(uint8_t* buffer, int page, int key0, int wave, int lane) {
    Side& y = VALUES ? v : k;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int access = NARROW ? i * W + wave : wave * kLoads + i;
      const int e = access * 64 + lane, row = e / kCached, at = e % kCached;
      const uint8_t* from;
      if constexpr (kWhole) {
        if (kItems % kThreads && access * 64 >= kItems) continue;
        const int first = access * kRowsAtOnce;
        from = row_at(y, __builtin_amdgcn_readlane(page, first), key0 + first);
#pragma unroll
        for (int g = 1; g < kGroups; ++g) {
          const int next = first + 4 * g;
          const uint8_t* there = row_at(y, __builtin_amdgcn_readlane(page, next), key0 + next);
          from = lane >= 64 / kGroups * g ? there : from;
        }
        from += y.lane;
      } else {
        const int pg = __shfl(page, row);
        if (kItems % kThreads && e >= kItems) continue;
        from = row_at(y, pg, key0 + row);
      }
      if constexpr (NARROW)
        y.x[i] = *reinterpret_cast<const u32x4*>(from + 16 * at);
      else
        load_lds(from + 16 * (VALUES ? S::v_piece(row, at) : S::k_piece(row, at)),
                 buffer + 1024 * access);
    }
  }
  template <bool VALUES>
  __device__ inline void lay_out(uint8_t* buffer, int wave, int lane) const {
    if constexpr (NARROW) {
      const Side& y = VALUES ? v : k;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int e = (i * W + wave) * 64 + lane;
        const int row = e / kCached, at = e % kCached;
        if (kItems % kThreads && e >= kItems) continue;
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int c = 2 * at + z;
          *reinterpret_cast<u32x4*>(buffer + row * S::kRow +
                                    16 * (VALUES ? S::v_place(row, c) : S::k_place(row, c))) =
              widen4(y.x[i][2 * z], y.x[i][2 * z + 1]);
        }
      }
    }
  }
  static __device__ inline u32x4 widen4(uint32_t x, uint32_t y) {
    return u32x4{Mma<T>::template widen<false>(x), Mma<T>::template widen<true>(x),
                 Mma<T>::template widen<false>(y), Mma<T>::template widen<true>(y)};
  }
};

// Four keys of one dim per lane: rows `row`.. of 16 dims for every 16 lanes.
__device__ inline u32x2 read_turned(const uint8_t* p) {
  typedef short v4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) v4 lds_v4;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4*)p));
}

// The sign bits of those of two values that are not finite.
template <class T>
__device__ inline uint32_t odd_ones(uint32_t w) {
  return ((w & 0x7fff7fffu) + Mma<T>::kExpStep) & 0x80008000u;
}

// The exponentials are taken of s - m + kLift (base 2), and the running maximum m is raised only once a
// score is kSlack above it, so the largest is 2^(kLift + kSlack): all that fp16 holds.  In fp16 the lift
// keeps a long tail under one large key; both cancel in o / l.
template <class T>
struct Soft;
template <>
struct Soft<f16> {
  static constexpr float kLift = 14.0f, kSlack = 1.9f, kUnlift = 0x1p-14f;
};
template <>
struct Soft<bf16> {
  static constexpr float kLift = 0.0f, kSlack = 8.0f, kUnlift = 1.0f;
};

template <class T>
__device__ inline float log_sum(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + log2f(l * Soft<T>::kUnlift)) * kLn2;
}

// A wave's 32 query rows; a lane has row lane % 32.
template <class T, bool NARROW, int D>
struct Rows {
  using S = Shape<T, NARROW, D>;
  static constexpr int KC = D / 16, OB = D / 32;
  using Scores = f32x16[S::kBlocks];
  using Keys = u32x4[KC][S::kBlocks];
  using Values = u32x4[S::kSteps][OB];
  u32x4 q[KC];
  f32x16 o[OB];
  float m, l;
  // of values that are not finite: whether dim 32 b + i (in o's order, bit 16 b + i) met one that is
  // not -inf, and one that is not inf
  uint64_t up[(OB + 3) / 4], down[(OB + 3) / 4];
  int lo, hi;  // the keys that the row sees

  static __device__ inline u32x4 read_keys(const uint8_t* keys, int block, int c, int lane) {
    const int row = 32 * block + (lane & 31);
    return *reinterpret_cast<const u32x4*>(keys + row * S::kRow +
                                           16 * S::k_place(row, 2 * c + (lane >> 5)));
  }
  // Raw scores; the scale is part of soften's multiply-add.
  __device__ inline void score(const Keys& k, Scores& s) const {
#pragma unroll
    for (int c = 0; c < KC; ++c)
#pragma unroll
      for (int b = 0; b < S::kBlocks; ++b)
        s[b] = Mma<T>::mul32(k[c][b], q[c], c == 0 ? f32x16{} : s[b]);
  }
  // Bit 16 b + i: the lane's row sees key 32 b + 8 (i / 4) + 4 h + i % 4.
  __device__ inline uint32_t seen(int key0, int page, int lane) const {
    const int h = lane >> 5;
    uint32_t bits = 0;
#pragma unroll
    for (int y = 0; y < 4 * S::kBlocks; ++y) {
      const int at = 32 * (y / 4) + 8 * (y % 4) + 4 * h;
      const bool paged = __shfl(page, at) >= 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = key0 + at + i;
        bits |= (paged && key >= lo && key < hi ? 1u : 0u) << (4 * y + i);
      }
    }
    return bits;
  }
  __device__ inline void mask_out(Scores& s, int key0, int page, int lane) const {
    const uint32_t bits = seen(key0, page, lane);
#pragma unroll
    for (int b = 0; b < S::kBlocks; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[b][i] = (bits >> (16 * b + i)) & 1u ? s[b][i] : -INFINITY;
  }
  // The running maximum; to_log2 > 0.
  __device__ inline void raise(const Scores& s, float to_log2) {
    float top = s[0][0];
#pragma unroll
    for (int b = 0; b < S::kBlocks; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
    // the row's other lane
    const auto both =
        __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
    top = fmaxf(__uint_as_float(both[0]), __uint_as_float(both[1])) * to_log2;
    if (!__any(top > m + Soft<T>::kSlack)) return;
    const float higher = fmaxf(m, top);
    const float f = higher == m ? 1.0f : __builtin_amdgcn_exp2f(m - higher);
    m = higher;
    l *= f;
#pragma unroll
    for (int b = 0; b < OB; ++b) o[b] *= f;
  }
  // Scores to p, in the second product's operand order, and their sums.
  __device__ inline void soften(const Scores& s, float to_log2, u32x4 (&p)[S::kSteps]) {
    const float base = (m == -INFINITY ? 0.0f : m) - Soft<T>::kLift;
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int t = 0; t < S::kSteps; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        typename Mma<T>::v2 x;
        const int at = 8 * (t % 2) + 2 * i;
        const float p0 = __builtin_amdgcn_exp2f(fmaf(s[t / 2][at], to_log2, -base));
        const float p1 = __builtin_amdgcn_exp2f(fmaf(s[t / 2][at + 1], to_log2, -base));
        sum[0] += p0;
        sum[1] += p1;
        x.x = (T)p0;
        x.y = (T)p1;
        p[t][i] = __builtin_bit_cast(uint32_t, x);
      }
    l += sum[0] + sum[1];
  }
  static __device__ inline u32x4 read_values(const uint8_t* values, int block, int step, int lane) {
    const int i = lane & 15, g = lane >> 4;
    const int row = 16 * step + 4 * (g >> 1) + (i >> 2);
    const int piece = 4 * block + 2 * (g & 1) + ((i & 3) >> 1);
    const uint8_t* p = values + row * S::kRow + 16 * S::v_place(row, piece) + 8 * (i & 1);
    // (eight rows on, a row's pieces are turned alike)
    const u32x2 x = read_turned(p), y = read_turned(p + 8 * S::kRow);
    return u32x4{x.x, x.y, y.x, y.y};
  }
  __device__ inline void take_values(const Values& v, const u32x4 (&p)[S::kSteps]) {
#pragma unroll
    for (int t = 0; t < S::kSteps; ++t)
#pragma unroll
      for (int b = 0; b < OB; ++b) o[b] = Mma<T>::mul32(v[t][b], p[t], o[b]);
  }
  // Notes which dims of the row meet a value that is not finite, which decides them whatever else
  // they meet.
  __device__ inline void note_odd(const uint8_t* values, int key0, int page, int lane) {
    const int h = lane >> 5;
    const uint32_t bits = seen(key0, page, lane), others = __shfl_xor(bits, 32);
#pragma unroll 1
    for (int key = 0; key < S::kKeys; ++key) {
      // bit 16 b + 4 g + i of half h is key 32 b + 8 g + 4 h + i
      const int at = 16 * (key >> 5) + 4 * ((key >> 3) & 3) + (key & 3);
      const uint32_t mine = ((key >> 2) & 1) == h ? bits : others;
      const uint32_t keep = (mine >> at) & 1u ? ~0u : 0u;
#pragma unroll 1
      for (int g = 0; g < 4 * OB; ++g) {  // dims 8 g + 4 h ..
        const u32x2 w = *reinterpret_cast<const u32x2*>(values + key * S::kRow +
                                                        16 * S::v_place(key, g) + 8 * h);
        uint64_t u = 0, d = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const typename Mma<T>::v2 x = __builtin_bit_cast(typename Mma<T>::v2, w[i / 2] & keep);
          const float f = (float)(i % 2 ? x.y : x.x);
          if (!(fabsf(f) < INFINITY)) {
            u |= f < 0.0f ? 0u : 1u << i;
            d |= f > 0.0f ? 0u : 1u << i;
          }
        }
        const int to = 4 * (g & 15);
        up[0] |= g < 16 ? u << to : 0;
        down[0] |= g < 16 ? d << to : 0;
        if constexpr (OB > 4) {
          up[1] |= g < 16 ? 0 : u << to;
          down[1] |= g < 16 ? 0 : d << to;
        }
      }
    }
  }
  __device__ inline float value(int b, int i) const {
    const uint64_t bit = (uint64_t)1 << (16 * (b % 4) + i);
    const bool u = up[b / 4] & bit, d = down[b / 4] & bit;
    return u || d ? o[b][i] + (u ? d ? NAN : INFINITY : -INFINITY) : o[b][i];
  }
};

template <class T, bool NARROW, int D, int W>
__global__ __launch_bounds__(64 * W, D >= 192 ? 1 : 2) void chunk_kernel(ChunkArgs a) {
  using S = Shape<T, NARROW, D>;
  using R = Rows<T, NARROW, D>;
  constexpr int kThreads = 64 * W;
  extern __shared__ __attribute__((aligned(256))) uint8_t lds[];  // two steps' keys and values
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5, r = lane & 31;
  // Workgroups go to the 8 XCDs in turn: the tiles of a key head, which read the same rows, meet on
  // few of them.  Later tiles of a sequence see more keys and are begun first.
  const int kvh = blockIdx.x % (unsigned)a.n_kv, rest = blockIdx.x / (unsigned)a.n_kv;
  const int piece = rest % a.pieces;
  const Tile tile = find_tile(a, a.tiles - 1 - rest / a.pieces, lane);
  if (tile.from == tile.to) return;

  Loader<T, NARROW, D, W> in;
  const Piece steps = piece_of(a, tile, piece, piece_steps(a, S::kKeys, lane), S::kKeys);
  if (piece > 0 && piece >= steps.pieces) return;
  in.lo = steps.lo;
  in.hi = steps.hi;
  float to_log2 = a.scale * kLog2e, v_mul = 1.0f;
  if constexpr (NARROW) {
    if (a.k_scale) to_log2 *= a.k_scale[kvh];
    if (a.v_scale) v_mul = a.v_scale[kvh];
  }
  in.k.base = (const uint8_t*)a.k + (int64_t)S::EB * kvh * a.k_head;
  in.v.base = (const uint8_t*)a.v + (int64_t)S::EB * kvh * a.v_head;
  in.table = a.table + tile.seq * a.table_stride;
  in.k.page = a.k_page; in.k.row = a.k_row; in.v.page = a.v_page; in.v.row = a.v_row;
  in.page_shift = a.page_shift; in.n_pages = a.n_pages;
  in.start(lane);

  // The scale is kept above zero, as the largest score is found before it is applied: a sign goes to
  // the queries, and a scale of zero makes them zeros.
  const uint32_t flip = to_log2 < 0.0f ? 0x80008000u : 0u, keep = to_log2 == 0.0f ? 0u : ~0u;
  to_log2 = to_log2 == 0.0f ? 1.0f : fabsf(to_log2);
  const int first = tile.from + 32 * wave;  // the wave's rows; past the last row, that one again
  const bool works = first < tile.to;
  const int last = first + 32 < tile.to ? first + 31 : tile.to - 1;
  const int lo_min = works ? lo_of(a, tile.position(first / a.group)) : 0;
  const int hi_max = works ? hi_of(tile.position(last / a.group)) : 0;
  const int row = first + r < tile.to ? first + r : tile.to - 1;
  const int token = row / a.group, head = kvh * a.group + row % a.group;
  R w;
  const uint8_t* q = (const uint8_t*)a.q + 2 * ((tile.first + token) * a.qt + head * a.qh);
#pragma unroll
  for (int c = 0; c < R::KC; ++c)
    w.q[c] = (*reinterpret_cast<const u32x4*>(q + 32 * c + 16 * h) ^ flip) & keep;
#pragma unroll
  for (int b = 0; b < R::OB; ++b) w.o[b] = f32x16{};
#pragma unroll
  for (int b = 0; b < (R::OB + 3) / 4; ++b) w.up[b] = w.down[b] = 0u;
  w.m = -INFINITY;
  w.l = 0.0f;
  w.lo = lo_of(a, tile.position(token));
  w.hi = hi_of(tile.position(token));
  // 0 * inf is NaN, so where some row does not see some key, values that are not finite are taken out
  // of the step and noted for the rows that do see them.
  __shared__ int odd_step[2];
  const int all_lo = lo_of(a, tile.position((tile.to - 1) / a.group));
  const int all_hi = hi_of(tile.position(tile.from / a.group));
  if (threadIdx.x < 2) odd_step[threadIdx.x] = 0;

  if (steps.count > 0) {
    const auto keys = [&](int i) { return lds + 2 * (i & 1) * S::kBuffer; };
    const auto values = [&](int i) { return lds + (2 * (i & 1) + 1) * S::kBuffer; };
    int key0 = steps.first * S::kKeys;
    int page = in.page_of(in.look_up(key0, lane), key0, lane);
    in.template load<false>(keys(0), page, key0, wave, lane);
    in.template load<true>(values(0), page, key0, wave, lane);
    int entry = in.look_up(key0 + S::kKeys, lane);
    in.template lay_out<false>(keys(0), wave, lane);
    in.template lay_out<true>(values(0), wave, lane);
    for (int i = 0; i < steps.count; ++i) {
      if constexpr (!NARROW) wait_loads();
      mask::lds_barrier();  // this step is laid out, the last one has been read
      const int next = key0 + S::kKeys;
      int next_page = -1;
      if (i + 1 < steps.count) {
        next_page = in.page_of(entry, next, lane);
        in.template load<false>(keys(i + 1), next_page, next, wave, lane);
        in.template load<true>(values(i + 1), next_page, next, wave, lane);
        entry = in.look_up(next + S::kKeys, lane);
      }
      const bool edge = !__all(page >= 0) || key0 < all_lo || key0 + S::kKeys > all_hi;
      if (edge) {
        uint8_t* v = values(i);
        constexpr int kMine = S::kBuffer / 16;
        uint32_t odd = 0u;
        for (int e = threadIdx.x; e < kMine; e += kThreads) {
          u32x4* at = reinterpret_cast<u32x4*>(v + 16 * e);
          const u32x4 x = *at;
          const int row = e / S::kPieces, key = key0 + row;
          const bool paged = __shfl(page, row) >= 0;  // (whole waves)
          const bool seen = paged && key >= in.lo && key < in.hi;
          const uint32_t bad = odd_ones<T>(x.x) | odd_ones<T>(x.y) | odd_ones<T>(x.z) | odd_ones<T>(x.w);
          if (!seen && bad) *at = u32x4{0u, 0u, 0u, 0u};  // whatever was left in unused rows
          odd |= seen ? bad : 0u;
        }
        if (__any(odd) && lane == 0) odd_step[i & 1] = 1;
        mask::lds_barrier();
        if (__builtin_amdgcn_readfirstlane(odd_step[i & 1])) {
          if (works) w.note_odd(v, key0, page, lane);
          mask::lds_barrier();
          for (int e = threadIdx.x; e < kMine; e += kThreads) {
            u32x4* at = reinterpret_cast<u32x4*>(v + 16 * e);
            u32x4 x = *at;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const uint32_t bad = odd_ones<T>(x[y]);
              x[y] &= ~(bad | (bad - (bad >> 15)));
            }
            *at = x;
          }
          mask::lds_barrier();
          if (threadIdx.x == 0) odd_step[i & 1] = 0;
        }
      }
      if (works && key0 + S::kKeys > lo_min && key0 < hi_max) {
        typename R::Scores s;
        {
          typename R::Keys k;
#pragma unroll
          for (int c = 0; c < R::KC; ++c)
#pragma unroll
            for (int b = 0; b < S::kBlocks; ++b) k[c][b] = R::read_keys(keys(i), b, c, lane);
          w.score(k, s);
        }
        if (edge) w.mask_out(s, key0, page, lane);
        w.raise(s, to_log2);
        __builtin_amdgcn_sched_barrier(0);
        u32x4 p[S::kSteps];
        w.soften(s, to_log2, p);
        __builtin_amdgcn_sched_barrier(0);
        typename R::Values v;
#pragma unroll
        for (int t = 0; t < S::kSteps; ++t)
#pragma unroll
          for (int b = 0; b < R::OB; ++b) v[t][b] = R::read_values(values(i), b, t, lane);
        w.take_values(v, p);
      }
      if (i + 1 < steps.count) {
        in.template lay_out<false>(keys(i + 1), wave, lane);
        in.template lay_out<true>(values(i + 1), wave, lane);
      }
      key0 = next;
      page = next_page;
    }
  }

  if (!works) return;
  w.l += __shfl_xor(w.l, 32);
  if (first + r >= tile.to) return;
  const int64_t at = (int64_t)(tile.first + token) * a.n_heads + head;
  if (steps.pieces <= 1) {
    const bool none = w.l == 0.0f;  // no key, or all scores -inf: zeros
    const float f = v_mul / w.l;
    T* out = (T*)a.out + (tile.first + token) * a.ot + head * a.oh;
#pragma unroll
    for (int b = 0; b < R::OB; ++b)
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = none ? 0.0f : w.value(b, 4 * y + i) * f;
        store_n<4>(out + 32 * b + 8 * y + 4 * h, x);
      }
    if (a.lse && h == 0) a.lse[at] = log_sum<T>(w.m, w.l);
    return;
  }
  const int64_t part = (int64_t)piece * a.n_tokens * a.n_heads + at;
#pragma unroll
  for (int b = 0; b < R::OB; ++b)
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      f32x4 x;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = w.value(b, 4 * y + i);
      *reinterpret_cast<f32x4*>(a.part_o + part * D + 32 * b + 8 * y + 4 * h) = x;
    }
  if (h == 0) {
    a.part_ml[2 * part] = w.m;
    a.part_ml[2 * part + 1] = w.l;
  }
}

// Joins the pieces of a row, a wave each: lane c has the maximum and the sum of piece c (at most 64),
// four dims a lane, D / 4 lanes a piece.  Rows whose tile is one piece have their result already.
constexpr int kJoinWaves = 4;
template <class T, int D>
__global__ __launch_bounds__(64 * kJoinWaves) void chunk_join_kernel(ChunkArgs a) {
  constexpr int kLanes = D / 4, kAtOnce = 64 / kLanes, kLoads = 8;
  constexpr int kKeys = D >= 192 ? 32 : 64;
  const int lane = threadIdx.x & 63;
  const int64_t at =
      (int64_t)blockIdx.x * kJoinWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int token = (int)(at / a.n_heads), head = (int)(at % a.n_heads);
  if (token >= a.n_tokens) return;
  Tile tile{0, 0, 0, 0, 0, 0};
  for (int base = 0; base < a.n_seqs; base += 64) {
    const Seq q = seq_at(a, base + lane);
    const uint64_t has = __ballot(token >= q.first && token - q.first < q.n_new);
    if (!has) continue;
    const int who = __builtin_ctzll(has);
    tile.seq = base + who;
    tile.first = __builtin_amdgcn_readlane(q.first, who);
    tile.n_new = __builtin_amdgcn_readlane(q.n_new, who);
    tile.len = __builtin_amdgcn_readfirstlane(clamp_to(a.lens[tile.seq], a.max_len));
    const int row = (token - tile.first) * a.group + head % a.group, rows = tile.n_new * a.group;
    tile.from = row / a.rows * a.rows;
    tile.to = tile.from + a.rows < rows ? tile.from + a.rows : rows;
    break;
  }
  if (tile.from == tile.to) return;
  const int pieces = piece_of(a, tile, 0, piece_steps(a, kKeys, lane), kKeys).pieces;
  if (pieces <= 1) return;
  const int64_t step = (int64_t)a.n_tokens * a.n_heads;
  const int slot = lane / kLanes, d = 4 * (lane % kLanes);
  const float* from = a.part_o + at * D + d;
  f32x4 x[kLoads];
#pragma unroll
  for (int y = 0; y < kLoads; ++y) {
    const int c = y * kAtOnce + slot;
    x[y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (slot < kAtOnce && c < pieces) x[y] = *reinterpret_cast<const f32x4*>(from + c * step * D);
  }
  const bool has = lane < pieces;
  const float pm = has ? a.part_ml[2 * (at + lane * step)] : -INFINITY;
  const float pl = has ? a.part_ml[2 * (at + lane * step) + 1] : 0.0f;
  float m = pm;
#pragma unroll
  for (int z = 32; z > 0; z >>= 1) m = fmaxf(m, __shfl_xor(m, z));
  const float f = has ? __builtin_amdgcn_exp2f(pm - (m == -INFINITY ? 0.0f : m)) : 0.0f;
  float l = f * pl;
#pragma unroll
  for (int z = 32; z > 0; z >>= 1) l += __shfl_xor(l, z);
  f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int c0 = 0;;) {
#pragma unroll
    for (int y = 0; y < kLoads; ++y) {
      const int c = c0 + y * kAtOnce + slot;
      sum += __shfl(f, c & 63) * x[y];
    }
    c0 += kLoads * kAtOnce;
    if (c0 >= pieces) break;
#pragma unroll
    for (int y = 0; y < kLoads; ++y) {
      const int c = c0 + y * kAtOnce + slot;
      x[y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (slot < kAtOnce && c < pieces) x[y] = *reinterpret_cast<const f32x4*>(from + c * step * D);
    }
  }
  if constexpr (kAtOnce > 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x = sum[i];
#pragma unroll
      for (int y = 1; y < kAtOnce; ++y) x += __shfl(sum[i], (lane + y * kLanes) & 63);
      sum[i] = x;
    }
  }
  if (slot > 0) return;
  const float inv = (a.v_scale ? a.v_scale[head / a.group] : 1.0f) / l;
  float out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = l == 0.0f ? 0.0f : sum[i] * inv;
  store_n<4>((T*)a.out + token * a.ot + head * a.oh + d, out);
  if (a.lse && d == 0) a.lse[at] = log_sum<T>(m, l);
}

template <class T, bool NARROW, int D, int W>
void start(const ChunkArgs& a, unsigned blocks, hipStream_t s) {
  constexpr int kLds = 4 * Shape<T, NARROW, D>::kBuffer;
  hipLaunchKernelGGL((chunk_kernel<T, NARROW, D, W>), dim3(blocks), dim3(64 * W), kLds, s, a);
}

template <class T, bool NARROW, int D>
int launch(const ChunkArgs& a, unsigned blocks, hipStream_t s) {
  if constexpr (!NARROW && D < 192) {
    if (a.rows == rows_of(8))
      start<T, NARROW, D, 8>(a, blocks, s);
    else
      start<T, NARROW, D, 4>(a, blocks, s);
  } else {
    start<T, NARROW, D, 4>(a, blocks, s);
  }
  SPAX_HIP_CHECK(hipGetLastError());
  if (a.pieces > 1) {
    const int64_t rows = (int64_t)a.n_tokens * a.n_heads;
    hipLaunchKernelGGL((chunk_join_kernel<T, D>), dim3((unsigned)((rows + kJoinWaves - 1) / kJoinWaves)),
                       dim3(64 * kJoinWaves), 0, s, a);
    SPAX_HIP_CHECK(hipGetLastError());
  }
  return SPAX_OK;
}

template <class T, bool NARROW>
int launch_dim(const ChunkArgs& a, int dim, unsigned blocks, hipStream_t s) {
  switch (dim) {
    case 64: return launch<T, NARROW, 64>(a, blocks, s);
    case 96: return launch<T, NARROW, 96>(a, blocks, s);
    case 128: return launch<T, NARROW, 128>(a, blocks, s);
    case 192: return launch<T, NARROW, 192>(a, blocks, s);
    default: return launch<T, NARROW, 256>(a, blocks, s);
  }
}

}  // namespace

ChunkPlan chunk_plan(const spax_chunk_attention_args* a) {
  const spax_kv_cache& c = *a->cache;
  ChunkPlan p{};
  if (a->n_tokens == 0) return p;
  const int64_t group = a->n_heads / c.n_kv_heads;
  const auto tiles = [&](int rows) {
    // every sequence with tokens has at most one tile that is not full
    return a->n_tokens * group / rows + (c.n_seqs < a->n_tokens ? c.n_seqs : a->n_tokens);
  };
  // Eight waves that share a step's keys bring half as many in for a row as two workgroups of four, and
  // have a unit to themselves (1 x 8192 of 16 bits: 657 us, 691 with four; 24 mixed 88 and 106), but
  // widen 8-bit keys all at the same time (8 x 512 over 15872: 1755 and 1350), and want one
  // workgroup for each unit (1 x 509 of 32 heads: 31 and 25).
  const bool wide = c.type != SPAX_E4M3 && c.head_dim < 192 &&
                    tiles(rows_of(8)) * c.n_kv_heads >= 256;
  p.rows = rows_of(wide ? 8 : 4);
  p.tiles = tiles(p.rows);
  int64_t keys = a->max_len;
  if (a->window > 0 && (int64_t)a->window + a->n_tokens < keys)
    keys = (int64_t)a->window + a->n_tokens;
  const int64_t width = c.head_dim >= 192 ? 32 : 64;
  const int64_t steps = (keys + width - 1) / width + 1;  // a window starts anywhere
  const int64_t items = p.tiles * c.n_kv_heads;
  int64_t pieces = 2048 / items;
  if (pieces > steps / kLeastSteps) pieces = steps / kLeastSteps;
  if (steps <= kWholeSteps) pieces = 1;
  pieces = pieces < 1 ? 1 : pieces > 64 ? 64 : pieces;
  p.least_steps = (int32_t)((steps + pieces - 1) / pieces);
  p.pieces = (int32_t)((steps + p.least_steps - 1) / p.least_steps);
  p.blocks = items * p.pieces;
  if (p.pieces > 1)
    p.ws_bytes = aligned_size((size_t)p.pieces * a->n_tokens * a->n_heads *
                              ((size_t)c.head_dim + 2) * sizeof(float));
  return p;
}

int launch_chunk_attention(const spax_chunk_attention_args* p, void* ws, hipStream_t s) {
  if (p->n_tokens == 0) return SPAX_OK;
  const spax_kv_cache& c = *p->cache;
  const ChunkPlan plan = chunk_plan(p);
  ChunkArgs a{};
  a.q = p->q; a.k = c.k; a.v = c.v; a.out = p->out; a.lse = p->lse;
  a.starts = p->starts; a.lens = p->lens; a.table = c.page_table;
  a.k_scale = c.k_scale; a.v_scale = c.v_scale;
  a.qt = p->q_token_stride; a.qh = p->q_head_stride;
  a.ot = p->out_token_stride; a.oh = p->out_head_stride;
  a.k_page = c.k_page_stride; a.k_head = c.k_head_stride; a.k_row = c.k_row_stride;
  a.v_page = c.v_page_stride; a.v_head = c.v_head_stride; a.v_row = c.v_row_stride;
  a.table_stride = c.table_stride;
  a.n_tokens = p->n_tokens; a.n_heads = p->n_heads; a.n_kv = c.n_kv_heads;
  a.group = p->n_heads / c.n_kv_heads; a.n_seqs = c.n_seqs; a.n_pages = c.n_pages;
  a.page_shift = __builtin_ctz((unsigned)c.page_size);
  a.max_len = p->max_len; a.window = p->window; a.scale = p->scale;
  a.rows = plan.rows; a.tiles = (int32_t)plan.tiles; a.pieces = plan.pieces;
  a.least_steps = plan.least_steps;
  a.part_o = (float*)ws;
  a.part_ml = (float*)ws + (size_t)plan.pieces * p->n_tokens * p->n_heads * c.head_dim;
  const unsigned blocks = (unsigned)plan.blocks;
  if (c.type == SPAX_E4M3)
    return p->type == SPAX_F16 ? launch_dim<f16, true>(a, c.head_dim, blocks, s)
                               : launch_dim<bf16, true>(a, c.head_dim, blocks, s);
  return p->type == SPAX_F16 ? launch_dim<f16, false>(a, c.head_dim, blocks, s)
                             : launch_dim<bf16, false>(a, c.head_dim, blocks, s);
}

}  // namespace spax
