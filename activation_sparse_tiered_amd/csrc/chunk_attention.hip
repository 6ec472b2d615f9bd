// spax_chunk_attention: a chunk of new query tokens per sequence over a paged cache, causal.
//
// A sequence's query rows for one key head, tokens times the group's heads, are laid end to end and
// cut into tiles, so any group fills them.  Per row with keys k_j, values v_j, in one pass:
//   s_j = scale q.k_j,  m = running max of s,  p = exp(s - m),
//   l <- l exp(m_old - m) + sum p,   o <- o exp(m_old - m) + sum p v,   out = o / l.
// Pieces of a tile's keys (m, l, o) join by the same rule.
//
// A wave has 32 rows.  Four or eight of them take a tile of 128 or 256 rows and walk over its keys a step
// at a time, which pass through LDS once for all (chunk_kernel); or four share the 32 rows of a small
// tile, each with its own keys (chunk_few_kernel); chunk_plan says when.
//   * S^T = K Q^T by 32x32x16 matrix instructions, keys as rows, query rows as columns.
//   * S^T's layout (lane: one row, keys 8 b + 4 h + i) is that of the second product's P operand if
//     that product counts keys in the order {4 h + i, 8 + 4 h + i} of every 16, so probabilities
//     never cross lanes and a row's maximum and sum are in two lanes.
//   * O^T = V^T P^T: eight keys of one dim come from LDS by transposing reads of four rows.
//   * p enters the product as one 16-bit value, in fp16 lifted by 2^14 (Soft): splitting it in two, as
//     the attention of single tokens does, would add half of the matrix work again where that is the
//     bound, for an error that is about that of rounding the result.
//   * The maximum is raised only where a score is kSlack above it: most steps leave o as it is.
//   * Masked keys get p = 0, but 0 * inf is NaN: in steps that some row does not see whole, values
//     that are not finite are zeroed in LDS and noted for the rows that see them (note_odd).
//
// What bounds it.  Many rows and keys: matrix instructions are under way for 0.43 of the SIMDs'
// cycles (counters; 0.37 from e4m3), vector instructions, the exponentials above all, for 0.47, and
// the two overlap in part only, with two waves on a SIMD: 1 x 8192 of 32 heads on 8, fp16, 600 us,
// 917 TFLOP/s; 8 x 512 over 15872 from e4m3 1236 us, 875 TFLOP/s; a large library product reaches
// 1400.  Two tiles of rows per wave, which would share its reads of keys and values, spilled (908 us
// for 620 then); scores of the next step between the products of this one 722 us for 620.  Few rows:
// the chain starts, table, keys, two products, join, second launch, 18.4 us for 1 x 5 over 8192, of
// which the keys' 33.6 MB need 4.7.
#include "attn_core.h"
#include "layer_ops.h"
#include "mask_core.h"
#include "staging.h"

namespace spax {
namespace {

using namespace elem;
using namespace staging;
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
  int32_t max_len, window, rows, tiles, pieces;  // rows: of a tile
  int32_t key_shift, least_steps, whole_steps, shares, join_groups, join_waves;   // a step is 2^key_shift keys
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

// Steps that hold [lo, hi).
__device__ inline int steps_in(const ChunkArgs& a, int lo, int hi) {
  return hi > lo ? ((hi - 1) >> a.key_shift) + 1 - (lo >> a.key_shift) : 0;
}

// The largest of the lanes up to each, of numbers from 0 up.
__device__ inline int wave_max_scan(int x) {
  const auto take = [](int x, int y) { return x > y ? x : y; };
  x = take(x, __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false));  // row_shr:1
  x = take(x, __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false));  // row_shr:2
  x = take(x, __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false));  // row_shr:4
  x = take(x, __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false));  // row_shr:8
  x = take(x, __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false));  // row_bcast:15
  x = take(x, __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false));  // row_bcast:31
  return x;
}

// Sequence base + lane: its first row, new tokens, tiles and length.  Starts count as their running
// maximum, so no row has two sequences and the tiles stay within the plan's, whatever the starts;
// `from` is that of the sequences before base.
struct Seq {
  int first, n_new, tiles, len;
  // of the last lane
  __device__ inline int end() const { return __builtin_amdgcn_readlane(first + n_new, 63); }
};
__device__ inline Seq seqs_at(const ChunkArgs& a, int base, int from, int lane) {
  const int s = base + lane;
  Seq q{from, 0, 0, 0};
  int end = from;
  if (s < a.n_seqs) {
    q.len = clamp_to(a.lens[s], a.max_len);
    q.first = clamp_to(a.starts[s], a.n_tokens);
    end = clamp_to(a.starts[s + 1], a.n_tokens);
  }
  // (starts that ascend, as they should, need no scan: 1 x 5 over 8192 18.7 us, 19.3 with it)
  if (__builtin_expect(__any(s < a.n_seqs && (q.first < from || end < q.first)), 0)) {
    const int most = q.first > end ? q.first : end;
    end = wave_max_scan(most > from ? most : from);
    const int before = __builtin_amdgcn_update_dpp(from, end, 0x138, 0xF, 0xF, false);  // wave_shr:1
    q.first = before > q.first ? before : q.first;
  }
  q.n_new = s < a.n_seqs ? end - q.first : 0;
  q.tiles = (q.n_new * a.group + a.rows - 1) / a.rows;
  return q;
}

// Tile `index` of all sequences' tiles laid end to end; lane l of `seqs` has sequence l.  Past the first
// 64, every 64 are a step of a chain of loads.
__device__ inline Tile find_tile(const ChunkArgs& a, const Seq& seqs, int index, int lane) {
  int before = 0;
  Seq q = seqs;
  for (int base = 0; base < a.n_seqs; base += 64) {
    if (base) q = seqs_at(a, base, q.end(), lane);
    const int upto = before + mask::wave_scan(q.tiles);
    const int last = __builtin_amdgcn_readlane(upto, 63);
    if (index < last) {
      const int who = __builtin_ctzll(__ballot(upto > index));
      Tile t;
      t.seq = base + who;
      t.first = __builtin_amdgcn_readlane(q.first, who);
      t.n_new = __builtin_amdgcn_readlane(q.n_new, who);
      t.len = __builtin_amdgcn_readlane(q.len, who);
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

// How many steps of a tile's keys make a piece, about: an equal share of all tiles' steps for each of the
// plan's shares, but no fewer than it has room for.  Every wave of both launches finds the same
// number, in integers, from at most kCounted sequences; with more the plan's own stands.
constexpr int kCounted = 256;
__device__ inline int piece_steps(const ChunkArgs& a, const Seq& seqs, int lane) {
  if (a.pieces == 1 || a.n_seqs > kCounted) return a.least_steps;
  int mine = 0;
  Seq q = seqs;
  for (int base = 0; base < a.n_seqs; base += 64) {
    if (base) q = seqs_at(a, base, q.end(), lane);
    const int len = q.len, p = len - q.n_new;
    // of the first token and of the last
    const int some = steps_in(a, lo_of(a, p), hi_of(p));
    const int more = steps_in(a, lo_of(a, len - 1), hi_of(len - 1));
    const int64_t units = (int64_t)q.tiles * ((some + more + 1) / 2);
    constexpr int kMost = 1 << 22;  // kCounted of them stay below 2^31
    mine += units < kMost ? (int)units : kMost;
  }
#pragma unroll
  for (int z = 32; z > 0; z >>= 1) mine += __shfl_xor(mine, z);
  mine = __builtin_amdgcn_readfirstlane(mine);
  const int64_t share = ((int64_t)mine * a.n_kv + a.shares - 1) / a.shares;
  return share > a.least_steps ? (int)share : a.least_steps;
}

// The tile's keys [lo, hi), the steps of one piece of them, and how many pieces there are.
struct Piece {
  int lo, hi, first, count, pieces;
};
__device__ inline Piece piece_of(const ChunkArgs& a, const Tile& t, int piece, int per) {
  Piece p;
  p.hi = hi_of(t.position((t.to - 1) / a.group));
  p.lo = lo_of(a, t.position(t.from / a.group));
  const int all = steps_in(a, p.lo, p.hi);
  const int n = all <= a.whole_steps ? 1 : (all + per / 2) / per;
  per = n > 1 ? (all + n - 1) / n : all;
  p.pieces = n > 1 ? (all + per - 1) / per : 1;
  const int from = piece * per < all ? piece * per : all;
  p.first = (p.lo >> a.key_shift) + from;
  p.count = from + per < all ? per : all - from;
  return p;
}

// How a step's keys and values lie in LDS: rows of D 16-bit values, in 16-byte pieces whose places
// within a row are turned by the row, so that the 16 rows of a pass over K (one piece each) lie on
// different banks, and the four rows of a transposing read of V (four pieces each) do.
template <class T, bool NARROW, int D, int KEYS>
struct Shape {
  static constexpr int kKeys = KEYS;                   // per step
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

// Brings a step's keys and values into LDS.  16-bit rows go there straight from memory, 8-bit ones
// through registers, where they are widened once for all of its waves.
template <class T, bool NARROW, int D, int KEYS, int W>
struct Loader {
  using S = Shape<T, NARROW, D, KEYS>;
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
  __device__ inline void open(const ChunkArgs& a, const Tile& t, const Piece& p, int kvh, int lane) {
    table = a.table + t.seq * a.table_stride;
    page_shift = a.page_shift; n_pages = a.n_pages; lo = p.lo; hi = p.hi;
    k.base = (const uint8_t*)a.k + (int64_t)S::EB * kvh * a.k_head;
    v.base = (const uint8_t*)a.v + (int64_t)S::EB * kvh * a.v_head;
    k.page = a.k_page; k.row = a.k_row; v.page = a.v_page; v.row = a.v_row;
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

// The sign bits of those of two values that are not finite.
template <class T>
__device__ inline uint32_t odd_ones(uint32_t w) {
  return ((w & 0x7fff7fffu) + Mma<T>::kExpStep) & 0x80008000u;
}

// Takes them out of `pieces` of 16 bytes.
template <class T>
__device__ inline void clear_odd(uint8_t* v, int pieces, int thread, int threads) {
  for (int e = thread; e < pieces; e += threads) {
    u32x4* at = reinterpret_cast<u32x4*>(v + 16 * e);
    u32x4 x = *at;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const uint32_t bad = odd_ones<T>(x[y]);
      x[y] &= ~(bad | (bad - (bad >> 15)));
    }
    *at = x;
  }
}

// The exponentials are taken of s - m + kLift (base 2), and the running maximum m is raised only once a
// score is kSlack above it, so the largest is 2^(kLift + kSlack), with 2^-13 of rounding (soften):
// all that fp16 holds.  In fp16 the lift keeps a long tail under one large key; both cancel in o / l.
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
template <class T, bool NARROW, int D, int KEYS>
struct Rows {
  using S = Shape<T, NARROW, D, KEYS>;
  static constexpr int KC = D / 16, OB = D / 32;
  using Scores = f32x16[S::kBlocks];
  using Keys = u32x4[KC][S::kBlocks];
  using Values = u32x4[S::kSteps][OB];
  u32x4 q[KC];
  f32x16 o[OB];
  float m, l;  // the running maximum of the raw scores, and the lane's part of the sum
  // of values that are not finite: whether dim 32 b + i (in o's order, bit 16 b + i) met one that is
  // not -inf, and one that is not inf
  uint64_t up[(OB + 3) / 4], down[(OB + 3) / 4];
  int lo, hi;  // the keys that the row sees

  // The row of this token and head, but for o: cleared here, it would be kept in memory longer (234 to 256
  // registers and spills in chunk_kernel).  The scale is kept above zero, as the largest score is found before it is
  // applied: a sign goes to the queries, and a scale of zero makes them zeros.
  __device__ inline void begin(const ChunkArgs& a, const Tile& t, int token, int head, float to_log2,
                               int lane) {
    const uint32_t flip = to_log2 < 0.0f ? 0x80008000u : 0u, keep = to_log2 == 0.0f ? 0u : ~0u;
    const uint8_t* from = (const uint8_t*)a.q + 2 * ((t.first + token) * a.qt + head * a.qh);
#pragma unroll
    for (int c = 0; c < KC; ++c)
      q[c] = (*reinterpret_cast<const u32x4*>(from + 32 * c + 16 * (lane >> 5)) ^ flip) & keep;
#pragma unroll
    for (int b = 0; b < (OB + 3) / 4; ++b) up[b] = down[b] = 0u;
    m = -INFINITY;
    l = 0.0f;
    lo = lo_of(a, t.position(token));
    hi = hi_of(t.position(token));
  }
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
  // The running maximum, raised where it pays; to_log2 > 0.
  __device__ inline void raise(const Scores& s, float to_log2) {
    float top = s[0][0];
#pragma unroll
    for (int b = 0; b < S::kBlocks; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
    // the row's other lane
    const auto both =
        __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
    top = fmaxf(__uint_as_float(both[0]), __uint_as_float(both[1]));
    if (!__any((top - m) * to_log2 > Soft<T>::kSlack)) return;
    const float higher = fmaxf(m, top);
    const float f = higher == m ? 1.0f : __builtin_amdgcn_exp2f((m - higher) * to_log2);
    m = higher;
    l *= f;
#pragma unroll
    for (int b = 0; b < OB; ++b) o[b] *= f;
  }
  // Scores to p, in the second product's operand order, and their sums.  The exponent is one
  // multiply-add from a base that is rounded once, to 2^-13 below kPlain; past it, where that
  // rounding would lift p by more than kLift + kSlack, the maximum is taken off first.
  static constexpr float kPlain = 4096.0f;
  __device__ inline void soften(Scores& s, float to_log2, u32x4 (&p)[S::kSteps]) {
    const float top = m == -INFINITY ? 0.0f : m;
    float base = fmaf(top, to_log2, -Soft<T>::kLift);
    if (!__all(fabsf(base) < kPlain)) {
#pragma unroll
      for (int b = 0; b < S::kBlocks; ++b) s[b] -= top;
      base = -Soft<T>::kLift;
    }
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
  // they meet and however small its weight: in dims 8 g + 4 h .. of one key,
  __device__ inline void note(u32x2 w, int g) {
    uint64_t u = 0, d = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t word = w[i / 2];  // (a cast of the element itself takes the first)
      const typename Mma<T>::v2 x = __builtin_bit_cast(typename Mma<T>::v2, word);
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
  // in a step's values in LDS,
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
        note(w & keep, g);
      }
    }
  }
  // and in memory, in every step-th kKeys keys from key0 up to stop: steps that all rows see whole
  // leave such a value in the product, where a weight that rounds to 0 makes it NaN.  Only where a
  // sum came out not finite though the weights are, so most tiles never get here.  (8-bit values
  // are finite or NaN, which the product keeps.)
  template <class In>
  __device__ inline void look_again(const In& in, int key0, int step, int stop, int lane) {
    float z = 0.0f;
#pragma unroll
    for (int b = 0; b < OB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) z = fmaf(o[b][i], 0.0f, z);
    if (!__any(z != 0.0f && fabsf(l) < INFINITY)) return;
#pragma unroll 1
    for (; key0 < stop; key0 += step) {
      const int page = in.page_of(in.look_up(key0, lane), key0, lane);
#pragma unroll 1
      for (int i = 0; i < S::kKeys; ++i) {
        const int pg = __shfl(page, i), key = key0 + i;
        const uint32_t keep = pg >= 0 && key >= lo && key < hi ? ~0u : 0u;
        const uint8_t* row = in.row_at(in.v, pg, key) + 8 * (lane >> 5);
#pragma unroll 1
        for (int g = 0; g < 4 * OB; ++g)
          note(*reinterpret_cast<const u32x2*>(row + 16 * g) & keep, g);
      }
    }
  }
  __device__ inline float value(int b, int i) const {
    const uint64_t bit = (uint64_t)1 << (16 * (b % 4) + i);
    const bool u = up[b / 4] & bit, d = down[b / 4] & bit;
    return u || d ? u ? d ? NAN : INFINITY : -INFINITY : o[b][i];
  }
};

template <bool NARROW>
__device__ inline float to_log2_of(const ChunkArgs& a, int kvh) {
  const float f = a.scale * kLog2e;
  return NARROW && a.k_scale ? f * a.k_scale[kvh] : f;
}
// The queries have its sign, and are zeros where it is zero (Rows::begin).
__device__ inline float positive(float to_log2) { return to_log2 == 0.0f ? 1.0f : fabsf(to_log2); }
template <bool NARROW>
__device__ inline float v_mul_of(const ChunkArgs& a, int kvh) {
  return NARROW && a.v_scale ? a.v_scale[kvh] : 1.0f;
}

// A piece of 32 rows of a tile leaves its sums as a wave holds them, dims 8 g + 4 h .. of row r in lane
// 32 h + r of group g, so that they go to memory and come back 1024 bytes at once (by rows, 8 x 128
// over 1000 took 88 us for 73 then), and its maxima (of raw scores) and weights.
__device__ inline int64_t part_of(const ChunkArgs& a, int piece, int rows32, int kvh) {
  return ((int64_t)piece * a.tiles * (a.rows / 32) + rows32) * a.n_kv + kvh;
}
template <int D>
__device__ inline f32x4* part_sums(const ChunkArgs& a, int64_t part, int group, int lane) {
  return reinterpret_cast<f32x4*>(a.part_o) + (part * (D / 8) + group) * 64 + lane;
}
// Sums that are not finite decide a joined one, whatever their weights (0 * inf is NaN).
__device__ inline bool is_finite(f32x4 x) {
  return fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w))) < INFINITY &&
         x.x == x.x && x.y == x.y && x.z == x.z && x.w == x.w;
}
__device__ inline f32x4 odd_ones(f32x4 x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = fabsf(x[i]) < INFINITY ? 0.0f : x[i];
  return x;
}
__device__ inline f32x4 decided(f32x4 sum, f32x4 odd) {
#pragma unroll
  for (int i = 0; i < 4; ++i) sum[i] = odd[i] == 0.0f ? sum[i] : odd[i];
  return sum;
}
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ inline f32x2* part_weight(const ChunkArgs& a, int64_t part, int r) {
  return reinterpret_cast<f32x2*>(a.part_ml) + part * 32 + r;
}

// Keys of a step that a workgroup's waves share.
constexpr int shared_keys(int dim) { return dim >= 192 ? 32 : 64; }

template <class T, bool NARROW, int D, int W>
__global__ __launch_bounds__(64 * W, D >= 192 ? 1 : 2) void chunk_kernel(ChunkArgs a) {
  constexpr int kKeys = shared_keys(D);
  using S = Shape<T, NARROW, D, kKeys>;
  using R = Rows<T, NARROW, D, kKeys>;
  constexpr int kThreads = 64 * W;
  extern __shared__ __attribute__((aligned(256))) uint8_t lds[];  // two steps' keys and values
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5, r = lane & 31;
  // Workgroups go to the 8 XCDs in turn: the tiles of a key head, which read the same rows, meet on
  // few of them.  Later tiles of a sequence see more keys and are begun first, and the pieces that
  // most tiles do not need come last (with a tile's pieces side by side 8 x 128 over 1000 took 72
  // us for 50 then).
  const int kvh = blockIdx.x % (unsigned)a.n_kv, rest = blockIdx.x / (unsigned)a.n_kv;
  const int piece = rest / a.tiles;
  const Seq seqs = seqs_at(a, 0, 0, lane);
  const int index = a.tiles - 1 - rest % a.tiles;
  const Tile tile = find_tile(a, seqs, index, lane);
  if (tile.from == tile.to) return;
  const Piece steps = piece_of(a, tile, piece, piece_steps(a, seqs, lane));
  if (piece > 0 && piece >= steps.pieces) return;
  Loader<T, NARROW, D, kKeys, W> in;
  in.open(a, tile, steps, kvh, lane);
  float to_log2 = to_log2_of<NARROW>(a, kvh);
  const int first = tile.from + 32 * wave;  // the wave's rows; past the last row, that one again
  const bool works = first < tile.to;
  const int last = first + 32 < tile.to ? first + 31 : tile.to - 1;
  const int lo_min = works ? lo_of(a, tile.position(first / a.group)) : 0;
  const int hi_max = works ? hi_of(tile.position(last / a.group)) : 0;
  const int row = first + r < tile.to ? first + r : tile.to - 1;
  const int token = row / a.group, head = kvh * a.group + row % a.group;
  R w;
  w.begin(a, tile, token, head, to_log2, lane);
#pragma unroll
  for (int b = 0; b < R::OB; ++b) w.o[b] = f32x16{};
  to_log2 = positive(to_log2);
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
          clear_odd<T>(v, kMine, threadIdx.x, kThreads);
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
  if constexpr (!NARROW)
    w.look_again(in, steps.first * S::kKeys, S::kKeys, (steps.first + steps.count) * S::kKeys, lane);
  if (first + r >= tile.to) return;
  const int64_t at = (int64_t)(tile.first + token) * a.n_heads + head;
  if (steps.pieces <= 1) {
    const bool none = w.l == 0.0f;  // no key, or all scores -inf: zeros
    const float f = v_mul_of<NARROW>(a, kvh) / w.l;
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
    if (a.lse && h == 0) a.lse[at] = log_sum<T>(w.m * to_log2, w.l);
    return;
  }
  const int64_t part = part_of(a, piece, index * W + wave, kvh);
#pragma unroll
  for (int b = 0; b < R::OB; ++b)
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      f32x4 x;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = w.value(b, 4 * y + i);
      *part_sums<D>(a, part, 4 * b + y, lane) = x;
    }
  if (h == 0) *part_weight(a, part, r) = f32x2{w.m, w.l};
}

// All loads but the last `N` are there.
template <int N>
__device__ inline void wait_loads_but() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}
// The wave's accesses to LDS are done.
__device__ inline void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); }

// A tile of 32 rows: its four waves take 32 keys of each step of 128, bring them in by themselves, without
// a barrier, and join at the end.  The next keys are asked for as soon as this step's have been read,
// and so are values, so one buffer of each does and two workgroups fit a unit (1 x 509 of 32 heads,
// fp16: 15.9 us, 23.7 in tiles of 128 rows).
constexpr int kFewRows = 32, kFewShift = 7;
template <class T, bool NARROW, int D>
__global__ __launch_bounds__(256, 2) void chunk_few_kernel(ChunkArgs a) {
  constexpr int kKeys = 32, kWaves = 4, kStep = 1 << kFewShift;
  using S = Shape<T, NARROW, D, kKeys>;
  using R = Rows<T, NARROW, D, kKeys>;
  using In = Loader<T, NARROW, D, kKeys, 1>;
  extern __shared__ __attribute__((aligned(256))) uint8_t lds[];
  __shared__ float ml[kWaves][32][2];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5, r = lane & 31;
  const int kvh = blockIdx.x % (unsigned)a.n_kv, rest = blockIdx.x / (unsigned)a.n_kv;
  const int piece = rest / a.tiles;
  const Seq seqs = seqs_at(a, 0, 0, lane);
  const int index = a.tiles - 1 - rest % a.tiles;
  const Tile tile = find_tile(a, seqs, index, lane);
  if (tile.from == tile.to) return;
  const Piece steps = piece_of(a, tile, piece, piece_steps(a, seqs, lane));
  if (piece > 0 && piece >= steps.pieces) return;
  In in;
  in.open(a, tile, steps, kvh, lane);
  float to_log2 = to_log2_of<NARROW>(a, kvh);
  const int row = tile.from + r < tile.to ? tile.from + r : tile.to - 1;
  const int token = row / a.group, head = kvh * a.group + row % a.group;
  R w;
  w.begin(a, tile, token, head, to_log2, lane);
#pragma unroll
  for (int b = 0; b < R::OB; ++b) w.o[b] = f32x16{};
  to_log2 = positive(to_log2);
  const int all_lo = lo_of(a, tile.position((tile.to - 1) / a.group));
  const int all_hi = hi_of(tile.position(tile.from / a.group));

  uint8_t* const keys = lds + wave * 2 * S::kBuffer;
  uint8_t* const values = keys + S::kBuffer;
  int key0 = steps.first * kStep + kKeys * wave;
  const int end = (steps.first + steps.count) * kStep;
  const int stop = steps.hi < end ? steps.hi : end;
  if (key0 + kKeys <= steps.lo) key0 += kStep;
  const int begin = key0;
  if (key0 < stop) {
    int page = in.page_of(in.look_up(key0, lane), key0, lane);
    in.template load<false>(keys, page, key0, 0, lane);
    in.template load<true>(values, page, key0, 0, lane);
    int entry = in.look_up(key0 + kStep, lane);
    for (; key0 < stop;) {
      const int next = key0 + kStep;
      const bool more = next < stop;
      if constexpr (NARROW) {
        in.template lay_out<false>(keys, 0, lane);
        in.template lay_out<true>(values, 0, lane);
        wait_lds();
      } else {
        wait_loads_but<In::kLoads>();
      }
      typename R::Scores s;
      {
        typename R::Keys k;
#pragma unroll
        for (int c = 0; c < R::KC; ++c)
#pragma unroll
          for (int b = 0; b < S::kBlocks; ++b) k[c][b] = R::read_keys(keys, b, c, lane);
        wait_lds();  // the next keys may take their place
        w.score(k, s);
      }
      int next_page = -1;
      if (more) {
        next_page = in.page_of(entry, next, lane);
        in.template load<false>(keys, next_page, next, 0, lane);
        if constexpr (NARROW) in.template load<true>(values, next_page, next, 0, lane);
        entry = in.look_up(next + kStep, lane);
      }
      const bool edge = !__all(page >= 0) || key0 < all_lo || key0 + kKeys > all_hi;
      if (edge) w.mask_out(s, key0, page, lane);
      w.raise(s, to_log2);
      u32x4 p[S::kSteps];
      w.soften(s, to_log2, p);
      if constexpr (!NARROW) {
        if (more)
          wait_loads_but<In::kLoads>();
        else
          wait_loads();
      }
      if (edge) {
        uint32_t odd = 0u;
#pragma unroll 1
        for (int e = lane; e < S::kBuffer / 16; e += 64) {
          u32x4* at = reinterpret_cast<u32x4*>(values + 16 * e);
          const u32x4 x = *at;
          const int row = e / S::kPieces, key = key0 + row;
          const bool paged = __shfl(page, row) >= 0;
          const bool seen = paged && key >= in.lo && key < in.hi;
          const uint32_t bad =
              odd_ones<T>(x.x) | odd_ones<T>(x.y) | odd_ones<T>(x.z) | odd_ones<T>(x.w);
          if (!seen && bad) *at = u32x4{0u, 0u, 0u, 0u};  // whatever was left in unused rows
          odd |= seen ? bad : 0u;
        }
        wait_lds();
        if (__any(odd)) {
          w.note_odd(values, key0, page, lane);
          wait_lds();
          clear_odd<T>(values, S::kBuffer / 16, lane, 64);
          wait_lds();
        }
      }
      typename R::Values v;
#pragma unroll
      for (int t = 0; t < S::kSteps; ++t)
#pragma unroll
        for (int b = 0; b < R::OB; ++b) v[t][b] = R::read_values(values, b, t, lane);
      wait_lds();
      if constexpr (!NARROW) {
        if (more) in.template load<true>(values, next_page, next, 0, lane);
      }
      w.take_values(v, p);
      key0 = next;
      page = next_page;
    }
  }

  // Join the waves: dims c .. c + 3 of all rows side by side.
  w.l += __shfl_xor(w.l, 32);
  if constexpr (!NARROW) w.look_again(in, begin, kStep, stop, lane);
  float* mine = reinterpret_cast<float*>(keys);
#pragma unroll
  for (int b = 0; b < R::OB; ++b)
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      f32x4 x;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = w.value(b, 4 * y + i);
      *reinterpret_cast<f32x4*>(mine + 4 * (32 * (8 * b + 2 * y + h) + r)) = x;
    }
  if (h == 0) {
    ml[wave][r][0] = w.m;
    ml[wave][r][1] = w.l;
  }
  mask::lds_barrier();
  if (tile.from + r >= tile.to) return;
  float m = -INFINITY, l = 0.0f, f[kWaves];
#pragma unroll
  for (int y = 0; y < kWaves; ++y) m = fmaxf(m, ml[y][r][0]);
#pragma unroll
  for (int y = 0; y < kWaves; ++y) {
    f[y] = __builtin_amdgcn_exp2f((ml[y][r][0] - (m == -INFINITY ? 0.0f : m)) * to_log2);
    l += f[y] * ml[y][r][1];
  }
  const int64_t at = (int64_t)(tile.first + token) * a.n_heads + head;
  const int64_t part = part_of(a, piece, index, kvh);
  const bool whole = steps.pieces <= 1, none = l == 0.0f;
  const float inv = v_mul_of<NARROW>(a, kvh) / l;
  constexpr int kShare = D / 4 / kWaves;  // of the dims, four at a time
  static_assert(kShare % 2 == 0, "two halves of a wave");
  const auto x_of = [&](int z, int c) {  // wave z's sums
    return *reinterpret_cast<const f32x4*>(
        reinterpret_cast<const float*>(lds + z * 2 * S::kBuffer) + 4 * (32 * c + r));
  };
#pragma unroll
  for (int y = 0; y < kShare / 2; ++y) {
    const int c = wave * kShare + 2 * y + h;
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int z = 0; z < kWaves; ++z)
      sum += f[z] * x_of(z, c);
    if (!NARROW && __any(!is_finite(sum))) {
      f32x4 odd = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int z = 0; z < kWaves; ++z) odd += odd_ones(x_of(z, c));
      sum = decided(sum, odd);
    }
    if (whole) {
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = none ? 0.0f : sum[i] * inv;
      store_n<4>((T*)a.out + (tile.first + token) * a.ot + head * a.oh + 4 * c, x);
    } else {
      *part_sums<D>(a, part, c / 2, lane) = sum;
    }
  }
  if (wave == 0 && h == 0) {
    if (!whole)
      *part_weight(a, part, r) = f32x2{m, l};
    else if (a.lse)
      a.lse[at] = log_sum<T>(m * to_log2, l);
  }
}

// Joins the pieces of 32 rows of a tile: a wave takes join_groups groups of 8 dims, and where there are
// many pieces join_waves waves take every join_waves-th.  Tiles of one piece have their result already.
constexpr int kJoinWaves = 4;
template <class T, int D>
__global__ __launch_bounds__(64 * kJoinWaves) void chunk_join_kernel(ChunkArgs a) {
  constexpr int kLoads = 8;  // pieces in flight
  __shared__ float others[kJoinWaves][6][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5, r = lane & 31;
  const int split = a.join_waves;
  const int item = split == 1 ? blockIdx.x * kJoinWaves + wave : blockIdx.x;
  const int shares = D / 8 / a.join_groups, per = a.rows / 32;
  const int share = item % shares, kvh = item / shares % a.n_kv, rows32 = item / shares / a.n_kv;
  if (rows32 >= a.tiles * per) return;
  // (scales come with 8-bit caches alone)
  const float v_mul = a.v_scale ? a.v_scale[kvh] : 1.0f;
  const float to_log2 = positive(a.scale * kLog2e * (a.k_scale ? a.k_scale[kvh] : 1.0f));
  const Seq seqs = seqs_at(a, 0, 0, lane);
  const Tile tile = find_tile(a, seqs, rows32 / per, lane);
  const int first = tile.from + rows32 % per * 32;
  if (first >= tile.to) return;
  const int pieces = piece_of(a, tile, 0, piece_steps(a, seqs, lane)).pieces;
  if (pieces <= 1) return;
  float pm[kLoads], pl[kLoads];
  f32x4 x[kLoads];
  const auto load_weights = [&](int c0) {
#pragma unroll
    for (int y = 0; y < kLoads; ++y) {
      const int c = c0 + y * split;
      pm[y] = -INFINITY;
      pl[y] = 0.0f;
      if (c < pieces) {
        const f32x2 w = *part_weight(a, part_of(a, c, rows32, kvh), r);
        pm[y] = w.x;
        pl[y] = w.y;
      }
    }
  };
  const auto load_sums = [&](int c0, int group) {
#pragma unroll
    for (int y = 0; y < kLoads; ++y) {
      const int c = c0 + y * split;
      x[y] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (c < pieces) x[y] = *part_sums<D>(a, part_of(a, c, rows32, kvh), group, lane);
    }
  };
  const int from = split == 1 ? 0 : wave, more = kLoads * split;
  const int row = first + r < tile.to ? first + r : tile.to - 1;
  const int token = tile.first + row / a.group, head = kvh * a.group + row % a.group;
  load_weights(from);
  load_sums(from, share * a.join_groups);
  for (int group = share * a.join_groups, last = group + a.join_groups - 1;;) {
    float m = -INFINITY, l = 0.0f;
    f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
    const auto add = [&](float m1, float l1, f32x4 x1, float base) {
      const float f = __builtin_amdgcn_exp2f((m1 - base) * to_log2);
      l += f * l1;
      sum += f * x1;
    };
    const auto raise = [&](float higher) {
      const float base = higher == -INFINITY ? 0.0f : higher;
      const float f = __builtin_amdgcn_exp2f((m - base) * to_log2);
      l *= f;
      sum *= f;
      m = higher;
      return base;
    };
    for (int c0 = from;;) {
      float top = m;
#pragma unroll
      for (int y = 0; y < kLoads; ++y) top = fmaxf(top, pm[y]);
      const float base = raise(top);
#pragma unroll
      for (int y = 0; y < kLoads; ++y) add(pm[y], pl[y], x[y], base);
      c0 += more;
      if (c0 >= pieces) break;
      load_weights(c0);
      load_sums(c0, group);
    }
    // A sum that is not finite decides, whatever its weight: looked for again, where there is one.
    if (__any(first + r < tile.to && !is_finite(sum))) {
      f32x4 odd = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
      for (int c = from; c < pieces; c += split)
        odd += odd_ones(*part_sums<D>(a, part_of(a, c, rows32, kvh), group, lane));
      sum = decided(sum, odd);
    }
    if (split > 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) others[wave][i][lane] = sum[i];
      others[wave][4][lane] = m;
      others[wave][5][lane] = l;
      mask::lds_barrier();
      if (wave > 0) return;
      f32x4 odd = odd_ones(sum);
#pragma unroll
      for (int y = 1; y < kJoinWaves; ++y) {
        const float m1 = others[y][4][lane];
        const f32x4 x1 = {others[y][0][lane], others[y][1][lane], others[y][2][lane],
                          others[y][3][lane]};
        add(m1, others[y][5][lane], x1, raise(fmaxf(m, m1)));
        odd += odd_ones(x1);
      }
      sum = decided(sum, odd);
    }
    const float inv = v_mul / l;
    float out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = l == 0.0f ? 0.0f : sum[i] * inv;
    if (first + r < tile.to) {
      store_n<4>((T*)a.out + token * a.ot + head * a.oh + 8 * group + 4 * h, out);
      if (a.lse && group == 0 && h == 0) a.lse[(int64_t)token * a.n_heads + head] = log_sum<T>(m * to_log2, l);
    }
    if (group == last) break;
    ++group;
    if (pieces > more) load_weights(0);
    load_sums(0, group);
  }
}

template <class T, bool NARROW, int D, int W>
void start(const ChunkArgs& a, unsigned blocks, hipStream_t s) {
  constexpr int kLds = 4 * Shape<T, NARROW, D, shared_keys(D)>::kBuffer;
  hipLaunchKernelGGL((chunk_kernel<T, NARROW, D, W>), dim3(blocks), dim3(64 * W), kLds, s, a);
}

template <class T, bool NARROW, int D>
int launch(const ChunkArgs& a, unsigned blocks, hipStream_t s) {
  if (a.rows == rows_of(4)) {
    start<T, NARROW, D, 4>(a, blocks, s);
  } else if constexpr (D < 192) {
    if (a.rows == kFewRows) {
      constexpr int kLds = 8 * Shape<T, NARROW, D, 32>::kBuffer;
      hipLaunchKernelGGL((chunk_few_kernel<T, NARROW, D>), dim3(blocks), dim3(256), kLds, s, a);
    } else if constexpr (!NARROW) {
      start<T, NARROW, D, 8>(a, blocks, s);
    }
  }
  SPAX_HIP_CHECK(hipGetLastError());
  if (a.pieces > 1) {
    const int64_t items = (int64_t)a.tiles * (a.rows / 32) * a.n_kv * (D / 8 / a.join_groups);
    hipLaunchKernelGGL((chunk_join_kernel<T, D>), dim3((unsigned)(a.join_waves > 1 ? items : (items + kJoinWaves - 1) / kJoinWaves)),
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

// A tile of up to kWholeSteps steps stays whole: its pieces' way through memory and the second launch take
// longer than the steps they save (1 x 509 tokens of 32 heads in tiles of 128 rows, eight steps: 23.5
// us whole, 30.8 in two).  Longer ones are cut down to kLeastSteps (1 x 5 over 8192 in such tiles: 23.9
// us with six, 20.2 with four, 21.2 with three).  The same for tiles of few rows, whose steps are
// twice as long: 1 x 509 15.5 us whole, 23.8 in two; 1 x 5 over 8192 18.7 us down to two steps, 22.6
// to four, 20.0 to one.
constexpr int kWholeSteps = 12, kLeastSteps = 4, kFewWhole = 6, kFewLeast = 2;
// Pieces of all tiles, those that a tile does not need included: their workgroups end at once, but 4096
// took 60 us for 8 x 128 over 1000 where 2048 took 53.
constexpr int64_t kMostPieces = 2048;

ChunkPlan chunk_plan(const spax_chunk_attention_args* a) {
  const spax_kv_cache& c = *a->cache;
  ChunkPlan p{};
  if (a->n_tokens == 0) return p;
  const int64_t group = a->n_heads / c.n_kv_heads;
  const auto tiles = [&](int rows) {
    // every sequence with tokens has at most one tile that is not full
    return a->n_tokens * group / rows + (c.n_seqs < a->n_tokens ? c.n_seqs : a->n_tokens);
  };
  int64_t keys = a->max_len;
  if (a->window > 0 && (int64_t)a->window + a->n_tokens < keys)
    keys = (int64_t)a->window + a->n_tokens;
  // Tiles of 32 rows, whose four waves take a step's keys in turn, where larger ones would stay empty (64
  // users' next token over 8192: 368 us, 406 in tiles of 128; 64 mixed of up to 256 tokens over
  // 2048, 93 rows a sequence: 63 and 89; 24 mixed, 158 rows: 73 and 70; 8 x 32 over 4096, 128 rows:
  // 61 and 53) or would not fill the units for long (1 x 509 of 32 heads: 16 and 24; 1 x 300 over 600:
  // 29 and 41; 1 x 1024: 37 and 42; 4 x 512 over 1024: 109 and 77; 1 x 512 over 16000: 260 and 180).
  const int64_t rows = a->n_tokens * group;
  const bool few = c.head_dim < 192 && (rows <= (int64_t)96 * c.n_seqs ||
                                        (keys <= 2048 && rows / rows_of(4) * c.n_kv_heads <= 256));
  // Eight waves that share a step's keys bring half as many in for a row as two workgroups of four, and
  // have a unit to themselves (1 x 8192 of 16 bits: 630 us, 660 with four; 24 mixed 71 and 65), but
  // widen 8-bit keys all at the same time (8 x 512 over 15872: 1755 and 1350 then), and want one
  // workgroup for each unit (1 x 512 of 32 key heads, without tiles of 32: 30 and 24).
  const bool wide = !few && c.type != SPAX_E4M3 && c.head_dim < 192 &&
                    tiles(rows_of(8)) * c.n_kv_heads >= 256;
  p.rows = few ? kFewRows : rows_of(wide ? 8 : 4);
  // as many as run at once (eight waves, with 512 for 256: 4 x 512 over 1024 101 for 79 us; four waves,
  // with 256 for 512: 8 x 32 over 4096 60 for 57)
  p.shares = wide ? 256 : 512;
  p.tiles = tiles(p.rows);
  p.key_shift = few ? kFewShift : c.head_dim >= 192 ? 5 : 6;
  p.whole_steps = few ? kFewWhole : kWholeSteps;
  const int64_t least = few ? kFewLeast : kLeastSteps;
  const int64_t width = (int64_t)1 << p.key_shift;
  const int64_t steps = (keys + width - 1) / width + (a->window > 0);  // a window starts anywhere
  const int64_t items = p.tiles * c.n_kv_heads;
  int64_t pieces = kMostPieces / items;
  if (pieces > steps / least) pieces = steps / least;
  if (steps <= p.whole_steps) pieces = 1;
  pieces = pieces < 1 ? 1 : pieces > 64 ? 64 : pieces;
  p.least_steps = (int32_t)((steps + pieces - 1) / pieces);
  p.pieces = (int32_t)((steps + p.least_steps - 1) / p.least_steps);
  p.blocks = items * p.pieces;
  if (p.pieces > 1)
    p.ws_bytes = aligned_size((size_t)(items * p.pieces) * p.rows * (c.head_dim + 2) * sizeof(float));
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
  a.least_steps = plan.least_steps; a.whole_steps = plan.whole_steps; a.key_shift = plan.key_shift; a.shares = plan.shares;
  a.part_o = (float*)ws;
  a.part_ml = (float*)ws + (size_t)plan.blocks * plan.rows * c.head_dim;
  // (32 pieces of 1 x 5 over 8192: 18.6 us by four waves, 20.5 by one)
  a.join_waves = plan.pieces > 16 ? kJoinWaves : 1;
  a.join_groups = a.join_waves == 1 && plan.tiles * (plan.rows / 32) * c.n_kv_heads * (c.head_dim / 8) > 8192
                      ? 4
                      : 1;
  const unsigned blocks = (unsigned)plan.blocks;
  if (c.type == SPAX_E4M3)
    return p->type == SPAX_F16 ? launch_dim<f16, true>(a, c.head_dim, blocks, s)
                               : launch_dim<bf16, true>(a, c.head_dim, blocks, s);
  return p->type == SPAX_F16 ? launch_dim<f16, false>(a, c.head_dim, blocks, s)
                             : launch_dim<bf16, false>(a, c.head_dim, blocks, s);
}

}  // namespace spax
