// attn_paged_common.cuh — what the kernels of attn_paged.cu share: arguments, the split of the
// batch's keys over the CTAs, the walk over a CTA's pieces, and places in the pages.
//
// Both kernels hold scores, maxima, sums and outputs in fp32 and round the weights once to the type of
// the values, because the matrix units multiply 16-bit operands of one type (thd_attn_fwd does the same).
// The output is divided by the sum of the rounded weights, so that their rounding does not shift its scale; the
// log-sum-exp takes the sum of the exact ones.  Error of the norm against 64 bits in bf16: 2.0e-3 to
// 2.3e-3, of which rounding the output alone is 1.7e-3; fp16 2.8e-4 and 2.1e-4.  Measured and left: weights in
// two 16-bit parts, with twice the products for the values, bring the error to the output's own rounding and
// cost 1 % on 500000 keys of heads of 128, 3 % on 262144 of 64, and 2 to 8 % in tiles of 128 rows.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"
#include "seq_rows.cuh"

namespace thd {
namespace {

constexpr int kUnit = 64;            // keys of a unit
constexpr int kNarrowRows = 16;      // rows of a narrow tile
constexpr int kMaxCtas = 320;        // CTAs of a launch at most (two on each of up to 160 SMs)

template <typename DT>
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// A tile that goes on from one CTA to the next: its rows, and the CTAs that share it.
struct alignas(16) Split {
  int n;        // CTAs (0: no such tile)
  int first;    // the first of them
  int second;   // whether the first one's partial is its second
  int q_start, row0, rows, head;
  int unused;
};

struct PagedArgs {
  const void* q;
  const void* kc;
  const void* vc;
  const int32_t* table;
  const int32_t* kv_lens;
  const int32_t* cu;
  const int32_t* padded;
  const long long* tree;
  void* out;
  float* lse;
  float* part_o;       // [ctas * 2][DP / 4][rows][4]
  float* part_m;       // [ctas * 2][3][rows]: maximum, sum of the rounded weights, sum of the weights
  uint32_t* call_status;
  uint32_t* status;    // [ctas]: THD_STATUS_* bits of each CTA
  uint64_t wait_limit_ns;
  uint32_t wait_check_mask, inject_wait;
  Split* splits;       // [ctas]
  float* key_weights;  // weights that the keys got, or null
  float* scores;       // narrow tiles with key_weights: the scores (score_places), room for score_room of them
  long long score_room;
  long long w_page, w_token, w_head;                                          // elements
  long long table_stride, k_page, k_token, k_head, v_page, v_token, v_head;   // elements
  int num_pages, page_size, max_pages;
  int page_shift;      // page_size = 2^page_shift, or -1
  int same_places;     // values lie in their cache as keys in theirs
  int tree_words;
  int win_left, sinks; // kWin: keys before its own slot that a token sees, and first keys that it sees besides
  int B, T, Hq, Hkv, group, d;
  float scale_log2;
};

// One sequence of the batch, clamped to the buffers.
struct SeqWork {
  int q_start, q_len, kv_len, tiles;
  int blocks;           // units of a tile: all of the sequence's, or (kWin) as many as a tile's rows see at most
  long long units;
};

// Units that hold first keys which every token sees (kWin).
__device__ __forceinline__ int sink_units(const PagedArgs& p, int kv_len) {
  return (min(p.sinks, kv_len) + kUnit - 1) / kUnit;
}

// First key of the window of new token `tok`.
__device__ __forceinline__ int window_first(const PagedArgs& p, int past, int tok) {
  return (int)max(0ll, (long long)past + tok - p.win_left);
}

template <bool kWin>
__device__ __forceinline__ SeqWork seq_work(const PagedArgs& p, int b, int rows_per_tile) {
  SeqWork s;
  const int c0 = p.cu[b], c1 = p.cu[b + 1];
  long long qs = p.padded ? p.padded[b] : c0, ql = (long long)c1 - c0;
  qs = qs < 0 ? 0 : (qs > p.T ? p.T : qs);
  ql = ql < 0 ? 0 : (ql > p.T - qs ? p.T - qs : ql);
  const long long room = (long long)p.max_pages * p.page_size;
  long long kv = p.kv_lens[b];
  kv = kv < 0 ? 0 : (kv > room ? room : kv);
  s.q_start = (int)qs;
  s.q_len = (int)ql;
  s.kv_len = (int)kv;
  const long long rows = ql * p.group;
  s.tiles = (int)((rows + rows_per_tile - 1) / rows_per_tile);
  s.blocks = (s.kv_len + kUnit - 1) / kUnit;
  if constexpr (kWin) {
    // a tile's tokens lie (rows - 1) / group apart at most, so its windows cover `span` keys one after another
    const long long span = (long long)p.win_left + (rows_per_tile - 1 + p.group - 1) / p.group + 1;
    s.blocks = (int)min((long long)s.blocks, sink_units(p, s.kv_len) + (span + kUnit - 2) / kUnit + 1);
  }
  s.units = (long long)s.tiles * s.blocks * p.Hkv;
  return s;
}

// The CTA's share of the batch's units, and the sequence its first unit lies in.  Every CTA
// adds up the whole batch: each thread a run of sequences, then a scan over the threads.
struct Share {
  long long begin, end, seq_base;   // units; seq_base: first unit of sequence seq
  long long total;
  int ctas;                         // CTAs that have units
  int seq;
};

__device__ __forceinline__ long long share_begin(long long total, int ctas, int c) { return total * c / ctas; }

// units(b): those of sequence b.
template <int kThreads, typename Units>
__device__ void find_share(const PagedArgs& p, Units units, Share* out) {
  __shared__ long long warp_sum[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += units(b);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  const long long excl = before + incl - mine;
  const int ctas = total < gridDim.x ? (int)total : (int)gridDim.x;
  if (tid == 0) {
    out->total = total;
    out->ctas = ctas;
    out->begin = out->end = 0;
    out->seq = 0;
    out->seq_base = 0;
  }
  __syncthreads();
  if ((int)blockIdx.x < ctas) {
    const long long begin = share_begin(total, ctas, blockIdx.x);
    if (begin >= excl && begin < excl + mine) {   // in this thread's run of sequences
      long long base = excl;
      int b = b0;
      for (; b < b1; ++b) {
        const long long u = units(b);
        if (begin < base + u) break;
        base += u;
      }
      out->seq = b;
      out->seq_base = base;
      out->begin = begin;
      out->end = share_begin(total, ctas, blockIdx.x + 1);
    }
  }
  __syncthreads();
}

// a / b for a >= 0, b > 0: in 32 bits where both fit, several times faster than in 64.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// One piece of a CTA's share: keys of units [blk0, blk0 + steps) of one row tile of one key/value head.
struct Piece {
  SeqWork s;
  int seq, head, tile;
  int row0, rows;       // the tile's rows of the sequence
  int past;             // keys before the new tokens (negative: fewer keys than tokens)
  int key_end;          // keys from here on no row of the tile sees
  int full_end;         // keys before here every row sees, but for the window
  int blk0, steps;      // units that some row sees (steps may be 0)
  // kWin: unit i is unit_of(i); the first row's window begins at win_lo and the last one's at win_hi; every row
  // sees the keys before `few` that it could see without a window
  int lead, skip, win_lo, win_hi, few;
  bool whole;           // all of the tile's units are in this piece
  bool first;           // the CTA's first piece
  long long tile_end;   // first unit after the tile's
};

// What of its sequence a tile (its s, row0 and rows set) sees: past, key_end and the window's fields.  Returns how many
// of the tile's units hold a key that some row sees.
template <bool kWin>
__device__ __forceinline__ int piece_bounds(const PagedArgs& p, Piece& x) {
  x.past = x.s.kv_len - x.s.q_len;
  x.key_end = p.tree ? x.s.kv_len : min(x.s.kv_len, max(0, x.past + (x.row0 + x.rows - 1) / p.group + 1));
  x.full_end = min(x.s.kv_len, p.tree ? x.past : x.past + x.row0 / p.group + 1);
  int last = (x.key_end + kUnit - 1) / kUnit;
  if constexpr (kWin) {
    const int tok0 = x.row0 / p.group, tok1 = (x.row0 + x.rows - 1) / p.group;
    x.win_lo = window_first(p, x.past, tok0);
    x.win_hi = window_first(p, x.past, tok1);
    x.few = min(p.sinks, x.key_end);
    // the units of the first keys, then from the window's first one on (one run where the two touch)
    const int first = sink_units(p, x.s.kv_len), from = x.win_lo / kUnit;
    x.lead = from > first ? first : 0;
    x.skip = from > first ? from - first : 0;
    last -= x.skip;   // a gap has the window's keys behind it
  }
  return last;
}

// Scores kept for the keys' weights, where they fit the call's room and every sequence is one narrow tile: of
// sequence b the units of its tile for each key/value head, 64 scores of each of its rows a unit, sequences one
// behind another.
__device__ __forceinline__ long long seq_scores(const PagedArgs& p, const SeqWork& s) {
  return (long long)p.Hkv * s.blocks * kUnit * s.q_len * p.group;
}
struct ScorePlaces {
  bool fit;         // the scores are kept
  long long base;   // first score of sequence `seq`
};
template <int kThreads, bool kWin>
__device__ ScorePlaces score_places(const PagedArgs& p, int seq) {
  __shared__ long long sums[2][kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long before = 0, all = 0;
  bool one = p.scores != nullptr;
  for (int b = threadIdx.x; b < p.B; b += kThreads) {
    const SeqWork s = seq_work<kWin>(p, b, kNarrowRows);
    const long long n = seq_scores(p, s);
    all += n;
    if (b < seq) before += n;
    one = one && s.tiles <= 1;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    all += __shfl_xor_sync(0xffffffffu, all, o);
  }
  if (lane == 0) {
    sums[0][warp] = before;
    sums[1][warp] = all;
  }
  one = __syncthreads_and(one ? 1 : 0) != 0;
  before = all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    before += sums[0][w];
    all += sums[1][w];
  }
  return {one && all <= p.score_room, before};
}

struct PieceWalk {
  long long u, end, base, begin;
  long long scores;   // first kept score of sequence b (kScores)
  int b;

  __device__ __forceinline__ explicit PieceWalk(const Share& share)
      : u(share.begin), end(share.end), base(share.seq_base), begin(share.begin), scores(0), b(share.seq) {}

  template <int MT, bool kWin, bool kScores = false>
  __device__ __forceinline__ bool next(const PagedArgs& p, Piece& x) {
    while (u < end) {
      x.s = seq_work<kWin>(p, b, MT);
      if (u - base >= x.s.units) {
        base += x.s.units;
        if (kScores) scores += seq_scores(p, x.s);
        ++b;
        continue;
      }
      const long long item = quotient(u - base, x.s.blocks);
      x.seq = b;
      x.blk0 = (int)(u - base - item * x.s.blocks);
      const int nblk = (int)min((long long)(x.s.blocks - x.blk0), end - u);
      x.head = (int)quotient(item, x.s.tiles);
      x.tile = (int)(item - (long long)x.head * x.s.tiles);
      x.whole = nblk == x.s.blocks;
      x.first = u == begin;
      x.row0 = x.tile * MT;
      x.rows = (int)min((long long)MT, (long long)x.s.q_len * p.group - x.row0);
      const int last = piece_bounds<kWin>(p, x);
      x.steps = min(nblk, max(0, last - x.blk0));
      x.tile_end = base + (item + 1) * x.s.blocks;
      u += nblk;
      return true;
    }
    return false;
  }
};

// Which unit of the sequence a tile's unit i is.
template <bool kWin>
__device__ __forceinline__ int unit_of(const Piece& x, int i) {
  return !kWin || i < x.lead ? i : i + x.skip;
}

// No row of the tile sees the key: it is not read.
template <bool kWin>
__device__ __forceinline__ bool key_hidden(const Piece& x, int key) {
  return key >= x.key_end || (kWin && key < x.win_lo && key >= x.few);
}

// Some key of the unit that begins with key `first` may be hidden from some row.
template <bool kWin>
__device__ __forceinline__ bool unit_cut(const PagedArgs& p, const Piece& x, int first) {
  return first + kUnit > x.full_end ||
         (kWin && first < x.win_hi && first + kUnit > x.few);
}

// The first word of a token's tree mask: read when the piece begins, needed at its last keys.
__device__ __forceinline__ uint64_t tree_word(const PagedArgs& p, const Piece& x, int tok) {
  return p.tree ? (uint64_t)p.tree[(long long)(x.s.q_start + tok) * p.tree_words] : 0ull;
}

// The lowest n of 64 bits set.
__device__ __forceinline__ uint64_t low_bits64(int n) { return n >= 64 ? ~0ull : (n <= 0 ? 0ull : (1ull << n) - 1); }

// Which of the 64 keys [first, first + 64) token `tok` of the piece's sequence sees; word0: its tree_word.
template <bool kWin>
__device__ __forceinline__ uint64_t seen_keys(const PagedArgs& p, const Piece& x, int tok, int first, uint64_t word0) {
  const int last = (p.tree ? x.s.kv_len : min(x.past + tok + 1, x.s.kv_len)) - first;   // keys before the end
  uint64_t m = low_bits64(last);
  if constexpr (kWin) m &= ~low_bits64(window_first(p, x.past, tok) - first) | low_bits64(p.sinks - first);
  if (p.tree) {
    const int j0 = first - x.past;   // index of the first key among the new tokens
    if (j0 > -64) {
      uint64_t t;
      if (j0 <= 0) {
        t = word0 << -j0;
        if (j0 < 0) t |= (1ull << -j0) - 1;   // cached keys
      } else {
        const long long* w = p.tree + (long long)(x.s.q_start + tok) * p.tree_words;
        const int at = j0 >> 6, sh = j0 & 63;
        t = at == 0 ? word0 >> sh : (at < p.tree_words ? (uint64_t)w[at] >> sh : 0ull);
        if (sh && at + 1 < p.tree_words) t |= (uint64_t)w[at + 1] << (64 - sh);
      }
      m &= t;
    }
  }
  return m;
}

// The CTA whose share unit u lies in.
__device__ __forceinline__ int cta_of(const Share& s, long long u) {
  return (int)quotient((u + 1) * s.ctas - 1, s.total);
}

// A tile that goes on in the next CTA: noted for the join.
__device__ __forceinline__ void note_split(const PagedArgs& p, const Piece& x, const Share& share) {
  if (x.tile_end <= share.end) return;
  const long long tile_begin = x.tile_end - x.s.blocks;
  Split sp;
  sp.first = cta_of(share, tile_begin);
  sp.n = cta_of(share, x.tile_end - 1) - sp.first + 1;
  sp.second = share_begin(share.total, share.ctas, sp.first) == tile_begin ? 0 : 1;
  sp.q_start = x.s.q_start;
  sp.row0 = x.row0;
  sp.rows = x.rows;
  sp.head = x.head;
  sp.unused = 0;
  p.splits[blockIdx.x] = sp;
}
// Place of the piece's partial result.
__device__ __forceinline__ int part_of_piece(const Piece& x) { return blockIdx.x * 2 + (x.first ? 0 : 1); }

// Element offset of a piece's key or value in its cache: -1 for one that is not read.
template <bool kWin>
__device__ __forceinline__ long long cache_offset(const PagedArgs& p, const Piece& x, const int32_t* table, int key,
                                                  bool values) {
  if (key_hidden<kWin>(x, key)) return -1;
  const int at = p.page_shift >= 0 ? key >> p.page_shift : key / p.page_size;
  int page = table[at];
  page = page < 0 ? 0 : (page >= p.num_pages ? p.num_pages - 1 : page);
  const int in = key - at * p.page_size;
  return values ? page * p.v_page + in * p.v_token + x.head * p.v_head
                : page * p.k_page + in * p.k_token + x.head * p.k_head;
}

}  // namespace
}  // namespace thd
