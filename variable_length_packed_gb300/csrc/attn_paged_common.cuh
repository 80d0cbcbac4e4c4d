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
constexpr int kMaxCtas = 320;        // CTAs of a launch at most (two on each of up to 160 SMs)

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
  long long table_stride, k_page, k_token, k_head, v_page, v_token, v_head;   // elements
  int num_pages, page_size, max_pages;
  int tree_words;
  int B, T, Hq, Hkv, group, d;
  float scale_log2;
};

// One sequence of the batch, clamped to the buffers.
struct SeqWork {
  int q_start, q_len, kv_len, tiles, blocks;
  long long units;
};

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

template <int kThreads>
__device__ void find_share(const PagedArgs& p, int rows_per_tile, Share* out) {
  __shared__ long long warp_sum[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += seq_work(p, b, rows_per_tile).units;
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
        const long long u = seq_work(p, b, rows_per_tile).units;
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
  int blk0, steps;      // units that some row sees (steps may be 0)
  bool whole;           // all of the tile's units are in this piece
  bool first;           // the CTA's first piece
  long long tile_end;   // first unit after the tile's
};

struct PieceWalk {
  long long u, end, base, begin;
  int b;

  __device__ __forceinline__ explicit PieceWalk(const Share& share)
      : u(share.begin), end(share.end), base(share.seq_base), begin(share.begin), b(share.seq) {}

  template <int MT>
  __device__ __forceinline__ bool next(const PagedArgs& p, Piece& x) {
    while (u < end) {
      x.s = seq_work(p, b, MT);
      if (u - base >= x.s.units) {
        base += x.s.units;
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
      x.past = x.s.kv_len - x.s.q_len;
      x.key_end = p.tree ? x.s.kv_len : min(x.s.kv_len, max(0, x.past + (x.row0 + x.rows - 1) / p.group + 1));
      x.steps = min(nblk, max(0, (x.key_end + kUnit - 1) / kUnit - x.blk0));
      x.tile_end = base + (item + 1) * x.s.blocks;
      u += nblk;
      return true;
    }
    return false;
  }
};

// The first word of a token's tree mask: read when the piece begins, needed at its last keys.
__device__ __forceinline__ uint64_t tree_word(const PagedArgs& p, const Piece& x, int tok) {
  return p.tree ? (uint64_t)p.tree[(long long)(x.s.q_start + tok) * p.tree_words] : 0ull;
}

// Which of the 64 keys [first, first + 64) token `tok` of the piece's sequence sees; word0: its tree_word.
__device__ __forceinline__ uint64_t seen_keys(const PagedArgs& p, const Piece& x, int tok, int first, uint64_t word0) {
  const int last = (p.tree ? x.s.kv_len : min(x.past + tok + 1, x.s.kv_len)) - first;   // keys before the end
  uint64_t m = last >= 64 ? ~0ull : (last <= 0 ? 0ull : (1ull << last) - 1);
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

// Element offset of a piece's key or value in its cache: 0 for one that is not read.
__device__ __forceinline__ long long cache_offset(const PagedArgs& p, const Piece& x, const int32_t* table, int key,
                                                  bool values) {
  if (key >= x.key_end) return 0;
  const int at = key / p.page_size;
  int page = table[at];
  page = page < 0 ? 0 : (page >= p.num_pages ? p.num_pages - 1 : page);
  const int in = key - at * p.page_size;
  return values ? page * p.v_page + in * p.v_token + x.head * p.v_head
                : page * p.k_page + in * p.k_token + x.head * p.k_head;
}

}  // namespace
}  // namespace thd
