// attn_paged.cu — attention of packed new tokens over a paged key/value cache
// (thd_attn_paged, include/thd_attn.h): decoding steps, chunks of new tokens, and trees of
// drafted tokens.
//
// For the new token i of a sequence with n new tokens and L cached keys (the new ones among
// them, last): scores s_j = scale q.k_j over the keys j it sees, out = sum_j softmax(s)_j v_j,
// lse = log sum_j exp(s_j).  It sees key j < L iff j <= L - n + i, or, with a tree mask, iff
// j < L - n or bit j - (L - n) of its mask is set.
//
// What bounds it is reading the keys and values once (4 d bytes per key and head against
// 4 d operations per query row), so the work is split along the keys over every SM:
//  * the query heads that share a key/value head are the rows of one tile (row = token * group
//    + head of the group), so a key is read once for all of them;
//  * a unit is kUnit keys of one (sequence, key/value head, row tile); the units of the batch
//    are laid end to end and every CTA takes an equal number of them, whatever the lengths.  Units that
//    the causal mask hides from a whole tile count too, although they are passed over: a share that has many
//    of them ends early (of one fresh prompt of 8192 the busiest CTA works on 1.97 times the mean, of 2048
//    new tokens after 30000 on 1.03; decoding steps and trees have none);
//  * a CTA whose share ends inside a tile writes an unnormalised partial (at most two per CTA),
//    and a second kernel, launched to overlap the first one's end, joins them.
// Tiles of more than 16 rows are attn_paged_wide.cuh's.  Here, with 16 rows (decoding: the heads of
// one group), the products are 128 of the warp-wide 16 x 8 x 16 ones per 32 KB, about a fifth of their rate when
// the keys come at memory speed, so each warp runs alone: it streams its own 16 keys of each unit
// through its own ring of shared memory with 16-byte asynchronous copies, keeps a running maximum, sums
// and output tile in registers, and meets the other warps only when the tile is done.
// Measured, with the join: 500000 keys of 64 sequences, 32 + 8 heads of 128, one token each, 310 us, 6.6 TB/s
// of the 6.8 that a copy reaches; 262144 keys of one sequence, 16 heads of 64, 172 us, 6.2 TB/s.  Four times as
// many CTAs with shorter shares (an SM that is slower takes fewer) gained nothing: 319 and 186 us.  Heads of 96, 80
// and 32 are padded to 128 and 64 in shared memory and in the products, though not read: 300000 keys of 64
// sequences, 16 + 8 heads, 0.64, 0.56 and 0.35 of the copy's rate.
// Under a window a tile has as many units as its rows see at most: the first keys' and the window's (seq_work), so
// that shares stay equal.  64 sequences, windows of 2048 keys: 98 us, 5.5 TB/s of the keys and values they see (the
// start and the tail are 15 us of it).
#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/thd_attn.h"
#include "attn_paged_common.cuh"
#include "attn_paged_weights.cuh"
#include "attn_paged_weights_wide.cuh"
#include "attn_paged_wide.cuh"

namespace thd {

// the library's settings of waits inside kernels (thd_attn.cu)
void wait_settings(uint64_t* limit_ns, uint32_t* check_mask, uint32_t* inject);

namespace {

constexpr int kWarps = 4;            // warps of a CTA, 16 keys of the unit each
constexpr int kWarpKeys = kUnit / kWarps;
constexpr int kStages = 3;           // units in flight per warp
// fp16 weights are held times 2^15 (the largest is 1, and fp16 ends below 2^16): without it one below 2^-14
// of the maximum rounds by 2^-25 of it, which 20000 keys at 2^-23.5 add up to a third of their sum.
constexpr float kNarrowLift = 15.f;
constexpr int kJoinThreads = 256;
constexpr int kJoinAhead = 4;        // partials read at once

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Shared memory of a CTA: each warp's ring of key and value tiles (16 rows of DP values,
// 16-byte chunks XORed with the row so that eight rows of one column of chunks lie in
// different banks); at a tile's end the warps' sums and outputs take its place.
template <int DP>
struct PagedSmem {
  static constexpr int kTileBytes = kWarpKeys * DP * 2;
  static constexpr int kRing = kWarps * kStages * 2 * kTileBytes;
  static constexpr int kJoin = kWarps * kNarrowRows * (DP + 3) * 4;
  static constexpr int kBytes = kRing > kJoin ? kRing : kJoin;
};

// kScores: the scores are kept for the keys' weights, in place of reading the keys once more.
template <typename DT, int DP, bool kWin, bool kScores>
__global__ void __launch_bounds__(kWarps * 32, 2) attn_paged_kernel(const PagedArgs p) {
  constexpr int MT = kNarrowRows;
  constexpr int kKSteps = DP / 16;      // of the score product
  constexpr int kNT = DP / 8;           // 8-column output fragments
  constexpr int kChunks = DP / 8;       // 16-byte chunks of a key
  constexpr int kLaneKeys = 32 / kChunks;               // keys one copy instruction covers
  constexpr int kCopies = kWarpKeys / kLaneKeys;
  constexpr int kTileBytes = PagedSmem<DP>::kTileBytes;
  constexpr float kLift = Pair16<DT>::kBF16 ? 0.f : kNarrowLift, kUnlift = Pair16<DT>::kBF16 ? 1.f : 0x1p-15f;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Share share;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  find_share<kWarps * 32>(p, [&](int b) { return seq_work<kWin>(p, b, MT).units; }, &share);
  if (tid == 0) {
    p.splits[blockIdx.x].n = 0;
    p.status[blockIdx.x] = 0u;
  }

  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * (kStages * 2 * kTileBytes);
  const int copy_key = lane / kChunks, copy_chunk = lane % kChunks;
  const bool copy_in = copy_chunk * 8 < p.d;
  const int ld_row = lane & 7, ld_mat = lane >> 3;   // ldmatrix: this lane's row of matrix ld_mat

  PieceWalk walk(share);
  Piece x;
  bool keep_scores = false;
  if constexpr (kScores) {
    const ScorePlaces at = score_places<kWarps * 32, kWin>(p, share.seq);
    keep_scores = at.fit;
    walk.scores = at.base;
  }
  while (walk.next<MT, kWin, kScores>(p, x)) {
    // ---- keys and values: this warp's 16 keys of unit blk0 + i ----
    const int32_t* table = p.table + (long long)x.seq * p.table_stride;
    // lane l < 16 holds the offset of key l, lane 16 + l that of value l
    auto offset_of = [&](int i) {
      return i < x.steps ? cache_offset<kWin>(p, x, table,
                                              unit_of<kWin>(x, x.blk0 + i) * kUnit + warp * kWarpKeys + (lane & 15),
                                              lane >= 16)
                         : 0ll;
    };
    auto issue = [&](int i, int stage, long long off) {
      if (i < x.steps) {
        const uint32_t dst = ring + stage * (2 * kTileBytes);
#pragma unroll
        for (int c = 0; c < kCopies; ++c) {
          const int key = c * kLaneKeys + copy_key;
          const uint32_t at = key * (DP * 2) + ((copy_chunk ^ (key & 7)) << 4);
          const long long ko = __shfl_sync(0xffffffffu, off, key), vo = __shfl_sync(0xffffffffu, off, 16 + key);
          const bool take = copy_in && ko >= 0;
          const int col = copy_chunk * 8;
          cp_async16(dst + at, static_cast<const DT*>(p.kc) + (take ? ko + col : 0), take);
          cp_async16(dst + kTileBytes + at, static_cast<const DT*>(p.vc) + (take ? vo + col : 0), take);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i, i, offset_of(i));
    long long next_off = offset_of(kStages - 1);

    // ---- queries: the A fragments of the tile ----
    uint32_t qf[kKSteps][4];
    int token[2];            // of the row, -1 past the last row
    const int qr = lane >> 2, qc = (lane & 3) * 2;
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int r = hh * 8 + qr;
      const int row = x.row0 + r;
      const int tok = row / p.group;
      const bool ok = r < x.rows;
      token[hh] = ok ? tok : -1;
      const DT* src = static_cast<const DT*>(p.q) +
                      ((long long)(x.s.q_start + tok) * p.Hq + x.head * p.group + (row - tok * p.group)) * p.d;
#pragma unroll
      for (int k = 0; k < kKSteps; ++k) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int col = k * 16 + half * 8 + qc;
          qf[k][half * 2 + hh] = ok && col < p.d ? *reinterpret_cast<const uint32_t*>(src + col) : 0u;
        }
      }
    }

    float o[kNT][4], m[2], l[2], lr[2];
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      m[hh] = -INFINITY;
      l[hh] = lr[hh] = 0.f;
    }

    int stage = 0;
    for (int i = 0; i < x.steps; ++i) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      {
        const int fill = stage == 0 ? kStages - 1 : stage - 1;   // the stage read in the step before
        issue(i + kStages - 1, fill, next_off);
        next_off = offset_of(i + kStages);
      }
      const uint32_t kt = ring + stage * (2 * kTileBytes), vt = kt + kTileBytes;
      const int unit0 = unit_of<kWin>(x, x.blk0 + i) * kUnit;
      // ---- scores ----
      float c[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[n][e] = 0.f;
#pragma unroll
      for (int k = 0; k < kKSteps; ++k) {
        uint32_t kb[4];   // keys 0-7 (both halves of the 16 columns), keys 8-15
        const int row = ld_row + (ld_mat >> 1) * 8, chunk = 2 * k + (ld_mat & 1);
        ldsm4(kt + row * (DP * 2) + ((chunk ^ ld_row) << 4), kb);
        mma16816<DT>(c[0], qf[k], kb[0], kb[1]);
        mma16816<DT>(c[1], qf[k], kb[2], kb[3]);
      }
      // ---- visibility ----
      const bool cut = unit_cut<kWin>(p, x, unit0);
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[n][e] *= p.scale_log2;
      if (cut) {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const uint64_t all = token[hh] >= 0 ? seen_keys<kWin>(p, x, token[hh], unit0, tree_word(p, x, token[hh])) : 0ull;
          const uint32_t seen = (uint32_t)(all >> (warp * kWarpKeys)) >> qc;   // this lane's: bits 0, 1, 8, 9
          if (!(seen & 1)) c[0][2 * hh] = -INFINITY;
          if (!(seen & 2)) c[0][2 * hh + 1] = -INFINITY;
          if (!(seen & 256)) c[1][2 * hh] = -INFINITY;
          if (!(seen & 512)) c[1][2 * hh + 1] = -INFINITY;
        }
      }
      if constexpr (kScores) {
        if (keep_scores) {
          float* dst = p.scores + walk.scores +
                       (((long long)x.head * x.s.blocks + x.blk0 + i) * x.rows + qr) * kUnit + warp * kWarpKeys + qc;
#pragma unroll
          for (int hh = 0; hh < 2; ++hh)
            if (token[hh] >= 0) {
              float2* to = reinterpret_cast<float2*>(dst + hh * 8 * kUnit);
              to[0] = make_float2(c[0][2 * hh], c[0][2 * hh + 1]);
              to[4] = make_float2(c[1][2 * hh], c[1][2 * hh + 1]);
            }
        }
      }
      // ---- running maximum and sums, weights ----
      uint32_t pf[4];
      float scale[2];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        float top = fmaxf(fmaxf(c[0][2 * hh], c[0][2 * hh + 1]), fmaxf(c[1][2 * hh], c[1][2 * hh + 1]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        top = fmaxf(m[hh], top);
        const float use = top == -INFINITY ? 0.f : top;
        scale[hh] = ex2_approx(m[hh] - use);
        m[hh] = top;
        const float lifted = use - kLift;
        float sum = 0.f, sum_r = 0.f;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float p0 = ex2_approx(c[n][2 * hh] - lifted), p1 = ex2_approx(c[n][2 * hh + 1] - lifted);
          sum += p0 + p1;
          const uint32_t w = Pair16<DT>::put(p0, p1);
          const float2 r = Pair16<DT>::get(w);
          sum_r += r.x + r.y;
          pf[n * 2 + hh] = w;
        }
        l[hh] = l[hh] * scale[hh] + sum;
        lr[hh] = lr[hh] * scale[hh] + sum_r;
      }
      if (__any_sync(0xffffffffu, scale[0] != 1.f || scale[1] != 1.f)) {
#pragma unroll
        for (int n = 0; n < kNT; ++n) {
          o[n][0] *= scale[0];
          o[n][1] *= scale[0];
          o[n][2] *= scale[1];
          o[n][3] *= scale[1];
        }
      }
      // ---- output ----
#pragma unroll
      for (int n = 0; n < kNT; n += 2) {
        uint32_t vb[4];   // columns n: keys 0-7, 8-15; columns n + 1: the same
        const int row = ld_row + (ld_mat & 1) * 8, chunk = n + (ld_mat >> 1);
        ldsm4_trans(vt + row * (DP * 2) + ((chunk ^ ld_row) << 4), vb);
        mma16816<DT>(o[n], pf, vb[0], vb[1]);
        mma16816<DT>(o[n + 1], pf, vb[2], vb[3]);
      }
      stage = stage == kStages - 1 ? 0 : stage + 1;
      __syncwarp();   // every lane has read the stage that the next step's copies fill
    }
    cp_async_wait<0>();

    // ---- the warps' results joined ----
    __syncthreads();   // no warp reads its ring any more
    float* jo = reinterpret_cast<float*>(smem);                 // [warp][row][DP]
    float* jm = jo + kWarps * MT * DP;                          // [warp][3][row]
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int r = hh * 8 + qr;
      float a = l[hh], ar = lr[hh];
      a += __shfl_xor_sync(0xffffffffu, a, 1);
      a += __shfl_xor_sync(0xffffffffu, a, 2);
      ar += __shfl_xor_sync(0xffffffffu, ar, 1);
      ar += __shfl_xor_sync(0xffffffffu, ar, 2);
      if ((lane & 3) == 0) {
        jm[(warp * 3 + 0) * MT + r] = m[hh];
        jm[(warp * 3 + 1) * MT + r] = ar;
        jm[(warp * 3 + 2) * MT + r] = a;
      }
#pragma unroll
      for (int n = 0; n < kNT; ++n)
        *reinterpret_cast<float2*>(jo + (warp * MT + r) * DP + n * 8 + qc) =
            make_float2(o[n][2 * hh], o[n][2 * hh + 1]);
    }
    __syncthreads();
    const int part = part_of_piece(x);
    for (int i = tid; i < x.rows * kChunks; i += kWarps * 32) {
      const int r = i / kChunks, chunk = i - r * kChunks;
      float top = -INFINITY, w[kWarps], sr = 0.f, se = 0.f, acc[8];
#pragma unroll
      for (int k = 0; k < kWarps; ++k) top = fmaxf(top, jm[(k * 3) * MT + r]);
      const float use = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        w[k] = ex2_approx(jm[(k * 3) * MT + r] - use) * kUnlift;
        sr += w[k] * jm[(k * 3 + 1) * MT + r];
        se += w[k] * jm[(k * 3 + 2) * MT + r];
        const float4* src = reinterpret_cast<const float4*>(jo + (k * MT + r) * DP + chunk * 8);
        const float4 a = src[0], c = src[1];
        acc[0] += w[k] * a.x, acc[1] += w[k] * a.y, acc[2] += w[k] * a.z, acc[3] += w[k] * a.w;
        acc[4] += w[k] * c.x, acc[5] += w[k] * c.y, acc[6] += w[k] * c.z, acc[7] += w[k] * c.w;
      }
      if (x.whole) {
        const int row = x.row0 + r, tok = row / p.group, hq = x.head * p.group + (row - tok * p.group);
        const float inv = sr == 0.f ? 0.f : 1.f / sr;   // a NaN sum stays one
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = sr == 0.f ? 0.f : acc[e] * inv;
        if (chunk * 8 < p.d)
          *reinterpret_cast<uint4*>(static_cast<DT*>(p.out) + ((long long)(x.s.q_start + tok) * p.Hq + hq) * p.d +
                                    chunk * 8) = pack8<DT>(acc);
        if (chunk == 0 && p.lse)
          p.lse[(long long)hq * p.T + x.s.q_start + tok] =
              se == 0.f ? -INFINITY : use * 0.69314718055994531f + logf(se);
      } else {
        float* dst = p.part_o + (long long)part * MT * DP + (2 * chunk * MT + r) * 4;
        *reinterpret_cast<float4*>(dst) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        *reinterpret_cast<float4*>(dst + MT * 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
        if (chunk == 0) {
          float* pm = p.part_m + (long long)part * 3 * MT;
          pm[r] = top;
          pm[MT + r] = sr;
          pm[2 * MT + r] = se;
        }
      }
    }
    if (tid == 0) note_split(p, x, share);
    __syncthreads();   // the ring is filled again
  }
}

// Joins the partials of the tiles that several CTAs share, and writes the rows that have no units: rows
// of no sequence and of sequences without keys.  Block x works on the tile that goes on from CTA x to
// the next, so a tile of n partials has n - 1 blocks.  They share its tasks of 32 rows (a lane each:
// partials lie rows side by side) and 16 columns; a warp takes a task, or, of many partials (a
// long sequence alone), a block does, its warps a part of the partials each.  The time is that of a
// few dependent loads, so kJoinAhead partials are read at once and weighed against the maximum so far.
template <typename DT, int DP, int MT>
__global__ void __launch_bounds__(kJoinThreads) attn_paged_join_kernel(const PagedArgs p) {
  constexpr int kJoinWarps = kJoinThreads / 32;
  constexpr int kColumnGroups = DP / 16;
  __shared__ float shared[kJoinWarps][32][19];   // 19: rows in different banks
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // from the last block on: the first ones have tiles to join
  for (int t = ((int)gridDim.x - 1 - (int)blockIdx.x) * kJoinWarps + warp; t < p.T; t += gridDim.x * kJoinWarps) {
    const RowSpan at = find_span(p.cu, p.padded, p.B, t);
    if (at.seq >= 0 && p.kv_lens[at.seq] > 0 && p.max_pages > 0) continue;
    uint4* dst = reinterpret_cast<uint4*>(static_cast<DT*>(p.out) + (long long)t * p.Hq * p.d);
    for (int i = lane; i < p.Hq * (p.d / 8); i += 32) dst[i] = make_uint4(0u, 0u, 0u, 0u);
    if (p.lse)
      for (int h = lane; h < p.Hq; h += 32) p.lse[(long long)h * p.T + t] = -INFINITY;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.x == gridDim.x - 1) {   // the call's status word, from the CTAs'
    uint32_t bits = 0u;
    for (int i = tid; i < (int)gridDim.x; i += kJoinThreads) bits |= p.status[i];
    bits = __syncthreads_or(bits != 0u) ? THD_STATUS_WAIT_TIMEOUT : 0u;
    if (tid == 0) *p.call_status = bits;
  }
  const Split sp = p.splits[blockIdx.x];
  if (sp.n == 0) return;
  const int tasks = (sp.rows + 31) / 32 * kColumnGroups, mine = (int)blockIdx.x - sp.first, others = sp.n - 1;
  // a warp takes a task alone where that means fewer rounds of reads one after another
  const bool alone = (tasks + others * kJoinWarps - 1) / (others * kJoinWarps) * ((sp.n + kJoinAhead - 1) / kJoinAhead) <=
                     (tasks + others - 1) / others * ((sp.n + kJoinAhead * kJoinWarps - 1) / (kJoinAhead * kJoinWarps));
  const int k0 = alone ? 0 : warp, step = alone ? 1 : kJoinWarps;
  for (int task = alone ? mine * kJoinWarps + warp : mine; task < tasks; task += alone ? others * kJoinWarps : others) {
    const int cg = task % kColumnGroups, r = task / kColumnGroups * 32 + lane;
    const bool have = r < sp.rows;
    float top = -INFINITY, sr = 0.f, se = 0.f, acc[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = 0.f;
    if (have) {
      for (int k = k0; k < sp.n; k += kJoinAhead * step) {
        float m[kJoinAhead], lr[kJoinAhead], le[kJoinAhead];
        float4 v[kJoinAhead][4];
#pragma unroll
        for (int i = 0; i < kJoinAhead; ++i) {
          const int kk = k + i * step;
          m[i] = -INFINITY;
          if (kk < sp.n) {
            const long long part = (sp.first + kk) * 2 + (kk == 0 ? sp.second : 0);
            const float* pm = p.part_m + part * 3 * MT + r;
            const float* src = p.part_o + part * MT * DP + (cg * 4 * MT + r) * 4;
            m[i] = pm[0];
            lr[i] = pm[MT];
            le[i] = pm[2 * MT];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[i][e] = *reinterpret_cast<const float4*>(src + e * MT * 4);
          }
        }
        float next = top;
#pragma unroll
        for (int i = 0; i < kJoinAhead; ++i) next = fmaxf(next, m[i]);
        const float use = next == -INFINITY ? 0.f : next;
        const float old = ex2_approx(top - use);
        top = next;
        sr *= old, se *= old;
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[e] *= old;
#pragma unroll
        for (int i = 0; i < kJoinAhead; ++i) {
          if (k + i * step < sp.n) {
            const float w = ex2_approx(m[i] - use);
            sr += w * lr[i];
            se += w * le[i];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              acc[4 * e] += w * v[i][e].x, acc[4 * e + 1] += w * v[i][e].y;
              acc[4 * e + 2] += w * v[i][e].z, acc[4 * e + 3] += w * v[i][e].w;
            }
          }
        }
      }
    }
    if (!alone) {   // over the warps, in their order
      float* own = shared[warp][lane];
      own[0] = top, own[1] = sr, own[2] = se;
#pragma unroll
      for (int e = 0; e < 16; ++e) own[3 + e] = acc[e];
      __syncthreads();
      if (warp == 0 && have) {
#pragma unroll
        for (int k = 1; k < kJoinWarps; ++k) top = fmaxf(top, shared[k][lane][0]);
        const float use = top == -INFINITY ? 0.f : top;
        const float w0 = ex2_approx(own[0] - use);
        sr *= w0, se *= w0;
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[e] *= w0;
        for (int k = 1; k < kJoinWarps; ++k) {
          const float* from = shared[k][lane];
          const float w = ex2_approx(from[0] - use);
          sr += w * from[1];
          se += w * from[2];
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[e] += w * from[3 + e];
        }
      }
      __syncthreads();
    }
    if (have && (alone || warp == 0)) {
      const int row = sp.row0 + r, tok = row / p.group, hq = sp.head * p.group + (row - tok * p.group);
      const long long t = sp.q_start + tok;
      DT* dst = static_cast<DT*>(p.out) + (t * p.Hq + hq) * p.d + cg * 16;
      const float inv = 1.f / sr;
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[e] = sr == 0.f ? 0.f : acc[e] * inv;
#pragma unroll
      for (int e = 0; e < 16; e += 8)
        if (cg * 16 + e < p.d) *reinterpret_cast<uint4*>(dst + e) = pack8<DT>(acc + e);
      if (cg == 0 && p.lse)
        p.lse[(long long)hq * p.T + t] =
            se == 0.f ? -INFINITY : (top == -INFINITY ? 0.f : top) * 0.69314718055994531f + logf(se);
    }
  }
}

// Workspace: the call's status word (byte 8), the CTAs' status words and split tiles, then the
// partial results (outputs, then maxima and sums).
constexpr int kMaxRows = 128;   // rows of a tile at most
constexpr size_t kStatusAt = 256, kSplitAt = kStatusAt + kMaxCtas * sizeof(uint32_t);
constexpr size_t kPartAt = kSplitAt + kMaxCtas * sizeof(Split);
constexpr size_t part_bytes(int dp) { return (size_t)kMaxCtas * 2 * kMaxRows * (dp + 3) * 4; }

// The keys' weights: tiles of 128 rows on the tensor cores where the attention took them, unless a group has more
// heads than such a tile rows.
template <typename DT, int DP, bool kWide, bool kWin>
int launch_key_weights(const PagedArgs& p, int sms, cudaStream_t st) {
  if constexpr (kWide) {
    if (p.group <= kWwRows) {
      const int tokens = kWwRows / p.group;
      CUtensorMap map;
      if (!encode_group_map(&map, p.q, p.T, p.Hq, p.d, p.group, tokens, Pair16<DT>::kBF16)) return THD_ERR_CUDA;
      auto kern = attn_key_weights_wide_kernel<DT, DP, kWin>;
      constexpr int smem = (int)sizeof(WwSmem<DP>) + 1024;
      static SmemGrant grant;
      if (!grant.ask(kern, smem)) return THD_ERR_CUDA;
      kern<<<sms, kWwThreads, smem, st>>>(map, p, tokens);
      return cudaGetLastError() == cudaSuccess ? THD_OK : THD_ERR_CUDA;
    }
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(4 * sms);
  cfg.blockDim = dim3(kWeightWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_key_weights_kernel<DT, DP, kWin>, p) == cudaSuccess ? THD_OK : THD_ERR_CUDA;
}

template <typename DT, int DP, int MT, bool kWin>
int launch_paged(PagedArgs& p, char* ws, int sms, cudaStream_t st) {
  p.call_status = reinterpret_cast<uint32_t*>(ws + 8);
  p.status = reinterpret_cast<uint32_t*>(ws + kStatusAt);
  p.splits = reinterpret_cast<Split*>(ws + kSplitAt);
  p.part_o = reinterpret_cast<float*>(ws + kPartAt);
  p.part_m = p.part_o + (size_t)kMaxCtas * 2 * MT * DP;
  if (MT != kNarrowRows || !p.key_weights || p.score_room <= 0) p.scores = nullptr;
  const int grid = 2 * sms < kMaxCtas ? 2 * sms : kMaxCtas;
  static SmemGrant grant;
  if constexpr (MT == kWideRows) {
    auto kern = attn_paged_wide_kernel<DT, DP, kWin>;
    constexpr int smem = (int)sizeof(WideSmem<DP>) + 1024;
    if (!grant.ask(kern, smem)) return THD_ERR_CUDA;
    kern<<<grid, kWideThreads, smem, st>>>(p);
  } else {
    auto kern = p.scores ? attn_paged_kernel<DT, DP, kWin, true> : attn_paged_kernel<DT, DP, kWin, false>;
    constexpr int smem = PagedSmem<DP>::kBytes;
    static SmemGrant grant_scores;
    if (!(p.scores ? grant_scores : grant).ask(kern, smem)) return THD_ERR_CUDA;
    kern<<<grid, kWarps * 32, smem, st>>>(p);
  }
  if (cudaGetLastError() != cudaSuccess) return THD_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, attn_paged_join_kernel<DT, DP, MT>, static_cast<const PagedArgs>(p)) != cudaSuccess)
    return THD_ERR_CUDA;
  return p.key_weights ? launch_key_weights<DT, DP, MT == kWideRows, kWin>(p, sms, st) : THD_OK;
}

// Tiles of 16 rows where no sequence has more, else of 128.  120000 keys of 16 sequences, 32 + 8 heads of 128,
// bf16, in us: 16 rows 89 narrow; 20 rows 94 wide, against 124 in narrow tiles of 32; 64 rows 98, against 229 in
// two such tiles.  Heads of 64 in fp16: 32 rows 62 and 70, 36 rows 68 and 117.  Wide tiles of 4 rows (a
// decoding batch called without the hint) cost 324 where narrow ones cost 317.
template <typename DT, bool kWin>
int launch_paged_rows(PagedArgs& p, long long row_hint, char* ws, int sms, cudaStream_t st) {
  if (p.d > 64) {
    if (row_hint <= kNarrowRows) return launch_paged<DT, 128, kNarrowRows, kWin>(p, ws, sms, st);
    return launch_paged<DT, 128, kWideRows, kWin>(p, ws, sms, st);
  }
  if (row_hint <= kNarrowRows) return launch_paged<DT, 64, kNarrowRows, kWin>(p, ws, sms, st);
  return launch_paged<DT, 64, kWideRows, kWin>(p, ws, sms, st);
}

// A window has kernels of its own: a call without one does what it did.
template <typename DT>
int launch_paged_of(PagedArgs& p, long long row_hint, char* ws, int sms, cudaStream_t st) {
  if (p.win_left >= 0) return launch_paged_rows<DT, true>(p, row_hint, ws, sms, st);
  return launch_paged_rows<DT, false>(p, row_hint, ws, sms, st);
}

}  // namespace
}  // namespace thd

extern "C" {

size_t thd_attn_paged_workspace_size(int head_dim) {
  if (head_dim < 8 || head_dim > 128 || head_dim % 8 != 0) return 0;
  return thd::kPartAt + thd::part_bytes(head_dim > 64 ? 128 : 64);
}

size_t thd_attn_paged_weights_workspace_size(int head_dim, int num_heads_q, int batch_size, int max_seqlen_q,
                                             int num_pages, int page_size, int max_pages, int window_left,
                                             int sink_tokens) {
  const size_t base = thd_attn_paged_workspace_size(head_dim);
  if (base == 0 || num_heads_q < 1 || batch_size < 0 || max_seqlen_q < 1 || num_pages < 0 || page_size < 1 ||
      max_pages < 0 || window_left < -1 || sink_tokens < 0)
    return 0;
  // keys in whole units: of a sequence at most, and, of sequences that share no pages, of all of them
  const double unit = thd::kUnit;
  double keys = (double)max_pages * page_size;
  if (window_left >= 0) {
    const double seen = (double)window_left + max_seqlen_q + sink_tokens + 3 * unit;
    keys = seen < keys ? seen : keys;
  }
  double all = (double)batch_size * (keys + unit);
  const double held = (double)num_pages * page_size + (double)batch_size * unit;
  if (held < all) all = held;
  const double bytes = all * num_heads_q * max_seqlen_q * 4.0;
  return bytes < 1e15 ? (base + 15) / 16 * 16 + (size_t)bytes : 0;
}

int thd_attn_paged_window(const void* q, const void* k_cache, const void* v_cache, const int64_t* cache_strides,
                   int num_pages, int page_size, const int32_t* page_table, int64_t page_table_stride, int max_pages,
                   const int32_t* kv_lens, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_q_padded,
                   int batch_size, int max_seqlen_q, const int64_t* tree_mask, int tree_words, int window_left,
                   int sink_tokens, float* key_weights, const int64_t* weight_strides, float softmax_scale, void* out, float* lse, int total_tokens, int num_heads_q, int num_heads_kv, int head_dim, int dtype,
                   void* workspace, size_t workspace_bytes, void* stream) {
  using namespace thd;
  if (batch_size < 0 || max_seqlen_q < 0 || total_tokens < 0) return THD_ERR_ARG;
  if (num_heads_q < 1 || num_heads_kv < 1 || num_pages < 0 || page_size < 1 || max_pages < 0) return THD_ERR_ARG;
  if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.f)) return THD_ERR_ARG;
  if (dtype != THD_BF16 && dtype != THD_FP16) return THD_ERR_UNSUPPORTED;
  if (head_dim < 8 || head_dim > 128 || head_dim % 8 != 0) return THD_ERR_UNSUPPORTED;
  if (num_heads_q % num_heads_kv != 0) return THD_ERR_UNSUPPORTED;
  const int group = num_heads_q / num_heads_kv;
  // rows of a sequence and keys of a table are 32-bit
  if ((long long)total_tokens * group >= (1ll << 30) || (long long)max_pages * page_size >= (1ll << 31) - kUnit)
    return THD_ERR_UNSUPPORTED;
  if ((long long)num_heads_q * head_dim >= (1ll << 31)) return THD_ERR_UNSUPPORTED;
  if (tree_mask && (tree_words < 1 || tree_words > (1 << 20))) return THD_ERR_ARG;
  if (window_left < -1 || sink_tokens < 0) return THD_ERR_ARG;
  // where drafted tokens stand to one another only their mask says, so a window has no meaning for them
  if (window_left >= 0 && tree_mask) return THD_ERR_UNSUPPORTED;
  if (!cache_strides || page_table_stride < max_pages) return THD_ERR_ARG;
  for (int i = 0; i < 6; ++i)
    if (cache_strides[i] < 0 || cache_strides[i] % 8 != 0) return THD_ERR_ARG;
  if (key_weights) {
    if (!weight_strides || !lse || !on4(key_weights)) return THD_ERR_ARG;
    for (int i = 0; i < 3; ++i)
      if (weight_strides[i] < 0) return THD_ERR_ARG;
  }
  if (total_tokens == 0) return THD_OK;
  if (!q || !out || !on16(q) || !on16(out) || !on4(lse)) return THD_ERR_ARG;
  if (!on4(page_table) || !on4(kv_lens) || !on4(cu_seqlens_q) || !on4(cu_seqlens_q_padded) ||
      (reinterpret_cast<uintptr_t>(tree_mask) & 7) != 0)
    return THD_ERR_ARG;
  if (batch_size > 0 && (!kv_lens || !cu_seqlens_q)) return THD_ERR_ARG;
  // without pages no sequence has keys
  if (num_pages == 0) max_pages = 0;
  if (batch_size > 0 && max_pages > 0 && (!page_table || !k_cache || !v_cache)) return THD_ERR_ARG;
  if (!on16(k_cache) || !on16(v_cache)) return THD_ERR_ARG;
  if (!workspace || !on16(workspace) || workspace_bytes < thd_attn_paged_workspace_size(head_dim))
    return THD_ERR_WORKSPACE;
  const int sms = device_sms();
  if (sms <= 0) return THD_ERR_CUDA;
  PagedArgs p{};
  p.q = q;
  p.kc = k_cache;
  p.vc = v_cache;
  p.table = page_table;
  p.kv_lens = kv_lens;
  p.cu = cu_seqlens_q;
  p.padded = cu_seqlens_q_padded;
  p.tree = reinterpret_cast<const long long*>(tree_mask);
  p.out = out;
  p.lse = lse;
  p.table_stride = page_table_stride;
  p.k_page = cache_strides[0];
  p.k_token = cache_strides[1];
  p.k_head = cache_strides[2];
  p.v_page = cache_strides[3];
  p.v_token = cache_strides[4];
  p.v_head = cache_strides[5];
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.max_pages = max_pages;
  p.page_shift = -1;
  for (int s = 0; s < 31; ++s)
    if (page_size == 1 << s) p.page_shift = s;
  p.same_places = p.k_page == p.v_page && p.k_token == p.v_token && p.k_head == p.v_head;
  p.tree_words = tree_mask ? tree_words : 0;
  p.B = batch_size;
  p.T = total_tokens;
  p.Hq = num_heads_q;
  p.Hkv = num_heads_kv;
  p.group = group;
  p.d = head_dim;
  // a window of as many keys as the table has room for hides none
  p.win_left = window_left < (long long)max_pages * page_size ? window_left : -1;
  p.sinks = p.win_left >= 0 ? sink_tokens : 0;
  if (key_weights && batch_size > 0 && max_pages > 0) {
    p.key_weights = key_weights;
    p.w_page = weight_strides[0];
    p.w_token = weight_strides[1];
    p.w_head = weight_strides[2];
    const size_t base = (thd_attn_paged_workspace_size(head_dim) + 15) / 16 * 16;
    p.scores = reinterpret_cast<float*>(static_cast<char*>(workspace) + base);
    p.score_room = workspace_bytes > base ? (long long)((workspace_bytes - base) / 4) : 0;
  }
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  wait_settings(&p.wait_limit_ns, &p.wait_check_mask, &p.inject_wait);
  long long longest = max_seqlen_q > 0 && max_seqlen_q < total_tokens ? max_seqlen_q : total_tokens;
  return dtype == THD_BF16
             ? launch_paged_of<__nv_bfloat16>(p, longest * group, static_cast<char*>(workspace), sms,
                                              static_cast<cudaStream_t>(stream))
             : launch_paged_of<__half>(p, longest * group, static_cast<char*>(workspace), sms,
                                       static_cast<cudaStream_t>(stream));
}

int thd_attn_paged(const void* q, const void* k_cache, const void* v_cache, const int64_t* cache_strides,
                   int num_pages, int page_size, const int32_t* page_table, int64_t page_table_stride, int max_pages,
                   const int32_t* kv_lens, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_q_padded,
                   int batch_size, int max_seqlen_q, const int64_t* tree_mask, int tree_words, float softmax_scale,
                   void* out, float* lse, int total_tokens, int num_heads_q, int num_heads_kv, int head_dim, int dtype,
                   void* workspace, size_t workspace_bytes, void* stream) {
  return thd_attn_paged_window(q, k_cache, v_cache, cache_strides, num_pages, page_size, page_table, page_table_stride,
                               max_pages, kv_lens, cu_seqlens_q, cu_seqlens_q_padded, batch_size, max_seqlen_q,
                               tree_mask, tree_words, -1, 0, nullptr, nullptr, softmax_scale, out, lse, total_tokens,
                               num_heads_q, num_heads_kv, head_dim, dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
