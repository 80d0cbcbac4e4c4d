// attn_paged_wide.cuh — attention over a paged cache for tiles of 128 query rows, on the
// fifth-generation tensor cores: chunks of new tokens and trees of drafted ones, where more
// than 32 rows share a key/value head.
//
// The same split of the batch's keys over the CTAs as the narrow kernel's (attn_paged.cu), one CTA
// per SM; inside a CTA the work is divided among warps:
//   warps 0-3, 4-7  softmax of the even and the odd units of a piece, one thread per row: scores out of
//                   tensor memory, weights back over them, a running maximum and sums; at the
//                   piece's end the two streams' outputs are added, half of the columns each
//   warps 8, 9      keys and values, out of the pages into the swizzled layout of the matrix unit:
//                   tensor copies of whole boxes of a page, or rows in pieces of 16 bytes
//   warp 10         issues the matrix products: S = Q K^T, O += P V
// What bounds it: with up to 128 rows for each key a unit's 32 KB take about 1400 cycles to come
// from memory on an SM, its two products 512 cycles of the tensor pipe, and the softmax of one
// unit 1000 to 1500.  So two softmax streams, each with two score tiles and an output tile of its
// own (all of tensor memory): up to four units' scores are computed ahead, and neither product waits
// for the other stream.  Two CTAs per SM with one stream and one score tile each ran scores,
// softmax and output of a unit one after another: 92 us where this takes @WIDE@ (trees of 27
// tokens, 108 rows, over 120000 keys of 8 heads; 74 us at the copy bandwidth).
//
// Every wait is bounded as in the other attention kernels: one that runs out sets the CTA's
// status word, and the CTA lets what it started finish and leaves.
#pragma once
#include "attn_paged_common.cuh"

namespace thd {
namespace {

constexpr int kWideRows = 128;
constexpr int kWideThreads = 384;
constexpr int kWideKStages = 5, kWideVStages = 6;   // units of keys, of values on the way
constexpr int kWideLag = 3;               // rows: units whose copies may still be flying when one is announced
constexpr uint32_t kWideTmemCols = 512;   // S (and P) of stream t, buffer s: 64 at 128 t + 64 s; O of stream t at 256 + 128 t

template <int DP>
struct WideSmem {
  static constexpr int kTileBytes = kUnit * DP * 2;   // panels of 64 rows x 128 bytes
  alignas(1024) uint8_t q[kWideRows * DP * 2];        // panels of 128 rows x 128 bytes
  alignas(1024) uint8_t k[kWideKStages][kTileBytes];
  alignas(1024) uint8_t v[kWideVStages][kTileBytes];
  // each stream's maximum, sum of the rounded weights, sum of the weights; by turns of pieces, since a
  // stream without units in a piece comes to its statistics while the others still read the last ones
  float stats[2][2][3][kWideRows];
  uint64_t places[2][kUnit];      // addresses of a unit's keys, values
  uint64_t k_full[kWideKStages], k_empty[kWideKStages], v_full[kWideVStages], v_empty[kWideVStages];
  // by stream and by turns of its units: a wait names a phase by its parity, so it must come at most one
  // phase late, and the scores of a unit say that the products of the unit two before it are done
  uint64_t s_full[2][2], p_full[2][2], o_full[2][2];
  uint64_t q_full, stats_full, o_free, drain, never;
  uint32_t tmem_base, abort;
  Share share;
};

// Waits of a whole warp, which leaves them together.
#define WIDE_WAIT(bar, parity)                                                                                     \
  (__all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, &p.status[blockIdx.x], THD_STATUS_WAIT_TIMEOUT,      \
                                     p.wait_limit_ns, p.wait_check_mask) ? 1 : 0) != 0)

// Copies the 64 rows of a unit out of the pages, by one warp in pieces of 16 bytes: each lane finds
// two rows (their pages given), and the addresses go round through shared memory, so that 512 bytes
// cost a load of an address, an add and the copy.  Rows that no query sees become zeros.
template <typename DT, int DP>
__device__ __forceinline__ void copy_rows(const PagedArgs& p, const Piece& x, const int (&page)[2], int first,
                                          bool values, const DT** places, uint8_t* tile) {
  constexpr int kChunks = DP / 8, kLaneKeys = 32 / kChunks, kCopies = kUnit / kLaneKeys;
  const int lane = threadIdx.x & 31;
  const int copy_key = lane / kChunks, copy_chunk = lane % kChunks;
  const bool copy_in = copy_chunk * 8 < p.d;
  const int col = copy_in ? copy_chunk * 8 : 0;
  const DT* cache = static_cast<const DT*>(values ? p.vc : p.kc);
  __syncwarp();   // the last addresses have been read
#pragma unroll
  for (int k = 0; k < 2; ++k)
    places[32 * k + lane] = cache + place_in_cache(p, x, page[k], first + 32 * k + lane, values);
  __syncwarp();
  const uint32_t at = smem_u32(tile) + (copy_chunk >> 3) * (kUnit * 128) + copy_key * 128;
  const int keys = copy_in ? x.key_end - first : 0;   // of the unit, that some row sees
#pragma unroll
  for (int c0 = 0; c0 < kCopies; c0 += 8) {   // eight addresses at a time, so that reading them overlaps
    const DT* from[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) from[c] = places[(c0 + c) * kLaneKeys + copy_key] + col;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int key = (c0 + c) * kLaneKeys + copy_key;
      const uint32_t swizzled = ((copy_chunk & 7) ^ (key & 7)) << 4;   // one of 8 / kLaneKeys values
      cp_async16(at + (c0 + c) * (kLaneKeys * 128) + swizzled, from[c], key < keys);
    }
  }
}

// Streams all of the CTA's units of keys (or values) through a ring of shared memory; one warp.  With any
// pages and head_dim: copies of 16 bytes, a unit announced kWideLag units later, when its own have landed.
template <typename DT, int DP, int kRing>
__device__ void wide_load_rows(const PagedArgs& p, PieceWalk walk, bool values,
                               uint8_t (*ring)[WideSmem<DP>::kTileBytes], uint64_t* places, uint64_t* full,
                               uint64_t* empty, volatile uint32_t* abort_flag) {
  const int lane = threadIdx.x & 31;
  uint32_t n = 0;   // units issued
  auto announce = [&](uint32_t i) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&full[i % kRing]);
  };
  Piece x;
  while (walk.next<kWideRows>(p, x)) {
    const int32_t* table = p.table + (long long)x.seq * p.table_stride;
    int page[2];   // of the lane's two rows of the unit issued next
#pragma unroll
    for (int k = 0; k < 2; ++k) page[k] = cache_page(p, x, table, x.blk0 * kUnit + 32 * k + lane);
    for (int i = 0; i < x.steps; ++i, ++n) {
      const int first = (x.blk0 + i) * kUnit;
      if (n >= kRing && !WIDE_WAIT(&empty[n % kRing], (n / kRing - 1) & 1)) {
        cp_async_wait<0>();
        return;
      }
      copy_rows<DT, DP>(p, x, page, first, values, reinterpret_cast<const DT**>(places), ring[n % kRing]);
      cp_async_commit();
      if (i + 1 < x.steps) {
#pragma unroll
        for (int k = 0; k < 2; ++k) page[k] = cache_page(p, x, table, first + kUnit + 32 * k + lane);
      }
      if (n >= kWideLag) {
        cp_async_wait<kWideLag>();
        announce(n - kWideLag);
      }
    }
  }
  cp_async_wait<0>();
  for (uint32_t i = n < kWideLag ? 0 : n - kWideLag; i < n; ++i) announce(i);
}

// The same by tensor copies, where a page is a multiple of 8 tokens and head_dim 64 or 128: boxes of `box`
// tokens (the largest power of two that divides the page and the unit) by 64 columns, a lane each.
// A box past the last visible key is left out; the unit of values that such a key ends in goes row by
// row instead, so that what lies behind it becomes zeros (the scores there are masked, whatever they are).
template <typename DT, int DP, int kRing>
__device__ void wide_load_boxes(const PagedArgs& p, const CUtensorMap* map, int box, PieceWalk walk, bool values,
                                uint8_t (*ring)[WideSmem<DP>::kTileBytes], uint64_t* places, uint64_t* full,
                                uint64_t* empty, volatile uint32_t* abort_flag) {
  constexpr int kPanels = DP / 64;
  const int lane = threadIdx.x & 31;
  const int panel = lane % kPanels, row = lane / kPanels * box;   // of this lane's box
  uint32_t n = 0;
  bool ok = true;
  Piece x;
  while (ok && walk.next<kWideRows>(p, x)) {
    const int32_t* table = p.table + (long long)x.seq * p.table_stride;
    int page = row < kUnit ? cache_page(p, x, table, x.blk0 * kUnit + row) : 0;
    for (int i = 0; i < x.steps; ++i, ++n) {
      const int first = (x.blk0 + i) * kUnit, keys = min(kUnit, x.key_end - first);
      const uint32_t st = n % kRing;
      if (n >= kRing && !WIDE_WAIT(&empty[st], (n / kRing - 1) & 1)) {
        ok = false;
        break;
      }
      if (values && keys < kUnit) {
        int pages[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) pages[k] = cache_page(p, x, table, first + 32 * k + lane);
        copy_rows<DT, DP>(p, x, pages, first, true, reinterpret_cast<const DT**>(places), ring[st]);
        cp_async_commit();
        cp_async_wait<0>();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
      } else {
        const int at = max(0, min(page, p.num_pages - 1)), token = (first + row) % p.page_size;
        if (lane == 0) mbar_arrive_expect_tx(&full[st], (keys + box - 1) / box * box * 128 * kPanels);
        __syncwarp();
        if (row < keys)
          tma_load_4d(ring[st] + panel * (kUnit * 128) + row * 128, map, &full[st], panel * 64, x.head, token, at);
      }
      if (i + 1 < x.steps && row < kUnit) page = cache_page(p, x, table, first + kUnit + row);
    }
  }
  if (!ok)   // the copies in flight land before the CTA leaves
    for (uint32_t i = n < kRing ? 0 : n - kRing; i < n; ++i) drain_wait(&full[i % kRing], (i / kRing) & 1);
}

template <typename DT, int DP, bool kBoxes>
__global__ void __launch_bounds__(kWideThreads, 1)
    attn_paged_wide_kernel(const PagedArgs p, const __grid_constant__ CUtensorMap key_map,
                           const __grid_constant__ CUtensorMap value_map, int box) {
  using Tr = Pair16<DT>;
  constexpr int kPanelBytes = kUnit * 128;
  constexpr uint32_t idesc_qk = umma_idesc_f16(Tr::kBF16, kWideRows, kUnit, false);
  constexpr uint32_t idesc_pv = umma_idesc_f16(Tr::kBF16, kWideRows, DP, true);
  extern __shared__ uint8_t smem_raw[];
  WideSmem<DP>& sm = *reinterpret_cast<WideSmem<DP>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                      ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile uint32_t* abort_flag = &sm.abort;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    for (int i = 0; i < kWideKStages; ++i) mbar_init(&sm.k_full[i], 1), mbar_init(&sm.k_empty[i], 1);
    for (int i = 0; i < kWideVStages; ++i) mbar_init(&sm.v_full[i], 1), mbar_init(&sm.v_empty[i], 1);
    for (int t = 0; t < 2; ++t) {
      for (int s = 0; s < 2; ++s) {
        mbar_init(&sm.s_full[t][s], 1);
        mbar_init(&sm.p_full[t][s], 4);   // one lane of each of the stream's warps
        mbar_init(&sm.o_full[t][s], 1);
      }
    }
    mbar_init(&sm.q_full, 8);             // one lane of each softmax warp
    mbar_init(&sm.stats_full, 8);
    mbar_init(&sm.o_free, 8);
    mbar_init(&sm.drain, 1);
    mbar_init(&sm.never, 1);
    fence_mbar_init();
    sm.abort = 0u;
    p.splits[blockIdx.x].n = 0;
    p.status[blockIdx.x] = 0u;
  }
  if (warp == 10) {
    tmem_alloc(&sm.tmem_base, kWideTmemCols);
    tmem_relinquish();
  }
  find_share<kWideThreads>(p, kWideRows, &sm.share);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const Share share = sm.share;
  PieceWalk walk(share);
  Piece x;

  if (warp == 8) {
    if constexpr (kBoxes)
      wide_load_boxes<DT, DP, kWideKStages>(p, &key_map, box, walk, false, sm.k, sm.places[0], sm.k_full, sm.k_empty,
                                            abort_flag);
    else
      wide_load_rows<DT, DP, kWideKStages>(p, walk, false, sm.k, sm.places[0], sm.k_full, sm.k_empty, abort_flag);
  } else if (warp == 9) {
    if constexpr (kBoxes)
      wide_load_boxes<DT, DP, kWideVStages>(p, &value_map, box, walk, true, sm.v, sm.places[1], sm.v_full, sm.v_empty,
                                            abort_flag);
    else
      wide_load_rows<DT, DP, kWideVStages>(p, walk, true, sm.v, sm.places[1], sm.v_full, sm.v_empty, abort_flag);
  } else if (warp == 10) {
    // ---------------------------------------------------------------- products
    const bool issue = elect_one_sync();
    auto ready = [&](uint64_t* bar, uint32_t parity) {   // lane 0's answer for the whole warp
      return __shfl_sync(0xffffffffu, mbar_test_wait(bar, parity) ? 1 : 0, 0) != 0;
    };
    uint32_t ns = 0, np = 0;         // units whose scores, whose outputs have been issued
    uint32_t cs[2] = {0, 0}, cp[2] = {0, 0};   // the same by stream
    uint32_t pieces = 0;
    const uint32_t hi = smem_desc_sw128_hi(1024), qlo = smem_desc_sw128_lo(smem_u32(sm.q), 16);
    bool ok = true;
    if (p.inject_wait) ok = WIDE_WAIT(&sm.never, 0);   // test setting: a wait that runs out, loads in flight
    while (ok && walk.next<kWideRows>(p, x)) {
      if (x.steps == 0) continue;
      if (!WIDE_WAIT(&sm.q_full, pieces & 1)) break;
      int is = 0, ip = 0;   // of this piece
      uint64_t since = globaltimer_ns();
      for (uint32_t polls = 1; ok && ip < x.steps; ++polls) {
        bool moved = false;
        // scores of the next unit: its tile of tensor memory is free once the outputs of the unit four
        // before it, which read its weights there, have been issued
        if (is < x.steps && is < ip + 4 && ready(&sm.k_full[ns % kWideKStages], (ns / kWideKStages) & 1)) {
          const int t = is & 1, s = cs[t] & 1;
          tc_fence_after();
          const uint32_t klo = smem_desc_sw128_lo(smem_u32(sm.k[ns % kWideKStages]), 16);
#pragma unroll
          for (int kk = 0; kk < DP / 16; ++kk)
            umma_ss_if(issue, tmem + 128 * t + 64 * s,
                       smem_desc_join(qlo + (((kk >> 2) * (kWideRows * 128) + (kk & 3) * 32) >> 4), hi),
                       smem_desc_join(klo + (((kk >> 2) * kPanelBytes + (kk & 3) * 32) >> 4), hi), idesc_qk,
                       kk > 0 ? 1u : 0u);
          umma_commit_if(issue, &sm.s_full[t][s]);
          umma_commit_if(issue, &sm.k_empty[ns % kWideKStages]);
          ++is, ++ns, ++cs[t];
          moved = true;
        }
        // outputs of the oldest unit
        const int t = ip & 1, s = cp[t] & 1;
        if (ip < is && ready(&sm.p_full[t][s], (cp[t] >> 1) & 1) &&
            ready(&sm.v_full[np % kWideVStages], (np / kWideVStages) & 1)) {
          if (ip == 0 && pieces > 0 && !WIDE_WAIT(&sm.o_free, (pieces - 1) & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t vlo = smem_desc_sw128_lo(smem_u32(sm.v[np % kWideVStages]), kPanelBytes);
#pragma unroll
          for (int kk = 0; kk < kUnit / 16; ++kk)
            umma_ts_if(issue, tmem + 256 + 128 * t, tmem + 128 * t + 64 * s + kk * 8,
                       smem_desc_join(vlo + ((kk * 16 * 128) >> 4), hi), idesc_pv, (ip > 1 || kk > 0) ? 1u : 0u);
          umma_commit_if(issue, &sm.o_full[t][s]);
          umma_commit_if(issue, &sm.v_empty[np % kWideVStages]);
          ++ip, ++np, ++cp[t];
          moved = true;
        }
        if (moved) {
          polls = 0;
        } else if ((polls & p.wait_check_mask) == 0) {   // bounded as mbar_wait is
          if (polls <= p.wait_check_mask + 1) since = globaltimer_ns();
          const bool late = lane == 0 && globaltimer_ns() - since > p.wait_limit_ns;
          if (late) {
            *abort_flag = 1u;
            atomicOr(&p.status[blockIdx.x], THD_STATUS_WAIT_TIMEOUT);
          }
          if (__any_sync(0xffffffffu, late || *abort_flag)) ok = false;
        }
      }
      ++pieces;
    }
    // what was issued completes before tensor memory is released
    umma_commit_if(issue, &sm.drain);
    drain_wait(&sm.drain, 0);
  } else if (warp < 8) {
    // ---------------------------------------------------------------- softmax
    const int t = warp >> 2, r = tid & 127;   // stream; row of the tile, lane of tensor memory
    const uint32_t t_lane = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + t_lane + 128 * t, tO = tmem + t_lane + 256;
    const float sl2 = p.scale_log2;
    uint32_t n[2] = {0, 0};   // units of each stream so far
    uint32_t pieces = 0;
    bool ok = true;
    while (ok && walk.next<kWideRows>(p, x)) {
      const int row = x.row0 + r, tok = row / p.group, hq = x.head * p.group + (row - tok * p.group);
      const bool valid = r < x.rows;
      const long long at = ((long long)(x.s.q_start + (valid ? tok : 0)) * p.Hq + (valid ? hq : 0)) * p.d;
      const int units[2] = {(x.steps + 1) / 2, x.steps / 2};
      if (x.steps > 0) {
        // this stream's half of the row's query; the last piece's products have read theirs
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const DT*>(p.q) + at);
#pragma unroll
        for (int e = 0; e < DP / 16; ++e) {
          const int c = t * (DP / 16) + e;
          uint4 w = make_uint4(0u, 0u, 0u, 0u);
          if (valid && c * 8 < p.d) w = src[c];
          *reinterpret_cast<uint4*>(sm.q + (c >> 3) * (kWideRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = w;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_full);
      }
      float m_run = -INFINITY, l_run = 0.f, l_exact = 0.f;
      for (int i = t; i < x.steps; i += 2) {
        const uint32_t c = n[t] + (i >> 1);
        const uint32_t tT = tS + 64 * (c & 1);
        if (!WIDE_WAIT(&sm.s_full[t][c & 1], (c >> 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t sr[64];
        tmem_ld32(tT, sr);
        tmem_ld32(tT + 32, sr + 32);
        tmem_ld_wait_regs32(sr);
        tmem_tie_regs32(sr + 32);
        const int first = (x.blk0 + i) * kUnit;
        if (first + kUnit > min(p.tree ? x.past : x.past + 1, x.s.kv_len)) {   // some key may be hidden from some row
          const uint64_t seen = valid ? seen_keys(p, x, tok, first) : 0ull;
          const uint32_t lo = (uint32_t)seen, hi = (uint32_t)(seen >> 32);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            if (!(lo >> e & 1)) sr[e] = __float_as_uint(-INFINITY);
            if (!(hi >> e & 1)) sr[32 + e] = __float_as_uint(-INFINITY);
          }
        }
        float mx[4] = {m_run, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 64; e += 8) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mx[k] = fmax3f(mx[k], __uint_as_float(sr[e + 2 * k]), __uint_as_float(sr[e + 2 * k + 1]));
        }
        const float m_new = fmax3f(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
        // the maximum moves only when it grows by more than 8 (log2): weights stay below 2^8 and the
        // output is seldom rescaled
        const bool need = (m_new - m_run) * sl2 > 8.f;   // false while both are -inf
        float alpha = 1.f;
        if (need) {
          alpha = ex2_approx((m_run - m_new) * sl2);
          m_run = m_new;
          l_run *= alpha;
          l_exact *= alpha;
        }
        const float mb = (m_run == -INFINITY ? 0.f : m_run) * sl2;
        float ex[4] = {0.f, 0.f, 0.f, 0.f}, rd[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t pk[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float a = ex2_approx(fmaf(__uint_as_float(sr[2 * e]), sl2, -mb));
          const float b = ex2_approx(fmaf(__uint_as_float(sr[2 * e + 1]), sl2, -mb));
          pk[e] = Tr::put(a, b);
          const float2 w = Tr::get(pk[e]);
          ex[(2 * e) & 3] += a;
          ex[(2 * e + 1) & 3] += b;
          rd[(2 * e) & 3] += w.x;
          rd[(2 * e + 1) & 3] += w.y;
        }
        l_exact += (ex[0] + ex[1]) + (ex[2] + ex[3]);
        l_run += (rd[0] + rd[1]) + (rd[2] + rd[3]);
        tmem_st32(tT, pk);
        if (i > 1 && __any_sync(0xffffffffu, need)) {
          if (!WIDE_WAIT(&sm.o_full[t][(c - 1) & 1], ((c - 1) >> 1) & 1)) {
            tmem_st_wait();
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < DP / 32; ++k) {
            uint32_t o[32];
            tmem_ld32(tO + 128 * t + 32 * k, o);
            tmem_ld_wait_regs32(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(tO + 128 * t + 32 * k, o);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[t][c & 1]);
      }
      if (!ok) break;
      // ---- the tile's output, or this piece's share of it: both streams' outputs, half of the columns ----
      float ms[2] = {-INFINITY, -INFINITY}, ls[2] = {0.f, 0.f}, le[2] = {0.f, 0.f}, w[2], sum = 0.f, se = 0.f;
      if (x.steps > 0) {
        auto& stats = sm.stats[pieces & 1];
        stats[t][0][r] = m_run;
        stats[t][1][r] = l_run;
        stats[t][2][r] = l_exact;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.stats_full);
        if (!WIDE_WAIT(&sm.stats_full, pieces & 1)) break;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          ms[k] = stats[k][0][r];
          ls[k] = stats[k][1][r];
          le[k] = stats[k][2][r];
        }
        // the last product of each stream, and with it those before
        n[0] += units[0];
        n[1] += units[1];
        for (int k = 0; ok && k < 2; ++k)
          if (units[k] > 0) ok = WIDE_WAIT(&sm.o_full[k][(n[k] - 1) & 1], ((n[k] - 1) >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        ++pieces;
      }
      const float mm = fmaxf(ms[0], ms[1]);
      const float top = mm * sl2;   // -inf: no key seen
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        w[k] = ms[k] == -INFINITY ? 0.f : ex2_approx((ms[k] - mm) * sl2);
        sum += w[k] * ls[k];
        se += w[k] * le[k];
      }
      const int part = part_of_piece(x);
      const float inv = x.whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
      const float w0 = w[0] * inv, w1 = w[1] * inv;
      DT* dst = static_cast<DT*>(p.out) + at;
      float* pdst = p.part_o + (long long)part * kWideRows * DP + r * 4;
#pragma unroll
      for (int k = 0; k < DP / 64; ++k) {
        const int col = t * (DP / 2) + 32 * k;
        float f[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) f[e] = 0.f;
        if (x.steps > 0) {
          uint32_t o[32];
          tmem_ld32(tO + col, o);
          tmem_ld_wait_regs32(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) f[e] = w0 == 0.f ? 0.f : w0 * __uint_as_float(o[e]);
          if (units[1] > 0) {
            tmem_ld32(tO + 128 + col, o);
            tmem_ld_wait_regs32(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] += w1 == 0.f ? 0.f : w1 * __uint_as_float(o[e]);
          }
        }
        if (valid) {
          if (x.whole) {
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              if (col + e < p.d) *reinterpret_cast<uint4*>(dst + col + e) = pack8<DT>(f + e);
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4*>(pdst + ((col + e) / 4) * (kWideRows * 4)) =
                  make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
          }
        }
      }
      if (x.steps > 0) {   // the outputs are read before the next piece's products write over them
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.o_free);
      }
      if (valid && t == 0) {
        if (x.whole) {
          if (p.lse)
            p.lse[(long long)hq * p.T + x.s.q_start + tok] =
                se == 0.f ? -INFINITY : top * 0.69314718055994531f + logf(se);
        } else {
          float* pm = p.part_m + (long long)part * 3 * kWideRows;
          pm[r] = top;
          pm[kWideRows + r] = sum;
          pm[2 * kWideRows + r] = se;
        }
      }
      if (tid == 0) note_split(p, x, share);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 10) {
    tc_fence_after();
    tmem_dealloc(tmem, kWideTmemCols);
  }
}

}  // namespace
}  // namespace thd
