// attn_paged_wide.cuh — attention over a paged cache for tiles of 128 query rows, on the
// fifth-generation tensor cores: chunks of new tokens and trees of drafted ones, where more
// than 16 rows share a key/value head.
//
// The same split of the batch's keys over the CTAs as the narrow kernel's (attn_paged.cu); inside a CTA
// the work is divided among warps:
//   warps 0-3  softmax, one thread per row: queries into tensor memory, scores out of it, weights
//              back over them, the running maximum and sums, the output at the end
//   warps 4-5  loads: 32 keys of each unit, 16-byte asynchronous copies out of the pages into
//              the swizzled layout of the matrix unit (any page size, order and stride)
//   warp 6     issues the matrix products: S = Q K^T (Q from tensor memory), O += P V
// What bounds it: with up to 128 rows for each key the unit's 32 KB take about 1400 cycles to
// come from memory on an SM, its two products 512 cycles of the tensor pipe and its softmax 1000 to
// 1500.  A CTA runs S, softmax, P V of a unit one after another; two CTAs per SM (half of the
// tensor memory and shared memory each) overlap one another's.  Queries in tensor memory leave
// shared memory for three units of keys and values.
// Measured (16 sequences, 27 drafted tokens of 32 + 8 heads of 128): each further 120000 keys take 73 us,
// 6.7 TB/s; 120000 keys 94 us, the rest being the start (17 us for 2000 keys: finding the share,
// first use of code, tables and pages one after another).  Measured and left: one CTA per SM with two
// softmax streams, two score tiles for each and the queries in shared memory took 107 us with
// keys and values by tensor copies of whole boxes of a page (16 tokens by 64 columns), 153 us with two
// warps copying rows; with the keys in the L2 it was slower too (78 against 60 us for 54 drafted tokens over
// 24000 keys).  Two CTAs leave a thread 128 registers; heads of 128 spill 8 to 16 bytes, under a
// window 20 to 24 (36 to 96 read back), heads of 64 there 8.
// Heads of 64 (68 us at 64 rows, where memory asks 37): a second score tile in the room they leave, twice the
// units on the way, and pages read a unit ahead changed nothing.
//
// Under a window (kWin) the loading warps bounded it while they looked up keys and values apart: 512 tokens of 8
// sequences over windows of 1023, 190 us, and 137 with one place for both.  Several tiles of many heads over a cache larger than
// the L2 are under way at once and read it again from memory: 1024 tokens of 4 sequences over 60000 keys, 0.99 ms and
// 5.6 GB read where the cache is 0.25.  Measured and left: two, three or four waves of shares, which keep a wave's keys in
// the L2 (0.97 ms there, but 166, 189 and 211 us against 137 on the windows); a second score tile with the queries in shared memory and two
// units on the way (194 us, and 1200 against 876 on 12500 keys of 8 sequences).
//
// Every wait is bounded as in the other attention kernels: one that runs out sets the CTA's
// status word, and the CTA lets what it started finish and leaves.
#pragma once
#include <type_traits>

#include "attn_paged_common.cuh"

namespace thd {
namespace {

constexpr int kWideRows = 128;
constexpr int kWideThreads = 224;   // seven warps: two CTAs leave a thread 128 registers
constexpr int kWideLoaders = 2;     // loading warps
constexpr int kWideStages = 3;
constexpr float kWideLag = 8.f;           // log2 by which weights may pass 1 before the maximum moves
constexpr float kWideLift = 7.f;          // as kNarrowLift (attn_paged.cu): fp16 weights stay below 2^(8 + 7)
constexpr uint32_t kWideTmemCols = 256;   // S and P [0, 64), Q [64, 128), O [128, 128 + DP)

template <int DP>
struct WideSmem {
  static constexpr int kTileBytes = kUnit * DP * 2;   // panels of 64 rows x 128 bytes
  alignas(1024) uint8_t k[kWideStages][kTileBytes];
  alignas(1024) uint8_t v[kWideStages][kTileBytes];
  uint64_t full[kWideStages], empty[kWideStages], q_full, s_full, p_full, o_full, drain, never;
  uint32_t tmem_base, abort;
  Share share;
};

// Waits of a whole warp, which leaves them together.
#define WIDE_WAIT(bar, parity)                                                                                     \
  (__all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, &p.status[blockIdx.x], THD_STATUS_WAIT_TIMEOUT,      \
                                     p.wait_limit_ns, p.wait_check_mask) ? 1 : 0) != 0)

template <typename DT, int DP, bool kWin>
__global__ void __launch_bounds__(kWideThreads, 2) attn_paged_wide_kernel(const PagedArgs p) {
  using Tr = Pair16<DT>;
  constexpr int kChunks = DP / 8;
  constexpr int kPanelBytes = kUnit * 128;
  constexpr float kLift = Tr::kBF16 ? 0.f : kWideLift, kUnlift = Tr::kBF16 ? 1.f : 0x1p-7f;
  constexpr uint32_t idesc_qk = umma_idesc_f16(Tr::kBF16, kWideRows, kUnit, false);
  constexpr uint32_t idesc_pv = umma_idesc_f16(Tr::kBF16, kWideRows, DP, true);
  extern __shared__ uint8_t smem_raw[];
  WideSmem<DP>& sm = *reinterpret_cast<WideSmem<DP>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                      ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile uint32_t* abort_flag = &sm.abort;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    for (int i = 0; i < kWideStages; ++i) {
      mbar_init(&sm.full[i], kWideLoaders);   // one lane of each loading warp
      mbar_init(&sm.empty[i], 1);   // the products that read the stage
    }
    mbar_init(&sm.q_full, 4);
    mbar_init(&sm.s_full, 1);
    mbar_init(&sm.p_full, 4);
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.drain, 1);
    mbar_init(&sm.never, 1);
    fence_mbar_init();
    sm.abort = 0u;
    p.splits[blockIdx.x].n = 0;
    p.status[blockIdx.x] = 0u;
  }
  if (warp == 6) {
    tmem_alloc(&sm.tmem_base, kWideTmemCols);
    tmem_relinquish();
  }
  find_share<kWideThreads>(p, [&](int b) { return seq_work<kWin>(p, b, kWideRows).units; }, &sm.share);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const Share share = sm.share;
  PieceWalk walk(share);
  Piece x;

  if (warp >= 4 && warp < 6) {
    // ---------------------------------------------------------------- loads
    constexpr int kWarpKeys = kUnit / kWideLoaders;
    constexpr int kLaneKeys = 32 / kChunks, kCopies = kWarpKeys / kLaneKeys;
    const int copy_key = lane / kChunks, copy_chunk = lane % kChunks;
    const bool copy_in = copy_chunk * 8 < p.d;
    uint32_t n = 0;   // units issued
    bool ok = true;
    // announces unit i, whose copies have landed
    auto announce = [&](uint32_t i) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.full[i % kWideStages]);
    };
    while (ok && walk.next<kWideRows, kWin>(p, x)) {
      const int32_t* table = p.table + (long long)x.seq * p.table_stride;
      for (int i = 0; i < x.steps; ++i, ++n) {
        const int first = unit_of<kWin>(x, x.blk0 + i) * kUnit + (warp - 4) * kWarpKeys;
        // each lane the place of one key and of its value
        const long long koff = cache_offset<kWin>(p, x, table, first + lane, false);
        const long long voff = p.same_places ? koff : cache_offset<kWin>(p, x, table, first + lane, true);
        const uint32_t st = n % kWideStages;
        if (n >= kWideStages && !WIDE_WAIT(&sm.empty[st], (n / kWideStages - 1) & 1)) {
          ok = false;
          break;
        }
        const uint32_t kt = smem_u32(sm.k[st]), vt = smem_u32(sm.v[st]);
        auto copy = [&](auto same) {
#pragma unroll
          for (int c = 0; c < kCopies; ++c) {
            const int key = c * kLaneKeys + copy_key, row = (warp - 4) * kWarpKeys + key;
            const uint32_t at = (copy_chunk >> 3) * kPanelBytes + row * 128 + (((copy_chunk & 7) ^ (row & 7)) << 4);
            const long long ko = __shfl_sync(0xffffffffu, koff, key);
            const long long vo = decltype(same)::value ? ko : __shfl_sync(0xffffffffu, voff, key);
            const bool take = copy_in && ko >= 0;
            const int col = copy_chunk * 8;
            cp_async16(kt + at, static_cast<const DT*>(p.kc) + (take ? ko + col : 0), take);
            cp_async16(vt + at, static_cast<const DT*>(p.vc) + (take ? vo + col : 0), take);
          }
        };
        if (p.same_places) copy(std::true_type{}); else copy(std::false_type{});
        cp_async_commit();
        if (n > 0) {
          cp_async_wait<1>();
          announce(n - 1);
        }
      }
    }
    cp_async_wait<0>();
    if (n > 0) announce(n - 1);
  } else if (warp == 6) {
    // ---------------------------------------------------------------- products
    const bool issue = elect_one_sync();
    uint32_t n = 0, pieces = 0;   // units, pieces
    bool ok = true;
    const uint32_t khi = smem_desc_sw128_hi(1024);
    if (p.inject_wait) ok = WIDE_WAIT(&sm.never, 0);   // test setting: a wait that runs out, loads in flight
    while (ok && walk.next<kWideRows, kWin>(p, x)) {
      if (x.steps == 0) continue;
      if (!WIDE_WAIT(&sm.q_full, pieces & 1)) break;
      ++pieces;
      for (int i = 0; i < x.steps; ++i, ++n) {
        const uint32_t st = n % kWideStages;
        if (!WIDE_WAIT(&sm.full[st], (n / kWideStages) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t klo = smem_desc_sw128_lo(smem_u32(sm.k[st]), 16);
        const uint32_t vlo = smem_desc_sw128_lo(smem_u32(sm.v[st]), kPanelBytes);
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk)
          umma_ts_if(issue, tmem, tmem + 64 + kk * 8,
                     smem_desc_join(klo + (((kk >> 2) * kPanelBytes + (kk & 3) * 32) >> 4), khi), idesc_qk,
                     kk > 0 ? 1u : 0u);
        umma_commit_if(issue, &sm.s_full);
        if (!WIDE_WAIT(&sm.p_full, n & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kUnit / 16; ++kk)
          umma_ts_if(issue, tmem + 128, tmem + kk * 8, smem_desc_join(vlo + ((kk * 16 * 128) >> 4), khi), idesc_pv,
                     (i > 0 || kk > 0) ? 1u : 0u);
        umma_commit_if(issue, &sm.empty[st]);
        umma_commit_if(issue, &sm.o_full);
      }
    }
    // what was issued completes before tensor memory is released
    umma_commit_if(issue, &sm.drain);
    drain_wait(&sm.drain, 0);
  } else {
    // ---------------------------------------------------------------- softmax
    const uint32_t t_lane = (uint32_t)(warp * 32) << 16;
    const uint32_t tS = tmem + t_lane, tQ = tS + 64, tO = tS + 128;
    const int r = tid;   // row of the tile, lane of tensor memory
    const float sl2 = p.scale_log2;
    uint32_t n = 0;      // units
    bool ok = true;
    while (ok && walk.next<kWideRows, kWin>(p, x)) {
      const int row = x.row0 + r, tok = row / p.group, hq = x.head * p.group + (row - tok * p.group);
      const bool valid = r < x.rows;
      // a warp past the tile's rows only keeps step: what its lanes of tensor memory hold reaches no row
      const bool idle = warp * 32 >= x.rows;
      const uint64_t word0 = tree_word(p, x, valid ? tok : 0);
      float m_run = -INFINITY, l_run = 0.f, l_exact = 0.f;
      if (x.steps > 0 && !idle) {
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const DT*>(p.q) + ((long long)(x.s.q_start + (valid ? tok : 0)) * p.Hq + (valid ? hq : 0)) * p.d);
#pragma unroll
        for (int c = 0; c < DP / 32; ++c) {
          uint32_t qv[16];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint4 w = make_uint4(0u, 0u, 0u, 0u);
            if (valid && (c * 4 + e) * 8 < p.d) w = src[c * 4 + e];
            qv[4 * e] = w.x, qv[4 * e + 1] = w.y, qv[4 * e + 2] = w.z, qv[4 * e + 3] = w.w;
          }
          tmem_st16(tQ + 16 * c, qv);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
      }
      if (x.steps > 0 && lane == 0) mbar_arrive(&sm.q_full);
      for (int i = 0; i < x.steps; ++i, ++n) {
        if (!WIDE_WAIT(&sm.s_full, n & 1)) {
          ok = false;
          break;
        }
        if (idle) {
          if (lane == 0) mbar_arrive(&sm.p_full);
          continue;
        }
        tc_fence_after();
        uint32_t sr[64];
        tmem_ld32(tS, sr);
        tmem_ld32(tS + 32, sr + 32);
        tmem_ld_wait_regs32(sr);
        tmem_tie_regs32(sr + 32);
        const int first = unit_of<kWin>(x, x.blk0 + i) * kUnit;
        if (unit_cut<kWin>(p, x, first)) {
          const uint64_t seen = valid ? seen_keys<kWin>(p, x, tok, first, word0) : 0ull;
          const uint32_t lo = (uint32_t)seen, hi = (uint32_t)(seen >> 32);
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            if (!(lo >> c & 1)) sr[c] = __float_as_uint(-INFINITY);
            if (!(hi >> c & 1)) sr[32 + c] = __float_as_uint(-INFINITY);
          }
        }
        float mx[4] = {m_run, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 64; c += 8) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mx[k] = fmax3f(mx[k], __uint_as_float(sr[c + 2 * k]), __uint_as_float(sr[c + 2 * k + 1]));
        }
        const float m_new = fmax3f(fmaxf(mx[0], mx[1]), mx[2], mx[3]);
        // the maximum moves only when it grows by more than kWideLag: the output is seldom rescaled
        const bool need = (m_new - m_run) * sl2 > kWideLag;   // false while both are -inf
        float alpha = 1.f;
        if (need) {
          alpha = ex2_approx((m_run - m_new) * sl2);
          m_run = m_new;
          l_run *= alpha;
          l_exact *= alpha;
        }
        const float mb = (m_run == -INFINITY ? 0.f : m_run) * sl2 - kLift;
        // sums of the weights and of the weights as rounded, in two chains of pairs each
        const float2 scale2 = make_float2(sl2, sl2), bias2 = make_float2(-mb, -mb);
        float2 ex[2], rd[2];
        ex[0] = ex[1] = rd[0] = rd[1] = make_float2(0.f, 0.f);
        uint32_t pk[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const float2 e =
              __ffma2_rn(make_float2(__uint_as_float(sr[2 * c]), __uint_as_float(sr[2 * c + 1])), scale2, bias2);
          const float2 w = make_float2(ex2_approx(e.x), ex2_approx(e.y));
          pk[c] = Tr::put(w.x, w.y);
          ex[c & 1] = __fadd2_rn(ex[c & 1], w);
          Tr::add(pk[c], rd[c & 1].x, rd[c & 1].y);
        }
        l_exact += (ex[0].x + ex[0].y) + (ex[1].x + ex[1].y);
        l_run += (rd[0].x + rd[0].y) + (rd[1].x + rd[1].y);
        tmem_st32(tS, pk);
        if (i > 0 && __any_sync(0xffffffffu, need)) {
          if (!WIDE_WAIT(&sm.o_full, (n - 1) & 1)) {
            tmem_st_wait();
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < DP / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * c, o);
            tmem_ld_wait_regs32(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(tO + 32 * c, o);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full);
      }
      if (!ok) break;
      if (idle) continue;
      // ---- the tile's output, or this piece's share of it ----
      if (x.steps > 0) {
        if (!WIDE_WAIT(&sm.o_full, (n - 1) & 1)) break;
        tc_fence_after();
      }
      const float top = m_run * sl2;   // -inf: no key seen
      const int part = part_of_piece(x);
      const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
      DT* dst = static_cast<DT*>(p.out) + ((long long)(x.s.q_start + (valid ? tok : 0)) * p.Hq + (valid ? hq : 0)) * p.d;
      float* pdst = p.part_o + (long long)part * kWideRows * DP + r * 4;
#pragma unroll
      for (int c = 0; c < DP / 32; ++c) {
        uint32_t o[32];
        if (x.steps > 0) {
          tmem_ld32(tO + 32 * c, o);
          tmem_ld_wait_regs32(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        if (valid) {
          if (x.whole) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              float f[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) f[k] = l_run == 0.f ? 0.f : __uint_as_float(o[e + k]) * inv;
              if (32 * c + e < p.d) *reinterpret_cast<uint4*>(dst + 32 * c + e) = pack8<DT>(f);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4*>(pdst + (8 * c + e / 4) * (kWideRows * 4)) =
                  make_float4(__uint_as_float(o[e]) * kUnlift, __uint_as_float(o[e + 1]) * kUnlift,
                              __uint_as_float(o[e + 2]) * kUnlift, __uint_as_float(o[e + 3]) * kUnlift);
          }
        }
      }
      tc_fence_before();   // the output is read before the next piece's products write over it
      if (valid) {
        if (x.whole) {
          if (p.lse)
            p.lse[(long long)hq * p.T + x.s.q_start + tok] =
                l_exact == 0.f ? -INFINITY : top * 0.69314718055994531f + logf(l_exact * kUnlift);
        } else {
          float* pm = p.part_m + (long long)part * 3 * kWideRows;
          pm[r] = top;
          pm[kWideRows + r] = l_run * kUnlift;
          pm[2 * kWideRows + r] = l_exact * kUnlift;
        }
      }
      if (tid == 0) note_split(p, x, share);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 6) {
    tc_fence_after();
    tmem_dealloc(tmem, kWideTmemCols);
  }
}

}  // namespace
}  // namespace thd
