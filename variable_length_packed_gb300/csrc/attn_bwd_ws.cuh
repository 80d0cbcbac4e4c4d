// attn_bwd_ws.cuh — the backward pass under a window with first keys that stay visible (p.sinks), warps
// specialised.  The mathematics, the items and the shared sums are attn_bwd.cuh's; the kernel there, which the
// calls without such keys keep, takes a step's parts one after another (3.9 us for 128 x 128 scores, of which
// the tensor pipe works 1.3 for heads of 128).  Here they overlap.  A step is 128 keys and kBQ queries of one head:
//
//   warp 0       scheduler and loads: K and V of an item, Q, dO and their row statistics of a step
//   warp 1       the products, in the order S(g+1) | dP(g+1), dV(g), dQ(g), dK(g): the elementwise
//                work on step g+1 runs while the last four do
//   warps 4-11   P^T and dS^T: four warps for each half of the queries, a thread a key; at an
//                item's end dK and dV
//   warps 12-15  dQ out of tensor memory into the fp32 accumulator
//
// S^T = K Q^T and dP^T = V dO^T have the keys on the lanes of tensor memory.  P^T goes back there, dS^T to
// shared memory, where dK += dS^T Q reads it by keys and the product for dQ by queries.
// Heads of 128: kBQ = 64 and dQ^T = K^T dS, a lane a value of the head: a warp's atomics are 128 bytes
// one after another.  Heads of 64: kBQ = 128 and dQ = dS K, a lane a query, out through shared memory
// by bulk reductions.  Tensor memory: dK, dV, S, dP, dQ and P, 480 and 512 columns of 512.
// Measured: 65536 rows of 64 sequences, 32 + 8 heads of 128, windows of 511: 1.74 ms of a call's 2.39 (0.39 row sums
// and zeros before it, 0.25 the conversion of dQ behind it), against 2.5 on the kernel of attn_bwd.cuh.  The tensor pipe is busy
// 42 % of the time.  Products of 64 columns read 6 KB of shared memory in the 32 cycles they take, so a
// step's operands, copies and dS^T are some 1900 cycles of it, and the 8.8 GB that are added to the accumulator pass at 5 TB/s.
// 65536 rows of one sequence, 16 + 4 heads of 64, fp16, window 1023: 1.04 of 1.20 ms (2.09 before).  Left: dQ of
// heads of 64 by 16 bytes a lane (1.83 ms) or by whole rows out of shared memory (1.48), a register split by setmaxnreg
// (more spills: heads of 64 store 88 bytes a thread in 128 registers and read 120 back, heads of 128 none).
#pragma once
#include "attn_bwd.cuh"

namespace thd {

constexpr int kBwsThreads = 512;
template <int DP> struct BwsShape {
  static constexpr int kBQ = DP == 128 ? 64 : 128;   // queries of a step
  static constexpr int kQ = 3;                       // steps whose Q and dO are in shared memory
  static constexpr int kDS = DP == 128 ? 2 : 1;      // and whose dS^T is
};

// An item as the producer hands it to the other warps.
struct BwsItem {
  int valid;
  int b, g, kv0, qblock, far;
  int t0, t1;      // query tiles of kBQ rows; a step for each and each query head of the group
  int shared;      // the sums of the first keys are added up by the post kernel
  SeqInfo s;
};

template <int DP>
struct BwsSmem {
  static constexpr int kBQ = BwsShape<DP>::kBQ, kQ = BwsShape<DP>::kQ, kDS = BwsShape<DP>::kDS;
  static constexpr int kKvBytes = kTileM * DP * 2, kQBytes = kBQ * DP * 2, kDsBytes = kTileM * kBQ * 2;
  alignas(1024) uint8_t k[kKvBytes];
  alignas(1024) uint8_t v[kKvBytes];
  alignas(1024) uint8_t q[kQ][kQBytes];
  alignas(1024) uint8_t dout[kQ][kQBytes];
  alignas(1024) uint8_t ds[kDS][kDsBytes];
  alignas(1024) uint8_t stage[DP == 64 ? kBQ * DP * 4 : 16];   // dQ on its way out (heads of 64)
  alignas(16) float lse2[kQ][kBQ], dd[kQ][kBQ];   // negative: -LSE * log2(e), -D of the step's queries
  uint64_t item_full[2], item_empty[2], k_full, v_full, k_empty, v_empty, q_full[kQ], q_empty[kQ];
  uint64_t s_full, s_empty, dp_full, ps_full, dv_done, ds_empty[kDS], dq_full, dq_empty, acc_full, acc_empty, drain;
  uint32_t tmem_base, abort;
  BwsItem items[2];
  SchedSmem sched;
};
static_assert(sizeof(BwsSmem<64>) + 1024 <= 227 * 1024 && sizeof(BwsSmem<128>) + 1024 <= 227 * 1024,
              "shared memory of the backward kernel");

#define BWS_WAIT(bar, parity) \
  mbar_wait((bar), (parity), abort_flag, p.status, THD_WAIT_TIMEOUT_BIT, p.wait_limit_ns, p.wait_check_mask)
#define BWS_WAIT_WARP(bar, parity) (__all_sync(0xffffffffu, BWS_WAIT((bar), (parity)) ? 1 : 0) != 0)

// One full warp: the next item of the CTA.
template <int DP>
__device__ BwsItem bws_next_item(SchedSmem& sched, const AttnParams& p, Claimer& claimer) {
  constexpr int kBQ = BwsShape<DP>::kBQ;
  const unsigned long long w = claim_item(claimer, p);
  const WorkItem it = sched_decode<kTileM, true>(sched, p, w);
  BwsItem x;
  x.valid = it.valid;
  if (!it.valid) return x;
  const SeqInfo& s = it.seq;
  x.s = s;
  x.b = it.b;
  x.g = it.h;
  x.qblock = it.qblock;
  x.kv0 = it.qblock * kTileM;
  x.far = it.far;
  const bool has_sinks = x.kv0 < p.sinks;
  const int sink_hi = s.causal ? 0 : kNoBound;
  const int all = (s.q_len + kBQ - 1) / kBQ;
  // queries that see a key of the tile: from first_q to last_q (attn_bwd.cuh)
  const long long first_q = (long long)x.kv0 - s.shift - (has_sinks ? sink_hi : s.hi_off);
  const long long last_q = (long long)x.kv0 + kTileM - 1 - s.shift + s.lo_off;
  x.t0 = first_q <= 0 ? 0 : (int)min(first_q / kBQ, (long long)all);
  x.t1 = last_q < 0 ? 0 : (int)min((long long)all, last_q / kBQ + 1);
  x.shared = 0;
  if (has_sinks) {
    constexpr int kPer = kTileM / kBQ;   // far items are cut at tiles of 128 queries
    const int near = near_query_tiles(s, x.kv0), tiles = (s.q_len + kTileM - 1) / kTileM;
    x.shared = p.far_tiles > 0 && near < tiles;
    if (it.far >= 0) {
      x.t0 = max(near, it.far * p.far_tiles) * kPer;
      x.t1 = min(all, (it.far + 1) * p.far_tiles * kPer);
    } else {
      x.t1 = x.shared ? near * kPer : all;
    }
  }
  x.t1 = max(x.t0, x.t1);
  return x;
}

// warp 0
template <int DP, bool kBF16>
__device__ void bws_producer(BwsSmem<DP>& sm, const BwdParams& bp, const CUtensorMap* tm_q, const CUtensorMap* tm_k,
                             const CUtensorMap* tm_v, const CUtensorMap* tm_do, volatile uint32_t* abort_flag) {
  constexpr int kBQ = BwsShape<DP>::kBQ, kQ = BwsShape<DP>::kQ, kPanels = DP / 64, kStats = kBQ / 32;
  constexpr int kKvPanel = kTileM * 128, kQPanel = kBQ * 128;
  constexpr float kLift = kBF16 ? 0.f : kBwdLift, kUnlift = kBF16 ? 1.f : kBwdUnlift;
  const AttnParams& p = bp.a;
  const int lane = threadIdx.x & 31;
  Claimer claimer{0ull, 0};
  uint32_t items = 0, kv = 0, n = 0;   // items, items with steps, steps
  bool ok = true;
  for (;;) {
    BwsItem x = bws_next_item<DP>(sm.sched, p, claimer);
    const int slot = items & 1;
    if (items >= 2) ok = BWS_WAIT_WARP(&sm.item_empty[slot], ((items >> 1) - 1) & 1);
    if (!ok) x.valid = 0;
    if (lane == 0) {
      sm.items[slot] = x;
      mbar_arrive(&sm.item_full[slot]);
    }
    ++items;
    if (!x.valid) break;
    const int tiles = x.t1 - x.t0;
    if (tiles == 0) continue;
    if (kv > 0) ok = BWS_WAIT_WARP(&sm.k_empty, (kv - 1) & 1) && BWS_WAIT_WARP(&sm.v_empty, (kv - 1) & 1);
    if (!ok) break;
    if (lane == 0) {
      mbar_arrive_expect_tx(&sm.k_full, BwsSmem<DP>::kKvBytes);
      mbar_arrive_expect_tx(&sm.v_full, BwsSmem<DP>::kKvBytes);
#pragma unroll
      for (int pn = 0; pn < kPanels; ++pn) {
        tma_load_2d(sm.k + pn * kKvPanel, tm_k, &sm.k_full, x.g * p.d + pn * 64, x.s.kv_start + x.kv0);
        tma_load_2d(sm.v + pn * kKvPanel, tm_v, &sm.v_full, x.g * p.d + pn * 64, x.s.kv_start + x.kv0);
      }
    }
    ++kv;
    // LSE * log2(e) and D of a step's rows (zero past the sequence), read a step ahead
    float l[kStats], dd[kStats];
    auto stats = [&](int h, int t) {
#pragma unroll
      for (int e = 0; e < kStats; ++e) {
        const int row = t * kBQ + e * 32 + lane;
        l[e] = dd[e] = 0.f;
        if (row < x.s.q_len) {
          const size_t at = (size_t)h * p.T + x.s.q_start + row;
          l[e] = p.lse[at] * 1.4426950408889634f;
          dd[e] = bp.D[at];
        }
      }
    };
    const int steps = tiles * p.group;
    int h = x.g * p.group, t = x.t0;
    stats(h, t);
    for (int i = 0; i < steps; ++i, ++n) {
      const uint32_t st = n % kQ;
      float l_now[kStats], d_now[kStats];
#pragma unroll
      for (int e = 0; e < kStats; ++e) {
        l_now[e] = kLift - l[e];
        d_now[e] = -dd[e] * kUnlift;
      }
      const int h_now = h, t_now = t;
      if (++t == x.t1) {
        t = x.t0;
        ++h;
      }
      if (i + 1 < steps) stats(h, t);
      if (n >= (uint32_t)kQ) ok = BWS_WAIT_WARP(&sm.q_empty[st], (n / kQ - 1) & 1);
      if (!ok) break;
#pragma unroll
      for (int e = 0; e < kStats; ++e) {
        sm.lse2[st][e * 32 + lane] = l_now[e];
        sm.dd[st][e * 32 + lane] = d_now[e];
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_expect_tx(&sm.q_full[st], 2 * BwsSmem<DP>::kQBytes);
#pragma unroll
        for (int pn = 0; pn < kPanels; ++pn) {
          tma_load_2d(sm.q[st] + pn * kQPanel, tm_q, &sm.q_full[st], h_now * p.d + pn * 64, x.s.q_start + t_now * kBQ);
          tma_load_2d(sm.dout[st] + pn * kQPanel, tm_do, &sm.q_full[st], h_now * p.d + pn * 64, x.s.q_start + t_now * kBQ);
        }
      }
    }
    if (!ok) break;
  }
  // copies still in flight land before the CTA can exit
  if (kv > 0) {
    drain_wait(&sm.k_full, (kv - 1) & 1);
    drain_wait(&sm.v_full, (kv - 1) & 1);
  }
  for (uint32_t c = n > (uint32_t)kQ ? n - kQ : 0; c < n; ++c) drain_wait(&sm.q_full[c % kQ], (c / kQ) & 1);
}

// warp 1
template <typename DT, int DP>
__device__ void bws_mma(BwsSmem<DP>& sm, const BwdParams& bp, uint32_t tmem, volatile uint32_t* abort_flag) {
  using Tr = DTypeTraits<DT>;
  constexpr int kBQ = BwsShape<DP>::kBQ, kQ = BwsShape<DP>::kQ, kDS = BwsShape<DP>::kDS;
  constexpr int kKvPanel = kTileM * 128, kQPanel = kBQ * 128;
  constexpr uint32_t idesc_s = umma_idesc_f16(Tr::kBF16, kTileM, kBQ, false);          // S^T, dP^T
  constexpr uint32_t idesc_acc = umma_idesc_f16(Tr::kBF16, kTileM, DP, true);          // dV, dK
  constexpr uint32_t idesc_dq = DP == 128 ? umma_idesc_f16_ab(Tr::kBF16, DP, kBQ, true, true)     // dQ^T = K^T dS
                                          : umma_idesc_f16_ab(Tr::kBF16, kBQ, DP, true, true);    // dQ = dS K
  constexpr uint32_t hi = smem_desc_sw128_hi(1024);
  const AttnParams& p = bp.a;
  const uint32_t tDK = tmem, tDV = tmem + DP, tS = tmem + 2 * DP, tDP = tS + kBQ, tDQ = tDP + kBQ, tP = tDQ + 64;
  const uint32_t k_K = smem_desc_sw128_lo(smem_u32(sm.k), 16), k_MN = smem_desc_sw128_lo(smem_u32(sm.k), kKvPanel);
  const uint32_t v_K = smem_desc_sw128_lo(smem_u32(sm.v), 16);
  const bool leader = elect_one_sync();
  uint32_t items = 0, kv = 0, g = 0;

  // K steps of 16 values of the head: 32 bytes inside a 128-byte row, panels of 64 values
  auto off_kv = [](int kk) { return (uint32_t)(((kk >> 2) * kKvPanel + (kk & 3) * 32) >> 4); };
  auto off_q = [](int kk) { return (uint32_t)(((kk >> 2) * kQPanel + (kk & 3) * 32) >> 4); };
  auto issue_s = [&](uint32_t n) {
    const uint32_t q_K = smem_desc_sw128_lo(smem_u32(sm.q[n % kQ]), 16);
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk)
      umma_ss_if(leader, tS, smem_desc_join(k_K + off_kv(kk), hi), smem_desc_join(q_K + off_q(kk), hi), idesc_s, kk > 0 ? 1u : 0u);
    umma_commit_if(leader, &sm.s_full);
  };
  auto issue_dp = [&](uint32_t n) {
    const uint32_t o_K = smem_desc_sw128_lo(smem_u32(sm.dout[n % kQ]), 16);
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk)
      umma_ss_if(leader, tDP, smem_desc_join(v_K + off_kv(kk), hi), smem_desc_join(o_K + off_q(kk), hi), idesc_s, kk > 0 ? 1u : 0u);
    umma_commit_if(leader, &sm.dp_full);
  };

  bool ok = true;
  while (ok) {
    const int slot = items & 1;
    if (!BWS_WAIT_WARP(&sm.item_full[slot], (items >> 1) & 1)) break;
    const int valid = sm.items[slot].valid, steps = valid ? (sm.items[slot].t1 - sm.items[slot].t0) * p.group : 0;
    __syncwarp();
    if (leader) mbar_arrive(&sm.item_empty[slot]);
    ++items;
    if (!valid) break;
    if (steps == 0) continue;
    ok = BWS_WAIT_WARP(&sm.k_full, kv & 1) && BWS_WAIT_WARP(&sm.v_full, kv & 1);
    for (int i = 0; ok && i < steps; ++i, ++g) {
      if (i == 0) {
        ok = BWS_WAIT_WARP(&sm.q_full[g % kQ], (g / kQ) & 1) && (g == 0 || BWS_WAIT_WARP(&sm.s_empty, (g - 1) & 1));
        if (!ok) break;
        tc_fence_after();
        issue_s(g);
        issue_dp(g);   // dP of the step before was read before its P came
      }
      if (i + 1 < steps) {
        ok = BWS_WAIT_WARP(&sm.q_full[(g + 1) % kQ], ((g + 1) / kQ) & 1) && BWS_WAIT_WARP(&sm.s_empty, g & 1);
        if (!ok) break;
        tc_fence_after();
        issue_s(g + 1);
      }
      ok = BWS_WAIT_WARP(&sm.ps_full, g & 1);
      if (!ok) break;
      tc_fence_after();
      if (i + 1 < steps) issue_dp(g + 1);
      if (i == 0 && kv > 0) {   // dK and dV of the item before are written
        ok = BWS_WAIT_WARP(&sm.acc_empty, (kv - 1) & 1);
        if (!ok) break;
        tc_fence_after();
      }
      const uint32_t st = g % kQ, buf = g % kDS;
      const uint32_t q_MN = smem_desc_sw128_lo(smem_u32(sm.q[st]), kQPanel);
      const uint32_t o_MN = smem_desc_sw128_lo(smem_u32(sm.dout[st]), kQPanel);
      // dS^T: rows of keys, panels of 64 queries
      const uint32_t ds_K = smem_desc_sw128_lo(smem_u32(sm.ds[buf]), 16);
      const uint32_t ds_MN = smem_desc_sw128_lo(smem_u32(sm.ds[buf]), kTileM * 128);
#pragma unroll
      for (int kk = 0; kk < kBQ / 16; ++kk)   // 16 queries a step: 8 columns of packed P, 16 rows of dO
        umma_ts_if(leader, tDV, tP + 8 * kk, smem_desc_join(o_MN + kk * 128, hi), idesc_acc, (i > 0 || kk > 0) ? 1u : 0u);
      umma_commit_if(leader, &sm.dv_done);
      if (g > 0) {
        ok = BWS_WAIT_WARP(&sm.dq_empty, (g - 1) & 1);
        if (!ok) break;
        tc_fence_after();
      }
#pragma unroll
      for (int kk = 0; kk < kTileM / 16; ++kk) {   // 16 keys a step: 16 rows of K and of dS^T
        if (DP == 128)
          umma_ss_if(leader, tDQ, smem_desc_join(k_MN + kk * 128, hi), smem_desc_join(ds_MN + kk * 128, hi), idesc_dq, kk > 0 ? 1u : 0u);
        else
          umma_ss_if(leader, tDQ, smem_desc_join(ds_MN + kk * 128, hi), smem_desc_join(k_MN + kk * 128, hi), idesc_dq, kk > 0 ? 1u : 0u);
      }
      umma_commit_if(leader, &sm.dq_full);
#pragma unroll
      for (int kk = 0; kk < kBQ / 16; ++kk)
        umma_ss_if(leader, tDK, smem_desc_join(ds_K + (((kk >> 2) * (kTileM * 128) + (kk & 3) * 32) >> 4), hi),
                   smem_desc_join(q_MN + kk * 128, hi), idesc_acc, (i > 0 || kk > 0) ? 1u : 0u);
      umma_commit_if(leader, &sm.q_empty[st]);
      umma_commit_if(leader, &sm.ds_empty[buf]);
      if (i == steps - 1) {
        umma_commit_if(leader, &sm.k_empty);
        umma_commit_if(leader, &sm.v_empty);
        umma_commit_if(leader, &sm.acc_full);
      }
    }
    ++kv;
  }
  // every MMA issued so far completes before TMEM is released
  umma_commit_if(leader, &sm.drain);
  drain_wait(&sm.drain, 0);
}

// warps 4-11: half 0 (warps 4-7) the first kBQ / 2 queries of a step, half 1 the others
template <typename DT, int DP>
__device__ void bws_elementwise(BwsSmem<DP>& sm, const BwdParams& bp, uint32_t tmem, int half, volatile uint32_t* abort_flag) {
  using Tr = DTypeTraits<DT>;
  constexpr int kBQ = BwsShape<DP>::kBQ, kQ = BwsShape<DP>::kQ, kDS = BwsShape<DP>::kDS, kCols = kBQ / 2;
  constexpr float kUnlift = Tr::kBF16 ? 1.f : kBwdUnlift;
  const AttnParams& p = bp.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = 32 * (warp & 3) + lane;   // key of the tile, lane of tensor memory
  const uint32_t t_lane = (uint32_t)(32 * (warp & 3)) << 16;
  const uint32_t tDK = tmem + t_lane, tDV = tDK + DP, tS = tDK + 2 * DP, tDP = tS + kBQ, tP = tDP + kBQ + 64;
  const float2 scale2 = make_float2(p.scale_log2, p.scale_log2), unlift2 = make_float2(kUnlift, kUnlift);
  uint32_t items = 0, kv = 0, g = 0;
  for (;;) {
    const int slot = items & 1;
    if (!BWS_WAIT_WARP(&sm.item_full[slot], (items >> 1) & 1)) break;
    const BwsItem x = sm.items[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.item_empty[slot]);
    ++items;
    if (!x.valid) break;
    const SeqInfo& s = x.s;
    const int key = x.kv0 + row;
    const bool kvalid = key < s.kv_len, sink = key < p.sinks;
    const int tiles = x.t1 - x.t0, steps = tiles * p.group;
    // query i sees the key iff lo_q <= i <= hi_q (attn_bwd.cuh)
    const long long at = (long long)key - s.shift;
    const long long lo_q = at - (sink ? (s.causal ? 0 : kNoBound) : s.hi_off), hi_q = at + (sink ? kNoBound : s.lo_off);
    bool ok = true;
    int t = x.t0;
    for (int i = 0; i < steps; ++i, ++g) {
      const int q0 = t * kBQ + half * kCols;   // first query of this half
      if (++t == x.t1) t = x.t0;
      const uint32_t st = g % kQ, buf = g % kDS;
      if (!BWS_WAIT_WARP(&sm.q_full[st], (g / kQ) & 1) || !BWS_WAIT_WARP(&sm.s_full, g & 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float pv[kCols];
#pragma unroll
      for (int c0 = 0; c0 < kCols; c0 += 32) {
        tmem_ld32(tS + half * kCols + c0, reinterpret_cast<uint32_t*>(pv) + c0);
        tmem_ld_wait_regs32(reinterpret_cast<uint32_t*>(pv) + c0);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.s_empty);
      // columns [c_lo, c_hi] of this half see the key
      const int c_lo = (int)min(max(lo_q - q0, -1ll), (long long)kCols);
      const int c_hi = kvalid ? (int)max(min(hi_q - q0, (long long)min(s.q_len - q0, kCols) - 1), -1ll) : -1;
      const float* lse2 = sm.lse2[st] + half * kCols;
      const float* dd = sm.dd[st] + half * kCols;
#pragma unroll
      for (int c = 0; c < kCols; c += 4) {
        const float4 l = *reinterpret_cast<const float4*>(lse2 + c);
        const float2 a = __ffma2_rn(make_float2(pv[c], pv[c + 1]), scale2, make_float2(l.x, l.y));
        const float2 b = __ffma2_rn(make_float2(pv[c + 2], pv[c + 3]), scale2, make_float2(l.z, l.w));
        pv[c] = ex2_approx(a.x);
        pv[c + 1] = ex2_approx(a.y);
        pv[c + 2] = ex2_approx(b.x);
        pv[c + 3] = ex2_approx(b.y);
      }
      if (!__all_sync(0xffffffffu, c_lo <= 0 && c_hi >= kCols - 1)) {
#pragma unroll
        for (int w = 0; w < kCols / 32; ++w) {
          const uint32_t seen = low_bits(c_hi + 1 - 32 * w) & ~low_bits(c_lo - 32 * w);
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (!(seen >> c & 1)) pv[32 * w + c] = 0.f;
        }
      }
      // Where a half is 64 queries, P^T goes out first: its values and dS^T's together are more than a thread's
      // registers.  Else both wait until they are ready, and only then for the products of the step before.
      constexpr bool kEarly = kCols > 32;
      auto put_p = [&]() {
        if (g > 0 && !BWS_WAIT_WARP(&sm.dv_done, (g - 1) & 1)) return false;
        tc_fence_after();
#pragma unroll
        for (int c0 = 0; c0 < kCols; c0 += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) pk[e] = Tr::pack2(pv[c0 + 2 * e], pv[c0 + 2 * e + 1]);
          tmem_st16(tP + (half * kCols + c0) / 2, pk);
        }
        return true;
      };
      ok = (!kEarly || put_p()) && BWS_WAIT_WARP(&sm.dp_full, g & 1);
      if (kEarly && ok && g >= (uint32_t)kDS) ok = BWS_WAIT_WARP(&sm.ds_empty[buf], (g / kDS - 1) & 1);
      if (!ok) {
        tmem_st_wait();   // stores above complete before TMEM can be released
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int c0 = 0; c0 < kCols; c0 += 32) {
        uint32_t dr[32], pd[16];
        tmem_ld32(tDP + half * kCols + c0, dr);
        tmem_ld_wait_regs32(dr);
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 d = *reinterpret_cast<const float4*>(dd + c0 + e);
          const float2 p0 = make_float2(pv[c0 + e], pv[c0 + e + 1]), p1 = make_float2(pv[c0 + e + 2], pv[c0 + e + 3]);
          const float2 w0 = make_float2(__uint_as_float(dr[e]), __uint_as_float(dr[e + 1]));
          const float2 w1 = make_float2(__uint_as_float(dr[e + 2]), __uint_as_float(dr[e + 3]));
          const float2 d0 = make_float2(d.x, d.y), d1 = make_float2(d.z, d.w);
          const float2 v0 = __fmul2_rn(p0, Tr::kBF16 ? __fadd2_rn(w0, d0) : __ffma2_rn(w0, unlift2, d0));
          const float2 v1 = __fmul2_rn(p1, Tr::kBF16 ? __fadd2_rn(w1, d1) : __ffma2_rn(w1, unlift2, d1));
          pd[e / 2] = Tr::pack2(v0.x, v0.y);
          pd[e / 2 + 1] = Tr::pack2(v1.x, v1.y);
        }
        if (!kEarly) {
          ok = put_p() && (g < (uint32_t)kDS || BWS_WAIT_WARP(&sm.ds_empty[buf], (g / kDS - 1) & 1));
          if (!ok) break;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int chunk = (half * kCols + c0) / 8 + e;   // 16 bytes: 8 queries
          *reinterpret_cast<uint4*>(sm.ds[buf] + sw128_offset(row, chunk)) =
              make_uint4(pd[4 * e], pd[4 * e + 1], pd[4 * e + 2], pd[4 * e + 3]);
        }
      }
      if (!ok) {
        tmem_st_wait();
        break;
      }
      tmem_st_wait();
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.ps_full);
        mbar_arrive(&sm.q_empty[st]);
      }
    }
    if (!ok) break;

    // ---- dK, dV of the tile (each half of the warps a half of the columns) ----
    const bool any = steps > 0;
    if (any) {
      if (!BWS_WAIT_WARP(&sm.acc_full, kv & 1)) break;
      ++kv;
      tc_fence_after();
    }
    const bool far = x.far >= 0;
    const bool to_sums = x.shared && key < min(p.sinks, s.kv_len), row_ok = kvalid && !to_sums && !far;
    if (any || !far) {   // a chunk of queries that are all near the tile has nothing to add
      const long long place = far ? far_slot(s, x.b, x.far) : (long long)x.b;
      float* sums = nullptr;
      if (to_sums)
        sums = (far ? bp.far_sums : bp.near_sums) +
               ((place * p.Hkv + x.g) * bp.far_key_tiles + x.qblock) * (2ll * bp.far_rows * p.d) + (long long)row * p.d;
      const size_t base = ((size_t)(s.kv_start + (row_ok ? key : 0)) * p.Hkv + x.g) * (size_t)p.d;
#pragma unroll
      for (int cc = 0; cc < DP / 64; ++cc) {
        const int c = (half * (DP / 64) + cc) * 32;
#pragma unroll
        for (int which = 0; which < 2; ++which) {   // dK, dV
          uint32_t a[32];
          if (any) {
            tmem_ld32((which ? tDV : tDK) + c, a);
            tmem_ld_wait_regs32(a);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) a[e] = 0u;
          }
          const float scale = which ? kUnlift : p.scale;
          if (row_ok) {
            DT* dst = static_cast<DT*>(which ? bp.dv : bp.dk) + base + c;
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint4 w;
              w.x = Tr::pack2(__uint_as_float(a[e]) * scale, __uint_as_float(a[e + 1]) * scale);
              w.y = Tr::pack2(__uint_as_float(a[e + 2]) * scale, __uint_as_float(a[e + 3]) * scale);
              w.z = Tr::pack2(__uint_as_float(a[e + 4]) * scale, __uint_as_float(a[e + 5]) * scale);
              w.w = Tr::pack2(__uint_as_float(a[e + 6]) * scale, __uint_as_float(a[e + 7]) * scale);
              *reinterpret_cast<uint4*>(dst + e) = w;
            }
          } else if (to_sums) {
            const float raw = which ? kUnlift : 1.f;
            float* dst = sums + (which ? (long long)bp.far_rows * p.d : 0ll) + c;
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4*>(dst + e) =
                  make_float4(__uint_as_float(a[e]) * raw, __uint_as_float(a[e + 1]) * raw, __uint_as_float(a[e + 2]) * raw,
                              __uint_as_float(a[e + 3]) * raw);
          }
        }
      }
    }
    if (any) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.acc_empty);
    }
  }
}

// warps 12-15: dQ of each step into the accumulator
template <int DP>
__device__ void bws_drain(BwsSmem<DP>& sm, const BwdParams& bp, uint32_t tmem, const CUtensorMap* tm_dq,
                          volatile uint32_t* abort_flag) {
  constexpr int kBQ = BwsShape<DP>::kBQ;
  const AttnParams& p = bp.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = 32 * (warp & 3) + lane;   // heads of 128: a value of the head; heads of 64: a query
  const uint32_t tDQ = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 2 * DP + 2 * kBQ;
  const size_t stride = (size_t)p.Hq * p.d;
  uint32_t items = 0, g = 0;
  // Heads of 64: the four warps meet at a barrier, so they leave together when a wait gave up for one of them.
  auto agreed = [&](bool mine) {
    if (DP != 64) return mine;
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "bar.red.and.pred p, 1, 128, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(all)
        : "r"(mine ? 1u : 0u)
        : "memory");
    return all != 0u;
  };
  bool ok = true;
  while (ok) {
    const int slot = items & 1;
    if (!agreed(BWS_WAIT_WARP(&sm.item_full[slot], (items >> 1) & 1))) break;
    const int valid = sm.items[slot].valid, t0 = sm.items[slot].t0, t1 = sm.items[slot].t1, kvh = sm.items[slot].g;
    const int q_start = sm.items[slot].s.q_start, q_len = sm.items[slot].s.q_len;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.item_empty[slot]);
    ++items;
    if (!valid) break;
    for (int h = kvh * p.group; ok && h < (kvh + 1) * p.group; ++h) {
      for (int t = t0; t < t1; ++t, ++g) {
        if (DP == 64 && threadIdx.x == 12 * 32) bulk_wait_group_read0();   // the step before's is read
        if (!agreed(BWS_WAIT_WARP(&sm.dq_full, g & 1))) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t o[64];
        tmem_ld32(tDQ, o);
        tmem_ld32(tDQ + 32, o + 32);
        tmem_ld_wait_regs32(o);
        tmem_tie_regs32(o + 32);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.dq_empty);
        const int q0 = t * kBQ, rows = min(kBQ, q_len - q0);
        if constexpr (DP == 128) {
          float* dst = bp.dacc + (size_t)(q_start + q0) * stride + (size_t)h * p.d + row;
          if (rows == kBQ) {
#pragma unroll
            for (int c = 0; c < kBQ; ++c) atomicAdd(dst + c * stride, __uint_as_float(o[c]));
          } else {
#pragma unroll
            for (int c = 0; c < kBQ; ++c)
              if (c < rows) atomicAdd(dst + c * stride, __uint_as_float(o[c]));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            *reinterpret_cast<uint4*>(sm.stage + (e >> 3) * (kBQ * 128) + row * 128 + (((e & 7) ^ (row & 7)) << 4)) =
                make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          fence_proxy_async_smem();
          asm volatile("bar.sync 1, 128;" ::: "memory");
          if (threadIdx.x == 12 * 32) {
            // rows past the sequence carry dS = 0, so their (zero) rows add nothing
            tma_reduce_add_2d(tm_dq, sm.stage, h * p.d, q_start + q0);
            tma_reduce_add_2d(tm_dq, sm.stage + kBQ * 128, h * p.d + 32, q_start + q0);
            bulk_commit_group();
          }
        }
      }
    }
  }
  if (DP == 64 && threadIdx.x == 12 * 32) bulk_wait_group0();
}

template <typename DT, int DP>
__global__ void __launch_bounds__(kBwsThreads, 1)
    attn_bwd_ws_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                       const __grid_constant__ CUtensorMap tm_dq, const BwdParams bp) {
  const AttnParams& p = bp.a;
  extern __shared__ uint8_t smem_raw[];
  BwsSmem<DP>& sm = *reinterpret_cast<BwsSmem<DP>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.item_full[i], 1);
      mbar_init(&sm.item_empty[i], 13);   // the MMA warp, eight elementwise ones, four of dQ
    }
    for (uint64_t* b : {&sm.k_full, &sm.v_full, &sm.k_empty, &sm.v_empty, &sm.s_full, &sm.dp_full, &sm.dv_done, &sm.dq_full,
                        &sm.acc_full, &sm.drain})
      mbar_init(b, 1);
    for (int i = 0; i < BwsShape<DP>::kQ; ++i) {
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.q_empty[i], 9);   // the products and the eight elementwise warps
    }
    for (int i = 0; i < BwsShape<DP>::kDS; ++i) mbar_init(&sm.ds_empty[i], 1);
    mbar_init(&sm.s_empty, 8);
    mbar_init(&sm.ps_full, 8);
    mbar_init(&sm.acc_empty, 8);
    mbar_init(&sm.dq_empty, 4);
    fence_mbar_init();
    sm.abort = 0;
    sched_init(sm.sched);
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_do);
    if (DP == 64) tma_prefetch_desc(&tm_dq);
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile uint32_t* abort_flag = &sm.abort;
  if (warp == 0) {
    bws_producer<DP, DTypeTraits<DT>::kBF16>(sm, bp, &tm_q, &tm_k, &tm_v, &tm_do, abort_flag);
  } else if (warp == 1) {
    bws_mma<DT, DP>(sm, bp, tmem, abort_flag);
  } else if (warp == 3) {
    // test setting: a wait that runs out while the pipeline runs (the drain barrier completes only at the end)
    if (p.inject_wait) inject_wait_timeout_warp(p, &sm.drain, abort_flag);
  } else if (warp >= 12) {
    bws_drain<DP>(sm, bp, tmem, &tm_dq, abort_flag);
  } else if (warp >= 4) {
    bws_elementwise<DT, DP>(sm, bp, tmem, (warp >> 2) - 1, abort_flag);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

#undef BWS_WAIT
#undef BWS_WAIT_WARP

}  // namespace thd
