// attn_paged_weights_wide.cuh — the weights that cached keys got from more than 16 rows each: chunks of new
// tokens and trees, on the fifth-generation tensor cores.
//
// A CTA takes 256 keys of a head at a time and all rows that see some of them, in tiles of 128:
// S^T = K Q^T with the keys on the lanes of tensor memory, so that a thread adds up its own key's
// weights exp2(s scale - lse) in a register and nothing crosses lanes, the sum has one order, and each
// weight is written once.  Inside a CTA:
//   warps 0-1   keys: 16-byte asynchronous copies out of the pages into the swizzled layout
//   warp 2      query tiles by tensor copies (a box of the group's heads of some tokens), and their log-sum-exps
//   warp 3      issues the products, two score tiles for each half of the keys
//   warps 4-7, 8-11  the exponentials of the first and second 128 keys
// What bounds it: a tile of 128 x 128 scores takes 512 cycles of the tensor pipe and as many of the
// exponential unit; 256 keys a query tile keep its 32 KB from the L2 below the rate of the packed
// forward kernel.  Measured, 1024 new tokens of 4 sequences over 60000 keys, 32 + 8 heads of 128: 0.50 ms, 1.0 PFLOP/s,
// the tensor pipe busy 40 % of the time: a scheduler has two warps of exponentials, whose steps wait for one another.
#pragma once
#include "attn_paged_weights.cuh"

namespace thd {

bool encode_group_map(CUtensorMap* map, const void* base, int T, int heads, int d, int heads_box, int tokens_box, bool bf16);

namespace {

constexpr int kWwThreads = 384;
constexpr int kWwKeys = 256;     // keys of an item
constexpr int kWwRows = 128;     // rows of a query tile at most: whole tokens
constexpr int kWwStats = 4;      // query tiles whose log-sum-exps are in shared memory: more than tiles, so that a tile's
                                 // place is free as soon as its products are done
template <int DP> struct WwDepth { static constexpr int kK = DP == 64 ? 3 : 2, kQ = DP == 64 ? 4 : 2; };

template <int DP>
struct WwSmem {
  static constexpr int kTileBytes = 128 * DP * 2;
  static constexpr int kK = WwDepth<DP>::kK, kQ = WwDepth<DP>::kQ;
  alignas(1024) uint8_t k[kK][2][kTileBytes];
  alignas(1024) uint8_t q[kQ][kTileBytes];
  alignas(16) float lse[kWwStats][kWwRows];   // -log2(e) * log-sum-exp of the tile's rows
  uint64_t k_full[kK], k_empty[kK], q_full[kQ], q_empty[kQ], l_full[kWwStats], l_empty[kWwStats], s_full[2][2], s_empty[2][2], drain, never;
  uint32_t tmem_base, abort;
  Share share;
};
static_assert(sizeof(WwSmem<128>) + 1024 <= 227 * 1024 && sizeof(WwSmem<64>) + 1024 <= 227 * 1024, "shared memory");

// 256 keys of a head, and the query tiles [tile0, tile1) whose rows see some of them (none: nothing to do).
struct WwItem {
  SeqWork s;
  int seq, head, key0, past, tile0, tile1;
};

// Items of a sequence's head; unsigned, as the last one may end at 2^31.
__device__ __forceinline__ int ww_items(int kv_len) { return (int)(((uint32_t)kv_len + kWwKeys - 1) / kWwKeys); }

// The items of a CTA's share, in order; an item costs its sequence's query tiles, and 2 for its keys.
template <bool kWin>
struct WwWalk {
  long long u, end, base;
  int b, tokens;   // tokens of a query tile

  __device__ __forceinline__ WwWalk(const Share& share, int tokens_)
      : u(share.begin), end(share.end), base(share.seq_base), b(share.seq), tokens(tokens_) {}

  __device__ static __forceinline__ long long cost(const SeqWork& s, int tokens) { return 2ll + (s.q_len + tokens - 1) / tokens; }
  __device__ static __forceinline__ long long items(const PagedArgs& p, const SeqWork& s) {
    return s.q_len > 0 ? (long long)p.Hkv * ww_items(s.kv_len) : 0ll;
  }

  __device__ __forceinline__ bool next(const PagedArgs& p, WwItem& x) {
    while (u < end) {
      x.s = seq_work<false>(p, b, kWwRows);
      const long long per = cost(x.s, tokens), n = items(p, x.s);
      const long long item = quotient(u - base + per - 1, per);   // the first that begins in the share
      if (item >= n) {
        base += n * per;
        u = max(u, base);
        ++b;
        continue;
      }
      u = base + item * per;
      if (u >= end) return false;
      u += per;
      const int blocks = ww_items(x.s.kv_len);
      x.seq = b;
      x.head = (int)quotient(item, blocks);
      x.key0 = (int)(item - (long long)x.head * blocks) * kWwKeys;
      x.past = x.s.kv_len - x.s.q_len;
      int tok0 = 0, tok1 = x.s.q_len;
      if (!p.tree) {
        tok0 = max(0, x.key0 - x.past);
        if (kWin && x.key0 >= p.sinks)
          tok1 = (int)max(0ll, min((long long)tok1, (long long)x.key0 + kWwKeys - x.past + p.win_left));
      }
      x.tile0 = tok0 / tokens;
      x.tile1 = tok1 > tok0 ? (tok1 + tokens - 1) / tokens : x.tile0;
      return true;
    }
    return false;
  }
};

#define WW_WAIT(bar, parity)                                                                                   \
  (__all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.call_status, THD_STATUS_WAIT_TIMEOUT,          \
                                     p.wait_limit_ns, p.wait_check_mask) ? 1 : 0) != 0)

template <typename DT, int DP, bool kWin>
__global__ void __launch_bounds__(kWwThreads, 1)
    attn_key_weights_wide_kernel(const __grid_constant__ CUtensorMap tm_q, const PagedArgs p, const int tokens) {
  using Tr = Pair16<DT>;
  constexpr int kK = WwSmem<DP>::kK, kQ = WwSmem<DP>::kQ, kPanels = DP / 64, kChunks = DP / 8;
  constexpr uint32_t idesc = umma_idesc_f16(Tr::kBF16, 128, kWwRows, false);
  extern __shared__ uint8_t smem_raw[];
  WwSmem<DP>& sm = *reinterpret_cast<WwSmem<DP>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                  ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile uint32_t* abort_flag = &sm.abort;
  if (tid == 0) {
    for (int i = 0; i < kK; ++i) {
      mbar_init(&sm.k_full[i], 2);    // one lane of each loading warp
      mbar_init(&sm.k_empty[i], 1);   // the products that read the stage
    }
    for (int i = 0; i < kQ; ++i) {
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.q_empty[i], 1);   // the products
    }
    for (int i = 0; i < kWwStats; ++i) {
      mbar_init(&sm.l_full[i], 1);
      mbar_init(&sm.l_empty[i], 8);   // the warps that read them
    }
    for (int i = 0; i < 2; ++i)
      for (int j = 0; j < 2; ++j) {
        mbar_init(&sm.s_full[i][j], 1);
        mbar_init(&sm.s_empty[i][j], 4);
      }
    mbar_init(&sm.drain, 1);
    mbar_init(&sm.never, 1);
    fence_mbar_init();
    sm.abort = 0u;
    tma_prefetch_desc(&tm_q);
  }
  if (warp == 3) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  find_share<kWwThreads>(
      p,
      [&](int b) {
        const SeqWork s = seq_work<false>(p, b, kWwRows);
        return WwWalk<kWin>::items(p, s) * WwWalk<kWin>::cost(s, tokens);
      },
      &sm.share);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  WwWalk<kWin> walk(sm.share, tokens);
  WwItem x;

  if (warp < 2) {
    // ---------------------------------------------------------------- keys
    constexpr int kLaneKeys = 32 / kChunks;
    const int copy_key = lane / kChunks, copy_chunk = lane % kChunks;
    const bool copy_in = copy_chunk * 8 < p.d;
    uint32_t n = 0, told = 0;   // items issued, items announced
    bool ok = true;
    auto announce = [&]() {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.k_full[told % kK]);
      ++told;
    };
    while (ok && walk.next(p, x)) {
      if (x.tile1 <= x.tile0) continue;
      const uint32_t st = n % kK, par = (n / kK - 1) & 1;
      if (n >= (uint32_t)kK) {
        // a stage that is not free yet: what is on the way is announced first
        const bool ready = __shfl_sync(0xffffffffu, mbar_test_wait(&sm.k_empty[st], par) ? 1 : 0, 0) != 0;
        if (!ready && told < n) {
          cp_async_wait<0>();
          announce();
        }
        if (!WW_WAIT(&sm.k_empty[st], par)) {
          ok = false;
          break;
        }
      }
      const int32_t* table = p.table + (long long)x.seq * p.table_stride;
      const uint32_t kt = smem_u32(sm.k[st][warp]);
#pragma unroll 1
      for (int r0 = 0; r0 < 128; r0 += 32) {
        const int first = x.key0 + warp * 128 + r0;
        long long off = -1;   // of this lane's key; -1: not read
        const int key = first + lane;
        if (key < x.s.kv_len && (!kWin || key < p.sinks || key >= window_first(p, x.past, 0))) {
          const int at = key / p.page_size, page = table[at];
          if (page >= 0 && page < p.num_pages)
            off = page * p.k_page + (key - at * p.page_size) * p.k_token + x.head * p.k_head;
        }
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          const int key_in = c * kLaneKeys + copy_key, row = r0 + key_in;
          const long long o = __shfl_sync(0xffffffffu, off, key_in);
          const bool take = copy_in && o >= 0;
          cp_async16(kt + (copy_chunk >> 3) * 16384 + row * 128 + (((copy_chunk & 7) ^ (row & 7)) << 4),
                     static_cast<const DT*>(p.kc) + (take ? o + copy_chunk * 8 : 0), take);
        }
      }
      cp_async_commit();
      ++n;
      if (n - told > 1) {
        cp_async_wait<1>();
        announce();
      }
    }
    cp_async_wait<0>();
    if (told < n) announce();
  } else if (warp == 2) {
    // ---------------------------------------------------------------- queries
    uint32_t n = 0;   // query tiles issued
    bool ok = true;
    const uint32_t bytes = (uint32_t)(kPanels * 128 * tokens * p.group);
    // the token and the head of this lane's columns
    int tok_of[kWwRows / 32], head_of[kWwRows / 32];
#pragma unroll
    for (int i = 0; i < kWwRows / 32; ++i) {
      tok_of[i] = (i * 32 + lane) / p.group;
      head_of[i] = i * 32 + lane - tok_of[i] * p.group;
    }
    float l[kWwRows / 32];
    auto stats = [&](int t) {   // read a tile ahead
#pragma unroll
      for (int i = 0; i < kWwRows / 32; ++i) {
        const int tok = t * tokens + tok_of[i];
        l[i] = tok_of[i] < tokens && tok < x.s.q_len
                   ? -1.4426950408889634f * p.lse[(long long)(x.head * p.group + head_of[i]) * p.T + x.s.q_start + tok]
                   : 0.f;
      }
    };
    while (ok && walk.next(p, x)) {
      if (x.tile1 > x.tile0) stats(x.tile0);
      for (int t = x.tile0; t < x.tile1; ++t, ++n) {
        const uint32_t st = n % kQ, ls = n % kWwStats;
        float now[kWwRows / 32];
#pragma unroll
        for (int i = 0; i < kWwRows / 32; ++i) now[i] = l[i];
        if (t + 1 < x.tile1) stats(t + 1);
        if (n >= (uint32_t)kQ && !WW_WAIT(&sm.q_empty[st], (n / kQ - 1) & 1)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(&sm.q_full[st], bytes);
#pragma unroll
          for (int pn = 0; pn < kPanels; ++pn)
            tma_load_3d(sm.q[st] + pn * 16384, &tm_q, &sm.q_full[st], pn * 64, x.head * p.group, x.s.q_start + t * tokens);
        }
        if (n >= (uint32_t)kWwStats && !WW_WAIT(&sm.l_empty[ls], (n / kWwStats - 1) & 1)) {
          ok = false;
          ++n;   // its copy is on the way
          break;
        }
#pragma unroll
        for (int i = 0; i < kWwRows / 32; ++i)   // a row that sees no key: its scores are all masked, by -inf
          sm.lse[ls][i * 32 + lane] = now[i] == INFINITY ? 0.f : now[i];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.l_full[ls]);
      }
    }
    // copies in flight land before the CTA can exit
    for (uint32_t c = n > (uint32_t)kQ ? n - kQ : 0; c < n; ++c) drain_wait(&sm.q_full[c % kQ], (c / kQ) & 1);
  } else if (warp == 3) {
    // ---------------------------------------------------------------- products
    const bool issue = elect_one_sync();
    constexpr uint32_t hi = smem_desc_sw128_hi(1024);
    uint32_t n = 0, nq = 0, ns[2] = {0, 0};   // items, query tiles, score tiles of each half
    bool ok = true;
    if (p.inject_wait) ok = WW_WAIT(&sm.never, 0);   // test setting: a wait that runs out, loads in flight
    while (ok && walk.next(p, x)) {
      if (x.tile1 <= x.tile0) continue;
      const uint32_t st = n % kK;
      if (!WW_WAIT(&sm.k_full[st], (n / kK) & 1)) break;
      ++n;
      const int halves = x.s.kv_len - x.key0 > 128 ? 2 : 1;
      for (int t = x.tile0; t < x.tile1; ++t, ++nq) {
        const uint32_t qs = nq % kQ;
        if (!WW_WAIT(&sm.q_full[qs], (nq / kQ) & 1)) {
          ok = false;
          break;
        }
        const uint32_t q_lo = smem_desc_sw128_lo(smem_u32(sm.q[qs]), 16);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h >= halves) break;
          const uint32_t buf = ns[h] & 1;
          if (ns[h] >= 2 && !WW_WAIT(&sm.s_empty[h][buf], (ns[h] / 2 - 1) & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t k_lo = smem_desc_sw128_lo(smem_u32(sm.k[st][h]), 16);
#pragma unroll
          for (int kk = 0; kk < DP / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
            umma_ss_if(issue, tmem + (h * 2 + buf) * 128, smem_desc_join(k_lo + off, hi), smem_desc_join(q_lo + off, hi),
                       idesc, kk > 0 ? 1u : 0u);
          }
          umma_commit_if(issue, &sm.s_full[h][buf]);
          ++ns[h];
        }
        if (!ok) break;
        umma_commit_if(issue, &sm.q_empty[qs]);
      }
      if (!ok) break;
      umma_commit_if(issue, &sm.k_empty[st]);
    }
    // what was issued completes before tensor memory is released
    umma_commit_if(issue, &sm.drain);
    drain_wait(&sm.drain, 0);
  } else {
    // ---------------------------------------------------------------- exponentials
    const int h = (warp >> 2) - 1, row = tid & 127;
    const uint32_t tS = tmem + h * 256 + ((uint32_t)((warp & 3) * 32) << 16);
    const float2 scale2 = make_float2(p.scale_log2, p.scale_log2);
    uint32_t nq = 0, ns = 0;
    bool ok = true;
    while (ok && walk.next(p, x)) {
      const bool mine = h == 0 || x.s.kv_len - x.key0 > 128;   // this half has keys
      const int key = x.key0 + h * 128 + row;
      const bool real = key < x.s.kv_len;
      const bool kept_visible = kWin && key < p.sinks;
      float2 sum[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] = make_float2(0.f, 0.f);
      for (int t = x.tile0; t < x.tile1; ++t, ++nq) {
        const uint32_t ls = nq % kWwStats;
        if (!WW_WAIT(&sm.l_full[ls], (nq / kWwStats) & 1)) {
          ok = false;
          break;
        }
        if (mine) {
          const uint32_t buf = ns & 1;
          if (!WW_WAIT(&sm.s_full[h][buf], (ns / 2) & 1)) {
            ok = false;
            break;
          }
          ++ns;
          tc_fence_after();
          // the columns whose rows see the key: [lo, end)
          const int tok0 = t * tokens;
          const int rows = min(tokens, x.s.q_len - tok0) * p.group;
          int lo = 0, end = real ? rows : 0;
          if (!p.tree) {
            lo = max(0, min(key - x.past - tok0, tokens)) * p.group;
            if (kWin && !kept_visible)
              end = (int)min((long long)end, max(0ll, (long long)key - x.past + p.win_left - tok0 + 1) * p.group);
          }
          const bool by_bits = p.tree && real && key >= x.past;
          const bool whole = __all_sync(0xffffffffu, lo == 0 && end == kWwRows && !by_bits);
#pragma unroll
          for (int c0 = 0; c0 < kWwRows; c0 += 64) {   // all 128 at once: 80 bytes of spills, 9 % slower
            uint32_t s[64];
            tmem_ld32(tS + buf * 128 + c0, s);
            tmem_ld32(tS + buf * 128 + c0 + 32, s + 32);
            tmem_ld_wait_regs32(s);
            tmem_tie_regs32(s + 32);
            if (c0 + 64 == kWwRows) {   // the scores are read
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&sm.s_empty[h][buf]);
            }
            if (!whole) {
#pragma unroll
              for (int w = 0; w < 2; ++w) {
                uint32_t seen = low_bits(end - c0 - 32 * w) & ~low_bits(lo - c0 - 32 * w);
                if (by_bits) {
                  const int j = key - x.past, at = j >> 6;
                  for (int c = 0; c < 32; ++c) {
                    const int tok = tok0 + (c0 + 32 * w + c) / p.group;
                    if ((seen >> c & 1) &&
                        !(at < p.tree_words &&
                          ((uint64_t)p.tree[(long long)(x.s.q_start + tok) * p.tree_words + at] >> (j & 63) & 1)))
                      seen &= ~(1u << c);
                  }
                }
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  if (!(seen >> c & 1)) s[32 * w + c] = __float_as_uint(-INFINITY);
              }
            }
            const float4* lse = reinterpret_cast<const float4*>(&sm.lse[ls][c0]);
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const float4 l = lse[c];
              const float2 a = __ffma2_rn(make_float2(__uint_as_float(s[4 * c]), __uint_as_float(s[4 * c + 1])), scale2,
                                          make_float2(l.x, l.y));
              const float2 b = __ffma2_rn(make_float2(__uint_as_float(s[4 * c + 2]), __uint_as_float(s[4 * c + 3])), scale2,
                                          make_float2(l.z, l.w));
              sum[(2 * c) & 3] = __fadd2_rn(sum[(2 * c) & 3], make_float2(ex2_approx(a.x), ex2_approx(a.y)));
              sum[(2 * c + 1) & 3] = __fadd2_rn(sum[(2 * c + 1) & 3], make_float2(ex2_approx(b.x), ex2_approx(b.y)));
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.l_empty[ls]);
      }
      if (!ok) break;
      // keys that no token sees are left alone: their pages may be another sequence's by now
      if (real && x.tile1 > x.tile0 && (!kWin || kept_visible || key >= window_first(p, x.past, 0))) {
        const int at = key / p.page_size, page = p.table[(long long)x.seq * p.table_stride + at];
        if (page >= 0 && page < p.num_pages) {
          const float2 a = __fadd2_rn(__fadd2_rn(sum[0], sum[1]), __fadd2_rn(sum[2], sum[3]));
          float* w = p.key_weights + page * p.w_page + (key - at * p.page_size) * p.w_token + x.head * p.w_head;
          *w = key >= x.past ? a.x + a.y : *w + (a.x + a.y);   // a new token's key had none before
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

#undef WW_WAIT

}  // namespace
}  // namespace thd
