// attn_paged_weights.cuh — the weight that each cached key got from the new tokens, added up beside the
// cache: w_j (+)= sum over the new tokens and the query heads of the group of exp(scale q.k_j - lse).
//
// The log-sum-exps are those that the attention before it wrote, so this pass needs the scores once more,
// not the values.  Of narrow tiles (decoding steps) the attention keeps them, 4 bytes a row and key where reading the
// key again is 2 d: here they only become weights.  Where they do not fit the workspace the products are taken
// again, by this kernel for a few rows, by the one of 128 rows for more.  Measured, 500000 keys of 64 sequences,
// 32 + 8 heads of 128, one token each: 380 us with the attention (310 without the weights), 42 of them this pass; with
// the products taken again 705.
#pragma once
#include "attn_paged_common.cuh"

namespace thd {
namespace {

constexpr int kWeightWarps = 4;   // 16 keys of a unit each

// Whether new token `tok` sees key `key` (both of the sequence, key < kv_len).
template <bool kWin>
__device__ __forceinline__ bool token_sees(const PagedArgs& p, const SeqWork& s, int tok, int key) {
  const int past = s.kv_len - s.q_len;
  if (p.tree) {
    const int j = key - past;
    if (j < 0) return true;
    const int at = j >> 6;
    return at < p.tree_words && ((uint64_t)p.tree[(long long)(s.q_start + tok) * p.tree_words + at] >> (j & 63) & 1);
  }
  const long long own = (long long)past + tok;
  return key <= own && (!kWin || key >= own - p.win_left || key < p.sinks);
}

// Units of a sequence's heads that have kept scores.
__device__ __forceinline__ long long score_units(const PagedArgs& p, const SeqWork& s) {
  return s.q_len > 0 ? (long long)p.Hkv * s.blocks : 0ll;
}

// From kept scores: a CTA takes a run of the units of all heads laid end to end, a warp every fourth of them, its
// lanes two keys each.
template <bool kWin>
__device__ void weights_of_scores(const PagedArgs& p, const Share& share, long long scores) {
  const int lane = threadIdx.x & 31;
  long long step = share.begin + (threadIdx.x >> 5), base = share.seq_base;
  for (int b = share.seq; step < share.end; ++b) {
    Piece x;
    x.s = seq_work<kWin>(p, b, kNarrowRows);
    const long long end = min(base + score_units(p, x.s), share.end);
    if (step < end) {
      x.row0 = 0;
      x.rows = x.s.q_len * p.group;
      const int last = piece_bounds<kWin>(p, x);
      const int32_t* table = p.table + (long long)b * p.table_stride;
      constexpr int kAhead = 4;   // units at once: a page, then a weight, then a sum each wait for the one before
      for (; step < end; step += kAhead * kWeightWarps) {
        float* place[kAhead][2];
        float had[kAhead][2];
        float2 sum[kAhead];
        const float2* src[kAhead];
        const float* lse[kAhead];
        int units = 0;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          place[k][0] = place[k][1] = nullptr;
          sum[k] = make_float2(0.f, 0.f);
          // a unit behind the last reads the first one's scores, and writes nothing
          const bool real = step + k * kWeightWarps < end;
          const int in = (int)((real ? step + k * kWeightWarps : step) - base), head = in / x.s.blocks, blk = in - head * x.s.blocks;
          src[k] = reinterpret_cast<const float2*>(p.scores + scores + (long long)in * x.rows * kUnit) + lane;
          lse[k] = p.lse + (long long)head * p.group * p.T + x.s.q_start;
          if (real && blk < last) {
            units = k + 1;
            const int key = unit_of<kWin>(x, blk) * kUnit + lane * 2;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int at_key = key + e;
              // a key that no token sees is left alone: its page may be another sequence's by now
              if (at_key < x.s.kv_len && (!kWin || at_key < p.sinks || at_key >= x.win_lo)) {
                const int at = p.page_shift >= 0 ? at_key >> p.page_shift : at_key / p.page_size, page = table[at];
                if (page >= 0 && page < p.num_pages)
                  place[k][e] = p.key_weights + page * p.w_page + (at_key - at * p.page_size) * p.w_token + head * p.w_head;
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e)   // a new token's key had none
            had[k][e] = place[k][e] && unit_of<kWin>(x, blk) * kUnit + lane * 2 + e < x.past ? *place[k][e] : 0.f;
        }
        if (units == 0) continue;
        for (int tok = 0, r = 0; tok < x.s.q_len; ++tok)
          for (int g = 0; g < p.group; ++g, ++r) {
            float2 s[kAhead];
            float l[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
              s[k] = src[k][r * (kUnit / 2)];
              l[k] = lse[k][(long long)g * p.T + tok];
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
              const float l2 = l[k] == -INFINITY ? 0.f : -1.4426950408889634f * l[k];   // such a row's scores are -inf
              sum[k].x += ex2_approx(s[k].x + l2);
              sum[k].y += ex2_approx(s[k].y + l2);
            }
          }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          if (place[k][0]) *place[k][0] = had[k][0] + sum[k].x;
          if (place[k][1]) *place[k][1] = had[k][1] + sum[k].y;
        }
      }
      // on with the first of this warp's units that was not taken
      step -= (step - end) / kWeightWarps * kWeightWarps;
    }
    base += score_units(p, x.s);
    scores += seq_scores(p, x.s);
  }
}

template <typename DT, int DP, bool kWin>
__global__ void __launch_bounds__(kWeightWarps * 32) attn_key_weights_kernel(const PagedArgs p) {
  constexpr int kKSteps = DP / 16;
  __shared__ Share share;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int qr = lane >> 2, qc = (lane & 3) * 2;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (p.scores) {
    find_share<kWeightWarps * 32>(p, [&](int b) { return score_units(p, seq_work<kWin>(p, b, kNarrowRows)); }, &share);
    const ScorePlaces at = score_places<kWeightWarps * 32, kWin>(p, share.seq);
    if (at.fit) {
      weights_of_scores<kWin>(p, share, at.base);
      return;
    }
  }
  // a unit of 64 keys of a head costs reading its keys and a step for every 8 rows
  auto cost = [&](const SeqWork& s) { return 2ll + (long long)s.q_len * p.group / 8; };
  auto whole = [&](int b) {
    SeqWork s = seq_work<false>(p, b, kNarrowRows);
    return (s.q_len > 0 ? (long long)p.Hkv * s.blocks : 0ll) * cost(s);
  };
  find_share<kWeightWarps * 32>(p, whole, &share);
  long long base = share.seq_base;
  int b = share.seq;
  for (long long u = share.begin; u < share.end;) {
    const SeqWork s = seq_work<false>(p, b, kNarrowRows);
    const long long per = cost(s), items = s.q_len > 0 ? (long long)p.Hkv * s.blocks : 0ll;
    const long long item = quotient(u - base + per - 1, per);   // the first unit that begins in the share
    if (item >= items) {
      base += items * per;
      u = max(u, base);
      ++b;
      continue;
    }
    u = base + item * per;
    if (u >= share.end) break;
    u += per;
    const int head = (int)quotient(item, s.blocks), blk = (int)(item - (long long)head * s.blocks);
    const int key0 = blk * kUnit + warp * 16, past = s.kv_len - s.q_len;
    const int32_t* table = p.table + (long long)b * p.table_stride;
    // ---- this warp's keys, and where their weights lie ----
    uint32_t kf[kKSteps][4];
    long long place[2];   // -1: no page
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      const int key = key0 + hh * 8 + qr;
      place[hh] = -1;
      const DT* src = static_cast<const DT*>(p.kc);
      // a key that no token sees is left alone: its page may be another sequence's by now
      bool ok = key < s.kv_len && (!kWin || key < p.sinks || key >= window_first(p, past, 0));
      if (ok) {
        const int at = key / p.page_size, page = table[at], in = key - at * p.page_size;
        ok = page >= 0 && page < p.num_pages;
        if (ok) {
          src += page * p.k_page + in * p.k_token + head * p.k_head;
          place[hh] = page * p.w_page + in * p.w_token + head * p.w_head;
        }
      }
#pragma unroll
      for (int k = 0; k < kKSteps; ++k)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int col = k * 16 + half * 8 + qc;
          kf[k][half * 2 + hh] = ok && col < p.d ? *reinterpret_cast<const uint32_t*>(src + col) : 0u;
        }
    }
    // ---- the rows that see some of them ----
    int tok0 = 0, tok1 = s.q_len;
    if (!p.tree) {
      tok0 = max(0, key0 - past);
      if (kWin && key0 >= p.sinks)
        tok1 = (int)max(0ll, min((long long)tok1, (long long)key0 + 16 - past + p.win_left));
    }
    float sum[2] = {0.f, 0.f};
    const int row_end = tok1 * p.group;
    for (int r0 = tok0 * p.group; r0 < row_end; r0 += 8) {
      float c[4] = {0.f, 0.f, 0.f, 0.f};
      {
        const int row = r0 + qr, tok = row / p.group;
        const bool ok = row < row_end;
        const DT* src = static_cast<const DT*>(p.q) +
                        ((long long)(s.q_start + (ok ? tok : 0)) * p.Hq + head * p.group + (ok ? row - tok * p.group : 0)) * p.d;
#pragma unroll
        for (int k = 0; k < kKSteps; ++k) {
          const int col = k * 16 + qc;
          const uint32_t b0 = ok && col < p.d ? *reinterpret_cast<const uint32_t*>(src + col) : 0u;
          const uint32_t b1 = ok && col + 8 < p.d ? *reinterpret_cast<const uint32_t*>(src + col + 8) : 0u;
          mma16816<DT>(c, kf[k], b0, b1);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = r0 + qc + e, tok = row / p.group;
        if (row >= row_end) continue;
        const float lse = p.lse[(long long)(head * p.group + row - tok * p.group) * p.T + s.q_start + tok];
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          const int key = key0 + hh * 8 + qr;
          if (key < s.kv_len && token_sees<kWin>(p, s, tok, key))
            sum[hh] += ex2_approx(fmaf(c[2 * hh + e], p.scale_log2, -1.4426950408889634f * lse));
        }
      }
    }
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      sum[hh] += __shfl_xor_sync(0xffffffffu, sum[hh], 1);
      sum[hh] += __shfl_xor_sync(0xffffffffu, sum[hh], 2);
      if ((lane & 3) == 0 && place[hh] >= 0) {
        float* w = p.key_weights + place[hh];
        *w = key0 + hh * 8 + qr >= past ? sum[hh] : *w + sum[hh];   // a new token's key had none before
      }
    }
  }
}

}  // namespace
}  // namespace thd
