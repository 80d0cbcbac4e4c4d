// kv_evict.cu — eviction of keys and values from a paged cache by the attention weight they got
// (thd_kv_evict, include/thd_attn.h).
//
// Of the L keys of a sequence and key/value head, K are kept: the first `sinks`, the last `recent`, and of
// the others those with the most weight (of equal ones the lower slot).  They keep their order and take
// slots 0 .. K - 1, in the same pages or in others.
//
// Two launches.  The first finds, for every (sequence, head), the weight of the last key to stay by
// counting digits from the top (three passes over the weights, read once into shared memory where they fit
// there), and writes the kept slots in order.  The second moves the keys, values and weights; it is bound by
// reading and writing 4 d + 4 bytes for each kept key and head.  Measured, 32 sequences of 500000 keys in all cut to
// 4000 to 8000, 8 heads of 128: 365 to 380 us into other pages, of which 281 move 1.69 GB (6.0 TB/s) and 60 select; 420 to
// 540 in place.  8 lists of 262144 keys cut to half: 364 us into other pages, 690 in place (a round's reads wait for the
// round before).  1000 keys cut to 500: 15 us on the GPU.
#include <cooperative_groups.h>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/thd_attn.h"
#include "seq_rows.cuh"

namespace thd {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelectThreads = 512;
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 32;                  // kept keys of a warp's step
constexpr int kDigit = 11;                     // bits of a pass, 10 in the last of three
constexpr int kBins = 1 << kDigit;             // the sign, the exponent and two bits more spread the first counts
constexpr int kCachedMax = 92 * 1024 / 4;      // weights of a run that are held in shared memory: two CTAs on an SM

struct EvictArgs {
  uint16_t* kc;
  uint16_t* vc;
  float* w;
  const int32_t* table;
  const int32_t* to_table;   // == table: in place
  const int32_t* kv_lens;
  const int32_t* keep_lens;
  int32_t* kept;             // [B, Hkv, max_keep]
  int32_t* new_lens;
  long long table_stride, to_stride, k_page, k_token, k_head, v_page, v_token, v_head;
  int w_page, w_token, w_head;   // 32-bit: a third of the select kernel's instructions were 64-bit products
  int num_pages, page_size, max_pages, to_pages;
  int page_shift;            // page_size = 2^page_shift, or -1
  int sinks, recent, max_keep, cached;
  int B, Hkv, d;
};

// Lengths before and after, clamped to the tables.
__device__ __forceinline__ int2 evict_lens(const EvictArgs& p, int b) {
  const long long room = (long long)p.max_pages * p.page_size, to_room = (long long)p.to_pages * p.page_size;
  const long long L = min(max((long long)p.kv_lens[b], 0ll), room);
  const long long K = min(min(max((long long)p.keep_lens[b], 0ll), L), min(to_room, (long long)p.max_keep));
  return make_int2((int)L, (int)K);
}

// Page and place in it of a slot; page -1 where the table names none.
__device__ __forceinline__ int2 slot_place(const EvictArgs& p, const int32_t* table, int slot) {
  const int at = p.page_shift >= 0 ? slot >> p.page_shift : slot / p.page_size, page = table[at];
  return make_int2(page >= 0 && page < p.num_pages ? page : -1, slot - at * p.page_size);
}

// Weights in the order of unsigned integers: NaN above all, zeros of both signs equal.
__device__ __forceinline__ uint32_t ordered(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

// A cluster of CTAs takes a list: each a run of its slots, the counts of all of them read out of one another's
// shared memory.
__global__ void __launch_bounds__(kSelectThreads, 3) kv_evict_select_kernel(const EvictArgs p) {
  constexpr int kWarps = kSelectThreads / 32;
  extern __shared__ __align__(16) uint32_t cache[];
  __shared__ __align__(16) uint32_t hist[2][kBins];
  __shared__ uint32_t s_warp[kWarps], s_digit, s_left;
  __shared__ int s_more[2][kWarps], s_same[2][kWarps];
  __shared__ int2 s_count;   // of this CTA's slots: those above the bound, and equal to it
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int list = blockIdx.x / C, b = list / p.Hkv, head = list - b * p.Hkv;
  const int2 len = evict_lens(p, b);
  const int L = len.x, K = len.y;
  const int first = min(p.sinks, K), last = min(p.recent, K - first);
  const int take = K - first - last, end = L - last;   // `take` of the slots [first, end)
  // this CTA's slots [from, to), whole warps of them
  const int run = ((L + C - 1) / C + 31) & ~31;
  const int from = (int)min((long long)L, (long long)rank * run), to = (int)min((long long)L, (long long)from + run);
  const int32_t* table = p.table + (long long)b * p.table_stride;
  const float* weights = p.w + (long long)head * p.w_head;
  auto weight_of = [&](int slot) {
    const int2 at = slot_place(p, table, slot);
    return at.x < 0 ? ordered(0.f) : ordered(weights[(long long)at.x * p.w_page + (long long)at.y * p.w_token]);
  };

  // ---- the least weight that stays, digit by digit ----
  uint32_t bound = take > 0 ? 0u : 0xFFFFFFFFu;   // keys above it stay
  int same = 0;                                   // and so many of those equal to it
  const int lo = max(from, first), hi = max(lo, min(to, end));
  const int n = hi - lo, held = min(n, p.cached);   // cache[j]: slot lo + j
  auto key_of = [&](int slot) { return slot - lo < held ? cache[slot - lo] : weight_of(slot); };
  if (take > 0) {
    constexpr int kAhead = 8;   // weights read at once: each waits for its page's entry first
    for (int j0 = tid; j0 < held; j0 += kSelectThreads * kAhead) {
      uint32_t u[kAhead];
#pragma unroll
      for (int e = 0; e < kAhead; ++e) u[e] = j0 + e * kSelectThreads < held ? weight_of(lo + j0 + e * kSelectThreads) : 0u;
#pragma unroll
      for (int e = 0; e < kAhead; ++e)
        if (j0 + e * kSelectThreads < held) cache[j0 + e * kSelectThreads] = u[e];
    }
    uint32_t left = take;
    for (int pass = 0; pass < 3; ++pass) {
      const int bits = pass < 2 ? kDigit : 32 - 2 * kDigit, shift = 32 - min(32, (pass + 1) * kDigit);
      uint32_t* mine = hist[pass & 1];
      for (int i = tid; i < kBins; i += kSelectThreads) mine[i] = 0u;
      __syncthreads();
      auto count = [&](uint32_t u) {
        if (pass == 0 || (u ^ bound) >> (shift + bits) == 0u) atomicAdd(&mine[(u >> shift) & ((1u << bits) - 1u)], 1u);
      };
      for (int j = tid * 4; j < held; j += kSelectThreads * 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(cache + j);   // what lies behind the last is not counted
        count(u.x);
        if (j + 1 < held) count(u.y);
        if (j + 2 < held) count(u.z);
        if (j + 3 < held) count(u.w);
      }
      for (int j0 = held + tid; j0 < n; j0 += kSelectThreads * kAhead) {
        uint32_t u[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e) u[e] = j0 + e * kSelectThreads < n ? weight_of(lo + j0 + e * kSelectThreads) : 0u;
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
          if (j0 + e * kSelectThreads < n) count(u[e]);
      }
      if (C > 1) cluster.sync(); else __syncthreads();
      // a thread adds up kBins / kSelectThreads digits; those above them are the threads' after it
      constexpr int kMine = kBins / kSelectThreads;
      static_assert(kMine == 4, "a thread's digits are one 16-byte word");
      uint4 d = make_uint4(0u, 0u, 0u, 0u);
      for (int c = 0; c < C; ++c) {
        const uint4* src = reinterpret_cast<const uint4*>(mine) + tid;
        const uint4 x = C > 1 ? *cluster.map_shared_rank(src, c) : *src;
        d.x += x.x, d.y += x.y, d.z += x.z, d.w += x.w;
      }
      const uint32_t sum = d.x + d.y + d.z + d.w;
      uint32_t above = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_down_sync(0xffffffffu, above, o);
        if (lane + o < 32) above += y;
      }
      if (lane == 0) s_warp[warp] = above;
      __syncthreads();
      above -= sum;
      for (int w = warp + 1; w < kWarps; ++w) above += s_warp[w];
      if (above < left && left <= above + sum) {
        const uint32_t of[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int e = 3; e >= 0; --e) {
          if (above < left && left <= above + of[e]) {
            s_digit = tid * 4 + e;
            s_left = left - above;
          }
          above += of[e];
        }
      }
      __syncthreads();
      bound |= s_digit << shift;
      left = s_left;
    }
    same = (int)left;
  }
  // whether a slot stays whatever its equals do, and whether it is one of those equal to the bound
  auto rank_of = [&](int i, bool& more, bool& equal) {
    more = equal = false;
    if (i < to) {
      if (i < first || i >= end) {
        more = true;
      } else if (take > 0) {
        const uint32_t u = key_of(i);
        more = u > bound;
        equal = u == bound;
      }
    }
  };

  // ---- what the CTAs before this one keep ----
  int more_before = 0, same_before = 0;
  if (C > 1) {
    int2 n = make_int2(0, 0);
    if (tid == 0) s_count = n;
    __syncthreads();
    for (int i = from + tid; i < to; i += kSelectThreads) {
      bool more, equal;
      rank_of(i, more, equal);
      n.x += more ? 1 : 0;
      n.y += equal ? 1 : 0;
    }
    n.x = __reduce_add_sync(0xffffffffu, n.x);
    n.y = __reduce_add_sync(0xffffffffu, n.y);
    if (lane == 0) {
      atomicAdd(&s_count.x, n.x);
      atomicAdd(&s_count.y, n.y);
    }
    cluster.sync();
    for (int c = 0; c < rank; ++c) {
      const int2 other = *cluster.map_shared_rank(&s_count, c);
      more_before += other.x;
      same_before += other.y;
    }
    cluster.sync();   // no CTA leaves while another may read its counts
  }

  // ---- the kept slots, in order: a warp 32 slots of each of kWords runs one after another ----
  constexpr int kWords = 4;
  int32_t* kept = p.kept + (long long)list * p.max_keep;
  for (int i0 = from, turn = 0; i0 < to; i0 += kSelectThreads * kWords, turn ^= 1) {
    uint32_t more_bits[kWords], same_bits[kWords];
    int m_sum = 0, e_sum = 0;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      bool more, equal;
      rank_of(i0 + (warp * kWords + w) * 32 + lane, more, equal);
      more_bits[w] = __ballot_sync(0xffffffffu, more);
      same_bits[w] = __ballot_sync(0xffffffffu, equal);
      m_sum += __popc(more_bits[w]);
      e_sum += __popc(same_bits[w]);
    }
    if (lane == 0) {
      s_more[turn][warp] = m_sum;
      s_same[turn][warp] = e_sum;
    }
    __syncthreads();
    // what the warps before this one keep, and all of them
    const int x = lane < kWarps ? s_more[turn][lane] : 0, y = lane < kWarps ? s_same[turn][lane] : 0;
    int m = more_before + __reduce_add_sync(0xffffffffu, lane < warp ? x : 0);
    int e = same_before + __reduce_add_sync(0xffffffffu, lane < warp ? y : 0);
    more_before += __reduce_add_sync(0xffffffffu, x);
    same_before += __reduce_add_sync(0xffffffffu, y);
    const uint32_t below = (1u << lane) - 1u;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
      const int me = m + __popc(more_bits[w] & below), ee = e + __popc(same_bits[w] & below);
      if ((more_bits[w] >> lane & 1) || ((same_bits[w] >> lane & 1) && ee < same))
        kept[me + min(ee, same)] = i0 + (warp * kWords + w) * 32 + lane;
      m += __popc(more_bits[w]);
      e += __popc(same_bits[w]);
    }
  }
  // 64 bits: a list may be as wide as 2^31 - 1, and the step behind its end passes that
  for (long long i = (long long)K + rank * kSelectThreads + tid; i < p.max_keep; i += C * kSelectThreads) kept[i] = -1;
  if (head == 0 && rank == 0 && tid == 0) p.new_lens[b] = K;
}

// Moves: a warp takes 32 kept keys.  A lane finds where one of them lies and goes; then the lanes carry
// 16 bytes each of as many of the 32 rows as fit a step, keys, then values.
struct Moves {
  long long from, to;   // this lane's key: element offsets in the weights (-1: not moved)
  long long kf, kt, vf, vt;
};

__device__ __forceinline__ Moves find_moves(const EvictArgs& p, int b, int head, int at, int K) {
  Moves m;
  m.from = m.to = -1;
  m.kf = m.kt = m.vf = m.vt = 0;
  if (at < K) {
    const int slot = p.kept[((long long)b * p.Hkv + head) * p.max_keep + at];
    const int2 f = slot_place(p, p.table + (long long)b * p.table_stride, slot);
    const int2 t = slot_place(p, p.to_table + (long long)b * p.to_stride, at);
    if (f.x >= 0 && t.x >= 0 && (f.x != t.x || f.y != t.y)) {
      m.from = (long long)f.x * p.w_page + (long long)f.y * p.w_token + (long long)head * p.w_head;
      m.to = (long long)t.x * p.w_page + (long long)t.y * p.w_token + (long long)head * p.w_head;
      m.kf = f.x * p.k_page + f.y * p.k_token + head * p.k_head;
      m.kt = t.x * p.k_page + t.y * p.k_token + head * p.k_head;
      m.vf = f.x * p.v_page + f.y * p.v_token + head * p.v_head;
      m.vt = t.x * p.v_page + t.y * p.v_token + head * p.v_head;
    }
  }
  return m;
}

// Lists of kept keys one CTA (or cluster of them) each, in rounds: all of a round's keys are read before any is
// written.  A key moves to its own slot or a lower one, so what a round writes lies below all that
// later rounds read, and rounds need no order among them but this.
__global__ void __launch_bounds__(kMoveThreads) kv_evict_within_kernel(const EvictArgs p) {
  constexpr int kWarps = kMoveThreads / 32;
  constexpr int kPieces = 16;   // 16-byte pieces of keys that a lane holds, and as many of values
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int list = blockIdx.x / C, b = list / p.Hkv, head = list - b * p.Hkv;
  const int K = evict_lens(p, b).y;
  const int chunks = p.d / 8, rows = 32 / chunks;   // rows of a step
  const int row = lane / chunks, col = (lane - row * chunks) * 8;
  // a warp's keys of a round: as many as its pieces hold
  const int mine = min(kMoveRows, kPieces * rows);
  const int round = C * kWarps * mine;
  for (int r0 = 0; r0 < K; r0 += round) {
    const int at = r0 + (rank * kWarps + warp) * mine;
    const Moves m = find_moves(p, b, head, lane < mine ? at + lane : K, K);
    uint4 k[kPieces], v[kPieces];
    float w = 0.f;
    if (m.to >= 0) w = p.w[m.from];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int src = i * rows + row;
      const long long kf = __shfl_sync(0xffffffffu, m.kf, src & 31), vf = __shfl_sync(0xffffffffu, m.vf, src & 31);
      const bool go = __shfl_sync(0xffffffffu, m.to, src & 31) >= 0 && src < mine && row < rows;
      if (go) {
        k[i] = *reinterpret_cast<const uint4*>(p.kc + kf + col);
        v[i] = *reinterpret_cast<const uint4*>(p.vc + vf + col);
      }
    }
    if (C > 1) cluster.sync(); else __syncthreads();
    if (m.to >= 0) p.w[m.to] = w;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int src = i * rows + row;
      const long long kt = __shfl_sync(0xffffffffu, m.kt, src & 31), vt = __shfl_sync(0xffffffffu, m.vt, src & 31);
      const bool go = __shfl_sync(0xffffffffu, m.to, src & 31) >= 0 && src < mine && row < rows;
      if (go) {
        *reinterpret_cast<uint4*>(p.kc + kt + col) = k[i];
        *reinterpret_cast<uint4*>(p.vc + vt + col) = v[i];
      }
    }
  }
}

// Into other pages: steps of 32 kept keys over all lists, laid end to end, a warp each.
__global__ void __launch_bounds__(kMoveThreads, 2) kv_evict_apart_kernel(const EvictArgs p) {
  constexpr int kWarps = kMoveThreads / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * kWarps;
  long long step = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5), base = 0;
  const int chunks = p.d / 8, rows = 32 / chunks;
  const int row = lane / chunks, col = (lane - row * chunks) * 8;
  for (int b = 0; b < p.B; ++b) {
    const int K = evict_lens(p, b).y, per = (K + kMoveRows - 1) / kMoveRows;
    for (; step < base + (long long)per * p.Hkv; step += warps) {
      const int in = (int)(step - base), head = in / per, at = (in - head * per) * kMoveRows;
      const Moves m = find_moves(p, b, head, at + lane, K);
      if (m.to >= 0) p.w[m.to] = p.w[m.from];
      constexpr int kPieces = 8;   // of keys and of values that a lane holds: reads on the way before the first write
#pragma unroll 1
      for (int i0 = 0; i0 < kMoveRows; i0 += rows * kPieces) {
        uint4 k[kPieces], v[kPieces];
#pragma unroll
        for (int e = 0; e < kPieces; ++e) {
          const int src = i0 + e * rows + row;
          const long long kf = __shfl_sync(0xffffffffu, m.kf, src & 31), vf = __shfl_sync(0xffffffffu, m.vf, src & 31);
          const bool go = __shfl_sync(0xffffffffu, m.to, src & 31) >= 0 && src < kMoveRows && row < rows;
          if (go) {
            k[e] = *reinterpret_cast<const uint4*>(p.kc + kf + col);
            v[e] = *reinterpret_cast<const uint4*>(p.vc + vf + col);
          }
        }
#pragma unroll
        for (int e = 0; e < kPieces; ++e) {
          const int src = i0 + e * rows + row;
          const long long kt = __shfl_sync(0xffffffffu, m.kt, src & 31), vt = __shfl_sync(0xffffffffu, m.vt, src & 31);
          const bool go = __shfl_sync(0xffffffffu, m.to, src & 31) >= 0 && src < kMoveRows && row < rows;
          if (go) {
            *reinterpret_cast<uint4*>(p.kc + kt + col) = k[e];
            *reinterpret_cast<uint4*>(p.vc + vt + col) = v[e];
          }
        }
      }
    }
    base += (long long)per * p.Hkv;
  }
}

}  // namespace
}  // namespace thd

extern "C" int thd_kv_evict(void* k_cache, void* v_cache, const int64_t* cache_strides, float* key_weights,
                            const int64_t* weight_strides, int num_pages, int page_size, const int32_t* page_table,
                            int64_t page_table_stride, int max_pages, const int32_t* new_page_table,
                            int64_t new_page_table_stride, int new_max_pages, const int32_t* kv_lens,
                            const int32_t* keep_lens, int batch_size, int sink_tokens, int recent_tokens, int32_t* kept,
                            int max_keep, int32_t* new_lens, int num_heads_kv, int head_dim, int dtype, void* stream) {
  using namespace thd;
  if (batch_size < 0 || num_heads_kv < 1 || num_pages < 0 || page_size < 1 || max_pages < 0) return THD_ERR_ARG;
  if (sink_tokens < 0 || recent_tokens < 0 || max_keep < 0) return THD_ERR_ARG;
  if (dtype != THD_BF16 && dtype != THD_FP16) return THD_ERR_UNSUPPORTED;
  if (head_dim < 8 || head_dim > 128 || head_dim % 8 != 0) return THD_ERR_UNSUPPORTED;
  // slots are 32-bit, and so are those of a round past the last
  if ((long long)max_pages * page_size >= (1ll << 31) - 4096) return THD_ERR_UNSUPPORTED;
  if ((long long)batch_size * num_heads_kv >= (1ll << 27)) return THD_ERR_UNSUPPORTED;
  if (!cache_strides || !weight_strides || page_table_stride < max_pages) return THD_ERR_ARG;
  for (int i = 0; i < 6; ++i)
    if (cache_strides[i] < 0 || cache_strides[i] % 8 != 0) return THD_ERR_ARG;
  for (int i = 0; i < 3; ++i)
    if (weight_strides[i] < 0) return THD_ERR_ARG;
  for (int i = 0; i < 3; ++i)
    if (weight_strides[i] >= (1ll << 31)) return THD_ERR_UNSUPPORTED;
  if (new_page_table) {
    if (new_max_pages < 0 || new_page_table_stride < new_max_pages) return THD_ERR_ARG;
    if ((long long)new_max_pages * page_size >= (1ll << 31) - 4096) return THD_ERR_UNSUPPORTED;
  }
  if (batch_size == 0) return THD_OK;
  if (!kv_lens || !keep_lens || !new_lens || (max_keep > 0 && !kept)) return THD_ERR_ARG;
  if (!on4(page_table) || !on4(new_page_table) || !on4(kv_lens) || !on4(keep_lens) || !on4(new_lens) || !on4(kept) ||
      !on4(key_weights) || !on16(k_cache) || !on16(v_cache))
    return THD_ERR_ARG;
  // every head reads the lengths while the first one writes the new ones
  for (const int32_t* lens : {kv_lens, keep_lens})
    if (new_lens < lens + batch_size && lens < new_lens + batch_size) return THD_ERR_ARG;
  if (num_pages == 0) max_pages = 0;   // no sequence has keys
  if (max_pages > 0 && (!page_table || !k_cache || !v_cache || !key_weights)) return THD_ERR_ARG;
  const bool within = !new_page_table || new_page_table == page_table;
  // the same rows, of which a narrower table names the first pages
  if (within && new_page_table && batch_size > 1 && new_page_table_stride != page_table_stride) return THD_ERR_ARG;
  const int sms = device_sms();
  if (sms <= 0) return THD_ERR_CUDA;
  EvictArgs p{};
  p.kc = static_cast<uint16_t*>(k_cache);
  p.vc = static_cast<uint16_t*>(v_cache);
  p.w = key_weights;
  p.table = page_table;
  p.table_stride = page_table_stride;
  p.to_table = within ? page_table : new_page_table;
  p.to_stride = within ? page_table_stride : new_page_table_stride;
  p.to_pages = new_page_table ? new_max_pages : max_pages;
  p.kv_lens = kv_lens;
  p.keep_lens = keep_lens;
  p.kept = kept;
  p.new_lens = new_lens;
  p.k_page = cache_strides[0];
  p.k_token = cache_strides[1];
  p.k_head = cache_strides[2];
  p.v_page = cache_strides[3];
  p.v_token = cache_strides[4];
  p.v_head = cache_strides[5];
  p.w_page = (int)weight_strides[0];
  p.w_token = (int)weight_strides[1];
  p.w_head = (int)weight_strides[2];
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.page_shift = -1;
  for (int s = 0; s < 31; ++s)
    if (page_size == 1 << s) p.page_shift = s;
  p.max_pages = max_pages;
  p.sinks = sink_tokens;
  p.recent = recent_tokens;
  p.max_keep = max_keep;
  p.B = batch_size;
  p.Hkv = num_heads_kv;
  p.d = head_dim;
  const long long room = (long long)max_pages * page_size;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int lists = batch_size * num_heads_kv;
  int C = 1;   // CTAs of a list: the lists alone may not fill the GPU
  while (C < 8 && 2ll * C * lists <= sms) C *= 2;
  // a list is selected by as many as hold its weights in shared memory (27000 of them read again from the L2 where
  // they did not fit cost 60 us of 94), or, of few lists, with 4096 slots each or more
  int Cs = 1;
  while (Cs < 8 && (room / Cs > kCachedMax || (Cs < C && room / Cs > 4096))) Cs *= 2;
  const long long run = ((room + Cs - 1) / Cs + 31) / 32 * 32;
  p.cached = (int)(run < kCachedMax ? (run + 3) / 4 * 4 : kCachedMax);
  static SmemGrant grant;
  if (!grant.ask(kv_evict_select_kernel, kCachedMax * 4)) return THD_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = Cs;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = Cs > 1 ? 1 : 0;
  cfg.stream = st;
  cfg.gridDim = dim3(lists * Cs);
  cfg.blockDim = dim3(kSelectThreads);
  cfg.dynamicSmemBytes = (size_t)p.cached * 4;
  if (cudaLaunchKernelEx(&cfg, kv_evict_select_kernel, static_cast<const EvictArgs>(p)) != cudaSuccess) return THD_ERR_CUDA;
  cfg.blockDim = dim3(kMoveThreads);
  cfg.dynamicSmemBytes = 0;
  cudaError_t e;
  if (within) {
    attr[0].val.clusterDim.x = C;
    cfg.attrs = C > 1 ? attr : attr + 1;
    cfg.numAttrs = C > 1 ? 2 : 1;
    cfg.gridDim = dim3(lists * C);
    e = cudaLaunchKernelEx(&cfg, kv_evict_within_kernel, static_cast<const EvictArgs>(p));
  } else {
    cfg.attrs = attr + 1;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(2 * sms);
    e = cudaLaunchKernelEx(&cfg, kv_evict_apart_kernel, static_cast<const EvictArgs>(p));
  }
  return e == cudaSuccess ? THD_OK : THD_ERR_CUDA;
}
