// kv_evict.cu — eviction of keys and values from a paged cache by the attention weight they got
// (thd_kv_evict, include/thd_attn.h).
//
// Of the L keys of a sequence and key/value head, K are kept: the first `sinks`, the last `recent`, and of
// the others those with the most weight (of equal ones the lower slot).  They keep their order and take
// slots 0 .. K - 1, in the same pages or in others.
//
// Two launches.  The first finds, for every (sequence, head), the weight of the last key to stay by
// counting digits of 8 bits from the top (four passes over the weights, which lie in shared memory after the
// first where they fit), and writes the kept slots in order.  The second moves the keys, values and weights;
// it is what takes the time: 8 d + 8 bytes for each kept key and head, read and written once.
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
constexpr int kCachedMax = 160 * 1024 / 4;     // weights of a head that are held in shared memory

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
  long long table_stride, to_stride, k_page, k_token, k_head, v_page, v_token, v_head, w_page, w_token, w_head;
  int num_pages, page_size, max_pages, to_pages;
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
  const int at = slot / p.page_size, page = table[at];
  return make_int2(page >= 0 && page < p.num_pages ? page : -1, slot - at * p.page_size);
}

// Weights in the order of unsigned integers: NaN above all, zeros of both signs equal.
__device__ __forceinline__ uint32_t ordered(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

__global__ void __launch_bounds__(kSelectThreads) kv_evict_select_kernel(const EvictArgs p) {
  constexpr int kWarps = kSelectThreads / 32;
  extern __shared__ uint32_t cache[];
  __shared__ uint32_t hist[256];
  __shared__ uint32_t s_digit, s_left;
  __shared__ int s_more[2][kWarps], s_same[2][kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int b = blockIdx.x / p.Hkv, head = blockIdx.x - b * p.Hkv;
  const int2 len = evict_lens(p, b);
  const int L = len.x, K = len.y;
  const int first = min(p.sinks, K), last = min(p.recent, K - first);
  const int take = K - first - last, end = L - last;   // `take` of the slots [first, end)
  const int32_t* table = p.table + (long long)b * p.table_stride;
  auto weight_of = [&](int slot) {
    const int2 at = slot_place(p, table, slot);
    return at.x < 0 ? ordered(0.f) : ordered(p.w[at.x * p.w_page + at.y * p.w_token + head * p.w_head]);
  };
  auto key_of = [&](int slot) { return slot - first < p.cached ? cache[slot - first] : weight_of(slot); };

  // ---- the least weight that stays, digit by digit ----
  uint32_t bound = take > 0 ? 0u : 0xFFFFFFFFu;   // keys above it stay
  int same = 0;                                   // and so many of those equal to it
  if (take > 0) {
    for (int i = first + tid; i < end && i - first < p.cached; i += kSelectThreads) cache[i - first] = weight_of(i);
    uint32_t left = take;
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0u;
      __syncthreads();
      for (int i0 = first + warp * 32; i0 < end; i0 += kSelectThreads) {
        const int i = i0 + lane;
        const uint32_t u = i < end ? key_of(i) : 0u;
        const bool in = i < end && (shift == 24 || (u >> (shift + 8)) == (bound >> (shift + 8)));
        const uint32_t digit = in ? (u >> shift) & 255u : 256u;
        const uint32_t peers = __match_any_sync(0xffffffffu, digit);
        if (in && lane == __ffs(peers) - 1) atomicAdd(&hist[digit], (uint32_t)__popc(peers));
      }
      __syncthreads();
      if (warp == 0) {   // lane l: digits [8 l, 8 l + 8); counted from the top
        uint32_t mine = 0;
        for (int e = 0; e < 8; ++e) mine += hist[lane * 8 + e];
        uint32_t above = mine;
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_down_sync(0xffffffffu, above, o);
          if (lane + o < 32) above += y;
        }
        above -= mine;   // of the digits of the lanes after this one
        if (above < left && left <= above + mine) {
          for (int e = 7; e >= 0; --e) {
            const uint32_t n = hist[lane * 8 + e];
            if (left <= above + n) {
              s_digit = lane * 8 + e;
              s_left = left - above;
              break;
            }
            above += n;
          }
        }
      }
      __syncthreads();
      bound |= s_digit << shift;
      left = s_left;
    }
    same = (int)left;
  }

  // ---- the kept slots, in order ----
  int32_t* kept = p.kept + (long long)blockIdx.x * p.max_keep;
  int more_before = 0, same_before = 0;
  for (int i0 = 0, turn = 0; i0 < L; i0 += kSelectThreads, turn ^= 1) {
    const int i = i0 + tid;
    bool more = false, equal = false;
    if (i < L) {
      if (i < first || i >= end) {
        more = true;
      } else if (take > 0) {
        const uint32_t u = key_of(i);
        more = u > bound;
        equal = u == bound;
      }
    }
    const uint32_t more_bits = __ballot_sync(0xffffffffu, more), same_bits = __ballot_sync(0xffffffffu, equal);
    if (lane == 0) {
      s_more[turn][warp] = __popc(more_bits);
      s_same[turn][warp] = __popc(same_bits);
    }
    __syncthreads();
    int m = more_before, e = same_before;
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) {
        m += __popc(more_bits & ((1u << lane) - 1u));
        e += __popc(same_bits & ((1u << lane) - 1u));
        if (more || (equal && e < same)) kept[m + min(e, same)] = i;
      }
      more_before += s_more[turn][w];
      same_before += s_same[turn][w];
      if (w < warp) {
        m += s_more[turn][w];
        e += s_same[turn][w];
      }
    }
  }
  for (int i = K + tid; i < p.max_keep; i += kSelectThreads) kept[i] = -1;
  if (head == 0 && tid == 0) p.new_lens[b] = K;
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
      m.from = f.x * p.w_page + f.y * p.w_token + head * p.w_head;
      m.to = t.x * p.w_page + t.y * p.w_token + head * p.w_head;
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
__global__ void __launch_bounds__(kMoveThreads) kv_evict_apart_kernel(const EvictArgs p) {
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
      for (int i = 0; i < kMoveRows; i += rows) {
        const int src = (i + row) & 31;
        const long long kf = __shfl_sync(0xffffffffu, m.kf, src), vf = __shfl_sync(0xffffffffu, m.vf, src);
        const long long kt = __shfl_sync(0xffffffffu, m.kt, src), vt = __shfl_sync(0xffffffffu, m.vt, src);
        const bool go = __shfl_sync(0xffffffffu, m.to, src) >= 0 && i + row < kMoveRows && row < rows;
        if (go) {
          const uint4 k = *reinterpret_cast<const uint4*>(p.kc + kf + col);
          const uint4 v = *reinterpret_cast<const uint4*>(p.vc + vf + col);
          *reinterpret_cast<uint4*>(p.kc + kt + col) = k;
          *reinterpret_cast<uint4*>(p.vc + vt + col) = v;
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
  const int sms = device_sms();
  if (sms <= 0) return THD_ERR_CUDA;
  const bool within = !new_page_table || new_page_table == page_table;
  EvictArgs p{};
  p.kc = static_cast<uint16_t*>(k_cache);
  p.vc = static_cast<uint16_t*>(v_cache);
  p.w = key_weights;
  p.table = page_table;
  p.table_stride = page_table_stride;
  p.to_table = within ? page_table : new_page_table;
  p.to_stride = within ? page_table_stride : new_page_table_stride;
  p.to_pages = within ? max_pages : new_max_pages;
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
  p.w_page = weight_strides[0];
  p.w_token = weight_strides[1];
  p.w_head = weight_strides[2];
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.max_pages = max_pages;
  p.sinks = sink_tokens;
  p.recent = recent_tokens;
  p.max_keep = max_keep;
  p.B = batch_size;
  p.Hkv = num_heads_kv;
  p.d = head_dim;
  const long long room = (long long)max_pages * page_size;
  p.cached = (int)(room < kCachedMax ? room : kCachedMax);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int lists = batch_size * num_heads_kv;
  static SmemGrant grant;
  if (!grant.ask(kv_evict_select_kernel, kCachedMax * 4)) return THD_ERR_CUDA;
  kv_evict_select_kernel<<<lists, kSelectThreads, (size_t)p.cached * 4, st>>>(p);
  if (cudaGetLastError() != cudaSuccess) return THD_ERR_CUDA;

  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = st;
  cudaError_t e;
  if (within) {
    int C = 1;   // CTAs of a list: the lists alone may not fill the GPU
    while (C < 8 && 2 * C * lists <= 2 * sms) C *= 2;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    cfg.gridDim = dim3(lists * C);
    e = cudaLaunchKernelEx(&cfg, kv_evict_within_kernel, static_cast<const EvictArgs>(p));
  } else {
    cfg.gridDim = dim3(4 * sms);
    e = cudaLaunchKernelEx(&cfg, kv_evict_apart_kernel, static_cast<const EvictArgs>(p));
  }
  return e == cudaSuccess ? THD_OK : THD_ERR_CUDA;
}
