// qk_norm_rope.cu — what a model does to its query and key heads between the projection and
// the attention: RMS norm of each head and the rotation by the row's position, for packed rows
// (thd_qk_norm_rope), its gradients (thd_qk_norm_rope_bwd), and the same on the way into a
// paged key/value cache (thd_kv_append).  Declared in include/thd_attn.h.
//
// For a head x of d values at position p:
//   n = x * r * w,  r = 1 / sqrt(mean(x^2) + eps)          (n = x without a weight)
//   y_i = n_i cos_i - n_j sin_i,  y_j = n_j cos_i + n_i sin_i   for each rotated pair (i, j)
// with cos / sin row p of the caller's tables; values past rotary_dim are left as n.
// Backward, with g the gradient of y:
//   h_i = g_i cos_i + g_j sin_i,  h_j = g_j cos_i - g_i sin_i   (the rotation by -p)
//   dw = sum over rows of h * x * r,   dx = r * (h * w - x * r^2 * mean(h * w * x))
// All in fp32, rounded once to the tensors' type.  dw is summed in fp32 too: a few terms one after another in
// a lane, then trees (2e-7 of its norm off over 200000 rows of 32 heads, where rounding it to fp32 alone is 3e-8).
//
// Layout: a head is d / 8 chunks of 16 bytes.  One lane holds two of them, the two whose values
// pair up under the half-split rotation (chunks s and s + rotary / 16; of the part behind, one of
// each half), so a rotation needs no exchange between lanes and a norm only the sum over
// the d / 16 lanes of a head.  A warp takes one row's block of heads: the row's sequence is
// found and its angles loaded once for all of them, while the heads' own loads are in flight.
#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/thd_attn.h"
#include "seq_rows.cuh"

namespace thd {
namespace {

struct HeadRows {            // rows of one kind of heads
  const void* src;
  void* dst;                 // packed rows (null: into the cache)
  const void* weight;        // null: no norm
  long long src_stride;      // elements from row to row
  long long dst_stride;
  int heads;
};

struct RowArgs {
  HeadRows q, k, v;
  const float* cos;
  const float* sin;
  const int32_t* cu;
  const int32_t* padded;
  const int32_t* offsets;    // added to the position of each row of sequence b (cache: its length so far)
  const int32_t* positions;  // cache: position of each row, or null
  long long rope_rows;
  float eps, inv_d;
  float sin_sign;            // -1 turns back
  int T, B, d, rotary;
  int interleaved, weight_fp32;
  int q_items, k_items;      // blocks of heads per row
  int row_items;             // of all kinds
  unsigned run;              // items of a warp
  // few heads: rows of an item and items of each kind
  int q_rows, k_rows, v_rows;
  unsigned q_total, k_total, v_total;
  // cache
  void* k_cache;
  void* v_cache;
  const int32_t* table;
  long long table_stride, k_page, k_token, k_head, v_page, v_token, v_head;   // elements
  int num_pages, page_size, max_pages;
};

constexpr int kRowWarps = 4;      // warps of a block
constexpr int kRowPasses = 4;     // 32 / lanes-per-head heads in each
constexpr int kRowStages = 2;     // the item worked on and one on the way
constexpr int kRowBlocksPerSm = 4;
constexpr int kRowRun = 6;        // items of a warp at most
// Per cent of the lanes at work below which items take whole rows (few_heads_kernel).  Share of the copy
// bandwidth, items of one row against whole rows, heads of 128, normed: 4 + 4 heads (25 %) 44 and 52,
// 8 + 1 (28 %) 49 and 54, 8 + 2 (31 %) 54 and 53, 16 + 2 (56 %) 79 and 57.  The lanes that heads of 48, 80, 96
// and 112 leave idle in both forms do not count: heads of 80 reach 35 to 42 % with whole rows, of 96 41 to 49 %.
constexpr int kFewShare = 30;

// Two fp32 values in one 64-bit register: multiplied and added by one instruction.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pair(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 split(f2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ f2 swapped(f2 x) {
  const float2 v = split(x);
  return pair(v.y, v.x);
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
template <typename DT>
__device__ __forceinline__ void unpack4(const uint4& x, f2* f) {
  const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = Pair16<DT>::get(u[i]);
    f[i] = pair(v.x, v.y);
  }
}
template <typename DT>
__device__ __forceinline__ uint4 pack4(const f2* f) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = split(f[i]);
    u[i] = Pair16<DT>::put(v.x, v.y);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ void copy16(void* dst, const void* src) {
  cp_async16(static_cast<uint32_t>(__cvta_generic_to_shared(dst)), src);
}

// The turn of a lane's two chunks by its angles, with a factor for each value before it:
// y0 = a0 x0 + b0 z0, y1 = a1 x1 + b1 z1, where z is the other chunk (half-split) or the same one with
// neighbours swapped (interleaved).  Half-split: value e of both chunks turns by angle 8 slot + e.
// Interleaved: pair e of the first chunk by 4 slot + e, of the second by 4 (slot + rotary / 16) + e.
struct Turn {
  f2 a0[4], b0[4], a1[4], b1[4];
};

// A lane's angles from its tables' row: cos 0-3, cos 4-7, sin 0-3, sin 4-7, into four 16-byte places
// that lie `apart` uint4s from one another.
__device__ __forceinline__ void fetch_angles(uint4* dst, int apart, const RowArgs& p, int slot, long long pos) {
  const long long row = pos < 0 ? 0 : (pos >= p.rope_rows ? p.rope_rows - 1 : pos);
  const int half = p.rotary >> 1;
  const long long at0 = row * half + (p.interleaved ? 4 * slot : 8 * slot);
  const long long at1 = row * half + (p.interleaved ? 4 * (slot + (p.rotary >> 4)) : 8 * slot + 4);
  copy16(dst, p.cos + at0);
  copy16(dst + apart, p.cos + at1);
  copy16(dst + 2 * apart, p.sin + at0);
  copy16(dst + 3 * apart, p.sin + at1);
}

__device__ __forceinline__ void read_angles(const uint4* src, int apart, f2* c, f2* s) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(src + i * apart);
    const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(src + (2 + i) * apart);
    c[2 * i] = a.x, c[2 * i + 1] = a.y;
    s[2 * i] = b.x, s[2 * i + 1] = b.y;
  }
}

__device__ __forceinline__ f2 negated(f2 x) { return x ^ 0x8000000080000000ull; }

__device__ __forceinline__ void make_turn(Turn& t, const f2* c, const f2* s, const f2* w0, const f2* w1, bool rot,
                                          int interleaved) {
  if (!rot) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t.a0[i] = w0[i];
      t.a1[i] = w1[i];
      t.b0[i] = t.b1[i] = 0ull;
    }
  } else if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 cl = split(c[i >> 1]), sl = split(s[i >> 1]), ch = split(c[2 + (i >> 1)]), sh = split(s[2 + (i >> 1)]);
      const float c0 = i & 1 ? cl.y : cl.x, s0 = i & 1 ? sl.y : sl.x, c1 = i & 1 ? ch.y : ch.x, s1 = i & 1 ? sh.y : sh.x;
      t.a0[i] = mul2(pair(c0, c0), w0[i]);
      t.b0[i] = mul2(pair(-s0, s0), swapped(w0[i]));
      t.a1[i] = mul2(pair(c1, c1), w1[i]);
      t.b1[i] = mul2(pair(-s1, s1), swapped(w1[i]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      t.a0[i] = mul2(c[i], w0[i]);
      t.b0[i] = mul2(negated(s[i]), w1[i]);
      t.a1[i] = mul2(c[i], w1[i]);
      t.b1[i] = mul2(s[i], w0[i]);
    }
  }
}

// A lane that holds no rotated values leaves out the other chunk, which need not be finite.
__device__ __forceinline__ void apply_turn(const Turn& t, const f2* x0, const f2* x1, f2* y0, f2* y1, bool rot,
                                           int interleaved) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y0[i] = mul2(x0[i], t.a0[i]);
    y1[i] = mul2(x1[i], t.a1[i]);
  }
  if (rot) {
    if (interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y0[i] = fma2(swapped(x0[i]), t.b0[i], y0[i]);
        y1[i] = fma2(swapped(x1[i]), t.b1[i], y1[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y0[i] = fma2(x1[i], t.b0[i], y0[i]);
        y1[i] = fma2(x0[i], t.b1[i], y1[i]);
      }
    }
  }
}

// A lane's two chunks of a head: rotated pairs first, then the chunks behind them, a half each, so that
// neighbouring lanes read neighbouring chunks (gradients of 32 + 32 heads of 64, with 32 values rotated 0.88 of the
// copy bandwidth, with none 1.00; a lane with two neighbouring chunks of its own: 0.80 and 0.69).
__device__ __forceinline__ void lane_chunks(int slot, int rotary, int d, int& c0, int& c1) {
  const int pairs = rotary >> 4, rest = (d >> 4) - pairs;
  c0 = slot < pairs ? slot : pairs + slot;   // 2 pairs + (slot - pairs)
  c1 = slot < pairs ? slot + pairs : c0 + rest;
}

template <typename DT>
__device__ __forceinline__ void load_weight(const void* w, int fp32, int chunk, f2* f) {
  if (fp32) {
    const ulonglong2 a = reinterpret_cast<const ulonglong2*>(w)[2 * chunk];
    const ulonglong2 b = reinterpret_cast<const ulonglong2*>(w)[2 * chunk + 1];
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
  } else {
    unpack4<DT>(reinterpret_cast<const uint4*>(w)[chunk], f);
  }
}

// The items of a warp: a run of them.  More blocks than fit at once, each with short runs, beat a grid
// of warps that stay (one long run each, or strided ones): the GPU's reads and writes then move
// through memory as one front, and an SM that is slower takes fewer blocks.  Packed batch of 65536 rows of
// 32 + 8 heads of 128, normed: 205 us against 225 (strided) and 255 (long runs); 131072 rows of
// 16 + 16 without a norm: 322 us against 379 and 374.
struct ItemWalk {
  unsigned item, end, row_items, t, part;

  __device__ __forceinline__ ItemWalk(unsigned total, unsigned row_items_, unsigned warp, unsigned run)
      : row_items(row_items_) {
    const unsigned long long first = (unsigned long long)warp * run;
    item = first < total ? (unsigned)first : total;
    end = total - item < run ? total : item + run;
    t = item / row_items;
    part = item - t * row_items;
  }
  __device__ __forceinline__ bool more() const { return item < end; }
  __device__ __forceinline__ void next() {
    ++item;
    if (++part == row_items) part = 0, ++t;
  }
};

// Shared memory of a warp: kRowStages items, each its heads' chunks ([pass][chunk][lane]) and the
// row's angles ([part][slot]).
template <int kPasses, int kChunks, int LPH>
struct alignas(16) RowStage {
  uint4 x[kPasses][kChunks][32];
  uint4 angle[4][LPH];
};

// LPH lanes per head (a power of two >= d / 16).  An item is a block of one row's heads of one
// kind; a warp takes a run of items.  While it works on one it has looked up the next one's row
// and copies its heads and angles into shared memory, so that only arithmetic is left
// when its turn comes; rows of no sequence are not read.  (One item ahead: three stages took 212 us
// where two take 205 on the batch above.)
template <typename DT, int LPH, bool kCache>
__global__ void __launch_bounds__(kRowWarps * 32, kRowBlocksPerSm) head_rows_kernel(const RowArgs p) {
  constexpr int kPerPass = 32 / LPH;
  constexpr int kAhead = kRowStages - 1;
  extern __shared__ __align__(16) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto* ring = reinterpret_cast<RowStage<kRowPasses, 2, LPH>*>(smem) + warp * kRowStages;
  ItemWalk ahead((unsigned)p.T * (unsigned)p.row_items, (unsigned)p.row_items, blockIdx.x * kRowWarps + warp,
                 p.run);
  ItemWalk now = ahead;
  const int slot = lane % LPH;
  const bool mine = slot < (p.d >> 4);
  int c0, c1;
  lane_chunks(slot, p.rotary, p.d, c0, c1);

  auto kind_of = [&](int part, int& block) {   // 0 queries, 1 keys, 2 values
    if (part < p.q_items) {
      block = part;
      return 0;
    }
    block = part - p.q_items;
    if (!kCache || block < p.k_items) return 1;
    block -= p.k_items;
    return 2;
  };
  auto rows_of = [&](int kind) -> const HeadRows& { return kind == 0 ? p.q : (kCache && kind == 2 ? p.v : p.k); };

  // What is known of an item when it is fetched: whether its row is of a sequence, and (cache) its
  // place: page (-1: none) and token in it.
  struct Item {
    int seq, page, in;
  };
  Item items[kAhead + 1];
  RowCursor cursor;
  auto fetch_next = [&](int stage) {
    Item it{-1, -1, 0};
    if (ahead.more()) {
      const unsigned ft = ahead.t, fpart = ahead.part;
      int block;
      const int kind = kind_of((int)fpart, block);
      const HeadRows& h = rows_of(kind);
      cursor.move(p.cu, p.padded, p.B, (int)ft);
      it.seq = cursor.span.seq;
      bool read = it.seq >= 0;
      if (read) {
        long long pos = (long long)ft - cursor.span.from + (p.offsets ? p.offsets[it.seq] : 0);
        if (kCache && kind != 0) {
          const long long page_at = pos / p.page_size;
          if (pos >= 0 && page_at < p.max_pages) {
            it.page = p.table[(long long)it.seq * p.table_stride + page_at];
            it.in = (int)(pos - page_at * p.page_size);
          }
          read = it.page >= 0 && it.page < p.num_pages;
          if (!read) it.page = -1;
        }
        if (read && kind != 2 && lane < (p.rotary >> 4))
          fetch_angles(&ring[stage].angle[0][lane], LPH, p, lane, kCache && p.positions ? (long long)p.positions[ft] : pos);
      }
      if (read && mine) {
        const DT* src = static_cast<const DT*>(h.src) + (long long)ft * h.src_stride;
        const int head0 = block * (kRowPasses * kPerPass) + lane / LPH;
#pragma unroll
        for (int i = 0; i < kRowPasses; ++i) {
          const int head = head0 + i * kPerPass;
          if (head < h.heads) {
            copy16(&ring[stage].x[i][0][lane], src + (long long)head * p.d + 8 * c0);
            copy16(&ring[stage].x[i][1][lane], src + (long long)head * p.d + 8 * c1);
          }
        }
      }
      ahead.next();
    }
    cp_async_commit();
    items[kAhead] = it;
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    fetch_next(i);
    items[i] = items[kAhead];
  }
  int stage = 0, turn_kind = -1;
  Turn turn;
  for (; now.more(); now.next()) {
    const unsigned t = now.t, part = now.part;
    __syncwarp();   // the stage filled now was read by every lane
    fetch_next(stage == 0 ? kRowStages - 1 : stage - 1);
    int block;
    const int kind = kind_of((int)part, block);
    const HeadRows& h = rows_of(kind);
    const Item it = items[0];
    DT* dst;
    long long dst_head = p.d;
    bool store = true;
    if (kCache && kind != 0) {   // a row without a page is not written
      store = it.page >= 0;
      dst = kind == 1 ? static_cast<DT*>(p.k_cache) + it.page * p.k_page + it.in * p.k_token
                      : static_cast<DT*>(p.v_cache) + it.page * p.v_page + it.in * p.v_token;
      dst_head = kind == 1 ? p.k_head : p.v_head;
    } else {
      dst = static_cast<DT*>(h.dst) + (long long)t * h.dst_stride;
    }
    const bool norm = kind != 2 && h.weight != nullptr;
    const bool turns = kind != 2 && p.rotary > 0;
    const bool rot = turns && slot < (p.rotary >> 4);
    const int head0 = block * (kRowPasses * kPerPass);
    DT* out = dst + (head0 + lane / LPH) * dst_head;
    cp_async_wait<kAhead>();
    __syncwarp();
    if (store && it.seq < 0) {
#pragma unroll
      for (int i = 0; i < kRowPasses; ++i) {
        if (mine && head0 + i * kPerPass + lane / LPH < h.heads) {
          *reinterpret_cast<uint4*>(out + i * kPerPass * dst_head + 8 * c0) = make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(out + i * kPerPass * dst_head + 8 * c1) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    } else if (store) {
      const auto& st = ring[stage];
      if ((norm || turns) && (block == 0 || turn_kind != kind)) {   // a row's blocks of one kind turn alike
        f2 c[4], s[4], w0[4], w1[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w0[e] = w1[e] = pair(1.f, 1.f);
        if (norm && mine) {
          load_weight<DT>(h.weight, p.weight_fp32, c0, w0);
          load_weight<DT>(h.weight, p.weight_fp32, c1, w1);
        }
        if (rot) {
          read_angles(&st.angle[0][slot], LPH, c, s);
          if (p.sin_sign < 0.f) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[e] = negated(s[e]);
          }
        }
        make_turn(turn, c, s, w0, w1, rot, p.interleaved);
        turn_kind = kind;
      }
      // two passes at a time, side by side
#pragma unroll
      for (int i = 0; i < kRowPasses; i += 2) {
        if (head0 + i * kPerPass >= h.heads) break;
        uint4 v[2][2];
        bool have[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          have[k] = mine && head0 + (i + k) * kPerPass + lane / LPH < h.heads;
          v[k][0] = v[k][1] = make_uint4(0u, 0u, 0u, 0u);
          if (have[k]) {
            v[k][0] = st.x[i + k][0][lane];
            v[k][1] = st.x[i + k][1][lane];
          }
        }
        if (norm || turns) {
          f2 y[2][2][4];
          float sum[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            f2 x0[4], x1[4];
            unpack4<DT>(v[k][0], x0);
            unpack4<DT>(v[k][1], x1);
            apply_turn(turn, x0, x1, y[k][0], y[k][1], rot, p.interleaved);
            f2 sq = mul2(x0[0], x0[0]), sq1 = mul2(x1[0], x1[0]);
#pragma unroll
            for (int e = 1; e < 4; ++e) {
              sq = fma2(x0[e], x0[e], sq);
              sq1 = fma2(x1[e], x1[e], sq1);
            }
            const float2 sqs = split(add2(sq, sq1));
            sum[k] = sqs.x + sqs.y;
          }
          if (norm) {
#pragma unroll
            for (int o = LPH / 2; o > 0; o >>= 1) {
#pragma unroll
              for (int k = 0; k < 2; ++k) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], o);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float r = rsqrtf(sum[k] * p.inv_d + p.eps);
              const f2 rr = pair(r, r);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                y[k][0][e] = mul2(y[k][0][e], rr);
                y[k][1][e] = mul2(y[k][1][e], rr);
              }
            }
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            v[k][0] = pack4<DT>(y[k][0]);
            v[k][1] = pack4<DT>(y[k][1]);
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (have[k]) {
            *reinterpret_cast<uint4*>(out + (i + k) * kPerPass * dst_head + 8 * c0) = v[k][0];
            *reinterpret_cast<uint4*>(out + (i + k) * kPerPass * dst_head + 8 * c1) = v[k][1];
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) items[i] = items[i + 1];
    stage = stage == kRowStages - 1 ? 0 : stage + 1;
  }
  cp_async_wait<0>();
}

// ---------------------------------------------------------------------------- few heads
// Where a row's heads would leave most lanes of an item idle (a model split over many GPUs, keys of
// one or two heads), an item takes as many whole rows as fit, and each lane group finds its row itself.

// The rows and heads of a lane's passes: pair i kPerPass + group of the item's (row, head) pairs.
template <int kPasses>
struct LaneRows {
  int tok[kPasses], head[kPasses];   // row of the item (or -1: nothing), head
  int seq[kPasses];                  // sequence of the row, -1: none
  long long pos[kPasses];            // place in it

  template <int LPH>
  __device__ __forceinline__ void find(const RowArgs& p, int heads, int rows, int block, unsigned t0, bool mine) {
    constexpr int kPerPass = 32 / LPH;
    const int group = (threadIdx.x & 31) / LPH;
    const long long end = min((long long)p.T, (long long)t0 + rows);
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int pair = i * kPerPass + group;
      tok[i] = rows > 1 ? pair / heads : 0;
      head[i] = rows > 1 ? pair - tok[i] * heads : block * (kPasses * kPerPass) + pair;
      if (!mine || tok[i] >= rows || head[i] >= heads || t0 + tok[i] >= end) tok[i] = -1;
      seq[i] = -1;
      pos[i] = 0;
    }
    for (long long t = t0; t < end;) {   // once for each stretch of rows of one sequence, or of none
      const RowSpan span = find_span(p.cu, p.padded, p.B, (int)t);
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const long long row = (long long)t0 + tok[i];
        if (span.seq >= 0 && tok[i] >= 0 && row >= t && row < span.to) {
          seq[i] = span.seq;
          pos[i] = row - span.from;
        }
      }
      t = span.to;
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
      if (seq[i] >= 0 && p.offsets) pos[i] += p.offsets[seq[i]];
  }
};

// A lane's angles, read at once; turned back where sin_sign is -1.
__device__ __forceinline__ void load_angles(f2* c, f2* s, const RowArgs& p, int slot, long long pos) {
  const long long row = pos < 0 ? 0 : (pos >= p.rope_rows ? p.rope_rows - 1 : pos);
  const int half = p.rotary >> 1;
  const long long at[2] = {row * half + (p.interleaved ? 4 * slot : 8 * slot),
                           row * half + (p.interleaved ? 4 * (slot + (p.rotary >> 4)) : 8 * slot + 4)};
  const f2 sign = pair(p.sin_sign, p.sin_sign);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(p.cos + at[i]);
    const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(p.sin + at[i]);
    c[2 * i] = a.x, c[2 * i + 1] = a.y;
    s[2 * i] = mul2(b.x, sign), s[2 * i + 1] = mul2(b.y, sign);
  }
}

// Turns a lane's two chunks.
__device__ __forceinline__ void turn_chunks(f2* x0, f2* x1, const f2* c, const f2* s, int interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 cl = split(c[i >> 1]), sl = split(s[i >> 1]), ch = split(c[2 + (i >> 1)]), sh = split(s[2 + (i >> 1)]);
      const float c0 = i & 1 ? cl.y : cl.x, s0 = i & 1 ? sl.y : sl.x, c1 = i & 1 ? ch.y : ch.x, s1 = i & 1 ? sh.y : sh.x;
      x0[i] = fma2(swapped(x0[i]), pair(-s0, s0), mul2(x0[i], pair(c0, c0)));
      x1[i] = fma2(swapped(x1[i]), pair(-s1, s1), mul2(x1[i], pair(c1, c1)));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f2 y0 = fma2(x1[i], negated(s[i]), mul2(x0[i], c[i]));
      x1[i] = fma2(x0[i], s[i], mul2(x1[i], c[i]));
      x0[i] = y0;
    }
  }
}

// A warp takes one item: queries' first, then keys', then values'.  Nothing is on the way while a warp looks
// for its rows, which other warps have to cover: five blocks an SM (96 registers a thread, up to 148 bytes
// spilled) reach 0.55 of the copy's rate at 1 + 1, 4 + 1 and 8 + 1 heads of 128 and 64, four
// blocks without spills 0.52.  Into a cache: four, 0.55 to 0.64.
template <typename DT, int LPH, bool kCache>
__global__ void __launch_bounds__(kRowWarps * 32, kCache ? 4 : 5) few_heads_kernel(const RowArgs p) {
  const int lane = threadIdx.x & 31;
  unsigned item = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  int kind = 0, rows = p.q_rows, blocks = p.q_items;
  const HeadRows* h = &p.q;
  if (item >= p.q_total) {
    item -= p.q_total;
    kind = 1, rows = p.k_rows, blocks = p.k_items, h = &p.k;
    if (item >= p.k_total) {
      item -= p.k_total;
      if (!kCache || item >= p.v_total) return;
      kind = 2, rows = p.v_rows, blocks = (int)(p.v_total / (unsigned)(((long long)p.T + rows - 1) / rows)), h = &p.v;
    }
  }
  const unsigned first = item / (unsigned)blocks;
  const int block = (int)(item - first * (unsigned)blocks);
  const unsigned t0 = first * (unsigned)rows;
  const int slot = lane % LPH;
  const bool mine = slot < (p.d >> 4);
  int c0, c1;
  lane_chunks(slot, p.rotary, p.d, c0, c1);
  LaneRows<kRowPasses> at;
  at.find<LPH>(p, h->heads, rows, block, t0, mine);
  uint4 v[kRowPasses][2];
  DT* dst[kRowPasses];
#pragma unroll
  for (int i = 0; i < kRowPasses; ++i) {
    const long long t = (long long)t0 + at.tok[i];
    v[i][0] = v[i][1] = make_uint4(0u, 0u, 0u, 0u);
    dst[i] = nullptr;
    if (at.tok[i] < 0) continue;
    if (kCache && kind != 0) {   // a row without a page is not written
      const long long page_at = at.pos[i] / p.page_size;
      int page = -1;
      if (at.seq[i] >= 0 && at.pos[i] >= 0 && page_at < p.max_pages)
        page = p.table[(long long)at.seq[i] * p.table_stride + page_at];
      if (page < 0 || page >= p.num_pages) continue;
      const long long in = at.pos[i] - page_at * p.page_size;
      dst[i] = kind == 1 ? static_cast<DT*>(p.k_cache) + page * p.k_page + in * p.k_token + at.head[i] * p.k_head
                         : static_cast<DT*>(p.v_cache) + page * p.v_page + in * p.v_token + at.head[i] * p.v_head;
    } else {
      dst[i] = static_cast<DT*>(h->dst) + t * h->dst_stride + (long long)at.head[i] * p.d;
    }
    if (at.seq[i] >= 0) {
      const DT* src = static_cast<const DT*>(h->src) + t * h->src_stride + (long long)at.head[i] * p.d;
      v[i][0] = *reinterpret_cast<const uint4*>(src + 8 * c0);
      v[i][1] = *reinterpret_cast<const uint4*>(src + 8 * c1);
    }
  }
  const bool norm = kind != 2 && h->weight != nullptr;
  const bool rot = kind != 2 && slot < (p.rotary >> 4);
  if (norm || (kind != 2 && p.rotary > 0)) {
    f2 w0[4], w1[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w0[e] = w1[e] = pair(1.f, 1.f);
    if (norm && mine) {
      load_weight<DT>(h->weight, p.weight_fp32, c0, w0);
      load_weight<DT>(h->weight, p.weight_fp32, c1, w1);
    }
#pragma unroll
    for (int i = 0; i < kRowPasses; ++i) {
      f2 x0[4], x1[4], c[4], s[4];
      const bool row = at.tok[i] >= 0 && at.seq[i] >= 0;
      if (row && rot)
        load_angles(c, s, p, slot, kCache && p.positions ? (long long)p.positions[(long long)t0 + at.tok[i]] : at.pos[i]);
      unpack4<DT>(v[i][0], x0);
      unpack4<DT>(v[i][1], x1);
      if (norm) {
        f2 sq = mul2(x0[0], x0[0]), sq1 = mul2(x1[0], x1[0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) {
          sq = fma2(x0[e], x0[e], sq);
          sq1 = fma2(x1[e], x1[e], sq1);
        }
        const float2 sqs = split(add2(sq, sq1));
        float sum = sqs.x + sqs.y;
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float r = rsqrtf(sum * p.inv_d + p.eps);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x0[e] = mul2(mul2(x0[e], w0[e]), pair(r, r));
          x1[e] = mul2(mul2(x1[e], w1[e]), pair(r, r));
        }
      }
      if (row && rot) turn_chunks(x0, x1, c, s, p.interleaved);
      if (row) {
        v[i][0] = pack4<DT>(x0);
        v[i][1] = pack4<DT>(x1);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kRowPasses; ++i) {
    if (dst[i]) {
      *reinterpret_cast<uint4*>(dst[i] + 8 * c0) = v[i][0];
      *reinterpret_cast<uint4*>(dst[i] + 8 * c1) = v[i][1];
    }
  }
}

// ---------------------------------------------------------------------------- backward
struct NormBwdArgs {
  RowArgs a;                 // src: x, dst: dx
  const void* gq;            // packed gradients of the outputs
  const void* gk;
  float* partial;            // [blocks][d]
  int q_blocks, k_blocks;
  unsigned run;              // items of a warp
};

constexpr int kBwdPasses = 2;
constexpr int kBwdWarps = 4;
constexpr int kBwdStages = 3;
// As kFewShare: 4 + 1 heads (31 %) 35 and 58, 8 + 1 (56 %) 58 and 63, 8 + 2 (62 %) 64 and 63, 16 + 2 (75 %) 75 and 65.
constexpr int kBwdFewShare = 60;
constexpr int kBwdRun = 6;        // items of a warp, more where that would give over kBwdMaxBlocks blocks
constexpr int kBwdBlocksPerSm = 3;
constexpr int kBwdMaxBlocks = 4096;

// The block's share of dw: over the warp's heads, then over the warps.
template <int LPH>
__device__ __forceinline__ void leave_weight_share(const f2* dw0, const f2* dw1, float (*sum)[128], int c0, int c1,
                                                   bool mine, float* dst, int d) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float2 a = split(dw0[e]), c = split(dw1[e]);
#pragma unroll
    for (int o = LPH; o < 32; o <<= 1) {
      a.x += __shfl_xor_sync(0xffffffffu, a.x, o);
      a.y += __shfl_xor_sync(0xffffffffu, a.y, o);
      c.x += __shfl_xor_sync(0xffffffffu, c.x, o);
      c.y += __shfl_xor_sync(0xffffffffu, c.y, o);
    }
    if (lane < LPH && mine) {
      sum[warp][8 * c0 + 2 * e] = a.x;
      sum[warp][8 * c0 + 2 * e + 1] = a.y;
      sum[warp][8 * c1 + 2 * e] = c.x;
      sum[warp][8 * c1 + 2 * e + 1] = c.y;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < d; i += blockDim.x) {
    float total = 0.f;
#pragma unroll
    for (int k = 0; k < kBwdWarps; ++k) total += sum[k][i];
    dst[i] = total;
  }
}

// A block works on one kind (queries or keys), so that a lane keeps one sum for dw.  Copies ahead as
// the forward does: gradients in chunks 0 and 1 of a stage, inputs in 2 and 3.
template <typename DT, int LPH>
__global__ void __launch_bounds__(kBwdWarps * 32, kBwdBlocksPerSm) head_rows_bwd_kernel(const NormBwdArgs b) {
  constexpr int kPerPass = 32 / LPH;
  constexpr int kAhead = kBwdStages - 1;
  extern __shared__ __align__(16) unsigned char smem[];
  const RowArgs& p = b.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto* ring = reinterpret_cast<RowStage<kBwdPasses, 4, LPH>*>(smem) + warp * kBwdStages;
  const bool is_q = (int)blockIdx.x < b.q_blocks;
  const HeadRows& h = is_q ? p.q : p.k;
  const DT* grad = static_cast<const DT*>(is_q ? b.gq : b.gk);
  const unsigned row_items = (unsigned)(is_q ? p.q_items : p.k_items);
  ItemWalk ahead((unsigned)p.T * row_items, row_items, (is_q ? blockIdx.x : blockIdx.x - b.q_blocks) * kBwdWarps + warp,
                 b.run);
  ItemWalk now = ahead;
  const int slot = lane % LPH;
  const bool mine = slot < (p.d >> 4);
  const bool norm = h.weight != nullptr;
  const bool rot = slot < (p.rotary >> 4);
  int c0, c1;
  lane_chunks(slot, p.rotary, p.d, c0, c1);
  f2 w0[4], w1[4], dw0[4], dw1[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w0[e] = w1[e] = dw0[e] = dw1[e] = 0ull;
  if (norm && mine) {
    load_weight<DT>(h.weight, p.weight_fp32, c0, w0);
    load_weight<DT>(h.weight, p.weight_fp32, c1, w1);
  }
  RowCursor cursor;
  bool inside[kAhead + 1];   // whether the item's row is of a sequence
  auto fetch_next = [&](int stage) {
    bool in = false;
    if (ahead.more()) {
      const unsigned ft = ahead.t, fpart = ahead.part;
      cursor.move(p.cu, p.padded, p.B, (int)ft);
      in = cursor.span.seq >= 0;
      if (in) {
        if (lane < (p.rotary >> 4))
          fetch_angles(&ring[stage].angle[0][lane], LPH, p, lane,
                       (long long)ft - cursor.span.from + (p.offsets ? p.offsets[cursor.span.seq] : 0));
        const DT* src = static_cast<const DT*>(h.src) + (long long)ft * h.src_stride;
        const DT* gsrc = grad + (long long)ft * h.heads * p.d;
#pragma unroll
        for (int i = 0; i < kBwdPasses; ++i) {
          const int head = ((int)fpart * kBwdPasses + i) * kPerPass + lane / LPH;
          if (mine && head < h.heads) {
            const long long at = (long long)head * p.d;
            copy16(&ring[stage].x[i][0][lane], gsrc + at + 8 * c0);
            copy16(&ring[stage].x[i][1][lane], gsrc + at + 8 * c1);
            if (norm) {
              copy16(&ring[stage].x[i][2][lane], src + at + 8 * c0);
              copy16(&ring[stage].x[i][3][lane], src + at + 8 * c1);
            }
          }
        }
      }
      ahead.next();
    }
    cp_async_commit();
    inside[kAhead] = in;
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    fetch_next(i);
    inside[i] = inside[kAhead];
  }
  int stage = 0;
  for (; now.more(); now.next()) {
    const unsigned t = now.t, part = now.part;
    __syncwarp();   // the stage filled now was read by every lane
    fetch_next(stage == 0 ? kBwdStages - 1 : stage - 1);
    const int head0 = (int)part * (kBwdPasses * kPerPass);
    DT* out = static_cast<DT*>(h.dst) + (long long)t * h.dst_stride + (long long)(head0 + lane / LPH) * p.d;
    cp_async_wait<kAhead>();
    __syncwarp();
    if (!inside[0]) {
#pragma unroll
      for (int i = 0; i < kBwdPasses; ++i) {
        if (mine && head0 + i * kPerPass + lane / LPH < h.heads) {
          *reinterpret_cast<uint4*>(out + (long long)i * kPerPass * p.d + 8 * c0) = make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(out + (long long)i * kPerPass * p.d + 8 * c1) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    } else {
      const auto& st = ring[stage];
      f2 c[4], s[4];
      if (rot) read_angles(&st.angle[0][slot], LPH, c, s);
      f2 h0[kBwdPasses][4], h1[kBwdPasses][4], x0[kBwdPasses][4], x1[kBwdPasses][4];
      float sum[kBwdPasses], along[kBwdPasses];
      bool have[kBwdPasses];
#pragma unroll
      for (int i = 0; i < kBwdPasses; ++i) {
        have[i] = mine && head0 + i * kPerPass + lane / LPH < h.heads;
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[k] = make_uint4(0u, 0u, 0u, 0u);
          if (have[i] && (k < 2 || norm)) v[k] = st.x[i][k][lane];
        }
        f2 g0[4], g1[4];
        unpack4<DT>(v[0], g0);
        unpack4<DT>(v[1], g1);
        unpack4<DT>(v[2], x0[i]);
        unpack4<DT>(v[3], x1[i]);
        if (rot) {   // turned back
          if (p.interleaved) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 cl = split(c[e >> 1]), sl = split(s[e >> 1]);
              const float2 ch = split(c[2 + (e >> 1)]), sh = split(s[2 + (e >> 1)]);
              const float ca = e & 1 ? cl.y : cl.x, sa = e & 1 ? sl.y : sl.x;
              const float cb = e & 1 ? ch.y : ch.x, sb = e & 1 ? sh.y : sh.x;
              h0[i][e] = fma2(swapped(g0[e]), pair(sa, -sa), mul2(g0[e], pair(ca, ca)));
              h1[i][e] = fma2(swapped(g1[e]), pair(sb, -sb), mul2(g1[e], pair(cb, cb)));
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              h0[i][e] = fma2(g1[e], s[e], mul2(g0[e], c[e]));
              h1[i][e] = fma2(negated(g0[e]), s[e], mul2(g1[e], c[e]));
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) h0[i][e] = g0[e], h1[i][e] = g1[e];
        }
        f2 sq0 = 0ull, sq1 = 0ull, dot0 = 0ull, dot1 = 0ull;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sq0 = fma2(x0[i][e], x0[i][e], sq0);
          sq1 = fma2(x1[i][e], x1[i][e], sq1);
          dot0 = fma2(mul2(h0[i][e], w0[e]), x0[i][e], dot0);
          dot1 = fma2(mul2(h1[i][e], w1[e]), x1[i][e], dot1);
        }
        const float2 sqs = split(add2(sq0, sq1)), dots = split(add2(dot0, dot1));
        sum[i] = sqs.x + sqs.y;
        along[i] = dots.x + dots.y;
      }
      if (norm) {
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) {
#pragma unroll
          for (int i = 0; i < kBwdPasses; ++i) {
            sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
            along[i] += __shfl_xor_sync(0xffffffffu, along[i], o);
          }
        }
#pragma unroll
        for (int i = 0; i < kBwdPasses; ++i) {
          // past the last head there is nothing, and with eps = 0 its 1 / rms has no value
          const float r = head0 + i * kPerPass + lane / LPH < h.heads ? rsqrtf(sum[i] * p.inv_d + p.eps) : 0.f;
          const float m = -(along[i] * p.inv_d * r) * r * r;   // in an order that stays in range for tiny heads
          const f2 rr = pair(r, r), mm = pair(m, m);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const f2 hr0 = mul2(h0[i][e], rr), hr1 = mul2(h1[i][e], rr);
            dw0[e] = fma2(hr0, x0[i][e], dw0[e]);
            dw1[e] = fma2(hr1, x1[i][e], dw1[e]);
            h0[i][e] = fma2(hr0, w0[e], mul2(x0[i][e], mm));
            h1[i][e] = fma2(hr1, w1[e], mul2(x1[i][e], mm));
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kBwdPasses; ++i) {
        if (have[i]) {
          *reinterpret_cast<uint4*>(out + (long long)i * kPerPass * p.d + 8 * c0) = pack4<DT>(h0[i]);
          *reinterpret_cast<uint4*>(out + (long long)i * kPerPass * p.d + 8 * c1) = pack4<DT>(h1[i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) inside[i] = inside[i + 1];
    stage = stage == kBwdStages - 1 ? 0 : stage + 1;
  }
  cp_async_wait<0>();
  if (!norm) return;
  __syncthreads();   // the ring is read no more
  leave_weight_share<LPH>(dw0, dw1, reinterpret_cast<float(*)[128]>(smem), c0, c1, mine,
                          b.partial + (long long)blockIdx.x * p.d, p.d);
}

// Few heads, as few_heads_kernel; a block works on one kind and a warp on a run of items.
template <typename DT, int LPH>
__global__ void __launch_bounds__(kBwdWarps * 32) few_heads_bwd_kernel(const NormBwdArgs b) {
  const RowArgs& p = b.a;
  __shared__ float sum[kBwdWarps][128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool is_q = (int)blockIdx.x < b.q_blocks;
  const HeadRows& h = is_q ? p.q : p.k;
  const DT* grad = static_cast<const DT*>(is_q ? b.gq : b.gk);
  const int rows = is_q ? p.q_rows : p.k_rows;
  const unsigned blocks = (unsigned)(is_q ? p.q_items : p.k_items);
  const int slot = lane % LPH;
  const bool mine = slot < (p.d >> 4);
  const bool norm = h.weight != nullptr;
  const bool rot = slot < (p.rotary >> 4);
  int c0, c1;
  lane_chunks(slot, p.rotary, p.d, c0, c1);
  f2 w0[4], w1[4], dw0[4], dw1[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w0[e] = w1[e] = dw0[e] = dw1[e] = 0ull;
  if (norm && mine) {
    load_weight<DT>(h.weight, p.weight_fp32, c0, w0);
    load_weight<DT>(h.weight, p.weight_fp32, c1, w1);
  }
  // row_items of the walk: blocks of heads of a group of rows
  for (ItemWalk now(is_q ? p.q_total : p.k_total, blocks, (is_q ? blockIdx.x : blockIdx.x - b.q_blocks) * kBwdWarps + warp,
                    b.run);
       now.more(); now.next()) {
    const unsigned t0 = now.t * (unsigned)rows;
    LaneRows<kBwdPasses> at;
    at.find<LPH>(p, h.heads, rows, (int)now.part, t0, mine);
    uint4 g[kBwdPasses][2], v[kBwdPasses][2];
#pragma unroll
    for (int i = 0; i < kBwdPasses; ++i) {
      g[i][0] = g[i][1] = v[i][0] = v[i][1] = make_uint4(0u, 0u, 0u, 0u);
      if (at.tok[i] >= 0 && at.seq[i] >= 0) {
        const long long t = (long long)t0 + at.tok[i], head = (long long)at.head[i] * p.d;
        const DT* gsrc = grad + t * h.heads * p.d + head;
        g[i][0] = *reinterpret_cast<const uint4*>(gsrc + 8 * c0);
        g[i][1] = *reinterpret_cast<const uint4*>(gsrc + 8 * c1);
        if (norm) {
          const DT* src = static_cast<const DT*>(h.src) + t * h.src_stride + head;
          v[i][0] = *reinterpret_cast<const uint4*>(src + 8 * c0);
          v[i][1] = *reinterpret_cast<const uint4*>(src + 8 * c1);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kBwdPasses; ++i) {
      const bool row = at.tok[i] >= 0 && at.seq[i] >= 0;
      f2 h0[4], h1[4];
      unpack4<DT>(g[i][0], h0);
      unpack4<DT>(g[i][1], h1);
      if (row && rot) {
        f2 c[4], s[4];
        load_angles(c, s, p, slot, at.pos[i]);   // turned back (sin_sign)
        turn_chunks(h0, h1, c, s, p.interleaved);
      }
      if (norm) {
        f2 x0[4], x1[4];
        unpack4<DT>(v[i][0], x0);
        unpack4<DT>(v[i][1], x1);
        f2 sq0 = 0ull, sq1 = 0ull, dot0 = 0ull, dot1 = 0ull;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sq0 = fma2(x0[e], x0[e], sq0);
          sq1 = fma2(x1[e], x1[e], sq1);
          dot0 = fma2(mul2(h0[e], w0[e]), x0[e], dot0);
          dot1 = fma2(mul2(h1[e], w1[e]), x1[e], dot1);
        }
        const float2 sqs = split(add2(sq0, sq1)), dots = split(add2(dot0, dot1));
        float ss = sqs.x + sqs.y, along = dots.x + dots.y;
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) {
          ss += __shfl_xor_sync(0xffffffffu, ss, o);
          along += __shfl_xor_sync(0xffffffffu, along, o);
        }
        // where there is no row there is nothing, and with eps = 0 its 1 / rms has no value; lanes past the
        // head's chunks hold zeros
        const float r = row ? rsqrtf(ss * p.inv_d + p.eps) : 0.f;
        const float m = -(along * p.inv_d * r) * r * r;   // in an order that stays in range for tiny heads
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f2 hr0 = mul2(h0[e], pair(r, r)), hr1 = mul2(h1[e], pair(r, r));
          dw0[e] = fma2(hr0, x0[e], dw0[e]);
          dw1[e] = fma2(hr1, x1[e], dw1[e]);
          h0[e] = fma2(hr0, w0[e], mul2(x0[e], pair(m, m)));
          h1[e] = fma2(hr1, w1[e], mul2(x1[e], pair(m, m)));
        }
      }
      if (at.tok[i] >= 0) {
        DT* dst = static_cast<DT*>(h.dst) + ((long long)t0 + at.tok[i]) * h.dst_stride + (long long)at.head[i] * p.d;
        *reinterpret_cast<uint4*>(dst + 8 * c0) = row ? pack4<DT>(h0) : make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(dst + 8 * c1) = row ? pack4<DT>(h1) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
  if (norm) leave_weight_share<LPH>(dw0, dw1, sum, c0, c1, mine, b.partial + (long long)blockIdx.x * p.d, p.d);
}

// dw = the blocks' shares summed in a fixed order; a block takes 8 columns of one kind.
constexpr int kSumRows = 128;
__global__ void __launch_bounds__(kSumRows * 8) weight_sum_kernel(const float* __restrict__ partial, int q_blocks,
                                                                  int k_blocks, int d, float* dwq, float* dwk) {
  const int kind = blockIdx.y;
  float* dst = kind == 0 ? dwq : dwk;
  if (!dst) return;
  const int col = blockIdx.x * 8 + (threadIdx.x & 7), row = threadIdx.x >> 3;
  const int begin = kind == 0 ? 0 : q_blocks, n = kind == 0 ? q_blocks : k_blocks;
  __shared__ float part[kSumRows][9];
  float s = 0.f;
#pragma unroll 8
  for (int i = row; i < n; i += kSumRows) s += partial[(long long)(begin + i) * d + col];
  part[row][threadIdx.x & 7] = s;
  __syncthreads();
#pragma unroll
  for (int half = kSumRows / 2; half > 0; half >>= 1) {
    if (row < half) part[row][threadIdx.x & 7] += part[row + half][threadIdx.x & 7];
    __syncthreads();
  }
  if (row == 0) dst[col] = part[0][threadIdx.x];
}

// ---------------------------------------------------------------------------- host
int lanes_per_head(int d) { return d <= 16 ? 1 : (d <= 32 ? 2 : (d <= 64 ? 4 : 8)); }

// The checks the three entry points share.
int check_common(int B, int T, int hq, int hkv, int d, int dtype, float eps, const void* wq, const void* wk,
                 int weight_fp32, const float* cos, const float* sin, int rope_rows, int rotary, const int32_t* cu,
                 const int32_t* padded, const int32_t* offsets) {
  if (B < 0 || T < 0 || hq < 0 || hkv < 0) return THD_ERR_ARG;
  if (dtype != THD_BF16 && dtype != THD_FP16) return THD_ERR_UNSUPPORTED;
  if (weight_fp32 != 0 && weight_fp32 != 1) return THD_ERR_ARG;
  if (d < 16 || d > 128 || d % 16 != 0) return THD_ERR_UNSUPPORTED;
  if (rotary < 0 || rotary > d || rotary % 16 != 0) return THD_ERR_UNSUPPORTED;
  if ((long long)hq * d >= (1ll << 31) || (long long)hkv * d >= (1ll << 31)) return THD_ERR_UNSUPPORTED;
  if ((wq || wk) && (!std::isfinite(eps) || eps < 0.f)) return THD_ERR_ARG;
  if (rotary > 0 && (!cos || !sin || rope_rows < 1)) return THD_ERR_ARG;
  if (rotary > 0 && (!on16(cos) || !on16(sin))) return THD_ERR_ARG;
  if ((wq && !on16(wq)) || (wk && !on16(wk))) return THD_ERR_ARG;
  if (!on4(cu) || !on4(padded) || !on4(offsets)) return THD_ERR_ARG;
  if (T > 0 && B > 0 && !cu) return THD_ERR_ARG;
  return THD_OK;
}

// Rows of `heads` heads: present, aligned, rows that do not overlap.
int check_rows(const void* x, long long stride, int heads, int d) {
  if (heads == 0) return THD_OK;
  if (!x || !on16(x) || stride < (long long)heads * d || stride % 8 != 0) return THD_ERR_ARG;
  return THD_OK;
}

int blocks_of_heads(int heads, int per) { return (heads + per - 1) / per; }

void fill_common(RowArgs& p, int B, int T, int d, float eps, int weight_fp32, const float* cos, const float* sin,
                 int rope_rows, int rotary, int interleaved, const int32_t* cu, const int32_t* padded,
                 const int32_t* offsets) {
  p.cos = cos;
  p.sin = sin;
  p.cu = cu;
  p.padded = padded;
  p.offsets = offsets;
  p.rope_rows = rope_rows;
  p.eps = eps;
  p.inv_d = 1.f / (float)d;
  p.sin_sign = 1.f;
  p.T = T;
  p.B = B;
  p.d = d;
  p.rotary = rotary;
  p.interleaved = interleaved;
  p.weight_fp32 = weight_fp32;
}

template <typename DT, int LPH, bool kCache>
int launch_rows_at(const RowArgs& p, unsigned grid, cudaStream_t st) {
  static SmemGrant grant;
  constexpr size_t smem = kRowWarps * kRowStages * sizeof(RowStage<kRowPasses, 2, LPH>);
  if (!grant.ask(head_rows_kernel<DT, LPH, kCache>, smem)) return THD_ERR_CUDA;
  head_rows_kernel<DT, LPH, kCache><<<grid, kRowWarps * 32, smem, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? THD_OK : THD_ERR_CUDA;
}

template <typename DT, int LPH, bool kCache>
int launch_few_at(const RowArgs& p, unsigned grid, cudaStream_t st) {
  few_heads_kernel<DT, LPH, kCache><<<grid, kRowWarps * 32, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? THD_OK : THD_ERR_CUDA;
}

template <typename DT, bool kCache>
int launch_few_of(const RowArgs& p, unsigned grid, cudaStream_t st) {
  switch (lanes_per_head(p.d)) {
    case 1: return launch_few_at<DT, 1, kCache>(p, grid, st);
    case 2: return launch_few_at<DT, 2, kCache>(p, grid, st);
    case 4: return launch_few_at<DT, 4, kCache>(p, grid, st);
    default: return launch_few_at<DT, 8, kCache>(p, grid, st);
  }
}

// Whether items of whole rows pay: kPasses * 32 / lanes-per-head pairs (`per`) fit one.
bool few_heads(const RowArgs& p, int per, int share) {
  const long long items = blocks_of_heads(p.q.heads, per) + blocks_of_heads(p.k.heads, per) + blocks_of_heads(p.v.heads, per);
  return 100ll * (p.q.heads + p.k.heads + p.v.heads) < share * per * items;
}

// Rows of an item and items of a kind of `heads` heads.
void rows_of_items(int heads, int per, int T, int& rows, long long& total) {
  rows = heads > 0 && per / heads > 1 ? per / heads : 1;
  total = heads > 0 ? ((long long)T + rows - 1) / rows * blocks_of_heads(heads, per) : 0;
}

template <typename DT, bool kCache>
int launch_rows_of(const RowArgs& p, unsigned grid, cudaStream_t st) {
  switch (lanes_per_head(p.d)) {
    case 1: return launch_rows_at<DT, 1, kCache>(p, grid, st);
    case 2: return launch_rows_at<DT, 2, kCache>(p, grid, st);
    case 4: return launch_rows_at<DT, 4, kCache>(p, grid, st);
    default: return launch_rows_at<DT, 8, kCache>(p, grid, st);
  }
}

template <bool kCache>
int launch_rows(RowArgs& p, int dtype, cudaStream_t st) {
  const int per = kRowPasses * (32 / lanes_per_head(p.d));
  p.q_items = blocks_of_heads(p.q.heads, per);
  p.k_items = blocks_of_heads(p.k.heads, per);
  const long long row_items = (long long)p.q_items + p.k_items + blocks_of_heads(p.v.heads, per);
  if (row_items == 0) return THD_OK;
  if (few_heads(p, per, kFewShare)) {
    long long qt, kt, vt;
    rows_of_items(p.q.heads, per, p.T, p.q_rows, qt);
    rows_of_items(p.k.heads, per, p.T, p.k_rows, kt);
    rows_of_items(p.v.heads, per, p.T, p.v_rows, vt);
    if (qt + kt + vt >= (1ll << 31)) return THD_ERR_UNSUPPORTED;   // item numbers are 32-bit
    p.q_total = (unsigned)qt, p.k_total = (unsigned)kt, p.v_total = (unsigned)vt;
    const unsigned grid = (unsigned)((qt + kt + vt + kRowWarps - 1) / kRowWarps);
    return dtype == THD_BF16 ? launch_few_of<__nv_bfloat16, kCache>(p, grid, st)
                             : launch_few_of<__half, kCache>(p, grid, st);
  }
  const long long items = row_items * p.T;
  if (items >= (1ll << 31)) return THD_ERR_UNSUPPORTED;   // item numbers are 32-bit
  p.row_items = (int)row_items;
  const int sms = device_sms();
  if (sms <= 0) return THD_ERR_CUDA;
  // as many items for a warp as leave all that fit at once one, kRowRun at most
  const long long per_warp = items / ((long long)sms * kRowBlocksPerSm * kRowWarps);
  p.run = per_warp < 1 ? 1u : (per_warp > kRowRun ? (unsigned)kRowRun : (unsigned)per_warp);
  const unsigned grid = (unsigned)((items + (long long)kRowWarps * p.run - 1) / ((long long)kRowWarps * p.run));
  return dtype == THD_BF16 ? launch_rows_of<__nv_bfloat16, kCache>(p, grid, st)
                           : launch_rows_of<__half, kCache>(p, grid, st);
}

template <typename DT, int LPH>
int launch_bwd_at(const NormBwdArgs& b, bool few, unsigned grid, cudaStream_t st) {
  if (few) {
    few_heads_bwd_kernel<DT, LPH><<<grid, kBwdWarps * 32, 0, st>>>(b);
    return cudaGetLastError() == cudaSuccess ? THD_OK : THD_ERR_CUDA;
  }
  static SmemGrant grant;
  constexpr size_t smem = kBwdWarps * kBwdStages * sizeof(RowStage<kBwdPasses, 4, LPH>);
  if (!grant.ask(head_rows_bwd_kernel<DT, LPH>, smem)) return THD_ERR_CUDA;
  head_rows_bwd_kernel<DT, LPH><<<grid, kBwdWarps * 32, smem, st>>>(b);
  return cudaGetLastError() == cudaSuccess ? THD_OK : THD_ERR_CUDA;
}

template <typename DT>
int launch_bwd_of(const NormBwdArgs& b, bool few, unsigned grid, cudaStream_t st) {
  switch (lanes_per_head(b.a.d)) {
    case 1: return launch_bwd_at<DT, 1>(b, few, grid, st);
    case 2: return launch_bwd_at<DT, 2>(b, few, grid, st);
    case 4: return launch_bwd_at<DT, 4>(b, few, grid, st);
    default: return launch_bwd_at<DT, 8>(b, few, grid, st);
  }
}

}  // namespace
}  // namespace thd

extern "C" {

int thd_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* q_weight,
                     const void* k_weight, int weight_fp32, float eps, const float* rope_cos, const float* rope_sin,
                     int rope_rows, int rotary_dim, int interleaved, const int32_t* cu_seqlens,
                     const int32_t* cu_seqlens_padded, const int32_t* position_offsets, int batch_size, void* q_out,
                     void* k_out, int total_tokens, int num_heads_q, int num_heads_kv, int head_dim, int dtype,
                     void* stream) {
  using namespace thd;
  int st = check_common(batch_size, total_tokens, num_heads_q, num_heads_kv, head_dim, dtype, eps, q_weight, k_weight,
                        weight_fp32, rope_cos, rope_sin, rope_rows, rotary_dim, cu_seqlens, cu_seqlens_padded,
                        position_offsets);
  if (st != THD_OK) return st;
  if (num_heads_q + (long long)num_heads_kv < 1) return THD_ERR_ARG;
  if (total_tokens == 0) return THD_OK;
  const long long qd = (long long)num_heads_q * head_dim, kd = (long long)num_heads_kv * head_dim;
  if ((st = check_rows(q, q_stride, num_heads_q, head_dim)) != THD_OK) return st;
  if ((st = check_rows(k, k_stride, num_heads_kv, head_dim)) != THD_OK) return st;
  if ((st = check_rows(q_out, qd, num_heads_q, head_dim)) != THD_OK) return st;
  if ((st = check_rows(k_out, kd, num_heads_kv, head_dim)) != THD_OK) return st;
  RowArgs p{};
  fill_common(p, batch_size, total_tokens, head_dim, eps, weight_fp32, rope_cos, rope_sin, rope_rows, rotary_dim,
              interleaved != 0, cu_seqlens, cu_seqlens_padded, position_offsets);
  p.q = HeadRows{q, q_out, q_weight, q_stride, qd, num_heads_q};
  p.k = HeadRows{k, k_out, k_weight, k_stride, kd, num_heads_kv};
  return launch_rows<false>(p, dtype, static_cast<cudaStream_t>(stream));
}

size_t thd_qk_norm_rope_bwd_workspace_size(int head_dim) {
  if (head_dim < 16 || head_dim > 128 || head_dim % 16 != 0) return 0;
  return (size_t)thd::kBwdMaxBlocks * head_dim * sizeof(float);
}

int thd_qk_norm_rope_bwd(const void* grad_q, const void* grad_k, const void* q, int64_t q_stride, const void* k,
                         int64_t k_stride, const void* q_weight, const void* k_weight, int weight_fp32, float eps,
                         const float* rope_cos, const float* rope_sin, int rope_rows, int rotary_dim, int interleaved,
                         const int32_t* cu_seqlens, const int32_t* cu_seqlens_padded, const int32_t* position_offsets,
                         int batch_size, void* dq, int64_t dq_stride, void* dk, int64_t dk_stride, float* dq_weight,
                         float* dk_weight, int total_tokens, int num_heads_q, int num_heads_kv, int head_dim,
                         int dtype, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace thd;
  int st = check_common(batch_size, total_tokens, num_heads_q, num_heads_kv, head_dim, dtype, eps, q_weight, k_weight,
                        weight_fp32, rope_cos, rope_sin, rope_rows, rotary_dim, cu_seqlens, cu_seqlens_padded,
                        position_offsets);
  if (st != THD_OK) return st;
  if (num_heads_q + (long long)num_heads_kv < 1) return THD_ERR_ARG;
  const bool nq = q_weight && num_heads_q > 0, nk = k_weight && num_heads_kv > 0;
  if (!q_weight != !dq_weight || !k_weight != !dk_weight || !on4(dq_weight) || !on4(dk_weight)) return THD_ERR_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const long long qd = (long long)num_heads_q * head_dim, kd = (long long)num_heads_kv * head_dim;
  if (total_tokens > 0) {
    if ((st = check_rows(grad_q, qd, num_heads_q, head_dim)) != THD_OK) return st;
    if ((st = check_rows(grad_k, kd, num_heads_kv, head_dim)) != THD_OK) return st;
    if (nq && (st = check_rows(q, q_stride, num_heads_q, head_dim)) != THD_OK) return st;
    if (nk && (st = check_rows(k, k_stride, num_heads_kv, head_dim)) != THD_OK) return st;
    if ((st = check_rows(dq, dq_stride, num_heads_q, head_dim)) != THD_OK) return st;
    if ((st = check_rows(dk, dk_stride, num_heads_kv, head_dim)) != THD_OK) return st;
  }
  RowArgs p{};
  fill_common(p, batch_size, total_tokens, head_dim, eps, weight_fp32, rope_cos, rope_sin, rope_rows, rotary_dim,
              interleaved != 0, cu_seqlens, cu_seqlens_padded, position_offsets);
  if (!q_weight && !k_weight) {   // the rotation alone: its transpose is the rotation back
    if (total_tokens == 0) return THD_OK;
    p.sin_sign = -1.f;
    p.q = HeadRows{grad_q, dq, nullptr, qd, dq_stride, num_heads_q};
    p.k = HeadRows{grad_k, dk, nullptr, kd, dk_stride, num_heads_kv};
    return launch_rows<false>(p, dtype, s);
  }
  if (!workspace || !on16(workspace) || workspace_bytes < thd_qk_norm_rope_bwd_workspace_size(head_dim))
    return THD_ERR_WORKSPACE;
  const int sms = device_sms();
  if (sms <= 0) return THD_ERR_CUDA;
  const int per = kBwdPasses * (32 / lanes_per_head(head_dim));
  NormBwdArgs b{};
  p.q = HeadRows{q, dq, q_weight, q_stride, dq_stride, num_heads_q};
  p.k = HeadRows{k, dk, k_weight, k_stride, dk_stride, num_heads_kv};
  p.q_items = blocks_of_heads(num_heads_q, per);
  p.k_items = blocks_of_heads(num_heads_kv, per);
  const bool few = few_heads(p, per, kBwdFewShare);
  long long qi = (long long)p.q_items * total_tokens, ki = (long long)p.k_items * total_tokens;
  if (few) {
    rows_of_items(num_heads_q, per, total_tokens, p.q_rows, qi);
    rows_of_items(num_heads_kv, per, total_tokens, p.k_rows, ki);
    p.sin_sign = -1.f;
  }
  if (qi >= (1ll << 31) || ki >= (1ll << 31)) return THD_ERR_UNSUPPORTED;   // item numbers are 32-bit
  // runs as in launch_rows, but of such a length that there are at most kBwdMaxBlocks blocks: each
  // leaves a share of dw to be summed
  const long long resident = (long long)sms * kBwdBlocksPerSm * kBwdWarps;
  const long long most = (long long)(kBwdMaxBlocks - 2) * kBwdWarps, least = (qi + ki + most - 1) / most;
  long long run = (qi + ki) / resident;
  run = run < 1 ? 1 : (run > kBwdRun ? kBwdRun : run);
  if (run < least) run = least;
  const long long per_block = run * kBwdWarps;
  const long long qb = (qi + per_block - 1) / per_block, kb = (ki + per_block - 1) / per_block;
  p.q_total = (unsigned)qi, p.k_total = (unsigned)ki;
  b.run = (unsigned)run;
  b.a = p;
  b.gq = grad_q;
  b.gk = grad_k;
  b.partial = static_cast<float*>(workspace);
  b.q_blocks = (int)qb;
  b.k_blocks = (int)kb;
  if (qb + kb > 0) {
    st = dtype == THD_BF16 ? launch_bwd_of<__nv_bfloat16>(b, few, (unsigned)(qb + kb), s)
                           : launch_bwd_of<__half>(b, few, (unsigned)(qb + kb), s);
    if (st != THD_OK) return st;
  }
  weight_sum_kernel<<<dim3(head_dim / 8, 2), kSumRows * 8, 0, s>>>(b.partial, b.q_blocks, b.k_blocks, head_dim,
                                                                   dq_weight, dk_weight);
  return cudaGetLastError() == cudaSuccess ? THD_OK : THD_ERR_CUDA;
}

int thd_kv_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                  const void* q_weight, const void* k_weight, int weight_fp32, float eps, const float* rope_cos,
                  const float* rope_sin, int rope_rows, int rotary_dim, int interleaved, const int32_t* positions,
                  const int32_t* cu_seqlens, const int32_t* cu_seqlens_padded, const int32_t* cache_lens,
                  int batch_size, void* q_out, void* k_cache, void* v_cache, const int64_t* cache_strides,
                  int num_pages, int page_size, const int32_t* page_table, int64_t page_table_stride, int max_pages,
                  int total_tokens, int num_heads_q, int num_heads_kv, int head_dim, int dtype, void* stream) {
  using namespace thd;
  int st = check_common(batch_size, total_tokens, num_heads_q, num_heads_kv, head_dim, dtype, eps, q_weight, k_weight,
                        weight_fp32, rope_cos, rope_sin, rope_rows, rotary_dim, cu_seqlens, cu_seqlens_padded,
                        cache_lens);
  if (st != THD_OK) return st;
  if (num_heads_kv < 1 || num_pages < 0 || page_size < 1 || max_pages < 0) return THD_ERR_ARG;
  if (!on4(positions) || !on4(page_table) || page_table_stride < max_pages) return THD_ERR_ARG;
  if (!cache_strides) return THD_ERR_ARG;
  for (int i = 0; i < 6; ++i)
    if (cache_strides[i] < 0 || cache_strides[i] % 8 != 0) return THD_ERR_ARG;
  if (total_tokens == 0) return THD_OK;
  if (batch_size > 0 && (!cache_lens || (!page_table && max_pages > 0))) return THD_ERR_ARG;
  const long long qd = (long long)num_heads_q * head_dim;
  if ((st = check_rows(q, q_stride, num_heads_q, head_dim)) != THD_OK) return st;
  if ((st = check_rows(k, k_stride, num_heads_kv, head_dim)) != THD_OK) return st;
  if ((st = check_rows(v, v_stride, num_heads_kv, head_dim)) != THD_OK) return st;
  if ((st = check_rows(q_out, qd, num_heads_q, head_dim)) != THD_OK) return st;
  if (num_pages > 0 && (!k_cache || !v_cache || !on16(k_cache) || !on16(v_cache))) return THD_ERR_ARG;
  RowArgs p{};
  fill_common(p, batch_size, total_tokens, head_dim, eps, weight_fp32, rope_cos, rope_sin, rope_rows, rotary_dim,
              interleaved != 0, cu_seqlens, cu_seqlens_padded, cache_lens);
  p.positions = positions;
  p.q = HeadRows{q, q_out, q_weight, q_stride, qd, num_heads_q};
  p.k = HeadRows{k, nullptr, k_weight, k_stride, 0, num_heads_kv};
  p.v = HeadRows{v, nullptr, nullptr, v_stride, 0, num_heads_kv};
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.k_page = cache_strides[0];
  p.k_token = cache_strides[1];
  p.k_head = cache_strides[2];
  p.v_page = cache_strides[3];
  p.v_token = cache_strides[4];
  p.v_head = cache_strides[5];
  p.table = page_table;
  p.table_stride = page_table_stride;
  p.num_pages = num_pages;
  p.page_size = page_size;
  p.max_pages = max_pages;
  return launch_rows<true>(p, dtype, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
