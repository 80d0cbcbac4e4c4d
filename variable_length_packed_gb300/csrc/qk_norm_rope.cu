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
// All in fp32, rounded once to the tensors' type.
//
// Layout: a head is d / 8 chunks of 16 bytes.  One lane holds two of them, the two whose values
// pair up under the half-split rotation (chunks s and s + rotary / 16; behind the rotated
// part, neighbours), so a rotation needs no exchange between lanes and a norm only the sum over
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
  // cache
  void* k_cache;
  void* v_cache;
  const int32_t* table;
  long long table_stride, k_page, k_token, k_head, v_page, v_token, v_head;   // elements
  int num_pages, page_size, max_pages;
};

constexpr int kRowWarps = 4;      // warps of a block
constexpr int kRowPasses = 4;     // 32 / lanes-per-head heads in each

// cos / sin of a lane's two chunks.  Half-split: element e of both chunks turns by angle
// 8 s + e.  Interleaved: pair e of the first chunk by 4 s + e, of the second by
// 4 (s + rotary / 16) + e.
struct Angles {
  float c[8], s[8];
};

__device__ __forceinline__ void load_angles(Angles& a, const RowArgs& p, int slot, long long pos) {
  const long long row = pos < 0 ? 0 : (pos >= p.rope_rows ? p.rope_rows - 1 : pos);
  const int half = p.rotary >> 1;
  const int at0 = p.interleaved ? 4 * slot : 8 * slot;
  const int at1 = p.interleaved ? 4 * (slot + (p.rotary >> 4)) : 8 * slot + 4;
  const float4 c0 = *reinterpret_cast<const float4*>(p.cos + row * half + at0);
  const float4 c1 = *reinterpret_cast<const float4*>(p.cos + row * half + at1);
  const float4 s0 = *reinterpret_cast<const float4*>(p.sin + row * half + at0);
  const float4 s1 = *reinterpret_cast<const float4*>(p.sin + row * half + at1);
  a.c[0] = c0.x, a.c[1] = c0.y, a.c[2] = c0.z, a.c[3] = c0.w;
  a.c[4] = c1.x, a.c[5] = c1.y, a.c[6] = c1.z, a.c[7] = c1.w;
  a.s[0] = s0.x, a.s[1] = s0.y, a.s[2] = s0.z, a.s[3] = s0.w;
  a.s[4] = s1.x, a.s[5] = s1.y, a.s[6] = s1.z, a.s[7] = s1.w;
}

// Turns a lane's two chunks; sign -1 turns back.
__device__ __forceinline__ void turn(float* x0, float* x1, const Angles& a, int interleaved, float sign) {
  if (interleaved) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float s0 = sign * a.s[e], s1 = sign * a.s[4 + e];
      const float u0 = x0[2 * e], w0 = x0[2 * e + 1], u1 = x1[2 * e], w1 = x1[2 * e + 1];
      x0[2 * e] = u0 * a.c[e] - w0 * s0;
      x0[2 * e + 1] = w0 * a.c[e] + u0 * s0;
      x1[2 * e] = u1 * a.c[4 + e] - w1 * s1;
      x1[2 * e + 1] = w1 * a.c[4 + e] + u1 * s1;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float s = sign * a.s[e];
      const float u = x0[e], w = x1[e];
      x0[e] = u * a.c[e] - w * s;
      x1[e] = w * a.c[e] + u * s;
    }
  }
}

// A lane's two chunks of a head: rotated pairs first, then neighbours.
__device__ __forceinline__ void lane_chunks(int slot, int rotary, int& c0, int& c1) {
  const int pairs = rotary >> 4;
  if (slot < pairs) {
    c0 = slot;
    c1 = slot + pairs;
  } else {
    c0 = 2 * slot;   // 2 * pairs + 2 * (slot - pairs)
    c1 = 2 * slot + 1;
  }
}

template <typename DT>
__device__ __forceinline__ void load_weight(const void* w, int fp32, int chunk, float* f) {
  if (fp32) {
    const float4 a = reinterpret_cast<const float4*>(w)[2 * chunk], b = reinterpret_cast<const float4*>(w)[2 * chunk + 1];
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    unpack8<DT>(reinterpret_cast<const uint4*>(w)[chunk], f);
  }
}

template <int LPH>
__device__ __forceinline__ float head_sum(float x) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// LPH lanes per head (a power of two >= d / 16).
template <typename DT, int LPH, bool kCache>
__global__ void __launch_bounds__(kRowWarps * 32) head_rows_kernel(const RowArgs p) {
  constexpr int kPerPass = 32 / LPH;
  const int lane = threadIdx.x & 31;
  const unsigned item = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  const unsigned t = item / (unsigned)p.row_items;
  if (t >= (unsigned)p.T) return;
  int part = (int)(item - t * (unsigned)p.row_items);
  int kind = 0;   // 0 queries, 1 keys, 2 values
  HeadRows h = p.q;
  if (part >= p.q_items) {
    part -= p.q_items;
    kind = 1;
    h = p.k;
    if (kCache && part >= p.k_items) {
      part -= p.k_items;
      kind = 2;
      h = p.v;
    }
  }
  const int slot = lane % LPH;
  const int head0 = part * (kRowPasses * kPerPass) + lane / LPH;
  const bool mine = slot < (p.d >> 4);
  int c0, c1;
  lane_chunks(slot, p.rotary, c0, c1);

  uint4 raw[kRowPasses][2];
  const DT* src = static_cast<const DT*>(h.src) + (long long)t * h.src_stride;
#pragma unroll
  for (int i = 0; i < kRowPasses; ++i) {
    const int head = head0 + i * kPerPass;
    raw[i][0] = raw[i][1] = make_uint4(0u, 0u, 0u, 0u);
    if (mine && head < h.heads) {
      raw[i][0] = *reinterpret_cast<const uint4*>(src + (long long)head * p.d + 8 * c0);
      raw[i][1] = *reinterpret_cast<const uint4*>(src + (long long)head * p.d + 8 * c1);
    }
  }
  const bool norm = kind != 2 && h.weight != nullptr;
  float w0[8], w1[8];
  if (norm && mine) {
    load_weight<DT>(h.weight, p.weight_fp32, c0, w0);
    load_weight<DT>(h.weight, p.weight_fp32, c1, w1);
  }
  const RowPlace at = find_row(p.cu, p.padded, p.B, (int)t);
  long long pos = at.pos;
  DT* dst;
  long long dst_head = p.d;
  if (at.seq >= 0) pos += p.offsets ? p.offsets[at.seq] : 0;
  if (kCache && kind != 0) {
    if (at.seq < 0 || pos < 0) return;
    const long long page_at = pos / p.page_size;
    if (page_at >= p.max_pages) return;
    const int page = p.table[(long long)at.seq * p.table_stride + page_at];
    if (page < 0 || page >= p.num_pages) return;
    const long long off = pos - page_at * p.page_size;
    dst = kind == 1 ? static_cast<DT*>(p.k_cache) + page * p.k_page + off * p.k_token
                    : static_cast<DT*>(p.v_cache) + page * p.v_page + off * p.v_token;
    dst_head = kind == 1 ? p.k_head : p.v_head;
  } else {
    dst = static_cast<DT*>(h.dst) + (long long)t * h.dst_stride;
  }
  const bool rot = kind != 2 && slot < (p.rotary >> 4);
  Angles a;
  if (at.seq >= 0 && rot) load_angles(a, p, slot, kCache && p.positions ? (long long)p.positions[t] : pos);
#pragma unroll
  for (int i = 0; i < kRowPasses; ++i) {
    const int head = head0 + i * kPerPass;
    uint4 o0 = make_uint4(0u, 0u, 0u, 0u), o1 = o0;   // a row of no sequence
    if (at.seq >= 0) {
      if (norm || rot) {
        float x0[8], x1[8];
        unpack8<DT>(raw[i][0], x0);
        unpack8<DT>(raw[i][1], x1);
        if (norm) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss += x0[e] * x0[e] + x1[e] * x1[e];
          const float r = rsqrtf(head_sum<LPH>(ss) * p.inv_d + p.eps);
          if (mine) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              x0[e] *= r * w0[e];
              x1[e] *= r * w1[e];
            }
          }
        }
        if (rot) turn(x0, x1, a, p.interleaved, p.sin_sign);
        o0 = pack8<DT>(x0);
        o1 = pack8<DT>(x1);
      } else {
        o0 = raw[i][0];
        o1 = raw[i][1];
      }
    }
    if (mine && head < h.heads) {
      *reinterpret_cast<uint4*>(dst + head * dst_head + 8 * c0) = o0;
      *reinterpret_cast<uint4*>(dst + head * dst_head + 8 * c1) = o1;
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
};

constexpr int kBwdPasses = 2;
constexpr int kBwdWarps = 4;
constexpr int kBwdBlocksPerSm = 4;
constexpr int kBwdMaxBlocks = 1024;

template <typename DT, int LPH>
__global__ void __launch_bounds__(kBwdWarps * 32) head_rows_bwd_kernel(const NormBwdArgs b) {
  constexpr int kPerPass = 32 / LPH;
  const RowArgs& p = b.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool is_q = (int)blockIdx.x < b.q_blocks;
  const HeadRows h = is_q ? p.q : p.k;
  const DT* grad = static_cast<const DT*>(is_q ? b.gq : b.gk);
  const unsigned items = (unsigned)(is_q ? p.q_items : p.k_items);
  const unsigned blocks = (unsigned)(is_q ? b.q_blocks : b.k_blocks);
  const unsigned first = (unsigned)(is_q ? blockIdx.x : blockIdx.x - b.q_blocks) * kBwdWarps + warp;
  const int slot = lane % LPH;
  const bool mine = slot < (p.d >> 4);
  const bool norm = h.weight != nullptr;
  int c0, c1;
  lane_chunks(slot, p.rotary, c0, c1);
  float w0[8], w1[8], dw0[8], dw1[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w0[e] = w1[e] = dw0[e] = dw1[e] = 0.f;
  if (norm && mine) {
    load_weight<DT>(h.weight, p.weight_fp32, c0, w0);
    load_weight<DT>(h.weight, p.weight_fp32, c1, w1);
  }
  const bool rot = slot < (p.rotary >> 4);
  const unsigned total = (unsigned)p.T * items;
  for (unsigned item = first; item < total; item += blocks * kBwdWarps) {
    const unsigned t = item / items;
    const int head0 = (int)(item - t * items) * (kBwdPasses * kPerPass) + lane / LPH;
    const DT* src = static_cast<const DT*>(h.src) + (long long)t * h.src_stride;
    const DT* gsrc = grad + (long long)t * h.heads * p.d;
    DT* dst = static_cast<DT*>(h.dst) + (long long)t * h.dst_stride;
    uint4 rx[kBwdPasses][2], rg[kBwdPasses][2];
#pragma unroll
    for (int i = 0; i < kBwdPasses; ++i) {
      const int head = head0 + i * kPerPass;
      rx[i][0] = rx[i][1] = rg[i][0] = rg[i][1] = make_uint4(0u, 0u, 0u, 0u);
      if (mine && head < h.heads) {
        const long long at = (long long)head * p.d;
        rg[i][0] = *reinterpret_cast<const uint4*>(gsrc + at + 8 * c0);
        rg[i][1] = *reinterpret_cast<const uint4*>(gsrc + at + 8 * c1);
        if (norm) {
          rx[i][0] = *reinterpret_cast<const uint4*>(src + at + 8 * c0);
          rx[i][1] = *reinterpret_cast<const uint4*>(src + at + 8 * c1);
        }
      }
    }
    const RowPlace at = find_row(p.cu, p.padded, p.B, (int)t);
    Angles a;
    if (at.seq >= 0 && rot) load_angles(a, p, slot, (long long)at.pos + (p.offsets ? p.offsets[at.seq] : 0));
#pragma unroll
    for (int i = 0; i < kBwdPasses; ++i) {
      const int head = head0 + i * kPerPass;
      uint4 o0 = make_uint4(0u, 0u, 0u, 0u), o1 = o0;
      if (at.seq >= 0) {
        float g0[8], g1[8];
        unpack8<DT>(rg[i][0], g0);
        unpack8<DT>(rg[i][1], g1);
        if (rot) turn(g0, g1, a, p.interleaved, -1.f);
        if (norm) {
          float x0[8], x1[8];
          unpack8<DT>(rx[i][0], x0);
          unpack8<DT>(rx[i][1], x1);
          float ss = 0.f, dot = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            ss += x0[e] * x0[e] + x1[e] * x1[e];
            dot += g0[e] * w0[e] * x0[e] + g1[e] * w1[e] * x1[e];
          }
          ss = head_sum<LPH>(ss);
          dot = head_sum<LPH>(dot);
          // past the last head there is nothing, and with eps = 0 its 1 / rms has no value
          const float r = head < h.heads ? rsqrtf(ss * p.inv_d + p.eps) : 0.f;
          const float m = dot * p.inv_d * r * r;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            dw0[e] += g0[e] * x0[e] * r;
            dw1[e] += g1[e] * x1[e] * r;
            g0[e] = r * (g0[e] * w0[e] - x0[e] * m);
            g1[e] = r * (g1[e] * w1[e] - x1[e] * m);
          }
        }
        o0 = pack8<DT>(g0);
        o1 = pack8<DT>(g1);
      }
      if (mine && head < h.heads) {
        *reinterpret_cast<uint4*>(dst + (long long)head * p.d + 8 * c0) = o0;
        *reinterpret_cast<uint4*>(dst + (long long)head * p.d + 8 * c1) = o1;
      }
    }
  }
  if (!norm) return;
  // the block's share of dw: over the warp's heads, then over the warps
  __shared__ float sum[kBwdWarps][128];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int o = LPH; o < 32; o <<= 1) {
      dw0[e] += __shfl_xor_sync(0xffffffffu, dw0[e], o);
      dw1[e] += __shfl_xor_sync(0xffffffffu, dw1[e], o);
    }
    if (lane < LPH && mine) {
      sum[warp][8 * c0 + e] = dw0[e];
      sum[warp][8 * c1 + e] = dw1[e];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.d; i += blockDim.x) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kBwdWarps; ++k) s += sum[k][i];
    b.partial[(long long)blockIdx.x * p.d + i] = s;
  }
}

// dw = the blocks' shares summed in a fixed order; a block takes 8 columns of one kind.
constexpr int kSumRows = 32;
__global__ void __launch_bounds__(kSumRows * 8) weight_sum_kernel(const float* __restrict__ partial, int q_blocks,
                                                                  int k_blocks, int d, float* dwq, float* dwk) {
  const int kind = blockIdx.y;
  float* dst = kind == 0 ? dwq : dwk;
  if (!dst) return;
  const int col = blockIdx.x * 8 + (threadIdx.x & 7), row = threadIdx.x >> 3;
  const int begin = kind == 0 ? 0 : q_blocks, n = kind == 0 ? q_blocks : k_blocks;
  __shared__ float part[kSumRows][9];
  float s = 0.f;
  for (int i = row; i < n; i += kSumRows) s += partial[(long long)(begin + i) * d + col];
  part[row][threadIdx.x & 7] = s;
  __syncthreads();
  if (row == 0) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kSumRows; ++i) s += part[i][threadIdx.x];
    dst[col] = s;
  }
}

// ---------------------------------------------------------------------------- host
bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool on4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

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

template <typename DT, bool kCache>
int launch_rows_of(const RowArgs& p, unsigned grid, cudaStream_t st) {
  const dim3 block(kRowWarps * 32);
  switch (lanes_per_head(p.d)) {
    case 1: head_rows_kernel<DT, 1, kCache><<<grid, block, 0, st>>>(p); break;
    case 2: head_rows_kernel<DT, 2, kCache><<<grid, block, 0, st>>>(p); break;
    case 4: head_rows_kernel<DT, 4, kCache><<<grid, block, 0, st>>>(p); break;
    default: head_rows_kernel<DT, 8, kCache><<<grid, block, 0, st>>>(p); break;
  }
  return cudaGetLastError() == cudaSuccess ? THD_OK : THD_ERR_CUDA;
}

template <bool kCache>
int launch_rows(RowArgs& p, int dtype, cudaStream_t st) {
  const int per = kRowPasses * (32 / lanes_per_head(p.d));
  p.q_items = blocks_of_heads(p.q.heads, per);
  p.k_items = blocks_of_heads(p.k.heads, per);
  const long long row_items = (long long)p.q_items + p.k_items + blocks_of_heads(p.v.heads, per);
  if (row_items == 0) return THD_OK;
  const long long items = row_items * p.T;
  if (items >= (1ll << 31)) return THD_ERR_UNSUPPORTED;   // item numbers are 32-bit
  p.row_items = (int)row_items;
  const unsigned grid = (unsigned)((items + kRowWarps - 1) / kRowWarps);
  return dtype == THD_BF16 ? launch_rows_of<__nv_bfloat16, kCache>(p, grid, st)
                           : launch_rows_of<__half, kCache>(p, grid, st);
}

template <typename DT>
int launch_bwd_of(const NormBwdArgs& b, unsigned grid, cudaStream_t st) {
  const dim3 block(kBwdWarps * 32);
  switch (lanes_per_head(b.a.d)) {
    case 1: head_rows_bwd_kernel<DT, 1><<<grid, block, 0, st>>>(b); break;
    case 2: head_rows_bwd_kernel<DT, 2><<<grid, block, 0, st>>>(b); break;
    case 4: head_rows_bwd_kernel<DT, 4><<<grid, block, 0, st>>>(b); break;
    default: head_rows_bwd_kernel<DT, 8><<<grid, block, 0, st>>>(b); break;
  }
  return cudaGetLastError() == cudaSuccess ? THD_OK : THD_ERR_CUDA;
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
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
    return THD_ERR_CUDA;
  const int per = kBwdPasses * (32 / lanes_per_head(head_dim));
  NormBwdArgs b{};
  p.q = HeadRows{q, dq, q_weight, q_stride, dq_stride, num_heads_q};
  p.k = HeadRows{k, dk, k_weight, k_stride, dk_stride, num_heads_kv};
  p.q_items = blocks_of_heads(num_heads_q, per);
  p.k_items = blocks_of_heads(num_heads_kv, per);
  const long long qi = (long long)p.q_items * total_tokens, ki = (long long)p.k_items * total_tokens;
  // item numbers are 32-bit, and the loop adds one stride of the grid past the last
  if (qi >= (1ll << 31) || ki >= (1ll << 31)) return THD_ERR_UNSUPPORTED;
  // blocks in proportion to the items of each kind, at most one item's worth of warps each
  long long blocks = (long long)sms * kBwdBlocksPerSm;
  if (blocks > kBwdMaxBlocks) blocks = kBwdMaxBlocks;
  const long long want_q = (qi + kBwdWarps - 1) / kBwdWarps, want_k = (ki + kBwdWarps - 1) / kBwdWarps;
  long long qb = want_q, kb = want_k;
  if (want_q + want_k > blocks) {
    qb = blocks * want_q / (want_q + want_k);
    if (want_q > 0 && qb < 1) qb = 1;
    if (want_k > 0 && qb > blocks - 1) qb = blocks - 1;
    kb = want_k < blocks - qb ? want_k : blocks - qb;
  }
  b.a = p;
  b.gq = grad_q;
  b.gk = grad_k;
  b.partial = static_cast<float*>(workspace);
  b.q_blocks = (int)qb;
  b.k_blocks = (int)kb;
  if (qb + kb > 0) {
    st = dtype == THD_BF16 ? launch_bwd_of<__nv_bfloat16>(b, (unsigned)(qb + kb), s)
                           : launch_bwd_of<__half>(b, (unsigned)(qb + kb), s);
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
