// seq_rows.cuh — what the operators around packed attention share: the sequence a packed row
// belongs to, 16-bit element conversion, asynchronous copies, launch settings and alignment checks.
//
// Packed rows, cu_seqlens and slot starts as everywhere in this library: sequence b holds rows
// [start_b, start_b + cu[b+1] - cu[b]), start_b = padded[b] or cu[b], starts ascending.
#pragma once
#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace thd {

// SM count of the current device, 0 on an error (looked up once per device).
inline int device_sms() {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < kDevices && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < kDevices) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

// Lets a kernel take `smem` bytes of dynamic shared memory on the current device.  One instance per
// kernel: what it has set is not set again (the call costs about a microsecond).
struct SmemGrant {
  std::atomic<uint64_t> granted{0};   // bit per device

  template <typename Kernel>
  bool ask(Kernel kern, size_t smem) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
    if (granted.load(std::memory_order_relaxed) & bit) return true;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return false;
    granted.fetch_or(bit, std::memory_order_relaxed);
    return true;
  }
};

inline bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline bool on4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }

// 16 bytes from global to shared memory, asynchronously; zeros (and nothing read) where `take` is false.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Where row t lies, found by the whole warp (every lane passes the same t and gets the same
// answer): its sequence and the rows [from, to) of it, or seq -1 and rows after t that are
// certainly of no sequence.  Each step probes 32 starts at once, so 4096 sequences take three
// dependent loads instead of the twelve of a bisection.  The answer is checked against the
// sequence's length, so metadata that does not ascend gives rows of no sequence, never a place
// outside one.
struct RowSpan {
  int seq;
  long long from, to;
};

__device__ __forceinline__ RowSpan find_span(const int32_t* __restrict__ cu, const int32_t* __restrict__ padded, int B,
                                             int t) {
  const int32_t* starts = padded ? padded : cu;
  const int lane = threadIdx.x & 31;
  const long long none = 1ll << 40;
  if (B <= 0) return {-1, t, none};
  int lo = 0, n = B;   // the last start <= t lies in [lo, lo + n)
  for (;;) {
    const int step = (n + 31) >> 5;
    const int at = lane * step;
    const bool le = at < n && starts[lo + at] <= t;
    const int cnt = __popc(__ballot_sync(0xffffffffu, le));
    if (cnt == 0) {
      const long long first = starts[lo];
      return {-1, t, first > t ? first : t + 1ll};
    }
    lo += (cnt - 1) * step;
    n = min(step, n - (cnt - 1) * step);
    if (n <= 1) break;
  }
  long long next = lo + 1 < B ? (long long)starts[lo + 1] : none;
  if (next <= t) next = t + 1ll;
  // sequences without rows may share a start with the one before them
  int b = lo;
  int len = cu[b + 1] - cu[b];
  while (len <= 0) {
    const int back = b - 1 - lane;
    const uint32_t some = __ballot_sync(0xffffffffu, back >= 0 && cu[max(back, 0) + 1] - cu[max(back, 0)] > 0);
    if (some) {
      b -= __ffs(some);
      len = cu[b + 1] - cu[b];
      break;
    }
    b -= 32;
    if (b <= 0) return {-1, t, next};
  }
  const long long from = starts[b], to = from + len;
  if (t < from || t >= to) return {-1, t, next};
  return {b, from, to};
}

// The places of rows that a warp visits in ascending order: the span of the last one is kept and
// looked up again only when a row leaves it.
struct RowCursor {
  RowSpan span{-1, 0, 0};

  __device__ __forceinline__ void move(const int32_t* cu, const int32_t* padded, int B, int t) {
    if (t < span.from || t >= span.to) span = find_span(cu, padded, B, t);
  }
};

template <typename DT>
struct Pair16;
template <>
struct Pair16<__nv_bfloat16> {
  static constexpr bool kBF16 = true;
  __device__ static __forceinline__ float2 get(uint32_t x) {
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
  }
  __device__ static __forceinline__ uint32_t put(float a, float b) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
  }
  // a += the pair's first value, b += its second (exact widening, one instruction each)
  __device__ static __forceinline__ void add(uint32_t x, float& a, float& b) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "add.rn.f32.bf16 %0, l, %0;\n\tadd.rn.f32.bf16 %1, h, %1;\n\t}"
        : "+f"(a), "+f"(b)
        : "r"(x));
  }
};
template <>
struct Pair16<__half> {
  static constexpr bool kBF16 = false;
  __device__ static __forceinline__ float2 get(uint32_t x) {
    return __half22float2(*reinterpret_cast<__half2*>(&x));
  }
  __device__ static __forceinline__ uint32_t put(float a, float b) {
    __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
  }
  __device__ static __forceinline__ void add(uint32_t x, float& a, float& b) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "add.rn.f32.f16 %0, l, %0;\n\tadd.rn.f32.f16 %1, h, %1;\n\t}"
        : "+f"(a), "+f"(b)
        : "r"(x));
  }
};

template <typename DT>
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(Pair16<DT>::put(f[0], f[1]), Pair16<DT>::put(f[2], f[3]), Pair16<DT>::put(f[4], f[5]),
                    Pair16<DT>::put(f[6], f[7]));
}

}  // namespace thd
