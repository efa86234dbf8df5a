// The paged key-value cache as the kernels of kv_append, kv_attend and
// kv_evict see it, and the conversions between its element types and fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "w4_device.cuh"
#include "w4_internal.h"

namespace w4kv {

using w4dev::ErrorWord;

// Quotients by a divisor of 1..2^30 of dividends below 2^31, by one high
// product: with l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1, n / d =
// (floor(m n / 2^32) + n) >> l.
struct Divisor {
  uint32_t d, m, l;
  __device__ __forceinline__ int32_t quotient(int32_t n) const {
    return static_cast<int32_t>((__umulhi(m, static_cast<uint32_t>(n)) + static_cast<uint32_t>(n)) >> l);
  }
};

// One layer's cache: page p holds, for each head, `page_size` slots of
// `head_dim` elements; pages lie `page_stride` elements apart (any 64-bit
// distance), `page_rows` rows of head_dim elements; scales
// [pages][heads][slots] are packed.
struct View {
  void* k;
  void* v;
  float* ks;
  float* vs;
  const int32_t* table;
  int32_t* lengths;
  int64_t page_stride;
  int64_t ldp;
  uint32_t page_rows;
  Divisor page;  // slots of a page
  int32_t num_pages, seqs, heads, slots_per_page, dim, capacity;
};

__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A stored length, held to [0, capacity]; one outside it is recorded.
__device__ __forceinline__ int32_t held_length(const View& c, int32_t b, ErrorWord* err, int32_t kernel) {
  const int32_t n = c.lengths[b];
  if (n >= 0 && n <= c.capacity) return n;
  w4dev::record_error(err, W4_ERR_VALUE, kernel, n);
  return n < 0 ? 0 : c.capacity;
}

// The page of a slot, or -1 (recorded) for an entry that names no page.
__device__ __forceinline__ int32_t page_of(const View& c, int32_t b, int32_t index, ErrorWord* err, int32_t kernel) {
  const int32_t p = c.table[static_cast<int64_t>(b) * c.ldp + index];
  if (p >= 0 && p < c.num_pages) return p;
  w4dev::record_error(err, W4_ERR_VALUE, kernel, p);
  return -1;
}

template <int TYPE>
struct Elem;

template <>
struct Elem<W4_KV_F32> {
  static constexpr int kBytes = 4, kPerVec = 4;
  __device__ static __forceinline__ void unpack(const uint4& w, float (&f)[4]) {
    f[0] = __uint_as_float(w.x);
    f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z);
    f[3] = __uint_as_float(w.w);
  }
};

template <>
struct Elem<W4_KV_F16> {
  static constexpr int kBytes = 2, kPerVec = 8;
  __device__ static __forceinline__ void unpack(const uint4& w, float (&f)[8]) {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&a[i]));
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    }
  }
};

template <>
struct Elem<W4_KV_BF16> {
  static constexpr int kBytes = 2, kPerVec = 8;
  __device__ static __forceinline__ void unpack(const uint4& w, float (&f)[8]) {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(a[i] << 16);
      f[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
  }
};

template <>
struct Elem<W4_KV_I8> {
  static constexpr int kBytes = 1, kPerVec = 16;
  // The code XOR 0x80 in the low byte of 2^23's mantissa is 2^23 + 128 + code
  // exactly; the subtraction is exact too.
  __device__ static __forceinline__ void unpack(const uint4& w, float (&f)[16]) {
    const uint32_t a[4] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u, w.z ^ 0x80808080u, w.w ^ 0x80808080u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[4 * i] = w4dev::byte_float<0>(a[i], 0x4B000000u) - 8388736.f;
      f[4 * i + 1] = w4dev::byte_float<1>(a[i], 0x4B000000u) - 8388736.f;
      f[4 * i + 2] = w4dev::byte_float<2>(a[i], 0x4B000000u) - 8388736.f;
      f[4 * i + 3] = w4dev::byte_float<3>(a[i], 0x4B000000u) - 8388736.f;
    }
  }
};

constexpr int elem_bytes(int type) { return type == W4_KV_F32 ? 4 : (type == W4_KV_I8 ? 1 : 2); }

// 2^x, the hardware's approximation (2 ulp); 2^-inf = 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace w4kv

namespace w4host {

w4kv::Divisor divisor(uint32_t d);

// Checks of a cache descriptor that need no device, and the kernels' view of
// it. `what` names the descriptor in the reason.
w4_status check_cache(const kv_cache* c, const char* what, w4kv::View* out);

// A launch whose start may overlap the end of the previous work on the stream
// (programmatic dependent launch); every kernel launched this way waits for
// that work before it reads or writes anything.
// cluster: CTAs of a cluster (1: none). most_shared: asks for the largest
// shared-memory split of an SM.
template <class... Args>
cudaError_t launch_pdl(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t st, unsigned cluster,
                       bool most_shared, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[3];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = cluster;
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs++].val.clusterDim.z = 1;
  }
  if (most_shared) {
    attr[cfg.numAttrs].id = cudaLaunchAttributePreferredSharedMemoryCarveout;
    attr[cfg.numAttrs++].val.sharedMemCarveout = cudaSharedmemCarveoutMaxShared;
  }
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace w4host
