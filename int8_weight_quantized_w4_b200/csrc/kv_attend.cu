// kv_attend's host side, and the small kernel behind the attention kernels: the
// partials of items that several CTAs shared joined, and attention weights
// summed over the query heads.
#include <algorithm>

#include "kv_attend.cuh"

namespace w4kv {

template <>
AttendKernel attend_kernel_for<W4_KV_F32>(int32_t dim, int32_t group, bool brief);
template <>
AttendKernel attend_kernel_for<W4_KV_F16>(int32_t dim, int32_t group, bool brief);
template <>
AttendKernel attend_kernel_for<W4_KV_BF16>(int32_t dim, int32_t group, bool brief);
template <>
AttendKernel attend_kernel_for<W4_KV_I8>(int32_t dim, int32_t group, bool brief);

}  // namespace w4kv

namespace {

using namespace w4kv;

constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kMostUnits = 16;
constexpr int kShortUnits = 4;
// Slots of a CTA in runs: fewer cost more to join than they save, more leave too
// few CTAs. One sequence of 1000 slots, 2 x 128 fp32, in a table for 40000, 8.9 us
// (with 16 9.9 us, with 256 13.6 us); of 6000 12.9 us (24.1 us, 15.5 us).
constexpr int kLeastSlots = 64;
// CTAs an SM that the weights are shared out for: 64 sequences of up to 2000 slots,
// 8 x 128 bf16 for 32 heads, 61.7 us (with 4 62.8 us, with 64 62.9 us); 8 of up to
// 4000, 32 x 96 fp16, 51.0 us (51.8 us, 51.0 us); one of 131072 119 us (110 us, 128 us).
constexpr int kGatherCtas = 16;
constexpr int kMaxLaneVecs = 2;  // float4s of a lane: 32 x 4 x 2 = 256, the largest head_dim

// The partials of an item: its first one, then the next CTAs' first ones.
__device__ __forceinline__ const float* partial(const AttendParams& p, const int2& meta, int32_t i) {
  const int64_t slot = i == 0 ? meta.x : 2 * int64_t(meta.x / 2 + i);
  return p.part + slot * p.part_stride;
}

__device__ __forceinline__ int2 meta_of(const AttendParams& p, int32_t b, int32_t qh, int* row) {
  const int32_t h = qh / p.group, in = qh - h * p.group, chunk = in / p.rows;
  *row = in - chunk * p.rows;
  return p.meta[(int64_t(b) * p.c.heads + h) * p.chunks + chunk];
}

// Query heads whose items several CTAs shared: `wpr` warps a head. wpr = 8
// spreads the partials of a few long rows, wpr = 1 passes over many rows that
// mostly have nothing to join.
__device__ __forceinline__ void join_heads(const AttendParams& p, int wpr) {
  __shared__ Triple sm[kJoinWarps][32 * kMaxLaneVecs];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q_heads = p.c.heads * p.group;
  const int64_t row = int64_t(blockIdx.x) * (kJoinWarps / wpr) + warp / wpr;
  const int sub = warp % wpr;
  const int D = p.c.dim, vecs = D / 4;
  Triple x[kMaxLaneVecs];
#pragma unroll
  for (int i = 0; i < kMaxLaneVecs; ++i) x[i] = no_slots();
  bool work = false;
  int32_t b = 0, qh = 0;
  if (row < int64_t(p.c.seqs) * q_heads) {
    b = static_cast<int32_t>(row / q_heads);
    qh = static_cast<int32_t>(row % q_heads);
    int32_t lo, n;
    int g = 0;
    attended(p, b, lo, n);
    const int2 meta = n > lo ? meta_of(p, b, qh, &g) : make_int2(0, 0);
    work = meta.y != 1;
#pragma unroll 8
    for (int32_t i = sub; i < (work ? meta.y : 0); i += wpr) {
      const float* part = partial(p, meta, i);
#pragma unroll
      for (int j = 0; j < kMaxLaneVecs; ++j)
        if (lane + 32 * j < vecs) join(x[j], stored(part, p.rows, D, g, 4 * (lane + 32 * j)));
    }
  }
  if (wpr > 1) {
#pragma unroll
    for (int j = 0; j < kMaxLaneVecs; ++j) sm[warp][lane + 32 * j] = x[j];
    __syncthreads();
    if (sub != 0) return;
    for (int w = warp + 1; w < warp + wpr; ++w) {
#pragma unroll
      for (int j = 0; j < kMaxLaneVecs; ++j) join(x[j], sm[w][lane + 32 * j]);
    }
  }
  if (!work) return;
#pragma unroll
  for (int j = 0; j < kMaxLaneVecs; ++j)
    if (lane + 32 * j < vecs) write_out(p, b, qh, 4 * (lane + 32 * j), x[j]);
}

// The query heads' log sums to base 2, 32 heads at a time by 8 lanes each: as
// the attention kernel wrote them, or from the partials, so that the weights
// need not wait for the join. -Inf: none of the attended slots is there (all on
// pages that do not exist), and nothing weighs anything.
__device__ __forceinline__ void log_sums(const AttendParams& p, int32_t b, int32_t q0, int heads, bool runs, float* z) {
  const int sub = threadIdx.x % 8;
  for (int i0 = 0; i0 < heads; i0 += kJoinThreads / 8) {
    const int i = i0 + threadIdx.x / 8;
    const bool live = i < heads;
    const int32_t qh = q0 + (live ? i : 0);
    Triple x = no_slots();
    int2 meta = make_int2(0, 1);
    if (runs) {
      int g;
      meta = meta_of(p, b, qh, &g);
      if (meta.y != 1) {
#pragma unroll 4
        for (int32_t k = sub; k < meta.y; k += 8) {
          const float* part = partial(p, meta, k) + p.rows * p.c.dim;
          join(x, {make_float4(0.f, 0.f, 0.f, 0.f), part[g], part[p.rows + g]});
        }
      }
    }
#pragma unroll
    for (int o = 1; o < 8; o *= 2) {
      const float m = __shfl_xor_sync(0xffffffffu, x.m, o), l = __shfl_xor_sync(0xffffffffu, x.l, o);
      // the lower lane's first: both sides the same sum
      Triple y = {x.a, sub & o ? m : x.m, sub & o ? l : x.l};
      join(y, {x.a, sub & o ? x.m : m, sub & o ? x.l : l});
      x = y;
    }
    if (live && sub == 0)
      z[i] = meta.y == 1 ? p.lse2[int64_t(b) * p.c.heads * p.group + qh] : (x.l == 0.f ? -INFINITY : x.m + log2f(x.l));
  }
}

// acc[b, j] += sum over the query heads of 2^(x - lse2). A warp takes 32 slots
// and every 8th head; the warps' sums are added in their order.
__device__ __forceinline__ void gather_weights(const AttendParams& p, int block, int blocks, int32_t b, float* acc,
                                               int64_t ldacc, bool runs) {
  constexpr int kAhead = 4;
  __shared__ float sums[kJoinWarps][32];
  __shared__ float z[kJoinThreads];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q_heads = p.c.heads * p.group;
  int32_t lo, n;
  attended(p, b, lo, n);
  for (int64_t j0 = lo + int64_t(block) * 32; j0 < n; j0 += int64_t(blocks) * 32) {
    const int64_t j = j0 + lane;
    float sum = 0.f;
    const float old = warp == 0 && j < n ? acc[int64_t(b) * ldacc + j] : 0.f;
    for (int q0 = 0; q0 < q_heads; q0 += kJoinThreads) {
      const int heads = min(kJoinThreads, q_heads - q0);
      const float* x = p.scores + (int64_t(b) * q_heads + q0) * p.c.capacity + j;
      float ahead[kAhead];  // on their way while the log sums are made
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = warp + u * kJoinWarps;
        ahead[u] = j < n && i < heads ? x[int64_t(i) * p.c.capacity] : 0.f;
      }
      if (q_heads > kJoinThreads || j0 == lo + int64_t(block) * 32) {
        __syncthreads();
        log_sums(p, b, q0, heads, runs, z);
        __syncthreads();
      }
      if (j < n) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
          const int i = warp + u * kJoinWarps;
          if (i < heads) sum += z[i] == -INFINITY ? 0.f : ex2(ahead[u] - z[i]);
        }
#pragma unroll 4
        for (int i = warp + kAhead * kJoinWarps; i < heads; i += kJoinWarps)
          sum += z[i] == -INFINITY ? 0.f : ex2(x[int64_t(i) * p.c.capacity] - z[i]);
      }
    }
    sums[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && j < n) {
#pragma unroll
      for (int w = 1; w < kJoinWarps; ++w) sum += sums[w][lane];
      acc[int64_t(b) * ldacc + j] = old + sum;
    }
    __syncthreads();
  }
}

// What is left behind the attention kernel: the first `joins` CTAs join, the
// others gather weights, `per_seq` for each sequence. It does not let the next
// kernel begin early, and asks for the attention's split of shared memory: a
// CTA that lies between those of the next call's attention leaves room for one
// less on its SM for as long as that runs (131072 slots of 8 x 128 bf16, call
// after call: 117 us with either, 90 us without).
__global__ void __launch_bounds__(kJoinThreads) behind_kernel(const AttendParams p, int joins, int wpr, int per_seq,
                                                              float* acc, int64_t ldacc) {
  pdl_wait();
  if (blockIdx.x < joins) {
    join_heads(p, wpr);
  } else {
    const int block = blockIdx.x - joins, b = block / per_seq;
    gather_weights(p, block - b * per_seq, per_seq, b, acc, ldacc, joins > 0);
  }
}

struct Layout {
  AttendKernel kernel;
  int32_t chunks;
  unsigned ranks;  // CTAs of an item's cluster; 0: not so
  bool warps;      // an item a warp; neither: runs of units, and a join
  unsigned ctas;
  int64_t part_stride;
  size_t meta, lse2, scores, bytes;  // offsets, and the total
};

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

// Brief: slots too few for the matrix body, whose staging of the queries is then
// most of its time. Plain lanes against matrices, 8 key-value heads:
//   a tile or two of slots, whatever the batch: 200 sequences of 32 slots of 256
//     bf16 for 32 heads 29.6 us against 35.6 us, of 128 int8 16.3 us against 17.2 us
//     (64 slots: 25.6 us against 20.6 us; 32 of 64 bf16: 9.1 us against 6.2 us);
//   little work: 4 x 300 slots of 128 fp16 for 32 heads 7.5 us against 8.2 us, for
//     64 heads 8.5 us against 8.8 us (4 x 1000 for 64: 15.4 us against 10.2 us);
//     int8 for 32 heads 4 x 300 7.4 us against 9.6 us, 4 x 1000 10.0 us against
//     11.2 us (16 x 1000: 24 us against 18 us).
// Rows of more than 128 elements of 16 bits are many registers to a plain lane
// (4 x 300 of 192 bf16 for 32 heads: 10.3 us against 7.9 us), and int8 rows of up to
// 64 are faster in matrices (1 x 1000 for 32 heads: 6.9 us against 5.6 us).
// slots: the most that a sequence attends.
AttendKernel choose(const w4kv::View& c, int type, int32_t group, int64_t slots) {
  const bool i8 = type == W4_KV_I8;
  const int64_t work = int64_t(c.seqs) * c.heads * ((group + 1) / 2) * slots;
  const bool brief = slots <= (c.dim < 128 ? 16 : 32) || (slots <= 1024 && work <= (i8 && c.dim <= 128 ? 65536 : 40960) &&
                                          (i8 ? c.dim > 64 : c.dim <= 128));
  switch (type) {
    case W4_KV_F32: return attend_kernel_for<W4_KV_F32>(c.dim, group, brief);
    case W4_KV_F16: return attend_kernel_for<W4_KV_F16>(c.dim, group, brief);
    case W4_KV_BF16: return attend_kernel_for<W4_KV_BF16>(c.dim, group, brief);
    default: return attend_kernel_for<W4_KV_I8>(c.dim, group, brief);
  }
}

constexpr int kRankLogs = 5;  // clusters of 1, 2, 4, 8 and 16 CTAs

// What a device holds of a kernel at once, asked once for each kernel and device.
struct Held {
  const void* fn;
  int dev;
  int per_sm, warp_per_sm;    // CTAs an SM, in runs of units and in warps' items
  int clusters[kRankLogs];    // clusters of 2^i CTAs: by GPC, so fewer than their CTAs alone
};

w4_status resident(const AttendKernel& k, const w4host::DeviceInfo& di, Held* out) {
  static thread_local Held known[32] = {};
  static thread_local int next = 0;
  const void* fn = reinterpret_cast<const void*>(k.fn);
  for (const Held& e : known)
    if (e.fn == fn && e.dev == di.dev) {
      *out = e;
      return W4_OK;
    }
  const auto allow = [](void (*f)(const AttendParams), size_t smem) {
    return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  };
  cudaError_t e = allow(k.fn, k.smem);
  if (e == cudaSuccess) e = allow(k.item_fn, k.smem);
  if (e == cudaSuccess) e = allow(k.warp_fn, k.warp_smem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k.item_fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return w4host::cuda_fail(e, "kv_attend kernel attributes");
  Held h = {fn, di.dev, 0, 0, {}};
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&h.per_sm, k.fn, kAttendThreads, k.smem);
  if (e == cudaSuccess)
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&h.warp_per_sm, k.warp_fn, kAttendThreads, k.warp_smem);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&h.clusters[0], k.item_fn, kAttendThreads, k.smem);
  if (e != cudaSuccess) return w4host::cuda_fail(e, "kv_attend occupancy");
  if (h.per_sm < 1 || h.warp_per_sm < 1 || h.clusters[0] < 1)
    return w4host::fail(W4_ERR_CUDA, "kv_attend: no CTA fits an SM");
  h.clusters[0] *= di.sms;
  for (int i = 1; i < kRankLogs; ++i) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(1u << i);
    cfg.blockDim = dim3(kAttendThreads);
    cfg.dynamicSmemBytes = k.smem;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << i;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributePreferredSharedMemoryCarveout;
    attr[1].val.sharedMemCarveout = cudaSharedmemCarveoutMaxShared;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaOccupancyMaxActiveClusters(&h.clusters[i], k.item_fn, &cfg) != cudaSuccess) {
      cudaGetLastError();  // no such cluster on this device
      h.clusters[i] = 0;
    }
  }
  known[next] = h;
  next = (next + 1) % 32;
  *out = h;
  return W4_OK;
}

// kernel: as chosen for `slots` or more. For one kernel, fewer slots never need
// more workspace.
w4_status lay_out(const w4kv::View& c, const AttendKernel& kernel, int64_t slots, int64_t q_heads, bool with_acc,
                  const w4host::DeviceInfo& di, Layout* out) {
  const int sms = di.sms;
  const int32_t group = static_cast<int32_t>(q_heads / c.heads);
  Layout L = {};
  L.kernel = kernel;
  L.chunks = (group + L.kernel.rows - 1) / L.kernel.rows;
  Held held = {};
  const w4_status rc = resident(L.kernel, di, &held);
  if (rc != W4_OK) return rc;
  const int64_t items = int64_t(c.seqs) * c.heads * L.chunks;
  const int64_t units = (slots + L.kernel.unit - 1) / L.kernel.unit;
  const int64_t most = items * (units + L.kernel.over);
  if (most > 0x7fffffff) return w4host::fail(W4_ERR_SHAPE, "seqs x heads x capacity are more slots than a call takes");
  const int64_t wave = int64_t(held.per_sm) * sms;
  // An item a cluster: the widest of up to 16 CTAs that one wave holds for all
  // items, where it leaves a CTA kMostUnits units (of 64 slots at most) of a full
  // sequence: runs balance the CTAs, clusters save the second launch. One
  // 12 x 64 fp32 sequence of 1021 slots: 5.7 us against 9.0 us as runs and a
  // join; 48 of 1024, bf16: 26 us against 32 us; 8 of 1000, 8 x 128 bf16 for 32
  // heads: 11.1 us against 14.4 us; with more units, 48 of up to 2048, 32.3 us
  // against 29.4 us; 32 of up to 2000, 8 x 128 int8 for 64 heads, 40 us against 31 us.
  // (As many as the GPCs hold, not as their SMs' sum does: 32 clusters of 16 are
  // one wave by the sum at 4 CTAs an SM, and took two.)
  int log = kRankLogs - 1;
  while (log > 0 && (items > held.clusters[log] || (1 << log) / 2 >= units)) --log;
  const int64_t most_slots = int64_t(kMostUnits) * std::min(64, L.kernel.unit) << log;
  L.ranks = items <= held.clusters[log] && slots <= most_slots ? 1u << log : 0;
  // More items than a wave of CTAs, and all of them short. 400 sequences of 64
  // slots, 12 x 64 bf16: 13.7 us against 29 us in runs; 1000 of 100, fp16: 57 us
  // against 79 us; 200 of 200, 8 x 128 bf16 for 32 heads: 46 us against 43 us.
  L.warps = L.ranks == 0 && items > wave && slots <= kShortUnits * L.kernel.unit;
  if (L.ranks != 0 || L.warps) {
    const int64_t by_warp = std::min((items + kWarps - 1) / kWarps, int64_t(held.warp_per_sm) * sms);
    L.ctas = static_cast<unsigned>(L.warps ? by_warp : items * L.ranks);
    L.lse2 = 0;
    L.scores = with_acc ? round256(static_cast<size_t>(c.seqs) * q_heads * 4) : 0;
    L.bytes = L.scores + (with_acc ? static_cast<size_t>(c.seqs) * q_heads * c.capacity * 4 : 0);
    *out = L;
    return W4_OK;
  }
  L.ctas = static_cast<unsigned>(most < wave ? (most > 0 ? most : 1) : wave);
  L.part_stride = (int64_t(L.kernel.rows) * (c.dim + 2) + 3) / 4 * 4;
  L.meta = round256(size_t(2) * L.ctas * L.part_stride * 4);
  L.lse2 = L.meta + round256(static_cast<size_t>(items) * sizeof(int2));
  L.scores = L.lse2 + (with_acc ? round256(static_cast<size_t>(c.seqs) * q_heads * 4) : 0);
  L.bytes = L.scores + (with_acc ? static_cast<size_t>(c.seqs) * q_heads * c.capacity * 4 : 0);
  *out = L;
  return W4_OK;
}

w4_status check_heads(const w4kv::View& c, int64_t q_heads) {
  if (q_heads < 1 || q_heads > (1 << 20) || q_heads % c.heads != 0)
    return w4host::fail(W4_ERR_SHAPE, "q_heads=%lld is not a multiple of kv_heads=%d", (long long)q_heads, int(c.heads));
  return W4_OK;
}

}  // namespace

extern "C" size_t kv_attend_workspace_size(const kv_cache* c, int64_t q_heads, int32_t with_acc) {
  using namespace w4host;
  w4kv::View v;
  const DeviceInfo* di = nullptr;
  if (check_cache(c, "cache", &v) != W4_OK || check_heads(v, q_heads) != W4_OK || c->seqs == 0 ||
      current_device(&di) != W4_OK)
    return 0;
  // a window may choose another kernel: the larger need of both
  const int32_t group = static_cast<int32_t>(q_heads / v.heads);
  size_t bytes = 0;
  for (const int64_t slots : {int64_t(v.capacity), int64_t(1)}) {
    Layout L;
    if (lay_out(v, choose(v, c->type, group, slots), v.capacity, q_heads, with_acc != 0, *di, &L) != W4_OK) return 0;
    bytes = std::max(bytes, L.bytes);
  }
  return bytes;
}

extern "C" w4_status kv_attend(const kv_cache* c, const float* q, int64_t ldq, int64_t q_heads, float scale,
                               int64_t window, float* out, int64_t ldo, float* lse, float* acc, int64_t ldacc,
                               void* workspace, size_t workspace_bytes, void* stream) {
  using namespace w4host;
  AttendParams p = {};
  w4_status rc = check_cache(c, "cache", &p.c);
  if (rc != W4_OK) return rc;
  rc = check_heads(p.c, q_heads);
  if (rc != W4_OK) return rc;
  if (window < 0) return fail(W4_ERR_VALUE, "window=%lld is negative", (long long)window);
  p.scale2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
  if (!(p.scale2 > -INFINITY && p.scale2 < INFINITY)) return fail(W4_ERR_VALUE, "scale is not finite, or too large");
  if (c->seqs == 0) return W4_OK;
  if (q == nullptr || out == nullptr) return fail(W4_ERR_NULL, "q and out must not be NULL");
  if (c->seqs > 1 && (ldq < q_heads * c->head_dim || ldo < q_heads * c->head_dim))
    return fail(W4_ERR_SHAPE, "ldq and ldo must be at least q_heads * head_dim");
  if (acc != nullptr && c->seqs > 1 && ldacc < p.c.capacity)
    return fail(W4_ERR_SHAPE, "ldacc=%lld is below the capacity of %d slots", (long long)ldacc, int(p.c.capacity));
  const auto bits = [](const void* x) { return reinterpret_cast<uintptr_t>(x); };
  if ((bits(q) | bits(out) | bits(lse) | bits(acc)) & 3)
    return fail(W4_ERR_ALIGN, "q, out, lse and acc must be 4-byte aligned");
  const DeviceInfo* di = nullptr;
  rc = current_device(&di);
  if (rc != W4_OK) return rc;
  Layout L;
  const int64_t slots = window > 0 ? std::min(window, int64_t(p.c.capacity)) : p.c.capacity;
  const AttendKernel kernel = choose(p.c, c->type, static_cast<int32_t>(q_heads / c->kv_heads), slots);
  rc = lay_out(p.c, kernel, slots, q_heads, acc != nullptr, *di, &L);
  if (rc != W4_OK) return rc;
  if (L.bytes > 0 && (workspace == nullptr || workspace_bytes < L.bytes))
    return fail(W4_ERR_WORKSPACE, "kv_attend needs a workspace of %zu bytes, %zu given", L.bytes,
                workspace == nullptr ? size_t(0) : workspace_bytes);
  if (bits(workspace) & 15) return fail(W4_ERR_WORKSPACE, "workspace must be 16-byte aligned");
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.q = q;
  p.ldq = ldq;
  p.out = out;
  p.ldo = ldo;
  p.lse = lse;
  p.part = reinterpret_cast<float*>(ws);
  p.meta = reinterpret_cast<int2*>(ws + L.meta);
  if (acc != nullptr) {
    p.lse2 = reinterpret_cast<float*>(ws + L.lse2);
    p.scores = reinterpret_cast<float*>(ws + L.scores);
  }
  p.part_stride = L.part_stride;
  p.window = window;
  p.group = static_cast<int32_t>(q_heads / c->kv_heads);
  p.rows = L.kernel.rows;
  p.over = L.kernel.over;
  p.least = std::max(1, kLeastSlots / L.kernel.unit);
  while ((1 << p.unit_log) < L.kernel.unit) ++p.unit_log;
  p.q_vec = (bits(q) & 15) == 0 && (c->seqs <= 1 || ldq % 4 == 0);
  p.chunks = L.chunks;
  p.err = di->err;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_pdl(L.ranks != 0 ? L.kernel.item_fn : (L.warps ? L.kernel.warp_fn : L.kernel.fn), dim3(L.ctas),
                             kAttendThreads, L.warps ? L.kernel.warp_smem : L.kernel.smem, st,
                             L.ranks != 0 ? L.ranks : 1, true, p);
  if (e != cudaSuccess) return cuda_fail(e, "launch kv_attend");
  int64_t joins = 0, gathers = 0, per_seq = 1;
  int wpr = 1;
  if (L.ranks == 0 && !L.warps) {
    const int64_t rows = c->seqs * q_heads;
    wpr = rows <= int64_t(di->sms) * kJoinWarps ? kJoinWarps : 1;
    const int64_t rows_per_cta = kJoinWarps / wpr;
    joins = (rows + rows_per_cta - 1) / rows_per_cta;
  }
  if (acc != nullptr && p.c.capacity > 0) {
    const int64_t tiles = (int64_t(p.c.capacity) + 31) / 32;
    const int64_t fair = std::max<int64_t>(1, int64_t(kGatherCtas) * di->sms / c->seqs);
    per_seq = std::min(tiles, fair);
    gathers = per_seq * c->seqs;
  }
  if (joins + gathers > 0) {
    e = launch_pdl(behind_kernel, dim3(static_cast<unsigned>(joins + gathers)), kJoinThreads, 0, st, 1, true, p,
                   static_cast<int>(joins), wpr, static_cast<int>(per_seq), acc, ldacc);
    if (e != cudaSuccess) return cuda_fail(e, "launch kv_attend (join)");
  }
  return W4_OK;
}
