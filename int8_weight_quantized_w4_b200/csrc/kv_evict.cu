// kv_evict: cuts sequences to the slots that the attention has used most.
//
// select_kernel: one cluster per sequence. The threshold, the key of the last
// slot that stays, is found exactly by four passes over 8-bit digits of an
// order-preserving key (a histogram a pass, in shared memory, added up over
// the cluster's CTAs); ties at the threshold stay from the lowest slot on. A
// last pass counts the slots before each one and writes the kept slots' list.
// move_kernel: the kept rows of keys, values and scales to the front. Row i
// comes from slot list[i] >= i, so a batch of rows that is read before any of
// it is written can be written in place, and never touches what a later
// batch reads: in place one CTA takes the batches of one (sequence, head,
// keys or values, 64-byte column) in order, elsewhere batches are dealt out.
#include <cooperative_groups.h>

#include "kv_cache.cuh"

namespace {

using namespace w4kv;
namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;

struct EvictParams {
  View c, d;
  const float* acc;
  float* acc_out;
  int64_t ldacc, ldacc_out;
  int32_t* list;  // the kept slots, rows of `ldlist`
  int64_t ldlist;
  int32_t pad;    // entries of a list row that are -1 behind the last (0: the caller wants no list)
  float* kept_acc;  // their weights, rows of `ldkept_acc`
  int64_t ldkept_acc;
  int32_t keep, recent;
  ErrorWord* err;
};

// The weight as an unsigned key of the same order; NaN below everything.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w == 0.f ? 0.f : w);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const EvictParams p) {
  __shared__ uint32_t hist[2][256];   // this CTA's counts: one pass fills one while others read the other
  __shared__ uint32_t total[256];
  __shared__ uint32_t picked[2];      // the digit, and how many of it are still wanted
  __shared__ uint32_t counts[2];      // slots of this CTA above the threshold, and at it
  __shared__ uint32_t warp_counts[2][kSelWarps];
  pdl_launch_dependents();
  pdl_wait();
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int32_t b = blockIdx.x / ranks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t n = held_length(p.c, b, p.err, w4dev::K_KV_EVICT);
  const float* acc = p.acc + b * p.ldacc;
  float* acc_out = p.acc_out + b * p.ldacc_out;
  int32_t* list = p.list + b * p.ldlist;
  float* kept_acc = p.kept_acc + b * p.ldkept_acc;
  int32_t fresh = min(n, p.keep);
  if (fresh > p.d.capacity) {
    if (rank == 0 && tid == 0) w4dev::record_error(p.err, W4_ERR_VALUE, w4dev::K_KV_EVICT, b);
    fresh = p.d.capacity;
  }
  const int32_t first = rank * kSelThreads + tid, step = ranks * kSelThreads;
  if (n <= p.keep) {
    for (int32_t i = first; i < fresh; i += step) {
      list[i] = i;
      if (acc_out != acc) acc_out[i] = acc[i];
    }
  } else {
    const int32_t recent = min(p.recent, p.keep);
    const int32_t m = n - recent;          // the slots that compete
    uint32_t want = p.keep - recent;       // and how many of them stay
    const int32_t chunk = ((n + ranks - 1) / ranks + kSelThreads - 1) / kSelThreads * kSelThreads;
    const int32_t c0 = min(n, rank * chunk), c1 = min(n, c0 + chunk);
    uint32_t prefix = 0;
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = 24 - 8 * pass;
      uint32_t* mine = hist[pass & 1];
      if (tid < 256) mine[tid] = 0;
      __syncthreads();
      for (int32_t i = c0 + tid; i < min(c1, m); i += kSelThreads) {
        const uint32_t k = weight_key(acc[i]);
        if (pass == 0 || (k >> (shift + 8)) == prefix) atomicAdd(&mine[(k >> shift) & 255u], 1u);
      }
      cluster.sync();
      if (tid < 256) {
        uint32_t sum = 0;
        for (int r = 0; r < ranks; ++r) sum += cluster.map_shared_rank(mine, r)[tid];
        total[tid] = sum;
      }
      __syncthreads();
      if (warp == 0) {
        // lane l takes digits 8 l .. 8 l + 7, the largest digits first
        uint32_t own = 0;
        for (int j = 0; j < 8; ++j) own += total[8 * lane + j];
        uint32_t above = own;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const uint32_t v = __shfl_down_sync(0xffffffffu, above, o);
          if (lane + o < 32) above += v;
        }
        above -= own;  // in the digits of the lanes above
        for (int j = 7; j >= 0; --j) {
          const uint32_t t = total[8 * lane + j];
          if (above < want && want <= above + t) {
            picked[0] = 8 * lane + j;
            picked[1] = want - above;
          }
          above += t;
        }
        if (want == 0 && lane == 0) {
          picked[0] = 255;
          picked[1] = 0;
        }
      }
      __syncthreads();
      prefix = (prefix << 8) | picked[0];
      want = picked[1];
      // the others read hist[pass & 1] until they pass the next cluster.sync,
      // behind which the pass after it fills it again
    }
    // `want` of the slots whose key is `prefix` stay, from the lowest on; with
    // nothing wanted from the start no key is above 2^32 - 1
    const bool none = p.keep == recent;
    uint32_t gt = 0, eq = 0;
    for (int32_t i = c0 + tid; i < c1; i += kSelThreads) {
      const uint32_t k = i < m ? weight_key(acc[i]) : 0u;
      gt += i >= m || (!none && k > prefix);
      eq += i < m && !none && k == prefix;
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
      gt += __shfl_xor_sync(0xffffffffu, gt, o);
      eq += __shfl_xor_sync(0xffffffffu, eq, o);
    }
    if (lane == 0) {
      warp_counts[0][warp] = gt;
      warp_counts[1][warp] = eq;
    }
    __syncthreads();
    if (tid < 2) {
      uint32_t sum = 0;
      for (int w = 0; w < kSelWarps; ++w) sum += warp_counts[tid][w];
      counts[tid] = sum;
    }
    cluster.sync();
    uint32_t gt_before = 0, eq_before = 0;
    for (int r = 0; r < rank; ++r) {
      const uint32_t* other = cluster.map_shared_rank(counts, r);
      gt_before += other[0];
      eq_before += other[1];
    }
    for (int32_t t = c0; t < c1; t += kSelThreads) {
      const int32_t i = t + tid;
      const float w = i < c1 ? acc[i] : 0.f;
      const uint32_t k = weight_key(w);
      const bool is_gt = i < c1 && (i >= m || (!none && k > prefix));
      const bool is_eq = i < c1 && i < m && !none && k == prefix;
      const uint32_t vg = __ballot_sync(0xffffffffu, is_gt), ve = __ballot_sync(0xffffffffu, is_eq);
      __syncthreads();
      if (lane == 0) {
        warp_counts[0][warp] = __popc(vg);
        warp_counts[1][warp] = __popc(ve);
      }
      __syncthreads();
      // each warp sums the counts of those before it (32 warps: one each lane)
      uint32_t sg = warp_counts[0][lane], se = warp_counts[1][lane];
      uint32_t bg = lane < warp ? sg : 0u, be = lane < warp ? se : 0u;
#pragma unroll
      for (int o = 16; o > 0; o /= 2) {
        sg += __shfl_xor_sync(0xffffffffu, sg, o);
        se += __shfl_xor_sync(0xffffffffu, se, o);
        bg += __shfl_xor_sync(0xffffffffu, bg, o);
        be += __shfl_xor_sync(0xffffffffu, be, o);
      }
      const uint32_t below = (1u << lane) - 1u;
      const uint32_t g = gt_before + bg + __popc(vg & below), e = eq_before + be + __popc(ve & below);
      if (is_gt || (is_eq && e < want)) {
        const int32_t at = static_cast<int32_t>(g + min(e, want));
        if (at < fresh) {
          list[at] = i;
          kept_acc[at] = w;
        }
      }
      gt_before += sg;
      eq_before += se;
    }
    // every weight has been read: the kept ones may take their new places
    __threadfence();
    cluster.sync();
    for (int32_t i = first; i < fresh; i += step) acc_out[i] = __ldcg(kept_acc + i);
  }
  for (int32_t i = fresh + first; i < n; i += step) acc_out[i] = 0.f;
  for (int32_t i = fresh + first; i < p.pad; i += step) list[i] = -1;
  // the length changes once all of the cluster have read it
  cluster.sync();
  if (rank == 0 && tid == 0) p.d.lengths[b] = fresh;
}

__device__ __forceinline__ int64_t row_of(const View& c, int32_t b, int32_t h, int32_t slot, int64_t* scale,
                                          ErrorWord* err) {
  const int32_t index = c.page.quotient(slot);
  const int32_t page = page_of(c, b, index, err, w4dev::K_KV_EVICT);
  if (page < 0) return -1;
  const int64_t inner = int64_t(h) * c.slots_per_page + (slot - index * c.slots_per_page);
  *scale = int64_t(page) * c.heads * c.slots_per_page + inner;
  return int64_t(page) * c.page_stride + inner * c.dim;
}

// vecs: 16-byte vectors of a row; per: those of this CTA's columns; in place
// the grid's x is the column, elsewhere the batch (and per == vecs).
template <bool IN_PLACE>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictParams p, int vecs, int per, int elem) {
  pdl_launch_dependents();
  pdl_wait();
  const int32_t b = blockIdx.z;
  const bool is_v = blockIdx.y >= static_cast<unsigned>(p.c.heads);
  const int32_t h = is_v ? blockIdx.y - p.c.heads : blockIdx.y;
  const int32_t fresh = p.d.lengths[b];
  const int32_t* list = p.list + b * p.ldlist;
  const uint8_t* src = static_cast<const uint8_t*>(is_v ? p.c.v : p.c.k);
  uint8_t* dst = static_cast<uint8_t*>(is_v ? p.d.v : p.d.k);
  const float* ss = is_v ? p.c.vs : p.c.ks;
  float* ds = is_v ? p.d.vs : p.d.ks;
  const int column = IN_PLACE ? blockIdx.x * per : 0;
  const int width = min(per, vecs - column);
  const int rows = kMoveThreads / width * kMoveUnroll;  // of a batch
  const int my_row = threadIdx.x / width, my_vec = threadIdx.x % width;
  const int stride = kMoveThreads / width;
  const bool live = my_row < stride;
  int32_t r0 = IN_PLACE ? 0 : static_cast<int32_t>(min(int64_t(fresh), int64_t(blockIdx.x) * rows));
  const int32_t end = IN_PLACE ? fresh : min(fresh, r0 + rows);
  for (; r0 < end; r0 += rows) {
    uint4 x[kMoveUnroll];
    float s[kMoveUnroll];
    int64_t to[kMoveUnroll], to_scale[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int32_t r = r0 + u * stride + my_row;
      to[u] = -1;
      if (live && r < end) {
        const int32_t slot = list[r];
        if (!(IN_PLACE && slot == r)) {
          int64_t at_scale = 0;
          const int64_t at = row_of(p.c, b, h, slot, &at_scale, p.err);
          to[u] = at < 0 ? -1 : row_of(p.d, b, h, r, &to_scale[u], p.err);
          if (to[u] >= 0) {
            x[u] = *reinterpret_cast<const uint4*>(src + at * elem + 16 * (column + my_vec));
            if (ss != nullptr && column + my_vec == 0) s[u] = ss[at_scale];
          }
        }
      }
    }
    if (IN_PLACE) __syncthreads();
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      if (to[u] >= 0) {
        *reinterpret_cast<uint4*>(dst + to[u] * elem + 16 * (column + my_vec)) = x[u];
        if (ss != nullptr && column + my_vec == 0) ds[to_scale[u]] = s[u];
      }
    }
  }
}

size_t round256(size_t b) { return (b + 255) / 256 * 256; }

int64_t list_width(const View& c, int64_t keep) { return keep < c.capacity ? keep : c.capacity; }

// [kept weights][kept slots], rows of the most that a sequence can keep
size_t evict_bytes(const View& c, int64_t keep) {
  return 2 * round256(static_cast<size_t>(c.seqs) * static_cast<size_t>(list_width(c, keep)) * 4);
}

}  // namespace

extern "C" size_t kv_evict_workspace_size(const kv_cache* src, int64_t keep) {
  View c;
  if (w4host::check_cache(src, "src", &c) != W4_OK || keep < 0) return 0;
  return evict_bytes(c, keep);
}

extern "C" w4_status kv_evict(const kv_cache* src, const float* acc, int64_t ldacc, int64_t keep, int64_t recent,
                              const kv_cache* dst, float* acc_out, int64_t ldacc_out, int32_t* kept, int64_t ldkept,
                              void* workspace, size_t workspace_bytes, void* stream) {
  using namespace w4host;
  EvictParams p = {};
  w4_status rc = check_cache(src, "src", &p.c);
  if (rc != W4_OK) return rc;
  rc = check_cache(dst, "dst", &p.d);
  if (rc != W4_OK) return rc;
  if (src->kv_heads != dst->kv_heads || src->page_size != dst->page_size || src->head_dim != dst->head_dim ||
      src->type != dst->type || src->seqs != dst->seqs)
    return fail(W4_ERR_SHAPE, "src and dst differ in seqs, heads, page_size, head_dim or type");
  if (keep < 0 || recent < 0 || keep > (int64_t(1) << 30) || recent > (int64_t(1) << 30))
    return fail(W4_ERR_VALUE, "keep and recent must lie in 0..2^30");
  if (src->seqs == 0) return W4_OK;
  const bool same_k = src->k == dst->k, same_v = src->v == dst->v, same_len = src->lengths == dst->lengths;
  const bool same_table = src->page_table == dst->page_table && src->ldp == dst->ldp && src->max_pages == dst->max_pages &&
                          src->page_stride == dst->page_stride && src->num_pages == dst->num_pages;
  const bool same_scales = src->k_scales == dst->k_scales && src->v_scales == dst->v_scales;
  const bool in_place = same_k && same_v && same_len && same_table && same_scales;
  if (!in_place && src->max_pages > 0 && dst->max_pages > 0 &&
      (same_k || same_v || (src->k_scales != nullptr && (src->k_scales == dst->k_scales || src->v_scales == dst->v_scales))))
    return fail(W4_ERR_VALUE, "dst shares pages with src but is not the same cache");
  if (!in_place && same_len) return fail(W4_ERR_VALUE, "dst shares its lengths with src but is not the same cache");
  if (dst->ldp == 0 && dst->seqs > 1 && dst->max_pages > 0)
    return fail(W4_ERR_VALUE, "sequences that share one row of pages (ldp == 0) cannot be evicted into");
  if (acc == nullptr || acc_out == nullptr) return fail(W4_ERR_NULL, "acc and acc_out must not be NULL");
  if (src->seqs > 1 && (ldacc < p.c.capacity || ldacc_out < p.c.capacity))
    return fail(W4_ERR_SHAPE, "ldacc and ldacc_out must be at least src's capacity of %d slots", int(p.c.capacity));
  if (acc == acc_out && ldacc != ldacc_out && src->seqs > 1)
    return fail(W4_ERR_SHAPE, "acc_out == acc needs ldacc_out == ldacc");
  if (kept != nullptr && src->seqs > 1 && ldkept < keep) return fail(W4_ERR_SHAPE, "ldkept=%lld < keep", (long long)ldkept);
  const auto bits = [](const void* x) { return reinterpret_cast<uintptr_t>(x); };
  if ((bits(acc) | bits(acc_out) | bits(kept)) & 3) return fail(W4_ERR_ALIGN, "acc, acc_out and kept must be 4-byte aligned");
  const DeviceInfo* di = nullptr;
  rc = current_device(&di);
  if (rc != W4_OK) return rc;
  const size_t need = evict_bytes(p.c, keep);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need))
    return fail(W4_ERR_WORKSPACE, "kv_evict needs a workspace of %zu bytes, %zu given", need,
                workspace == nullptr ? size_t(0) : workspace_bytes);
  if (bits(workspace) & 15) return fail(W4_ERR_WORKSPACE, "workspace must be 16-byte aligned");
  p.acc = acc;
  p.ldacc = ldacc;
  p.acc_out = acc_out;
  p.ldacc_out = ldacc_out;
  p.keep = static_cast<int32_t>(keep);
  p.recent = static_cast<int32_t>(recent);
  p.err = di->err;
  const int64_t width = list_width(p.c, keep);
  p.kept_acc = static_cast<float*>(workspace);
  p.ldkept_acc = width;
  if (kept != nullptr) {
    p.list = kept;
    p.ldlist = ldkept;
    p.pad = p.keep;
  } else {
    p.list = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + need / 2);
    p.ldlist = width;
  }
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  // one cluster per sequence: 8 CTAs while the sequences alone do not fill the
  // SMs and a CTA's share is a few thousand slots or more
  unsigned ranks = 1;
  while (ranks < 8 && src->seqs * ranks * 2 <= di->sms && p.c.capacity / (ranks * 2) >= 2 * kSelThreads) ranks *= 2;
  cudaError_t e = launch_pdl(select_kernel, dim3(static_cast<unsigned>(src->seqs) * ranks), kSelThreads, 0, st, ranks, false, p);
  if (e != cudaSuccess) return cuda_fail(e, "launch kv_evict (select)");
  const int elem = elem_bytes(src->type), vecs = src->head_dim * elem / 16;
  const int64_t most = width < p.d.capacity ? width : p.d.capacity;
  if (most == 0) return W4_OK;
  if (in_place) {
    const int per = vecs < 4 ? vecs : 4;
    const dim3 grid((vecs + per - 1) / per, 2 * src->kv_heads, static_cast<unsigned>(src->seqs));
    e = launch_pdl(move_kernel<true>, grid, kMoveThreads, 0, st, 1, false, p, vecs, per, elem);
  } else {
    const int rows = kMoveThreads / vecs * kMoveUnroll;
    const dim3 grid(static_cast<unsigned>((most + rows - 1) / rows), 2 * src->kv_heads, static_cast<unsigned>(src->seqs));
    e = launch_pdl(move_kernel<false>, grid, kMoveThreads, 0, st, 1, false, p, vecs, vecs, elem);
  }
  return e == cudaSuccess ? W4_OK : cuda_fail(e, "launch kv_evict (move)");
}
