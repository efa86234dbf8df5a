// kv_evict: cuts sequences to the slots that the attention has used most.
//
// select_kernel: one cluster per sequence. The threshold, the key of the last
// slot that stays, is found exactly by four passes over 8-bit digits of an
// order-preserving key (a histogram a pass, in shared memory, added up over
// the cluster's CTAs); ties at the threshold stay from the lowest slot on. A
// CTA reads its weights once and keeps their keys in shared memory, up to
// 16384 of them. Then each thread places four neighbouring slots behind the
// kept ones before them: the kept slots' list.
// move_kernel: the kept rows of keys, values and scales to the front. A CTA
// looks up the places of its rows once and moves them for several heads, the
// next head's rows on their way while one's are written. Row i comes from slot
// list[i] >= i, so a batch of rows that is read before any of it is written can
// be written in place, and never touches what a later batch reads: in place
// one CTA takes the batches of one 64-byte column in order, elsewhere batches
// are dealt out.
#include <cooperative_groups.h>

#include "kv_cache.cuh"

namespace {

using namespace w4kv;
namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;
constexpr int kMoveCtas = 4;        // CTAs an SM that the heads are shared out for
constexpr int kHeldKeys = 16384;    // keys that a selecting CTA keeps in shared memory

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

__global__ void __launch_bounds__(kSelThreads) select_kernel(const EvictParams p, int32_t held_keys) {
  extern __shared__ uint32_t keys[];  // of this CTA's slots, where there is room for them
  __shared__ uint32_t hist[2][256];   // this CTA's counts: one pass fills one while others read the other
  __shared__ uint32_t total[256];
  __shared__ uint32_t picked[4];      // the digit, how many of it are wanted; this CTA's slots above and at it
  __shared__ uint32_t counts[2];      // slots of this CTA that stay for sure, and at the threshold
  __shared__ uint32_t warp_counts[kSelWarps];
  pdl_launch_dependents();
  pdl_wait();
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const auto sync_all = [&]() {
    if (ranks > 1) {
      cluster.sync();
    } else {
      __syncthreads();
    }
  };
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
    const bool none = want == 0;
    const int32_t chunk = ((n + ranks - 1) / ranks + 3) / 4 * 4;
    const int32_t c0 = min(n, rank * chunk), c1 = min(n, c0 + chunk), m1 = min(c1, m);
    const bool held = chunk <= held_keys;
    const auto key_of = [&](int32_t i) { return held ? keys[i - c0] : weight_key(acc[i]); };
    if (tid < 256) hist[0][tid] = 0;
    __syncthreads();
    uint32_t prefix = 0, sure = 0, at_it = 0;  // the last two: this CTA's, of the slots that compete
    for (int pass = 0; pass < 4 && !none; ++pass) {
      const int shift = 24 - 8 * pass;
      uint32_t* mine = hist[pass & 1];
      if (pass == 0) {
#pragma unroll 4
        for (int32_t i = c0 + tid; i < m1; i += kSelThreads) {
          const uint32_t k = weight_key(acc[i]);
          if (held) keys[i - c0] = k;
          atomicAdd(&mine[k >> 24], 1u);
        }
      } else {
#pragma unroll 4
        for (int32_t i = c0 + tid; i < m1; i += kSelThreads) {
          const uint32_t k = key_of(i);
          if ((k >> (shift + 8)) == prefix) atomicAdd(&mine[(k >> shift) & 255u], 1u);
        }
      }
      sync_all();
      if (tid < 256) {
        uint32_t sum = mine[tid];
        if (ranks > 1) {
          sum = 0;
          for (int r = 0; r < ranks; ++r) sum += cluster.map_shared_rank(mine, r)[tid];
        }
        total[tid] = sum;
        hist[(pass + 1) & 1][tid] = 0;  // its readers are behind the barrier above
      }
      __syncthreads();
      if (warp == 0) {
        // lane l takes digits 8 l .. 8 l + 7, the largest digits first
        uint32_t t[8], c[8], own = 0, own_c = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          t[j] = total[8 * lane + j];
          c[j] = mine[8 * lane + j];
          own += t[j];
          own_c += c[j];
        }
        uint32_t above = own, above_c = own_c;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const uint32_t v = __shfl_down_sync(0xffffffffu, above, o), w = __shfl_down_sync(0xffffffffu, above_c, o);
          if (lane + o < 32) {
            above += v;
            above_c += w;
          }
        }
        above -= own;  // in the digits of the lanes above
        above_c -= own_c;
#pragma unroll
        for (int j = 7; j >= 0; --j) {
          if (above < want && want <= above + t[j]) {
            picked[0] = 8 * lane + j;
            picked[1] = want - above;
            picked[2] = above_c;
            picked[3] = c[j];
          }
          above += t[j];
          above_c += c[j];
        }
      }
      __syncthreads();
      prefix = (prefix << 8) | picked[0];
      want = picked[1];
      sure += picked[2];
      at_it = picked[3];
    }
    // `want` of the slots whose key is `prefix` stay, from the lowest on
    uint32_t sure_before = 0, at_before = 0;
    if (ranks > 1) {
      if (tid == 0) {
        counts[0] = sure + max(0, c1 - max(c0, m));
        counts[1] = at_it;
      }
      cluster.sync();
      for (int r = 0; r < rank; ++r) {
        const uint32_t* other = cluster.map_shared_rank(counts, r);
        sure_before += other[0];
        at_before += other[1];
      }
    }
    for (int32_t t0 = c0; t0 < c1; t0 += 4 * kSelThreads) {
      const int32_t i0 = t0 + 4 * tid;
      uint32_t is_sure = 0, is_at = 0;  // a bit for each of the four
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int32_t i = i0 + j;
        if (i < m1) {
          const uint32_t k = key_of(i);
          is_sure |= static_cast<uint32_t>(!none && k > prefix) << j;
          is_at |= static_cast<uint32_t>(!none && k == prefix) << j;
        } else if (i < c1) {
          is_sure |= 1u << j;
        }
      }
      // both counts in one word: a tile's are below 2^16
      const uint32_t own = static_cast<uint32_t>(__popc(is_sure)) | static_cast<uint32_t>(__popc(is_at)) << 16;
      uint32_t up = own;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += v;
      }
      __syncthreads();
      if (lane == 31) warp_counts[warp] = up;
      __syncthreads();
      const uint32_t wc = warp_counts[lane];
      const uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? wc : 0u) + up - own;
      const uint32_t all = __reduce_add_sync(0xffffffffu, wc);
      uint32_t g = sure_before + (before & 0xFFFFu), e = at_before + (before >> 16);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool a = (is_sure >> j) & 1u, t = (is_at >> j) & 1u;
        if (a || (t && e < want)) {
          const int32_t at = static_cast<int32_t>(g + min(e, want));
          if (at < fresh) {
            list[at] = i0 + j;
            kept_acc[at] = acc[i0 + j];
          }
        }
        g += a;
        e += t;
      }
      sure_before += all & 0xFFFFu;
      at_before += all >> 16;
    }
    // every weight has been read: the kept ones may take their new places
    __threadfence();
    sync_all();
    for (int32_t i = first; i < fresh; i += step) acc_out[i] = __ldcg(kept_acc + i);
  }
  for (int32_t i = fresh + first; i < n; i += step) acc_out[i] = 0.f;
  for (int32_t i = fresh + first; i < p.pad; i += step) list[i] = -1;
  // the length changes once all of the cluster have read it
  sync_all();
  if (rank == 0 && tid == 0) p.d.lengths[b] = fresh;
}

// Where slot `slot`'s row of head 0 lies: elements into k and v, and its scale.
__device__ __forceinline__ int64_t row_of(const View& c, int32_t b, int32_t slot, int64_t* scale, ErrorWord* err) {
  const int32_t index = c.page.quotient(slot);
  const int32_t page = page_of(c, b, index, err, w4dev::K_KV_EVICT);
  if (page < 0) return -1;
  const int32_t inner = slot - index * c.slots_per_page;
  *scale = int64_t(page) * c.heads * c.slots_per_page + inner;
  return int64_t(page) * c.page_stride + int64_t(inner) * c.dim;
}

// A batch's rows of one head's keys or values.
struct Batch {
  uint4 x[kMoveUnroll];
  float s[kMoveUnroll];
};

// vecs: 16-byte vectors of a row; per: those of this CTA's columns; in place
// the grid's x is the column, elsewhere the batch (and per == vecs). y: a group
// of `group` heads. rows_of: row and column of a thread.
template <bool IN_PLACE>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictParams p, int vecs, int per, int elem, int group) {
  pdl_launch_dependents();
  pdl_wait();
  const int32_t b = blockIdx.z;
  const int32_t h0 = blockIdx.y * group, h1 = min(p.c.heads, h0 + group);
  const int32_t fresh = p.d.lengths[b];
  const int32_t* list = p.list + b * p.ldlist;
  const int column = IN_PLACE ? blockIdx.x * per : 0;
  const int width = min(per, vecs - column);
  const int stride = kMoveThreads / width;
  const int my_row = threadIdx.x / width, my_vec = column + threadIdx.x % width;
  const int rows = stride * kMoveUnroll;  // of a batch
  const bool live = my_row < stride;
  const bool scales = p.c.ks != nullptr && my_vec == 0;
  const int64_t head = int64_t(p.c.slots_per_page) * p.c.dim * elem;  // bytes from a head to the next
  int32_t r0 = IN_PLACE ? 0 : static_cast<int32_t>(min(int64_t(fresh), int64_t(blockIdx.x) * rows));
  const int32_t end = IN_PLACE ? fresh : min(fresh, r0 + rows);
  for (; r0 < end; r0 += rows) {
    int64_t from[kMoveUnroll], to[kMoveUnroll], from_scale[kMoveUnroll], to_scale[kMoveUnroll];
    int32_t slot[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int32_t r = r0 + u * stride + my_row;
      slot[u] = live && r < end ? list[r] : -1;
    }
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int32_t r = r0 + u * stride + my_row;
      from_scale[u] = to_scale[u] = 0;
      from[u] = to[u] = -1;
      if (slot[u] >= 0 && !(IN_PLACE && slot[u] == r)) {
        from[u] = row_of(p.c, b, slot[u], &from_scale[u], p.err);
        to[u] = row_of(p.d, b, r, &to_scale[u], p.err);
        if (from[u] < 0) to[u] = -1;
        from[u] = from[u] * elem + 16 * my_vec;
        if (to[u] >= 0) to[u] = to[u] * elem + 16 * my_vec;
      }
    }
    const auto load = [&](Batch& x, int i) {  // keys of heads h0 .. h1 - 1, then values
      const int32_t h = i < h1 - h0 ? h0 + i : i - (h1 - h0) + h0;
      const uint8_t* src = static_cast<const uint8_t*>(i < h1 - h0 ? p.c.k : p.c.v) + h * head;
      const float* ss = (i < h1 - h0 ? p.c.ks : p.c.vs) + int64_t(h) * p.c.slots_per_page;
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u) {
        if (to[u] >= 0) {
          x.x[u] = *reinterpret_cast<const uint4*>(src + from[u]);
          if (scales) x.s[u] = ss[from_scale[u]];
        }
      }
    };
    const auto store = [&](const Batch& x, int i) {
      const int32_t h = i < h1 - h0 ? h0 + i : i - (h1 - h0) + h0;
      uint8_t* dst = static_cast<uint8_t*>(i < h1 - h0 ? p.d.k : p.d.v) + h * head;
      float* ds = (i < h1 - h0 ? p.d.ks : p.d.vs) + int64_t(h) * p.c.slots_per_page;
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u) {
        if (to[u] >= 0) {
          *reinterpret_cast<uint4*>(dst + to[u]) = x.x[u];
          if (scales) ds[to_scale[u]] = x.s[u];
        }
      }
    };
    Batch even, odd;
    const int count = 2 * (h1 - h0);  // even
    load(even, 0);
    for (int i = 0; i < count; i += 2) {
      load(odd, i + 1);
      if (IN_PLACE) __syncthreads();  // all rows of i and i + 1 have been read
      store(even, i);
      if (i + 2 < count) load(even, i + 2);
      store(odd, i + 1);
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
  // one cluster per sequence: up to 8 CTAs while the sequences alone do not fill
  // the SMs and a CTA's share is a few thousand slots or more
  unsigned ranks = 1;
  while (ranks < 8 && src->seqs * ranks * 2 <= di->sms && p.c.capacity / (ranks * 2) >= 2 * kSelThreads) ranks *= 2;
  const int64_t share = (p.c.capacity + ranks - 1) / ranks + 4;
  const int32_t held_keys = share <= kHeldKeys ? static_cast<int32_t>(share) : kHeldKeys;
  static thread_local int ready = -1;
  if (ready != di->dev) {
    const cudaError_t e = cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeldKeys * 4);
    if (e != cudaSuccess) return cuda_fail(e, "kv_evict shared memory");
    ready = di->dev;
  }
  cudaError_t e = launch_pdl(select_kernel, dim3(static_cast<unsigned>(src->seqs) * ranks), kSelThreads,
                             static_cast<size_t>(held_keys) * 4, st, ranks, false, p, held_keys);
  if (e != cudaSuccess) return cuda_fail(e, "launch kv_evict (select)");
  const int elem = elem_bytes(src->type), vecs = src->head_dim * elem / 16;
  const int64_t most = width < p.d.capacity ? width : p.d.capacity;
  if (most == 0) return W4_OK;
  // heads of a CTA: as many as leave every SM a few CTAs
  const int per = in_place ? (vecs < 4 ? vecs : 4) : vecs;
  const int rows = kMoveThreads / per * kMoveUnroll;
  const int64_t pieces = in_place ? (vecs + per - 1) / per : (most + rows - 1) / rows;
  int group = src->kv_heads;
  while (group > 1 && pieces * src->seqs * ((src->kv_heads + group - 1) / group) < int64_t(kMoveCtas) * di->sms)
    group = (group + 1) / 2;
  const dim3 grid(static_cast<unsigned>(pieces), (src->kv_heads + group - 1) / group, static_cast<unsigned>(src->seqs));
  if (in_place) {
    e = launch_pdl(move_kernel<true>, grid, kMoveThreads, 0, st, 1, false, p, vecs, per, elem, group);
  } else {
    e = launch_pdl(move_kernel<false>, grid, kMoveThreads, 0, st, 1, false, p, vecs, per, elem, group);
  }
  return e == cudaSuccess ? W4_OK : cuda_fail(e, "launch kv_evict (move)");
}
