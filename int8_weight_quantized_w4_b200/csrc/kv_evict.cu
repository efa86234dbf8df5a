// kv_evict: cuts sequences to the slots that the attention has used most.
//
// select_kernel: one cluster per sequence, whose CTAs hold its weights in shared
// memory (up to 16640 each). The threshold, the key of the last slot that
// stays, is found exactly by passes over the digits of an order-preserving key:
// a histogram a pass, in shared memory, added up over the cluster's CTAs, and
// searched from above. A digit has 12 bits (10 for short sequences, whose CTAs
// are small), since a first one of 8 has a float's exponent in few bins, which
// the adding threads wait for (16 sequences of up to 16000 slots: 24 us), and
// two passes tell most thresholds apart. Ties at it stay from the lowest slot
// on. Then each thread places four neighbouring slots behind the kept ones
// before them: the kept slots' list. Slots on pages that do not exist leave it
// again, in a pass of their own that only broken page tables bring about.
// move_kernel: the kept rows of keys, values and scales to the front. A CTA
// looks up the places of its rows once and moves them for several heads, the
// next head's rows on their way while one's are written. Row i comes from slot
// list[i] >= i, so a batch of rows that is read before any of it is written can
// be written in place, and never touches what a later batch reads: in place
// one CTA takes the batches of one 64-byte column in order, elsewhere batches
// are dealt out.
// Measured: 16 sequences of up to 16000 slots cut to 2045, 8 x 128 bf16 into
// other pages, 51 us: 15 us to select, bound by its passes' barriers, and 36 us
// to move, 6.3 TB/s; in place 57 us; one 12 x 64 fp32 sequence of 1024 slots cut to
// 512, 8.0 us, in place 10.6 us.
#include <cooperative_groups.h>

#include "kv_cache.cuh"

namespace {

using namespace w4kv;
namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024;
constexpr int kSelSmall = 256;      // for sequences of up to kSmall slots: 9 us against 10 us with 1024 threads
constexpr int kSmall = 2048;
constexpr int kMaxRanks = 8;        // CTAs of a selecting cluster
constexpr int kMoveThreads = 256;
// CTAs an SM that the heads are shared out for: one sequence of 131072 slots, 8 x
// 128 bf16, cut to 8192, 29.3 us (with 2 28.5 us, with 8 31.1 us); one of 5000, 12 x
// 64 fp32, 15.2 us (15.9 us, 15.2 us).
constexpr int kMoveCtas = 4;
// Slots that a sequence grows by another CTA at: 16 of up to 16000 slots 52.1 us
// (with 2080 54.4 us, with 8320 53.8 us); one of 8000 17.6 us (17.1 us, 18.5 us).
constexpr int kShare = 4160;
constexpr int kHeld = 16640;        // weights that a selecting CTA keeps in shared memory

// Rows of a moving thread at a time. In place a batch is read as a whole before
// it is written, and int8 rows are short: 4 (16 x <= 16000 slots of 128 bf16 in place
// 58 us, 66 us with 2; int8 into other pages 39.5 us, 41 us); else 2 (64 x <= 2000
// fp16 73 us, 75.5 us with 4; one 12 x 64 sequence of 1024 8.0 us, 9.1 us).
constexpr int move_unroll(bool in_place, bool scales) { return in_place || scales ? 4 : 2; }

struct EvictParams {
  View c, d;
  const float* acc;
  float* acc_out;
  int64_t ldacc, ldacc_out;
  int32_t* list;  // the kept slots, rows of `ldlist`
  int64_t ldlist;
  int32_t pad;    // entries of a list row that are -1 behind the last (0: the caller wants no list)
  float* kept_acc;  // their weights, rows of `ldkept_acc` (where a CTA does not hold them)
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

// Both with those of the lanes above added.
__device__ __forceinline__ void suffix_sums(uint32_t& a, uint32_t& b, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const uint32_t v = __shfl_down_sync(0xffffffffu, a, o), w = __shfl_down_sync(0xffffffffu, b, o);
    if (lane + o < 32) {
      a += v;
      b += w;
    }
  }
}

// A digit has a bin for each quarter of a thread.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) select_kernel(const EvictParams p, int32_t room) {
  constexpr int kBits = THREADS == 1024 ? 12 : 10, kBins = 1 << kBits, kWarps = THREADS / 32;
  static_assert(kBins == 4 * THREADS, "four digits a thread");
  extern __shared__ float weights[];  // of this CTA's slots, where there is room for them
  __shared__ __align__(16) uint32_t hist[2][kBins];  // this CTA's counts: one pass fills one while others read the other
  __shared__ uint32_t coarse[2][32];  // each warp's digits', of this CTA
  __shared__ uint32_t picked[5];      // see below
  __shared__ uint32_t warp_counts[2][32];
  __shared__ int32_t broken;  // of the first CTA: whether a page id of the sequence names no page
  if (threadIdx.x == 0) broken = 0;
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
  const int32_t first = rank * THREADS + tid, step = ranks * THREADS;
  const int32_t* table = p.c.table + b * p.c.ldp;
  const auto no_page = [&](int32_t id) { return id < 0 || id >= p.c.num_pages; };
  bool bad = false;
  int32_t id = p.c.num_pages - 1;  // looked at last, when it has long arrived
  if (n <= p.keep) {
    const int32_t pages = n > 0 ? p.c.page.quotient(n - 1) + 1 : 0;
    for (int32_t i = first; i < pages; i += step) bad = bad || no_page(table[i]);
    for (int32_t i = first; i < fresh; i += step) {
      list[i] = i;
      if (acc_out != acc) acc_out[i] = acc[i];
    }
    sync_all();  // `broken` is 0 from here on
  } else {
    const int32_t recent = min(p.recent, p.keep);
    const int32_t m = n - recent;          // the slots that compete
    uint32_t want = p.keep - recent;       // and how many of them stay
    const bool none = want == 0;
    const int32_t chunk = ((n + ranks - 1) / ranks + 3) / 4 * 4;
    const int32_t c0 = min(n, rank * chunk), c1 = min(n, c0 + chunk), m1 = min(c1, m);
    const bool held = chunk <= room;
    const auto weight = [&](int32_t i) { return held ? weights[i - c0] : acc[i]; };
    *reinterpret_cast<uint4*>(&hist[0][4 * tid]) = make_uint4(0, 0, 0, 0);
    __syncthreads();
    // the first page ids are on their way while the weights are read
    const int32_t page0 = p.c.page.quotient(c0), pages = c1 > c0 ? p.c.page.quotient(c1 - 1) - page0 + 1 : 0;
    if (tid < pages) id = table[page0 + tid];
    constexpr int kAhead = 8;
    for (int32_t i0 = c0 + tid; i0 < c1; i0 += kAhead * THREADS) {
      float w[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) w[j] = i0 + j * THREADS < c1 ? acc[i0 + j * THREADS] : 0.f;
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int32_t i = i0 + j * THREADS;
        if (i < c1 && held) weights[i - c0] = w[j];
        if (i < m1) atomicAdd(&hist[0][weight_key(w[j]) >> (32 - kBits)], 1u);
      }
    }
    for (int32_t i = tid + THREADS; i < pages; i += THREADS) bad = bad || no_page(table[page0 + i]);
    if (none) sync_all();
    uint32_t prefix = 0;
    uint32_t sure_before = max(0, c0 - m), at_before = 0;  // of the CTAs before: slots that stay for sure, and at the threshold
    int low = 32;                                          // `prefix` holds a key's bits from here on
    for (int pass = 0; low > 0 && !none; ++pass) {
      const int bits = min(low, kBits), shift = low - bits;
      const uint32_t mask = (1u << bits) - 1u;
      uint32_t* mine = hist[pass & 1];
      if (pass > 0) {
#pragma unroll 4
        for (int32_t i = c0 + tid; i < m1; i += THREADS) {
          const uint32_t k = weight_key(weight(i));
          if ((k >> low) == prefix) atomicAdd(&mine[(k >> shift) & mask], 1u);
        }
      }
      __syncthreads();
      const uint4 own4 = *reinterpret_cast<const uint4*>(mine + 4 * tid);
      uint32_t t[4] = {own4.x, own4.y, own4.z, own4.w}, lower[4] = {0, 0, 0, 0};
      uint32_t own = t[0] + t[1] + t[2] + t[3], above = own, above_b = 0;
      if (ranks == 1) suffix_sums(above, above_b, lane);
      const uint32_t sum = ranks == 1 ? above : __reduce_add_sync(0xffffffffu, own);
      if (lane == 0) coarse[pass & 1][warp] = sum;
      sync_all();
      // The digit, by the warp among whose 128 digits it lies: each knows by the
      // cluster's sums of each warp's. Only that one then adds up the digits
      // themselves. `t`: of the cluster, `lower`: of the CTAs before this one;
      // `above`: with all that lies above. (By every warp, 64 KB a CTA through
      // the cluster: 55 us for 51 us.)
      uint32_t tw = 0, bw = 0;
#pragma unroll
      for (int r = 0; r < kMaxRanks; ++r) {  // all on their way at once
        if (r < ranks) {
          const uint32_t x = lane < kWarps ? cluster.map_shared_rank(coarse[pass & 1], r)[lane] : 0u;
          tw += x;
          bw += r < rank ? x : 0u;
        }
      }
      const uint32_t base = __reduce_add_sync(0xffffffffu, lane > warp ? tw : 0u);
      if (base < want && want <= base + __shfl_sync(0xffffffffu, tw, warp)) {
        if (ranks > 1) {
          t[0] = t[1] = t[2] = t[3] = 0;
#pragma unroll
          for (int r = 0; r < kMaxRanks; ++r) {
            if (r < ranks) {
              const uint4 x = *reinterpret_cast<const uint4*>(cluster.map_shared_rank(mine, r) + 4 * tid);
              const uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                t[j] += e[j];
                lower[j] += r < rank ? e[j] : 0u;
              }
            }
          }
          above = own = t[0] + t[1] + t[2] + t[3];
          const uint32_t own_b = lower[0] + lower[1] + lower[2] + lower[3];
          above_b = own_b;
          suffix_sums(above, above_b, lane);
          above_b += __reduce_add_sync(0xffffffffu, lane > warp ? bw : 0u) - own_b;
        }
        above += base - own;
#pragma unroll
        for (int j = 3; j >= 0; --j) {
          if (above < want && want <= above + t[j]) {
            picked[0] = 4 * tid + j;
            picked[1] = want - above;  // how many of the digit stay
            picked[2] = t[j];          // of how many
            picked[3] = above_b;       // above it in the CTAs before
            picked[4] = lower[j];      // and of it
          }
          above += t[j];
          above_b += lower[j];
        }
      }
      // the other buffer's readers are behind the barrier above
      *reinterpret_cast<uint4*>(&hist[(pass + 1) & 1][4 * tid]) = make_uint4(0, 0, 0, 0);
      __syncthreads();
      prefix = pass == 0 ? picked[0] : (prefix << bits) | picked[0];
      want = picked[1];
      sure_before += picked[3];
      at_before = picked[4];
      low = shift;
      if (picked[2] == want) break;  // all of this digit stay: the rest decides nothing
    }
    // `want` of the slots whose key begins with `prefix` stay, from the lowest on
    // Where all CTAs hold their weights (each has as many slots as another or
    // fewer) they have all been read, and may be written over.
    float* out = held ? acc_out : kept_acc;
    int turn = 0;
    for (int32_t t0 = c0; t0 < c1; t0 += 4 * THREADS, turn ^= 1) {
      const int32_t i0 = t0 + 4 * tid;
      uint32_t is_sure = 0, is_at = 0;  // a bit for each of the four
      float w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int32_t i = i0 + j;
        w[j] = i < c1 ? weight(i) : 0.f;
        const uint32_t k = none ? 0u : weight_key(w[j]) >> low;
        if (i < m1) {
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
      if (lane == 31) warp_counts[turn][warp] = up;
      __syncthreads();
      const uint32_t wc = lane < kWarps ? warp_counts[turn][lane] : 0u;
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
            out[at] = w[j];
          }
        }
        g += a;
        e += t;
      }
      sure_before += all & 0xFFFFu;
      at_before += all >> 16;
    }
    if (!held) {  // every weight has been read once all are here: the kept ones may take their new places
      __threadfence();
      sync_all();
      for (int32_t i = first; i < fresh; i += step) acc_out[i] = __ldcg(kept_acc + i);
    }
  }
  for (int32_t i = fresh + first; i < n; i += step) acc_out[i] = 0.f;
  for (int32_t i = fresh + first; i < p.pad; i += step) list[i] = -1;
  if (bad || no_page(id)) *cluster.map_shared_rank(&broken, 0) = 1;
  // the length changes once all of the cluster have read it
  sync_all();
  if (rank != 0) return;
  if (broken != 0) {  // kept slots without a page count as empty: the others close up
    int32_t m = 0;
    int turn = 0;
    for (int32_t i0 = 0; i0 < fresh; i0 += THREADS, turn ^= 1) {
      const int32_t i = i0 + tid, slot = i < fresh ? __ldcg(list + i) : 0;
      const float w = i < fresh ? __ldcg(acc_out + i) : 0.f;
      const bool stays = i < fresh && page_of(p.c, b, p.c.page.quotient(slot), p.err, w4dev::K_KV_EVICT) >= 0;
      const uint32_t votes = __ballot_sync(0xffffffffu, stays);
      if (lane == 0) warp_counts[turn][warp] = __popc(votes);
      __syncthreads();  // and all of this tile has been read
      const uint32_t wc = lane < kWarps ? warp_counts[turn][lane] : 0u;
      const int32_t at = m + __reduce_add_sync(0xffffffffu, lane < warp ? wc : 0u) + __popc(votes & ((1u << lane) - 1u));
      if (stays) {
        list[at] = slot;
        acc_out[at] = w;
      }
      m += __reduce_add_sync(0xffffffffu, wc);
    }
    __syncthreads();
    for (int32_t i = m + tid; i < fresh; i += THREADS) {
      acc_out[i] = 0.f;
      if (i < p.pad) list[i] = -1;
    }
    fresh = m;
  }
  if (tid == 0) p.d.lengths[b] = fresh;
}

// Where slot `slot`'s row of head 0 lies: its number among the rows of k and v,
// and among the scales.
constexpr uint32_t kNoRow = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t row_of(const View& c, int32_t b, int32_t slot, uint32_t* scale, ErrorWord* err) {
  const int32_t index = c.page.quotient(slot);
  const int32_t page = page_of(c, b, index, err, w4dev::K_KV_EVICT);
  if (page < 0) return kNoRow;
  const uint32_t inner = slot - index * c.slots_per_page;
  *scale = static_cast<uint32_t>(page) * (c.heads * c.slots_per_page) + inner;
  return static_cast<uint32_t>(page) * c.page_rows + inner;
}

// A batch's rows of one head's keys or values.
template <int ROWS, bool SCALES>
struct Batch {
  uint4 x[ROWS];
  float s[SCALES ? ROWS : 1];
};

// vecs: 16-byte vectors of a row; per: those of this CTA's columns; in place
// the grid's x is the column, elsewhere the batch (and per == vecs). y: a group
// of `group` heads.
template <bool IN_PLACE, bool SCALES>
__global__ void __launch_bounds__(kMoveThreads, 3) move_kernel(const EvictParams p, int vecs, int per, int group) {
  constexpr int kRows = move_unroll(IN_PLACE, SCALES);
  using Rows = Batch<kRows, SCALES>;
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
  const int rows = stride * kRows;  // of a batch
  const bool live = my_row < stride;
  const bool scales = SCALES && my_vec == 0;
  int32_t r0 = IN_PLACE ? 0 : static_cast<int32_t>(min(int64_t(fresh), int64_t(blockIdx.x) * rows));
  const int32_t end = IN_PLACE ? fresh : min(fresh, r0 + rows);
  for (; r0 < end; r0 += rows) {
    uint32_t from[kRows], to[kRows], from_scale[kRows], to_scale[kRows];
    int32_t slot[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int32_t r = r0 + u * stride + my_row;
      slot[u] = live && r < end ? list[r] : -1;
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int32_t r = r0 + u * stride + my_row;
      from_scale[u] = to_scale[u] = 0;
      from[u] = to[u] = kNoRow;
      if (slot[u] >= 0 && !(IN_PLACE && slot[u] == r)) {
        from[u] = row_of(p.c, b, slot[u], &from_scale[u], p.err);
        to[u] = row_of(p.d, b, r, &to_scale[u], p.err);
        if (from[u] == kNoRow) to[u] = kNoRow;
      }
    }
    // step i: keys of heads h0 .. h1 - 1, then their values
    const auto head = [&](int i) { return i < h1 - h0 ? h0 + i : i - (h1 - h0) + h0; };
    const auto load = [&](Rows& x, int i) {
      const uint32_t h = head(i) * p.c.slots_per_page;
      const uint4* src = static_cast<const uint4*>(i < h1 - h0 ? p.c.k : p.c.v) + my_vec;
      const float* ss = i < h1 - h0 ? p.c.ks : p.c.vs;
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        if (to[u] != kNoRow) {
          x.x[u] = src[uint64_t(from[u] + h) * vecs];
          if (scales) x.s[u] = ss[from_scale[u] + h];
        }
      }
    };
    const auto store = [&](const Rows& x, int i) {
      const uint32_t h = head(i) * p.c.slots_per_page;
      uint4* dst = static_cast<uint4*>(i < h1 - h0 ? p.d.k : p.d.v) + my_vec;
      float* ds = i < h1 - h0 ? p.d.ks : p.d.vs;
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        if (to[u] != kNoRow) {
          dst[uint64_t(to[u] + h) * vecs] = x.x[u];
          if (scales) ds[to_scale[u] + h] = x.s[u];
        }
      }
    };
    Rows even, odd;
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

// CTAs of a sequence's cluster: as many as hold its weights, up to 8, while the
// sequences alone do not fill the SMs.
unsigned select_ranks(const View& c, int sms) {
  unsigned ranks = 1;
  while (ranks < kMaxRanks && int64_t(c.seqs) * ranks * 2 <= sms && (c.capacity + ranks - 1) / ranks + 4 > kShare) ranks *= 2;
  return ranks;
}

// The most slots of a CTA.
int64_t select_share(const View& c, unsigned ranks) { return (int64_t(c.capacity) + ranks - 1) / ranks + 4; }

// [kept weights, unless the CTAs hold them][kept slots, unless the caller gives
// the room], rows of the most that a sequence can keep
size_t kept_bytes(const View& c, int64_t keep) {
  return round256(static_cast<size_t>(c.seqs) * static_cast<size_t>(list_width(c, keep)) * 4);
}
size_t evict_bytes(const View& c, int64_t keep, bool with_kept, int sms) {
  return (select_share(c, select_ranks(c, sms)) > kHeld ? kept_bytes(c, keep) : 0) + (with_kept ? 0 : kept_bytes(c, keep));
}

}  // namespace

extern "C" size_t kv_evict_workspace_size(const kv_cache* src, int64_t keep, int32_t with_kept) {
  View c;
  const w4host::DeviceInfo* di = nullptr;
  if (w4host::check_cache(src, "src", &c) != W4_OK || keep < 0 || w4host::current_device(&di) != W4_OK) return 0;
  return evict_bytes(c, keep, with_kept != 0, di->sms);
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
  const auto overlap = [](const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
  };
  if (!in_place && !same_len &&
      overlap(src->lengths, static_cast<size_t>(src->seqs) * 4, dst->lengths, static_cast<size_t>(src->seqs) * 4))
    return fail(W4_ERR_VALUE, "dst's lengths overlap src's in part");
  if (!in_place && same_len) return fail(W4_ERR_VALUE, "dst shares its lengths with src but is not the same cache");
  if (dst->ldp == 0 && dst->seqs > 1 && dst->max_pages > 0)
    return fail(W4_ERR_VALUE, "sequences that share one row of pages (ldp == 0) cannot be evicted into");
  if (acc == nullptr || acc_out == nullptr) return fail(W4_ERR_NULL, "acc and acc_out must not be NULL");
  if (src->seqs > 1 && (ldacc < p.c.capacity || ldacc_out < p.c.capacity))
    return fail(W4_ERR_SHAPE, "ldacc and ldacc_out must be at least src's capacity of %d slots", int(p.c.capacity));
  if (acc == acc_out && ldacc != ldacc_out && src->seqs > 1)
    return fail(W4_ERR_SHAPE, "acc_out == acc needs ldacc_out == ldacc");
  if (acc != acc_out) {
    // rows apart from each other may lie between those of the other
    const int64_t cap = p.c.capacity, rows = src->seqs - 1;
    const size_t na = static_cast<size_t>(rows * ldacc + cap) * 4, nb = static_cast<size_t>(rows * ldacc_out + cap) * 4;
    if (overlap(acc, rows > 0 ? na : cap * 4, acc_out, rows > 0 ? nb : cap * 4)) {
      const int64_t off = (reinterpret_cast<intptr_t>(acc_out) - reinterpret_cast<intptr_t>(acc)) / 4;
      const int64_t in = rows > 0 && ldacc == ldacc_out ? ((off % ldacc) + ldacc) % ldacc : 0;
      if (in < cap || ldacc - in < cap) return fail(W4_ERR_VALUE, "acc_out overlaps acc in part");
    }
  }
  if (kept != nullptr && src->seqs > 1 && ldkept < keep) return fail(W4_ERR_SHAPE, "ldkept=%lld < keep", (long long)ldkept);
  const auto bits = [](const void* x) { return reinterpret_cast<uintptr_t>(x); };
  if ((bits(acc) | bits(acc_out) | bits(kept)) & 3) return fail(W4_ERR_ALIGN, "acc, acc_out and kept must be 4-byte aligned");
  const DeviceInfo* di = nullptr;
  rc = current_device(&di);
  if (rc != W4_OK) return rc;
  const size_t need = evict_bytes(p.c, keep, kept != nullptr, di->sms);
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
  const unsigned ranks = select_ranks(p.c, di->sms);
  const int64_t share = select_share(p.c, ranks);
  p.kept_acc = static_cast<float*>(workspace);  // not used where the CTAs hold the weights
  p.ldkept_acc = share > kHeld ? width : 0;
  if (kept != nullptr) {
    p.list = kept;
    p.ldlist = ldkept;
    p.pad = p.keep;
  } else {
    p.list = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + (need - kept_bytes(p.c, keep)));
    p.ldlist = width;
  }
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int32_t room = share <= kHeld ? static_cast<int32_t>(share) : kHeld;
  static thread_local int ready = -1;
  if (ready != di->dev) {
    const cudaError_t e =
        cudaFuncSetAttribute(select_kernel<kSelThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeld * 4);
    if (e != cudaSuccess) return cuda_fail(e, "kv_evict shared memory");
    ready = di->dev;
  }
  const bool small = p.c.capacity <= kSmall;
  cudaError_t e = launch_pdl(small ? select_kernel<kSelSmall> : select_kernel<kSelThreads>,
                             dim3(static_cast<unsigned>(src->seqs) * ranks), small ? kSelSmall : kSelThreads,
                             static_cast<size_t>(room) * 4, st, ranks, false, p, room);
  if (e != cudaSuccess) return cuda_fail(e, "launch kv_evict (select)");
  const int vecs = src->head_dim * elem_bytes(src->type) / 16;
  const int64_t most = width < p.d.capacity ? width : p.d.capacity;
  if (most == 0) return W4_OK;
  // heads of a CTA: as many as leave every SM a few CTAs
  const int per = in_place ? (vecs < 4 ? vecs : 4) : vecs;
  const int rows = kMoveThreads / per * move_unroll(in_place, src->type == W4_KV_I8);
  const int64_t pieces = in_place ? (vecs + per - 1) / per : (most + rows - 1) / rows;
  int group = src->kv_heads;
  while (group > 1 && pieces * src->seqs * ((src->kv_heads + group - 1) / group) < int64_t(kMoveCtas) * di->sms)
    group = (group + 1) / 2;
  const dim3 grid(static_cast<unsigned>(pieces), (src->kv_heads + group - 1) / group, static_cast<unsigned>(src->seqs));
  void (*const move)(const EvictParams, int, int, int) =
      src->type == W4_KV_I8 ? (in_place ? move_kernel<true, true> : move_kernel<false, true>)
                            : (in_place ? move_kernel<true, false> : move_kernel<false, false>);
  e = launch_pdl(move, grid, kMoveThreads, 0, st, 1, false, p, vecs, per, group);
  return e == cudaSuccess ? W4_OK : cuda_fail(e, "launch kv_evict (move)");
}
