// The attention kernels of kv_attend: one new token per sequence over a paged
// cache.
//
// Mathematics. For one key-value head of one sequence and the query heads g
// that share it, x_gj = scale * q_g . k_j over the attended slots j,
//   m_g = max_j x_gj, l_g = sum_j 2^(x_gj - m_g), a_g = sum_j 2^(x_gj - m_g) v_j
// (x taken to base 2: scale * log2 e is applied to the product), and
// out_g = a_g / l_g. A triple (m, l, a) of any set of slots joins another one
// exactly by rescaling both to the larger m, so the slots can be shared out
// freely and each is read once.
//
// Work. The slots of one (sequence, key-value head, chunk of query heads), an
// item, are cut into units of 16 to 128, a tile for each warp. All units of all
// items, in that order, are dealt to the CTAs in equal contiguous runs, by the
// lengths on the device: a batch of unequal lengths, one long sequence and many
// short ones all load every SM alike, and a CUDA graph stays valid while the
// lengths grow. An item counts one to three units more than it has, what
// beginning and ending it costs. A CTA holds at most one item that began before its run and one that goes on
// behind it; those leave (m, l, a) in the workspace and behind_kernel joins them
// in the order of the slots. So no result depends on timing, and nothing has
// to be zero beforehand. Where one wave of clusters holds all items with a few
// units for each CTA, an item is a cluster instead, and its CTAs join theirs
// through shared memory: one launch, no workspace traffic. And where there are
// more items than that but all are short, each warp takes items of its own.
//
// Latency. Each warp feeds itself: its tiles of 4 to 32 slots follow one another
// across the segments of its CTA's run, and while it works on one the next
// ones are on their way into its ring of stages in shared memory (cp.async,
// which also writes the zeros of slots that are not there), whichever segments
// they belong to; their entries of the page table were fetched a tile earlier.
//
// Measured, on the device: 131072 slots of 8 x 128 bf16 for 32 query heads
// 90 us, 5.9 TB/s of keys and values (0.92 of what a plain copy moves); 48
// sequences of up to 1024 slots, 12 x 64 bf16, 17.4 us (4.4 TB/s), of 1024 all
// 26.1 us (5.8 TB/s); one of 1021 slots, 12 x 64 fp32, 5.7 us, bound by its chain
// of reads.
#pragma once

#include <cooperative_groups.h>

#include "kv_cache.cuh"

namespace w4kv {

namespace cg = cooperative_groups;

constexpr int kWarps = 4;
constexpr int kAttendThreads = kWarps * 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 7.f;  // see the bodies: how far, to base 2, a maximum may pass its reference

struct AttendParams {
  View c;
  const float* q;
  float* out;
  float* lse;      // [seqs][q_heads], NULL: not wanted
  float* lse2;     // the same to base 2, NULL unless weights are gathered
  float* scores;   // x of every attended slot, [seqs][q_heads][capacity], NULL unless weights are gathered
  float* part;     // two partials a CTA, `part_stride` floats each: a [rows][dim], m [rows], l [rows]
  int2* meta;      // an item's first partial and how many CTAs it took
  int64_t ldq, ldo, part_stride;
  int64_t window;  // 0: every slot
  float scale2;    // scale * log2 e
  int32_t group, rows, chunks;  // query heads of a key-value head, of an item, items of a key-value head
  int32_t unit_log;             // slots of a unit: a tile for each warp
  int32_t over;                 // an item's own cost, in units
  int32_t least;                // units that a CTA takes at least
  int32_t q_vec;                // the rows of q are 16-byte aligned
  ErrorWord* err;
};

// The attended slots [lo, n) of sequence b.
__device__ __forceinline__ void attended(const AttendParams& p, int32_t b, int32_t& lo, int32_t& n) {
  n = held_length(p.c, b, p.err, w4dev::K_KV_ATTEND);
  lo = p.window > 0 && p.window < n ? n - static_cast<int32_t>(p.window) : 0;
}

__device__ __forceinline__ int32_t units_of(const AttendParams& p, int32_t slots) {
  return (slots + (1 << p.unit_log) - 1) >> p.unit_log;
}

// What an item of sequence b counts.
__device__ __forceinline__ int32_t cost_of(const AttendParams& p, int32_t b) {
  int32_t lo, n;
  attended(p, b, lo, n);
  return n > lo ? units_of(p, n - lo) + p.over : 0;
}

// How the units are dealt (shared by the CTA): each CTA takes `share` of them,
// the first `extra` one more; this CTA's run ends before unit `end`. The host
// keeps all units below 2^31.
struct Run {
  int32_t share, extra, end;

  // The CTA that holds unit u.
  __device__ __forceinline__ int32_t owner(int32_t u) const {
    const int32_t more = extra * (share + 1);
    return u < more ? u / (share + 1) : extra + (u - more) / share;
  }
};

// What is left of this CTA's run, in units that count `over` more an item.
struct Walk {
  int32_t left;
  int32_t b, item, unit;  // sequence, item within it, unit within that
  int32_t lo, n;          // attended slots of sequence b; n < 0: not read yet
};

// The slots [s0, s1) of one item.
struct Segment {
  int32_t b, h, q0, ng;               // sequence, key-value head, first query head and how many
  int32_t s0, s1;
  int32_t item, count;                // count: CTAs that the item takes, where it begins here; else 0
  bool whole;
};

// Where this CTA's run begins; false if it has none. Every thread of the CTA
// calls it; `s` is shared scratch.
__device__ inline bool find_run(const AttendParams& p, Walk& w, Run& run, int32_t (&s)[kWarps + 3]) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t items = p.c.heads * p.chunks;
  int32_t sum = 0;  // of all sequences' costs, where one pass does not hold them
  if (p.c.seqs > kAttendThreads) {
    int32_t mine = 0;
    for (int32_t b = tid; b < p.c.seqs; b += kAttendThreads) mine += cost_of(p, b);
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) s[warp] = mine;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; ++i) sum += s[i];
  }
  int32_t before = 0, want = 0, u = 0;
  for (int32_t b0 = 0; b0 < p.c.seqs; b0 += kAttendThreads) {
    const int32_t b = b0 + tid;
    const int32_t n = b < p.c.seqs ? cost_of(p, b) : 0;
    int32_t up = n;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int32_t v = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += v;
    }
    __syncthreads();
    if (lane == 31) s[warp] = up;
    if (tid == 0) s[kWarps] = -1;
    __syncthreads();
    int32_t all = before;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) up += s[i];
      all += s[i];
    }
    up += before;
    if (b0 == 0) {
      if (p.c.seqs <= kAttendThreads) sum = all;
      const int32_t total = sum * items, c = blockIdx.x;
      const int32_t ctas = max(min(total, 1), min(total / p.least, static_cast<int32_t>(gridDim.x)));
      if (c >= ctas) return false;
      const int32_t share = total / ctas, extra = total - share * ctas;
      u = c * share + min(c, extra);
      w.left = share + (c < extra ? 1 : 0);
      if (tid == 0) run = {share, extra, u + w.left};
      want = u / items;
    }
    if (up - n <= want && want < up) {
      s[kWarps] = b;
      s[kWarps + 1] = up - n;
      s[kWarps + 2] = n;
    }
    __syncthreads();
    if (s[kWarps] >= 0) {
      const int32_t inside = u - s[kWarps + 1] * items, cost = s[kWarps + 2];
      w.b = s[kWarps];
      w.n = -1;
      w.item = inside / cost;
      w.unit = inside - w.item * cost;
      return true;
    }
    before = all;
  }
  return false;
}

// The next segment of the run; false at its end.
__device__ __forceinline__ bool next_segment(const AttendParams& p, const Run& run, Walk& w, Segment& s) {
  const int32_t items = p.c.heads * p.chunks;
  while (w.left > 0 && w.b < p.c.seqs) {
    if (w.n < 0) attended(p, w.b, w.lo, w.n);  // a sequence's first item
    if (w.n == w.lo) {
      ++w.b;
      w.n = -1;
      continue;
    }
    const int32_t units = units_of(p, w.n - w.lo), cost = units + p.over;
    const int32_t stop = min(cost - w.unit, w.left) + w.unit;
    const int32_t from = max(0, w.unit - p.over), to = max(0, stop - p.over);
    const int32_t last = run.end - w.left + (cost - w.unit) - 1;  // the item's last unit
    s.b = w.b;
    s.item = w.item;
    s.s0 = w.lo + (from << p.unit_log);
    s.s1 = s.s0 + min(w.n - s.s0, (to - from) << p.unit_log);
    w.left -= stop - w.unit;
    w.unit = 0;
    if (stop == cost && ++w.item == items) {
      w.item = 0;
      ++w.b;
      w.n = -1;
    }
    if (from == to) continue;
    s.h = p.chunks == 1 ? s.item : s.item / p.chunks;
    const int32_t g0 = (s.item - s.h * p.chunks) * p.rows;
    s.q0 = s.h * p.group + g0;
    s.ng = min(p.rows, p.group - g0);
    s.whole = from == 0 && to == units;
    s.count = 0;
    if (from == 0) s.count = s.whole ? 1 : run.owner(last) - static_cast<int32_t>(blockIdx.x) + 1;
    return true;
  }
  return false;
}

// A warp's tiles, ahead of the work on them.
template <int TS>
struct Ahead {
  Walk w;
  int32_t b, h, tile, s1;
  int32_t stride;  // slots to this warp's next tile
  bool live;

  __device__ __forceinline__ void open(const AttendParams& p, const Run& run) {
    Segment s;
    do {
      live = next_segment(p, run, w, s);
      if (!live) return;
      b = s.b;
      h = s.h;
      s1 = s.s1;
      stride = kWarps * TS;
      tile = s.s0 + static_cast<int32_t>(threadIdx.x >> 5) * TS;
    } while (tile >= s1);
  }
  // One segment only: the first tile of warp `warp` of `team`.
  __device__ __forceinline__ void only(const Segment& s, int warp, int team) {
    w.left = 0;
    b = s.b;
    h = s.h;
    s1 = s.s1;
    stride = team * TS;
    tile = s.s0 + warp * TS;
    live = tile < s1;
  }
  __device__ __forceinline__ void step(const AttendParams& p, const Run& run) {
    if (!live) return;
    tile += stride;
    if (tile >= s1) open(p, run);
  }
};

// Queries of a segment on their way to shared memory: rows of WIDTH floats,
// zeros behind head_dim and the last row.
template <int ROWS, int WIDTH>
struct Queries {
  static constexpr int N = (ROWS * WIDTH / 4 + kAttendThreads - 1) / kAttendThreads;
  float4 x[N];

  __device__ __forceinline__ void fetch(const AttendParams& p, const Segment& s) {
    const int D = p.c.dim;
    const float* q = p.q + s.b * p.ldq + int64_t(s.q0) * D;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int i = threadIdx.x + n * kAttendThreads, g = i / (WIDTH / 4), d = i % (WIDTH / 4) * 4;
      x[n] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (g < s.ng && d < D) {
        const float* from = q + g * D + d;
        x[n] = p.q_vec ? *reinterpret_cast<const float4*>(from) : make_float4(from[0], from[1], from[2], from[3]);
      }
    }
  }
  __device__ __forceinline__ void store(float* sq) const {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int i = threadIdx.x + n * kAttendThreads;
      if (i < ROWS * WIDTH / 4) *reinterpret_cast<float4*>(sq + 4 * i) = x[n];
    }
  }
};

// A score as it is, or NaN for an infinite one: of a key with an Inf the bodies'
// products are an Inf of either sign or a NaN, and -Inf would weigh nothing.
__device__ __forceinline__ float finite(float x) { return fmaf(x, 0.f, x); }

// (a, m, l) of one quad of a query head's sums.
struct Triple {
  float4 a;
  float m, l;
};

__device__ __forceinline__ Triple no_slots() { return {make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, 0.f}; }

// b into a. A triple without a score (m = -Inf) holds zeros, or a NaN that stays one.
__device__ __forceinline__ void join(Triple& a, const Triple& b) {
  const float m = fmaxf(a.m, b.m);
  const float f = a.m == -INFINITY ? 1.f : ex2(a.m - m), g = b.m == -INFINITY ? 1.f : ex2(b.m - m);
  a.a = make_float4(a.a.x * f + b.a.x * g, a.a.y * f + b.a.y * g, a.a.z * f + b.a.z * g, a.a.w * f + b.a.w * g);
  a.l = a.l * f + b.l * g;
  a.m = m;
}

// A stored triple's quad: a [rows][dim], m [rows], l [rows].
__device__ __forceinline__ Triple stored(const float* t, int rows, int D, int g, int d) {
  return {*reinterpret_cast<const float4*>(t + g * D + d), t[rows * D + g], t[rows * D + rows + g]};
}

__device__ __forceinline__ void store(float* t, int rows, int D, int g, int d, const Triple& x) {
  *reinterpret_cast<float4*>(t + g * D + d) = x.a;
  if (d == 0) {
    t[rows * D + g] = x.m;
    t[rows * D + rows + g] = x.l;
  }
}

// The result of a whole item's quad, query head q of sequence b.
__device__ __forceinline__ void write_out(const AttendParams& p, int32_t b, int32_t q, int d, const Triple& x) {
  float* o = p.out + b * p.ldo + int64_t(q) * p.c.dim + d;
  const float by = x.l == 0.f ? 0.f : 1.f / x.l;  // no slot with a weight: a is 0 too
  o[0] = x.a.x * by;
  o[1] = x.a.y * by;
  o[2] = x.a.z * by;
  o[3] = x.a.w * by;
  if (d == 0) {
    const float z = x.l == 0.f ? -INFINITY : x.m + log2f(x.l);
    const int64_t at = int64_t(b) * p.c.heads * p.group + q;
    if (p.lse != nullptr) p.lse[at] = z * kLn2;
    if (p.lse2 != nullptr) p.lse2[at] = z;
  }
}

// The four warps' triples of a segment (each in a stage of the warp's ring)
// joined, quad by quad: sink(g, d, triple).
template <int ROWS, class Sink>
__device__ __forceinline__ void join_warps(const AttendParams& p, int ng, float* const (&triple)[kWarps], Sink sink) {
  const int D = p.c.dim, quads = D / 4;
  for (int i = threadIdx.x; i < ng * quads; i += kAttendThreads) {
    const int g = i / quads, d = 4 * (i - g * quads);
    Triple x = stored(triple[0], ROWS, D, g, d);
#pragma unroll
    for (int w = 1; w < kWarps; ++w) join(x, stored(triple[w], ROWS, D, g, d));
    sink(g, d, x);
  }
}

// A segment's result, or partial.
template <int ROWS>
__device__ __forceinline__ void finish(const AttendParams& p, const Segment& s, bool first, float* const (&triple)[kWarps]) {
  const int64_t slot = 2 * int64_t(blockIdx.x) + (first ? 0 : 1);
  float* part = p.part + slot * p.part_stride;
  join_warps<ROWS>(p, s.ng, triple, [&](int g, int d, const Triple& x) {
    if (s.whole) {
      write_out(p, s.b, s.q0 + g, d, x);
    } else {
      store(part, ROWS, p.c.dim, g, d, x);
    }
  });
  if (s.count > 0 && threadIdx.x == 0)
    p.meta[int64_t(s.b) * p.c.heads * p.chunks + s.item] = make_int2(static_cast<int32_t>(slot), s.count);
}

// One CTA's run. Body::segment leaves each warp's triple of a segment in the
// free stage of its ring, where it stays until that warp's next tile is begun.
template <class Body, int ROWS>
__device__ __forceinline__ void attend_runs(const AttendParams& p, uint8_t* smem) {
  __shared__ int32_t scratch[kWarps + 3];
  __shared__ Run run;
  __shared__ float* triple[kWarps];
  float* sq = reinterpret_cast<float*>(smem + kWarps * Body::Feed::kRing);
  float* body = sq + ROWS * (Body::kWidth + 2);
  Walk w;
  if (!find_run(p, w, run, scratch)) return;
  __syncthreads();
  Segment s = {}, prev = {};
  Queries<ROWS, Body::kWidth> queries;
  typename Body::Feed feed;
  feed.ahead.w = w;
  bool more = next_segment(p, run, w, s);
  if (more) queries.fetch(p, s);
  feed.ahead.open(p, run);
  feed.begin(p, run, smem + (threadIdx.x >> 5) * Body::Feed::kRing);
  for (int k = 0;; ++k) {
    if (k > 0) {
      more = next_segment(p, run, w, s);
      if (more) queries.fetch(p, s);
      __syncthreads();  // every warp has left the segment before
      finish<ROWS>(p, prev, k == 1, triple);
    }
    if (!more) break;
    queries.store(sq);
    __syncthreads();
    float* to = Body::template segment<kWarps>(p, run, s, feed, sq, body);
    if ((threadIdx.x & 31) == 0) triple[threadIdx.x >> 5] = to;
    prev = s;
  }
}

// One item by a cluster: each CTA takes an equal share of its units, and their
// triples meet in shared memory.
template <class Body, int ROWS>
__device__ __forceinline__ void attend_item(const AttendParams& p, uint8_t* smem) {
  __shared__ float* triple[kWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int32_t ranks = cluster.num_blocks(), rank = cluster.block_rank();
  float* sq = reinterpret_cast<float*>(smem + kWarps * Body::Feed::kRing);
  float* body = sq + ROWS * (Body::kWidth + 2);
  float* mine = sq;  // this CTA's triple, once no warp reads the queries
  const int32_t item = blockIdx.x / ranks, items = p.c.heads * p.chunks;
  const int D = p.c.dim;
  int32_t lo, n;
  Segment s = {};
  s.b = item / items;
  s.item = item - s.b * items;
  attended(p, s.b, lo, n);
  const int32_t units = units_of(p, n - lo);
  const int32_t from = units * rank / ranks, to = units * (rank + 1) / ranks;
  s.h = s.item / p.chunks;
  const int32_t g0 = (s.item - s.h * p.chunks) * p.rows;
  s.q0 = s.h * p.group + g0;
  s.ng = min(p.rows, p.group - g0);
  s.s0 = lo + (from << p.unit_log);
  s.s1 = min(n, lo + (to << p.unit_log));
  const Run run = {};  // not asked: the walk holds no further unit
  typename Body::Feed feed;
  feed.ahead.only(s, threadIdx.x >> 5, kWarps);
  Queries<ROWS, Body::kWidth> queries;
  queries.fetch(p, s);
  feed.begin(p, run, smem + (threadIdx.x >> 5) * Body::Feed::kRing);
  queries.store(sq);
  __syncthreads();
  float* own = Body::template segment<kWarps>(p, run, s, feed, sq, body);
  if ((threadIdx.x & 31) == 0) triple[threadIdx.x >> 5] = own;
  __syncthreads();
  join_warps<ROWS>(p, s.ng, triple, [&](int g, int d, const Triple& x) {
    if (ranks == 1) {
      write_out(p, s.b, s.q0 + g, d, x);
    } else {
      store(mine, ROWS, D, g, d, x);
    }
  });
  if (ranks == 1) return;
  cluster.sync();
  const int quads = D / 4;
  for (int i = rank * kAttendThreads + threadIdx.x; i < s.ng * quads; i += ranks * kAttendThreads) {
    const int g = i / quads, d = 4 * (i - g * quads);
    Triple x = no_slots();
    for (int r = 0; r < ranks; ++r) join(x, stored(cluster.map_shared_rank(mine, r), ROWS, D, g, d));
    write_out(p, s.b, s.q0 + g, d, x);
  }
  cluster.sync();  // no CTA leaves while its triple is read
}

// Short items, one after the other, by each warp.
template <class Body, int ROWS>
__device__ __forceinline__ void attend_warps(const AttendParams& p, uint8_t* smem) {
  constexpr int kOwn = (Body::Feed::kRing + (ROWS * (Body::kWidth + 2) + Body::kBodyFloats) * 4 + 127) / 128 * 128;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint8_t* own = smem + warp * kOwn;
  float* sq = reinterpret_cast<float*>(own + Body::Feed::kRing);
  float* body = sq + ROWS * (Body::kWidth + 2);
  const int32_t items = p.c.heads * p.chunks, all = p.c.seqs * items, D = p.c.dim, quads = D / 4;
  const Run run = {};
  for (int32_t item = blockIdx.x * kWarps + warp; item < all; item += gridDim.x * kWarps) {
    Segment s = {};
    s.b = item / items;
    s.item = item - s.b * items;
    s.h = p.chunks == 1 ? s.item : s.item / p.chunks;
    const int32_t g0 = (s.item - s.h * p.chunks) * p.rows;
    s.q0 = s.h * p.group + g0;
    s.ng = min(p.rows, p.group - g0);
    attended(p, s.b, s.s0, s.s1);
    typename Body::Feed feed;
    feed.ahead.only(s, 0, 1);
    feed.begin(p, run, own);
    const float* q = p.q + s.b * p.ldq + int64_t(s.q0) * D;
    for (int i = lane; i < ROWS * Body::kWidth / 4; i += 32) {
      const int g = i / (Body::kWidth / 4), d = i % (Body::kWidth / 4) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (g < s.ng && d < D) {
        const float* from = q + g * D + d;
        x = p.q_vec ? *reinterpret_cast<const float4*>(from) : make_float4(from[0], from[1], from[2], from[3]);
      }
      *reinterpret_cast<float4*>(sq + 4 * i) = x;
    }
    __syncwarp();
    const float* t = Body::template segment<1>(p, run, s, feed, sq, body);
    __syncwarp();
    for (int i = lane; i < s.ng * quads; i += 32) {
      const int g = i / quads, d = 4 * (i - g * quads);
      write_out(p, s.b, s.q0 + g, d, stored(t, ROWS, D, g, d));
    }
    __syncwarp();  // the next item's first tile may come to where the triple lies
  }
}

// ---------------------------------------------------------------- plain lanes

// A row's entry in the page table on its way from memory: looked at a tile
// later, when it has arrived.
struct Entry {
  int32_t page, inner;  // inner < 0: no row
};

// How a warp's tiles of TS slots come to shared memory. CL lanes copy a row's
// 16-byte vectors, CV each; rows lie PITCH vectors apart. SWIZZLED: the vectors
// of each 128 bytes change places by the row's number in its tile, so that the
// matrix body's reads (4 neighbours of 2 neighbouring rows, or 2 neighbours of
// every other row) meet 8 different places.
template <int TYPE, int TS_, int CL, int CV, int PITCH, bool SWIZZLED, int STAGES, int TRIPLE>
struct Ring {
  static constexpr int TS = TS_;
  static constexpr bool I8 = TYPE == W4_KV_I8;
  static constexpr int kSide = TS * PITCH * 16;  // bytes of a tile's keys, or values
  static constexpr int kScales = 2 * kSide;      // then its int8 scales: keys' [TS], values' [TS]
  static constexpr int kNeed = kScales + (I8 ? 8 * TS : 0);
  static constexpr int kStage = ((kNeed > TRIPLE * 4 ? kNeed : TRIPLE * 4) + 127) / 128 * 128;
  static constexpr int kRing = STAGES * kStage;
  static constexpr int kRows = 32 / CL;          // rows of a copy instruction
  static constexpr uint32_t kAll = 0xFFFFFFFFu >> (32 - TS);  // every slot of a tile

  Ahead<TS> ahead;
  Entry entry;              // of the tile to be copied next
  uint32_t held[STAGES];    // slots that are there, by lane: this tile's, the next one's ...
  uint8_t* ring;
  int put;                  // stage that is free: the next tile's

  // Where vector `vec` of row `row` lies in a side of a stage.
  __device__ static __forceinline__ int place(int row, int vec) {
    if constexpr (SWIZZLED) vec ^= (((row >> 1) ^ (row << 1)) & 3) << 1;
    return (row * PITCH + vec) * 16;
  }

  __device__ __forceinline__ void fetch_entry(const AttendParams& p) {
    const int32_t slot = ahead.tile + static_cast<int32_t>(threadIdx.x) % TS;
    entry = {0, -1};
    if (ahead.live && slot < ahead.s1) {
      const int32_t index = p.c.page.quotient(slot);
      entry.inner = ahead.h * p.c.slots_per_page + (slot - index * p.c.slots_per_page);
      entry.page = p.c.table[ahead.b * p.c.ldp + index];
    }
  }

  // The copies of the next tile into the free stage, as one group.
  __device__ __forceinline__ void push(const AttendParams& p, const Run& run) {
    const int lane = threadIdx.x & 31;
    uint8_t* stage = ring + put * kStage;
    put = put + 1 == STAGES ? 0 : put + 1;
    bool there = entry.inner >= 0;
    if (there && (entry.page < 0 || entry.page >= p.c.num_pages)) {
      w4dev::record_error(p.err, W4_ERR_VALUE, w4dev::K_KV_ATTEND, entry.page);
      there = false;
    }
    const uint32_t mask = __ballot_sync(0xffffffffu, there) & kAll;
#pragma unroll
    for (int i = 0; i + 1 < STAGES; ++i) held[i] = held[i + 1];
    held[STAGES - 1] = mask;
    if (ahead.live) {
      const uint32_t at = there ? static_cast<uint32_t>(entry.page) * p.c.page_rows + entry.inner : 0u;
      const uint32_t n16 = p.c.dim / Elem<TYPE>::kPerVec;
      const int vec = lane % CL;
      const uint32_t to = w4dev::smem_u32(stage);
      const uint8_t* base = static_cast<const uint8_t*>(p.c.k) + vec * 16;
      const int64_t v_off = static_cast<const uint8_t*>(p.c.v) - static_cast<const uint8_t*>(p.c.k);
      if (mask == kAll && n16 == CL * CV) {
#pragma unroll
        for (int i = 0; i < TS / kRows; ++i) {
          const int row = i * kRows + lane / CL;
          const uint8_t* k = base + uint64_t(__shfl_sync(0xffffffffu, at, row)) * (n16 * 16);
#pragma unroll
          for (int j = 0; j < CV; ++j) {
            copy16(to + place(row, vec + j * CL), k + j * CL * 16, 16);
            copy16(to + kSide + place(row, vec + j * CL), k + v_off + j * CL * 16, 16);
          }
        }
      } else {  // zeros for slots that are not there and behind the row's end: nothing is read for them
#pragma unroll 1
        for (int i = 0; i < TS / kRows; ++i) {
          const int row = i * kRows + lane / CL;
          const uint8_t* k = base + uint64_t(__shfl_sync(0xffffffffu, at, row)) * (n16 * 16);
          const bool copy = (mask >> row) & 1u;
#pragma unroll
          for (int j = 0; j < CV; ++j) {
            const bool in = copy && vec + j * CL < n16;
            const uint8_t* from = in ? k + j * CL * 16 : static_cast<const uint8_t*>(p.c.k);
            copy16(to + place(row, vec + j * CL), from, in ? 16 : 0);
            copy16(to + kSide + place(row, vec + j * CL), from + v_off, in ? 16 : 0);
          }
        }
      }
      if constexpr (I8) {  // keys' scales, then values': half the lanes each, or all of them twice
        const int64_t scale = there ? int64_t(entry.page) * (p.c.heads * p.c.slots_per_page) + entry.inner : 0;
#pragma unroll
        for (int i = lane; i < 2 * TS; i += 32)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to + kScales + 4 * i),
                       "l"((i < TS ? p.c.ks : p.c.vs) + scale), "r"(there ? 4 : 0)
                       : "memory");
      }
    }
    w4dev::cp_async_commit();
    ahead.step(p, run);
    fetch_entry(p);
  }

  __device__ static __forceinline__ void copy16(uint32_t to, const uint8_t* from, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
  }

  // The first tiles, once `ahead` is at the very first.
  __device__ __forceinline__ void begin(const AttendParams& p, const Run& run, uint8_t* own) {
    ring = own;
    put = 0;
    fetch_entry(p);
#pragma unroll
    for (int i = 0; i < STAGES; ++i) held[i] = 0;
#pragma unroll
    for (int i = 0; i + 1 < STAGES; ++i) push(p, run);
  }

  // The next tile, arrived: its stage and its slots' mask; the one behind the
  // stages ahead is begun. The tile before is given up.
  __device__ __forceinline__ const uint8_t* take(const AttendParams& p, const Run& run, uint32_t& mask) {
    w4dev::cp_async_wait_group<STAGES - 2>();
    __syncwarp();
    const int at = put + 1 == STAGES ? 0 : put + 1;
    push(p, run);
    mask = held[0];
    return ring + at * kStage;
  }

  // The stage that no tile is in: free until the next take().
  __device__ __forceinline__ float* spare() const {
    __syncwarp();  // the last tile may lie there
    return reinterpret_cast<float*>(ring + put * kStage);
  }
};

// LPR lanes read a row, VPL 16-byte vectors each; a warp reads 32 / LPR rows at
// a time. A lane keeps its part of every row's product with q, so the sum over
// a row's lanes leaves the score with each of them and the same lanes add the
// row's values without an exchange; each group of LPR lanes carries its own
// (m, l, a) and the groups join at the end. Tiles are 4 KB (K and V) or a
// little less, 16, 8 or 4 slots; fp32 rows of more than 128 elements 6 or 8 KB,
// 4 slots.
template <int TYPE, int LPR, int VPL, int GT>
struct PlainLanes {
  using E = Elem<TYPE>;
  static constexpr int EPV = E::kPerVec;
  static constexpr int RPW = 32 / LPR;
  static constexpr int kRowBytes = LPR * VPL * 16;
  static constexpr int NP = kRowBytes * 16 <= 2048 && RPW < 16 ? 16 / RPW : (kRowBytes * 8 <= 2048 && RPW <= 8 ? 8 / RPW : 1);
  static constexpr int TS = NP * RPW;
  static constexpr int kWidth = LPR * VPL * EPV;  // of a row of queries in shared memory
  static constexpr int kBodyFloats = 0;
  static constexpr int kOver = 1;
  static constexpr int kMinCtas = GT * VPL * EPV <= 16 ? 5 : (GT * VPL * EPV <= 32 ? 4 : (GT * VPL * EPV <= 64 ? 3 : 2));
  using Feed = Ring<TYPE, TS, LPR, VPL, LPR * VPL, false, 2, GT * (kWidth + 2)>;

  // The warp's triple of its share (one of TEAM) of the segment: where it has been put.
  template <int TEAM>
  __device__ static __forceinline__ float* segment(const AttendParams& p, const Run& run, const Segment& seg, Feed& feed,
                                                   const float* sq, float*) {
    const int lane = threadIdx.x & 31, warp = TEAM == 1 ? 0 : threadIdx.x >> 5, sub = lane % LPR, rg = lane / LPR;
    const int D = p.c.dim, n16 = D / EPV;
    constexpr int W = kWidth;
    const int32_t s1 = seg.s1;
    float m[GT], l[GT], a[GT][VPL * EPV];
#pragma unroll
    for (int g = 0; g < GT; ++g) {
      m[g] = -INFINITY;
      l[g] = 0.f;
#pragma unroll
      for (int d = 0; d < VPL * EPV; ++d) a[g][d] = 0.f;
    }
#pragma unroll 1
    for (int32_t t = seg.s0 + warp * TS; t < s1; t += TEAM * TS) {
      uint32_t held;
      const uint8_t* stage = feed.take(p, run, held);
      const uint8_t* mine = stage + Feed::place(rg, sub);
      const float* scales = reinterpret_cast<const float*>(stage + Feed::kScales);
      float x[GT][NP];
#pragma unroll
      for (int g = 0; g < GT; ++g)
#pragma unroll
        for (int i = 0; i < NP; ++i) x[g][i] = 0.f;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        float qv[GT][EPV];
#pragma unroll
        for (int g = 0; g < GT; ++g)
#pragma unroll
          for (int e = 0; e < EPV; e += 4)
            *reinterpret_cast<float4*>(&qv[g][e]) =
                *reinterpret_cast<const float4*>(sq + g * W + (sub + j * LPR) * EPV + e);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          float f[EPV];
          E::unpack(*reinterpret_cast<const uint4*>(mine + i * RPW * kRowBytes + j * LPR * 16), f);
#pragma unroll
          for (int g = 0; g < GT; ++g)
#pragma unroll
            for (int e = 0; e < EPV; ++e) x[g][i] = fmaf(qv[g][e], f[e], x[g][i]);
        }
      }
#pragma unroll
      for (int g = 0; g < GT; ++g)
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
          for (int o = 1; o < LPR; o *= 2) x[g][i] += __shfl_xor_sync(0xffffffffu, x[g][i], o);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        float f = p.scale2;
        if constexpr (TYPE == W4_KV_I8) f *= scales[i * RPW + rg];
#pragma unroll
        for (int g = 0; g < GT; ++g) x[g][i] = finite(x[g][i] * f);
      }
      if (held != Feed::kAll) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const bool there = (held >> (i * RPW + rg)) & 1u;
#pragma unroll
          for (int g = 0; g < GT; ++g) x[g][i] = there ? x[g][i] : -INFINITY;
        }
      }
      if (p.scores != nullptr) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const int32_t slot = t + i * RPW + rg;
#pragma unroll
          for (int g = 0; g < GT; ++g)
            if (sub == g % LPR && g < seg.ng && slot < s1)
              p.scores[(int64_t(seg.b) * p.c.heads * p.group + seg.q0 + g) * p.c.capacity + slot] = x[g][i];
        }
      }
#pragma unroll
      for (int g = 0; g < GT; ++g) {
        float top = m[g];
#pragma unroll
        for (int i = 0; i < NP; ++i) top = fmaxf(top, x[g][i]);
        // the reference follows the maximum once it lies kSlack below: weights of up to 2^kSlack are as good
        if (top > m[g] + kSlack) {
          if (m[g] != -INFINITY) {
            const float f = ex2(m[g] - top);
            l[g] *= f;
#pragma unroll
            for (int d = 0; d < VPL * EPV; ++d) a[g][d] *= f;
          }
          m[g] = top;
        }
        const float ref = m[g] == -INFINITY ? 0.f : m[g];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          x[g][i] = ex2(x[g][i] - ref);
          l[g] += x[g][i];
          if constexpr (TYPE == W4_KV_I8) x[g][i] *= scales[TS + i * RPW + rg];
        }
      }
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
          float f[EPV];
          E::unpack(*reinterpret_cast<const uint4*>(mine + Feed::kSide + i * RPW * kRowBytes + j * LPR * 16), f);
#pragma unroll
          for (int g = 0; g < GT; ++g)
#pragma unroll
            for (int e = 0; e < EPV; ++e) a[g][j * EPV + e] = fmaf(x[g][i], f[e], a[g][j * EPV + e]);
        }
    }
    // the groups' triples into one
    float* to = feed.spare();
#pragma unroll
    for (int g = 0; g < GT; ++g) {
      float top = m[g];
#pragma unroll
      for (int o = LPR; o < 32; o *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float f = m[g] == -INFINITY ? 1.f : ex2(m[g] - top);  // without a score it holds zeros, or a NaN
      l[g] *= f;
#pragma unroll
      for (int o = LPR; o < 32; o *= 2) l[g] += __shfl_xor_sync(0xffffffffu, l[g], o);
#pragma unroll
      for (int d = 0; d < VPL * EPV; ++d) {
        a[g][d] *= f;
#pragma unroll
        for (int o = LPR; o < 32; o *= 2) a[g][d] += __shfl_xor_sync(0xffffffffu, a[g][d], o);
      }
      if (lane == 0) {
        to[GT * D + g] = top;
        to[GT * D + GT + g] = l[g];
      }
      if (rg == 0) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
          const int vec = sub + j * LPR;
          if (vec < n16) {
#pragma unroll
            for (int e = 0; e < EPV; e += 4)
              *reinterpret_cast<float4*>(to + g * D + vec * EPV + e) = *reinterpret_cast<const float4*>(&a[g][j * EPV + e]);
          }
        }
      }
    }
    return to;
  }
};

template <class Body, int ROWS>
__global__ void __launch_bounds__(kAttendThreads, Body::kMinCtas) attend_kernel(const AttendParams p) {
  extern __shared__ __align__(128) uint8_t attend_smem[];
  pdl_launch_dependents();
  pdl_wait();
  attend_runs<Body, ROWS>(p, attend_smem);
}

template <class Body, int ROWS>
__global__ void __launch_bounds__(kAttendThreads, Body::kMinCtas) attend_warp_kernel(const AttendParams p) {
  extern __shared__ __align__(128) uint8_t attend_smem[];
  pdl_launch_dependents();
  pdl_wait();
  attend_warps<Body, ROWS>(p, attend_smem);
}

template <class Body, int ROWS>
__global__ void __launch_bounds__(kAttendThreads, Body::kMinCtas) attend_item_kernel(const AttendParams p) {
  extern __shared__ __align__(128) uint8_t attend_smem[];
  pdl_launch_dependents();
  pdl_wait();
  attend_item<Body, ROWS>(p, attend_smem);
}

// A kernel of the table: how it is launched, what it takes.
struct AttendKernel {
  void (*fn)(const AttendParams);       // runs of units
  void (*item_fn)(const AttendParams);  // an item a cluster
  void (*warp_fn)(const AttendParams);  // an item a warp
  int rows;         // query heads of an item
  int unit;         // slots of a unit
  int over;         // an item's own cost, in units
  size_t smem;      // bytes of shared memory; of warp_fn's
  size_t warp_smem;
};

template <class Body, int ROWS>
AttendKernel attend_kernel_of() {
  return {attend_kernel<Body, ROWS>, attend_item_kernel<Body, ROWS>, attend_warp_kernel<Body, ROWS>, ROWS, kWarps * Body::TS, Body::kOver,
          size_t(kWarps) * Body::Feed::kRing + (size_t(ROWS) * (Body::kWidth + 2) + Body::kBodyFloats) * 4,
          size_t(kWarps) *
              ((Body::Feed::kRing + (ROWS * (Body::kWidth + 2) + Body::kBodyFloats) * 4 + 127) / 128 * 128)};
}

// The kernel for a call of this element type (one translation unit a type).
// brief: too few slots for the matrix body, whose staging of the queries is then
// most of its time.
template <int TYPE>
AttendKernel attend_kernel_for(int32_t dim, int32_t group, bool brief);

// Query heads at once: up to 2, and for fp32, whose rows have no exact matrix
// operands, 4, or 8 where their sums fit the registers.
template <int TYPE, int LPR, int VPL>
AttendKernel plain_kernel_for(int32_t group) {
  if (group == 1) return attend_kernel_of<PlainLanes<TYPE, LPR, VPL, 1>, 1>();
  if constexpr (TYPE == W4_KV_F32) {
    if constexpr (VPL <= 4) {
      if (group > 4) return attend_kernel_of<PlainLanes<TYPE, LPR, VPL, 8>, 8>();
    }
    if (group > 2) return attend_kernel_of<PlainLanes<TYPE, LPR, VPL, 4>, 4>();
  }
  return attend_kernel_of<PlainLanes<TYPE, LPR, VPL, 2>, 2>();
}

// The narrowest shape that holds a row's vectors.
template <int TYPE>
AttendKernel plain_kernel_for(int32_t dim, int32_t group) {
  const int n16 = dim / Elem<TYPE>::kPerVec;
  if (n16 <= 4) return plain_kernel_for<TYPE, 4, 1>(group);
  if (n16 <= 8) return plain_kernel_for<TYPE, 8, 1>(group);
  if (n16 <= 12) return plain_kernel_for<TYPE, 4, 3>(group);
  if constexpr (TYPE != W4_KV_I8) {
    if (n16 <= 16) return plain_kernel_for<TYPE, 8, 2>(group);
    if (n16 <= 24) return plain_kernel_for<TYPE, 8, 3>(group);
    if constexpr (TYPE == W4_KV_F32) {
      if (n16 <= 32) return plain_kernel_for<TYPE, 8, 4>(group);
      if (n16 <= 48) return plain_kernel_for<TYPE, 8, 6>(group);
      return plain_kernel_for<TYPE, 8, 8>(group);
    } else {
      return plain_kernel_for<TYPE, 8, 4>(group);
    }
  } else {
    return plain_kernel_for<TYPE, 8, 2>(group);
  }
}

}  // namespace w4kv
