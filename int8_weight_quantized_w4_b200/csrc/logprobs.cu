// token_logprobs: log probabilities of given tokens, entropy and the most
// likely alternatives from rows of logits, in one pass.
//
// Mathematics. With m = max x, l = sum e^(x - m) and t = sum e^(x - m) (x - m):
// lse = m + log l, entropy = log l - t / l. (m, l, t) of two sets of logits
// join by rescaling to the larger m. The alternatives are the largest of
// 64-bit keys (the logit's order above, the complement of the id below), so
// ties need no rule of their own.
//
// Work. A row is one cluster of CTAs, as many as fill the SMs when there are
// few rows; its parts meet in the first one's shared memory. A thread takes 16
// logits at a time: their maximum decides both whether the sums have to be
// rescaled and whether any of them can be an alternative. Each warp keeps its
// best 32 keys sorted, one a lane, and drops what lies below the last wanted
// one of any warp of the CTA (of n unordered logits about top * ln(n / top)
// pass); to begin with, the top-th largest of the threads' first maxima is such
// a bound. Lists and sums are joined pairwise by as many warps. Bound by
// reading the logits (2048 rows of 50257: 69 us on the device, 6.0 TB/s; with 20
// alternatives by the insertions, 94 us), by latency where there are few (one row
// with 5 alternatives: 6.9 us; 58 rows with 20: 11.3 us).
#include <cooperative_groups.h>

#include "kv_cache.cuh"

namespace {

using namespace w4kv;
namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarpsLp = kThreads / 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct LogprobParams {
  const float* logits;
  int64_t ldl;
  const int32_t* tokens;
  int32_t V, top;
  float* logp;
  float* entropy;
  float* top_logp;
  int32_t* top_ids;
  ErrorWord* err;
};

using Key = unsigned long long;

// head_key with NaN below everything (and above 0, the key of no logit).
__device__ __forceinline__ Key logit_key(float x, uint32_t id) {
  if (x != x) return static_cast<Key>(0xFFFFFFFFu - id);
  return w4dev::head_key(x, id);
}

__device__ __forceinline__ float key_logit(Key k) {
  const uint32_t o = static_cast<uint32_t>(k >> 32);
  if (o == 0u) return __int_as_float(0x7fc00000);
  return __uint_as_float((o & 0x80000000u) ? o ^ 0x80000000u : ~o);
}

struct Sums {
  float m, l, t;
};

// l and t about a maximum that lies d <= 0 above the old one's (new = old - d).
// A factor of 0 leaves no t: d times l may have overflowed.
__device__ __forceinline__ void shift(float& l, float& t, float d) {
  const float f = ex2(d * kLog2e);
  t = f > 0.f ? f * fmaf(d, l, t) : 0.f;
  l *= f;
}

// b into a; -Inf for m means that only logits of -Inf (or none) were seen.
__device__ __forceinline__ void join(Sums& a, Sums b) {
  const float m = fmaxf(a.m, b.m);
  if (a.m != -INFINITY) shift(a.l, a.t, a.m - m);
  if (b.m != -INFINITY) shift(b.l, b.t, b.m - m);
  a.l += b.l;
  a.t += b.t;
  a.m = m;
}

// N logits of which `top` is the largest (NaN aside).
template <int N>
__device__ __forceinline__ void add(Sums& s, const float (&x)[N], float top) {
  if (top > s.m) {
    if (s.m != -INFINITY) shift(s.l, s.t, s.m - top);
    s.m = top;
  }
  const float ref = s.m == -INFINITY ? 0.f : s.m;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float d = x[i] - ref;
    const float e = ex2(d * kLog2e);  // NaN goes on: it makes l NaN
    s.l += e;
    s.t = fmaf(e, fmaxf(d, -1e30f), s.t);  // d may be -Inf, where e is 0
  }
}

__device__ __forceinline__ Key shfl_key(Key k, int src) { return __shfl_sync(0xffffffffu, k, src); }

// `k` of some lanes into the warp's sorted list (largest in lane 0).
__device__ __forceinline__ void insert(Key& list, Key k, bool want, int lane) {
  uint32_t votes = __ballot_sync(0xffffffffu, want);
  while (votes != 0) {
    const int src = __ffs(votes) - 1;
    votes &= votes - 1;
    const Key c = shfl_key(k, src);
    const Key up = __shfl_up_sync(0xffffffffu, list, 1);
    if (c > list) list = (lane == 0 || c <= up) ? c : up;
  }
}

// The best 32 of two sorted lists, sorted.
__device__ __forceinline__ Key merge(Key a, Key b, int lane) {
  const Key r = shfl_key(b, 31 - lane);
  Key x = a > r ? a : r;  // bitonic, and the 32 largest of both
#pragma unroll
  for (int o = 16; o > 0; o /= 2) {
    const Key y = __shfl_xor_sync(0xffffffffu, x, o);
    x = (lane & o) == 0 ? (x > y ? x : y) : (x < y ? x : y);
  }
  return x;
}

// The lanes' values sorted, the largest in lane 0.
__device__ __forceinline__ float sort(float x, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k *= 2)
#pragma unroll
    for (int o = k / 2; o > 0; o /= 2) {
      const float y = __shfl_xor_sync(0xffffffffu, x, o);
      x = ((lane & o) == 0) == ((lane & k) == 0 || k == 32) ? fmaxf(x, y) : fminf(x, y);
    }
  return x;
}

// The largest 32 of two sorted lists of values, sorted.
__device__ __forceinline__ float merge(float a, float b, int lane) {
  float x = fmaxf(a, __shfl_sync(0xffffffffu, b, 31 - lane));
#pragma unroll
  for (int o = 16; o > 0; o /= 2) {
    const float y = __shfl_xor_sync(0xffffffffu, x, o);
    x = (lane & o) == 0 ? fmaxf(x, y) : fminf(x, y);
  }
  return x;
}

// The sums and lists of warps 0 .. count - 1 joined into warp 0's, in a fixed
// order; every thread of the CTA calls it.
template <bool TOP>
__device__ __forceinline__ void join_all(Sums& s, Key& list, int count, Sums (&sums)[kWarpsLp],
                                         Key (&keys)[TOP ? kWarpsLp : 1][32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int o = 1; o < count; o *= 2) {
    if (warp < count && (warp & (2 * o - 1)) == o) {
      if (lane == 0) sums[warp] = s;
      if (TOP) keys[TOP ? warp : 0][lane] = list;
    }
    __syncthreads();
    if ((warp & (2 * o - 1)) == 0 && warp + o < count) {
      join(s, sums[warp + o]);
      if (TOP) list = merge(list, keys[TOP ? warp + o : 0][lane], lane);
    }
  }
}

template <bool TOP>
__global__ void __launch_bounds__(kThreads, 4) logprob_kernel(const LogprobParams p) {
  __shared__ Sums sm_sums[kWarpsLp];
  __shared__ Key sm_keys[TOP ? kWarpsLp : 1][32];
  __shared__ Sums cta_sums;
  __shared__ Key cta_keys[32];
  __shared__ Key cta_bar;
  __shared__ float sm_top[TOP ? kWarpsLp : 1][32];
  pdl_launch_dependents();
  pdl_wait();
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int64_t row = blockIdx.x / ranks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float* x = p.logits + row * p.ldl;
  // this CTA's part of the row: whole float4s of an aligned middle, the ragged
  // ends with the first and the last part
  const int32_t lead = min(p.V, static_cast<int32_t>((16 - (reinterpret_cast<uintptr_t>(x) & 15)) % 16 / 4));
  const int32_t quads = (p.V - lead) / 4;
  const int32_t share = (quads + ranks - 1) / ranks;
  const int32_t q0 = min(quads, rank * share), q1 = min(quads, q0 + share);
  const float4* xq = reinterpret_cast<const float4*>(x + lead);

  Sums s = {-INFINITY, 0.f, 0.f};
  Key list = 0;
  Key bar = 0;  // a bound that the wanted keys of the CTA's part do not lie below, and its logit
  float bar_x = -INFINITY;
  const auto raise = [&](Key k) {
    if (k > bar) {
      bar = k;
      const float b = key_logit(bar);
      bar_x = b == b ? b : -INFINITY;
    }
  };
  const auto offer = [&](float v, int32_t id, bool there) {
    const bool maybe = there && !(v < bar_x);
    if (__any_sync(0xffffffffu, maybe)) {
      const Key k = maybe ? logit_key(v, static_cast<uint32_t>(id)) : 0;
      insert(list, k, maybe && k >= bar, lane);
    }
  };
  constexpr int kQuads = 4;  // float4s of a thread at a time
  int32_t q = q0 + warp * 32;
  float4 v[kQuads];
  const auto load = [&](int32_t from) {
#pragma unroll
    for (int u = 0; u < kQuads; ++u) {
      const int32_t at = from + u * kThreads + lane;
      v[u] = at < q1 ? __ldg(xq + at) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    }
  };
  if (q < q1) load(q);
  if (TOP) {
    // `top` logits lie at or above the top-th largest of the threads' first maxima
    float top = -INFINITY;
    if (q < q1) {
#pragma unroll
      for (int u = 0; u < kQuads; ++u) top = fmaxf(top, fmaxf(fmaxf(v[u].x, v[u].y), fmaxf(v[u].z, v[u].w)));
    }
    top = sort(top, lane);
#pragma unroll
    for (int o = 1; o < kWarpsLp; o *= 2) {
      if ((warp & (2 * o - 1)) == o) sm_top[TOP ? warp : 0][lane] = top;
      __syncthreads();
      if ((warp & (2 * o - 1)) == 0) top = merge(top, sm_top[TOP ? warp + o : 0][lane], lane);
    }
    if (warp == 0 && lane == p.top - 1) cta_bar = top > -INFINITY ? logit_key(top, 0xFFFFFFFFu) : 0;
    __syncthreads();
    raise(cta_bar);
  }
  if (warp == kWarpsLp - 1) {
    const int32_t tail = lead + 4 * quads;
    if (rank == 0 && lead > 0) {
      const bool there = lane < lead;
      const float w[1] = {there ? x[lane] : -INFINITY};
      add(s, w, w[0]);
      if (TOP) offer(w[0], lane, there);
    }
    if (rank == ranks - 1 && tail < p.V) {
      const bool there = tail + lane < p.V;
      const float w[1] = {there ? x[tail + lane] : -INFINITY};
      add(s, w, w[0]);
      if (TOP) offer(w[0], tail + lane, there);
    }
  }
  for (; q < q1; q += kQuads * kThreads) {
    float w[4 * kQuads];
#pragma unroll
    for (int u = 0; u < kQuads; ++u) {
      w[4 * u] = v[u].x;
      w[4 * u + 1] = v[u].y;
      w[4 * u + 2] = v[u].z;
      w[4 * u + 3] = v[u].w;
    }
    const int32_t next = q + kQuads * kThreads;
    if (next < q1) load(next);
    float top = w[0];
#pragma unroll
    for (int i = 1; i < 4 * kQuads; ++i) top = fmaxf(top, w[i]);
    add(s, w, top);
    if (TOP) {
      // NaN is never the maximum, and only matters where fewer than `top` others are there
      if (__any_sync(0xffffffffu, !(top < bar_x))) {
        raise(*static_cast<volatile Key*>(&cta_bar));
        // those that may be wanted, a bit each; a warp takes one of each lane at a time
        uint32_t hits = 0;
#pragma unroll
        for (int i = 0; i < 4 * kQuads; ++i)
          hits |= static_cast<uint32_t>(!(w[i] < bar_x)) << i;
        if (bar_x == -INFINITY) {  // which is also what is not there
#pragma unroll
          for (int u = 0; u < kQuads; ++u)
            if (q + u * kThreads + lane >= q1) hits &= ~(15u << (4 * u));
        }
        while (__any_sync(0xffffffffu, hits != 0)) {
          const int i = hits != 0 ? __ffs(hits) - 1 : 0;
          const int32_t id = lead + 4 * (q + i / 4 * kThreads + lane) + i % 4;
          const Key k = hits != 0 ? logit_key(__ldg(x + id), static_cast<uint32_t>(id)) : 0;  // near: it was just read
          insert(list, k, hits != 0 && k >= bar, lane);
          hits &= hits - 1;
        }
        const Key last = shfl_key(list, p.top - 1);
        if (last > bar) {
          raise(last);
          if (lane == 0) atomicMax(&cta_bar, last);
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o /= 2) {
    const Sums b = {__shfl_xor_sync(0xffffffffu, s.m, o), __shfl_xor_sync(0xffffffffu, s.l, o),
                    __shfl_xor_sync(0xffffffffu, s.t, o)};
    join(s, b);
  }
  join_all<TOP>(s, list, kWarpsLp, sm_sums, sm_keys);
  if (ranks > 1) {
    if (warp == 0) {
      if (lane == 0) cta_sums = s;
      if (TOP) cta_keys[lane] = list;
    }
    cluster.sync();
    if (rank == 0) {
      if (warp > 0 && warp < ranks) {
        s = *cluster.map_shared_rank(&cta_sums, warp);
        if (TOP) list = cluster.map_shared_rank(cta_keys, warp)[lane];
      }
      join_all<TOP>(s, list, ranks, sm_sums, sm_keys);
    }
  }
  if (rank == 0 && warp == 0) {
    // l is 0 without a logit above -Inf, NaN with a NaN or +Inf: no distribution
    const float bad = __int_as_float(0x7fc00000);
    const bool none = !(s.l > 0.f);
    const float log_l = log2f(s.l) * kLn2;
    if (lane == 0) {
      if (p.logp != nullptr) {
        const int32_t t = p.tokens[row];
        float out = 0.f;
        if (t >= 0 && t < p.V) {
          out = none ? bad : (x[t] - s.m) - log_l;  // a large m would drown the logarithm in m + log l
        } else if (t != -1) {
          out = bad;
          w4dev::record_error(p.err, W4_ERR_VALUE, w4dev::K_LOGPROBS, t);
        }
        p.logp[row] = out;
      }
      if (p.entropy != nullptr) p.entropy[row] = none ? bad : log_l - s.t / s.l;
    }
    if (TOP && lane < p.top) {
      if (p.top_logp != nullptr) p.top_logp[row * p.top + lane] = none ? bad : (key_logit(list) - s.m) - log_l;
      if (p.top_ids != nullptr)
        p.top_ids[row * p.top + lane] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(list));
    }
  }
  if (ranks > 1) cluster.sync();  // no CTA leaves while its shared memory is read
}

}  // namespace

extern "C" w4_status token_logprobs(const float* logits, int64_t ldl, const int32_t* tokens, int64_t M, int64_t V,
                                    int32_t top, float* logp, float* entropy, float* top_logp, int32_t* top_ids,
                                    void* stream) {
  using namespace w4host;
  if (M < 0 || V < 0) return fail(W4_ERR_SHAPE, "negative size");
  if (top < 0 || top > W4_TOP_MAX) return fail(W4_ERR_VALUE, "top=%d is outside 0..%d", int(top), W4_TOP_MAX);
  if (M == 0) return W4_OK;
  if (V == 0) return fail(W4_ERR_SHAPE, "V == 0: no token to score");
  if (V > 0x7fffffff || M > 0x0fffffff) return fail(W4_ERR_SHAPE, "V must be below 2^31 and M below 2^28");
  if (top > V) return fail(W4_ERR_VALUE, "top=%d is above V=%lld", int(top), (long long)V);
  if (M > 1 && ldl < V) return fail(W4_ERR_SHAPE, "ldl < V");
  if (logits == nullptr) return fail(W4_ERR_NULL, "logits is NULL");
  if (logp != nullptr && tokens == nullptr) return fail(W4_ERR_NULL, "logp needs tokens");
  const auto bits = [](const void* x) { return reinterpret_cast<uintptr_t>(x); };
  if ((bits(logits) | bits(tokens) | bits(logp) | bits(entropy) | bits(top_logp) | bits(top_ids)) & 3)
    return fail(W4_ERR_ALIGN, "all pointers must be 4-byte aligned");
  const DeviceInfo* di = nullptr;
  const w4_status rc = current_device(&di);
  if (rc != W4_OK) return rc;
  const LogprobParams p = {logits, ldl, tokens, static_cast<int32_t>(V), top, logp, entropy, top_logp, top_ids, di->err};
  // CTAs of a row: up to 8, while the rows alone do not give every SM four and
  // a CTA has a few thousand logits or more. 134 rows of 95490: 1 CTA 19.2 us, 2
  // 15.4, 4 (this rule's) 12.0, 8 15.6; 618 of 45918: 1 (this rule's) 27 us, 2 29 us
  unsigned ranks = 1;
  while (ranks < 8 && M * ranks * 2 <= 4 * di->sms && V / (ranks * 2) >= 8 * kThreads) ranks *= 2;
  const cudaError_t e = launch_pdl(top > 0 ? logprob_kernel<true> : logprob_kernel<false>,
                                   dim3(static_cast<unsigned>(M) * ranks), kThreads, 0,
                                   static_cast<cudaStream_t>(stream), ranks, false, p);
  return e == cudaSuccess ? W4_OK : cuda_fail(e, "launch token_logprobs");
}
