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
// item, are cut into units of 64. All units of all items, in that order, are
// dealt to the CTAs in equal contiguous runs, by the lengths on the device: a
// batch of unequal lengths, one long sequence and many short ones all load
// every SM alike, and a CUDA graph stays valid while the lengths grow. A CTA
// holds at most one item that began before its run and one that goes on
// behind it; those leave (m, l, a) in the workspace and join_kernel joins them
// in the order of the slots. So no result depends on timing, and nothing has
// to be zero beforehand.
#pragma once

#include "kv_cache.cuh"

namespace w4kv {

constexpr int kWarps = 4;
constexpr int kAttendThreads = kWarps * 32;
constexpr int kUnit = 64;  // slots of a unit: 4 warps x 16
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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
  ErrorWord* err;
};

// The attended slots [lo, n) of sequence b.
__device__ __forceinline__ void attended(const AttendParams& p, int32_t b, int32_t& lo, int32_t& n) {
  n = held_length(p.c, b, p.err, w4dev::K_KV_ATTEND);
  lo = p.window > 0 && p.window < n ? n - static_cast<int32_t>(p.window) : 0;
}

__device__ __forceinline__ int32_t units_of(const AttendParams& p, int32_t b) {
  int32_t lo, n;
  attended(p, b, lo, n);
  return (n - lo + kUnit - 1) / kUnit;
}

// The CTA that holds unit u, when `total` units are dealt to `ctas` of them:
// the first total % ctas take one more than the others.
__device__ __forceinline__ int64_t owner_of(int64_t u, int64_t total, int64_t ctas) {
  const int64_t q = total / ctas, r = total % ctas;
  return u < r * (q + 1) ? u / (q + 1) : r + (u - r * (q + 1)) / q;
}

// Where this CTA's run of units begins, and its end.
struct Run {
  int64_t total, ctas, u, end;  // all units, CTAs that have any, this one's
  int32_t b, item, unit;        // sequence, item within it, unit within that
};

__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Every thread of the CTA calls it; `s` is shared scratch of kWarps + 3 words.
__device__ inline bool find_run(const AttendParams& p, Run& r, int64_t* s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t items = int64_t(p.c.heads) * p.chunks;
  int64_t mine = 0;
  for (int32_t b = tid; b < p.c.seqs; b += kAttendThreads) mine += units_of(p, b);
  mine = warp_sum(mine);
  if (lane == 0) s[warp] = mine;
  __syncthreads();
  int64_t sum = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) sum += s[w];
  r.total = sum * items;
  r.ctas = r.total < gridDim.x ? r.total : gridDim.x;
  const int64_t c = blockIdx.x;
  if (c >= r.ctas) return false;
  const int64_t q = r.total / r.ctas, rest = r.total % r.ctas;
  r.u = c * q + (c < rest ? c : rest);
  r.end = r.u + q + (c < rest ? 1 : 0);
  // the sequence of unit u: its predecessors hold at most u / items units per item
  const int64_t want = r.u / items;
  int64_t before = 0;
  bool found = false;
  for (int32_t b0 = 0; b0 < p.c.seqs && !found; b0 += kAttendThreads) {
    const int32_t b = b0 + tid;
    const int64_t n = b < p.c.seqs ? units_of(p, b) : 0;
    int64_t up = n;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t v = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += v;
    }
    __syncthreads();
    if (lane == 31) s[warp] = up;
    if (tid == 0) s[kWarps] = -1;
    __syncthreads();
    int64_t all = before;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) up += s[w];
      all += s[w];
    }
    up += before;
    if (up - n <= want && want < up) {
      s[kWarps] = b;
      s[kWarps + 1] = up - n;
      s[kWarps + 2] = n;
    }
    __syncthreads();
    found = s[kWarps] >= 0;
    before = all;
  }
  if (!found) return false;
  r.b = static_cast<int32_t>(s[kWarps]);
  const int64_t inside = r.u - s[kWarps + 1] * items, n = s[kWarps + 2];
  r.item = static_cast<int32_t>(inside / n);
  r.unit = static_cast<int32_t>(inside % n);
  return true;
}

// One CTA's run, segment by segment. Body::run leaves each warp's triple of
// the segment in shared memory (m, l [kWarps][ROWS], a [kWarps][ROWS][dim]);
// the CTA joins the four and writes the result, or a partial.
template <class Body, int ROWS>
__device__ __forceinline__ void attend_runs(const AttendParams& p, float* smem) {
  __shared__ int64_t scratch[kWarps + 3];
  const int D = p.c.dim;
  float* sm_a = smem;
  float* sm_m = sm_a + kWarps * ROWS * D;
  float* sm_l = sm_m + kWarps * ROWS;
  float* sm_body = sm_l + kWarps * ROWS;
  Run r;
  if (!find_run(p, r, scratch)) return;
  const int q_heads = p.c.heads * p.group;
  bool first = true;
  while (r.u < r.end && r.b < p.c.seqs) {
    int32_t lo, n;
    attended(p, r.b, lo, n);
    const int32_t units = (n - lo + kUnit - 1) / kUnit;
    if (units == 0) {
      ++r.b;
      continue;
    }
    const int32_t stop = static_cast<int32_t>(min(int64_t(units), r.unit + (r.end - r.u)));
    const int32_t h = r.item / p.chunks, g0 = (r.item % p.chunks) * p.rows;
    const int ng = min(p.rows, p.group - g0);
    const int32_t q0 = h * p.group + g0;
    const int32_t s0 = lo + r.unit * kUnit, s1 = min(int64_t(n), lo + int64_t(stop) * kUnit);
    Body::run(p, r.b, h, q0, ng, s0, s1, sm_a, sm_m, sm_l, sm_body);
    __syncthreads();
    const bool whole = r.unit == 0 && stop == units;
    const int64_t slot = 2 * int64_t(blockIdx.x) + (first ? 0 : 1);
    float* part = p.part + slot * p.part_stride;
    for (int i = threadIdx.x; i < ng * D; i += kAttendThreads) {
      const int g = i / D, d = i - g * D;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w * ROWS + g]);
      float l = 0.f, a = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float m = sm_m[w * ROWS + g];
        const float f = m == -INFINITY ? 0.f : ex2(m - M);
        // a warp without slots holds zeros; a NaN that it holds stays one
        l += m == -INFINITY ? sm_l[w * ROWS + g] : sm_l[w * ROWS + g] * f;
        a += m == -INFINITY ? sm_a[(w * ROWS + g) * D + d] : sm_a[(w * ROWS + g) * D + d] * f;
      }
      if (whole) {
        p.out[r.b * p.ldo + int64_t(q0 + g) * D + d] = l == 0.f ? 0.f : a / l;
        if (d == 0) {
          const float z = l == 0.f ? -INFINITY : M + log2f(l);
          const int64_t at = int64_t(r.b) * q_heads + q0 + g;
          if (p.lse != nullptr) p.lse[at] = z * kLn2;
          if (p.lse2 != nullptr) p.lse2[at] = z;
        }
      } else {
        part[g * D + d] = a;
        if (d == 0) {
          part[p.rows * D + g] = M;
          part[p.rows * D + p.rows + g] = l;
        }
      }
    }
    if (r.unit == 0 && threadIdx.x == 0) {
      const int64_t last = owner_of(r.u + units - 1, r.total, r.ctas);
      p.meta[int64_t(r.b) * p.c.heads * p.chunks + r.item] =
          make_int2(static_cast<int32_t>(slot), whole ? 1 : static_cast<int32_t>(last - blockIdx.x + 1));
    }
    first = false;
    r.u += stop - r.unit;
    r.unit = 0;
    if (stop == units && ++r.item == p.c.heads * p.chunks) {
      r.item = 0;
      ++r.b;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- plain lanes

// Loads of one tile's rows: which are there, and where.
struct Row {
  int64_t vec;    // first 16-byte vector of the slot's row in k and in v; -1: none
  float ks, vs;   // int8 scales
};

template <int TYPE>
__device__ __forceinline__ Row find_row(const AttendParams& p, int32_t b, int32_t h, int32_t slot, int32_t s1) {
  Row r = {-1, 0.f, 0.f};
  if (slot < s1) {
    const int32_t page = page_of(p.c, b, slot / p.c.slots_per_page, p.err, w4dev::K_KV_ATTEND);
    if (page >= 0) {
      const int32_t inner = h * p.c.slots_per_page + slot % p.c.slots_per_page;
      r.vec = (int64_t(page) * p.c.page_stride + int64_t(inner) * p.c.dim) / Elem<TYPE>::kPerVec;
      if constexpr (TYPE == W4_KV_I8) {
        const int64_t at = int64_t(page) * p.c.heads * p.c.slots_per_page + inner;
        r.ks = p.c.ks[at];
        r.vs = p.c.vs[at];
      }
    }
  }
  return r;
}

// LPR lanes read a row, VPL 16-byte vectors each (interleaved, so that a load
// instruction covers LPR * 16 contiguous bytes of it); a warp's tile is
// 32 / LPR rows at a time, NP times. A lane keeps its part of every row's
// product with q, so the sum over a row's lanes leaves the score with each
// of them and the same lanes add the row's values without an exchange; each
// group of LPR lanes carries its own (m, l, a) and the groups join at the end.
template <int TYPE, int LPR, int VPL, int GT>
struct PlainLanes {
  using E = Elem<TYPE>;
  static constexpr int EPV = E::kPerVec;
  static constexpr int RPW = 32 / LPR;
  static constexpr int NP = LPR == 4 ? 2 : (VPL * GT >= 8 || VPL > 4 ? 2 : 4);
  static constexpr int TS = NP * RPW;
  static constexpr int kBodyFloats = GT * LPR * VPL * EPV;

  __device__ static __forceinline__ void load(uint4 (&x)[NP][VPL], const void* base, const Row& row, int n16) {
    const int lane = threadIdx.x & 31, sub = lane % LPR, rg = lane / LPR;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int64_t at = __shfl_sync(0xffffffffu, row.vec, i * RPW + rg);
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        const int vec = sub + j * LPR;
        x[i][j] = make_uint4(0, 0, 0, 0);
        if (at >= 0 && vec < n16) x[i][j] = __ldg(static_cast<const uint4*>(base) + at + vec);
      }
    }
  }

  __device__ static __forceinline__ void run(const AttendParams& p, int32_t b, int32_t h, int32_t q0, int ng,
                                             int32_t s0, int32_t s1, float* sm_a, float* sm_m, float* sm_l,
                                             float* sq) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % LPR, rg = lane / LPR;
    const int D = p.c.dim, n16 = D / EPV;
    constexpr int W = LPR * VPL * EPV;
    for (int i = threadIdx.x; i < GT * W; i += kAttendThreads) {
      const int g = i / W, d = i % W;
      sq[i] = g < ng && d < D ? p.q[b * p.ldq + int64_t(q0 + g) * D + d] : 0.f;
    }
    __syncthreads();
    float m[GT], l[GT], a[GT][VPL * EPV];
#pragma unroll
    for (int g = 0; g < GT; ++g) {
      m[g] = -INFINITY;
      l[g] = 0.f;
#pragma unroll
      for (int d = 0; d < VPL * EPV; ++d) a[g][d] = 0.f;
    }
    uint4 kx[NP][VPL], vx[NP][VPL];
    int32_t t = s0 + warp * TS;
    Row row = find_row<TYPE>(p, b, h, t + lane, min(s1, t + TS));
    load(kx, p.c.k, row, n16);
    load(vx, p.c.v, row, n16);
#pragma unroll 1
    while (t < s1) {
      const int32_t next = t + kWarps * TS;
      const Row next_row = find_row<TYPE>(p, b, h, next + lane, min(s1, next + TS));
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
          E::unpack(kx[i][j], f);
#pragma unroll
          for (int g = 0; g < GT; ++g)
#pragma unroll
            for (int e = 0; e < EPV; ++e) x[g][i] = fmaf(qv[g][e], f[e], x[g][i]);
        }
      }
      load(kx, p.c.k, next_row, n16);
#pragma unroll
      for (int g = 0; g < GT; ++g)
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
          for (int o = 1; o < LPR; o *= 2) x[g][i] += __shfl_xor_sync(0xffffffffu, x[g][i], o);
      float vs[NP];
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const bool there = __shfl_sync(0xffffffffu, row.vec, i * RPW + rg) >= 0;
        float f = p.scale2;
        if constexpr (TYPE == W4_KV_I8) {
          f *= __shfl_sync(0xffffffffu, row.ks, i * RPW + rg);
          vs[i] = __shfl_sync(0xffffffffu, row.vs, i * RPW + rg);
        }
#pragma unroll
        for (int g = 0; g < GT; ++g) x[g][i] = there ? x[g][i] * f : -INFINITY;
      }
      if (p.scores != nullptr) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const int32_t slot = t + i * RPW + rg;
#pragma unroll
          for (int g = 0; g < GT; ++g)
            if (sub == g % LPR && g < ng && slot < s1)
              p.scores[(int64_t(b) * p.c.heads * p.group + q0 + g) * p.c.capacity + slot] = x[g][i];
        }
      }
#pragma unroll
      for (int g = 0; g < GT; ++g) {
        float top = m[g];
#pragma unroll
        for (int i = 0; i < NP; ++i) top = fmaxf(top, x[g][i]);
        if (top > m[g]) {
          const float f = m[g] == -INFINITY ? 0.f : ex2(m[g] - top);
          if (m[g] != -INFINITY) {
            l[g] *= f;
#pragma unroll
            for (int d = 0; d < VPL * EPV; ++d) a[g][d] *= f;
          }
          m[g] = top;
        }
        const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          x[g][i] = ex2(x[g][i] - ref);
          l[g] += x[g][i];
          if constexpr (TYPE == W4_KV_I8) x[g][i] = x[g][i] * vs[i];
        }
      }
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
          float f[EPV];
          E::unpack(vx[i][j], f);
#pragma unroll
          for (int g = 0; g < GT; ++g)
#pragma unroll
            for (int e = 0; e < EPV; ++e) a[g][j * EPV + e] = fmaf(x[g][i], f[e], a[g][j * EPV + e]);
        }
      load(vx, p.c.v, next_row, n16);
      row = next_row;
      t = next;
    }
    // the groups' triples into one
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
        sm_m[warp * GT + g] = top;
        sm_l[warp * GT + g] = l[g];
      }
      if (rg == 0) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
          const int vec = sub + j * LPR;
          if (vec < n16) {
#pragma unroll
            for (int e = 0; e < EPV; ++e) sm_a[(warp * GT + g) * D + vec * EPV + e] = a[g][j * EPV + e];
          }
        }
      }
    }
  }
};

template <class Body, int ROWS>
__global__ void __launch_bounds__(kAttendThreads) attend_kernel(const AttendParams p) {
  extern __shared__ __align__(16) float attend_smem[];
  pdl_launch_dependents();
  pdl_wait();
  attend_runs<Body, ROWS>(p, attend_smem);
}

// A kernel of the table: how it is launched, what it takes.
struct AttendKernel {
  void (*fn)(const AttendParams);
  int rows;        // query heads of an item
  int body_floats; // shared memory of the body
};

// The kernel for a call of this element type (one translation unit a type).
template <int TYPE>
AttendKernel attend_kernel_for(int32_t dim, int32_t group);

template <int TYPE, int LPR, int VPL>
AttendKernel plain_kernel_for(int32_t group) {
  if (group == 1)
    return {attend_kernel<PlainLanes<TYPE, LPR, VPL, 1>, 1>, 1, PlainLanes<TYPE, LPR, VPL, 1>::kBodyFloats};
  if (group == 2)
    return {attend_kernel<PlainLanes<TYPE, LPR, VPL, 2>, 2>, 2, PlainLanes<TYPE, LPR, VPL, 2>::kBodyFloats};
  return {attend_kernel<PlainLanes<TYPE, LPR, VPL, 4>, 4>, 4, PlainLanes<TYPE, LPR, VPL, 4>::kBodyFloats};
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
