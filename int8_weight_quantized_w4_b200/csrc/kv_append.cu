// kv_append: new tokens' keys and values into the pages of a cache, and the
// descriptor checks that the cache's entry points share.
//
// Bound by its bytes (fp32 rows in, stored rows out) for prompts and by
// latency for a decode step. A token is one CTA, or a few warps of one where it
// is short, so that its place in the cache (a search in cu_tokens, the length,
// the page: three dependent reads) is found once, while the token's first
// values are already on their way. int8 rows go to half-warps, 16 lanes of 4
// elements wide, which a row's maximum is reduced over; the others are copied
// as they come, 4 elements a thread. Measured: 7254 tokens of 32 x 96 to bf16
// 48.5 us, 5.5 TB/s (0.85 of a plain copy; 44.4 us where part of the rows lies in
// L2), to int8 74.5 us: a half-warp has one further row on its way; 8 tokens of
// 12 x 64 3.1 us.
#include "kv_cache.cuh"

namespace w4host {

w4kv::Divisor divisor(uint32_t d) {
  uint32_t l = 0;
  while ((1u << l) < d) ++l;
  return {d, static_cast<uint32_t>(((uint64_t((1u << l) - d) << 32) / d) + 1), l};
}

w4_status check_cache(const kv_cache* c, const char* what, w4kv::View* out) {
  if (c == nullptr) return fail(W4_ERR_NULL, "%s is NULL", what);
  if (c->type < W4_KV_F32 || c->type > W4_KV_I8) return fail(W4_ERR_VALUE, "%s: unknown element type %d", what, int(c->type));
  if (c->seqs < 0 || c->num_pages < 0 || c->max_pages < 0) return fail(W4_ERR_SHAPE, "%s: negative size", what);
  if (c->kv_heads < 1 || c->kv_heads > 4096) return fail(W4_ERR_SHAPE, "%s: kv_heads=%d is outside 1..4096", what, int(c->kv_heads));
  if (c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16 != 0)
    return fail(W4_ERR_SHAPE, "%s: head_dim=%d is not a multiple of 16 up to 256", what, int(c->head_dim));
  if (c->page_size < 1 || c->page_size > 65536) return fail(W4_ERR_SHAPE, "%s: page_size=%d is outside 1..65536", what, int(c->page_size));
  if (c->num_pages > 0x7fffffff || c->seqs > 65535)
    return fail(W4_ERR_SHAPE, "%s: num_pages must be below 2^31 and seqs at most 65535", what);
  if (c->max_pages > (int64_t(1) << 30) / c->page_size)
    return fail(W4_ERR_SHAPE, "%s: max_pages * page_size is above 2^30", what);
  const int64_t page = int64_t(c->kv_heads) * c->page_size * c->head_dim;
  if (c->page_stride < page || c->page_stride > (int64_t(1) << 40) || c->page_stride % c->head_dim != 0)
    return fail(W4_ERR_SHAPE, "%s: page_stride=%lld is below a page's %lld elements or no multiple of head_dim", what,
                (long long)c->page_stride, (long long)page);
  if (c->num_pages * (c->page_stride / c->head_dim) > 0xFFFFFFFFll)
    return fail(W4_ERR_SHAPE, "%s: num_pages * page_stride is above 2^32 rows of head_dim elements", what);
  if (c->ldp != 0 && c->ldp < c->max_pages) return fail(W4_ERR_SHAPE, "%s: ldp=%lld < max_pages", what, (long long)c->ldp);
  if (c->seqs > 0) {
    if (c->lengths == nullptr) return fail(W4_ERR_NULL, "%s: lengths is NULL", what);
    if (c->max_pages > 0 && (c->page_table == nullptr || c->k == nullptr || c->v == nullptr))
      return fail(W4_ERR_NULL, "%s: k, v and page_table must not be NULL", what);
    if (c->type == W4_KV_I8 && c->max_pages > 0 && (c->k_scales == nullptr || c->v_scales == nullptr))
      return fail(W4_ERR_NULL, "%s: an int8 cache needs k_scales and v_scales", what);
  }
  if (c->type != W4_KV_I8 && (c->k_scales != nullptr || c->v_scales != nullptr))
    return fail(W4_ERR_VALUE, "%s: scales belong to an int8 cache only", what);
  const auto bits = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
  if ((bits(c->k) | bits(c->v)) & 15) return fail(W4_ERR_ALIGN, "%s: k and v must be 16-byte aligned", what);
  if ((bits(c->k_scales) | bits(c->v_scales) | bits(c->page_table) | bits(c->lengths)) & 3)
    return fail(W4_ERR_ALIGN, "%s: scales, page_table and lengths must be 4-byte aligned", what);
  out->k = c->k;
  out->v = c->v;
  out->ks = c->k_scales;
  out->vs = c->v_scales;
  out->table = c->page_table;
  out->lengths = c->lengths;
  out->page_stride = c->page_stride;
  out->ldp = c->ldp;
  out->num_pages = static_cast<int32_t>(c->num_pages);
  out->seqs = static_cast<int32_t>(c->seqs);
  out->heads = c->kv_heads;
  out->slots_per_page = c->page_size;
  out->page_rows = static_cast<uint32_t>(c->page_stride / c->head_dim);
  out->page = divisor(static_cast<uint32_t>(c->page_size));
  out->dim = c->head_dim;
  out->capacity = static_cast<int32_t>(c->max_pages * c->page_size);
  return W4_OK;
}

}  // namespace w4host

namespace {

using namespace w4kv;

constexpr int kThreads = 256;
constexpr int kRowLanes = 16;
constexpr float kSmallScale = 1e-30f;  // below it the inverse may overflow

struct AppendParams {
  View c;
  const float* k;
  const float* v;
  int64_t ldk, ldv;
  const int32_t* cu;
  int64_t tokens;
  int32_t* lengths_out;  // NULL: written by advance_kernel
  int32_t vec;           // both inputs' rows are 16-byte aligned
  Divisor quads;         // float4s of a row of head_dim elements
  int32_t group_log;     // threads of a token
  ErrorWord* err;
};

// Rows of sequence b, by cu_tokens (one each without it), of those there are.
__device__ __forceinline__ int32_t rows_of(const AppendParams& p, int32_t b) {
  if (p.cu == nullptr) return 1;
  const int64_t from = p.cu[b], to = p.cu[b + 1];
  if (from < 0 || to < from || to > p.tokens) w4dev::record_error(p.err, W4_ERR_VALUE, w4dev::K_KV_APPEND, b);
  const int64_t n = min(to, p.tokens) - max(from, int64_t(0));
  return n < 0 ? 0 : static_cast<int32_t>(min(n, int64_t(0x3fffffff)));
}

// Where a sequence's rows begin: its length. One below 0 (recorded) is no
// place: it takes no rows, and stays.
__device__ __forceinline__ int32_t start_of(const AppendParams& p, int32_t b) {
  const int32_t n = p.c.lengths[b], held = held_length(p.c, b, p.err, w4dev::K_KV_APPEND);
  return n < 0 ? n : held;
}

__device__ __forceinline__ int32_t advanced(const AppendParams& p, int32_t b) {
  const int32_t n = start_of(p, b);
  return n < 0 ? n : min(n + rows_of(p, b), p.c.capacity);
}

// The sequence whose rows hold row t: how many of cu[1..seqs] are <= t, by
// whole-warp steps that cut the range 32-fold.
__device__ int32_t sequence_of(const AppendParams& p, int64_t t) {
  const int lane = threadIdx.x & 31;
  int32_t lo = 0, n = p.c.seqs;  // the answer lies in [lo, lo + n]
  while (n > 0) {
    const int32_t step = (n + 31) / 32;
    const int32_t at = lo + (lane + 1) * step;  // counts entries 1..at
    const bool below = (lane + 1) * step <= n && p.cu[at] <= t;
    const int32_t hit = __popc(__ballot_sync(0xffffffffu, below));
    const int32_t skip = hit * step;
    n = min(n - skip, step - 1);
    lo += skip;
  }
  return lo;
}

template <int TYPE>
__device__ __forceinline__ void store4(void* dst, int64_t at, float4 x) {
  if constexpr (TYPE == W4_KV_F32) {
    reinterpret_cast<float4*>(dst)[at / 4] = x;
  } else if constexpr (TYPE == W4_KV_F16) {
    const __half2 a = __floats2half2_rn(x.x, x.y), b = __floats2half2_rn(x.z, x.w);
    uint2 w;
    w.x = *reinterpret_cast<const uint32_t*>(&a);
    w.y = *reinterpret_cast<const uint32_t*>(&b);
    reinterpret_cast<uint2*>(dst)[at / 4] = w;
  } else {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
    uint2 w;
    w.x = *reinterpret_cast<const uint32_t*>(&a);
    w.y = *reinterpret_cast<const uint32_t*>(&b);
    reinterpret_cast<uint2*>(dst)[at / 4] = w;
  }
}

__device__ __forceinline__ float4 load4(const AppendParams& p, const float* src) {
  return p.vec ? __ldg(reinterpret_cast<const float4*>(src)) : make_float4(src[0], src[1], src[2], src[3]);
}

// Rows without a scale: float4 i of the token's keys, then of its values.
template <int TYPE>
struct Copied {
  static constexpr int kAhead = 8;
  float4 x[kAhead];

  __device__ __forceinline__ void load(const AppendParams& p, int64_t t, int32_t from, int32_t tid) {
    const int32_t half = p.c.heads * p.c.dim / 4;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int32_t i = from + tid + (j << p.group_log);
      if (i < half) x[j] = load4(p, p.k + t * p.ldk + 4 * i);
      else if (i < 2 * half) x[j] = load4(p, p.v + t * p.ldv + 4 * (i - half));
    }
  }
  // page_at: elements to the page; inner: the slot in it
  __device__ __forceinline__ void store(const AppendParams& p, int64_t page_at, int32_t inner, int32_t from,
                                        int32_t tid) const {
    const int32_t half = p.c.heads * p.c.dim / 4;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int32_t i = from + tid + (j << p.group_log);
      if (i < 2 * half) {
        const int32_t r = i < half ? i : i - half, h = p.quads.quotient(r), d = r - h * (p.c.dim / 4);
        const int64_t at = page_at + (int64_t(h) * p.c.slots_per_page + inner) * p.c.dim + 4 * d;
        store4<TYPE>(i < half ? p.c.k : p.c.v, at, x[j]);
      }
    }
  }
};

// int8: a row of head_dim elements for each 16 lanes, VECS float4s a lane; keys'
// rows, then values'.
template <int VECS>
struct Quantised {
  float4 x[VECS];

  __device__ __forceinline__ void load(const AppendParams& p, int64_t t, int32_t from, int32_t tid) {
    const int lane = threadIdx.x % kRowLanes;
    const int32_t r = from + tid / kRowLanes;
    const float* src = r < p.c.heads ? p.k + t * p.ldk + int64_t(r) * p.c.dim : p.v + t * p.ldv + int64_t(r - p.c.heads) * p.c.dim;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int at = lane + i * kRowLanes;
      x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < 2 * p.c.heads && at < p.c.dim / 4) x[i] = load4(p, src + 4 * at);
    }
  }
  __device__ __forceinline__ void store(const AppendParams& p, int32_t page, int32_t inner, int32_t from, int32_t tid) {
    const View& c = p.c;
    const int lane = threadIdx.x % kRowLanes;
    const int32_t r = from + tid / kRowLanes;
    const bool live = r < 2 * c.heads, is_v = r >= c.heads;
    const int32_t h = is_v ? r - c.heads : r;
    float top = 0.f, poison = 0.f;  // NaN for an Inf or NaN in the row
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      top = fmaxf(fmaxf(top, fmaxf(fabsf(x[i].x), fabsf(x[i].y))), fmaxf(fabsf(x[i].z), fabsf(x[i].w)));
      poison = fmaf(x[i].x, 0.f, fmaf(x[i].y, 0.f, fmaf(x[i].z, 0.f, fmaf(x[i].w, 0.f, poison))));
    }
#pragma unroll
    for (int o = kRowLanes / 2; o > 0; o /= 2) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      poison += __shfl_xor_sync(0xffffffffu, poison, o);
    }
    // the fp64 quotient rounded to fp32 is the correctly rounded fp32 one
    const bool bad = poison != 0.f;
    const float sc = bad ? __int_as_float(0x7fc00000) : (top > 0.f ? __fdiv_rn(top, 127.f) : 1.f);
    if (!live) return;
    const int64_t row = int64_t(h) * c.slots_per_page + inner;
    if (lane == 0) (is_v ? c.vs : c.ks)[int64_t(page) * c.heads * c.slots_per_page + row] = sc;
    uint32_t* base = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(is_v ? c.v : c.k) + int64_t(page) * c.page_stride +
                                                 row * c.dim);
    // a scale that underflows to 0 stores zeros, which it also stands for
    const bool zeros = bad || sc == 0.f;
    const float inverse = sc >= kSmallScale ? 1.f / sc : __int_as_float(0x7fc00000);  // NaN: every code the long way
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
      const int at = lane + i * kRowLanes;
      if (at < c.dim / 4) base[at] = zeros ? 0u : codes(x[i], sc, inverse);
    }
  }
  // rint(x / s) of the fp64 quotient, as the definition has it, of four x. x
  // times the rounded inverse is off by at most 3 roundings, 127 x 3 x 2^-24 =
  // 2.3e-5, so only a value within that of a half can round to another code and
  // takes the quotient itself. 1.5 x 2^23 + x rounds x to an integer, whose low
  // byte is the sum's. (7254 tokens of 32 x 96: all by quotients 139 us.)
  __device__ static __forceinline__ uint32_t codes(float4 f, float s, float inverse) {
    const float t[4] = {f.x * inverse, f.y * inverse, f.z * inverse, f.w * inverse};
    uint32_t b[4];
    bool sure = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float m = __fadd_rn(t[i], 12582912.f);
      sure = sure && fabsf(t[i] - __fadd_rn(m, -12582912.f)) < 0.49995f;
      b[i] = __float_as_uint(m);
    }
    if (!sure) {
      const float g[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const double q = rint(static_cast<double>(g[i]) / static_cast<double>(s));
        b[i] = static_cast<uint32_t>(static_cast<int>(fmin(fmax(q, -127.0), 127.0)));
      }
    }
    return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  }
};

// VECS: int8 only, float4s of a lane (head_dim up to 64 VECS).
template <int TYPE, int VECS>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p) {
  constexpr bool I8 = TYPE == W4_KV_I8;
  pdl_launch_dependents();
  pdl_wait();
  const View& c = p.c;
  using Data = typename std::conditional<I8, Quantised<VECS>, Copied<TYPE>>::type;
  Data data;
  const int32_t threads = 1 << p.group_log, tid = threadIdx.x & (threads - 1);
  const int32_t step = I8 ? threads / kRowLanes : Copied<TYPE>::kAhead * threads;
  const int32_t count = I8 ? 2 * c.heads : 2 * c.heads * c.dim / 4;
  const int64_t t = int64_t(blockIdx.x) * (kThreads >> p.group_log) + (threadIdx.x >> p.group_log);
  if (t < p.tokens) data.load(p, t, 0, tid);
  // the new lengths, where they go to memory of their own
  const int64_t b_of_thread = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (p.lengths_out != nullptr && p.cu != nullptr && b_of_thread < c.seqs)
    p.lengths_out[b_of_thread] = advanced(p, static_cast<int32_t>(b_of_thread));
  int32_t b = static_cast<int32_t>(t), slot = 0;
  if (p.cu == nullptr) {
    if (t < p.tokens) slot = start_of(p, b);
    __syncthreads();  // these threads alone read lengths[b], so it may be advanced in place
    if (t < p.tokens && tid == 0) p.lengths_out[b] = slot < 0 ? slot : min(slot + 1, c.capacity);
  }
  if (t >= p.tokens) return;
  if (p.cu != nullptr) {
    b = sequence_of(p, t);
    if (b >= c.seqs || p.cu[b] > t || p.cu[b + 1] <= t) return;  // a row of no sequence
    slot = start_of(p, b);
    if (slot >= 0) {
      const int64_t at = slot + (t - max(p.cu[b], 0));
      slot = static_cast<int32_t>(at < c.capacity ? at : c.capacity);
    }
  }
  if (slot < 0) return;
  if (slot >= c.capacity) {
    if (tid == 0) w4dev::record_error(p.err, W4_ERR_VALUE, w4dev::K_KV_APPEND, b);
    return;
  }
  const int32_t index = c.page.quotient(slot);
  const int32_t page = page_of(c, b, index, p.err, w4dev::K_KV_APPEND);
  if (page < 0) return;
  const int32_t inner = slot - index * c.slots_per_page;
  for (int32_t from = 0; from < count; from += step) {
    if constexpr (I8) {
      Data next;  // a row's rounding takes as long as the next one's loads
      if (from + step < count) next.load(p, t, from + step, tid);
      data.store(p, page, inner, from, tid);
      data = next;
    } else {
      if (from > 0) data.load(p, t, from, tid);
      data.store(p, int64_t(page) * c.page_stride, inner, from, tid);
    }
  }
}

// The lengths advanced in place, once every row has been placed by the old ones.
__global__ void __launch_bounds__(kThreads) advance_kernel(const AppendParams p, int32_t* lengths_out) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t b = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (b < p.c.seqs) lengths_out[b] = advanced(p, static_cast<int32_t>(b));
}

}  // namespace

extern "C" w4_status kv_append(const kv_cache* c, const float* k, int64_t ldk, const float* v, int64_t ldv,
                               const int32_t* cu_tokens, int64_t tokens, int32_t* lengths_out, void* stream) {
  using namespace w4host;
  AppendParams p = {};
  w4_status rc = check_cache(c, "cache", &p.c);
  if (rc != W4_OK) return rc;
  const int64_t wide = int64_t(c->kv_heads) * c->head_dim;
  if (tokens < 0 || tokens > 0x7fffffff) return fail(W4_ERR_SHAPE, "tokens=%lld is outside 0..2^31-1", (long long)tokens);
  if (cu_tokens == nullptr && tokens != c->seqs)
    return fail(W4_ERR_SHAPE, "without cu_tokens there is one row for each sequence: tokens=%lld, seqs=%lld",
                (long long)tokens, (long long)c->seqs);
  if (c->seqs == 0) return W4_OK;
  if (c->ldp == 0 && c->seqs > 1 && tokens > 0)
    return fail(W4_ERR_VALUE, "sequences that share one row of pages (ldp == 0) cannot be appended to");
  if (lengths_out == nullptr) return fail(W4_ERR_NULL, "lengths_out is NULL");
  if (tokens > 0 && (k == nullptr || v == nullptr)) return fail(W4_ERR_NULL, "k and v must not be NULL");
  if (tokens > 1 && (ldk < wide || ldv < wide)) return fail(W4_ERR_SHAPE, "ldk and ldv must be at least kv_heads * head_dim");
  const auto bits = [](const void* q) { return reinterpret_cast<uintptr_t>(q); };
  if ((bits(k) | bits(v) | bits(cu_tokens) | bits(lengths_out)) & 3)
    return fail(W4_ERR_ALIGN, "k, v, cu_tokens and lengths_out must be 4-byte aligned");
  if (lengths_out != c->lengths) {
    const uintptr_t a = bits(lengths_out), b = bits(c->lengths), n = static_cast<uintptr_t>(c->seqs) * 4;
    if (a < b + n && b < a + n) return fail(W4_ERR_VALUE, "lengths_out overlaps the cache's lengths in part");
  }
  const DeviceInfo* di = nullptr;
  rc = current_device(&di);
  if (rc != W4_OK) return rc;
  p.k = k;
  p.v = v;
  p.ldk = ldk;
  p.ldv = ldv;
  p.cu = cu_tokens;
  p.tokens = tokens;
  p.err = di->err;
  p.quads = divisor(static_cast<uint32_t>(c->head_dim) / 4);
  p.vec = ((bits(k) | bits(v)) & 15) == 0 && (tokens <= 1 || ((ldk | ldv) & 3) == 0);
  const bool in_place = cu_tokens != nullptr && lengths_out == c->lengths;
  p.lengths_out = in_place ? nullptr : lengths_out;
  // threads of a token: as many as its first loads keep busy (int8: a half-warp for each row)
  const int64_t busy = c->type == W4_KV_I8 ? 2 * int64_t(c->kv_heads) * kRowLanes : 2 * wide / 4 / Copied<W4_KV_F32>::kAhead;
  p.group_log = 5;
  while ((1 << p.group_log) < busy && (1 << p.group_log) < kThreads) ++p.group_log;
  const int64_t by_seq = (c->seqs + kThreads - 1) / kThreads, per_cta = kThreads >> p.group_log;
  const int64_t by_token = (tokens + per_cta - 1) / per_cta;
  const dim3 grid(static_cast<unsigned>(by_token > by_seq ? by_token : by_seq));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  void (*kernel)(const AppendParams) = append_kernel<W4_KV_F32, 1>;
  if (c->type == W4_KV_F16) kernel = append_kernel<W4_KV_F16, 1>;
  if (c->type == W4_KV_BF16) kernel = append_kernel<W4_KV_BF16, 1>;
  if (c->type == W4_KV_I8) {
    kernel = c->head_dim <= 64    ? append_kernel<W4_KV_I8, 1>
             : c->head_dim <= 128 ? append_kernel<W4_KV_I8, 2>
             : c->head_dim <= 192 ? append_kernel<W4_KV_I8, 3>
                                  : append_kernel<W4_KV_I8, 4>;
  }
  cudaError_t e = launch_pdl(kernel, grid, kThreads, 0, st, 1, false, p);
  if (e != cudaSuccess) return cuda_fail(e, "launch kv_append");
  if (in_place) {
    e = launch_pdl(advance_kernel, dim3(static_cast<unsigned>(by_seq)), kThreads, 0, st, 1, false, p, lengths_out);
    if (e != cudaSuccess) return cuda_fail(e, "launch kv_append (lengths)");
  }
  return W4_OK;
}
