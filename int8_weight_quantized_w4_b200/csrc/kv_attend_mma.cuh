// The matrix-instruction body of kv_attend, for several query heads on one
// key-value head: from 3 heads on the plain lanes' fused multiply-adds
// (one for each head and stored element) take longer than the loads.
//
// Exactness. A stored key or value is an exact fp16 (fp16, int8 codes) or
// bf16 operand; the fp32 queries and softmax weights are taken apart into
// pieces of that type, which lie in different rows of the 16-row A operand
// and are added up in fp32 behind the product:
//   fp16, int8: 8 heads x 2 pieces, 11 + 11 bits: the second one holds the
//               exact rest, scaled by 2^11. Queries are scaled by a power of
//               two so that their largest lies at 2^14, weights so that it lies
//               from 2^7 to 2^14: what is left out is below 2^-22 of each of
//               them or 2^-43 of the largest. int8's weights have the value's
//               scale in them, and the largest of those products counts, each
//               head's own and from 2^8 on (2^-44): a slot whose scale is
//               large but whose weight is not takes no bits from the others.
//               Nor does a row of zeros, whatever its scale (kv_append gives
//               it 1): where a product would raise the power, such rows'
//               are set to 0 first;
//   bf16:       4 heads x 3 pieces (8 + 8 + 8 bits, all of them) in one
//               instruction, or 8 heads in two (pieces 0 and 1, then 2).
//
// Layout. mma.m16n8k16 sums over k in any order, and its n columns may be any
// 8 values, so both operands are read from the stages as they were stored, 16
// bytes a lane (values: VB), without a transposing load: lane (g, t) =
// (lane / 4, lane % 4) reads
//   keys:   vectors t, t + 4, ... of slots g and g + 8 of a tile's 16; the 8
//           elements of a vector are two k-steps' 4 each;
//   values: vectors g, g + 8 of slots 2t, 2t+1, 2t+8, 2t+9; byte permutes pair
//           the slots, element j of all vectors makes one product's columns.
// The scores' accumulators are then the A operand of the second product.
//
// Why not the larger matrix instructions: the rows of A are the query heads of
// one key-value head, so a 128-row operand would be mostly zeros, and int8
// codes have to pass the registers anyway. Rate is not what is short: on
// 131072 slots of 8 x 128 bf16 for 32 heads the tensor pipe is busy a fifth of
// the time and DRAM delivers 6.1 TB/s; int8 (32 sequences of up to 4096 slots,
// 8 x 128 for 64 heads: 54 us, 3.6 TB/s) is held by the conversions' dependent
// instructions at the 12 warps that an SM's registers hold.
#pragma once

#include "kv_attend.cuh"

namespace w4kv {

template <int TYPE>
__device__ __forceinline__ void mma16816(float (&c)[4], uint4 a, uint32_t b0, uint32_t b1) {
  if constexpr (TYPE == W4_KV_BF16) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
  } else {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
  }
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }

// Two bytes (code XOR 0x80) under the high byte of fp16 1024 are 1024 + 128 +
// code; the subtraction is exact.
__device__ __forceinline__ uint32_t code_pair(uint32_t biased, uint32_t sel) {
  const uint32_t w = prmt(biased, 0x64646464u, sel);
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&w), __floats2half2_rn(1152.f, 1152.f));
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Piece `piece` of x (two neighbours packed): fp16's second one is scaled by 2^11.
__device__ __forceinline__ uint32_t half_piece(float a, float b, int piece) {
  if (piece == 0) return pack_half(a, b);
  return pack_half((a - __half2float(__float2half_rn(a))) * 2048.f, (b - __half2float(__float2half_rn(b))) * 2048.f);
}

__device__ __forceinline__ float bf16_rest(float x) { return x - __bfloat162float(__float2bfloat16_rn(x)); }

__device__ __forceinline__ uint32_t bf16_piece(float a, float b, int piece) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (i < piece) {
      a = bf16_rest(a);
      b = bf16_rest(b);
    }
  }
  return pack_bf16(a, b);
}

__device__ __forceinline__ float power_of_two(int exponent) {  // exponent in -126..127
  return __uint_as_float(static_cast<uint32_t>(exponent + 127) << 23);
}

// ROWS query heads, rows of at most MAXD elements.
template <int TYPE, int ROWS, int MAXD>
struct MatrixLanes {
  using E = Elem<TYPE>;
  static constexpr bool BF = TYPE == W4_KV_BF16, I8 = TYPE == W4_KV_I8;
  static_assert(BF || ROWS == 8, "fp16 pieces of 8 heads fill the 16 rows");
  static constexpr int SETS = BF && ROWS == 8 ? 2 : 1;  // A operands
  static constexpr int EPV = E::kPerVec;
  static constexpr int NI = (MAXD / EPV + 3) / 4;       // key vectors of a lane
  static constexpr int STEPS = NI * EPV / 4;            // k-steps of the scores
  // bytes of a value load: shorter ones need fewer registers at a time. 32
  // sequences of up to 6000 slots of 128 int8: 60.5 us with 16 bytes, 53.7 us with
  // 8; fp16 57.9 us, 54.2 us; bf16 of 256 for 2 heads 24.6 us, 25.8 us
  static constexpr int VB = BF && MAXD == 256 ? 16 : 8;
  static constexpr int VE = VB / E::kBytes;             // its elements
  static constexpr int NC = (MAXD / VE + 7) / 8;        // value vectors of a lane
  static constexpr int NT = I8 && MAXD <= 128 ? 2 : 1;  // 16 slots each, at once: int8's stages have room for two
  static constexpr int TS = 16 * NT;
  static constexpr int kLift = 14;  // fp16 pieces: the exponent of the largest query, and of the largest weight
  static constexpr float kBelow = BF || I8 ? 0.f : kLift - kSlack;  // a new reference lies this far below the maximum
  static constexpr int kFresh = 8;  // int8: a new power lifts the largest product of weight and scale to here,
                                    // and stands until one passes 2^(kLift + 1)
  static constexpr int kMostUp = 126;  // the largest power
  static constexpr int kFrag = SETS * STEPS * 32 * 4;   // words of the queries' operands
  static constexpr int kWidth = MAXD;  // of a row of queries in shared memory
  static constexpr int kBodyFloats = kFrag;
  // Beginning and ending a segment takes about as long as two units: 32 sequences of
  // up to 6000 slots of 128 int8 for 64 heads 54 us (with 1 57.6 us), one of 131072 bf16
  // for 32 heads 89.5 us (91 us).
  static constexpr int kOver = 3;
  static constexpr int kMinCtas = MAXD <= 128 ? 3 : (MAXD == 256 && !I8 ? 1 : 2);
  static constexpr int CV = MAXD / EPV % 3 == 0 ? 3 : (MAXD / EPV == 32 ? 2 : 1);  // copies: vectors of a lane,
  static constexpr int CL = MAXD / EPV / CV;                                       // lanes of a row
  using Feed = Ring<TYPE, TS, CL, CV, (MAXD / EPV + 7) / 8 * 8, true, 2, ROWS * (MAXD + 2)>;
  using VVec = typename std::conditional<VB == 16, uint4, uint2>::type;

  __device__ static __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
  __device__ static __forceinline__ uint32_t word(const uint2& v, int i) { return i == 0 ? v.x : v.y; }

  // The queries as A operands in shared memory, in the order the lanes read
  // them; returns what this lane's head's scores are multiplied by for it.
  template <int TEAM>
  __device__ static __forceinline__ float stage_queries(uint32_t* frag, const float* sq) {
    const int lane = threadIdx.x & 31, warp = TEAM == 1 ? 0 : threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    float factor = 1.f, scale = 1.f;
    if constexpr (!BF) {
      // 2^(14 - e), 2^e the power below the largest |q| of each row; the scores take it back
#pragma unroll
      for (int h = 0; h < ROWS; ++h) {
        uint32_t top = 0;
#pragma unroll
        for (int d = 0; d < MAXD; d += 128) {
          if (d + 4 * lane < MAXD) {
            const float4 x = *reinterpret_cast<const float4*>(sq + h * MAXD + d + 4 * lane);
            top = max(top, max(max(__float_as_uint(fabsf(x.x)), __float_as_uint(fabsf(x.y))),
                               max(__float_as_uint(fabsf(x.z)), __float_as_uint(fabsf(x.w)))));
          }
        }
        top = __reduce_max_sync(0xffffffffu, top);
        if (h == g) factor = power_of_two(max(kLift + 1, min(253, static_cast<int>(top >> 23))) - 127 - kLift);
      }
      scale = 1.f / factor;
    }
    for (int s = warp; s < SETS * STEPS; s += TEAM) {
      const int set = s / STEPS, st = s % STEPS;
      const int d = (t + 4 * (st / (EPV / 4))) * EPV + 4 * (st % (EPV / 4));
      uint32_t a[4];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = g + 8 * half;
        const int h = r % ROWS, piece = ROWS == 4 ? r / 4 : (set == 0 ? r / 8 : 2 + r / 8);
        const float4 x = *reinterpret_cast<const float4*>(sq + h * MAXD + d);  // zeros behind head_dim
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float u = (e == 0 ? x.x : x.z) * scale, v = (e == 0 ? x.y : x.w) * scale;
          if constexpr (BF) {
            a[half + 2 * e] = piece < 3 ? bf16_piece(u, v, piece) : 0u;
          } else {
            a[half + 2 * e] = half_piece(u, v, piece);
          }
        }
      }
      *reinterpret_cast<uint4*>(frag + (s * 32 + lane) * 4) = make_uint4(a[0], a[1], a[2], a[3]);
    }
    if (TEAM == 1) {
      __syncwarp();
    } else {
      __syncthreads();
    }
    return factor;
  }

  // Rows of one head's pieces summed: in a lane, and over the two lanes that
  // share a head where there are 4.
  __device__ static __forceinline__ float in_lane(float lo, float hi) { return BF ? lo + hi : fmaf(hi, 1.f / 2048.f, lo); }
  __device__ static __forceinline__ float over_lanes(float v) {
    if constexpr (ROWS == 4) v += __shfl_xor_sync(0xffffffffu, v, 16);
    return v;
  }
  __device__ static __forceinline__ float joined(float lo, float hi) { return over_lanes(in_lane(lo, hi)); }
  // A product's two columns to acc, as packed pairs; bf16's 8 rows have no
  // registers for their alignment (16 x 4096 slots of 128 for 64 heads: 62 us
  // packed, 58 us so; fp16: 54 us).
  __device__ static __forceinline__ void add(float (&acc)[2], const float (&c)[4]) {
    if constexpr (BF && ROWS == 8) {
      acc[0] += in_lane(c[0], c[2]);
      acc[1] += in_lane(c[1], c[3]);
      return;
    }
    unsigned long long a, lo, hi;
    asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(acc[0]), "f"(acc[1]));
    asm("mov.b64 %0, {%1, %2};" : "=l"(lo) : "f"(c[0]), "f"(c[1]));
    asm("mov.b64 %0, {%1, %2};" : "=l"(hi) : "f"(c[2]), "f"(c[3]));
    if constexpr (BF) {
      asm("add.rn.f32x2 %0, %0, %1;" : "+l"(lo) : "l"(hi));
    } else {
      asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(lo) : "l"(hi), "l"(0x3A0000003A000000ull));  // 2^-11 twice
    }
    asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(lo));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(acc[0]), "=f"(acc[1]) : "l"(a));
  }

  // 2^by, by <= 0; below fp32's normal numbers nothing is left but a NaN.
  __device__ static __forceinline__ float falling(int by) { return by < -126 ? 0.f : power_of_two(by); }

  // The largest of this lane's weights in a tile.
  __device__ static __forceinline__ float largest(const float (&x)[2 * NT][2]) {
    float top = 0.f;
#pragma unroll
    for (int n = 0; n < 2 * NT; ++n) top = fmaxf(top, fmaxf(fabsf(x[n][0]), fabsf(x[n][1])));
    return top;
  }
  __device__ static __forceinline__ int exponent(float x) { return static_cast<int>(__float_as_uint(x) >> 23) - 127; }

  // The warp's triple of its share (one of TEAM) of the segment: where it has been put.
  template <int TEAM>
  __device__ static __forceinline__ float* segment(const AttendParams& p, const Run& run, const Segment& seg, Feed& feed,
                                                   const float* sq, float* body) {
    uint32_t* frag = reinterpret_cast<uint32_t*>(body);
    const int lane = threadIdx.x & 31, warp = TEAM == 1 ? 0 : threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int D = p.c.dim, head = g % ROWS;
    const int32_t s1 = seg.s1;
    const float scale = stage_queries<TEAM>(frag, sq) * p.scale2;
    float m = -INFINITY, l = 0.f;
    float acc[NC * VE][2];  // the lane's pieces added up
#pragma unroll
    for (int i = 0; i < NC * VE; ++i) acc[i][0] = acc[i][1] = 0.f;
    int up = kMostUp;  // int8: the weights' products with the values' scales enter times 2^up, which acc is in
#pragma unroll 1
    for (int32_t tile = seg.s0 + warp * TS; tile < s1; tile += TEAM * TS) {
      uint32_t held;
      const uint8_t* stage = feed.take(p, run, held);
      const float* scales = reinterpret_cast<const float*>(stage + Feed::kScales);
      uint4 kx[2 * NT][NI];
#pragma unroll
      for (int n = 0; n < 2 * NT; ++n)
#pragma unroll
        for (int i = 0; i < NI; ++i) kx[n][i] = *reinterpret_cast<const uint4*>(stage + Feed::place(8 * n + g, t + 4 * i));
      float c[2 * NT][4] = {};
#pragma unroll
      for (int st = 0; st < STEPS; ++st) {
        const int i = st / (EPV / 4), j = st % (EPV / 4);
        uint4 a[SETS];
#pragma unroll
        for (int s = 0; s < SETS; ++s) a[s] = *reinterpret_cast<const uint4*>(frag + ((s * STEPS + st) * 32 + lane) * 4);
#pragma unroll
        for (int n = 0; n < 2 * NT; ++n) {
          uint32_t b0, b1;
          if constexpr (I8) {
            const uint32_t w = word(kx[n][i], j) ^ 0x80808080u;
            b0 = code_pair(w, 0x4140);
            b1 = code_pair(w, 0x4342);
          } else {
            b0 = word(kx[n][i], 2 * j);
            b1 = word(kx[n][i], 2 * j + 1);
          }
#pragma unroll
          for (int s = 0; s < SETS; ++s) mma16816<TYPE>(c[n], a[s], b0, b1);
        }
      }
      VVec vx[4 * NT][NC];
#pragma unroll
      for (int n = 0; n < 4 * NT; ++n)
#pragma unroll
        for (int cc = 0; cc < NC; ++cc) {
          const int row = 2 * t + (n & 1) + (n >> 1) * 8, byte = (g + 8 * cc) * VB;
          vx[n][cc] = *reinterpret_cast<const VVec*>(stage + Feed::kSide + Feed::place(row, byte / 16) + byte % 16);
        }
      // scores of this lane's head at slots 8 n + 2 t + e
      float x[2 * NT][2];
      float top = -INFINITY;
#pragma unroll
      for (int n = 0; n < 2 * NT; ++n) {
        float2 f = make_float2(1.f, 1.f);
        if constexpr (I8) f = *reinterpret_cast<const float2*>(scales + 8 * n + 2 * t);
        x[n][0] = finite(joined(c[n][0], c[n][2]) * (scale * f.x));
        x[n][1] = finite(joined(c[n][1], c[n][3]) * (scale * f.y));
      }
      if (held != Feed::kAll) {
#pragma unroll
        for (int n = 0; n < 2 * NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (!((held >> (8 * n + 2 * t + e)) & 1u)) x[n][e] = -INFINITY;
      }
#pragma unroll
      for (int n = 0; n < 2 * NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) top = fmaxf(top, x[n][e]);
      if (p.scores != nullptr && head < seg.ng && g < ROWS) {
        float* to = p.scores + (int64_t(seg.b) * p.c.heads * p.group + seg.q0 + head) * p.c.capacity + tile + 2 * t;
#pragma unroll
        for (int n = 0; n < 2 * NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (tile + 8 * n + 2 * t + e < s1) to[8 * n + e] = x[n][e];
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // weights are 2^(x - m): m follows the maximum when that passes it by more
      // than what keeps the largest weight below 2^kLift
      float back = 1.f;  // what acc is multiplied by
      if (top - kBelow > m + kSlack) {
        top -= kBelow;
        if constexpr (I8) top = ceilf(top);  // references whole powers apart: acc keeps its own
        const float fall = m == -INFINITY ? 1.f : ex2(m - top);  // without a score so far there are zeros, or a NaN
        l *= fall;
        if constexpr (I8) {
          const int to = up + static_cast<int>(fminf(top - m, 1000.f));
          up = min(to, kMostUp);
          back = falling(up - to);
        } else {
          back = fall;
        }
        m = top;
      }
      const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int n = 0; n < 2 * NT; ++n) {
        float2 f = make_float2(1.f, 1.f);
        if constexpr (I8) f = *reinterpret_cast<const float2*>(scales + TS + 8 * n + 2 * t);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x[n][e] = ex2(x[n][e] - ref);
          l += x[n][e];
          if constexpr (I8) x[n][e] *= e == 0 ? f.x : f.y;
        }
      }
      bool rescale = back != 1.f;
      if constexpr (I8) rescale = rescale || exponent(largest(x)) + up > kLift;
      if (__any_sync(0xffffffffu, rescale)) {
        if constexpr (I8) {
          uint32_t codes = 0;  // which of this lane's slots hold other codes than 0
#pragma unroll
          for (int n = 0; n < 4 * NT; ++n)
#pragma unroll
            for (int cc = 0; cc < NC; ++cc)
#pragma unroll
              for (int i = 0; i < VB / 4; ++i)
                if ((g + 8 * cc) * VB < D && word(vx[n][cc], i) != 0u) codes |= 1u << n;
#pragma unroll
          for (int o = 4; o < 32; o *= 2) codes |= __shfl_xor_sync(0xffffffffu, codes, o);
#pragma unroll
          for (int n = 0; n < 2 * NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!((codes >> (2 * n + e)) & 1u)) x[n][e] *= 0.f;  // a scale of NaN stays
          float most = largest(x);  // of the head's four lanes
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
          if (exponent(most) + up > kLift) {
            back *= falling(kFresh - exponent(most) - up);
            up = kFresh - exponent(most);
          }
        }
#pragma unroll
        for (int i = 0; i < NC * VE; ++i) {
          acc[i][0] *= back;
          acc[i][1] *= back;
        }
      }
      if constexpr (I8) {
        const float unit = power_of_two(up);
#pragma unroll
        for (int n = 0; n < 2 * NT; ++n) {
          x[n][0] *= unit;
          x[n][1] *= unit;
        }
      }
      uint4 w[NT][SETS];
#pragma unroll
      for (int k = 0; k < NT; ++k) {
        const float(&x0)[2] = x[2 * k];
        const float(&x1)[2] = x[2 * k + 1];
        if constexpr (!BF) {
          w[k][0] = make_uint4(half_piece(x0[0], x0[1], 0), half_piece(x0[0], x0[1], 1), half_piece(x1[0], x1[1], 0),
                               half_piece(x1[0], x1[1], 1));
        } else {
          uint32_t piece[3][2];
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            piece[i][0] = bf16_piece(x0[0], x0[1], i);
            piece[i][1] = bf16_piece(x1[0], x1[1], i);
          }
          if constexpr (ROWS == 4) {
            const bool low = g < 4;  // rows 0-3 and 8-11: pieces 0 and 2; rows 4-7: piece 1
            w[k][0] = make_uint4(low ? piece[0][0] : piece[1][0], low ? piece[2][0] : 0u,
                                 low ? piece[0][1] : piece[1][1], low ? piece[2][1] : 0u);
          } else {
            w[k][0] = make_uint4(piece[0][0], piece[1][0], piece[0][1], piece[1][1]);
            w[k][SETS - 1] = make_uint4(piece[2][0], 0u, piece[2][1], 0u);
          }
        }
      }
      // A tile's products begin at zero and are added here: the matrix pipe cuts
      // its sums off instead of rounding them, which over a warp's thousands of
      // slots of one sign came to 1.4e-5 of the result. (A score's sum, of 4 to 32
      // instructions, stays there: 256 products of one sign lose 1.4e-6 of it, all
      // slots alike, which the log sum shows and the weights do not.)
#pragma unroll
      for (int cc = 0; cc < NC; ++cc) {
        if constexpr (I8) {
#pragma unroll
          for (int q = 0; q < VE / 4; ++q) {
            float c[4][4] = {};
#pragma unroll
            for (int k = 0; k < NT; ++k) {
              uint32_t s[4];
#pragma unroll
              for (int n = 0; n < 4; ++n) s[n] = word(vx[4 * k + n][cc], q) ^ 0x80808080u;
              const uint32_t lo0 = prmt(s[0], s[1], 0x5140), hi0 = prmt(s[0], s[1], 0x7362);
              const uint32_t lo1 = prmt(s[2], s[3], 0x5140), hi1 = prmt(s[2], s[3], 0x7362);
              mma16816<TYPE>(c[0], w[k][0], code_pair(lo0, 0x4140), code_pair(lo1, 0x4140));
              mma16816<TYPE>(c[1], w[k][0], code_pair(lo0, 0x4342), code_pair(lo1, 0x4342));
              mma16816<TYPE>(c[2], w[k][0], code_pair(hi0, 0x4140), code_pair(hi1, 0x4140));
              mma16816<TYPE>(c[3], w[k][0], code_pair(hi0, 0x4342), code_pair(hi1, 0x4342));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) add(acc[cc * VE + 4 * q + j], c[j]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            const uint32_t sel = j & 1 ? 0x7632 : 0x5410;
            float c[4] = {};
#pragma unroll
            for (int k = 0; k < NT; ++k) {
              const uint32_t b0 = prmt(word(vx[4 * k][cc], j / 2), word(vx[4 * k + 1][cc], j / 2), sel);
              const uint32_t b1 = prmt(word(vx[4 * k + 2][cc], j / 2), word(vx[4 * k + 3][cc], j / 2), sel);
#pragma unroll
              for (int s = 0; s < SETS; ++s) mma16816<TYPE>(c, w[k][s], b0, b1);
            }
            add(acc[cc * VE + j], c);
          }
        }
      }
    }
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    const float unit = I8 ? power_of_two(-up) : 1.f;
    float* to = feed.spare();
    if (t == 0 && g < ROWS) {
      to[ROWS * D + head] = m;
      to[ROWS * D + ROWS + head] = l;
    }
#pragma unroll
    for (int i = 0; i < NC * VE; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float v = over_lanes(acc[i][e]) * unit;
        const int d = (2 * t + e + 8 * (i / VE)) * VE + i % VE;
        if (g < ROWS && d < D) to[head * D + d] = v;
      }
    return to;
  }
};

// Query heads of a key-value head from which on the matrices are taken, where
// there are slots enough. Two heads, 16 sequences of 4000 slots of 8 key-value heads:
// 160 bf16 101 us in plain lanes, 61 us in matrices; 256 int8 112 us, 65 us. Rows
// of up to 128 gain little from them (64 bf16 29.4 us, 24.6 us; 128 int8 42.9 us,
// 40.6 us) and keep the lanes' whole fp32 queries and weights. Three heads, 8
// sequences of 6000 slots of 16 x 128 bf16: 123 us, 67 us.
inline int32_t least_group(int32_t dim) { return dim > 128 ? 2 : 3; }

// The matrix kernel for this many query heads, where there is one.
template <int TYPE, int ROWS>
AttendKernel matrix_kernel_for(int32_t dim) {
  if (dim <= 64) return attend_kernel_of<MatrixLanes<TYPE, ROWS, 64>, ROWS>();
  if constexpr (TYPE != W4_KV_I8) {
    if (dim <= 96) return attend_kernel_of<MatrixLanes<TYPE, ROWS, 96>, ROWS>();
  }
  if (dim <= 128) return attend_kernel_of<MatrixLanes<TYPE, ROWS, 128>, ROWS>();
  if (dim <= 192) return attend_kernel_of<MatrixLanes<TYPE, ROWS, 192>, ROWS>();
  return attend_kernel_of<MatrixLanes<TYPE, ROWS, 256>, ROWS>();
}

}  // namespace w4kv
