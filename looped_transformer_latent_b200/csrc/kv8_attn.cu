// Attention over the 8-bit K/V cache and the exact tokens after it.
//
// A CTA serves RT = 8 NT query rows of one (sequence, cache head) over one
// split of the cached tokens.  Each warp streams its own token tiles from
// global memory straight into registers in the operand order of the f16
// m16n8k16 product, widens the 8-bit codes to f16 there (exact), and keeps its
// own running maximum, sum and accumulator; warps are joined through shared
// memory, splits by kv8_join.
//   S^T [tokens x rows] = K q^T   K codes as the A operand, q as B
//   O^T [d x rows]     += V^T P^T V codes as A (pairs of tokens interleaved
//                                 while widening), P from S^T by movmatrix
// so any number of rows up to 8 NT shares each widened code.  A lane's bytes
// of a row are contiguous: which element a product index stands for is free as
// long as both operands agree.
#include "kernels.cuh"

namespace lla {
namespace {

constexpr int AT = 128;          // threads
constexpr int AW = AT / 32;

struct Tokens {                  // what one sequence's rows see
  int len, tail;
  int64_t pos0;                  // position of the oldest exact token
  __device__ Tokens(const lla_kv8_attn_params& p, int b) {
    len = min(max(kv8_at(p.len, b), 0), p.cache.Ncap);
    tail = 0; pos0 = 0;
    if (p.win_k) {
      tail = min(max(kv8_at(p.tail, b), 0), p.Wcap);
      pos0 = (int64_t)kv8_at(p.ctx, b) - tail;
    }
  }
};

// exact tokens, of `tail`, that query position qp of nq sees
__device__ __forceinline__ int visible(int tail, int qp, int nq) { return max(0, tail - (nq - 1 - qp)); }

__device__ __forceinline__ int slot_of(int64_t pos, int cap) {
  const int64_t r = pos % cap;
  return (int)(r < 0 ? r + cap : r);
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Widening of codes to f16, exact.  int8: the byte plus 128 in the low mantissa
// bits of 1024, less 1152.  e4m3: its bits moved to f16's places, which is the
// value times 2^-8 (subnormals included; kCodeGain undoes it in fp32).
template <int CODE>
struct Widen;
template <>
struct Widen<LLA_KV8_I8> {
  static constexpr float gain = 1.f;
  static __device__ __forceinline__ uint32_t prep(uint32_t w) { return w ^ 0x80808080u; }
  static __device__ __forceinline__ uint32_t lo(uint32_t w) { return sub_f16x2(prmt(w, 0x64646464u, 0x4140), 0x64806480u); }
  static __device__ __forceinline__ uint32_t hi(uint32_t w) { return sub_f16x2(prmt(w, 0x64646464u, 0x4342), 0x64806480u); }
};
template <>
struct Widen<LLA_KV8_E4M3> {
  static constexpr float gain = 256.f;
  static __device__ __forceinline__ uint32_t prep(uint32_t w) { return w; }
  static __device__ __forceinline__ uint32_t put(uint32_t p) { return ((p >> 1) & 0x3f803f80u) | (p & 0x80008000u); }
  static __device__ __forceinline__ uint32_t lo(uint32_t w) { return put(prmt(w, 0u, 0x1404)); }
  static __device__ __forceinline__ uint32_t hi(uint32_t w) { return put(prmt(w, 0u, 0x3424)); }
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t h) {
  float2 r;
  asm("{.reg .f16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}" : "=f"(r.x), "=f"(r.y) : "r"(h));
  return r;
}
// 8 x 8 transpose across the warp: lane (g, t) of (row g, columns 2t, 2t + 1)
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Cache bytes are read once: no allocation in L1.
template <int W>
__device__ __forceinline__ void load_words(uint32_t* r, const uint8_t* p, bool ok) {
  if constexpr (W == 4) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (ok) asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
  } else if constexpr (W == 2) {
    uint2 v = make_uint2(0, 0);
    if (ok) asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    r[0] = v.x; r[1] = v.y;
  } else {
    uint32_t v = 0;
    if (ok) asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(v) : "l"(p));
    r[0] = v;
  }
}

// Element offset of a lane's word of a row, D elements padded: K rows are
// shared by the 4 lanes t of a group (D / 16 words each), V rows by the 8
// groups g (D / 32 words each); in both, pieces of 16 bytes, then of what is
// left.
template <int LANES>
__device__ __forceinline__ constexpr int word_at(int D, int w, int lane) {
  const int full = D / (16 * LANES);             // pieces of 16 bytes
  if (w < 4 * full) return 16 * LANES * (w / 4) + 16 * lane + 4 * (w % 4);
  const int left = D / LANES - 16 * full;        // bytes of the last pieces: 8, 4 or 12
  const int w2 = w - 4 * full;
  if (left >= 8 && w2 < 2) return 16 * LANES * full + 8 * lane + 4 * w2;
  return 16 * LANES * full + (left >= 8 ? 8 * LANES : 0) + 4 * lane;
}

template <int LANES, int D>
__device__ __forceinline__ void load_row(uint32_t* r, const uint8_t* row, int lane, int d) {
  constexpr int W = D / (4 * LANES), full = W / 4, left = W % 4;
#pragma unroll
  for (int i = 0; i < full; ++i) {
    const int at = word_at<LANES>(D, 4 * i, lane);
    load_words<4>(r + 4 * i, row + at, at < d);
  }
  if constexpr (left >= 2) {
    const int at = word_at<LANES>(D, 4 * full, lane);
    load_words<2>(r + 4 * full, row + at, at < d);
  }
  if constexpr (left % 2) {
    const int at = word_at<LANES>(D, W - 1, lane);
    load_words<1>(r + W - 1, row + at, at < d);
  }
}

// Queries enter as f16 under a power of two per row that puts the row's largest
// magnitude into [2^13, 2^14): a bf16 query is exact, a second term adds the
// next 11 bits of an fp32 one.
constexpr int kQExp = 13;
// Running references of a row, both base-2 exponents: m of the probabilities
// p = exp2(s - m), a of what meets the value codes, w = exp2(s + log2(scale) - a),
// so that a block whose values are 2^60 times another's does not drown it.  A
// reference is set kOff below a new maximum and follows it only when it is
// exceeded by kSlack more: w stays below 2^12 in f16, the largest above 2^-8,
// and most tiles need neither a shuffle nor a rescaling.
constexpr float kOff = 4.f, kSlack = 12.f, kUnset = -1e30f;

template <int D, int NT>
struct AttnSmem {
  static constexpr int RT = 8 * NT;
  uint2 q[2][D / 16][NT][32];    // query terms, B operand order
  float rowf[RT];                // row exponent times scale log2(e)
  float2 ml[2][RT];              // join of the warps
  float y[2][D * RT];
};

template <int CODE, int D, int NT, int QT>
__global__ void __launch_bounds__(AT, NT == 1 ? 3 : 2) kv8_attn_kernel(const Kv8AttnArgs a) {
  constexpr int RT = 8 * NT;
  constexpr int KW = D / 16, VW = D / 32;        // words per lane of a K and of a V row
  constexpr int MT = D > 128 || NT > 1 ? 1 : 2;  // tiles of 16 tokens a warp holds at a time
  constexpr int STEP = 16 * MT;
  using Wd = Widen<CODE>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  AttnSmem<D, NT>& sm = *reinterpret_cast<AttnSmem<D, NT>*>(smem_raw);
  griddep_wait();
  const lla_kv8_attn_params& p = a.p;
  const lla_kv8_cache& c = p.cache;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int split = blockIdx.x, rt = blockIdx.y / c.H, h = blockIdx.y % c.H, b = blockIdx.z;
  const int len = min(max(kv8_at(p.len, b), 0), c.Ncap);
  const int first = split * a.tps, last = min(len, first + a.tps);   // this split's tokens
  const int row0 = rt * RT;                      // of this pass
  const int64_t bh = (int64_t)b * c.H + h;
  if (first >= last) {                           // nothing: the join must not read what was there
    if (tid < RT && row0 + tid < a.rows)
      a.part_ml[(bh * a.rows + row0 + tid) * a.ST + split] = make_float2(-INFINITY, 0.f);
    return;
  }

  // ---- queries: a warp takes RT / 4 rows
  for (int r = warp; r < RT; r += AW) {
    const int row = a.row0 + row0 + r;           // of the call
    const bool there = row0 + r < a.rows;
    const int qp = row / p.G, gq = row % p.G;
    const int64_t qo = (int64_t)b * p.q_stride_b + (int64_t)qp * p.q_stride_n + (int64_t)(h * p.G + gq) * c.d;
    float top = 0.f;
    for (int e = lane; e < c.d; e += 32) {
      const float x = there ? fabsf(load_elem(p.q, qo + e, p.dtype)) : 0.f;
      top = x > top || x != x ? x : top;         // NaN stays
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float x = __shfl_xor_sync(0xffffffffu, top, o);
      top = x > top || x != x ? x : top;
    }
    int ex = 0;
    if (top > 0.f && top < INFINITY) ex = max(ilogbf(top) - kQExp, -100);
    if (lane == 0) sm.rowf[r] = ldexpf(a.qmul, ex) * Wd::gain;
    for (int i = lane; i < KW * 4; i += 32) {    // word w, group lane tt
      const int w = i / 4, tt = i % 4, at = word_at<4>(D, w, tt);
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = there && at < c.d ? ldexpf(load_elem(p.q, qo + at + e, p.dtype), -ex) : 0.f;
      uint2 v = make_uint2(pack_f16(x[0], x[1]), pack_f16(x[2], x[3]));
      sm.q[0][w][r / 8][(r % 8) * 4 + tt] = v;
      if (QT == 2) {
        const float2 u0 = unpack_f16(v.x), u1 = unpack_f16(v.y);
        sm.q[1][w][r / 8][(r % 8) * 4 + tt] =
            make_uint2(pack_f16(x[0] - u0.x, x[1] - u0.y), pack_f16(x[2] - u1.x, x[3] - u1.y));
      }
    }
  }
  __syncthreads();

  const uint8_t* kc = static_cast<const uint8_t*>(c.k) + (int64_t)b * c.stride_b + (int64_t)h * c.stride_h;
  const uint8_t* vc = static_cast<const uint8_t*>(c.v) + (int64_t)b * c.stride_b + (int64_t)h * c.stride_h;
  const float* ksc = c.k_scale + (int64_t)b * c.scale_stride_b + (int64_t)h * c.scale_stride_h;
  const float* vsc = c.v_scale + (int64_t)b * c.scale_stride_b + (int64_t)h * c.scale_stride_h;
  const int bshift = 31 - __clz(c.block);

  float acc[D / 16][NT][4];
  float mo[2 * NT], ao[2 * NT], F[2 * NT], l[2 * NT];   // references, F = exp2(mo - ao)
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][n][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mo[2 * n + e] = ao[2 * n + e] = kUnset; F[2 * n + e] = 1.f; l[2 * n + e] = 0.f;
    }
  }

  uint32_t kr[MT][2][KW], vr[MT][4][VW];
  float ks[MT], vs[MT];
  // a tile of 16 tokens that starts before `last` lies inside one block of the cache
  auto load_k = [&](int tb) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int s = tb + 16 * m < last ? tb + 16 * m : first;
#pragma unroll
      for (int i = 0; i < 2; ++i) load_row<4, D>(kr[m][i], kc + (int64_t)(s + g + 8 * i) * c.d, t, c.d);
      ks[m] = __ldg(ksc + (s >> bshift));
    }
  };
  auto load_v = [&](int tb) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int s = tb + 16 * m < last ? tb + 16 * m : first;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        load_row<8, D>(vr[m][i], vc + (int64_t)(s + 2 * t + (i & 1) + 8 * (i >> 1)) * c.d, g, c.d);
      vs[m] = __ldg(vsc + (s >> bshift));
    }
  };

  int tb = first + warp * STEP;
  if (tb < last) { load_k(tb); load_v(tb); }
  for (; tb < last; tb += AW * STEP) {
    // ---- S^T = K q^T
    float s[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[m][n][e] = 0.f;
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      uint2 q0[NT], q1[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        q0[n] = sm.q[0][w][n][lane];
        if (QT == 2) q1[n] = sm.q[1][w][n][lane];
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const uint32_t x0 = Wd::prep(kr[m][0][w]), x1 = Wd::prep(kr[m][1][w]);
        const uint32_t op[4] = {Wd::lo(x0), Wd::lo(x1), Wd::hi(x0), Wd::hi(x1)};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_f16(s[m][n], op, q0[n].x, q0[n].y);
          if (QT == 2) mma_f16(s[m][n], op, q1[n].x, q1[n].y);
        }
      }
    }
    bool rise = false;
    float lv[MT];                                // log2 of the values' scales
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      lv[m] = __log2f(fabsf(vs[m]));
      const int j0 = tb + 16 * m + g;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float2 rf = *reinterpret_cast<const float2*>(&sm.rowf[8 * n + 2 * t]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float f = (e ? rf.y : rf.x) * ks[m];
          const float edge = fminf(mo[2 * n + e], ao[2 * n + e] - lv[m]) + kSlack;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float x = s[m][n][e + 2 * i] * f;
            s[m][n][e + 2 * i] = j0 + 8 * i < last ? x : -INFINITY;
            rise |= s[m][n][e + 2 * i] > edge;
          }
        }
      }
    }
    if (a.scores) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = row0 + 8 * n + 2 * t + (e & 1), j = tb + 16 * m + g + 8 * (e >> 1);
            if (r < a.rows && j < last) a.scores[(bh * a.rows + r) * c.Ncap + j] = s[m][n][e];
          }
    }
    if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = -INFINITY, atop = -INFINITY;
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const float x = fmaxf(s[m][n][e], s[m][n][e + 2]);
            top = fmaxf(top, x);
            atop = fmaxf(atop, x + lv[m]);       // a NaN (no token of a block of zeros) is passed over
          }
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            atop = fmaxf(atop, __shfl_xor_sync(0xffffffffu, atop, o));
          }
          const float m0 = mo[2 * n + e], a0 = ao[2 * n + e];
          const float m1 = fmaxf(m0, top - kOff);
          // F = exp2(m1 - a1) stays finite: a block of tiny values cannot lie more than 2^100 below
          const float a1 = fmaxf(fmaxf(a0, atop - kOff), m1 - 100.f);
          mo[2 * n + e] = m1;
          ao[2 * n + e] = a1;
          F[2 * n + e] = exp2f(m1 - a1);
          l[2 * n + e] *= exp2f(m0 - m1);
          const float f = exp2f(a0 - a1);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) { acc[i][n][e] *= f; acc[i][n][e + 2] *= f; }
        }
    }
    // ---- P, and O^T += V^T P^T
    const bool more = tb + AW * STEP < last;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      uint32_t p0[NT][2], p1[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = exp2f(s[m][n][e] - mo[2 * n + (e & 1)]);
          l[2 * n + (e & 1)] += x;
          w[e] = x * (vs[m] * F[2 * n + (e & 1)]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t hi = pack_f16(w[2 * i], w[2 * i + 1]);
          p0[n][i] = transpose8(hi);
          if (QT == 2) {
            const float2 u = unpack_f16(hi);
            p1[n][i] = transpose8(pack_f16(w[2 * i] - u.x, w[2 * i + 1] - u.y));
          }
        }
      }
      if (m == 0 && more) {
        // the next step's keys are under way while this step's values are used
        load_k(tb + AW * STEP);
      }
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        const uint32_t x0 = Wd::prep(vr[m][0][w]), x1 = Wd::prep(vr[m][1][w]);
        const uint32_t x2 = Wd::prep(vr[m][2][w]), x3 = Wd::prep(vr[m][3][w]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t sel = e ? 0x7362 : 0x5140;
          const uint32_t u = prmt(x0, x1, sel), v = prmt(x2, x3, sel);
          const uint32_t op[4] = {Wd::lo(u), Wd::hi(u), Wd::lo(v), Wd::hi(v)};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_f16(acc[2 * w + e][n], op, p0[n][0], p0[n][1]);
            if (QT == 2) mma_f16(acc[2 * w + e][n], op, p1[n][0], p1[n][1]);
          }
        }
      }
    }
    if (more) load_v(tb + AW * STEP);
  }

  // ---- join the warps: 3 -> 1 and 2 -> 0, then 1 -> 0
  // in units of exp2(m): sums and accumulators
  float m[2 * NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * n + e;
      m[i] = mo[i] > kUnset ? mo[i] + kOff : -INFINITY;
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
      l[i] *= 0.0625f;                           // 2^-kOff
      const float unit = Wd::gain * 0.0625f / F[i];
#pragma unroll
      for (int k = 0; k < D / 16; ++k) { acc[k][n][e] *= unit; acc[k][n][e + 2] *= unit; }
    }
#pragma unroll
  for (int half = AW / 2; half > 0; half /= 2) {
    __syncthreads();
    if (warp >= half && warp < 2 * half) {
      float* y = sm.y[warp - half];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) y[((n * (D / 16) + i) * 4 + e) * 32 + lane] = acc[i][n][e];
      if (g == 0)
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) sm.ml[warp - half][8 * (i / 2) + 2 * t + i % 2] = make_float2(m[i], l[i]);
    }
    __syncthreads();
    if (warp < half) {
      const float* y = sm.y[warp];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 o = sm.ml[warp][8 * n + 2 * t + e];
          const float mn = fmaxf(m[2 * n + e], o.x), z = mn == -INFINITY ? 0.f : mn;
          const float f0 = exp2f(m[2 * n + e] - z), f1 = exp2f(o.x - z);
          m[2 * n + e] = mn;
          l[2 * n + e] = l[2 * n + e] * f0 + o.y * f1;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            acc[i][n][e] = acc[i][n][e] * f0 + f1 * y[((n * (D / 16) + i) * 4 + e) * 32 + lane];
            acc[i][n][e + 2] = acc[i][n][e + 2] * f0 + f1 * y[((n * (D / 16) + i) * 4 + e + 2) * 32 + lane];
          }
        }
    }
  }
  if (warp) return;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = row0 + 8 * n + 2 * t + e;
      if (r >= a.rows) continue;
      const int64_t at = (bh * a.rows + r) * a.ST + split;
      if (g == 0) a.part_ml[at] = make_float2(m[2 * n + e], l[2 * n + e]);
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        const int dim = word_at<8>(D, w, g);
        if (dim < c.d)
          *reinterpret_cast<float4*>(a.part_y + at * c.d + dim) =
              make_float4(acc[2 * w][n][e], acc[2 * w][n][e + 2], acc[2 * w + 1][n][e], acc[2 * w + 1][n][e + 2]);
      }
    }
}

// Exact tokens: TT tokens at a time in shared memory as fp32; a lane's token
// against the warp's rows for the scores, a lane's elements for the values.
// fp32 throughout; the ring is small beside the cache.
constexpr int TT = 32, TR = 8;   // tokens of a tile, rows of a CTA

__global__ void __launch_bounds__(AT) kv8_tail_kernel(const Kv8AttnArgs a) {
  extern __shared__ __align__(16) float tsm[];
  griddep_wait();
  const lla_kv8_attn_params& p = a.p;
  const lla_kv8_cache& c = p.cache;
  const int d = c.d, pitch = d + 4, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float* tk = tsm;                               // [TT][pitch]
  float* tv = tk + TT * pitch;
  float* tq = tv + TT * pitch;                   // [TR][d]
  float* tp = tq + TR * d;                       // [TR][TT]
  const int chunk = blockIdx.x, rt = blockIdx.y / c.H, h = blockIdx.y % c.H, b = blockIdx.z;
  const Tokens tok(p, b);
  const int row0 = rt * TR, rows = min(TR, a.rows - row0);
  const int64_t bh = (int64_t)b * c.H + h;
  const int first = chunk * a.tpc;
  const int last = min(min(tok.tail, first + a.tpc), visible(tok.tail, (a.row0 + row0 + rows - 1) / p.G, p.nq));
  if (first >= last) {
    if (tid < rows) a.part_ml[(bh * a.rows + row0 + tid) * a.ST + a.S + chunk] = make_float2(-INFINITY, 0.f);
    return;
  }
  for (int i = tid; i < rows * d; i += AT) {
    const int row = a.row0 + row0 + i / d;
    tq[i] = a.qmul * load_elem(p.q, (int64_t)b * p.q_stride_b + (int64_t)(row / p.G) * p.q_stride_n +
                                        (int64_t)(h * p.G + row % p.G) * d + i % d, p.dtype);
  }
  constexpr int RW = TR / AW;                    // rows of a warp: warp, warp + AW
  int vis[RW];
  float m[RW], l[RW], acc[RW][8];
#pragma unroll
  for (int r = 0; r < RW; ++r) {
    const int row = row0 + warp + AW * r;
    vis[r] = row < a.rows ? visible(tok.tail, (a.row0 + row) / p.G, p.nq) : 0;
    m[r] = -INFINITY; l[r] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[r][i] = 0.f;
  }
  const int64_t wb = (int64_t)b * p.win_stride_b + (int64_t)h * p.win_stride_h;
  for (int t0 = first; t0 < last; t0 += TT) {
    __syncthreads();
    const int n = min(TT, last - t0);
    for (int i = tid; i < TT * (d / 4); i += AT) {
      const int j = i / (d / 4), e = 4 * (i % (d / 4));
      float4 k = make_float4(0, 0, 0, 0), v = k;
      if (j < n) {
        const int64_t at = wb + (int64_t)slot_of(tok.pos0 + t0 + j, p.Wcap) * p.win_stride_n + e;
        if (p.win_dtype == LLA_BF16) {
          const uint2 x = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.win_k) + at));
          const uint2 y = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.win_v) + at));
          k = make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u), __uint_as_float(x.y << 16),
                          __uint_as_float(x.y & 0xffff0000u));
          v = make_float4(__uint_as_float(y.x << 16), __uint_as_float(y.x & 0xffff0000u), __uint_as_float(y.y << 16),
                          __uint_as_float(y.y & 0xffff0000u));
        } else {
          k = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.win_k) + at));
          v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.win_v) + at));
        }
      }
      *reinterpret_cast<float4*>(tk + j * pitch + e) = k;
      *reinterpret_cast<float4*>(tv + j * pitch + e) = v;
    }
    __syncthreads();
    float s[RW];
#pragma unroll
    for (int r = 0; r < RW; ++r) s[r] = 0.f;
    for (int e = 0; e < d; e += 4) {
      const float4 k = *reinterpret_cast<const float4*>(tk + lane * pitch + e);
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        const float4 q = *reinterpret_cast<const float4*>(tq + (warp + AW * r) * d + e);
        s[r] += q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
      }
    }
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      const bool see = t0 + lane < min(vis[r], last);
      const float x = see ? s[r] : -INFINITY;
      const float mn = fmaxf(m[r], warp_max(x)), z = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(m[r] - z), e = see ? exp2f(x - z) : 0.f;
      m[r] = mn;
      l[r] = l[r] * f + warp_sum(e);
      tp[(warp + AW * r) * TT + lane] = e;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[r][i] *= f;
    }
    __syncwarp();
    // a row that does not see a token must not meet its value: 0 times a NaN is one
    for (int j = 0; j < n; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = lane + 32 * i;
        if (e >= d) break;
        const float v = tv[j * pitch + e];
#pragma unroll
        for (int r = 0; r < RW; ++r)
          if (t0 + j < vis[r]) acc[r][i] += tp[(warp + AW * r) * TT + j] * v;
      }
    }
  }
#pragma unroll
  for (int r = 0; r < RW; ++r) {
    const int row = row0 + warp + AW * r;
    if (row >= a.rows) continue;
    const int64_t at = (bh * a.rows + row) * a.ST + a.S + chunk;
    if (lane == 0) a.part_ml[at] = make_float2(m[r], l[r]);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane + 32 * i < d) a.part_y[at * d + lane + 32 * i] = acc[r][i];
  }
}

// Joins the splits of a row: (m, 1 / l) over all of them, by one warp.
__device__ __forceinline__ float2 row_ml(const float2* ml, int ST) {
  const int lane = threadIdx.x & 31;
  float m = -INFINITY, l = 0.f;
  for (int i = lane; i < ST; i += 32) {
    const float2 x = ml[i];
    const float mn = fmaxf(m, x.x), z = mn == -INFINITY ? 0.f : mn;
    l = l * exp2f(m - z) + x.y * exp2f(x.x - z);
    m = mn;
  }
  const float top = warp_max(m), z = top == -INFINITY ? 0.f : top;
  l = warp_sum(l * exp2f(m - z));
  return make_float2(z, l == 0.f ? 0.f : 1.f / l);
}

constexpr int JT = 512;          // cached tokens of a weights CTA

// CTAs below `joins` write the outputs, a warp for each row; the others add a
// stretch of the head's weights: each token's terms over the rows in order.
__global__ void __launch_bounds__(AT) kv8_join_kernel(const Kv8AttnArgs a, int joins) {
  __shared__ float2 sml[32];
  griddep_wait();
  const lla_kv8_attn_params& p = a.p;
  const lla_kv8_cache& c = p.cache;
  const int h = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t bh = (int64_t)b * c.H + h;
  if ((int)blockIdx.x < joins) {
    const int r = blockIdx.x * AW + warp;
    if (r >= a.rows) return;
    const float2* ml = a.part_ml + (bh * a.rows + r) * a.ST;
    const float2 all = row_ml(ml, a.ST);
    const float* y = a.part_y + (bh * a.rows + r) * a.ST * c.d;
    const int row = a.row0 + r, qp = row / p.G, gq = row % p.G;
    const int64_t o = (int64_t)b * p.out_stride_b + (int64_t)qp * p.out_stride_n + (int64_t)(h * p.G + gq) * c.d;
    for (int e = 4 * lane; e < c.d; e += 128) {
      float4 s = make_float4(0, 0, 0, 0);
      for (int i = 0; i < a.ST; ++i) {
        const float2 x = ml[i];
        if (x.x == -INFINITY && x.y == 0.f) continue;     // an empty split wrote no y
        const float f = exp2f(x.x - all.x);
        const float4 v = *reinterpret_cast<const float4*>(y + (int64_t)i * c.d + e);
        s.x += f * v.x; s.y += f * v.y; s.z += f * v.z; s.w += f * v.w;
      }
      store_elem(p.out, o + e, p.dtype, s.x * all.y);
      store_elem(p.out, o + e + 1, p.dtype, s.y * all.y);
      store_elem(p.out, o + e + 2, p.dtype, s.z * all.y);
      store_elem(p.out, o + e + 3, p.dtype, s.w * all.y);
    }
    return;
  }
  const int len = min(max(kv8_at(p.len, b), 0), c.Ncap), j0 = (blockIdx.x - joins) * JT;
  if (j0 >= len) return;
  float sum[JT / AT];
#pragma unroll
  for (int i = 0; i < JT / AT; ++i) sum[i] = 0.f;
  for (int r0 = 0; r0 < a.rows; r0 += 32) {
    const int n = min(32, a.rows - r0);
    __syncthreads();
    for (int r = warp; r < n; r += AW) {
      const float2 x = row_ml(a.part_ml + (bh * a.rows + r0 + r) * a.ST, a.ST);
      if (lane == 0) sml[r] = x;
    }
    __syncthreads();
    for (int r = 0; r < n; ++r) {
      const float* s = a.scores + (bh * a.rows + r0 + r) * c.Ncap;
#pragma unroll
      for (int i = 0; i < JT / AT; ++i) {
        const int j = j0 + threadIdx.x + AT * i;
        if (j < len) sum[i] += exp2f(s[j] - sml[r].x) * sml[r].y;
      }
    }
  }
  float* w = p.weights + (int64_t)b * p.weights_stride_b + (int64_t)h * p.weights_stride_h;
#pragma unroll
  for (int i = 0; i < JT / AT; ++i) {
    const int j = j0 + threadIdx.x + AT * i;
    if (j < len) w[j] += sum[i];
  }
}

template <int CODE, int D, int NT, int QT>
cudaError_t launch_split(const Kv8AttnArgs& a, cudaStream_t st) {
  const lla_kv8_cache& c = a.p.cache;
  constexpr size_t smem = sizeof(AttnSmem<D, NT>);
  auto* kern = kv8_attn_kernel<CODE, D, NT, QT>;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(kern, dim3(a.S, ceil_div(a.rows, 8 * NT) * c.H, c.B), dim3(AT), smem, st, 1, a);
}

template <int CODE, int D, int QT>
cudaError_t launch_rows(const Kv8AttnArgs& a, cudaStream_t st) {
  if (a.nt == 1) return launch_split<CODE, D, 1, QT>(a, st);
  if constexpr (D <= 128)
    if (a.nt == 4) return launch_split<CODE, D, 4, QT>(a, st);
  return launch_split<CODE, D, 2, QT>(a, st);
}

template <int CODE, int QT>
cudaError_t launch_d(const Kv8AttnArgs& a, cudaStream_t st) {
  const int d = a.p.cache.d;
  if (d <= 64) return launch_rows<CODE, 64, QT>(a, st);
  if (d <= 96) return launch_rows<CODE, 96, QT>(a, st);
  if (d <= 128) return launch_rows<CODE, 128, QT>(a, st);
  return launch_rows<CODE, 256, QT>(a, st);
}

}  // namespace

cudaError_t launch_kv8_attn(const Kv8AttnArgs& a0, cudaStream_t st) {
  const lla_kv8_cache& c = a0.p.cache;
  const int total = a0.rows;
  for (int row0 = 0; row0 < total; row0 += a0.rows_pass) {
    Kv8AttnArgs a = a0;
    a.row0 = row0;
    a.rows = total - row0 < a0.rows_pass ? total - row0 : a0.rows_pass;
    cudaError_t e = cudaSuccess;
    if (a.S) {
      if (c.code == LLA_KV8_I8) e = a.p.dtype == LLA_F32 ? launch_d<LLA_KV8_I8, 2>(a, st) : launch_d<LLA_KV8_I8, 1>(a, st);
      else e = a.p.dtype == LLA_F32 ? launch_d<LLA_KV8_E4M3, 2>(a, st) : launch_d<LLA_KV8_E4M3, 1>(a, st);
    }
    if (e == cudaSuccess && a.ST > a.S) {
      const size_t smem = (size_t)(2 * TT * (c.d + 4) + TR * c.d + TR * TT) * sizeof(float);
      if (smem > 48 * 1024)
        e = cudaFuncSetAttribute(kv8_tail_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e == cudaSuccess)
        e = launch_kernel(kv8_tail_kernel, dim3(a.ST - a.S, ceil_div(a.rows, TR) * c.H, c.B), dim3(AT), smem, st, 1, a);
    }
    if (e != cudaSuccess) return e;
    const int joins = ceil_div(a.rows, AW);
    e = launch_kernel(kv8_join_kernel, dim3(joins + (a.p.weights ? ceil_div(c.Ncap, JT) : 0), c.H, c.B), dim3(AT), 0, st,
                      1, a, joins);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace lla
