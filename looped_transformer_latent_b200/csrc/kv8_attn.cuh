// Attention over the 8-bit K/V cache and the exact tokens after it: the split
// kernel, included by one source per code format.
//
// A CTA serves RT = 8 NT query rows of one (sequence, cache head) over one
// split of the cached tokens.  Each warp streams its own tiles of 16 tokens
// through its own ring of shared memory (cp.async, no barrier beyond the warp),
// reads the bytes in the operand order of the f16 m16n8k16 product, widens the
// 8-bit codes to f16 in registers (exact), and keeps its own running maximum,
// sum and accumulator; warps are joined through shared memory, splits by
// kv8_join_kernel.
//   S^T [tokens x rows] = K q^T   K codes as the A operand, q as B
//   O^T [d x rows]     += V^T P^T V codes as A (pairs of tokens interleaved
//                                 while widening), P from S^T by movmatrix
// so any number of rows up to 8 NT shares each widened code.  A lane's bytes
// of a row are contiguous: which element a product index stands for is free as
// long as both operands agree.
// CTAs past the cached splits serve the exact tokens, with bf16 products of as
// many terms as the types need.
// Up to 8 rows it is bound by HBM: 32 x 16 heads of 128, 4096 e4m3 tokens and 129
// exact ones take 108 us, 5.3 TB/s, 81 % of the copy rate; widened by shifts and
// masks instead of the conversion instruction the same read took 196.  Beyond, by
// the latency of instructions that wait for one another: with 32 rows a thread
// needs 255 registers, which leaves 8 warps an SM, and these issue 1.9 of 4
// instructions a cycle (545 for 16 tokens, 48 of them products, 33 % of their
// pipe); 16 x 55 heads of 96, 32 rows, 4096 int8 tokens take 235 us (3.0 TB/s).
// fp32 queries double the products and add their sums apart: 585 instructions for
// 16 tokens of one tile of 8 rows, 2.2 a cycle from 15 warps an SM, 300 MB of
// 96-element heads with their weights in 103 us.  Rings and not register prefetch:
// with 8 warps an SM the registers held 24 KB under way, half of what the memory's
// latency asks for (462 us).
#pragma once

#include "kernels.cuh"
#include "kv8_math.cuh"
#include "tc_ptx.cuh"

namespace lla {
namespace kv8 {

using ptx::ex2;                  // below 2^-126 it is 0

constexpr int AT = 128;          // threads
constexpr int AW = AT / 32;

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
// Widening of codes to f16, exact.  lo, hi: the two lower and the two upper
// bytes of a word; pairs: byte i of a beside byte i of b, for i = 0, 1 and 2, 3.
// int8: the byte plus 128 in the low mantissa bits of 1024, less 1152 (1.25
// integer and half instructions an element; 1.5 with the interleave).  e4m3:
// the conversion instruction, two elements each (0.75; 1 with the interleave).
template <int CODE>
struct Widen;
template <>
struct Widen<LLA_KV8_I8> {
  static __device__ __forceinline__ uint32_t prep(uint32_t w) { return w ^ 0x80808080u; }
  static __device__ __forceinline__ uint32_t lo(uint32_t w) { return sub_f16x2(prmt(w, 0x64646464u, 0x4140), 0x64806480u); }
  static __device__ __forceinline__ uint32_t hi(uint32_t w) { return sub_f16x2(prmt(w, 0x64646464u, 0x4342), 0x64806480u); }
  static __device__ __forceinline__ void pairs(uint32_t a, uint32_t b, uint32_t (&o)[4]) {
    const uint32_t u = prmt(a, b, 0x5140), v = prmt(a, b, 0x7362);
    o[0] = lo(u); o[1] = hi(u); o[2] = lo(v); o[3] = hi(v);
  }
};
template <>
struct Widen<LLA_KV8_E4M3> {
  static __device__ __forceinline__ uint32_t prep(uint32_t w) { return w; }
  static __device__ __forceinline__ uint32_t lo(uint32_t w) { return e4m3_f16x2(w); }
  static __device__ __forceinline__ uint32_t hi(uint32_t w) { return e4m3_f16x2(w >> 16); }
  static __device__ __forceinline__ void pairs(uint32_t a, uint32_t b, uint32_t (&o)[4]) {
    o[0] = e4m3_f16x2(prmt(a, b, 0x0040)); o[1] = e4m3_f16x2(prmt(a, b, 0x0051));
    o[2] = e4m3_f16x2(prmt(a, b, 0x0062)); o[3] = e4m3_f16x2(prmt(a, b, 0x0073));
  }
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float2 unpack_f16(uint32_t h) {
  float2 r;
  asm("{.reg .f16 l, h; mov.b32 {l, h}, %2; cvt.f32.f16 %0, l; cvt.f32.f16 %1, h;}" : "=f"(r.x), "=f"(r.y) : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_bf16(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
// T terms of bf16 whose sum is x to 8 T bits
template <int T>
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t (&o)[T]) {
#pragma unroll
  for (int i = 0; i < T; ++i) {
    o[i] = pack_bf16(x, y);
    const float2 u = unpack_bf16(o[i]);
    x -= u.x; y -= u.y;
  }
}
// 8 x 8 transpose across the warp: lane (g, t) of (row g, columns 2t, 2t + 1)
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
// 16 bytes, or zeros without a read where !ok
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int W>
__device__ __forceinline__ void lds(uint32_t* r, uint32_t at) {
  if constexpr (W == 4)
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at));
  else if constexpr (W == 2)
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(at));
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r[0]) : "r"(at));
}

// Byte offset of a lane's word w (4 codes) in a row of D codes: K rows are
// shared by the 4 lanes t of a group (D / 16 words each), V rows by the 8 groups
// g (D / 32 words each); in both, pieces of 16 bytes, then of what is left.
template <int LANES>
__host__ __device__ __forceinline__ constexpr int word_at(int D, int w, int lane) {
  const int full = D / (16 * LANES);             // pieces of 16 bytes
  if (w < 4 * full) return 16 * LANES * (w / 4) + 16 * lane + 4 * (w % 4);
  const int left = D / LANES - 16 * full;        // bytes of the last pieces: 8, 4 or 12
  const int w2 = w - 4 * full;
  if (left >= 8 && w2 < 2) return 16 * LANES * full + 8 * lane + 4 * w2;
  return 16 * LANES * full + (left >= 8 ? 8 * LANES : 0) + 4 * lane;
}
// The same for exact rows of 2- or 4-byte elements: element offset of a lane's
// group w of 4 elements.
__device__ __forceinline__ int quad_k(int w, int t) { return 32 * (w / 2) + 8 * t + 4 * (w % 2); }
template <int D>
__device__ __forceinline__ int quad_v(int w, int g) {
  return w < 2 * (D / 64) ? 64 * (w / 2) + 8 * g + 4 * (w % 2) : 64 * (D / 64) + 4 * g;
}

// A row of a tile in shared memory: pitch bytes, its 16-byte pieces exchanged
// so that neither the K reads (rows 2i, 2i + 1 in one phase) nor the V reads
// (rows 2t of four t) meet in a bank.
template <int D>
struct Row {
  static constexpr int pitch = D <= 64 ? 64 : D <= 128 ? 128 : 256;
  static __device__ __forceinline__ int at(int r, int byte) {
    const int sw = ((((r >> 2) ^ r) & 1) << 2 | (r & 2)) & (pitch / 16 - 1);
    return r * pitch + (((byte >> 4) ^ sw) << 4) + (byte & 15);
  }
};

// LANES lanes' words of row r, in order
template <int LANES, int D>
__device__ __forceinline__ void read_row(uint32_t* w, uint32_t base, int r, int lane) {
  constexpr int W = D / (4 * LANES), full = W / 4, left = W % 4;
#pragma unroll
  for (int i = 0; i < full; ++i) lds<4>(w + 4 * i, base + Row<D>::at(r, word_at<LANES>(D, 4 * i, lane)));
  if constexpr (left >= 2) lds<2>(w + 4 * full, base + Row<D>::at(r, word_at<LANES>(D, 4 * full, lane)));
  if constexpr (left % 2) lds<1>(w + W - 1, base + Row<D>::at(r, word_at<LANES>(D, W - 1, lane)));
}

// Queries enter as f16 under a power of two per row that puts the row's largest
// magnitude into [2^13, 2^14): a bf16 query is exact, a second term adds the
// next 11 bits of an fp32 one.
constexpr int kQExp = 13;
// Running references of a row, both base-2 exponents: m of the probabilities
// p = exp2(s - m), a of what meets the value codes, w = 2^kMost exp2(s + log2(scale) - a),
// so that a block whose values are 2^60 times another's does not drown it.  A
// reference is set kSlack above a new maximum and moves only when a logit
// exceeds it: p <= 1, w <= 2^15 in f16 and the largest of them above 2^2, and
// most tiles need neither a shuffle nor a rescaling.  One f16 term loses what lies
// 27 bits below the largest.  fp32: the second term is what the first leaves of w,
// times kLow, and meets the codes first; its products are taken back by that
// power of two, and what is lost lies 39 bits below the largest (without it a flat
// rest of 4096 tokens of a warp, 25 bits below a peak, was lost: 1e-4 of the output).
// References are whole numbers, so that moving one is exact, and of a only m - a is
// kept, which means the same however large the logits are.
constexpr float kSlack = 12.f, kMost = 15.f, kUnset = -3.4e38f;
constexpr float kLow = 0x1p12f, kLowInv = 0x1p-12f;
// from here on the rounding of a product exceeds the slack of f16, and the difference to a reference is taken from
// the rounded logit, which lies below it
constexpr float kHuge = 16777216.f;


// MT: tiles of 16 tokens that a warp takes at a time.
template <int D, int NT, int MT>
struct Smem {
  static constexpr int RT = 8 * NT;
  static constexpr int STAGES = MT == 1 ? 3 : 2;                      // of a warp's ring, one of them in use
  static constexpr int tile = 16 * MT * Row<D>::pitch;                // bytes of a stage's rows
  uint2 q[3][D / 16][NT][32];    // query terms, B operand order
  float rowf[RT];                // row exponent times scale log2(e)
  float2 ml[2][RT];              // join of the warps
  union {
    struct {
      uint8_t kv[AW][STAGES][2][tile];
      float scales[AW][STAGES][2];
    } ring;
    float y[2][D * RT];          // join of the warps; probabilities of a tile of exact tokens
  };
};

// The CTA's rows in a launch, and the call's row numbers.
struct Place {
  int split, h, b, row0;
  int64_t bh;
  __device__ Place(const Kv8AttnArgs& a, int RT) {
    split = blockIdx.x + a.split0;
    h = blockIdx.y % a.p.cache.H;
    row0 = blockIdx.y / a.p.cache.H * RT;
    b = blockIdx.z;
    bh = (int64_t)b * a.p.cache.H + h;
  }
  __device__ int64_t query(const Kv8AttnArgs& a, int r) const {       // element offset of row r's query
    const int row = a.row0 + row0 + r, qp = row / a.p.G, gq = row % a.p.G;
    return (int64_t)b * a.p.q_stride_b + (int64_t)qp * a.p.q_stride_n + (int64_t)(h * a.p.G + gq) * a.p.cache.d;
  }
  __device__ int64_t output(const Kv8AttnArgs& a, int r) const {      // and of its output
    const int row = a.row0 + row0 + r, qp = row / a.p.G, gq = row % a.p.G;
    return (int64_t)b * a.p.out_stride_b + (int64_t)qp * a.p.out_stride_n + (int64_t)(h * a.p.G + gq) * a.p.cache.d;
  }
};

// Join of the warps, 3 -> 1 and 2 -> 0, then 1 -> 0, and the split's partial
// results.  acc, l in units of exp2(m); base(w): first element of quad w.
template <int D, int NT, int MT, class Base>
__device__ __forceinline__ void join_store(const Kv8AttnArgs& a, Smem<D, NT, MT>& sm, const Place& at_, float (&acc)[D / 16][NT][4],
                                           float (&m)[2 * NT], float (&l)[2 * NT], Base base) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
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
  const int d = a.p.cache.d;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = at_.row0 + 8 * n + 2 * t + e;
      if (r >= a.rows) continue;
      if (a.direct) {                            // the only split: these are the sums
        const float inv = l[2 * n + e] == 0.f ? 0.f : 1.f / l[2 * n + e];
        const int64_t o = at_.output(a, r - at_.row0);
#pragma unroll
        for (int w = 0; w < D / 32; ++w)
          if (base(w) < d)
            store_quad(a.p.out, o + base(w), a.p.dtype,
                       make_float4(acc[2 * w][n][e], acc[2 * w][n][e + 2], acc[2 * w + 1][n][e], acc[2 * w + 1][n][e + 2]), inv);
        continue;
      }
      if (a.cluster) {                           // for the other CTAs of the cluster to read (y[1] and ml[1] are done with)
        if (g == 0) sm.ml[1][r - at_.row0] = make_float2(m[2 * n + e], l[2 * n + e]);
#pragma unroll
        for (int w = 0; w < D / 32; ++w)
          if (base(w) < d)
            *reinterpret_cast<float4*>(&sm.y[1][(r - at_.row0) * D + base(w)]) =
                make_float4(acc[2 * w][n][e], acc[2 * w][n][e + 2], acc[2 * w + 1][n][e], acc[2 * w + 1][n][e + 2]);
        continue;
      }
      const int64_t at = (at_.bh * a.rows + r) * a.ST + at_.split;
      if (g == 0) a.part_ml[at] = make_float2(m[2 * n + e], l[2 * n + e]);
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        const int dim = base(w);
        if (dim < d)
          *reinterpret_cast<float4*>(a.part_y + at * d + dim) =
              make_float4(acc[2 * w][n][e], acc[2 * w][n][e + 2], acc[2 * w + 1][n][e], acc[2 * w + 1][n][e + 2]);
      }
    }
}

// Nothing to see in this split: the join must not read what was there.
template <int RT>
__device__ __forceinline__ void empty_split(const Kv8AttnArgs& a, const Place& at, float2 (&ml)[2][RT]) {
  if (a.cluster) {
    if ((int)threadIdx.x < RT) ml[1][threadIdx.x] = make_float2(-INFINITY, 0.f);
    return;
  }
  if (a.direct) {
    for (int i = threadIdx.x; i < RT * (a.p.cache.d / 4); i += AT) {
      const int r = i / (a.p.cache.d / 4);
      if (at.row0 + r < a.rows)
        store_quad(a.p.out, at.output(a, r) + 4 * (i % (a.p.cache.d / 4)), a.p.dtype, make_float4(0, 0, 0, 0), 0.f);
    }
    return;
  }
  if ((int)threadIdx.x < RT && at.row0 + (int)threadIdx.x < a.rows)
    a.part_ml[(at.bh * a.rows + at.row0 + threadIdx.x) * a.ST + at.split] = make_float2(-INFINITY, 0.f);
}

// Join of the splits of a cluster through its shared memory: a warp for each
// row, the rows over the CTAs.  Lane k reads CTA k's maximum and sum; the loads
// of all CTAs' y are under way together.
template <int D, int NT, int MT>
__device__ __forceinline__ void cluster_join(const Kv8AttnArgs& a, Smem<D, NT, MT>& sm) {
  const Place at(a, 8 * NT);
  const int d = a.p.cache.d, rows = min(8 * NT, a.rows - at.row0), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  ptx::cluster_sync_all();
  const uint32_t ml = smem_addr(sm.ml[1]), y = smem_addr(sm.y[1]);
  for (int r = at.split * AW + warp; r < rows; r += a.ST * AW) {
    float m = -INFINITY, l = 0.f;
    if (lane < a.ST) {
      const uint32_t x = ptx::mapa_shared(ml + 8 * r, lane);
      m = ptx::ld_shared_cluster(x);
      l = ptx::ld_shared_cluster(x + 4);
    }
    const unsigned some = __ballot_sync(0xffffffffu, !(m == -INFINITY && l == 0.f));   // an empty split wrote no y
    const float top = warp_max(m), f = exp2f(m - (top == -INFINITY ? 0.f : top)), sum = warp_sum(l * f);
    for (int e = 4 * lane; e - 4 * lane < d; e += 128) {
      float4 s = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int k0 = 0; k0 < 16; k0 += 8) {
        float4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          v[k] = make_float4(0, 0, 0, 0);
          if (e < d && some >> (k0 + k) & 1)
            asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                         : "=f"(v[k].x), "=f"(v[k].y), "=f"(v[k].z), "=f"(v[k].w)
                         : "r"(ptx::mapa_shared(y + 4 * (r * D + e), k0 + k)));
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float g = __shfl_sync(0xffffffffu, f, k0 + k);
          s.x += g * v[k].x; s.y += g * v[k].y; s.z += g * v[k].z; s.w += g * v[k].w;
        }
        if (k0 + 8 >= a.ST) break;
      }
      if (e < d) store_quad(a.p.out, at.output(a, r) + e, a.p.dtype, s, sum == 0.f ? 0.f : 1.f / sum);
    }
  }
  ptx::cluster_sync_all();                       // a CTA's shared memory stays until all have read it
}

// ------------------------------------------------------------ exact tokens --
// exact tokens, of `tail`, that query position qp of nq sees
__device__ __forceinline__ int visible(int tail, int qp, int nq) { return max(0, tail - (nq - 1 - qp)); }

// 4 elements as WT bf16 terms, two words each
template <int WT>
__device__ __forceinline__ void load_quad(uint32_t (&o)[WT][2], const void* x, int64_t at, bool ok) {
  if constexpr (WT == 1) {
    const uint2 v = ok ? __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(x) + at)) : make_uint2(0, 0);
    o[0][0] = v.x; o[0][1] = v.y;
  } else {
    const float4 v = ok ? __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(x) + at)) : make_float4(0, 0, 0, 0);
    uint32_t u[WT], w[WT];
    split_bf16<WT>(v.x, v.y, u);
    split_bf16<WT>(v.z, v.w, w);
#pragma unroll
    for (int i = 0; i < WT; ++i) { o[i][0] = u[i]; o[i][1] = w[i]; }
  }
}
// Whether one of 4 elements is an infinity or a NaN, or becomes one as a bf16 term.
template <int WT>
__device__ __forceinline__ bool no_number(const void* x, int64_t at) {
  if constexpr (WT == 1) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(x) + at));
    const uint32_t m = __vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu);
    return (m & 0xffffu) >= 0x7f80u || m >= 0x7f800000u;
  } else {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(static_cast<const float*>(x) + at));
    const uint32_t m = 0x7fffffffu;
    return max(max(v.x & m, v.y & m), max(v.z & m, v.w & m)) >= 0x7f7f8000u;
  }
}

// s += the products of 16 elements, of WT terms on one side and YT on the other.
// fp32 (QT 2): summed apart, the smallest terms first, and added to nearest: the
// product unit's sums are not, and 48 of them in a row (heads of 128) shrank the
// logits by 48 x 2^-25, an error of 3e-6 where a call's tokens were mostly exact.
template <int QT, int WT, int YT, class Y>
__device__ __forceinline__ void sum_terms(float (&s)[4], const uint32_t (&x)[WT][4], Y y) {
  if constexpr (QT == 1) {
#pragma unroll
    for (int i = 0; i < WT; ++i)
#pragma unroll
      for (int k = 0; k < YT && i + k <= 2; ++k) mma_bf16(s, x[i], y(k).x, y(k).y);
  } else {
    float u[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int o = 2; o >= 0; --o)
#pragma unroll
      for (int i = 0; i < WT && i <= o; ++i)
        if (o - i < YT) mma_bf16(u, x[i], y(o - i).x, y(o - i).y);
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] += u[e];
  }
}

// WT: terms of the ring's elements (bf16 1, fp32 3).  QT 1: bf16 queries, one
// exact term, probabilities in two; QT 2: fp32, three of each.  Products of
// terms whose order exceeds the third are left out: they are below 2^-24.
template <int D, int NT, int MT, int QT, int WT>
__device__ __noinline__ void exact_split(const Kv8AttnArgs& a, Smem<D, NT, MT>& sm) {
  constexpr int RT = 8 * NT, QB = QT == 1 ? 1 : 3, PB = QT == 1 ? 2 : 3;
  const lla_kv8_attn_params& p = a.p;
  const int d = p.cache.d, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const Place at(a, RT);
  const int ctx = max(kv8_at(p.ctx, at.b), 0), tail = min(max(kv8_at(p.tail, at.b), 0), min(p.Wcap, ctx));
  const int slot0 = (ctx - tail) % p.Wcap;       // of the oldest exact token
  const int rows = min(RT, a.rows - at.row0);
  const int first = (at.split - a.S) * a.tpc;
  const int last = min(first + a.tpc, visible(tail, (a.row0 + at.row0 + rows - 1) / p.G, p.nq));
  if (first >= last) { empty_split<RT>(a, at, sm.ml); return; }

  for (int i = threadIdx.x; i < RT * (D / 4); i += AT) {
    const int r = i / (D / 4), w = i % (D / 4) / 4, tt = i % 4, e = quad_k(w, tt);
    float x[4];
    load_query(x, p.q, at.query(a, r) + e, p.dtype, r < rows && e < d);
    uint32_t u[QB], v[QB];
    split_bf16<QB>(x[0], x[1], u);
    split_bf16<QB>(x[2], x[3], v);
#pragma unroll
    for (int k = 0; k < QB; ++k) sm.q[k][w][r / 8][(r % 8) * 4 + tt] = make_uint2(u[k], v[k]);
  }
  __syncthreads();

  float acc[D / 16][NT][4], mo[2 * NT], l[2 * NT];
  int vis[2 * NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][n][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = 8 * n + 2 * t + e;
      mo[2 * n + e] = kUnset; l[2 * n + e] = 0.f;
      vis[2 * n + e] = r < rows ? min(last, visible(tail, (a.row0 + at.row0 + r) / p.G, p.nq)) : last;
    }
  }
  const int64_t wb = (int64_t)at.b * p.win_stride_b + (int64_t)at.h * p.win_stride_h;
  auto row_of = [&](int j) {                     // element offset of exact token j; any valid one where there is none
    int s = slot0 + min(j, last - 1);
    if (s >= p.Wcap) s -= p.Wcap;
    return wb + (int64_t)s * p.win_stride_n;
  };
  for (int tb = first + 16 * warp; tb < last; tb += 16 * AW) {
    int64_t vrow[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) vrow[i] = row_of(tb + 2 * t + (i & 1) + 8 * (i >> 1));
    float s[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
    const int64_t k0 = row_of(tb + g), k1 = row_of(tb + g + 8);
    const bool ok0 = tb + g < last, ok1 = tb + g + 8 < last;
#pragma unroll
    for (int w = 0; w < D / 16; ++w) {
      const int e = quad_k(w, t);
      uint32_t x0[WT][2], x1[WT][2];
      load_quad<WT>(x0, p.win_k, k0 + e, ok0 && e < d);
      load_quad<WT>(x1, p.win_k, k1 + e, ok1 && e < d);
      uint32_t op[WT][4];
#pragma unroll
      for (int i = 0; i < WT; ++i) { op[i][0] = x0[i][0]; op[i][1] = x1[i][0]; op[i][2] = x0[i][1]; op[i][3] = x1[i][1]; }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint2 q[QB];
#pragma unroll
        for (int k = 0; k < QB; ++k) q[k] = sm.q[k][w][n][lane];
        sum_terms<QT, WT, QB>(s[n], op, [&](int k) { return q[k]; });
      }
    }
    float pr[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = 2 * n + e;
        const float u = tb + g < vis[i] ? __fmul_rn(s[n][e], a.qmul) : -INFINITY;
        const float v = tb + g + 8 < vis[i] ? __fmul_rn(s[n][e + 2], a.qmul) : -INFINITY;
        float top = fmaxf(u, v);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float m1 = fmaxf(mo[i], top), f = ex2(mo[i] - m1);
        mo[i] = m1;
        // fp32: the difference to the reference is rounded once
        const bool once = QT == 2 && fabsf(m1) < kHuge;
        pr[n][e] = tb + g < vis[i] ? ex2(once ? fmaf(s[n][e], a.qmul, -m1) : u - m1) : 0.f;
        pr[n][e + 2] = tb + g + 8 < vis[i] ? ex2(once ? fmaf(s[n][e + 2], a.qmul, -m1) : v - m1) : 0.f;
        l[i] = l[i] * f + (pr[n][e] + pr[n][e + 2]);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) { acc[k][n][e] *= f; acc[k][n][e + 2] *= f; }
      }
    // values that are no numbers, where a query may not see all tokens (or they have no terms)
    bool odd = false;
    if (p.nq > 1 || WT > 1)
#pragma unroll
      for (int w = 0; w < D / 32; ++w)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = quad_v<D>(w, g);
          odd |= tb + 2 * t + (i & 1) + 8 * (i >> 1) < last && e < d && no_number<WT>(p.win_v, vrow[i] + e);
        }
    if (!__any_sync(0xffffffffu, odd)) {
      uint32_t pt[NT][2][PB];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          split_bf16<PB>(pr[n][2 * i], pr[n][2 * i + 1], pt[n][i]);
#pragma unroll
          for (int k = 0; k < PB; ++k) pt[n][i][k] = transpose8(pt[n][i][k]);
        }
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        const int e = quad_v<D>(w, g);
        uint32_t x[4][WT][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          load_quad<WT>(x[i], p.win_v, vrow[i] + e, tb + 2 * t + (i & 1) + 8 * (i >> 1) < last && e < d);
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            uint32_t op[WT][4];
#pragma unroll
            for (int i = 0; i < WT; ++i) {
              op[i][0] = prmt(x[0][i][k], x[1][i][k], 0x5410); op[i][1] = prmt(x[0][i][k], x[1][i][k], 0x7632);
              op[i][2] = prmt(x[2][i][k], x[3][i][k], 0x5410); op[i][3] = prmt(x[2][i][k], x[3][i][k], 0x7632);
            }
            sum_terms<QT, WT, PB>(acc[2 * w + k][n], op, [&](int o) { return make_uint2(pt[n][0][o], pt[n][1][o]); });
          }
      }
      continue;
    }
    // a query that does not see a token must not meet its value: 0 times infinity is a NaN
    float* ps = &sm.y[0][0] + warp * 16 * RT;    // [16 tokens][RT]
    __syncwarp();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) ps[(g + 8 * (i >> 1)) * RT + 8 * n + 2 * t + (i & 1)] = pr[n][i];
    __syncwarp();
#pragma unroll 1
    for (int j = 0; j < 16 && tb + j < last; ++j) {
      const int64_t row = row_of(tb + j);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int e = quad_v<D>(k / 2, g) + 2 * (k & 1) + i;
          const float v = e < d ? load_elem(p.win_v, row + e, p.win_dtype) : 0.f;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c)
              if (tb + j < vis[2 * n + c]) acc[k][n][c + 2 * i] += ps[j * RT + 8 * n + 2 * t + c] * v;
        }
    }
  }
  float m[2 * NT];
#pragma unroll
  for (int i = 0; i < 2 * NT; ++i) {
    m[i] = mo[i] > kUnset ? mo[i] : -INFINITY;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
  }
  join_store<D, NT, MT>(a, sm, at, acc, m, l, [&](int w) { return quad_v<D>(w, g); });
}

// ----------------------------------------------------------- cached tokens --
template <int CODE, int D, int NT, int MT, int QT>
__device__ __forceinline__ void cached_split(const Kv8AttnArgs& a, Smem<D, NT, MT>& sm) {
  constexpr int RT = 8 * NT, STEP = 16 * MT, STAGES = Smem<D, NT, MT>::STAGES;
  constexpr int KW = D / 16, VW = D / 32;        // words per lane of a K and of a V row
  constexpr int PIECES = MT * (D / 16) / 2;      // 16-byte pieces of a stage that a lane copies
  using Wd = Widen<CODE>;
  const lla_kv8_attn_params& p = a.p;
  const lla_kv8_cache& c = p.cache;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const Place at(a, RT);
  const int h = at.h, b = at.b;
  const int len = min(max(kv8_at(p.len, b), 0), c.Ncap);
  const int first = at.split * a.tps, last = min(len, first + a.tps);   // this split's tokens
  if (first >= last) { empty_split<RT>(a, at, sm.ml); return; }

  const uint8_t* kc = static_cast<const uint8_t*>(c.k) + (int64_t)b * c.stride_b + (int64_t)h * c.stride_h;
  const uint8_t* vc = static_cast<const uint8_t*>(c.v) + (int64_t)b * c.stride_b + (int64_t)h * c.stride_h;
  const float* ksc = c.k_scale + (int64_t)b * c.scale_stride_b + (int64_t)h * c.scale_stride_h;
  const float* vsc = c.v_scale + (int64_t)b * c.scale_stride_b + (int64_t)h * c.scale_stride_h;
  const int bshift = 31 - __clz(c.block);

  // a step of STEP tokens lies inside one block of the cache; rows past `last` are zeros
  auto copy_step = [&](int tb, int stage) {
    const uint32_t ks = smem_addr(sm.ring.kv[warp][stage][0]), vs = smem_addr(sm.ring.kv[warp][stage][1]);
    const uint8_t *kf = kc + (int64_t)tb * c.d, *vf = vc + (int64_t)tb * c.d;
    if (c.d == D && tb + STEP <= last) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const int id = lane + 32 * i, r = id / (D / 16), e = 16 * (id % (D / 16));
        copy16(ks + Row<D>::at(r, e), kf + 16 * id);
        copy16(vs + Row<D>::at(r, e), vf + 16 * id);
      }
    } else
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int id = lane + 32 * i, r = id / (D / 16), e = 16 * (id % (D / 16));
      const bool ok = tb + r < last && e < c.d;
      const int from = ok ? r * c.d + e : 0;
      copy16(ks + Row<D>::at(r, e), kf + from, ok);
      copy16(vs + Row<D>::at(r, e), vf + from, ok);
    }
    if (lane < 2) copy4(smem_addr(&sm.ring.scales[warp][stage][lane]), (lane ? vsc : ksc) + (tb >> bshift));
  };
  int tb = first + STEP * warp;
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) {
    if (tb + STEP * AW * i < last) copy_step(tb + STEP * AW * i, i);
    copy_commit();
  }

  // ---- queries: a warp takes RT / 4 rows, a lane one or two quads of each
  constexpr int QL = (D / 4 + 31) / 32;
#pragma unroll 2
  for (int r = warp; r < RT; r += AW) {
    const bool there = at.row0 + r < a.rows;
    const int64_t qo = at.query(a, r);
    float x[QL][4], top = 0.f;
#pragma unroll
    for (int i = 0; i < QL; ++i) {
      const int id = lane + 32 * i, e = id < D / 4 ? word_at<4>(D, id / 4, id % 4) : D;
      load_query(x[i], p.q, qo + e, p.dtype, there && e < c.d);
#pragma unroll
      for (int k = 0; k < 4; ++k) top = fabsf(x[i][k]) > top || x[i][k] != x[i][k] ? fabsf(x[i][k]) : top;   // NaN stays
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float u = __shfl_xor_sync(0xffffffffu, top, o);
      top = u > top || u != u ? u : top;
    }
    // ilogb of the largest magnitude (of a subnormal: -127) less kQExp; 0 where that is zero or no number
    const int ex = top > 0.f && top < INFINITY ? max((__float_as_int(top) >> 23) - 127 - kQExp, -100) : 0;
    if (lane == 0) sm.rowf[r] = a.qmul * pow2(ex);
    const float down = pow2(-ex);
#pragma unroll
    for (int i = 0; i < QL; ++i) {
      const int id = lane + 32 * i;
      if (id >= D / 4) break;
#pragma unroll
      for (int k = 0; k < 4; ++k) x[i][k] *= down;
      const uint2 v = make_uint2(pack_f16(x[i][0], x[i][1]), pack_f16(x[i][2], x[i][3]));
      sm.q[0][id / 4][r / 8][(r % 8) * 4 + id % 4] = v;
      if (QT == 2) {
        const float2 u0 = unpack_f16(v.x), u1 = unpack_f16(v.y);
        sm.q[1][id / 4][r / 8][(r % 8) * 4 + id % 4] =
            make_uint2(pack_f16(x[i][0] - u0.x, x[i][1] - u0.y), pack_f16(x[i][2] - u1.x, x[i][3] - u1.y));
      }
    }
  }
  __syncthreads();

  float acc[D / 16][NT][4];
  float mo[2 * NT], da[2 * NT], F[2 * NT], l[2 * NT];   // reference m, m - a, F = 2^kMost exp2(m - a), sums
  bool huge = false;                                    // the warp has seen an |m| >= kHuge
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][n][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mo[2 * n + e] = kUnset; da[2 * n + e] = 0.f; F[2 * n + e] = 1.f; l[2 * n + e] = 0.f;
    }
  }

  int stage = 0;
  for (; tb < last; tb += STEP * AW) {
    if (STAGES > 2) copy_wait<STAGES - 2>();
    else copy_wait<0>();
    __syncwarp();                                // every lane's part is there, and the step before is done with
    {
      const int next = tb + STEP * AW * (STAGES - 1), to = stage == 0 ? STAGES - 1 : stage - 1;
      if (next < last) copy_step(next, to);
      copy_commit();
    }
    const uint32_t kt = smem_addr(sm.ring.kv[warp][stage][0]), vt = smem_addr(sm.ring.kv[warp][stage][1]);
    const float ks = sm.ring.scales[warp][stage][0], vs = sm.ring.scales[warp][stage][1];
    stage = stage == STAGES - 1 ? 0 : stage + 1;
    // ---- S^T = K q^T
    float s[MT][NT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[m][n][e] = 0.f;
    {
      uint32_t k[MT][2][KW];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        read_row<4, D>(k[m][0], kt, 16 * m + g, t);
        read_row<4, D>(k[m][1], kt, 16 * m + g + 8, t);
      }
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        uint32_t op[MT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const uint32_t x0 = Wd::prep(k[m][0][w]), x1 = Wd::prep(k[m][1][w]);
          op[m][0] = Wd::lo(x0); op[m][1] = Wd::lo(x1); op[m][2] = Wd::hi(x0); op[m][3] = Wd::hi(x1);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint2 q0 = sm.q[0][w][n][lane];
          if (QT == 1) {
#pragma unroll
            for (int m = 0; m < MT; ++m) mma_f16(s[m][n], op[m], q0.x, q0.y);
          } else {
            // 16 elements' products are summed apart: the product unit's sums are not rounded to nearest
            const uint2 q1 = sm.q[1][w][n][lane];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              float y[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16(y, op[m], q1.x, q1.y);
              mma_f16(y, op[m], q0.x, q0.y);
#pragma unroll
              for (int e = 0; e < 4; ++e) s[m][n][e] += y[e];
            }
          }
        }
      }
    }
    // ---- logits (base 2); one beyond its reference moves that
    const float lv = __log2f(fabsf(vs));         // of a block of zeros -inf: never a rise
    const bool whole = tb + STEP <= last;
    float cv[2 * NT], keep_f[2 * NT], raw_s[MT][NT][4];
    bool rise = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float2 rf = *reinterpret_cast<const float2*>(&sm.rowf[8 * n + 2 * t]);
      const float f[2] = {rf.x * ks, rf.y * ks};
      if (QT == 2) { keep_f[2 * n] = f[0]; keep_f[2 * n + 1] = f[1]; }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (QT == 2) raw_s[m][n][e] = s[m][n][e];
          s[m][n][e] = __fmul_rn(s[m][n][e], f[e & 1]);
        }
    }
    if (!whole)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (tb + 16 * m + g + 8 * (e >> 1) >= last) s[m][n][e] = -INFINITY;
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) {
      float most = fmaxf(s[0][i / 2][i % 2], s[0][i / 2][i % 2 + 2]);
#pragma unroll
      for (int m = 1; m < MT; ++m) most = fmaxf(most, fmaxf(s[m][i / 2][i % 2], s[m][i / 2][i % 2 + 2]));
      rise |= most - mo[i] > fminf(0.f, -da[i] - lv);
      cv[i] = vs * F[i];
      rise |= cv[i] > 1e30f;                     // kept finite: a probability of 0 may meet it
    }
    if (a.scores) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = at.row0 + 8 * n + 2 * t + (e & 1), j = tb + 16 * m + g + 8 * (e >> 1);
            if (r < a.rows && j < last) a.scores[(at.bh * a.rows + r) * c.Ncap + j] = s[m][n][e];
          }
    }
    if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = 2 * n + e;
          float top = -INFINITY;
#pragma unroll
          for (int m = 0; m < MT; ++m) top = fmaxf(top, fmaxf(s[m][n][e], s[m][n][e + 2]));
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const bool over = top > mo[i];
          const float m1 = over ? ceilf(top) + kSlack : mo[i], up = over ? m1 - mo[i] : 0.f;
          const float a0 = -da[i] - up, v = top - m1 + lv;     // a, and the tile's largest s + log2(scale), less m1
          // F vs stays below 2^100 and F below 2^115: blocks of tiny values lie at most 2^100 below
          const float a1 = fmaxf(v > a0 ? ceilf(v) + kSlack : a0, fmaxf(-100.f, ceilf(lv) - 80.f));
          mo[i] = m1;
          da[i] = -a1;
          huge |= QT == 2 && fabsf(m1) >= kHuge;
          F[i] = ex2(QT == 1 ? kMost - a1 : kMost - kSlack - a1);
          cv[i] = vs * F[i];
          l[i] *= ex2(-up);
          const float r = ex2(a0 - a1);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) { acc[k][n][e] *= r; acc[k][n][e + 2] *= r; }
        }
      if (QT == 2) huge = __any_sync(0xffffffffu, huge);
    }
    float ref[2 * NT];
    if (QT == 2) {
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i) ref[i] = kSlack - mo[i];
      if (huge)
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) {
          const bool h = fabsf(mo[i]) >= kHuge;
          if (h) { keep_f[i] = 1.f; ref[i] = kSlack; }
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = i % 2; e < 4; e += 2)
              if (h) raw_s[m][i / 2][e] = s[m][i / 2][e] - mo[i];
        }
    }
    // ---- P, and O^T += V^T P^T
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      uint32_t p0[NT][2], p1[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          // fp32: one rounding, of the difference to 2^kSlack below the reference, which is small where p is large
          const int i = 2 * n + (e & 1);
          float x;
          if (QT == 1) x = ex2(s[m][n][e] - mo[i]);
          else if (whole || s[m][n][e] > -INFINITY) x = ex2(fmaf(raw_s[m][n][e], keep_f[i], ref[i]));
          else x = s[m][n][e] == -INFINITY ? 0.f : s[m][n][e];
          l[i] += x;
          w[e] = x * cv[i];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t hi = pack_f16(w[2 * i], w[2 * i + 1]);
          p0[n][i] = transpose8(hi);
          if (QT == 2) {
            const float2 u = unpack_f16(hi);
            p1[n][i] = transpose8(pack_f16((w[2 * i] - u.x) * kLow, (w[2 * i + 1] - u.y) * kLow));
          }
        }
      }
      uint32_t vw[4][VW];
#pragma unroll
      for (int i = 0; i < 4; ++i) read_row<8, D>(vw[i], vt, 16 * m + 2 * t + (i & 1) + 8 * (i >> 1), g);
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        uint32_t u[4], v[4];
        Wd::pairs(Wd::prep(vw[0][w]), Wd::prep(vw[1][w]), u);
        Wd::pairs(Wd::prep(vw[2][w]), Wd::prep(vw[3][w]), v);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t op[4] = {u[2 * e], u[2 * e + 1], v[2 * e], v[2 * e + 1]};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (QT == 1) {
              mma_f16(acc[2 * w + e][n], op, p0[n][0], p0[n][1]);
            } else {
              // as above
              float y[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16(y, op, p1[n][0], p1[n][1]);
#pragma unroll
              for (int i = 0; i < 4; ++i) y[i] *= kLowInv;
              mma_f16(y, op, p0[n][0], p0[n][1]);
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[2 * w + e][n][i] += y[i];
            }
          }
        }
      }
    }
  }
  copy_wait<0>();

  // in units of exp2(m): sums and accumulators
  float m[2 * NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * n + e;
      m[i] = mo[i] > kUnset ? mo[i] : -INFINITY;
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
      // QT 2 summed p 2^kSlack; a power of two less here, as m less kSlack is m again where logits are huge
      const float less = QT == 1 ? 1.f : 0x1p-12f, unit = less / F[i];
      static_assert(kSlack == 12.f, "its power of two");
      l[i] *= less;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) { acc[k][n][e] *= unit; acc[k][n][e + 2] *= unit; }
    }
  join_store<D, NT, MT>(a, sm, at, acc, m, l, [&](int w) { return word_at<8>(D, w, g); });
}

template <int CODE, int D, int NT, int MT, int QT>
__global__ void __launch_bounds__(AT, kv8_ctas_per_sm(D, NT, QT))
kv8_attn_kernel(const __grid_constant__ Kv8AttnArgs a) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem<D, NT, MT>& sm = *reinterpret_cast<Smem<D, NT, MT>*>(smem_raw);
  griddep_wait();
  if ((int)blockIdx.x + a.split0 < a.S) cached_split<CODE, D, NT, MT, QT>(a, sm);
  else if (a.p.win_dtype == LLA_BF16) exact_split<D, NT, MT, QT, 1>(a, sm);
  else exact_split<D, NT, MT, QT, 3>(a, sm);
  if (a.cluster) cluster_join<D, NT, MT>(a, sm);
}

template <int CODE, int D, int NT, int MT, int QT>
cudaError_t launch_split(const Kv8AttnArgs& a, cudaStream_t st) {
  const lla_kv8_cache& c = a.p.cache;
  constexpr size_t smem = sizeof(Smem<D, NT, MT>);
  auto* kern = kv8_attn_kernel<CODE, D, NT, MT, QT>;
  static std::atomic<uint64_t> done{0}, wide_clusters{0};
  cudaError_t e = smem > 48 * 1024 ? allow_smem(kern, smem, done) : cudaSuccess;
  if (e == cudaSuccess && a.cluster > 8)
    e = allow_once(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1, wide_clusters);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(a.ST - a.split0, ceil_div(a.rows, 8 * NT) * c.H, c.B), dim3(AT), smem, st,
                       a.cluster ? a.cluster : 1, a);
}

// the planner chooses nt; a step of two tiles needs blocks of 32 tokens
template <int CODE, int D, int QT>
cudaError_t launch_rows(const Kv8AttnArgs& a, cudaStream_t st) {
  if (a.nt == 1) return launch_split<CODE, D, 1, 1, QT>(a, st);
  if (a.p.cache.block < 32) return launch_split<CODE, D, 2, 1, QT>(a, st);
  if constexpr (D <= 128 && QT == 1)
    if (a.nt == 4) return launch_split<CODE, D, 4, 2, QT>(a, st);
  return launch_split<CODE, D, 2, 2, QT>(a, st);
}

template <int CODE, int QT>
cudaError_t launch_d(const Kv8AttnArgs& a, cudaStream_t st) {
  const int d = a.p.cache.d;
  if (d <= 64) return launch_rows<CODE, 64, QT>(a, st);
  if (d <= 96) return launch_rows<CODE, 96, QT>(a, st);
  if (d <= 128) return launch_rows<CODE, 128, QT>(a, st);
  return launch_rows<CODE, 256, QT>(a, st);
}

}  // namespace kv8
}  // namespace lla
