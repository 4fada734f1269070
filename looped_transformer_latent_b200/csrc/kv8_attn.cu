// Attention over the 8-bit K/V cache: join of the splits, weights, launches.
#include "kernels.cuh"
#include "tc_ptx.cuh"

namespace lla {
namespace {

constexpr int AT = 128;          // threads
constexpr int AW = AT / 32;

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

// Sum of a row's splits [i0, ST) in steps of `step`, by one warp; a lane holds 4 elements.
// Loads of 8 splits are under way at a time; an empty split's y is not there.
__device__ __forceinline__ float4 row_sum(const float2* ml, const float* y, int ST, int d, int e, float m, int i0, int step) {
  const int lane = threadIdx.x & 31;
  float4 s = make_float4(0, 0, 0, 0);
  for (int base = i0; base < ST; base += 32 * step) {
    const int mine = base + lane * step;
    const float2 x = mine < ST ? ml[mine] : make_float2(-INFINITY, 0.f);
    const bool there = !(x.x == -INFINITY && x.y == 0.f);
    const float f = there ? exp2f(x.x - m) : 0.f;
    const unsigned some = __ballot_sync(0xffffffffu, there);
    const int n = min(32, (ST - base + step - 1) / step);
    for (int k0 = 0; k0 < n; k0 += 8) {
      float4 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        v[k] = e < d && (some >> (k0 + k) & 1) ? *reinterpret_cast<const float4*>(y + (int64_t)(base + (k0 + k) * step) * d + e)
                                               : make_float4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float g = __shfl_sync(0xffffffffu, f, k0 + k);
        s.x += g * v[k].x; s.y += g * v[k].y; s.z += g * v[k].z; s.w += g * v[k].w;
      }
    }
  }
  return s;
}

// 8 x 16 heads, 16384 tokens, one row: 12 us with the weights (scores read, weights
// read and written: 25 MB, 2.1 TB/s: latency; 15 us with the weights' loads last), 4 us without.
// CTAs below `joins` write the outputs, a warp (a.wide: a CTA) for each row;
// the others add a stretch of the head's weights: each token's terms over the
// rows in order.
__global__ void __launch_bounds__(AT) kv8_join_kernel(const __grid_constant__ Kv8AttnArgs a, int joins, int wide) {
  __shared__ float2 sml[32];
  __shared__ float4 sy[AW][64];
  griddep_wait();
  const lla_kv8_attn_params& p = a.p;
  const lla_kv8_cache& c = p.cache;
  const int h = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t bh = (int64_t)b * c.H + h;
  if ((int)blockIdx.x < joins) {
    const int r = wide ? blockIdx.x : blockIdx.x * AW + warp;
    if (r >= a.rows) return;
    const float2* ml = a.part_ml + (bh * a.rows + r) * a.ST;
    const float2 all = row_ml(ml, a.ST);
    const float* y = a.part_y + (bh * a.rows + r) * a.ST * c.d;
    const int row = a.row0 + r, qp = row / p.G, gq = row % p.G;
    const int64_t o = (int64_t)b * p.out_stride_b + (int64_t)qp * p.out_stride_n + (int64_t)(h * p.G + gq) * c.d;
    for (int e0 = 0; e0 < c.d; e0 += 128) {
      const int e = e0 + 4 * lane;
      float4 s = row_sum(ml, y, a.ST, c.d, e, all.x, wide ? warp : 0, wide ? AW : 1);
      if (wide) sy[warp][e / 4] = s;
      else if (e < c.d) store_quad(p.out, o + e, p.dtype, s, all.y);
    }
    if (!wide) return;
    __syncthreads();
    const int e = 4 * threadIdx.x;
    if (e < c.d) {
      float4 s = sy[0][e / 4];
#pragma unroll
      for (int w = 1; w < AW; ++w) {
        const float4 v = sy[w][e / 4];
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
      }
      store_quad(p.out, o + e, p.dtype, s, all.y);
    }
    return;
  }
  const int len = min(max(kv8_at(p.len, b), 0), c.Ncap), j0 = (blockIdx.x - joins) * JT;
  if (j0 >= len) return;
  float* w = p.weights + (int64_t)b * p.weights_stride_b + (int64_t)h * p.weights_stride_h;
  float sum[JT / AT], was[JT / AT];              // the weights' loads go out before the splits' and the scores'
#pragma unroll
  for (int i = 0; i < JT / AT; ++i) {
    const int j = j0 + threadIdx.x + AT * i;
    sum[i] = 0.f;
    was[i] = j < len ? w[j] : 0.f;
  }
  for (int r0 = 0; r0 < a.rows; r0 += 32) {
    const int n = min(32, a.rows - r0);
    __syncthreads();
    for (int r = warp; r < n; r += AW) {
      const float2 x = row_ml(a.part_ml + (bh * a.rows + r0 + r) * a.ST, a.ST);
      if (lane == 0) sml[r] = x;
    }
    __syncthreads();
    // four rows' scores under way at a time; each token's terms are added in the rows' order
    for (int r = 0; r < n; r += 4) {
      const float* s = a.scores + (bh * a.rows + r0 + r) * c.Ncap;
      float x[4][JT / AT];
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < JT / AT; ++i) {
          const int j = j0 + threadIdx.x + AT * i;
          x[k][i] = r + k < n && j < len ? s[(int64_t)k * c.Ncap + j] : -INFINITY;
        }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (r + k >= n) break;
#pragma unroll
        for (int i = 0; i < JT / AT; ++i) sum[i] += ptx::ex2(x[k][i] - sml[r + k].x) * sml[r + k].y;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < JT / AT; ++i) {
    const int j = j0 + threadIdx.x + AT * i;
    if (j < len) w[j] = was[i] + sum[i];
  }
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
    if (a.wide && a.S) {
      e = launch_kv8_wide(a, st);
      a.split0 = a.S;
    }
    if (e == cudaSuccess && a.ST > a.split0) {
      const bool f32 = a.p.dtype == LLA_F32;
      if (c.code == LLA_KV8_I8) e = f32 ? launch_kv8_attn_i8_f32(a, st) : launch_kv8_attn_i8_bf16(a, st);
      else e = f32 ? launch_kv8_attn_e4m3_f32(a, st) : launch_kv8_attn_e4m3_bf16(a, st);
    }
    if (e != cudaSuccess) return e;
    if (a.direct || a.cluster) continue;
    const int wide = a.ST >= 8;                  // many splits: a CTA for each row shortens the chain of loads
    const int joins = wide ? a.rows : ceil_div(a.rows, AW);
    e = launch_kernel(kv8_join_kernel, dim3(joins + (a.p.weights ? ceil_div(c.Ncap, JT) : 0), c.H, c.B), dim3(AT), 0, st,
                      1, a, joins, wide);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace lla
