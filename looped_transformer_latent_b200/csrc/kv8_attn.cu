// Attention over the 8-bit K/V cache and the exact tokens after it.
#include <cuda_fp8.h>

#include "kernels.cuh"

namespace lla {
namespace {

constexpr int AT = 128;          // threads
constexpr int AW = AT / 32;
constexpr int EPL = 8;           // elements per lane: d <= 256

__device__ __forceinline__ float code_value(uint8_t c, int code) {
  if (code == LLA_KV8_I8) return (float)(int8_t)c;
  const __nv_fp8_storage_t s = c;
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(s, __NV_E4M3)));
}

struct Tokens {                  // what one sequence's rows see
  int len, tail;
  int64_t pos0;                  // position of the oldest exact token
  int ctx;
  __device__ Tokens(const lla_kv8_attn_params& p, int b) {
    len = min(max(kv8_at(p.len, b), 0), p.cache.Ncap);
    tail = 0; ctx = 0; pos0 = 0;
    if (p.win_k) {
      tail = min(max(kv8_at(p.tail, b), 0), p.Wcap);
      ctx = kv8_at(p.ctx, b);
      pos0 = (int64_t)ctx - tail;
    }
  }
  // exact tokens that query position qp of nq sees
  __device__ int visible(int qp, int nq) const { return max(0, min(tail, tail - (nq - 1 - qp))); }
};

__device__ __forceinline__ int slot_of(int64_t pos, int cap) {
  const int64_t r = pos % cap;
  return (int)(r < 0 ? r + cap : r);
}

// One CTA per query row: its warps take tokens in turn with a running maximum
// and sum, joined in shared memory.
__global__ void __launch_bounds__(AT) kv8_attn_row_kernel(const Kv8AttnArgs a) {
  griddep_wait();
  const lla_kv8_attn_params& p = a.p;
  const lla_kv8_cache& c = p.cache;
  const int row = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int qp = row / p.G, g = row % p.G, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const Tokens tk(p, b);
  const int vis = tk.visible(qp, p.nq);
  float q[EPL], acc[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 32 * i;
    q[i] = e < c.d ? a.qmul * load_elem(p.q, (int64_t)b * p.q_stride_b + (int64_t)qp * p.q_stride_n +
                                                 (int64_t)(h * p.G + g) * c.d + e, p.dtype) : 0.f;
    acc[i] = 0.f;
  }
  const int64_t cb = (int64_t)b * c.stride_b + (int64_t)h * c.stride_h;
  const int64_t sb = (int64_t)b * c.scale_stride_b + (int64_t)h * c.scale_stride_h;
  const int64_t wb = (int64_t)b * p.win_stride_b + (int64_t)h * p.win_stride_h;
  float m = -INFINITY, l = 0.f;
  for (int j = w; j < tk.len + vis; j += AW) {
    float k[EPL], v[EPL], s = 0.f;
    const bool cached = j < tk.len;
    const int64_t at = cached ? cb + (int64_t)j * c.d
                              : wb + (int64_t)slot_of(tk.pos0 + (j - tk.len), p.Wcap) * p.win_stride_n;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 32 * i;
      if (e >= c.d) { k[i] = v[i] = 0.f; continue; }
      if (cached) {
        k[i] = code_value(static_cast<const uint8_t*>(c.k)[at + e], c.code);
        v[i] = code_value(static_cast<const uint8_t*>(c.v)[at + e], c.code);
      } else {
        k[i] = load_elem(p.win_k, at + e, p.win_dtype);
        v[i] = load_elem(p.win_v, at + e, p.win_dtype);
      }
      s += q[i] * k[i];
    }
    s = warp_sum(s);
    const float vs = cached ? c.v_scale[sb + j / c.block] : 1.f;
    if (cached) s *= c.k_scale[sb + j / c.block];
    const float mn = s > m ? s : m;
    const float f = m == -INFINITY ? 0.f : exp2f(m - mn), e = exp2f(s - mn);
    l = l * f + e;
#pragma unroll
    for (int i = 0; i < EPL; ++i) acc[i] = acc[i] * f + (e * vs) * v[i];
    m = mn;
  }
  __shared__ float sm[AW], sl[AW], sa[AW][256];
  if (lane == 0) { sm[w] = m; sl[w] = l; }
#pragma unroll
  for (int i = 0; i < EPL; ++i) sa[w][lane + 32 * i] = acc[i];
  __syncthreads();
  float mt = sm[0], lt = 0.f;
  for (int i = 1; i < AW; ++i) mt = fmaxf(mt, sm[i]);
  float f[AW];
  for (int i = 0; i < AW; ++i) {
    f[i] = sm[i] == -INFINITY ? 0.f : exp2f(sm[i] - mt);
    lt += sl[i] * f[i];
  }
  const float inv = lt == 0.f ? 0.f : 1.f / lt;
  for (int e = threadIdx.x; e < c.d; e += AT) {
    float o = 0.f;
    for (int i = 0; i < AW; ++i) o += sa[i][e] * f[i];
    store_elem(p.out, (int64_t)b * p.out_stride_b + (int64_t)qp * p.out_stride_n + (int64_t)(h * p.G + g) * c.d + e,
               p.dtype, o * inv);
  }
  if (a.ml && threadIdx.x == 0) a.ml[((int64_t)b * c.H + h) * a.rows + row] = make_float2(mt, inv);
}

// A warp per cached token: its weight summed over the head's rows in order.
__global__ void __launch_bounds__(AT) kv8_weights_kernel(const Kv8AttnArgs a) {
  griddep_wait();
  const lla_kv8_attn_params& p = a.p;
  const lla_kv8_cache& c = p.cache;
  const int h = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 31;
  const int len = min(max(kv8_at(p.len, b), 0), c.Ncap);
  const float2* ml = a.ml + ((int64_t)b * c.H + h) * a.rows;
  const int64_t cb = (int64_t)b * c.stride_b + (int64_t)h * c.stride_h;
  const int64_t sb = (int64_t)b * c.scale_stride_b + (int64_t)h * c.scale_stride_h;
  for (int j = blockIdx.x * AW + (threadIdx.x >> 5); j < len; j += gridDim.x * AW) {
    float k[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 32 * i;
      k[i] = e < c.d ? code_value(static_cast<const uint8_t*>(c.k)[cb + (int64_t)j * c.d + e], c.code) : 0.f;
    }
    const float ks = c.k_scale[sb + j / c.block];
    float sum = 0.f;
    for (int row = 0; row < a.rows; ++row) {
      const int qp = row / p.G, g = row % p.G;
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = lane + 32 * i;
        if (e < c.d)
          s += a.qmul * load_elem(p.q, (int64_t)b * p.q_stride_b + (int64_t)qp * p.q_stride_n +
                                           (int64_t)(h * p.G + g) * c.d + e, p.dtype) * k[i];
      }
      s = warp_sum(s) * ks;
      sum += exp2f(s - ml[row].x) * ml[row].y;
    }
    if (lane == 0) p.weights[(int64_t)b * p.weights_stride_b + (int64_t)h * p.weights_stride_h + j] += sum;
  }
}

}  // namespace

cudaError_t launch_kv8_attn(const Kv8AttnArgs& a, cudaStream_t st) {
  const lla_kv8_cache& c = a.p.cache;
  cudaError_t e = launch_kernel(kv8_attn_row_kernel, dim3(a.rows, c.H, c.B), dim3(AT), 0, st, 1, a);
  if (e != cudaSuccess || !a.p.weights) return e;
  const int ctas = ceil_div(c.Ncap, AW * 8);
  return launch_kernel(kv8_weights_kernel, dim3(ctas, c.H, c.B), dim3(AT), 0, st, 1, a);
}

}  // namespace lla
