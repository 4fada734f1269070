// Writer and eviction of the 8-bit K/V cache: codes with one scale per block
// of tokens and head.
#include <cuda_fp8.h>

#include "kernels.cuh"

namespace lla {
namespace {

constexpr int WT = 128;          // threads of the writer

// Largest magnitude as ordered bits: a NaN is above infinity, which is above
// every finite value.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
constexpr uint32_t kInfBits = 0x7f800000u;

__device__ __forceinline__ uint8_t quantise(float x, float s, int code) {
  const float y = x / s;         // fp32 quotient: the codes are a function of x and s alone
  if (code == LLA_KV8_I8) return (uint8_t)(int8_t)fminf(fmaxf(rintf(y), -127.f), 127.f);
  const __nv_fp8_e4m3 c(y);      // nearest-even, saturating to +-448
  return *reinterpret_cast<const uint8_t*>(&c);
}

// One CTA quantises one block of one head of one part: amax over its tokens,
// then the codes.
__global__ void __launch_bounds__(WT) kv8_write_kernel(const lla_kv8_write_params p) {
  griddep_wait();
  const lla_kv8_cache& c = p.cache;
  const int h = blockIdx.y, b = blockIdx.z >> 1, part = blockIdx.z & 1;
  const int n = min(max(kv8_at(p.n, b), 0), p.max_n);
  const int t0 = blockIdx.x * c.block;
  const int64_t src0 = kv8_at(p.src0, b), row0 = kv8_at(p.row0, b);
  const bool fits = row0 >= 0 && row0 % c.block == 0 && row0 + n <= c.Ncap &&
                    (p.ring ? n <= p.rows : src0 >= 0 && src0 + n <= p.rows);
  if (t0 >= n || !fits) return;
  const int m = min(c.block, n - t0);
  const void* x = part ? p.x_v : p.x_k;
  const int64_t xb = (int64_t)b * p.x_stride_b + (int64_t)h * p.x_stride_h;
  auto src = [&](int j) -> int64_t {
    int64_t r = src0 + t0 + j;
    if (p.ring) { r %= p.rows; if (r < 0) r += p.rows; }
    return xb + r * p.x_stride_n;
  };
  uint32_t top = 0;
  for (int e = threadIdx.x; e < m * c.d; e += WT)
    top = max(top, abs_bits(load_elem(x, src(e / c.d) + e % c.d, p.dtype)));
  __shared__ uint32_t tops[WT / 32];
  top = __reduce_max_sync(0xffffffffu, top);
  if (threadIdx.x % 32 == 0) tops[threadIdx.x / 32] = top;
  __syncthreads();
  for (int w = 0; w < WT / 32; ++w) top = max(top, tops[w]);
  const bool bad = top >= kInfBits;
  const float s = bad ? __int_as_float(0x7fc00000) : __uint_as_float(top) / (c.code == LLA_KV8_I8 ? 127.f : 448.f);
  uint8_t* out = static_cast<uint8_t*>(part ? c.v : c.k) + (int64_t)b * c.stride_b + (int64_t)h * c.stride_h +
                 (row0 + t0) * c.d;
  for (int e = threadIdx.x; e < m * c.d; e += WT)
    out[e] = s > 0.f ? quantise(load_elem(x, src(e / c.d) + e % c.d, p.dtype), s, c.code) : 0;
  if (threadIdx.x == 0)
    (part ? c.v_scale : c.k_scale)[(int64_t)b * c.scale_stride_b + (int64_t)h * c.scale_stride_h +
                                   (row0 + t0) / c.block] = s;
}

// ---------------------------------------------------------------- eviction --
constexpr int ST = 256;          // threads of the selection

// Order-preserving map of fp32 to unsigned; NaN is the lowest.
__device__ __forceinline__ uint32_t mass_key(float x) {
  if (x != x) return 0;
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {   // exclusive, ST threads
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[w] = x;
  __syncthreads();
  int before = 0, all = 0;
  for (int i = 0; i < ST / 32; ++i) {
    if (i < w) before += warp_sums[i];
    all += warp_sums[i];
  }
  *total = all;
  return before + x - v;
}

// One CTA chooses the blocks of one head: the sum of each block, then the
// key of the lowest kept sum by four passes of an 8-bit histogram, then an
// ordered scan.
__global__ void __launch_bounds__(ST) kv8_select_kernel(const Kv8EvictArgs a) {
  extern __shared__ uint32_t keys[];        // one per block
  __shared__ int hist[256];
  __shared__ int sums[ST / 32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  griddep_wait();
  const lla_kv8_evict_params& p = a.p;
  const int h = blockIdx.x, b = blockIdx.y, blk = p.src.block;
  const int len = min(max(p.len[b], 0), p.src.Ncap);
  const int nb = (len + blk - 1) / blk;
  int* kept = a.kept + ((int64_t)b * p.src.H + h) * p.keep;
  if (h == 0 && threadIdx.x == 0)
    a.info[b] = make_int2(len, nb <= p.keep ? len : len - (nb - p.keep) * blk);
  if (nb <= p.keep) {
    for (int i = threadIdx.x; i < p.keep; i += ST) kept[i] = i < nb ? i : -1;
    return;
  }
  const float* w = p.weights + (int64_t)b * p.weights_stride_b + (int64_t)h * p.weights_stride_h;
  const int lo = p.first, hi = nb - p.last;  // candidates [lo, hi): all of them whole blocks
  for (int i = lo + threadIdx.x; i < hi; i += ST) {
    double s = 0.0;
    for (int j = 0; j < blk; ++j) s += (double)w[(int64_t)i * blk + j];
    keys[i] = mass_key((float)s);
  }
  if (threadIdx.x == 0) { s_prefix = 0; s_need = p.keep - p.first - p.last; }
  for (int shift = 24; shift >= 0; shift -= 8) {
    hist[threadIdx.x] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix;
    const int need = s_need;
    for (int i = lo + threadIdx.x; i < hi; i += ST)
      if (shift == 24 || (keys[i] ^ prefix) >> (shift + 8) == 0) atomicAdd(&hist[keys[i] >> shift & 255], 1);
    __syncthreads();
    // how many keys lie in higher buckets than this thread's
    int total;
    const int v = hist[255 - threadIdx.x];
    const int above = block_scan(v, sums, &total);
    if (need > 0 && above < need && above + v >= need) {
      s_prefix = prefix | (uint32_t)(255 - threadIdx.x) << shift;
      s_need = need - above;
    }
    __syncthreads();
  }
  const uint32_t edge = s_prefix;
  const int ties = s_need;                  // keys equal to the edge that are kept, the lowest blocks first
  const bool any = p.keep > p.first + p.last;
  int at = 0, tied = 0;
  for (int i0 = 0; i0 < nb; i0 += ST) {
    const int i = i0 + threadIdx.x;
    const bool cand = i >= lo && i < hi;
    const bool tie = any && cand && keys[i] == edge;
    int total;
    const int rank = tied + block_scan(tie, sums, &total);
    tied += total;
    const bool keep = i < nb && (!cand || (any && keys[i] > edge) || (tie && rank < ties));
    const int to = at + block_scan(keep, sums, &total);
    at += total;
    if (keep) kept[to] = i;
  }
}

constexpr int MT = 128;          // threads of the move
constexpr int MU = 8;            // blocks a CTA moves at a time

// One CTA moves one 2 KB slice of every kept block of one head and part; the
// last slice index moves the scales and weights.  Kept blocks stay in order,
// so block i's source is at or after i: a CTA that reads MU blocks before it
// writes them never reads what it has written, and slices share no byte.
__global__ void __launch_bounds__(MT) kv8_move_kernel(const Kv8EvictArgs a, int slices) {
  griddep_wait();
  const lla_kv8_evict_params& p = a.p;
  const int h = blockIdx.y, b = blockIdx.z, blk = p.src.block, d = p.src.d;
  const int* kept = a.kept + ((int64_t)b * p.src.H + h) * p.keep;
  const int2 info = a.info[b];
  const int nk = (info.y + blk - 1) / blk;  // blocks that stay
  if ((int)blockIdx.x < 2 * slices) {
    const int part = blockIdx.x / slices, off = (blockIdx.x % slices) * MT * 16 + threadIdx.x * 16;
    const uint8_t* src = static_cast<const uint8_t*>(part ? p.src.v : p.src.k) + (int64_t)b * p.src.stride_b +
                         (int64_t)h * p.src.stride_h;
    uint8_t* dst = static_cast<uint8_t*>(part ? p.dst.v : p.dst.k) + (int64_t)b * p.dst.stride_b +
                   (int64_t)h * p.dst.stride_h;
    const int64_t unit = (int64_t)blk * d;
    for (int i0 = 0; i0 < nk; i0 += MU) {
      uint4 r[MU];
      bool go[MU];
#pragma unroll
      for (int u = 0; u < MU; ++u) {
        const int i = i0 + u;
        go[u] = false;
        if (i < nk) {
          const int s = kept[i];
          const int64_t bytes = (int64_t)min(blk, info.y - i * blk) * d;
          go[u] = off < bytes && !(a.inplace && s == i);
          if (go[u]) r[u] = *reinterpret_cast<const uint4*>(src + s * unit + off);
        }
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < MU; ++u)
        if (go[u]) *reinterpret_cast<uint4*>(dst + (i0 + u) * unit + off) = r[u];
      __syncthreads();
    }
    return;
  }
  const float* ss[2] = {p.src.k_scale, p.src.v_scale};
  float* ds[2] = {p.dst.k_scale, p.dst.v_scale};
  for (int part = 0; part < 2; ++part) {
    const float* s = ss[part] + (int64_t)b * p.src.scale_stride_b + (int64_t)h * p.src.scale_stride_h;
    float* t = ds[part] + (int64_t)b * p.dst.scale_stride_b + (int64_t)h * p.dst.scale_stride_h;
    for (int i0 = 0; i0 < nk; i0 += MT) {
      const int i = i0 + threadIdx.x;
      const float x = i < nk ? s[kept[i]] : 0.f;
      __syncthreads();
      if (i < nk) t[i] = x;
      __syncthreads();
    }
  }
  const float* w = p.weights + (int64_t)b * p.weights_stride_b + (int64_t)h * p.weights_stride_h;
  float* t = p.dst_weights + (int64_t)b * p.dst_weights_stride_b + (int64_t)h * p.dst_weights_stride_h;
  for (int j0 = 0; j0 < info.y; j0 += MT) {
    const int j = j0 + threadIdx.x;
    const float x = j < info.y ? w[(int64_t)kept[j / blk] * blk + j % blk] : 0.f;
    __syncthreads();
    if (j < info.y) t[j] = x;
    __syncthreads();
  }
  for (int j = info.y + threadIdx.x; j < min(info.x, p.dst.Ncap); j += MT) t[j] = 0.f;
  if (h == 0 && threadIdx.x == 0) p.dst_len[b] = info.y;
}

}  // namespace

cudaError_t launch_kv8_write(const lla_kv8_write_params& p, cudaStream_t st) {
  const dim3 grid(ceil_div(p.max_n, p.cache.block), p.cache.H, 2 * p.cache.B);
  return launch_kernel(kv8_write_kernel, grid, dim3(WT), 0, st, 1, p);
}

cudaError_t launch_kv8_evict(const Kv8EvictArgs& a, cudaStream_t st) {
  const lla_kv8_cache& c = a.p.src;
  const size_t smem = (size_t)(c.Ncap / c.block) * sizeof(uint32_t);
  cudaError_t e = launch_kernel(kv8_select_kernel, dim3(c.H, c.B), dim3(ST), smem, st, 1, a);
  if (e != cudaSuccess) return e;
  const int slices = ceil_div(c.block * c.d, MT * 16);
  return launch_kernel(kv8_move_kernel, dim3(2 * slices + 1, c.H, c.B), dim3(MT), 0, st, 1, a, slices);
}

}  // namespace lla
