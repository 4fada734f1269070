// Writer and eviction of the 8-bit K/V cache: codes with one scale per block
// of tokens and head.
#include <cuda_fp8.h>

#include <climits>

#include "kernels.cuh"
#include "tc_ptx.cuh"

namespace lla {
namespace {

constexpr uint32_t kInfBits = 0x7f800000u;

// 8 consecutive elements as they come: bf16 in one 16-byte word, fp32 in two.
template <int DT>
struct Vec;
template <>
struct Vec<LLA_BF16> {
  uint4 v;
  __device__ __forceinline__ void load(const void* x, int64_t at) {
    v = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(x) + at));
  }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  // magnitude bits of the largest element, in fp32's places: NaN above infinity above every number
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t m = 0x7fff7fffu;
    const uint32_t a = __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
    return max(a << 16, a & 0xffff0000u);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Vec<LLA_F32> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* x, int64_t at) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
    a = __ldg(p);
    b = __ldg(p + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0, 0, 0, 0); }
  __device__ __forceinline__ uint32_t top() const {
    float f[8];
    get(f);
    uint32_t t = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) t = max(t, __float_as_uint(f[i]) & 0x7fffffffu);
    return t;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);   // nearest-even, +-448
}
__device__ __forceinline__ uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// The codes of 8 elements: fp32 quotients x / s, rounded to nearest-even.  The
// quotient and x * (1 / s) are off by 2^-24 and 2 x 2^-24 relative, so they round to
// the same code unless they lie that near to a boundary between two; only then
// is the division done (it is about ten instructions an element).  `fast`: 1 / s
// is an ordinary number.
template <int CODE>
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float s, float inv, bool fast) {
  bool sure = fast;
  uint2 r;
  if constexpr (CODE == LLA_KV8_I8) {
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = fmaf(x[i], inv, 12582912.f);         // 1.5 x 2^23: the integer in the low bits
      const float off = fmaf(x[i], inv, 12582912.f - t);   // exact to 2^-25
      c[i] = __float_as_uint(t);
      sure = sure && fabsf(off) < 0.49998f;                // |x / s| <= 127: both are off by 127 x 2^-24 = 7.6e-6 at most
    }
    r.x = bytes4(c[0], c[1], c[2], c[3]);
    r.y = bytes4(c[4], c[5], c[6], c[7]);
  } else {
    // a little below and a little above the quotient: 2^-21 covers 3 x 2^-24 and the products' own rounding
    const float lo = inv * (1.f - 0x1p-21f), hi = inv * (1.f + 0x1p-21f);
    uint32_t a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = e4m3_pair(x[2 * i] * lo, x[2 * i + 1] * lo);
      sure = sure && a[i] == e4m3_pair(x[2 * i] * hi, x[2 * i + 1] * hi);
    }
    r.x = a[0] | a[1] << 16;
    r.y = a[2] | a[3] << 16;
  }
  if (!sure) {
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = x[i] / s;
      c[i] = CODE == LLA_KV8_I8 ? (uint32_t)(int)fminf(fmaxf(rintf(q), -127.f), 127.f) : e4m3_pair(q, 0.f);
    }
    r.x = bytes4(c[0], c[1], c[2], c[3]);
    r.y = bytes4(c[4], c[5], c[6], c[7]);
  }
  return r;
}

// One CTA quantises one block of one head of one part.  NV vectors of 8 elements
// a thread stay in registers between the maximum and the codes, so each element
// is read once; NV = 0 reads them again (blocks of more than 16K elements).
// Bound by HBM for fp32 (16384 tokens of 16 heads of 128 to int8: 57 us, 5.9
// TB/s, 90 % of the copy rate) and by instruction issue for bf16 (41 us to int8,
// 48 to e4m3, 4.9 and 4.2 TB/s): e4m3 values of a block whose maximum is 7 times
// a power of two lie on ties often, and those are divided.
template <int CODE, int DT, int T, int NV>
__global__ void __launch_bounds__(T) kv8_write_kernel(const lla_kv8_write_params p) {
  griddep_wait();
  const lla_kv8_cache& c = p.cache;
  const int h = blockIdx.y, b = blockIdx.z >> 1, part = blockIdx.z & 1;
  const int n = min(max(kv8_at(p.n, b), 0), p.max_n);
  const int bshift = 31 - __clz(c.block), t0 = blockIdx.x << bshift;
  if (t0 >= n) return;
  const int src0 = kv8_at(p.src0, b), row0 = kv8_at(p.row0, b);
  // n <= Ncap and n <= rows: the differences do not overflow
  const bool fits = row0 >= 0 && (row0 & (c.block - 1)) == 0 && row0 <= c.Ncap - n &&
                    (p.ring ? n <= p.rows : src0 >= 0 && src0 <= p.rows - n);
  if (!fits) return;
  const uint32_t vpr = c.d >> 3;                           // vectors of a row
  const int nv = min(c.block, n - t0) * vpr;               // and of the block
  const void* x = part ? p.x_v : p.x_k;
  int first = src0 + t0;                                   // source row of the block's first token
  if (p.ring) {
    first = src0 % p.rows;
    if (first < 0) first += p.rows;
    first = (int)(((uint32_t)first + (uint32_t)t0) % (uint32_t)p.rows);
  }
  // threads run through the rows of the block; a ring's rows turn once at most (n <= rows)
  const int64_t xb = (int64_t)b * p.x_stride_b + (int64_t)h * p.x_stride_h + first * p.x_stride_n;
  const int64_t turn = p.ring ? (int64_t)p.rows * p.x_stride_n : 0;
  const int turn_row = p.ring ? p.rows - first : INT_MAX;
  const int row_step = T / vpr, col_step = T % vpr;
  int row = threadIdx.x / vpr, col = threadIdx.x % vpr;
  auto next = [&]() -> int64_t {                           // element offset of the thread's next vector
    const int64_t at = xb + row * p.x_stride_n + 8 * col - (row >= turn_row ? turn : 0);
    row += row_step; col += col_step;
    if (col >= (int)vpr) { col -= vpr; ++row; }
    return at;
  };
  constexpr int HOLD = NV ? NV : 1;
  Vec<DT> v[HOLD];
  uint32_t top = 0;
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t at = next();
      if ((int)threadIdx.x + i * T < nv) v[i].load(x, at);
      else v[i].zero();
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) top = max(top, v[i].top());
  } else {
    for (int i = threadIdx.x; i < nv; i += T) {
      v[0].load(x, next());
      top = max(top, v[0].top());
    }
  }
  __shared__ uint32_t tops[T / 32];
  top = __reduce_max_sync(0xffffffffu, top);
  if (threadIdx.x % 32 == 0) tops[threadIdx.x / 32] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < T / 32; ++w) top = max(top, tops[w]);
  const bool bad = top >= kInfBits;
  const float s = bad ? __int_as_float(0x7fc00000) : __uint_as_float(top) / (CODE == LLA_KV8_I8 ? 127.f : 448.f);
  const float inv = 1.f / s;
  const bool some = s > 0.f, fast = s > 1e-37f;
  uint8_t* out = static_cast<uint8_t*>(part ? c.v : c.k) + (int64_t)b * c.stride_b + (int64_t)h * c.stride_h +
                 (int64_t)(row0 + t0) * c.d;
  auto put = [&](int i, const Vec<DT>& y) {
    float f[8];
    y.get(f);
    const uint2 r = some ? quantise8<CODE>(f, s, inv, fast) : make_uint2(0, 0);
    *reinterpret_cast<uint2*>(out + 8 * (int64_t)i) = r;
  };
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((int)threadIdx.x + i * T < nv) put(threadIdx.x + i * T, v[i]);
  } else {
    row = threadIdx.x / vpr; col = threadIdx.x % vpr;
    for (int i = threadIdx.x; i < nv; i += T) {
      v[0].load(x, next());
      put(i, v[0]);
    }
  }
  if (threadIdx.x == 0)
    (part ? c.v_scale : c.k_scale)[(int64_t)b * c.scale_stride_b + (int64_t)h * c.scale_stride_h +
                                   ((row0 + t0) >> bshift)] = s;
}

template <int CODE, int DT>
cudaError_t launch_write(const lla_kv8_write_params& p, cudaStream_t st) {
  const dim3 grid(ceil_div(p.max_n, p.cache.block), p.cache.H, 2 * p.cache.B);
  const int nv = p.cache.block * p.cache.d / 8;
  if (nv <= 128) return launch_kernel(kv8_write_kernel<CODE, DT, 128, 1>, grid, dim3(128), 0, st, 1, p);
  if (nv <= 256) return launch_kernel(kv8_write_kernel<CODE, DT, 128, 2>, grid, dim3(128), 0, st, 1, p);
  if (nv <= 512) return launch_kernel(kv8_write_kernel<CODE, DT, 128, 4>, grid, dim3(128), 0, st, 1, p);
  if constexpr (DT == LLA_BF16) {
    if (nv <= 1024) return launch_kernel(kv8_write_kernel<CODE, DT, 128, 8>, grid, dim3(128), 0, st, 1, p);
  } else {
    if (nv <= 1024) return launch_kernel(kv8_write_kernel<CODE, DT, 256, 4>, grid, dim3(256), 0, st, 1, p);
  }
  if (nv <= 2048) return launch_kernel(kv8_write_kernel<CODE, DT, 256, 8>, grid, dim3(256), 0, st, 1, p);
  return launch_kernel(kv8_write_kernel<CODE, DT, 256, 0>, grid, dim3(256), 0, st, 1, p);
}

// ---------------------------------------------------------------- eviction --
constexpr int ST = 256;          // threads of a CTA

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

constexpr int EC = 8;            // CTAs that move a head's blocks
constexpr int MU = 8;            // blocks that a thread moves at a time

// What becomes of a sequence.
struct Cut {
  int len, nb, left, nk;         // tokens, blocks; tokens that are left, blocks that stay
  bool cut;
  __device__ Cut(const lla_kv8_evict_params& p, int b) {
    const int blk = p.src.block;
    len = min(max(p.len[b], 0), p.src.Ncap);
    nb = (len + blk - 1) / blk;
    cut = nb > p.keep;
    left = cut ? len - (nb - p.keep) * blk : len;
    nk = cut ? p.keep : nb;
  }
};

// Keys of blocks i, i + step, .. below hi by one warp, four blocks' loads under way at a time.
__device__ __forceinline__ void block_keys(uint32_t* keys, const float* w, int i, int step, int hi, int blk) {
  const int lane = threadIdx.x & 31;
  for (; i < hi; i += 4 * step) {
    double s[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      s[u] = 0.0;
      if (i + u * step < hi)
        for (int k = lane; k < blk; k += 32) s[u] += (double)w[(int64_t)(i + u * step) * blk + k];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int u = 0; u < 4; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], o);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (lane == u && i + u * step < hi) keys[i + u * step] = mass_key((float)s[u]);
  }
}

// One CTA's choice among the candidates [lo, hi) by their keys: the lowest kept
// key by four passes of an 8-bit histogram, then an ordered scan into `list`.
__device__ __forceinline__ void choose_blocks(const lla_kv8_evict_params& p, const uint32_t* keys, int lo, int hi, int nb, int* list) {
  __shared__ int hist[256];
  __shared__ int sums[ST / 32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int tid = threadIdx.x;
  if (tid == 0) { s_prefix = 0; s_need = p.keep - p.first - p.last; }
  __syncthreads();
  for (int shift = 24; shift >= 0; shift -= 8) {
    hist[tid] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix;
    const int need = s_need;
    for (int i = lo + tid; i < hi; i += ST)
      if (shift == 24 || (keys[i] ^ prefix) >> (shift + 8) == 0) atomicAdd(&hist[keys[i] >> shift & 255], 1);
    __syncthreads();
    // how many keys lie in higher buckets than this thread's
    int total;
    const int v = hist[255 - tid];
    const int above = block_scan(v, sums, &total);
    if (need > 0 && above < need && above + v >= need) {
      s_prefix = prefix | (uint32_t)(255 - tid) << shift;
      s_need = need - above;
    }
    __syncthreads();
  }
  const uint32_t edge = s_prefix;
  const int ties = s_need;                     // keys equal to the edge that are kept, the lowest blocks first
  const bool any = p.keep > p.first + p.last;
  int at = 0, tied = 0;
  for (int i0 = 0; i0 < nb; i0 += ST) {
    const int i = i0 + tid;
    const bool cand = i >= lo && i < hi;
    const bool tie = any && cand && keys[i] == edge;
    int total;
    const int place = tied + block_scan(tie, sums, &total);
    tied += total;
    const bool keep = i < nb && (!cand || (any && keys[i] > edge) || (tie && place < ties));
    const int to = at + block_scan(keep, sums, &total);
    at += total;
    if (keep) list[to] = i;
  }
}

// CTA `rank` of EC moves its own share of every kept block's K and V bytes.  Kept
// blocks stay in order, so block i's source is at or after i: in place, a CTA
// that reads a run of blocks before it writes them never reads what it has
// written, and the CTAs' bytes are apart.  Ranks 0 to 2 move the scales and the
// weights, too, which no CTA may still be reading.
__device__ __forceinline__ void move_blocks(const Kv8EvictArgs& a, const Cut& c, int rank, int h, int b, const int* list) {
  const lla_kv8_evict_params& p = a.p;
  const int blk = p.src.block, d = p.src.d, nk = c.nk, left = c.left, len = c.len, tid = threadIdx.x;
  if (a.inplace && !c.cut) return;
  const float* w = p.weights + (int64_t)b * p.weights_stride_b + (int64_t)h * p.weights_stride_h;
  // ---- K and V: the CTA's 16-byte pieces of a block, a thread to each and as many runs of blocks as threads allow
  const int unit = blk * d / 16, all = 2 * unit, p0 = rank * all / EC, p1 = (rank + 1) * all / EC;
  for (int q0 = p0; q0 < p1; q0 += ST) {
    const int pieces = min(ST, p1 - q0), runs = ST / pieces, run = tid / pieces, q = q0 + tid % pieces;
    const bool v = q >= unit;
    const int off = 16 * (v ? q - unit : q);
    const uint8_t* src = static_cast<const uint8_t*>(v ? p.src.v : p.src.k) + (int64_t)b * p.src.stride_b +
                         (int64_t)h * p.src.stride_h + off;
    uint8_t* dst = static_cast<uint8_t*>(v ? p.dst.v : p.dst.k) + (int64_t)b * p.dst.stride_b +
                   (int64_t)h * p.dst.stride_h + off;
    for (int i0 = 0; i0 < nk; i0 += runs * MU) {
      uint4 r[MU];
      bool go[MU];
#pragma unroll
      for (int u = 0; u < MU; ++u) {
        const int i = i0 + run * MU + u;
        go[u] = false;
        if (run < runs && i < nk) {
          const int s = list[i];
          go[u] = off < min(blk, left - i * blk) * d && !(a.inplace && s == i);
          if (go[u]) r[u] = *reinterpret_cast<const uint4*>(src + (int64_t)s * 16 * unit);
        }
      }
      if (a.inplace) __syncthreads();            // all of the run's sources are read; what is written lies before the next's
#pragma unroll
      for (int u = 0; u < MU; ++u)
        if (go[u]) *reinterpret_cast<uint4*>(dst + (int64_t)(i0 + run * MU + u) * 16 * unit) = r[u];
    }
  }
  if (rank < 2) {                                // scales
    const float* s = (rank ? p.src.v_scale : p.src.k_scale) + (int64_t)b * p.src.scale_stride_b + (int64_t)h * p.src.scale_stride_h;
    float* t = (rank ? p.dst.v_scale : p.dst.k_scale) + (int64_t)b * p.dst.scale_stride_b + (int64_t)h * p.dst.scale_stride_h;
    for (int i0 = 0; i0 < nk; i0 += ST) {
      const int i = i0 + tid;
      const float x = i < nk ? s[list[i]] : 0.f;
      __syncthreads();
      if (i < nk) t[i] = x;
      __syncthreads();
    }
  } else if (rank == 2) {                        // weights
    float* t = p.dst_weights + (int64_t)b * p.dst_weights_stride_b + (int64_t)h * p.dst_weights_stride_h;
    constexpr int TU = 4;
    for (int j0 = 0; j0 < left; j0 += TU * ST) {
      float x[TU];
#pragma unroll
      for (int u = 0; u < TU; ++u) {
        const int j = j0 + u * ST + tid;
        x[u] = j < left ? w[(int64_t)list[j / blk] * blk + j % blk] : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < TU; ++u) {
        const int j = j0 + u * ST + tid;
        if (j < left) t[j] = x[u];
      }
      __syncthreads();
    }
    for (int j = left + tid; j < min(len, p.dst.Ncap); j += ST) t[j] = 0.f;
  }
}

// Few heads (16 of 64 blocks of 8 KB, half kept: 11 us, latency): a cluster of EC CTAs evicts from one head in one launch.  Its warps
// sum the blocks' weights in turn, the keys go to all CTAs through the cluster's
// shared memory, and each CTA makes the same choice for itself.
__global__ void __launch_bounds__(ST) kv8_evict_kernel(const Kv8EvictArgs a) {
  extern __shared__ uint32_t keys[];             // one per block, then the list of kept blocks
  griddep_wait();
  const lla_kv8_evict_params& p = a.p;
  const int rank = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, warp = tid >> 5;
  const Cut c(p, b);
  int* list = reinterpret_cast<int*>(keys + p.src.Ncap / p.src.block);
  if (c.cut) {
    const float* w = p.weights + (int64_t)b * p.weights_stride_b + (int64_t)h * p.weights_stride_h;
    const int lo = p.first, hi = c.nb - p.last;  // candidates: all of them whole blocks
    block_keys(keys, w, lo + rank + EC * warp, EC * (ST / 32), hi, p.src.block);
    __syncthreads();
    ptx::cluster_sync_all();
    for (int i = lo + tid; i < hi; i += ST) {
      const int owner = (i - lo) % EC;
      if (owner != rank)
        keys[i] = __float_as_uint(ptx::ld_shared_cluster(ptx::mapa_shared((uint32_t)__cvta_generic_to_shared(keys + i), owner)));
    }
    __syncthreads();
    ptx::cluster_sync_all();                     // all have read: keys may go, weights may move
    choose_blocks(p, keys, lo, hi, c.nb, list);
  } else {
    for (int i = tid; i < c.nb; i += ST) list[i] = i;
  }
  __syncthreads();
  if (rank == 0) {
    if (p.kept)
      for (int i = tid; i < p.keep; i += ST) p.kept[((int64_t)b * p.src.H + h) * p.keep + i] = i < c.nk ? list[i] : -1;
    if (h == 0 && tid == 0 && p.dst_len != p.len) p.dst_len[b] = c.left;
  }
  move_blocks(a, c, rank, h, b, list);
}

// Many heads: a CTA chooses for each, then EC CTAs move each head's blocks.  512
// heads of 64 to 128 blocks of 4 KB, 32 kept: 16 us for the choice (latency of its
// passes), 44 us for the moves (5.6 TB/s, 85 % of the copy rate).
__global__ void __launch_bounds__(ST) kv8_select_kernel(const Kv8EvictArgs a) {
  extern __shared__ uint32_t keys[];
  griddep_wait();
  const lla_kv8_evict_params& p = a.p;
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5;
  const Cut c(p, b);
  int* list = a.kept + ((int64_t)b * p.src.H + h) * p.keep;
  if (c.cut) {
    const float* w = p.weights + (int64_t)b * p.weights_stride_b + (int64_t)h * p.weights_stride_h;
    const int lo = p.first, hi = c.nb - p.last;
    block_keys(keys, w, lo + warp, ST / 32, hi, p.src.block);
    __syncthreads();
    choose_blocks(p, keys, lo, hi, c.nb, list);
  } else {
    for (int i = tid; i < p.keep; i += ST) list[i] = i < c.nb ? i : -1;
  }
}
__global__ void __launch_bounds__(ST) kv8_move_kernel(const Kv8EvictArgs a) {
  griddep_wait();
  const lla_kv8_evict_params& p = a.p;
  const int rank = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const Cut c(p, b);
  if (rank == 0 && h == 0 && threadIdx.x == 0 && p.dst_len != p.len) p.dst_len[b] = c.left;
  move_blocks(a, c, rank, h, b, a.kept + ((int64_t)b * p.src.H + h) * p.keep);
}

// Lengths in place: after every head has read them.
__global__ void kv8_evict_len_kernel(const Kv8EvictArgs a) {
  griddep_wait();
  const int b = blockIdx.x * ST + threadIdx.x;
  if (b < a.p.src.B) a.p.dst_len[b] = Cut(a.p, b).left;
}

}  // namespace

cudaError_t launch_kv8_write(const lla_kv8_write_params& p, cudaStream_t st) {
  if (p.cache.code == LLA_KV8_I8)
    return p.dtype == LLA_BF16 ? launch_write<LLA_KV8_I8, LLA_BF16>(p, st) : launch_write<LLA_KV8_I8, LLA_F32>(p, st);
  return p.dtype == LLA_BF16 ? launch_write<LLA_KV8_E4M3, LLA_BF16>(p, st) : launch_write<LLA_KV8_E4M3, LLA_F32>(p, st);
}

cudaError_t launch_kv8_evict(const Kv8EvictArgs& a, cudaStream_t st) {
  const lla_kv8_cache& c = a.p.src;
  const size_t keys = (size_t)(c.Ncap / c.block) * sizeof(uint32_t), smem = keys + a.p.keep * sizeof(int);
  cudaError_t e = cudaSuccess;
  if (a.fused) {
    static std::atomic<uint64_t> done{0};
    if (smem > 40 * 1024) e = allow_smem(kv8_evict_kernel, 2 * kv8_max_evict_blocks() * sizeof(uint32_t), done);
    if (e == cudaSuccess) e = launch_kernel(kv8_evict_kernel, dim3(EC, c.H, c.B), dim3(ST), smem, st, EC, a);
  } else {
    e = launch_kernel(kv8_select_kernel, dim3(c.H, c.B), dim3(ST), keys, st, 1, a);
    if (e == cudaSuccess) e = launch_kernel(kv8_move_kernel, dim3(EC, c.H, c.B), dim3(ST), 0, st, 1, a);
  }
  if (e != cudaSuccess || a.p.dst_len != a.p.len) return e;
  return launch_kernel(kv8_evict_len_kernel, dim3(ceil_div(c.B, ST)), dim3(ST), 0, st, 1, a);
}

}  // namespace lla
