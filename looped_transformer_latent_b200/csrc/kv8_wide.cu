// Attention over the 8-bit K/V cache for many query rows of a head (bf16):
// tcgen05 products with all accumulators in TMEM.
//
//   S [128 lanes x 128 tokens] = q K^T     M = 128
//   O [128 lanes x d]         += P V       M = 128
// K and V codes are widened to f16 once for all rows (exact), by warps that do
// nothing else, into the swizzled layouts that the products read.  A lane is a
// query row and its softmax thread, which keeps the row's maximum and sum in
// registers; nothing is exchanged between threads in the loop.  With 64 rows the
// queries stand in the lanes twice, each copy serves its own half of a tile's
// tokens (its P is zero elsewhere), and the copies are joined at the end like
// splits.  Two groups of four softmax warps
// take tiles in turn, each with its own scores, P and O, so that one's waits
// are the other's work.
// A row's reference is set kSlack above a new maximum; a tile whose logits pass
// it is done again under a new one, twice at most, and the row's accumulators
// are rescaled.
// Bound by the chain from tile to tile, 5800 cycles each with 128 rows: K and V
// have one f16 stage each that the same four warps fill, K of a tile after V of
// the tile before, which waits for that stage's products, and these for the
// softmax (39 % of the issue slots are used, the tensor pipe 18 % of the time).
// Shared memory alone would take 1800 cycles (64 KB of widened codes and 32 KB of
// P written, 128 KB read by the products), the exponentials 1024.  256 heads of 128,
// 4096 e4m3 tokens: 48 rows 149 us, 128 rows 205 (335 TFLOP/s).  A softmax thread
// for each token instead of each row (and rows walked in registers) took 170 and
// 270: it votes on every tile and its sums do not fit registers.
// Every wait is bounded; a CTA that gives up writes NaN.
#include <type_traits>

#include "kernels.cuh"
#include "kv8_math.cuh"
#include "tc_ptx.cuh"

namespace lla {
namespace {

using namespace ptx;
using namespace kv8;

constexpr int TOK = 128;                       // tokens of a tile
constexpr int CHUNK = TOK * 128;               // bytes of 128 rows of 64 f16 elements
constexpr int TILE = 2 * CHUNK;                // K, V, P or q: 128 rows of up to 128 f16 elements
constexpr int RAW = TOK * 128;                 // bytes of a tile's codes, up to 128 a row; two stages of K and V
constexpr int CT = 128;                        // widening threads
// 8 softmax, 4 widening, 2 product warps: an SM quarter's 16K registers go to four warps, 128 for a thread
constexpr int THREADS = 256 + CT + 64, PWARP = 8 + CT / 32;
constexpr uint32_t TMEM_COLS = 512, O_COL = 256;   // two score tiles, two O
constexpr int YP = 132;                        // pitch (floats) of the rows of O in the final join
constexpr long long WAIT_CYCLES = 1ll << 32;   // about 2 s
constexpr float kSlack = 12.f, kUnset = -3.4e38f;
constexpr float kMost = 15.f, kHead = 3.f;     // log2 of the largest P, and of where a new lf puts it
constexpr float kScale = kMost - 90.f;
constexpr float kFar = 65536.f;                // beyond it a difference of references says nothing about a scale

struct Smem {
  uint64_t rawfull[2], kfull, kfree, vfull, vfree, sfull[2], sfree[2], pfull[2], pfree[2], qfull, odone, fin[2];
  uint32_t tmem;
  int abort;
  uint32_t qtop[128];                          // bits of each query row's largest magnitude
};

__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const uint32_t b = smem_u32(bar);
  if (mbar_try_wait(b, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (*abort) return false;
    if (mbar_try_wait(b, parity)) return true;
    if (clock64() - t0 > WAIT_CYCLES) {
      *abort = 1;
      return false;
    }
  }
}

// Two elements at a time, each rounded by itself (never one operation with the next).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{.reg .b64 a, b, r; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; mul.rn.f32x2 r, a, b; mov.b64 {%0, %1}, r;}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{.reg .b64 a, b, r; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %5}; add.rn.f32x2 r, a, b; mov.b64 {%0, %1}, r;}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
// 4 codes to f16, in order (int8: the byte plus 128 in the low bits of 1024, less 1152)
template <int CODE>
__device__ __forceinline__ uint2 widen4(uint32_t w) {
  if constexpr (CODE == LLA_KV8_I8) {
    w ^= 0x80808080u;
    return make_uint2(sub_f16x2(__byte_perm(w, 0x64646464u, 0x4140), 0x64806480u),
                      sub_f16x2(__byte_perm(w, 0x64646464u, 0x4342), 0x64806480u));
  } else {
    return make_uint2(e4m3_f16x2(w), e4m3_f16x2(w >> 16));
  }
}

// Shared memory by its own addresses: the aligned base is no pointer that the
// compiler can tell from a global one.
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// 32 columns of the thread's lane, straight into the registers that are used
// after load_wait, which names them so that nothing touches them before it.
__device__ __forceinline__ void load32(uint32_t at, float (&v)[32]) {
#pragma unroll
  for (int h = 0; h < 32; h += 16)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(v[h]), "=f"(v[h + 1]), "=f"(v[h + 2]), "=f"(v[h + 3]), "=f"(v[h + 4]), "=f"(v[h + 5]), "=f"(v[h + 6]),
          "=f"(v[h + 7]), "=f"(v[h + 8]), "=f"(v[h + 9]), "=f"(v[h + 10]), "=f"(v[h + 11]), "=f"(v[h + 12]),
          "=f"(v[h + 13]), "=f"(v[h + 14]), "=f"(v[h + 15])
        : "r"(at + h));
}
__device__ __forceinline__ void load_wait(float (&v)[32]) {
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3]), "+f"(v[i + 4]), "+f"(v[i + 5]),
                 "+f"(v[i + 6]), "+f"(v[i + 7]));
}

// R: rows of a CTA (64 or 128).  PC: 16-byte pieces of a row of codes.
template <int CODE, int PC, int R>
__global__ void __launch_bounds__(THREADS, 1) kv8_wide_kernel(const __grid_constant__ Kv8AttnArgs a) {
  constexpr int REP = 128 / R;
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_s = base;
  uint8_t* k_s = q_s + TILE;
  uint8_t* v_s = k_s + TILE;
  uint8_t* p_s = v_s + TILE;
  uint8_t* raw_s = p_s + 2 * TILE;
  Smem& bar = *reinterpret_cast<Smem*>(raw_s + 4 * RAW);
  volatile int* abort = &bar.abort;
  griddep_wait();

  const lla_kv8_attn_params& p = a.p;
  const lla_kv8_cache& c = p.cache;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = blockIdx.x, h = blockIdx.y % c.H, row0 = blockIdx.y / c.H * R, b = blockIdx.z;
  const int64_t bh = (int64_t)b * c.H + h;
  const int len = min(max(kv8_at(p.len, b), 0), c.Ncap);
  const int first = split * a.tps, last = min(len, first + a.tps);
  const int rows = min(R, a.rows - row0);
  auto place = [&](int r, int64_t sb, int64_t sn) -> int64_t {
    const int row = a.row0 + row0 + r, qp = row / p.G, gq = row - qp * p.G;
    return (int64_t)b * sb + (int64_t)qp * sn + (int64_t)(h * p.G + gq) * c.d;
  };
  if (first >= last) {
    if (a.direct) {
      for (int i = tid; i < rows * (c.d / 4); i += THREADS)
        store_quad(p.out, place(i / (c.d / 4), p.out_stride_b, p.out_stride_n) + 4 * (i % (c.d / 4)), p.dtype,
                   make_float4(0, 0, 0, 0), 0.f);
    } else if (tid < rows) {
      a.part_ml[(bh * a.rows + row0 + tid) * a.ST + split] = make_float2(-INFINITY, 0.f);
    }
    return;
  }
  const int ntiles = (last - first + TOK - 1) / TOK;
  const int bshift = 31 - __clz(c.block);
  const float* ksc = c.k_scale + (int64_t)b * c.scale_stride_b + (int64_t)h * c.scale_stride_h;
  const float* vsc = c.v_scale + (int64_t)b * c.scale_stride_b + (int64_t)h * c.scale_stride_h;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bar.rawfull[i]), 1);
      mbar_init(smem_u32(&bar.sfull[i]), 1);
      mbar_init(smem_u32(&bar.sfree[i]), 128);
      mbar_init(smem_u32(&bar.pfull[i]), 128);
      mbar_init(smem_u32(&bar.pfree[i]), 1);
      mbar_init(smem_u32(&bar.fin[i]), 1);
    }
    mbar_init(smem_u32(&bar.kfull), CT);
    mbar_init(smem_u32(&bar.kfree), 1);
    mbar_init(smem_u32(&bar.vfull), CT);
    mbar_init(smem_u32(&bar.vfree), 1);
    mbar_init(smem_u32(&bar.qfull), 256);
    mbar_init(smem_u32(&bar.odone), 1);
    fence_mbar_init();
    bar.abort = 0;
  }
  if (tid < R) bar.qtop[tid] = 0;
  if (warp == PWARP) {
    tmem_alloc(smem_u32(&bar.tmem), TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;

  if (warp >= 8 && warp < PWARP) {
    // ------------------------------------------------------- widening warps --
    // A tile's codes are one run of bytes: one bulk copy for K, one for V, two
    // tiles ahead.  A thread widens 8 codes at a time; GU lanes share a row, so
    // that neither the loads (rows d bytes apart) nor the swizzled stores meet in
    // a bank (96: the stores of two rows do).
    constexpr int GU = PC == 8 ? 16 : PC == 4 ? 8 : 4, RPI = CT / GU;
    const int t = tid - 256, u0 = t % GU, r0 = t / GU;
    const int64_t at = (int64_t)b * c.stride_b + (int64_t)h * c.stride_h + (int64_t)first * c.d;
    const uint8_t* kc = static_cast<const uint8_t*>(c.k) + at;
    const uint8_t* vc = static_cast<const uint8_t*>(c.v) + at;
    int issued = 0;
    auto copy = [&](int n) {
      const uint32_t bytes = min(TOK, last - first - n * TOK) * c.d, full = smem_u32(&bar.rawfull[n & 1]);
      mbar_arrive_tx(full, 2 * bytes);
      bulk_load(smem_u32(raw_s + (n & 1) * 2 * RAW), kc + (int64_t)n * TOK * c.d, bytes, full);
      bulk_load(smem_u32(raw_s + (n & 1) * 2 * RAW + RAW), vc + (int64_t)n * TOK * c.d, bytes, full);
      issued = n + 1;
    };
    auto widen = [&](uint32_t from, uint32_t to, int valid) {
#pragma unroll
      for (int g = 0; g < 2 * PC / GU; ++g) {
        const int u = u0 + GU * g;
        if (8 * u < c.d) {
          constexpr int IT = TOK / RPI, HALF = IT > 8 ? 8 : IT;
          const uint32_t src = from + r0 * c.d + 8 * u, dst = to + u / 8 * CHUNK;
#pragma unroll
          for (int i0 = 0; i0 < IT; i0 += HALF) {
            uint2 w[HALF];
#pragma unroll
            for (int i = 0; i < HALF; ++i) w[i] = lds64(src + RPI * (i0 + i) * c.d);
#pragma unroll
            for (int i = 0; i < HALF; ++i) {
              const int r = r0 + RPI * (i0 + i);
              if (r >= valid) w[i] = make_uint2(0, 0);     // rows past the end are zeros
              const uint2 x = widen4<CODE>(w[i].x), y = widen4<CODE>(w[i].y);
              sts128(dst + r * 128 + ((u % 8 ^ (r & 7)) << 4), x.x, x.y, y.x, y.y);
            }
          }
        }
      }
      fence_proxy_async_smem();
    };
    if (t == 0) {
      copy(0);
      if (ntiles > 1) copy(1);
    }
    bool ok = true;
    for (int n = 0; n < ntiles; ++n) {
      const uint32_t from = smem_u32(raw_s) + (n & 1) * 2 * RAW;
      const int valid = last - first - n * TOK;
      ok = ok && wait_bar(&bar.rawfull[n & 1], (n / 2) & 1, abort) && (n == 0 || wait_bar(&bar.kfree, (n - 1) & 1, abort));
      widen(from, smem_u32(k_s), valid);
      mbar_arrive(smem_u32(&bar.kfull));
      ok = ok && (n == 0 || wait_bar(&bar.vfree, (n - 1) & 1, abort));
      widen(from + RAW, smem_u32(v_s), valid);
      mbar_arrive(smem_u32(&bar.vfull));
      __syncwarp();
      if (named_any(2, CT, !ok)) break;
      if (t == 0 && n + 2 < ntiles) copy(n + 2);           // the stage has been read by all
    }
    if (t == 0 && *abort) {                                // copies under way land before the CTA ends
      int never = 0;
      for (int n = max(0, issued - 2); n < issued; ++n) wait_bar(&bar.rawfull[n & 1], (n / 2) & 1, &never);
    }
  } else if (warp >= PWARP) {
    // --------------------------------------------------------- product warps --
    if (lane == 0) {
      bool ok = true;
      const bool scores = warp == PWARP;
      if (scores) {
        const uint32_t id = idesc_f16(128, TOK, false, false);
        const uint64_t qd = smem_desc_sw128(smem_u32(q_s), 16, 1024);
        const int steps = c.d / 16;
        ok = wait_bar(&bar.qfull, 0, abort);
        for (int n = 0; n < ntiles && ok; ++n) {
          const int buf = n & 1;
          ok = wait_bar(&bar.kfull, n & 1, abort) && (n < 2 || wait_bar(&bar.sfree[buf], (n / 2 - 1) & 1, abort));
          if (!ok) break;
          tc_fence_after();
          const uint64_t kd = smem_desc_sw128(smem_u32(k_s), 16, 1024);
          for (int j = 0; j < steps; ++j) {
            const uint64_t off = (uint64_t)((j / 4 * CHUNK + j % 4 * 32) >> 4);
            mma_bf16(tmem + buf * TOK, qd + off, kd + off, id, j > 0);
          }
          mma_commit(smem_u32(&bar.kfree));
          mma_commit(smem_u32(&bar.sfull[buf]));
        }
      } else {
        const uint32_t id = idesc_f16(128, 16 * PC, false, true);
        for (int n = 0; n < ntiles; ++n) {
          const int buf = n & 1;
          ok = wait_bar(&bar.vfull, n & 1, abort) && wait_bar(&bar.pfull[buf], (n / 2) & 1, abort);
          if (!ok) break;
          tc_fence_after();
          const uint64_t pd = smem_desc_sw128(smem_u32(p_s) + buf * TILE, 16, 1024);
          const uint64_t vd = smem_desc_sw128(smem_u32(v_s), CHUNK, 1024);
#pragma unroll
          for (int j = 0; j < TOK / 16; ++j)
            mma_bf16(tmem + O_COL + buf * 128, pd + (uint64_t)((j / 4 * CHUNK + j % 4 * 32) >> 4), vd + 128 * j, id,
                     n > 1 || j > 0);
          mma_commit(smem_u32(&bar.vfree));
          mma_commit(smem_u32(&bar.pfree[buf]));
        }
        if (ok) mma_commit(smem_u32(&bar.odone));
      }
      if (!ok) {
        // every product issued must end before TMEM is freed
        int never = 0;
        mma_commit(smem_u32(&bar.fin[scores]));
        wait_bar(&bar.fin[scores], 0, &never);
      }
    }
  } else {
    // --------------------------------------------------------- softmax warps --
    const int wg = warp / 4, q4 = warp & 3, at128 = 32 * q4 + lane;   // group, TMEM lane
    const int row = at128 % R, c0 = at128 / R * R;                    // row, first of its R tokens of a tile
    const uint32_t lanes = (uint32_t)(32 * q4) << 16;
    const uint32_t s_at = tmem + wg * TOK + c0 + lanes, o_at = tmem + O_COL + wg * 128 + lanes;
    // ---- queries to f16 under a power of two per row that puts the row's largest magnitude into [2^13, 2^14): each row
    // keeps its bits whatever the others hold, and a row that is no number is its own
    auto exponent = [](uint32_t top) {           // of a row; 0 where it is zero or no number
      return top > 0 && top < 0x7f800000u ? max((int)(top >> 23) - 127 - 13, -100) : 0;
    };
    {
      constexpr int ALL = R * PC * 2, UNITS = (ALL + 255) / 256;    // pieces of 8 elements
      uint4 u[UNITS];
#pragma unroll
      for (int i = 0; i < UNITS; ++i) {
        const int id = tid + 256 * i, r = id / (PC * 2), e = 8 * (id % (PC * 2));
        u[i] = id < ALL && r < rows && e < c.d ? __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                                          place(r, p.q_stride_b, p.q_stride_n) + e))
                                   : make_uint4(0, 0, 0, 0);
      }
      if (REP > 1)                               // P outside a copy's own tokens
        for (int i = tid; i < 2 * TILE / 16; i += 256) reinterpret_cast<uint4*>(p_s)[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < UNITS; ++i) {
        const uint32_t m = 0x7fff7fffu;
        const uint32_t w = __vmaxu2(__vmaxu2(u[i].x & m, u[i].y & m), __vmaxu2(u[i].z & m, u[i].w & m));
        if (w) atomicMax(&bar.qtop[(tid + 256 * i) / (PC * 2)], max(w << 16, w & 0xffff0000u));
      }
      named_sync(1, 256);
#pragma unroll
      for (int i = 0; i < UNITS; ++i) {
        const int id = tid + 256 * i, r = id / (PC * 2), k = id % (PC * 2);
        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
        if (id >= ALL) break;
        const float down = pow2(-exponent(bar.qtop[r]));
        uint32_t o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          o[q] = pack_f16(__uint_as_float(w[q] << 16) * down, __uint_as_float(w[q] & 0xffff0000u) * down);
#pragma unroll
        for (int y = 0; y < REP; ++y)            // r + R y: the same residue mod 8
          *reinterpret_cast<uint4*>(q_s + k / 8 * CHUNK + (r + R * y) * 128 + ((k % 8 ^ (r & 7)) << 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
      }
      fence_proxy_async_smem();
      mbar_arrive(smem_u32(&bar.qfull));
    }
    const float rowf = a.qmul * pow2(exponent(bar.qtop[row]));
    // Probabilities p = exp2(s - m) <= 1 meet the codes times scale * F, F = 2^lf of the row: w = exp2(s + log2 scale - m
    // + lf) <= 2^15 in f16, and the largest of them above 2^2 when lf is set, so that what f16 leaves out of the small
    // ones (below 2^-24) stays 26 bits below the largest, whatever block that lies in.  References are whole numbers,
    // so that moving one is exact; lf is kept by itself, so that it means the same however large the logits are.
    float m = kUnset, lf = 0.f, l = 0.f;        // reference, log2 F, sum
    bool ok = true;
    {
      // lanes 0-7 hold the K scales of a tile's groups of 16 tokens, 8-15 the V scales; read a turn ahead
      const float* sc = lane & 8 ? vsc : ksc;
      auto scale_of = [&](int n) { return __ldg(sc + (min(first + n * TOK + 16 * (lane & 7), last - 1) >> bshift)); };
      float ahead = wg < ntiles ? scale_of(wg) : 0.f;
      for (int n = wg; n < ntiles; n += 2) {
        const float scales = ahead;
        if (n + 2 < ntiles) ahead = scale_of(n + 2);
        const int j0 = first + n * TOK + c0;     // the thread's first token
        const bool whole = first + (n + 1) * TOK <= last;
        ok = ok && wait_bar(&bar.sfull[wg], (n / 2) & 1, abort);
        ok = ok && (n < 2 || wait_bar(&bar.pfree[wg], (n / 2 - 1) & 1, abort));   // P and O of the turn before are done
        __syncwarp();
        tc_fence_after();
        const uint32_t prow = smem_u32(p_s) + wg * TILE + at128 * 128;
        // one turn over the tile's 32-token groups, the next one's scores on their way; MAX: only the maxima (under
        // m = 0); ALL: every token is there.  top: the largest logit; atop: the largest logit + log2 scale, less m
        auto turn = [&](auto only_max, auto all, float& top, float& atop, float& sum) {
          constexpr bool MAX = decltype(only_max)::value, ALL = decltype(all)::value;
          const float F = ex2(lf);
          auto group = [&](int g, float (&x)[32]) {
#pragma unroll
            for (int hf = 0; hf < 32; hf += 16) {
              const int grp = (c0 + g + hf) / 16;
              const float f = __shfl_sync(0xffffffffu, scales, grp) * rowf, vs = __shfl_sync(0xffffffffu, scales, grp + 8);
              float t[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                // rounded, and not summed with m in one: no logit passes a reference above the largest
                float2 y = mul2(make_float2(x[hf + i], x[hf + i + 1]), make_float2(f, f));
                if (!ALL && j0 + g + hf + i >= last) y.x = -INFINITY;
                if (!ALL && j0 + g + hf + i + 1 >= last) y.y = -INFINITY;
                x[hf + i] = y.x; x[hf + i + 1] = y.y;
                t[i & 2] = fmaxf(t[i & 2], y.x); t[i & 2 | 1] = fmaxf(t[i & 2 | 1], y.y);
              }
              const float most = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
              top = fmaxf(top, most);
              // kScale: scale * F stays below 2^90, as a probability of 0 may meet it
              atop = fmaxf(atop, (MAX ? most : fmaxf(most - m, kScale)) + __log2f(fabsf(vs)));
              if (MAX) continue;
              if (a.scores && row < rows) {
                float* to = a.scores + (bh * a.rows + row0 + row) * c.Ncap + j0 + g + hf;
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  if (ALL || j0 + g + hf + i < last) to[i] = x[hf + i];
              }
              const float vF = vs * F;
#pragma unroll
              for (int i = 0; i < 16; i += 8) {
                float w[8], part[2] = {0.f, 0.f};
#pragma unroll
                for (int k = 0; k < 8; k += 2) {
                  const float2 y = make_float2(x[hf + i + k], x[hf + i + k + 1]), s = add2(y, make_float2(-m, -m));
                  const float2 e = make_float2(ex2(s.x), ex2(s.y)), v = mul2(e, make_float2(vF, vF));
                  part[0] += e.x; part[1] += e.y;
                  w[k] = ALL || y.x != -INFINITY ? v.x : 0.f;    // a scale that is no number meets no absent token
                  w[k + 1] = ALL || y.y != -INFINITY ? v.y : 0.f;
                }
                sum += part[0] + part[1];
                const int tk = c0 + g + hf + i;
                sts128(prow + tk / 64 * CHUNK + ((tk % 64 / 8 ^ (at128 & 7)) << 4), pack_f16(w[0], w[1]),
                       pack_f16(w[2], w[3]), pack_f16(w[4], w[5]), pack_f16(w[6], w[7]));
              }
            }
          };
          float x[32], z[32];
          load32(s_at, x);
          load_wait(x);
#pragma unroll 1
          for (int g = 0; g < R; g += 64) {
            load32(s_at + g + 32, z);
            group(g, x);
            load_wait(z);
            if (g + 64 < R) load32(s_at + g + 64, x);
            group(g + 32, z);
            if (g + 64 < R) load_wait(x);
          }
        };
        if (n == wg) {                           // the first turn sets the references
          float top = -INFINITY, atop = -INFINITY, none = 0.f;
          if (whole) turn(std::true_type{}, std::true_type{}, top, atop, none);
          else turn(std::true_type{}, std::false_type{}, top, atop, none);
          if (top > -INFINITY) {
            m = ceilf(top) + kSlack;
            lf = fabsf(m) < kFar ? fminf(kHead + m - ceilf(atop), 100.f) : 100.f;
          }
        }
        // At most two more turns: no logit passes the first new m, and under that atop is exact, so that the next lf
        // holds.  Where m went up far, atop says nothing yet: lf takes its largest value, which the next turn sees.
        for (int again = 2;; --again) {
          float top = -INFINITY, atop = -INFINITY, sum = l;
          if (whole) turn(std::false_type{}, std::true_type{}, top, atop, sum);
          else turn(std::false_type{}, std::false_type{}, top, atop, sum);
          if (!__any_sync(0xffffffffu, top > m || atop + lf > kMost) || again == 0) {
            l = sum;
            break;
          }
          const float m1 = top > m ? ceilf(top) + kSlack : m, up = m1 - m;
          const float l1 = fminf(up < kFar ? (atop + lf > kMost ? kHead - ceilf(atop - up) : lf + up) : 100.f, 100.f);
          const float r = ex2(l1 - lf - up);
          l *= ex2(-up);
          m = m1;
          lf = l1;
          if (n > 1) {
#pragma unroll 1
            for (int i = 0; i < 16 * PC; i += 16) {
              float y[16];
              tmem_ld16(o_at + i, y);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) y[k] *= r;
              tmem_st16(o_at + i, y);
            }
            tmem_wait_st();
          }
        }
        tc_fence_before();
        mbar_arrive(smem_u32(&bar.sfree[wg]));
        fence_proxy_async_smem();
        mbar_arrive(smem_u32(&bar.pfull[wg]));
      }
    }
    ok = ok && wait_bar(&bar.odone, 0, abort);
    __syncwarp();
    tc_fence_after();
    // ---- join of the groups and copies through shared memory (the tiles are done with)
    float* y_s = reinterpret_cast<float*>(k_s);          // [2][128][YP], then m and l of the 256 lanes
    float2* ml_s = reinterpret_cast<float2*>(y_s + 256 * YP);
    const bool some = wg < ntiles && m > kUnset;
    const float unit = some ? ex2(-lf) : 0.f;
    float* mine = y_s + tid * YP;
#pragma unroll 1
    for (int i = 0; i < 16 * PC; i += 16) {
      float y[16];
      tmem_ld16(o_at + i, y);
      tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < 16; k += 4)
        *reinterpret_cast<float4*>(mine + i + k) =
            some ? make_float4(y[k] * unit, y[k + 1] * unit, y[k + 2] * unit, y[k + 3] * unit) : make_float4(0, 0, 0, 0);
    }
    tc_fence_before();
    ml_s[tid] = make_float2(some ? m : -INFINITY, ok ? l : __int_as_float(0x7fc00000));
    named_sync(1, 256);
    for (int i = tid; i < rows * (c.d / 4); i += 256) {
      const int r = i / (c.d / 4), e = 4 * (i % (c.d / 4));
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int k = 0; k < 2 * REP; ++k) top = fmaxf(top, ml_s[r + R * k].x);
      const float z = top == -INFINITY ? 0.f : top;
      float4 s = make_float4(0, 0, 0, 0);
#pragma unroll
      for (int k = 0; k < 2 * REP; ++k) {
        const float2 x = ml_s[r + R * k];
        const float g = ex2(x.x - z);
        sum += g * x.y;
        const float4 v = *reinterpret_cast<const float4*>(y_s + (r + R * k) * YP + e);
        s.x += g * v.x; s.y += g * v.y; s.z += g * v.z; s.w += g * v.w;
      }
      if (a.direct) {
        store_quad(p.out, place(r, p.out_stride_b, p.out_stride_n) + e, p.dtype, s, sum == 0.f ? 0.f : 1.f / sum);
      } else {
        const int64_t at = (bh * a.rows + row0 + r) * a.ST + split;
        if (e == 0) a.part_ml[at] = make_float2(top, sum);
        *reinterpret_cast<float4*>(a.part_y + at * c.d + e) = s;
      }
    }
  }
  __syncthreads();
  if (warp == PWARP) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

template <int CODE, int PC, int R>
cudaError_t launch_wide(const Kv8AttnArgs& a, cudaStream_t st) {
  constexpr size_t smem = 1024 + 5 * TILE + 4 * RAW + sizeof(Smem);
  static_assert(smem <= 227 * 1024, "one CTA to an SM");
  static_assert(256 * (YP * sizeof(float) + sizeof(float2)) <= 4 * TILE + 4 * RAW, "the join fits the tiles");
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(kv8_wide_kernel<CODE, PC, R>, smem, done);
  if (e != cudaSuccess) return e;
  return launch_kernel(kv8_wide_kernel<CODE, PC, R>, dim3(a.S, ceil_div(a.rows, R) * a.p.cache.H, a.p.cache.B),
                       dim3(THREADS), smem, st, 1, a);
}

template <int CODE, int PC>
cudaError_t launch_r(const Kv8AttnArgs& a, cudaStream_t st) {
  return a.wide == 64 ? launch_wide<CODE, PC, 64>(a, st) : launch_wide<CODE, PC, 128>(a, st);
}

template <int CODE>
cudaError_t launch_pieces(const Kv8AttnArgs& a, cudaStream_t st) {
  const int d = a.p.cache.d;
  return d <= 64 ? launch_r<CODE, 4>(a, st) : d <= 96 ? launch_r<CODE, 6>(a, st) : launch_r<CODE, 8>(a, st);
}

}  // namespace

cudaError_t launch_kv8_wide(const Kv8AttnArgs& a, cudaStream_t st) {
  return a.p.cache.code == LLA_KV8_I8 ? launch_pieces<LLA_KV8_I8>(a, st) : launch_pieces<LLA_KV8_E4M3>(a, st);
}

}  // namespace lla
