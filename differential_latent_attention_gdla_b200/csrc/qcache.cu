// qcache.cu -- the 8-bit latent cache: rows quantised as they are written, and read
// back. A cached row is e4m3 with one fp32 scale per block of scale_block tokens.
//
// Write (one pass over the new tokens): with c = gamma (.) c_kv / sqrt(mean(c_kv^2) + eps)
// and k = RoPE(k_rope, position),
//   s   = the smallest power of two >= 2^-40 with max |c|, |k| of the block <= 448 s,
//   row = e4m3([c | k] / s), round to nearest even, once.
// A scale moves by a factor of two where the block's maximum passes 448 2^e. The maximum is
// formed in fp32, to 2^-19; a token whose maximum comes nearer than 2^-16 to such a border
// (one in some 20,000 of normally distributed ones), or is past fp32's range, is looked at
// again in 64 bits, so that the choice does not depend on the order of a sum. Elements are rounded from values that are off by a few 2^-24.
//
// The floor is the bytes: 1152 in and 576 out per bf16 token of the report's sizes, 37 us for
// 131072 tokens; the kernel of many tokens takes 79, see there.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace gdla {
namespace {

// the smallest e with top <= 448 2^e (448 = 1.75 2^8), at least kQcacheMinExp; a top that
// is not positive and finite asks for nothing
__device__ __forceinline__ int scale_exp(double top) {
  if (!(top > 0.0) || !(top < 1e300)) return kQcacheMinExp;
  const unsigned long long u = (unsigned long long)__double_as_longlong(top);
  const int k = (int)(u >> 52) - 1023;
  const int e = (u & 0xFFFFFFFFFFFFFull) <= 0xC000000000000ull ? k - 8 : k - 7;
  return max(e, kQcacheMinExp);
}
__device__ __forceinline__ float exp_to_float(int e) { return __int_as_float((e + 127) << 23); }

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xFFFFu), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// an infinity would saturate to 448: stored as NaN, like every value that is not finite
__device__ __forceinline__ float finite_or_nan(float x) { return fabsf(x) < INFINITY ? x : NAN; }

// eight consecutive inputs of a lane
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = __bfloat1622float2(h[i]);
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    }
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};

template <typename F>
__device__ __forceinline__ F warp_sum(F x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
// the same of an fp32 value that is off by 2^-19 at most, and whether fp32 cannot tell: the
// border is too near (128 steps of 2^-23), or the value is past fp32's range
__device__ __forceinline__ int scale_exp_fast(float top, bool& near) {
  const uint32_t u = __float_as_uint(top);
  near |= u == 0x7F800000u;
  if (u >= 0x7F800000u) return kQcacheMinExp;  // (a NaN asks for nothing)
  const int k = (int)(u >> 23) - 127, m = (int)(u & 0x7FFFFFu) - 0x600000;
  near |= m > -128 && m < 128;
  return max(m <= 0 ? k - 8 : k - 7, kQcacheMinExp);
}

// whether sequence b's new tokens lie inside its cache
__device__ __forceinline__ bool range_ok(const QcacheWriteParams& p, int b) {
  const int n = p.lens ? p.lens[b] : p.L, p0 = p.start ? p.start[b] : 0;
  return n >= 0 && n <= p.L && p0 >= 0 && p0 <= p.T_max && n <= p.T_max - p0;
}

// the exponent that one token asks for, in 64 bits, of its finite values (the whole warp)
template <typename T>
__device__ __forceinline__ int exact_exp(const QcacheWriteParams& p, long long row, int t) {
  const int lane = threadIdx.x & 31, half = p.d_rope >> 1;
  const T* c = reinterpret_cast<const T*>(p.c_kv) + row * p.d_c;
  const T* g = reinterpret_cast<const T*>(p.gamma);
  double ss = 0.0, mx = 0.0, r = 1.0;
#pragma unroll 1
  for (int i = lane; i < p.d_c; i += 32) {
    const double x = (double)to_f(c[i]), v = fabs(g ? x * (double)to_f(g[i]) : x);
    ss = fma(x, x, ss);
    if (v < (double)INFINITY && v > mx) mx = v;
  }
  if (g) {
    // 1/sqrt(m): the fp32 estimate and two Newton steps y (3 - m y^2) / 2 (d_c divides 512)
    const double m = warp_sum(ss) * ((512 / p.d_c) * 0x1p-9) + (double)p.eps;
    r = (double)rsqrtf((float)m);
    if (m < (double)INFINITY) {
      r *= 1.5 - 0.5 * m * r * r;
      r *= 1.5 - 0.5 * m * r * r;
    }
  }
  int e = scale_exp(mx * r);
  if (lane < half) {
    const T* kr = reinterpret_cast<const T*>(p.k_rope) + row * p.d_rope;
    double z1 = (double)to_f(kr[lane]), z2 = (double)to_f(kr[lane + half]);
    if (g) {
      const double cs = (double)p.cos_tab[(long long)t * half + lane], sn = (double)p.sin_tab[(long long)t * half + lane];
      const double w1 = z1 * cs - z2 * sn, w2 = z2 * cs + z1 * sn;
      z1 = w1;
      z2 = w2;
    }
    e = max(e, max(scale_exp(fabs(z1)), scale_exp(fabs(z2))));
  }
  return e;
}

// What a lane holds of a token: NS slots of 8 latents, a pair of the rotary key.
template <typename T, int NS>
struct Token {
  Eight<T> x[NS];
  float k1, k2, cs, sn;  // (not used by the kernel of many tokens)
  __device__ __forceinline__ void load(const QcacheWriteParams& p, long long row, int t, bool on) {
    const int lane = threadIdx.x & 31, half = p.d_rope >> 1;
    const T* c = reinterpret_cast<const T*>(p.c_kv) + row * p.d_c;
    k1 = k2 = sn = 0.f;
    cs = 1.f;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      x[s].zero();
      if (on && (lane + 32 * s) * 8 < p.d_c) x[s].load(c + (lane + 32 * s) * 8);
    }
    if (on && lane < half) {
      const T* kr = reinterpret_cast<const T*>(p.k_rope) + row * p.d_rope;
      k1 = to_f(kr[lane]);
      k2 = to_f(kr[lane + half]);
      if (p.gamma) {
        cs = __ldg(p.cos_tab + (long long)t * half + lane);
        sn = __ldg(p.sin_tab + (long long)t * half + lane);
      }
    }
  }
};
// 1 / rms of the token, its rotated pair, and whether one of the lane's values is infinite
struct Derived {
  float r, y1, y2;
  bool odd;
};

// 1 / sqrt(m) to about an fp32 rounding: the estimate, and a Newton step whose residual
// 1 - m y^2 is formed with the products' rounding errors. (m = inf, from an infinite input or
// squares past the range of fp32: 0, and inf x 0 = NaN.)
__device__ __forceinline__ float inv_sqrt(float m) {
  const float y = rsqrtf(m), t = __fmul_rn(m, y);
  const float e = fmaf(-t, y, 1.f) - fmaf(m, y, -t) * y;
  return m < INFINITY ? fmaf(0.5f * y, e, y) : y;
}
// the rotated pair of (x1, x2), each product with its rounding error
__device__ __forceinline__ float2 rotate(float x1, float x2, float cs, float sn) {
  const float a = __fmul_rn(x1, cs), b = __fmul_rn(x2, sn), c = __fmul_rn(x2, cs), e = __fmul_rn(x1, sn);
  return make_float2(__fadd_rn(__fsub_rn(a, b), __fsub_rn(fmaf(x1, cs, -a), fmaf(x2, sn, -b))),
                     __fadd_rn(__fadd_rn(c, e), __fadd_rn(fmaf(x2, cs, -c), fmaf(x1, sn, -e))));
}

// cs, sn: the lane's angle (1 and 0 without a rotation)
template <typename T, int NS>
__device__ __forceinline__ int derive(const QcacheWriteParams& p, const Token<T, NS>& k, const Eight<T> (&gam)[NS], float x1,
                                      float x2, float cs, float sn, Derived& d, bool& unsure) {
  const bool norm = p.gamma != nullptr;
  float ss = 0.f, mx = 0.f;  // (fmaxf passes over a NaN)
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    float f[8], g[8];
    k.x[s].get(f);
    gam[s].get(g);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      ss = fmaf(f[q], f[q], ss);
      mx = fmaxf(mx, fabsf(norm ? f[q] * g[q] : f[q]));
    }
  }
  d.r = 1.f;
  d.y1 = x1;
  d.y2 = x2;
  if (norm) {
    d.r = inv_sqrt(fmaf(warp_sum(ss), (512 / p.d_c) * 0x1p-9f, p.eps));  // (d_c divides 512)
    const float2 y = rotate(x1, x2, cs, sn);
    d.y1 = y.x;
    d.y2 = y.y;
  }
  // near a border, or an infinity among the values: decided in 64 bits
  const float k_top = fmaxf(fabsf(d.y1), fabsf(d.y2));
  d.odd = mx == INFINITY || k_top == INFINITY;
  unsure = d.odd;
  return scale_exp_fast(fmaxf(mx * d.r, k_top), unsure);
}

// eight stored values before their rounding
template <typename T>
__device__ __forceinline__ void values(const Eight<T>& x, const Eight<T>& gam, bool norm, float r, float inv, float (&f)[8]) {
  float g[8];
  x.get(f);
  gam.get(g);
  const float ri = r * inv;
#pragma unroll
  for (int q = 0; q < 8; ++q) f[q] = finite_or_nan(norm ? (f[q] * g[q]) * ri : f[q] * inv);
}
__device__ __forceinline__ void store_pair(const QcacheWriteParams& p, long long row, int lane, int half, float y1, float y2,
                                           float inv) {
  const uint32_t two = e4m3x4(finite_or_nan(y1) * inv, finite_or_nan(y2) * inv, 0.f, 0.f);
  p.kr8[row * p.d_rope + lane] = (uint8_t)(two & 0xFFu);
  p.kr8[row * p.d_rope + half + lane] = (uint8_t)((two >> 8) & 0xFFu);
}
template <typename T, int NS>
__device__ __forceinline__ void store(const QcacheWriteParams& p, const Token<T, NS>& k, const Eight<T> (&gam)[NS],
                                      const Derived& d, long long row, float inv) {
  const int lane = threadIdx.x & 31, half = p.d_rope >> 1;
  const bool norm = p.gamma != nullptr;
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    if ((lane + 32 * s) * 8 >= p.d_c) continue;
    float f[8];
    values<T>(k.x[s], gam[s], norm, d.r, inv, f);
    *reinterpret_cast<uint2*>(p.c8 + row * p.d_c + (lane + 32 * s) * 8) =
        make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
  }
  if (lane < half) store_pair(p, row, lane, half, d.y1, d.y2, inv);
}
// rows [t0, t1) of a block, which held earlier tokens, to the block's larger scale
__device__ __forceinline__ void bring_rows(const QcacheWriteParams& p, int b, long long t0, int t1, int warp, int n_warps,
                                           float by) {
  const int lane = threadIdx.x & 31;
  for (long long t = t0 + warp; t < t1; t += n_warps) {
    const long long row = (long long)b * p.T_max + t;
    for (int q = lane; q < (p.d_c + p.d_rope) / 16; q += 32) {
      uint4* at = q < p.d_c / 16 ? reinterpret_cast<uint4*>(p.c8 + row * p.d_c) + q
                                 : reinterpret_cast<uint4*>(p.kr8 + row * p.d_rope) + (q - p.d_c / 16);
      uint4 v = *at;
      uint32_t* u = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 a = e4m3x2_to_float2(u[j]), c = e4m3x2_to_float2(u[j] >> 16);
        u[j] = e4m3x4(a.x * by, a.y * by, c.x * by, c.y * by);
      }
      *at = v;
    }
  }
}

// One unit = one block of 2^sl tokens of a sequence, taken by WU = min(2^sl, 16) warps with
// TPW = 2^sl / WU tokens each; a CTA of 8 warps holds 8 / 2^sl units of up to 8 tokens, one
// of 16 warps one unit of 16 .. 128 tokens. NS = 8-element slots of a lane in a latent row.
// Up to 4 tokens of a warp are loaded before any is used and stay in registers until the
// unit's scale is known; KEEP = false (8 tokens) reads them a second time, from L2.
template <typename T, int NS, int TPW, bool KEEP>
__global__ void __launch_bounds__(512, sizeof(T) == 2 && (!KEEP || TPW == 1) ? 2 : 1) qcache_write_kernel(const QcacheWriteParams p) {
  __shared__ int warp_exp[16];
  __shared__ float unit_old[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
  const int b = blockIdx.y;
  const int SB = 1 << p.sl, WU = min(SB, n_warps), UPC = n_warps / WU;
  // the first CTA sets the status word, in the place of a memset in front of the kernel (no other
  // reads it or reports to it)
  if (blockIdx.x == 0 && b == 0) {
    bool bad = false;
    for (int i = threadIdx.x; i < p.B; i += blockDim.x) bad |= !range_ok(p, i);
    bad = __syncthreads_or(bad);
    if (threadIdx.x < kStatusBytes / 4) p.status[threadIdx.x] = threadIdx.x == 0 && bad ? (int)GDLA_ERR_INVALID_ARG : 0;
  }
  if (!range_ok(p, b)) return;
  const int n = p.lens ? p.lens[b] : p.L, p0 = p.start ? p.start[b] : 0;
  const int ul = warp / WU, wi = warp % WU;
  const long long blk = (long long)(p0 >> p.sl) + (long long)blockIdx.x * UPC + ul;
  const long long first = blk << p.sl;
  const int lo = (int)max((long long)p0, first), hi = (int)min((long long)p0 + n, first + SB);
  const bool unit_on = lo < hi;  // (a unit beyond the sequence's tokens does nothing)
  float* scale_at = p.scales + (long long)b * p.n_blocks + blk;
  const long long in0 = (long long)b * p.L - p0;  // + t: the input's row

  constexpr int HELD = KEEP ? TPW : 1;
  Token<T, NS> k[HELD];
  Derived d[HELD];
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      const int t = lo + wi + i * WU;
      k[i].load(p, in0 + t, t, unit_on && t < hi);
    }
  }
  if (unit_on && wi == 0 && lane == 0) unit_old[ul] = first < p0 ? *scale_at : 0.f;
  Eight<T> gam[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    gam[s].zero();
    if (p.gamma && (lane + 32 * s) * 8 < p.d_c)
      gam[s].load(reinterpret_cast<const T*>(p.gamma) + (lane + 32 * s) * 8);
  }
  int exps = kQcacheMinExp;
  uint32_t again = 0;  // tokens to look at again
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      const int t = lo + wi + i * WU;
      const bool on = unit_on && t < hi;
      bool unsure;
      const int e = derive<T, NS>(p, k[i], gam, k[i].k1, k[i].k2, k[i].cs, k[i].sn, d[i], unsure);
      if (on) {
        if (unsure)
          again |= 1u << i;
        else
          exps = max(exps, e);
      }
    }
  } else {
#pragma unroll 2
    for (int i = 0; i < TPW; ++i) {
      const int t = lo + wi + i * WU;
      const bool on = unit_on && t < hi;
      k[0].load(p, in0 + t, t, on);
      bool unsure;
      const int e = derive<T, NS>(p, k[0], gam, k[0].k1, k[0].k2, k[0].cs, k[0].sn, d[0], unsure);
      if (on) {
        if (unsure)
          again |= 1u << i;
        else
          exps = max(exps, e);
      }
    }
  }
  again = __reduce_or_sync(0xffffffffu, again);
#pragma unroll 1
  for (int i = 0; again >> i; ++i) {
    const int t = lo + wi + i * WU;
    if ((again >> i) & 1u) exps = max(exps, exact_exp<T>(p, in0 + t, t));
  }
  exps = __reduce_max_sync(0xffffffffu, exps);
  if (WU > 1) {
    if (lane == 0) warp_exp[warp] = exps;
    __syncthreads();
    for (int w = 0; w < WU; ++w) exps = max(exps, warp_exp[ul * WU + w]);
  } else {
    __syncwarp();
  }
  if (!unit_on) return;
  float scale = exp_to_float(exps);
  // earlier tokens of the block: keep their scale, or bring them to the larger one
  const float old = unit_old[ul];
  if (first < p0 && old > 0.f && old < INFINITY) {
    if (scale <= old) {
      scale = old;
    } else {
      bring_rows(p, b, first, p0, wi, WU, old / scale);
    }
  }
  if (wi == 0 && lane == 0) *scale_at = scale;
  const float inv = 1.f / scale;
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < TPW; ++i) {
      const int t = lo + wi + i * WU;
      if (t < hi) store<T, NS>(p, k[i], gam, d[i], (long long)b * p.T_max + t, inv);
    }
  } else {
#pragma unroll 2
    for (int i = 0; i < TPW; ++i) {
      const int t = lo + wi + i * WU;
      if (t >= hi) break;
      k[0].load(p, in0 + t, t, true);
      bool unsure;
      derive<T, NS>(p, k[0], gam, k[0].k1, k[0].k2, k[0].cs, k[0].sn, d[0], unsure);
      store<T, NS>(p, k[0], gam, d[0], (long long)b * p.T_max + t, inv);
    }
  }
}

// Many bf16 tokens: a CTA takes a chunk of 2^lc tokens (whole blocks). Its latent rows come in
// by one bulk copy and stay in shared memory for both passes, so that few registers are held,
// and a warp takes its tokens four at a time through each step. 131072 tokens, a scale per 64:
// 81 us, the kernel above 110; a scale per token: 76 and 104. Below 16384 tokens the kernel
// above is the faster one (8192: 13 and 11 us), and so it is for fp32 rows (32768 tokens, a
// scale per token: 44 and 38 us) and where a chunk leaves no room for a second one (a scale
// per 128: 109 and 106 us).
constexpr int kBulkTokens = 16384;       // B L from which it is taken
constexpr int kBulkMaxSmem = 100 << 10;  // two chunks an SM
constexpr int kBulkBatch = 4;  // tokens of a warp whose rotary keys are loaded together
template <typename T>
__global__ void __launch_bounds__(512, 2) qcache_write_bulk_kernel(const QcacheWriteParams p, int lc) {
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ uint64_t bar;
  __shared__ int blk_exp[32];
  __shared__ float blk_scale[32];
  __shared__ int odd_any;     // a value of the chunk is infinite
  __shared__ float first_by;  // factor of the first block's earlier rows, 1 if they stay
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int b = blockIdx.y, C = 1 << lc;
  // (the status word is cleared before the kernel: its CTAs' waits read it)
  if (blockIdx.x == 0 && b == 0) {
    bool bad = false;
    for (int i = threadIdx.x; i < p.B; i += blockDim.x) bad |= !range_ok(p, i);
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0 && bad) atomicCAS(p.status, 0, (int)GDLA_ERR_INVALID_ARG);
  }
  if (!range_ok(p, b)) return;
  const int n = p.lens ? p.lens[b] : p.L, p0 = p.start ? p.start[b] : 0;
  const long long first = (long long)((p0 >> lc) + (int)blockIdx.x) << lc;
  const int lo = (int)max((long long)p0, first), hi = (int)min((long long)p0 + n, first + C);
  if (lo >= hi) return;
  const int half = p.d_rope >> 1, es = (int)sizeof(T);
  const bool norm = p.gamma != nullptr;
  const long long in0 = (long long)b * p.L - p0;  // + t: the input's row
  T* xs = reinterpret_cast<T*>(sm);                                           // [C][d_c]
  float2* ys = reinterpret_cast<float2*>(sm + (size_t)C * p.d_c * es);        // [C][half]: rotated pairs
  float* rs = reinterpret_cast<float*>(ys + (size_t)C * half);                // [C]: 1 / rms
  if (threadIdx.x == 0) {
    sm100::mbar_init(sm100::smem_u32(&bar), 1);
    sm100::fence_mbar_init();
    const uint32_t bytes = (uint32_t)(hi - lo) * p.d_c * es;
    sm100::mbar_expect_tx(sm100::smem_u32(&bar), bytes);
    sm100::bulk_load(sm100::smem_u32(xs), reinterpret_cast<const T*>(p.c_kv) + (in0 + lo) * p.d_c, bytes,
                     sm100::smem_u32(&bar));
  }
  const int n_blk = ((hi - 1) >> p.sl) - (lo >> p.sl) + 1, blk0 = lo >> p.sl;
  if (threadIdx.x < 32) blk_exp[threadIdx.x] = kQcacheMinExp;
  if (threadIdx.x == 0) odd_any = 0;
  // 16 consecutive latents of a lane; a gain of 1 and r = 1 where the rows are normalised already
  const bool in_row = lane * 16 < p.d_c;
  float2 gam[8];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    Eight<T> g;
    g.zero();
    if (norm && in_row) g.load(reinterpret_cast<const T*>(p.gamma) + lane * 16 + 8 * s);
    float f[8];
    g.get(f);
#pragma unroll
    for (int q = 0; q < 4; ++q) gam[4 * s + q] = norm ? make_float2(f[2 * q], f[2 * q + 1]) : make_float2(1.f, 1.f);
  }
  auto latents = [&](int i, float2 (&x)[8]) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      Eight<T> v;
      v.zero();
      if (in_row) v.load(xs + (size_t)i * p.d_c + lane * 16 + 8 * s);
      float f[8];
      v.get(f);
#pragma unroll
      for (int q = 0; q < 4; ++q) x[4 * s + q] = make_float2(f[2 * q], f[2 * q + 1]);
    }
  };
  const float inv_dc = (512 / p.d_c) * 0x1p-9f;  // (d_c divides 512)
  const int cnt = hi - lo;
  __syncthreads();
  bool landed = false, failed = false;
  // a warp's tokens four at a time, each step for all four: their latencies overlap
  for (int i0 = warp; i0 < cnt; i0 += nw * kBulkBatch) {
    float k1[kBulkBatch], k2[kBulkBatch], cs[kBulkBatch], sn[kBulkBatch], ss[kBulkBatch], mx[kBulkBatch];
#pragma unroll
    for (int u = 0; u < kBulkBatch; ++u) {
      const int i = min(i0 + u * nw, cnt - 1);  // (the last token again, where there are fewer)
      k1[u] = k2[u] = sn[u] = 0.f;
      cs[u] = 1.f;
      if (lane < half) {
        const T* kr = reinterpret_cast<const T*>(p.k_rope) + (in0 + lo + i) * p.d_rope;
        k1[u] = to_f(kr[lane]);
        k2[u] = to_f(kr[lane + half]);
        if (norm) {
          cs[u] = __ldg(p.cos_tab + (long long)(lo + i) * half + lane);
          sn[u] = __ldg(p.sin_tab + (long long)(lo + i) * half + lane);
        }
      }
    }
    // the first of a warp's rounds waits for the chunk; a warp that gives up looks at none of it
    if (!landed) landed = sm100::mbar_wait(sm100::smem_u32(&bar), 0, p.status, 561);
    if (!__all_sync(0xffffffffu, landed)) {
      failed = true;
      break;
    }
#pragma unroll
    for (int u = 0; u < kBulkBatch; ++u) {
      float2 x[8], s2 = make_float2(0.f, 0.f);
      latents(min(i0 + u * nw, cnt - 1), x);
      mx[u] = 0.f;  // (the maximum passes over a NaN)
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        s2 = sm100::ffma2(x[q], x[q], s2);
        const float2 v = sm100::fmul2(x[q], gam[q]);
        mx[u] = sm100::fmax3(mx[u], fabsf(v.x), fabsf(v.y));
      }
      ss[u] = s2.x + s2.y;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
      for (int u = 0; u < kBulkBatch; ++u) ss[u] += __shfl_xor_sync(0xffffffffu, ss[u], o);
    int e[kBulkBatch];
    uint32_t again = 0;  // tokens near a border or with an infinity: decided in 64 bits
#pragma unroll
    for (int u = 0; u < kBulkBatch; ++u) {
      const float r = norm ? inv_sqrt(fmaf(ss[u], inv_dc, p.eps)) : 1.f;
      const float2 y = norm ? rotate(k1[u], k2[u], cs[u], sn[u]) : make_float2(k1[u], k2[u]);
      const float k_top = fmaxf(fabsf(y.x), fabsf(y.y));
      bool unsure = mx[u] == INFINITY || k_top == INFINITY;
      if (unsure) *reinterpret_cast<volatile int*>(&odd_any) = 1;
      e[u] = scale_exp_fast(fmaxf(mx[u] * r, k_top), unsure);
      if (unsure) again |= 1u << u;
      const int i = i0 + u * nw;
      if (i < cnt) {
        if (lane == 0) rs[i] = r;
        if (lane < half) ys[i * half + lane] = y;
      }
    }
    again = __reduce_or_sync(0xffffffffu, again);
#pragma unroll
    for (int u = 0; u < kBulkBatch; ++u) e[u] = __reduce_max_sync(0xffffffffu, e[u]);
#pragma unroll
    for (int u = 0; u < kBulkBatch; ++u) {
      const int i = i0 + u * nw;
      if (i >= cnt) break;
      if (lane == 0 && !((again >> u) & 1u)) atomicMax(&blk_exp[((lo + i) >> p.sl) - blk0], e[u]);
    }
#pragma unroll 1
    for (int u = 0; again >> u; ++u) {
      const int i = i0 + u * nw;
      if (i >= cnt || !((again >> u) & 1u)) continue;
      const int x = __reduce_max_sync(0xffffffffu, exact_exp<T>(p, in0 + lo + i, lo + i));
      if (lane == 0) atomicMax(&blk_exp[((lo + i) >> p.sl) - blk0], x);
    }
  }
  if (__syncthreads_or(failed)) {  // (reported; nothing is written)
    if (threadIdx.x == 0) sm100::mbar_wait(sm100::smem_u32(&bar), 0, nullptr, 0);  // no copy is in flight at exit
    return;
  }
  if ((int)threadIdx.x < n_blk) {
    float* at = p.scales + (long long)b * p.n_blocks + blk0 + threadIdx.x;
    float scale = exp_to_float(blk_exp[threadIdx.x]), by = 1.f;
    if ((long long)(blk0 + (int)threadIdx.x) << p.sl < p0) {  // (the first block, which holds earlier tokens)
      const float old = *at;
      if (old > 0.f && old < INFINITY) {
        if (scale > old) by = old / scale;
        scale = fmaxf(scale, old);
      }
    }
    *at = blk_scale[threadIdx.x] = scale;
    if (threadIdx.x == 0) first_by = by;
  }
  __syncthreads();
  if (first_by != 1.f) bring_rows(p, b, (long long)blk0 << p.sl, p0, warp, nw, first_by);
  const bool odd = odd_any != 0;
#pragma unroll 2
  for (int i = warp; i < cnt; i += nw) {
    const float inv = 1.f / blk_scale[((lo + i) >> p.sl) - blk0];
    const long long row = (long long)b * p.T_max + lo + i;
    if (in_row) {
      const float ri = rs[i] * inv;
      float2 x[8];
      latents(i, x);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        x[q] = sm100::fmul2(sm100::fmul2(x[q], gam[q]), make_float2(ri, ri));
        if (odd) x[q] = make_float2(finite_or_nan(x[q].x), finite_or_nan(x[q].y));
      }
      *reinterpret_cast<uint4*>(p.c8 + row * p.d_c + lane * 16) =
          make_uint4(e4m3x4(x[0].x, x[0].y, x[1].x, x[1].y), e4m3x4(x[2].x, x[2].y, x[3].x, x[3].y),
                     e4m3x4(x[4].x, x[4].y, x[5].x, x[5].y), e4m3x4(x[6].x, x[6].y, x[7].x, x[7].y));
    }
    if (lane < half) {
      const float2 y = ys[i * half + lane];
      store_pair(p, row, lane, half, y.x, y.y, inv);
    }
  }
}

template <typename T, int NS>
cudaError_t write_ns(const QcacheWriteParams& p, cudaStream_t s) {
  const int SB = 1 << p.sl, warps = SB <= 8 ? 8 : 16, upc = SB <= 8 ? 8 / SB : 1;
  // blocks that L tokens touch, whatever their start
  const long long units = (((long long)p.L + SB - 2) >> p.sl) + 1;
  const dim3 grid((unsigned)((units + upc - 1) / upc), (unsigned)p.B);
  switch (SB <= 16 ? 1 : SB / 16) {
    case 1: qcache_write_kernel<T, NS, 1, true><<<grid, warps * 32, 0, s>>>(p); break;
    case 2: qcache_write_kernel<T, NS, 2, true><<<grid, warps * 32, 0, s>>>(p); break;
    case 4: qcache_write_kernel<T, NS, 4, false><<<grid, warps * 32, 0, s>>>(p); break;
    default: qcache_write_kernel<T, NS, 8, false><<<grid, warps * 32, 0, s>>>(p); break;
  }
  return cudaGetLastError();
}

// chunks of about 40 KB (five CTAs of an SM), or a block where that is larger
cudaError_t write_bulk(const QcacheWriteParams& p, int lc, size_t smem, cudaStream_t s) {
  auto k = qcache_write_bulk_kernel<__nv_bfloat16>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(k, kBulkMaxSmem, allowed);
  if (e == cudaSuccess) e = cudaMemsetAsync(p.status, 0, kStatusBytes, s);
  if (e != cudaSuccess) return e;
  const long long chunks = (((long long)p.L + (1 << lc) - 2) >> lc) + 1;
  k<<<dim3((unsigned)chunks, (unsigned)p.B), smem > (size_t)(60 << 10) ? 512 : 256, smem, s>>>(p, lc);
  return cudaGetLastError();
}
template <typename T>
cudaError_t write_t(const QcacheWriteParams& p, cudaStream_t s) {
  if (sizeof(T) == 2 && (long long)p.B * p.L >= kBulkTokens) {
    const size_t row = (size_t)p.d_c * sizeof(T) + (size_t)p.d_rope * 4 + 4;
    int lc = p.sl > 3 ? p.sl : 3;
    while (lc < 5 && row << (lc + 1) <= (size_t)(44 << 10)) ++lc;
    if (row << lc <= (size_t)kBulkMaxSmem) return write_bulk(p, lc, row << lc, s);
  }
  return p.d_c > 256 ? write_ns<T, 2>(p, s) : write_ns<T, 1>(p, s);
}

// ------------------------------------------------------------------------ read
// A thread turns 16 cached bytes (piece q of a row) into 16 values, in kReadRows rows a block's
// rows apart, all loaded before any is used.
constexpr int kReadRows = 4;
template <typename T>
__global__ void __launch_bounds__(256) qcache_read_kernel(const QcacheReadParams p, int pc, int rpb) {
  const int cc = p.d_c >> 4, b = blockIdx.y;
  const int r = (int)threadIdx.x / pc, q = (int)threadIdx.x % pc;
  if (r >= rpb) return;
  const long long i0 = (long long)blockIdx.x * (rpb * kReadRows) + r;
  const int n = p.lens ? min(max(p.lens[b], 0), p.L) : p.L;
  uint4 v[kReadRows];
  float s[kReadRows];
#pragma unroll
  for (int u = 0; u < kReadRows; ++u) {
    const long long i = i0 + u * rpb;
    v[u] = make_uint4(0, 0, 0, 0);
    s[u] = 0.f;
    if (i < n) {
      const long long row = (long long)b * p.T_max + p.first + i;
      s[u] = __ldg(p.scales + (long long)b * p.n_blocks + ((p.first + i) >> p.sl));
      v[u] = __ldg(q < cc ? reinterpret_cast<const uint4*>(p.c8 + row * p.d_c) + q
                          : reinterpret_cast<const uint4*>(p.kr8 + row * p.d_rope) + (q - cc));
    }
  }
#pragma unroll
  for (int u = 0; u < kReadRows; ++u) {
    const long long i = i0 + u * rpb;
    if (i >= p.L) break;
    float f[16];
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&v[u]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = e4m3x2_to_float2(w[j]), c = e4m3x2_to_float2(w[j] >> 16);
      f[4 * j] = a.x * s[u]; f[4 * j + 1] = a.y * s[u]; f[4 * j + 2] = c.x * s[u]; f[4 * j + 3] = c.y * s[u];
    }
    const long long o = (long long)b * p.L + i;
    T* dst = q < cc ? reinterpret_cast<T*>(p.c_hat) + o * p.d_c + q * 16
                    : reinterpret_cast<T*>(p.k_rope) + o * p.d_rope + (q - cc) * 16;
    if constexpr (sizeof(T) == 2) {
      uint4 h[2];
      __nv_bfloat162* h2 = reinterpret_cast<__nv_bfloat162*>(h);
#pragma unroll
      for (int j = 0; j < 8; ++j) h2[j] = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
      reinterpret_cast<uint4*>(dst)[0] = h[0];
      reinterpret_cast<uint4*>(dst)[1] = h[1];
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        reinterpret_cast<float4*>(dst)[j] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
    }
  }
}

}  // namespace

cudaError_t launch_qcache_write(const QcacheWriteParams& p, gdla_dtype dt, cudaStream_t s) {
  return dt == GDLA_BF16 ? write_t<__nv_bfloat16>(p, s) : write_t<float>(p, s);
}

cudaError_t launch_qcache_read(const QcacheReadParams& p, gdla_dtype dt, cudaStream_t s) {
  const int pc = (p.d_c + p.d_rope) / 16, rpb = 256 / pc;
  const long long per = (long long)rpb * kReadRows;
  const dim3 grid((unsigned)((p.L + per - 1) / per), (unsigned)p.B);
  if (dt == GDLA_BF16)
    qcache_read_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(p, pc, rpb);
  else
    qcache_read_kernel<float><<<grid, 256, 0, s>>>(p, pc, rpb);
  return cudaGetLastError();
}

}  // namespace gdla
