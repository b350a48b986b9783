// qcache.cu -- the 8-bit latent cache: rows quantised as they are written, and read
// back. A cached row is e4m3 with one fp32 scale per block of scale_block tokens.
//
// Write (one pass over the new tokens): with c = gamma (.) c_kv / sqrt(mean(c_kv^2) + eps)
// and k = RoPE(k_rope, position),
//   s   = the smallest power of two >= 2^-40 with max |c|, |k| of the block <= 448 s,
//   row = e4m3([c | k] / s), round to nearest even, once.
// A scale moves by a factor of two where the block's maximum passes 448 2^e, so the
// maximum is compared with that border in 64-bit arithmetic (the sum of squares exact to
// ~2^-45, the maximum of |gamma c| exact, one product): the choice does not depend on the
// order of a sum. Elements are rounded from values correct to an fp32 rounding.
//
// Bound by the bytes: 1152 in and 576 out per bf16 token of the report's sizes.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

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

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// whether sequence b's new tokens lie inside its cache
__device__ __forceinline__ bool range_ok(const QcacheWriteParams& p, int b) {
  const int n = p.lens ? p.lens[b] : p.L, p0 = p.start ? p.start[b] : 0;
  return n >= 0 && n <= p.L && p0 >= 0 && p0 <= p.T_max && n <= p.T_max - p0;
}

// One unit = one block of 2^sl tokens of a sequence, taken by WU = min(2^sl, 16) warps with
// TPW = 2^sl / WU tokens each; a CTA of 8 warps holds 8 / 2^sl units of up to 8 tokens, one
// of 16 warps one unit of 16 .. 128 tokens. NS = 8-element slots of a lane in a latent row.
// The inputs of all of a warp's tokens are loaded before any is used, and stay in registers
// until the unit's scale is known.
template <typename T, int NS, int TPW>
__global__ void __launch_bounds__(512) qcache_write_kernel(const QcacheWriteParams p) {
  __shared__ int warp_exp[16];
  __shared__ float unit_old[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
  const int b = blockIdx.y;
  const int SB = 1 << p.sl, WU = min(SB, n_warps), UPC = n_warps / WU;
  // the first CTA sets the status word, in the place of a memset in front of the kernel
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
  const int half = p.d_rope >> 1;
  float* scale_at = p.scales + (long long)b * p.n_blocks + blk;

  Eight<T> x[TPW][NS];
  T k1[TPW], k2[TPW];
  int exps = kQcacheMinExp;
#pragma unroll
  for (int i = 0; i < TPW; ++i) {
    const int t = lo + wi + i * WU;
    k1[i] = k2[i] = from_f<T>(0.f);
#pragma unroll
    for (int s = 0; s < NS; ++s) x[i][s].zero();
    if (unit_on && t < hi) {
      const long long row = (long long)b * p.L + (t - p0);
      const T* c = reinterpret_cast<const T*>(p.c_kv) + row * p.d_c;
#pragma unroll
      for (int s = 0; s < NS; ++s)
        if ((lane + 32 * s) * 8 < p.d_c) x[i][s].load(c + (lane + 32 * s) * 8);
      if (lane < half) {
        const T* kr = reinterpret_cast<const T*>(p.k_rope) + row * p.d_rope;
        k1[i] = kr[lane];
        k2[i] = kr[lane + half];
      }
    }
  }
  if (unit_on && wi == 0 && lane == 0) unit_old[ul] = first < p0 ? *scale_at : 0.f;

  // gain; without one the rows are normalised already and r = 1
  Eight<T> gam[NS];
  const bool norm = p.gamma != nullptr;
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    gam[s].zero();
    if (norm && (lane + 32 * s) * 8 < p.d_c)
      gam[s].load(reinterpret_cast<const T*>(p.gamma) + (lane + 32 * s) * 8);
  }
  float rh[TPW], rl[TPW], y1[TPW], y2[TPW];  // 1/rms as a sum of two floats; the rotated pair
#pragma unroll
  for (int i = 0; i < TPW; ++i) {
    const int t = lo + wi + i * WU;
    const bool on = unit_on && t < hi;
    double r = 1.0, top = 0.0;
    if (norm) {
      double ss;
      if constexpr (sizeof(T) == 2) {
        // squares of bf16 values are exact in fp32; their sum is kept with its error
        float sum = 0.f, err = 0.f;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          float f[8];
          x[i][s].get(f);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float sq = __fmul_rn(f[q], f[q]);
            const float a = __fadd_rn(sum, sq), bb = __fsub_rn(a, sum);
            err += __fadd_rn(__fsub_rn(sum, __fsub_rn(a, bb)), __fsub_rn(sq, bb));
            sum = a;
          }
        }
        ss = (double)sum + (double)err;
      } else {
        ss = 0.0;
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          float f[8];
          x[i][s].get(f);
#pragma unroll
          for (int q = 0; q < 8; ++q) ss = fma((double)f[q], (double)f[q], ss);
        }
      }
      const double m = warp_sum(ss) / (double)p.d_c + (double)p.eps;
      // 1/sqrt(m): the fp32 estimate and two Newton steps y (3 - m y^2) / 2
      double y = (double)rsqrtf((float)m);
      y *= 1.5 - 0.5 * m * y * y;
      y *= 1.5 - 0.5 * m * y * y;
      r = y;
    }
    rh[i] = (float)r;
    rl[i] = (float)(r - (double)rh[i]);
    // the largest |gamma c|, times r
    if constexpr (sizeof(T) == 2) {
      float mx = 0.f;  // (products of two bf16 values are exact; fmaxf passes over a NaN)
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        float f[8], g[8];
        x[i][s].get(f);
        gam[s].get(g);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float v = fabsf(norm ? f[q] * g[q] : f[q]);
          mx = fmaxf(mx, v < INFINITY ? v : 0.f);
        }
      }
      top = (double)mx * r;
    } else {
      double mx = 0.0;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        float f[8], g[8];
        x[i][s].get(f);
        gam[s].get(g);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const double v = fabs(norm ? (double)f[q] * (double)g[q] : (double)f[q]);
          mx = v < (double)INFINITY && v > mx ? v : mx;
        }
      }
      top = mx * r;
    }
    double z1 = (double)to_f(k1[i]), z2 = (double)to_f(k2[i]);
    if (norm && on && lane < half) {
      const double cs = (double)p.cos_tab[(long long)t * half + lane], sn = (double)p.sin_tab[(long long)t * half + lane];
      const double w1 = z1 * cs - z2 * sn, w2 = z2 * cs + z1 * sn;
      z1 = w1;
      z2 = w2;
    }
    y1[i] = (float)z1;
    y2[i] = (float)z2;
    int e = scale_exp(top);
    e = max(e, scale_exp(fabs(z1)));
    e = max(e, scale_exp(fabs(z2)));
    if (on) exps = max(exps, e);
  }
  exps = __reduce_max_sync(0xffffffffu, exps);
  if (lane == 0) warp_exp[warp] = exps;
  __syncthreads();
  if (!unit_on) return;
  for (int w = 0; w < WU; ++w) exps = max(exps, warp_exp[ul * WU + w]);
  float scale = exp_to_float(exps);
  // earlier tokens of the block: keep their scale, or bring them to the larger one
  const float old = unit_old[ul];
  if (first < p0 && old > 0.f && old < INFINITY) {
    if (scale <= old) {
      scale = old;
    } else {
      const float by = old / scale;
      for (long long t = first + wi; t < p0; t += WU) {
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
  }
  if (wi == 0 && lane == 0) *scale_at = scale;
  const float inv = 1.f / scale;
#pragma unroll
  for (int i = 0; i < TPW; ++i) {
    const int t = lo + wi + i * WU;
    if (t >= hi) continue;
    const long long row = (long long)b * p.T_max + t;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      if ((lane + 32 * s) * 8 >= p.d_c) continue;
      float f[8], g[8];
      x[i][s].get(f);
      gam[s].get(g);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        if (norm) {
          if constexpr (sizeof(T) == 2) {
            // (gamma c) r with r = rh + rl: the product's rounding error is added back
            const float v = f[q] * g[q], ph = __fmul_rn(v, rh[i]);
            f[q] = __fadd_rn(ph, fmaf(v, rl[i], fmaf(v, rh[i], -ph)));
          } else {
            f[q] = (float)((double)f[q] * (double)g[q] * ((double)rh[i] + (double)rl[i]));
          }
        }
        f[q] = finite_or_nan(f[q]) * inv;
      }
      *reinterpret_cast<uint2*>(p.c8 + row * p.d_c + (lane + 32 * s) * 8) =
          make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
    }
    if (lane < half) {
      const uint32_t two = e4m3x4(finite_or_nan(y1[i]) * inv, finite_or_nan(y2[i]) * inv, 0.f, 0.f);
      p.kr8[row * p.d_rope + lane] = (uint8_t)(two & 0xFFu);
      p.kr8[row * p.d_rope + half + lane] = (uint8_t)((two >> 8) & 0xFFu);
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
    case 1: qcache_write_kernel<T, NS, 1><<<grid, warps * 32, 0, s>>>(p); break;
    case 2: qcache_write_kernel<T, NS, 2><<<grid, warps * 32, 0, s>>>(p); break;
    case 4: qcache_write_kernel<T, NS, 4><<<grid, warps * 32, 0, s>>>(p); break;
    default: qcache_write_kernel<T, NS, 8><<<grid, warps * 32, 0, s>>>(p); break;
  }
  return cudaGetLastError();
}

// ------------------------------------------------------------------------ read
// One thread turns 16 cached bytes into 16 values; a row is (d_c + d_rope) / 16 pieces.
template <typename T>
__global__ void __launch_bounds__(256) qcache_read_kernel(const QcacheReadParams p) {
  const int pc = (p.d_c + p.d_rope) >> 4, cc = p.d_c >> 4;
  const long long e = (long long)blockIdx.x * 256 + threadIdx.x;
  const int b = blockIdx.y;
  if (e >= (long long)p.L * pc) return;
  const int i = (int)(e / pc), q = (int)(e % pc);
  const int n = p.lens ? min(max(p.lens[b], 0), p.L) : p.L;
  float f[16];
  if (i < n) {
    const long long row = (long long)b * p.T_max + p.first + i;
    const float s = p.scales[(long long)b * p.n_blocks + ((p.first + i) >> p.sl)];
    const uint4 v = q < cc ? reinterpret_cast<const uint4*>(p.c8 + row * p.d_c)[q]
                           : reinterpret_cast<const uint4*>(p.kr8 + row * p.d_rope)[q - cc];
    const uint32_t* u = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = e4m3x2_to_float2(u[j]), c = e4m3x2_to_float2(u[j] >> 16);
      f[4 * j] = a.x * s; f[4 * j + 1] = a.y * s; f[4 * j + 2] = c.x * s; f[4 * j + 3] = c.y * s;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) f[j] = 0.f;
  }
  const long long o = (long long)b * p.L + i;
  T* dst = q < cc ? reinterpret_cast<T*>(p.c_hat) + o * p.d_c + q * 16
                  : reinterpret_cast<T*>(p.k_rope) + o * p.d_rope + (q - cc) * 16;
  if constexpr (sizeof(T) == 2) {
    uint4 w[2];
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(w);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
    reinterpret_cast<uint4*>(dst)[0] = w[0];
    reinterpret_cast<uint4*>(dst)[1] = w[1];
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      reinterpret_cast<float4*>(dst)[j] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
  }
}

}  // namespace

cudaError_t launch_qcache_write(const QcacheWriteParams& p, gdla_dtype dt, cudaStream_t s) {
  if (dt == GDLA_BF16) return p.d_c > 256 ? write_ns<__nv_bfloat16, 2>(p, s) : write_ns<__nv_bfloat16, 1>(p, s);
  return p.d_c > 256 ? write_ns<float, 2>(p, s) : write_ns<float, 1>(p, s);
}

cudaError_t launch_qcache_read(const QcacheReadParams& p, gdla_dtype dt, cudaStream_t s) {
  const long long n = (long long)p.L * ((p.d_c + p.d_rope) / 16);
  const dim3 grid((unsigned)((n + 255) / 256), (unsigned)p.B);
  if (dt == GDLA_BF16)
    qcache_read_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(p);
  else
    qcache_read_kernel<float><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace gdla
