// qdecode.cu -- the split-KV pass over the 8-bit latent cache on the CUDA cores, for the
// shapes and fp32 tensors that the tensor-core kernel does not take. It stands between
// the absorb and combine kernels of the bf16 / fp32 cache, whose records it writes:
//   S_hj = tau log2e s_j (q_abs,h . c8_j + q_rot,h . k8_j), O_h = sum_j 2^(S - m) s_j c8_j.
#include <cuda_fp8.h>
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace gdla {

// Block (split s, sequence b), 256 threads: tiles of 32 tokens are turned into fp32 rows in
// shared memory (16 bytes per thread and load) and used for the scores (lane = token, one
// warp per head) and the weighted sum (thread: heads warp + 8 i, columns lane + 32 c).
// A row's scale multiplies its values once, as it is unpacked.
template <int HPT, int CPT>
__global__ void __launch_bounds__(256) qdecode_split_simt_kernel(const QdecodeParams qp) {
  constexpr int BT = 32;
  const DecodeParams& p = qp.d;
  const int s = blockIdx.x, b = blockIdx.y;
  const int n_S = p.g * p.n_kv, H_q = n_S + p.n_kv;
  const int d_c = p.d_c, d_r = p.d_rope, RW = d_c + d_r + 1;  // padded row
  extern __shared__ float sm[];
  float* qa = sm;               // [H_q][d_c]
  float* qr = qa + H_q * d_c;   // [H_q][d_r]
  float* ct = qr + H_q * d_r;   // [BT][RW]
  float* ps = ct + BT * RW;     // [H_q][BT]
  float* mrow = ps + H_q * BT;  // [H_q]
  float* lrow = mrow + H_q;
  float* arow = lrow + H_q;
  const uint8_t* cc = reinterpret_cast<const uint8_t*>(p.c_cache);
  const uint8_t* kc = reinterpret_cast<const uint8_t*>(p.kr_cache);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float sl2 = p.scale * kLog2e;

  // (started while the absorb kernel still runs; the combine kernel in turn beside this one)
  sm100::grid_dep_launch();
  sm100::grid_dep_wait();
  for (int e = tid; e < H_q * d_c; e += 256) qa[e] = p.q_abs[(long long)b * H_q * d_c + e];
  for (int e = tid; e < H_q * d_r; e += 256) qr[e] = p.q_rot[(long long)b * H_q * d_r + e];
  for (int e = tid; e < H_q; e += 256) {
    mrow[e] = -INFINITY;
    lrow[e] = 0.f;
  }
  const int raw = p.seqlens[b];
  if ((raw < 0 || raw > p.T_max) && s == 0 && tid == 0) atomicCAS(p.status, 0, (int)GDLA_ERR_INVALID_ARG);
  const int Tb = min(max(raw, 0), p.T_max);
  const int lo = p.sliding ? max(0, Tb - p.window) : 0;
  const long long s0 = (long long)s * p.split_len;
  const int t0 = (int)max((long long)lo, s0), t1 = (int)min((long long)Tb, s0 + p.split_len);

  float acc[HPT][CPT];
#pragma unroll
  for (int a = 0; a < HPT; ++a)
#pragma unroll
    for (int c = 0; c < CPT; ++c) acc[a][c] = 0.f;

  const int pieces = (d_c + d_r) >> 4;
  for (int j0 = t0; j0 < t1; j0 += BT) {
    __syncthreads();
    for (int e = tid; e < BT * pieces; e += 256) {
      const int r = e / pieces, q = e % pieces, j = j0 + r;
      uint4 v = make_uint4(0, 0, 0, 0);
      float sc = 0.f;
      if (j < t1) {
        const long long row = (long long)b * p.T_max + j;
        v = q < (d_c >> 4) ? reinterpret_cast<const uint4*>(cc + row * d_c)[q]
                           : reinterpret_cast<const uint4*>(kc + row * d_r)[q - (d_c >> 4)];
        sc = qp.scales[(long long)b * qp.n_blocks + (j >> qp.sl)];
      }
      const uint32_t* u = reinterpret_cast<const uint32_t*>(&v);
      float* dst = ct + r * RW + q * 16;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((u[i >> 1] >> (16 * (i & 1))) & 0xFFFFu),
                                                         __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        dst[2 * i] = f.x * sc;
        dst[2 * i + 1] = f.y * sc;
      }
    }
    __syncthreads();
    for (int hh = warp; hh < H_q; hh += 8) {
      const float* qh = qa + hh * d_c;
      const float* crow = ct + lane * RW;
      float d0 = 0.f, d1 = 0.f, d2 = 0.f, d3 = 0.f;
      for (int k = 0; k < d_c; k += 4) {
        d0 = fmaf(qh[k], crow[k], d0);
        d1 = fmaf(qh[k + 1], crow[k + 1], d1);
        d2 = fmaf(qh[k + 2], crow[k + 2], d2);
        d3 = fmaf(qh[k + 3], crow[k + 3], d3);
      }
      const float* qrh = qr + hh * d_r;
      for (int k = 0; k < d_r; k += 4) {
        d0 = fmaf(qrh[k], crow[d_c + k], d0);
        d1 = fmaf(qrh[k + 1], crow[d_c + k + 1], d1);
        d2 = fmaf(qrh[k + 2], crow[d_c + k + 2], d2);
        d3 = fmaf(qrh[k + 3], crow[d_c + k + 3], d3);
      }
      const float sv = j0 + lane < t1 ? ((d0 + d1) + (d2 + d3)) * sl2 : -INFINITY;
      float mx = sv;
#pragma unroll
      for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float m_old = mrow[hh], m_new = fmaxf(m_old, mx);
      // (m_new stays -inf only where every score so far is NaN: the weights are then NaN too)
      const float pe = j0 + lane < t1 ? exp2f(sv - m_new) : 0.f;
      float sum = pe;
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      ps[hh * BT + lane] = pe;
      __syncwarp();
      if (lane == 0) {
        const float al = m_old == -INFINITY ? (m_new == -INFINITY ? 1.f : 0.f) : exp2f(m_old - m_new);
        arow[hh] = al;
        lrow[hh] = lrow[hh] * al + sum;
        mrow[hh] = m_new;
      }
    }
    __syncthreads();
#pragma unroll
    for (int a = 0; a < HPT; ++a) {
      const int hh = warp + 8 * a;
      if (hh >= H_q) break;
      const float al = arow[hh];
#pragma unroll
      for (int c = 0; c < CPT; ++c) acc[a][c] *= al;
      for (int j = 0; j < BT; ++j) {
        const float pj = ps[hh * BT + j];
#pragma unroll
        for (int c = 0; c < CPT; ++c) acc[a][c] = fmaf(pj, ct[j * RW + lane + 32 * c], acc[a][c]);
      }
    }
  }
  __syncthreads();
  const long long base = ((long long)b * p.n_splits + s) * p.part_heads;
#pragma unroll
  for (int a = 0; a < HPT; ++a) {
    const int hh = warp + 8 * a;
    if (hh >= H_q) break;
#pragma unroll
    for (int c = 0; c < CPT; ++c) p.part_o[(base + hh) * d_c + lane + 32 * c] = acc[a][c];
  }
  for (int e = tid; e < H_q; e += 256) {
    p.part_ml[(base + e) * 2 + 0] = mrow[e];
    p.part_ml[(base + e) * 2 + 1] = lrow[e];
  }
}

namespace {

template <int HPT, int CPT>
cudaError_t one(const QdecodeParams& p, cudaStream_t s) {
  const DecodeParams& d = p.d;
  const int H_q = d.n_kv * (d.g + 1);
  const size_t smem = sizeof(float) * ((size_t)H_q * d.d_c + (size_t)H_q * d.d_rope +
                                       32 * (size_t)(d.d_c + d.d_rope + 1) + (size_t)H_q * 32 + 3 * (size_t)H_q);
  auto k = qdecode_split_simt_kernel<HPT, CPT>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)d.n_splits, (unsigned)d.B);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, p);
}
template <int HPT>
cudaError_t by_width(const QdecodeParams& p, cudaStream_t s) {
  switch (p.d.d_c) {
    case 64: return one<HPT, 2>(p, s);
    case 128: return one<HPT, 4>(p, s);
    case 256: return one<HPT, 8>(p, s);
    case 512: return one<HPT, 16>(p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_qdecode_split_simt(const QdecodeParams& p, cudaStream_t s) {
  const int H_q = p.d.n_kv * (p.d.g + 1);
  if (H_q <= 16) return by_width<2>(p, s);
  if (H_q <= 32) return by_width<4>(p, s);
  if (H_q <= 48) return by_width<6>(p, s);
  if (H_q <= 64) return by_width<8>(p, s);
  return cudaErrorInvalidValue;
}

}  // namespace gdla
