// qdecode_tc.cu -- split-KV GDLA decode over the 8-bit latent cache on the 5th-generation
// tensor cores. A cached row is 512 + 64 e4m3 values times a scale s_j (one per block of
// tokens), and both products of the attention run on it as it is stored:
//   S_hj = s_j (q~_h . row8_j)            q~ = tau log2e [W_UK q_nope | RoPE(q_rope)]
//   O_h  = sum_j 2^(S_hj) s_j c8_j        (over the sum of 2^(S_hj))
//   S^T[tokens x 2 heads] = row8[tokens x 576] . q8^T                  (M = 128, N = 96)
//   O^T[512 x 2 heads]   += c8^T[512 x tokens] . w8^T[tokens x 2 heads]  (M = 4 x 128, N = 96)
// The tensor cores take 8-bit operands on both sides, so the other operand of each product
// is split into two e4m3 terms, x = hi + lo / 16 (4 + 4 significant bits and the sign of the
// remainder: relative rounding at most 2^-8, 6e-4 rms; bf16's is 1.6e-3 rms). Both terms are
// columns of one MMA, which so reads the cached tile from shared memory once (the rate of an
// 8-bit MMA of this width is that of its shared-memory reads), and the two halves are added
// when the accumulator is read:
//   * q~ / 2^k, 2^k chosen for each head: its largest element fills the e4m3 range;
//   * w = 2^(S + log2 s_j - M + 6) <= 2^8.75 < 448. Its rounding is relative down to 2^-6;
//     below, the step is 2^-13, and a weight under 2^-14 is lost. That counts where many small
//     weights stand behind few large ones (a sink over a long flat context), so:
//     - Where M has risen by 2^6 at least to a tile's maximum, and then at most 64 of the tile's
//       weights are 2^-6 and more and all the others smaller by 2^14 at least, or by 2^8 and a
//       crowd (an eighth of them within 2^8 of their largest; in a broad softmax they add up to
//       nothing), M goes to 2^4 times the largest of the others (2^8 if they are no crowd: then
//       the tiles' maxima vary more). The few go around the MMA: they are added to O^T in fp32.
//     - At every 8th tile M goes down to 2^4 times the tile's largest weight where all of them
//       are below 2^-6 and a crowd. Until then a tile's 128 weights lose 2^-13 of the largest
//       weight at most.
//     M stays within 2^60 of the largest reference before: O^T and the sum hold 2^66 and more.
//     Logits of 1 / 2 / 4 / 8 nats deviation, 64 x 32768 tokens, 48 heads: 296 / 355 / 422 / 651
//     us a call (287 / 325 / 353 / 349 with an M that only rises, and its lost weights). What
//     is not seen: several heights above the others with none of the gaps, whose values vanish.
// A scale enters twice, both times outside the products: it multiplies the score, and it
// is part of the weight (the reference M follows the maxima of S + log2 s). The sum of
// 2^S is kept in fp32 from the weights before their rounding.
//
// Split: the visible 128-token tiles of all sequences are numbered in sequence order, and
// CTA r of a head group takes tiles [r W / R, (r + 1) W / R): equal shares, no tail wave.
// A share writes one partial (M, l, O) per sequence it touches, to record r + b; the
// combine kernel merges the records of a sequence.
//
// Block: warp 0 loads tiles (TMA, two stages of 72 KB), warp 1 issues the MMAs, warp 2 loads
// query images, warp 3 reports what failed before; the others are the softmax, a group of four warps for each 16 of
// the up to 48 heads: a thread owns one token (TMEM lane) and 16 heads, and the four warps of
// a group agree on their heads' references by a barrier of their own. Every wait is bounded
// and reports GDLA_ERR_TIMEOUT.
//
// What bounds it (B=64 over 32768 tokens, 48 heads: this kernel 286 us by itself, 4.2 TB/s of cache): a
// tile's way through its stage -- load, scores (1015 cycles of shared-memory reads), softmax
// (~1750), values (905) -- with two of them in flight; the loads alone run at the memory's
// rate (without the MMAs: 211 us). Tried and slower: prefetches into L2 (337 us a call without,
// 344 to 363 with one to four tiles ahead), stages released in halves (the same) or quarters
// (+5 %), box by box (+30 %: a row's 512 bytes are then read at four times), and three stages
// of 96 tokens (+13 %: the softmax's work a tile is the same for fewer tokens).
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>

#include "kernels.h"
#include "sm100.cuh"

namespace gdla {
namespace q8 {

constexpr int DC = 512, DR = 64;
constexpr int TT = kQdecTile;                  // cache tokens per tile (M of the score MMA)
constexpr int HT = 16;                         // heads per softmax thread
constexpr int BOX = TT * 128, RBOX = TT * 64;  // a 128-column box of the tile; the rotary box
constexpr int TILE = 4 * BOX + RBOX;
constexpr int STAGES = 2;
constexpr int PBYTES = TT * 128;               // weights: TT tokens x (hi, lo) heads, one byte each
constexpr uint32_t COL_S = 0;                  // S^T; then O^T of M-tile mt at NQ (1 + mt)
constexpr float kBase = 6.f;                   // weights are 2^(S + log2 s - M + kBase)
constexpr float kThr = 2.75f;                  // M moves when exceeded by this: w <= 2^8.75 < 448
constexpr float kLow = -6.f;                   // weights from 2^kLow on are rounded relatively
constexpr int kFew = 64;                       // tokens of a tile that may go around the MMA
constexpr int kBatch = 16;                     // so many at a time
constexpr float kGap = 8.f;                    // and how far the others are below them
constexpr float kFar = 14.f;                   // so far below, they are kept even if they are no crowd
constexpr int kCrowd = 8;                      // a crowd: 1 / 8 within 2^kGap of the largest
constexpr float kRise = 6.f;                   // M has risen by this at least
constexpr float kRoom = 4.f;                   // M over the others then: the next tiles' maxima vary
constexpr int kLook = 8;                       // tiles from one look down to the next
constexpr float kSpan = 60.f;                  // M goes down this far at most
constexpr float kMinScale = 8.6736174e-19f;    // 2^-60: keeps 1/s finite whatever the scales hold

// the layout for head groups of 16 HG heads
template <int HG>
struct Lay {
  static constexpr int NH = HT * HG, NQ = 2 * NH;          // heads; hi and lo rows of the query operand
  static constexpr int QBOX = NQ * 128, QIMG = NQ * 576;   // 128-column box of the query image; the image
  static constexpr int OFF_TILES = QIMG, OFF_P = OFF_TILES + STAGES * TILE, OFF_SH = OFF_P + PBYTES;
  static constexpr int NSW = 4 * HG, NT = 32 * (4 + NSW);  // softmax warps; threads
  struct Shared {
    uint64_t full[STAGES], empty[STAGES];
    uint64_t s_full, s_free, p_full, p_free;
    uint64_t q_full, q_free, seg_done, mma_done;
    uint32_t tmem_slot;
    int abort_flag;
    int b0;
    int R;
    long long p0, start, end, W;
    long long red[NT / 32];
    float4 hx[NH / 4], hm[NH / 4];  // per head: scale of the query; kBase - M
    float wmax[4][NH];
    float alpha[NH], move[NH];  // of a moved reference: 2^(old - new); the old less the new
    // a moving reference: of each warp the tokens at 2^kLow and above (as a mask), the smallest
    // S + log2 s of these, how many are below; the largest reference of the sequence share
    uint32_t big[4][NH];
    float wmin[4][NH];
    int small[4][NH];
    float top[NH];
    int n_out[NH];                  // tokens of the tile that go around the MMA
    // the same for the groups: the warps' tokens that some head takes out; a batch of them and
    // their weights
    uint32_t out_mask[HG][4];
    int out_row[HG][kBatch];
    float4 out_w[HG][kBatch][HT / 4];
  };
  static constexpr int SMEM = OFF_SH + (int)sizeof(Shared);
  static_assert(QIMG % 1024 == 0 && TILE % 1024 == 0, "1024-byte swizzle atoms");
  static_assert(NQ * 5 <= 512, "TMEM columns");
  static_assert(SMEM <= 232448, "shared memory of one CTA");
};

struct Args {
  int B, T_max, sliding, window, H_q, n_hg, hpc, n_ranges, sl, n_blocks, img_bytes;
  const int* seqlens;
  const uint8_t* c8;
  const uint8_t* kr8;
  const float* scales;
  const uint8_t* qimg;
  int2* seqinfo;
  float* part_o;   // [records][heads of a group][512]
  float* part_ml;  // [records][heads of a group][2]
  int* status;
  const int* failed;  // of the absorb kernel's CTAs
  int n_absorb;
};

// the visible tiles of a sequence: tokens [lo, Tb), tiles jt0 .. jt0 + n - 1
struct SeqTiles {
  int Tb, lo, jt0, n;
};
__device__ __forceinline__ SeqTiles seq_tiles(const Args& a, int b) {
  SeqTiles s;
  s.Tb = min(max(__ldg(a.seqlens + b), 0), a.T_max);
  s.lo = a.sliding ? max(0, s.Tb - a.window) : 0;
  s.jt0 = s.lo / TT;
  s.n = (int)(((long long)s.Tb + TT - 1) / TT) - s.jt0;
  return s;
}
// failures of the absorb kernel's CTAs, as they are left in their records
constexpr int kAbsorbLoad = 541, kAbsorbMma = 542, kAbsorbAlignment = 598;
// these are reported, and lengths outside [0, T_max], which are clamped
__device__ __forceinline__ void report(const Args& a, int t, int nt) {
  for (int c = t; c < a.n_absorb; c += nt) {
    const int code = a.failed[c];
    if (code) {
      atomicCAS(a.status, 0, (int)(code == kAbsorbAlignment ? GDLA_ERR_CUDA : GDLA_ERR_TIMEOUT));
      atomicCAS(a.status + 1, 0, code);
    }
  }
  for (int b = t; b < a.B; b += nt) {
    const int raw = __ldg(a.seqlens + b);
    if (raw < 0 || raw > a.T_max) atomicCAS(a.status, 0, (int)GDLA_ERR_INVALID_ARG);
  }
}
struct Walker {
  const Args* a;
  int b;
  long long pb;  // global index of sequence b's first tile
  SeqTiles st;
  __device__ void init(const Args& args, int b0, long long p0) {
    a = &args;
    b = b0;
    pb = p0;
    st = seq_tiles(args, b0);
  }
  __device__ void seek(long long t) {  // (t never decreases)
    while (t >= pb + st.n) {
      pb += st.n;
      ++b;
      st = seq_tiles(*a, b);
    }
  }
  __device__ int token0(long long t) const { return (st.jt0 + (int)(t - pb)) * TT; }
};
// the share that holds global tile t: the largest r with floor(r W / R) <= t
__device__ __forceinline__ int range_of(long long t, long long W, int R) {
  return (int)(((t + 1) * (long long)R - 1) / W);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t e4m3x2(__half2 h) {
  return __nv_cvt_halfraw2_to_fp8x2(*reinterpret_cast<const __half2_raw*>(&h), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ __half2 e4m3x2_to_half2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return *reinterpret_cast<const __half2*>(&h);
}
// two weights as pairs of hi and 16 lo. The remainder is formed in fp16, whose 11 bits hold
// the 4 of hi and more than the 4 of lo
__device__ __forceinline__ void split_weights(float w0, float w1, uint32_t& hi, uint32_t& lo) {
  const __half2 w = __floats2half2_rn(w0, w1);
  hi = e4m3x2(w);
  lo = e4m3x2(__hmul2(__hsub2(w, e4m3x2_to_half2(hi)), __float2half2_rn(16.f)));
}
__device__ __forceinline__ float2 f2(const uint32_t (&r)[HT], int i) {
  return make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
}
// the largest value of a warp (one that is not a number is passed over)
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
// pair i of 16 per-head values
__device__ __forceinline__ float2 pair(const float4* v, int i) {
  const float4 x = v[i >> 1];
  return i & 1 ? make_float2(x.z, x.w) : make_float2(x.x, x.y);
}

// The MMAs of a tile in stage ST. The stage is a constant so that every descriptor is one plus
// a constant.
template <int HG, int ST>
__device__ __forceinline__ void score_mmas(uint32_t smem, uint32_t tmem) {
  using namespace sm100;
  using L = Lay<HG>;
  constexpr uint32_t id = idesc_f8_f32(TT, L::NQ, kF8E4m3, kF8E4m3, false, false);
  const uint64_t q128 = sdesc_sw128(smem, 16, 1024), q64 = sdesc_sw64(smem + 4 * L::QBOX, 16, 512);
  const uint64_t c128 = sdesc_sw128(smem + L::OFF_TILES + ST * TILE, 16, 1024);
  const uint64_t c64 = sdesc_sw64(smem + L::OFF_TILES + ST * TILE + 4 * BOX, 16, 512);
#pragma unroll
  for (int kk = 0; kk < 16; ++kk) {
    const uint32_t bx = kk >> 2, off = (kk & 3) * 32;
    mma_f8_ss(tmem + COL_S, c128 + ((bx * BOX + off) >> 4), q128 + ((bx * L::QBOX + off) >> 4), id, kk > 0);
  }
#pragma unroll
  for (int kk = 0; kk < 2; ++kk) mma_f8_ss(tmem + COL_S, c64 + 2 * kk, q64 + 2 * kk, id, 1);
}
// (O^T starts from the zeros that the softmax warps write)
template <int HG, int ST>
__device__ __forceinline__ void value_mmas(uint32_t smem, uint32_t tmem) {
  using namespace sm100;
  using L = Lay<HG>;
  constexpr uint32_t id = idesc_f8_f32(128, L::NQ, kF8E4m3, kF8E4m3, true, true);
  const uint64_t c = sdesc_sw128(smem + L::OFF_TILES + ST * TILE, BOX, 1024);
  const uint64_t wd = sdesc_sw128(smem + L::OFF_P, BOX, 1024);
#pragma unroll
  for (int kk = 0; kk < TT / 32; ++kk)  // 32 tokens: 4096 bytes of a box and of the weights
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
      mma_f8_ss(tmem + L::NQ * (1 + mt), c + ((mt * BOX + kk * 4096) >> 4), wd + ((kk * 4096) >> 4), id, 1u);
}

}  // namespace q8

template <int HG>
__global__ void __launch_bounds__(q8::Lay<HG>::NT, 1)
    qdecode_split_kernel(const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmR,
                         const q8::Args a) {
  using namespace sm100;
  using namespace q8;
  using L = Lay<HG>;
  constexpr int NH = L::NH, NQ = L::NQ, NT = L::NT, NSW = L::NSW;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* qs = smem;                     // query image: 4 boxes of [NQ x 128 B], one of [NQ x 64 B]
  uint8_t* tiles = smem + L::OFF_TILES;   // stages: 4 boxes of [128 tokens x 128 B], one of [128 x 64 B]
  uint8_t* ps = smem + L::OFF_P;          // weights [128 tokens x 128 B]: NH hi, NH lo
  typename L::Shared& sh = *reinterpret_cast<typename L::Shared*>(smem + L::OFF_SH);
  volatile int& abort_flag = sh.abort_flag;

  grid_dep_launch();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hg = blockIdx.x, r = blockIdx.y;
  if (smem_u32(smem) & 1023u) {  // the swizzled operands need it: report instead of computing garbage
    if (tid == 0) {
      atomicCAS(a.status, 0, (int)GDLA_ERR_CUDA);
      atomicCAS(a.status + 1, 0, 599);
    }
    grid_dep_wait();
    return;
  }

  // ---- this CTA's share of the W tiles, and the sequence that holds its first tile
  {
    long long loc = 0;
    for (int b = tid; b < a.B; b += NT) {
      loc += seq_tiles(a, b).n;
    }
    for (int o = 16; o; o >>= 1) loc += __shfl_xor_sync(0xffffffffu, loc, o);
    if (lane == 0) sh.red[warp] = loc;
    __syncthreads();
    if (tid == 0) {
      long long W = 0;
      for (int w = 0; w < NT / 32; ++w) W += sh.red[w];
      const long long R = min((long long)a.n_ranges, W);
      sh.start = r < R ? (long long)r * W / R : 0;
      sh.end = r < R ? (long long)(r + 1) * W / R : 0;
      sh.R = (int)R;
      sh.b0 = -1;
      sh.W = W;
    }
    __syncthreads();
    const long long start = sh.start;
    if (start < sh.end) {
      long long base = 0;
      for (int c0 = 0; c0 < a.B; c0 += NT) {
        const int b = c0 + tid;
        const long long n = b < a.B ? seq_tiles(a, b).n : 0;
        long long incl = n;
        for (int o = 1; o < 32; o <<= 1) {
          const long long v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        if (lane == 31) sh.red[warp] = incl;
        __syncthreads();
        long long wbase = base;
        for (int w = 0; w < warp; ++w) wbase += sh.red[w];
        long long total = 0;
        for (int w = 0; w < NT / 32; ++w) total += sh.red[w];
        const long long p = wbase + incl - n;
        if (b < a.B && n > 0 && p <= start && start < p + n) {
          sh.b0 = b;
          sh.p0 = p;
        }
        base += total;
        __syncthreads();
        if (sh.b0 >= 0) break;
      }
    }
  }
  const long long start = sh.start, end = sh.end, W = sh.W;
  const int R = sh.R;
  if (start >= end || sh.b0 < 0) {  // a range beyond the tiles
    grid_dep_wait();                // (this grid never completes before the one it overlaps)
    if (r == 0 && hg == 0) report(a, tid, NT);
    return;
  }
  const int b0 = sh.b0;
  const long long p0 = sh.p0;
  const int n_tiles = (int)(end - start);
  const int nh = min(a.hpc, a.H_q - hg * a.hpc);  // query heads of this head group

  if (tid == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(smem_u32(&sh.full[i]), 1);
      mbar_init(smem_u32(&sh.empty[i]), 1);
    }
    mbar_init(smem_u32(&sh.s_full), 1);
    mbar_init(smem_u32(&sh.s_free), NSW);
    mbar_init(smem_u32(&sh.p_full), NSW);
    mbar_init(smem_u32(&sh.p_free), 1);
    mbar_init(smem_u32(&sh.q_full), 1);
    mbar_init(smem_u32(&sh.q_free), 1);
    mbar_init(smem_u32(&sh.seg_done), 1);
    mbar_init(smem_u32(&sh.mma_done), 1);
    fence_mbar_init();
    abort_flag = 0;
    prefetch_tmap(&tmC);
    prefetch_tmap(&tmR);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&sh.tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      Walker wl;
      wl.init(a, b0, p0);
      int k = 0;
      for (; k < n_tiles && !abort_flag; ++k) {
        const int st = k % STAGES;
        const long long t = start + k;
        wl.seek(t);
        if (t == wl.pb && hg == 0)  // this CTA holds the sequence's first tile: record who covers it
          a.seqinfo[wl.b] = make_int2(r, range_of(wl.pb + wl.st.n - 1, W, R));
        const int j0 = wl.token0(t);
        const uint32_t bar = smem_u32(&sh.full[st]);
        const uint32_t dst = smem_u32(tiles + st * TILE);
        if (k >= STAGES &&
            !mbar_wait(smem_u32(&sh.empty[st]), ((k / STAGES) & 1) ^ 1, a.status, 501, &abort_flag)) {
          abort_flag = 1;
          break;
        }
        mbar_expect_tx(bar, TILE);
        for (int bx = 0; bx < 4; ++bx) tma_load_3d(dst + bx * BOX, &tmC, bar, bx * 128, j0, wl.b);
        tma_load_3d(dst + 4 * BOX, &tmR, bar, 0, j0, wl.b);
      }
      // no copy is in flight at exit, also where another warp gives up after the last load
      for (int q = (k > STAGES ? k - STAGES : 0); q < k; ++q)
        mbar_wait(smem_u32(&sh.full[q % STAGES]), (q / STAGES) & 1, nullptr, 0);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMAs
    // One thread issues both products, so that neither's MMAs are interleaved with the other's:
    // the scores of tile k + 1 as soon as they can run, which the softmax waits for, then the
    // values of tile k.
    if (lane == 0) {
      Walker ws, wv;
      ws.init(a, b0, p0);
      wv.init(a, b0, p0);
      int ks = 0, kv = 0, seg = 0;  // next tile of the scores, of the values; query images used
      bool new_seq = true;          // tile ks starts a sequence
      bool ok = true;
      uint64_t t0 = 0;
      for (uint32_t idle = 0; kv < n_tiles && ok;) {
        // the score's operands: the tile, a sequence's query image, S^T read by the softmax
        if (ks < n_tiles && mbar_try_wait(smem_u32(&sh.full[ks % STAGES]), (ks / STAGES) & 1) &&
            (!new_seq || mbar_try_wait(smem_u32(&sh.q_full), seg & 1)) &&
            (ks == 0 || mbar_try_wait(smem_u32(&sh.s_free), (ks - 1) & 1))) {
          tc_fence_after();
          if (ks & 1)
            score_mmas<HG, 1>(smem_u32(smem), tmem);
          else
            score_mmas<HG, 0>(smem_u32(smem), tmem);
          mma_commit(smem_u32(&sh.s_full));
          ws.seek(start + ks);
          seg += new_seq;
          new_seq = start + ks == ws.pb + ws.st.n - 1;
          if (new_seq || ks == n_tiles - 1) mma_commit(smem_u32(&sh.q_free));  // the query image may be replaced
          ++ks;
          idle = 0;
        }
        // the weights of tile kv are written; their softmax has also read the previous sequence's
        // O^T and cleared it
        if (kv < ks && mbar_try_wait(smem_u32(&sh.p_full), kv & 1)) {
          const long long t = start + kv;
          wv.seek(t);
          tc_fence_after();
          if (kv & 1)
            value_mmas<HG, 1>(smem_u32(smem), tmem);
          else
            value_mmas<HG, 0>(smem_u32(smem), tmem);
          mma_commit(smem_u32(&sh.empty[kv % STAGES]));
          mma_commit(smem_u32(&sh.p_free));
          if (kv == n_tiles - 1 || t == wv.pb + wv.st.n - 1) mma_commit(smem_u32(&sh.seg_done));  // O^T holds the share
          ++kv;
          idle = 0;
        }
        if ((++idle & 255u) == 0) {  // bounded, like mbar_wait
          const uint64_t now = globaltimer_ns();
          if (idle == 256) t0 = now;
          const bool gave_up = now - t0 > kWaitLimitNs;
          if (gave_up) {
            atomicCAS(a.status, 0, (int)GDLA_ERR_TIMEOUT);
            atomicCAS(a.status + 1, 0, 511);
          }
          ok = !gave_up && !abort_flag && !earlier_failure(a.status);
        }
      }
      if (!ok) abort_flag = 1;
      mma_commit(smem_u32(&sh.mma_done));  // every MMA issued completes before TMEM is released
      mbar_wait(smem_u32(&sh.mma_done), 0, nullptr, 514);
    }
  } else if (warp == 2) {
    // -------------------------------------------------------- query images
    grid_dep_wait();  // the absorb kernel wrote them
    if (lane == 0) {
      Walker w;
      w.init(a, b0, p0);
      bool ok = true;
      int seg = 0;
      for (long long t = start; t < end && ok; ++seg) {
        w.seek(t);
        if (seg > 0) ok = mbar_wait(smem_u32(&sh.q_free), (seg - 1) & 1, a.status, 531, &abort_flag);
        if (!ok) break;
        const uint32_t bar = smem_u32(&sh.q_full);
        mbar_expect_tx(bar, L::QIMG);
        bulk_load(smem_u32(qs), a.qimg + ((long long)w.b * a.n_hg + hg) * a.img_bytes, L::QIMG, bar);
        t = w.pb + w.st.n;  // the next sequence's first tile
      }
      if (!ok) abort_flag = 1;
      if (seg > 0) mbar_wait(smem_u32(&sh.q_full), (seg - 1) & 1, nullptr, 0);  // no copy is in flight at exit
    }
  } else if (warp == 3) {
    grid_dep_wait();  // the absorb kernel cleared the status word
    if (r == 0 && hg == 0) report(a, lane, 32);
  } else {
    // ------------------------------------------------------------- softmax
    const int grp = (warp - 4) >> 2, q4 = warp & 3, hb = grp * HT;
    const int tl = q4 * 32 + lane;  // this thread's token of the tile; its index in the group
    const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
    const uint32_t tS = tmem + lane_base + COL_S + hb;
    float4* hx = sh.hx + hb / 4;
    float4* hm = sh.hm + hb / 4;
    float* hm1 = reinterpret_cast<float*>(hm);
    auto grp_or = [&](bool pred) { return named_bar_or(1 + grp, 128, pred); };
    auto grp_sync = [&]() { named_bar_sync(1 + grp, 128); };
    auto clear_o = [&]() {  // O^T of the sequence that comes
      uint32_t zero[HT];
#pragma unroll
      for (int h = 0; h < HT; ++h) zero[h] = 0;
#pragma unroll 1
      for (int c = 0; c < 8; ++c) tmem_st16(tmem + lane_base + NQ * (1 + (c >> 1)) + NH * (c & 1) + hb, zero);
      tmem_wait_st();
    };
    clear_o();
    Walker w, wn;
    w.init(a, b0, p0);
    wn.init(a, b0, p0);
    grid_dep_wait();
    // the scale of this thread's token of tile t (1 where the token is not visible)
    auto load_scale = [&](long long t) {
      wn.seek(t);
      const int j = wn.token0(t) + tl;
      return j >= wn.st.lo && j < wn.st.Tb ? __ldg(a.scales + (long long)wn.b * a.n_blocks + (j >> a.sl)) : 1.f;
    };
    float s_next = load_scale(start);
    float2 lp[HT / 2];
    int seg = -1;
    bool ok = true, bad = false;
    for (int k = 0; k < n_tiles; ++k) {
      const long long t = start + k;
      w.seek(t);
      const bool first = k == 0 || t == w.pb, last = k == n_tiles - 1 || t == w.pb + w.st.n - 1;
      const float sc = fmaxf(s_next, kMinScale);
      if (k + 1 < n_tiles) s_next = load_scale(t + 1);
      const int j = w.token0(t) + tl;
      const bool valid = j >= w.st.lo && j < w.st.Tb;
      if (first) {
        ++seg;
        if (tl < HT) {
          const float* hs = reinterpret_cast<const float*>(
              a.qimg + ((long long)w.b * a.n_hg + hg) * a.img_bytes + L::QIMG);
          reinterpret_cast<float*>(hx)[tl] = hs[hb + tl];
          hm1[tl] = kBase;
          sh.top[hb + tl] = -INFINITY;  // (no reference yet)
        }
#pragma unroll
        for (int i = 0; i < HT / 2; ++i) lp[i] = make_float2(0.f, 0.f);
        grp_sync();
      }
      const float ls = __log2f(sc), inv_s = __frcp_rn(sc);
      const float2 s2 = make_float2(sc, sc), ls2 = make_float2(ls, ls), i2 = make_float2(inv_s, inv_s);
      // the score's factor and offset, ready before the score
      float2 fa[HT / 2], fb[HT / 2];
#pragma unroll
      for (int i = 0; i < HT / 2; ++i) {
        fa[i] = fmul2(pair(hx, i), s2);
        fb[i] = fadd2(pair(hm, i), ls2);
        asm volatile("" : "+f"(fa[i].x), "+f"(fa[i].y), "+f"(fb[i].x), "+f"(fb[i].y));
      }
      bad |= !mbar_wait(smem_u32(&sh.s_full), k & 1, a.status, 522, &abort_flag);
      __syncwarp();
      float2 e[HT / 2];
      {
        tc_fence_after();
        uint32_t xh[HT], xl[HT];
        tmem_ld16(tS, xh);
        tmem_ld16(tS + NH, xl);
        tmem_wait_ld();
        tc_fence_before();
        mbar_arrive_warp(smem_u32(&sh.s_free));
#pragma unroll
        for (int i = 0; i < HT / 2; ++i)
          e[i] = ffma2(ffma2(f2(xl, i), make_float2(0.0625f, 0.0625f), f2(xh, i)), fa[i], fb[i]);
      }
      if (!valid) {  // (whatever the row held)
#pragma unroll
        for (int i = 0; i < HT / 2; ++i) e[i] = make_float2(-INFINITY, -INFINITY);
      }
      float mx = fmaxf(e[0].x, e[0].y);
#pragma unroll
      for (int i = 1; i < HT / 2; ++i) mx = fmax3(mx, e[i].x, e[i].y);
      bool look = false;
      if (k % kLook == kLook - 1) {
        float mn = INFINITY;
#pragma unroll
        for (int i = 0; i < HT / 2; ++i) mn = fmin3(mn, e[i].x, e[i].y);
        if (__any_sync(0xffffffffu, valid && mn < kLow)) {
#pragma unroll
          for (int i = 0; i < HT; ++i)  // a head without any above, in this warp at least
            look |= !__any_sync(0xffffffffu, (i & 1 ? e[i / 2].y : e[i / 2].x) >= kLow);
          look = look && __any_sync(0xffffffffu, valid);
        }
      }
      if (grp_or(mx > kBase + kThr || first || look || bad)) {
        if (grp_or(bad)) {
          ok = false;
          break;
        }
        // Some head's reference may have to move. It goes up to the tile's maximum of S + log2 s
        auto e1 = [&](int i) { return i & 1 ? e[i / 2].y : e[i / 2].x; };
        auto v1 = [&](int i) { return e1(i) - hm1[i]; };  // S + log2 s
        const int h1 = hb + (tl & (HT - 1));  // threads below HT: their head
        auto tile_max = [&]() { return fmaxf(fmaxf(sh.wmax[0][h1], sh.wmax[1][h1]), fmaxf(sh.wmax[2][h1], sh.wmax[3][h1])); };
#pragma unroll
        for (int i = 0; i < HT; ++i) {
          const float v = warp_max(v1(i));  // (-inf where the token is not visible)
          if (lane == 0) sh.wmax[q4][hb + i] = v;
        }
        look = grp_or(look);
        if (look) {
#pragma unroll
          for (int i = 0; i < HT; ++i) {
            const int h = hb + i;
            const float tm = fmaxf(fmaxf(sh.wmax[0][h], sh.wmax[1][h]), fmaxf(sh.wmax[2][h], sh.wmax[3][h]));
            const uint32_t near = __ballot_sync(0xffffffffu, valid && v1(i) >= tm - kGap);
            if (lane == 0) sh.small[q4][h] = __popc(near);
          }
          grp_sync();
        }
        float m_old = 0.f, ref = 0.f;
        bool resc = false;
        auto move_to = [&](float to) {
          sh.move[h1] = ref - to;
          ref = to;
          resc = !first && ref != m_old;
          sh.alpha[h1] = first ? 0.f : ex2_approx(m_old - ref);
          hm1[tl] = kBase - ref;
        };
        if (tl < HT) {
          const float tm = tile_max();
          m_old = ref = kBase - hm1[tl];
          float to = ref;
          if (tm > m_old || (first && tm > -INFINITY)) {  // (a first tile of NaN leaves it at 0)
            to = tm;
          } else if (look && tm < m_old + (kLow - kBase)) {
            const int near = (sh.small[0][h1] + sh.small[1][h1]) + (sh.small[2][h1] + sh.small[3][h1]);
            const int seen = min(w.st.Tb, w.token0(t) + TT) - max(w.st.lo, w.token0(t));
            if (near * kCrowd >= seen) to = tm + kRoom;
          }
          move_to(fmaxf(to, sh.top[h1] - kSpan));
          sh.top[h1] = fmaxf(sh.top[h1], ref);
        }
        bool any = grp_or(resc);  // (also publishes hm and alpha)
        auto rescore = [&]() {
#pragma unroll
          for (int i = 0; i < HT / 2; ++i) e[i] = fadd2(e[i], make_float2(sh.move[hb + 2 * i], sh.move[hb + 2 * i + 1]));
        };
        rescore();
        float low = INFINITY;
#pragma unroll
        for (int i = 0; i < HT / 2; ++i) low = fmin3(low, e[i].x, e[i].y);
        bool few = false, out = false;
        float rise = INFINITY;
#pragma unroll
        for (int i = 0; i < HT; ++i) rise = fminf(rise, sh.move[hb + i]);
        if ((first || rise <= -kRise) && __any_sync(0xffffffffu, valid && low < kLow)) {
          // kFew of a full tile: some warp has kFew / 4 at most. (No branches between the votes)
          const int lim = w.token0(t) >= w.st.lo && w.token0(t) + TT <= w.st.Tb ? kFew / 4 : kFew;
#pragma unroll
          for (int i = 0; i < HT; ++i) {
            const int n_big = __popc(__ballot_sync(0xffffffffu, e1(i) >= kLow));
            few |= (n_big <= lim) & (e1(i) < kLow) & (first | (sh.move[hb + i] <= -kRise));
          }
          few &= valid;
        }
        if (grp_or(few)) {
          // the few that are far above all the others
#pragma unroll
          for (int i = 0; i < HT; ++i) {
            const float v = v1(i), x = e1(i);
            const uint32_t big = __ballot_sync(0xffffffffu, x >= kLow);
            const uint32_t small = __ballot_sync(0xffffffffu, valid && x < kLow);
            const float mx_small = warp_max(x < kLow ? v : -INFINITY);
            const float mn_big = -warp_max(x >= kLow ? -v : -INFINITY);
            if (lane == 0) {
              sh.big[q4][hb + i] = big;
              sh.small[q4][hb + i] = __popc(small);
              sh.wmax[q4][hb + i] = mx_small;
              sh.wmin[q4][hb + i] = mn_big;
            }
          }
          grp_sync();
          int n_big = 0, n_small = 0;
          float lower = 0.f;
          bool far = false;
          if (tl < HT) {
            for (int q = 0; q < 4; ++q) {
              n_big += __popc(sh.big[q][h1]);
              n_small += sh.small[q][h1];
            }
            const float over = fminf(fminf(sh.wmin[0][h1], sh.wmin[1][h1]), fminf(sh.wmin[2][h1], sh.wmin[3][h1]));
            const float rest = tile_max();
            far = over - rest >= kFar;
            lower = fmaxf(rest + kRoom, sh.top[h1] - kSpan);
            out = n_big > 0 && n_big <= kFew && n_small > 0 && over - rest >= kGap && lower < ref;
            sh.wmin[0][h1] = out ? rest - kGap : INFINITY;
            sh.n_out[h1] = 0;
            sh.move[h1] = 0.f;
          }
          if (grp_or(out)) {
#pragma unroll
            for (int i = 0; i < HT; ++i) {
              const uint32_t near = __ballot_sync(0xffffffffu, e1(i) < kLow && v1(i) >= sh.wmin[0][hb + i]);
              if (lane == 0) sh.small[q4][hb + i] = __popc(near);
            }
            grp_sync();
            if (tl < HT) {
              const int near = (sh.small[0][h1] + sh.small[1][h1]) + (sh.small[2][h1] + sh.small[3][h1]);
              const bool crowd = near * kCrowd >= n_small;
              out = out && (far || crowd);
              if (out) {
                sh.n_out[h1] = n_big;
                move_to(crowd ? lower : lower + kRoom);
              }
            }
          }
          out = grp_or(out);
          any = grp_or(resc);
          rescore();
        }
#pragma unroll
        for (int i = 0; i < HT / 2; ++i)
          lp[i] = fmul2(lp[i], make_float2(sh.alpha[hb + 2 * i], sh.alpha[hb + 2 * i + 1]));
        // O^T holds the tiles before k once the value MMAs of tile k - 1 have landed
        if ((any || out) && k >= 1) {
          bad |= !mbar_wait(smem_u32(&sh.p_free), (k - 1) & 1, a.status, 523, &abort_flag);
          __syncwarp();
          tc_fence_after();
        }
        if (any) {
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {  // M-tile c / 2, hi or lo columns
            uint32_t o[HT];
            const uint32_t ta = tmem + lane_base + NQ * (1 + (c >> 1)) + NH * (c & 1) + hb;
            tmem_ld16(ta, o);
            tmem_wait_ld();
#pragma unroll
            for (int h = 0; h < HT; ++h) o[h] = __float_as_uint(__uint_as_float(o[h]) * sh.alpha[hb + h]);
            tmem_st16(ta, o);
          }
          tmem_wait_st();
        }
        if (out) {
          // this token's weights where it is one of the few; those go into the sum here, and to
          // O^T in the order of the tokens, a batch of tokens at a time
          uint32_t mine = 0;
#pragma unroll
          for (int i = 0; i < HT; ++i)
            if (sh.n_out[hb + i] > 0) mine |= ((sh.big[q4][hb + i] >> lane) & 1u) << i;
          const uint32_t mask = __ballot_sync(0xffffffffu, mine != 0);
          if (lane == 0) sh.out_mask[grp][q4] = mask;
          // (the tile's rows, which only the MMAs have waited for so far)
          bad |= !mbar_wait(smem_u32(&sh.full[k % STAGES]), (k / STAGES) & 1, a.status, 526, &abort_flag);
          __syncwarp();
          grp_sync();
          int at = __popc(mask & ((1u << lane) - 1u)), n = 0;
          for (int q = 0; q < 4; ++q) {
            if (q < q4) at += __popc(sh.out_mask[grp][q]);
            n += __popc(sh.out_mask[grp][q]);
          }
#pragma unroll 1
          for (int n0 = 0; n0 < n; n0 += kBatch) {
            if (mine && at >= n0 && at < n0 + kBatch) {
              float* to = reinterpret_cast<float*>(sh.out_w[grp][at - n0]);
              sh.out_row[grp][at - n0] = tl;
#pragma unroll
              for (int i = 0; i < HT; ++i) {
                const bool one = (mine >> i) & 1u;
                float& x = i & 1 ? e[i / 2].y : e[i / 2].x;
                float& l = i & 1 ? lp[i / 2].y : lp[i / 2].x;
                const float p = one ? ex2_approx(x) : 0.f;
                to[i] = p;
                l = fmaf(p, inv_s, l);
                if (one) x = -INFINITY;  // (its weight in the MMA is 0)
              }
            }
            grp_sync();
#pragma unroll 1
            for (int mt = 0; mt < 4; ++mt) {
              uint32_t o[HT];
              const uint32_t ta = tmem + lane_base + NQ * (1 + mt) + hb;
              tmem_ld16(ta, o);
              tmem_wait_ld();
              const uint8_t* box = tiles + (k % STAGES) * TILE + mt * BOX;
#pragma unroll 1
              for (int u = 0; u < min(kBatch, n - n0); ++u) {
                const int r = sh.out_row[grp][u];  // row r, column tl of the box
                const uint32_t byte = box[r * 128 + (((tl >> 4) ^ (r & 7)) << 4) + (tl & 15)];
                const float c = __low2float(e4m3x2_to_half2(byte));
#pragma unroll
                for (int q = 0; q < HT / 4; ++q) {
                  const float4 p = sh.out_w[grp][u][q];
                  o[4 * q] = __float_as_uint(fmaf(p.x, c, __uint_as_float(o[4 * q])));
                  o[4 * q + 1] = __float_as_uint(fmaf(p.y, c, __uint_as_float(o[4 * q + 1])));
                  o[4 * q + 2] = __float_as_uint(fmaf(p.z, c, __uint_as_float(o[4 * q + 2])));
                  o[4 * q + 3] = __float_as_uint(fmaf(p.w, c, __uint_as_float(o[4 * q + 3])));
                }
              }
              tmem_st16(ta, o);
            }
            tmem_wait_st();
            grp_sync();
          }
        }
      }
      // weights of this token: hi and lo bytes of 16 heads
      uint32_t wh[HT / 4], wl[HT / 4];
#pragma unroll
      for (int q = 0; q < HT / 4; ++q) {
        uint32_t h[2], l[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float2 p = make_float2(ex2_approx(e[2 * q + u].x), ex2_approx(e[2 * q + u].y));
          lp[2 * q + u] = ffma2(p, i2, lp[2 * q + u]);
          split_weights(p.x, p.y, h[u], l[u]);
        }
        wh[q] = h[0] | (h[1] << 16);
        wl[q] = l[0] | (l[1] << 16);
      }
      // a row that is not visible may hold anything: its weight is zero, but 0 x NaN is NaN
      if (!valid) {
        uint8_t* tb = tiles + (k % STAGES) * TILE + tl * 128;
        for (int bx = grp; bx < 4; bx += HG)
#pragma unroll
          for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(tb + bx * BOX + c * 16) = make_uint4(0, 0, 0, 0);
      }
      // the weights of tile k - 1 have been consumed
      if (k >= 1) bad |= !mbar_wait(smem_u32(&sh.p_free), (k - 1) & 1, a.status, 524, &abort_flag);
      __syncwarp();
      // token row of 128 bytes, 16-byte chunks (16 heads: hi of the groups, then lo) swizzled
      // by the token's low bits
      *reinterpret_cast<uint4*>(ps + tl * 128 + ((grp ^ (tl & 7)) << 4)) = make_uint4(wh[0], wh[1], wh[2], wh[3]);
      *reinterpret_cast<uint4*>(ps + tl * 128 + (((HG + grp) ^ (tl & 7)) << 4)) = make_uint4(wl[0], wl[1], wl[2], wl[3]);
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive_warp(smem_u32(&sh.p_full));

      if (last) {
        // ---- partial of this sequence share: (M, l) per head and O^T
        const bool d_ok = mbar_wait(smem_u32(&sh.seg_done), seg & 1, a.status, 525, &abort_flag);
        if (grp_or(!d_ok || bad)) {
          ok = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < HT / 2; ++i) {
          float2 v = lp[i];
#pragma unroll
          for (int o = 16; o; o >>= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
          }
          if (lane == 0) {
            sh.wmax[q4][hb + 2 * i] = v.x;
            sh.wmax[q4][hb + 2 * i + 1] = v.y;
          }
        }
        grp_sync();
        const long long rec = ((long long)(r + w.b) * a.n_hg + hg) * NH;
        if (tl < HT && hb + tl < nh) {
          const int h = hb + tl;
          a.part_ml[(rec + h) * 2 + 0] = kBase - hm1[tl];
          a.part_ml[(rec + h) * 2 + 1] = (sh.wmax[0][h] + sh.wmax[1][h]) + (sh.wmax[2][h] + sh.wmax[3][h]);
        }
#pragma unroll 1
        for (int mt = 0; mt < 4; ++mt) {
          uint32_t oh[HT], ol[HT];
          const uint32_t ta = tmem + lane_base + NQ * (1 + mt) + hb;
          tmem_ld16(ta, oh);
          tmem_ld16(ta + NH, ol);
          tmem_wait_ld();
          float* dst = a.part_o + (rec + hb) * DC + mt * 128 + tl;
#pragma unroll
          for (int h = 0; h < HT; ++h)
            if (hb + h < nh) dst[h * DC] = fmaf(__uint_as_float(ol[h]), 0.0625f, __uint_as_float(oh[h]));
        }
        clear_o();
        tc_fence_before();
        grp_sync();
      }
    }
    if (!ok || bad) abort_flag = 1;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- absorb
// q~ = tau log2e [W_UK q_nope | RoPE(q_rope)], quantised into the split kernel's images. For
// KV group h and 128 query rows (row = (sequence b, head u of the group)) a cluster of four
// CTAs computes the 512 latent columns, 128 each, on the tensor cores; the largest magnitude
// of a row is exchanged through distributed shared memory, so that the row is scaled by one
// power of two and written once. Each CTA adds a quarter of the rotary part.
namespace q8 {
constexpr int AB = kQdecAbsorbRows;
static_assert(DC / AB == kQdecAbsorbSplit, "one CTA of the cluster for each 128 columns");
constexpr int AB_OP = AB * AB * 2;  // an operand: two 64-column chunks of [128 rows x 128 B]
constexpr int AB_SMEM = 2 * AB_OP + 64;
struct AbsorbArgs {
  int B, T_max, n_kv, g, H_q, n_hg, hpc, NH;  // NH: heads of an image (kQdecHeads at most)
  float isc;
  const __nv_bfloat16* q;
  const int* seqlens;
  const float* cos_tab;
  const float* sin_tab;
  uint8_t* qimg;
  int* status;
  int* failed;
};
// byte of dimension d of image row (hi: head; lo: NH + head)
__device__ __forceinline__ int image_offset(int NH, int row, int d) {
  return d < DC ? (d >> 7) * (2 * NH * 128) + row * 128 + ((((d & 127) >> 4) ^ (row & 7)) << 4) + (d & 15)
                : 4 * (2 * NH * 128) + row * 64 + ((((d - DC) >> 4) ^ ((row >> 1) & 3)) << 4) + (d & 15);
}
// values (already divided by the row's scale) into the hi and lo rows
__device__ __forceinline__ void split4(const float* x, uint32_t& hi, uint32_t& lo) {
  uint32_t hh[2], ll[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    hh[u] = e4m3x2(x[2 * u], x[2 * u + 1]);
    const float2 f = __half22float2(e4m3x2_to_half2(hh[u]));
    ll[u] = e4m3x2((x[2 * u] - f.x) * 16.f, (x[2 * u + 1] - f.y) * 16.f);
  }
  hi = hh[0] | (hh[1] << 16);
  lo = ll[0] | (ll[1] << 16);
}
__device__ __forceinline__ void store16(uint8_t* img, int NH, int head, int d, const float (&x)[16]) {
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) split4(x + 4 * q, hi[q], lo[q]);
  *reinterpret_cast<uint4*>(img + image_offset(NH, head, d)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  *reinterpret_cast<uint4*>(img + image_offset(NH, NH + head, d)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}
__device__ __forceinline__ void store8(uint8_t* img, int NH, int head, int d, const float (&x)[8]) {
  uint32_t hi[2], lo[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) split4(x + 4 * q, hi[q], lo[q]);
  *reinterpret_cast<uint2*>(img + image_offset(NH, head, d)) = make_uint2(hi[0], hi[1]);
  *reinterpret_cast<uint2*>(img + image_offset(NH, NH + head, d)) = make_uint2(lo[0], lo[1]);
}
}  // namespace q8

__global__ void __cluster_dims__(1, 1, 4) __launch_bounds__(256, 1)
    qdecode_absorb_kernel(const __grid_constant__ CUtensorMap tmW, const q8::AbsorbArgs a) {
  using namespace sm100;
  using namespace q8;
  // The call's status word, before the split kernel can report to it. Nothing orders this store
  // and the other CTAs of this grid, so they neither read the word nor report to it: each leaves
  // its own record of a failure (0: none), which the split kernel reports
  int* const failed = a.failed + (blockIdx.y * gridDim.x + blockIdx.x) * gridDim.z + blockIdx.z;
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x < kStatusBytes / 4) {
    a.status[threadIdx.x] = 0;
    __threadfence();
  }
  __syncthreads();
  grid_dep_launch();
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* as = smem;
  uint8_t* bs = smem + AB_OP;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + 2 * AB_OP);  // [0] W landed, [1] MMAs done
  __shared__ uint32_t tmem_slot;
  __shared__ int w_landed;
  __shared__ float part_max[2][AB], row_max[AB];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x, z = blockIdx.z;
  const int G1 = a.g + 1, n_S = a.g * a.n_kv, rows = a.B * G1, r0 = blockIdx.y * AB;
  const int NH = a.NH, img_data = qdec_image_data(NH), img_bytes = qdec_image_bytes(NH);
  // (the cluster's CTAs have the same shared-memory layout: all four or none pass this)
  if (smem_u32(smem) & 1023u) {
    if (tid == 0) *failed = kAbsorbAlignment;
    return;
  }
  if (tid == 0) {
    w_landed = 0;
    mbar_init(smem_u32(&bar[0]), 1);
    mbar_init(smem_u32(&bar[1]), 1);
    fence_mbar_init();
    prefetch_tmap(&tmW);
    mbar_expect_tx(smem_u32(&bar[0]), AB_OP);
    for (int kc = 0; kc < 2; ++kc)
      tma_load_2d(smem_u32(bs + kc * (AB_OP / 2)), &tmW, smem_u32(&bar[0]), h * 256 + kc * 64, z * AB);
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&tmem_slot), AB);
    tmem_relinquish();
  }
  auto head_of = [&](int u) { return u < a.g ? h * a.g + u : n_S + h; };
  constexpr int kPieces = AB * 16 / 256;
  uint4 qv[kPieces];
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int e = tid + 256 * u, rr = e >> 4, pc = e & 15, R = r0 + rr;
    qv[u] = make_uint4(0, 0, 0, 0);
    if (R < rows)
      qv[u] = *reinterpret_cast<const uint4*>(a.q + ((long long)(R / G1) * a.H_q + head_of(R % G1)) * 192 + pc * 8);
  }
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int e = tid + 256 * u, rr = e >> 4, pc = e & 15;
    *reinterpret_cast<uint4*>(as + (pc >> 3) * (AB_OP / 2) + rr * 128 + (((pc & 7) ^ (rr & 7)) << 4)) = qv[u];
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  if (tid == 32) {
    if (mbar_wait(smem_u32(&bar[0]), 0, nullptr, 0)) {
      w_landed = 1;
      tc_fence_after();
      constexpr uint32_t id = idesc_bf16_f32(AB, AB, false, false);
#pragma unroll
      for (int kk = 0; kk < AB / 16; ++kk) {
        const uint32_t off = (uint32_t)((kk & 3) * 32);
        mma_ss(tmem, sdesc_sw128(smem_u32(as + (kk >> 2) * (AB_OP / 2)) + off, 16, 1024),
               sdesc_sw128(smem_u32(bs + (kk >> 2) * (AB_OP / 2)) + off, 16, 1024), id, kk > 0);
      }
    } else {
      mbar_wait(smem_u32(&bar[0]), 0, nullptr, 0);  // no copy is in flight at exit
    }
    mma_commit(smem_u32(&bar[1]));
  }
  __syncwarp();
  const int q4 = warp & 3, ch = warp >> 2;  // TMEM lane quarter; half of the 128 columns
  const int rl = q4 * 32 + lane, R = r0 + rl;
  const bool real = R < rows;
  const int b = real ? R / G1 : 0, head = real ? head_of(R % G1) : 0;
  // this CTA's rotary pairs (k, k + 32), k = 8z .. 8z + 7, at position seqlen - 1
  const bool rot = ch == 0 && real;
  float lo[8], hi[8], mx = 0.f;
  if (rot) {
    const int pos = min(max(__ldg(a.seqlens + b), 1), a.T_max) - 1;
    const __nv_bfloat16* qr = a.q + ((long long)b * a.H_q + head) * 192 + 128 + 8 * z;
    const uint4 xl = *reinterpret_cast<const uint4*>(qr), xh = *reinterpret_cast<const uint4*>(qr + 32);
    const float4* c4 = reinterpret_cast<const float4*>(a.cos_tab + (long long)pos * 32 + 8 * z);
    const float4* s4 = reinterpret_cast<const float4*>(a.sin_tab + (long long)pos * 32 + 8 * z);
    const float4 cq[2] = {__ldg(c4), __ldg(c4 + 1)}, sq[2] = {__ldg(s4), __ldg(s4 + 1)};
    const float* cs = reinterpret_cast<const float*>(cq);
    const float* sn = reinterpret_cast<const float*>(sq);
    const __nv_bfloat162* l2 = reinterpret_cast<const __nv_bfloat162*>(&xl);
    const __nv_bfloat162* h2 = reinterpret_cast<const __nv_bfloat162*>(&xh);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 x1 = __bfloat1622float2(l2[e]), x2 = __bfloat1622float2(h2[e]);
      lo[2 * e] = (x1.x * cs[2 * e] - x2.x * sn[2 * e]) * a.isc;
      lo[2 * e + 1] = (x1.y * cs[2 * e + 1] - x2.y * sn[2 * e + 1]) * a.isc;
      hi[2 * e] = (x2.x * cs[2 * e] + x1.x * sn[2 * e]) * a.isc;
      hi[2 * e + 1] = (x2.y * cs[2 * e + 1] + x1.y * sn[2 * e + 1]) * a.isc;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fmaxf(fabsf(lo[e]), fabsf(hi[e])));
  }
  const bool done = mbar_wait(smem_u32(&bar[1]), 0, nullptr, 0);
  __syncwarp();
  tc_fence_after();
  uint32_t v0[32], v1[32];
  tmem_ld32(tmem + ((uint32_t)(q4 * 32) << 16) + ch * 64, v0);
  tmem_ld32(tmem + ((uint32_t)(q4 * 32) << 16) + ch * 64 + 32, v1);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    v0[i] = __float_as_uint(__uint_as_float(v0[i]) * a.isc);
    v1[i] = __float_as_uint(__uint_as_float(v1[i]) * a.isc);
    mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(v0[i])), fabsf(__uint_as_float(v1[i]))));
  }
  part_max[ch][rl] = mx;
  __syncthreads();
  if (tid < AB) row_max[tid] = fmaxf(part_max[0][tid], part_max[1][tid]);
  cluster_sync();
  float top = 0.f;
#pragma unroll
  for (uint32_t c = 0; c < 4; ++c) top = fmaxf(top, ld_shared_cluster(mapa_shared(smem_u32(&row_max[rl]), c)));
  // the row's scale: a power of two with top <= 448 scale (448 = 1.75 2^8)
  int ex = 0;
  if (top > 0.f && top < INFINITY) {
    const uint32_t u = __float_as_uint(top);
    ex = max((int)(u >> 23) - 127 - ((u & 0x7FFFFFu) <= 0x600000u ? 8 : 7), -100);
  }
  const float inv = __int_as_float((127 - ex) << 23);
  if (real && done && w_landed) {
    const int hgi = head / a.hpc, lh = head - hgi * a.hpc;
    uint8_t* img = a.qimg + ((long long)b * a.n_hg + hgi) * img_bytes;
    // (an infinity would saturate: a query that is not finite gives NaN, as its scores would)
    const float bad = top < INFINITY ? 0.f : NAN;
    float x[16];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        x[i] = fmaf(__uint_as_float(c < 2 ? v0[16 * (c & 1) + i] : v1[16 * (c & 1) + i]), inv, bad);
      store16(img, NH, lh, z * AB + ch * 64 + 16 * c, x);
    }
    if (rot) {
      if (z == 0) *reinterpret_cast<float*>(img + img_data + 4 * lh) = __int_as_float((127 + ex) << 23);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        lo[e] = fmaf(lo[e], inv, bad);
        hi[e] = fmaf(hi[e], inv, bad);
      }
      store8(img, NH, lh, DC + 8 * z, lo);
      store8(img, NH, lh, DC + 32 + 8 * z, hi);
    }
  }
  // image rows of the padding heads of each head group are zero (their scale is 1): the blocks
  // of KV group 0 clear them for the sequences whose first row falls in their tile
  if (h == 0 && z == 0) {
    const int b_lo = (r0 + G1 - 1) / G1, b_hi = min(a.B, (r0 + AB + G1 - 1) / G1);
    for (int bb = b_lo; bb < b_hi; ++bb)
      for (int hg2 = 0; hg2 < a.n_hg; ++hg2) {
        const int nhd = min(a.hpc, a.H_q - hg2 * a.hpc);
        uint8_t* im = a.qimg + ((long long)bb * a.n_hg + hg2) * img_bytes;
        for (int e = tid; e < (NH - nhd) * 72; e += 256) {
          const int lh = nhd + e / 72, c = e % 72, part = c / 36, d = (c % 36) * 16;
          *reinterpret_cast<uint4*>(im + image_offset(NH, part * NH + lh, d)) = make_uint4(0, 0, 0, 0);
          if (c == 0) *reinterpret_cast<float*>(im + img_data + 4 * lh) = 1.f;
        }
      }
  }
  cluster_sync();  // (no CTA of the cluster leaves while another reads its row maxima)
  tc_fence_before();
  const bool all_done = __syncthreads_and(done);
  tc_fence_after();
  if (tid == 0) *failed = !w_landed ? kAbsorbLoad : !all_done ? kAbsorbMma : 0;
  if (warp == 0) tmem_dealloc(tmem, AB);
}

// --------------------------------------------------------------- combine
// Merge of the partials, W_UV product and output epilogue. Block = (KV group h, whole
// sequences: up to 32 query rows, row = (sequence b, head u of the group)):
//   O_lat = sum_s 2^(M_s - M) O_s / sum_s 2^(M_s - M) l_s;  H = O_lat W_UV;
//   D = H_S - sigmoid(lambda) H_N;  Y = sigmoid(G) D.
// The product runs on the tensor cores with O_lat as the sum of two bf16 values, rows 0..31
// of the M = 64 operand the rounded ones and rows 32..63 what the rounding left, added in the
// epilogue: the difference of two heads with nearly equal outputs keeps its precision.
namespace q8 {
constexpr int CB_R = 32, CB_N = 128;
constexpr int CB_A = 64 * DC * 2;        // 8 chunks of [64 rows x 128 B]
constexpr int CB_B = DC * CB_N * 2;      // 2 MN blocks of [512 K rows x 128 B]
constexpr int CB_W = CB_R * kQdecSMs * 4;  // weights of a row's partials
constexpr int CB_SMEM = CB_A + CB_B + CB_W + 64;
constexpr int CB_T = 512;
struct CombineArgs {
  int B, T_max, n_kv, g, H_q, n_hg, hpc, NH, n_ranges, spb;
  const int* seqlens;
  const int2* seqinfo;
  const float* part_o;
  const float* part_ml;
  const float* lam;
  const __nv_bfloat16* gate;
  __nv_bfloat16* out;
  int* status;
};
}  // namespace q8

__global__ void __launch_bounds__(q8::CB_T, 1)
    qdecode_combine_kernel(const __grid_constant__ CUtensorMap tmW, const q8::CombineArgs a) {
  using namespace sm100;
  using namespace q8;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* as = smem;         // O_lat; later H (fp32 [64 x 128])
  uint8_t* bs = smem + CB_A;  // W_UV,h
  float* wgt = reinterpret_cast<float*>(smem + CB_A + CB_B);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + CB_A + CB_B + CB_W);
  __shared__ long long rec0[CB_R];
  __shared__ int n_parts[CB_R];
  __shared__ uint32_t tmem_slot;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(smem) & 1023u) {
    if (tid == 0) {
      atomicCAS(a.status, 0, (int)GDLA_ERR_CUDA);
      atomicCAS(a.status + 1, 0, 597);
    }
    grid_dep_wait();
    return;
  }
  const int h = blockIdx.x, G1 = a.g + 1, n_S = a.g * a.n_kv;
  const int b0 = blockIdx.y * a.spb, nb = min(a.spb, a.B - b0), R = nb * G1;
  const long long rstep = (long long)a.n_hg * a.NH;
  if (tid == 0) {
    mbar_init(smem_u32(&bar[0]), 1);
    mbar_init(smem_u32(&bar[1]), 1);
    fence_mbar_init();
    prefetch_tmap(&tmW);
    mbar_expect_tx(smem_u32(&bar[0]), CB_B);
    for (int j = 0; j < 2; ++j)
      for (int kh = 0; kh < 2; ++kh)
        tma_load_2d(smem_u32(bs + j * (CB_B / 2) + kh * (CB_B / 4)), &tmW, smem_u32(&bar[0]), h * 256 + 128 + 64 * j,
                    256 * kh);
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&tmem_slot), CB_N);
    tmem_relinquish();
  }
  // lambda and the gate logits of this thread's eight outputs (inputs of the caller)
  const int e_out = tid, n_out = nb * a.g * (CB_N / 8);  // (at most 32 x 16)
  const int o_bl = e_out / (a.g * (CB_N / 8)), o_u = (e_out / (CB_N / 8)) % a.g, o_c = e_out % (CB_N / 8);
  const long long o_idx = ((long long)(b0 + o_bl) * n_S + h * a.g + o_u) * CB_N + o_c * 8;
  uint4 gv = make_uint4(0, 0, 0, 0);
  float lamv = 0.f;
  if (e_out < n_out) {
    gv = *reinterpret_cast<const uint4*>(a.gate + o_idx);
    lamv = sigmoidf_(__ldg(a.lam + (long long)(b0 + o_bl) * n_S + h * a.g + o_u));
  }
  grid_dep_wait();  // the partials come from the split kernel
  if (tid < CB_R) {
    n_parts[tid] = 0;
    rec0[tid] = 0;
    if (tid < R) {
      const int b = b0 + tid / G1, u = tid % G1, head = u < a.g ? h * a.g + u : n_S + h;
      const int hgi = head / a.hpc, lh = head - hgi * a.hpc;
      if (__ldg(a.seqlens + b) > 0) {
        // first and last share of the sequence (clamped: a call whose split kernel gave up
        // early still reads inside the records); an empty sequence has none and gives zeros
        const int2 info = a.seqinfo[b];
        const int x = min(max(info.x, 0), a.n_ranges - 1), y = min(max(info.y, x), a.n_ranges - 1);
        rec0[tid] = ((long long)(x + b) * a.n_hg + hgi) * a.NH + lh;
        n_parts[tid] = y - x + 1;
      }
    }
  }
  __syncthreads();
  // weights of a row's partials: one warp per row
  for (int r = warp; r < R; r += CB_T / 32) {
    const int np = n_parts[r];
    const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + rec0[r];
    float* wr = wgt + r * kQdecSMs;
    constexpr int kPL = (kQdecSMs + 31) / 32;  // partials of a lane
    float2 v[kPL];
    float M = -INFINITY;
#pragma unroll
    for (int q = 0; q < kPL; ++q) {
      v[q] = lane + 32 * q < np ? ml[(lane + 32 * q) * rstep] : make_float2(-INFINITY, 0.f);
      M = fmaxf(M, v[q].x);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float den = 0.f;
#pragma unroll
    for (int q = 0; q < kPL; ++q) {
      // (an l that is NaN, of a share that saw one, is passed on)
      const float f = v[q].x == -INFINITY ? 1.f : exp2f(v[q].x - M);
      den += f * v[q].y;
      v[q].x = f;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    const float inv = den == 0.f ? 0.f : 1.f / den;
#pragma unroll
    for (int q = 0; q < kPL; ++q)
      if (lane + 32 * q < np) wr[lane + 32 * q] = v[q].x * inv;
  }
  __syncthreads();
  constexpr int kMB = 8;  // partials in flight per thread
  for (int e = tid; e < CB_R * (DC / 8); e += CB_T) {
    const int r = e / (DC / 8), c8 = e % (DC / 8);
    float acc[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] = 0.f;
    if (r < R) {
      const int np = n_parts[r];
      const float* src = a.part_o + rec0[r] * DC + c8 * 8;
      const float* wr = wgt + r * kQdecSMs;
      for (int sp0 = 0; sp0 < np; sp0 += kMB) {
        float4 x[kMB][2];
#pragma unroll
        for (int q = 0; q < kMB; ++q) {
          x[q][0] = x[q][1] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (sp0 + q < np) {
            const float4* s4 = reinterpret_cast<const float4*>(src + (sp0 + q) * rstep * DC);
            x[q][0] = s4[0];
            x[q][1] = s4[1];
          }
        }
#pragma unroll
        for (int q = 0; q < kMB; ++q) {
          if (sp0 + q >= np) continue;
          const float f = wr[sp0 + q];
          acc[0] = fmaf(f, x[q][0].x, acc[0]); acc[1] = fmaf(f, x[q][0].y, acc[1]);
          acc[2] = fmaf(f, x[q][0].z, acc[2]); acc[3] = fmaf(f, x[q][0].w, acc[3]);
          acc[4] = fmaf(f, x[q][1].x, acc[4]); acc[5] = fmaf(f, x[q][1].y, acc[5]);
          acc[6] = fmaf(f, x[q][1].z, acc[6]); acc[7] = fmaf(f, x[q][1].w, acc[7]);
        }
      }
    }
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      hi[q] = pack_bf16x2(acc[2 * q], acc[2 * q + 1]);
      const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&hi[q]));
      lo[q] = pack_bf16x2(acc[2 * q] - f.x, acc[2 * q + 1] - f.y);
    }
    uint8_t* at = as + (c8 >> 3) * (64 * 128) + r * 128 + (((c8 & 7) ^ (r & 7)) << 4);
    *reinterpret_cast<uint4*>(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(at + CB_R * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  if (tid == 32) {
    if (mbar_wait(smem_u32(&bar[0]), 0, a.status, 551)) {
      tc_fence_after();
      constexpr uint32_t id = idesc_bf16_f32(64, CB_N, false, true);
#pragma unroll
      for (int kk = 0; kk < DC / 16; ++kk)
        mma_ss(tmem, sdesc_sw128(smem_u32(as + (kk >> 2) * (64 * 128)) + (kk & 3) * 32, 16, 1024),
               sdesc_sw128(smem_u32(bs) + kk * 2048, CB_B / 2, 1024), id, kk > 0);
    } else {
      mbar_wait(smem_u32(&bar[0]), 0, nullptr, 0);  // no copy is in flight at exit
    }
    mma_commit(smem_u32(&bar[1]));
  }
  __syncwarp();
  const bool done = mbar_wait(smem_u32(&bar[1]), 0, a.status, 552);
  __syncwarp();
  tc_fence_after();
  // the M = 64 accumulator: row 16 q + l in lane l < 16 of quarter q
  float* hs = reinterpret_cast<float*>(as);
  {
    const int q4 = warp & 3, c = warp >> 2;
    uint32_t v[32];
    tmem_ld32(tmem + ((uint32_t)(q4 * 32) << 16) + c * 32, v);
    tmem_wait_ld();
    if (lane < 16) {
      float* dst = hs + (q4 * 16 + lane) * CB_N + c * 32;
#pragma unroll
      for (int q = 0; q < 8; ++q)
        reinterpret_cast<float4*>(dst)[q] = make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]),
                                                        __uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3]));
    }
  }
  __syncthreads();
  if (e_out < n_out && done && !earlier_failure(a.status)) {
    const __nv_bfloat162* g2 = reinterpret_cast<const __nv_bfloat162*>(&gv);
    const float* hsr = hs + (o_bl * G1 + o_u) * CB_N + o_c * 8;
    const float* hnr = hs + (o_bl * G1 + a.g) * CB_N + o_c * 8;
    uint32_t o[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 gf = __bfloat1622float2(g2[q]);
      float d[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        d[i] = (hsr[2 * q + i] + hsr[CB_R * CB_N + 2 * q + i]) - lamv * (hnr[2 * q + i] + hnr[CB_R * CB_N + 2 * q + i]);
      o[q] = pack_bf16x2(d[0] * sigmoidf_(gf.x), d[1] * sigmoidf_(gf.y));
    }
    *reinterpret_cast<uint4*>(a.out + o_idx) = make_uint4(o[0], o[1], o[2], o[3]);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, CB_N);
}

// ---------------------------------------------------------------- launches
namespace {

template <auto K, typename... A>
cudaError_t launch_dependent(dim3 grid, int threads, int smem, cudaStream_t s, A... args) {
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(K, smem, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, K, args...);
}

bool w_map(CUtensorMap* m, const DecodeParams& d, uint32_t rows) {
  const int ncol = d.n_kv * (d.d_nope + d.d_v);
  const uint64_t dims[2] = {(uint64_t)ncol, (uint64_t)d.d_c}, str[1] = {(uint64_t)ncol * 2};
  const uint32_t box[2] = {64, rows};
  return make_tmap_bf16(m, d.w_ukv, 2, dims, str, box);
}

}  // namespace

cudaError_t launch_qdecode_tc(const QdecodeParams& p, cudaStream_t s) {
  using namespace q8;
  const DecodeParams& d = p.d;
  const int H_q = d.n_kv * (d.g + 1);
  {
    CUtensorMap tw;
    if (!w_map(&tw, d, AB)) return cudaErrorInvalidValue;
    AbsorbArgs a{};
    a.B = d.B; a.T_max = d.T_max; a.n_kv = d.n_kv; a.g = d.g; a.H_q = H_q; a.n_hg = d.n_hg; a.hpc = d.hpc;
    a.NH = d.part_heads;
    a.isc = d.scale * kLog2e;
    a.q = reinterpret_cast<const __nv_bfloat16*>(d.q); a.seqlens = d.seqlens; a.cos_tab = d.cos_tab;
    a.sin_tab = d.sin_tab; a.qimg = d.qimg; a.status = d.status; a.failed = p.failed;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_smem(qdecode_absorb_kernel, AB_SMEM, allowed);
    if (e != cudaSuccess) return e;
    const unsigned tiles = (unsigned)qdec_absorb_tiles(d.B, d.g);
    qdecode_absorb_kernel<<<dim3((unsigned)d.n_kv, tiles, kQdecAbsorbSplit), 256, AB_SMEM, s>>>(tw, a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  {
    CUtensorMap tc, tr;
    const uint64_t cd[3] = {(uint64_t)DC, (uint64_t)d.T_max, (uint64_t)d.B};
    const uint64_t cs[2] = {(uint64_t)DC, (uint64_t)d.T_max * DC};
    const uint32_t cb[3] = {128, (uint32_t)TT, 1};
    const uint64_t rd[3] = {(uint64_t)DR, (uint64_t)d.T_max, (uint64_t)d.B};
    const uint64_t rs[2] = {(uint64_t)DR, (uint64_t)d.T_max * DR};
    const uint32_t rb[3] = {64, (uint32_t)TT, 1};
    if (!make_tmap_u8(&tc, d.c_cache, 3, cd, cs, cb, 128) || !make_tmap_u8(&tr, d.kr_cache, 3, rd, rs, rb, 64))
      return cudaErrorInvalidValue;
    Args a{};
    a.B = d.B; a.T_max = d.T_max; a.sliding = d.sliding; a.window = d.window; a.H_q = H_q; a.n_hg = d.n_hg;
    a.hpc = d.hpc; a.n_ranges = d.n_ranges; a.sl = p.sl; a.n_blocks = p.n_blocks;
    a.img_bytes = qdec_image_bytes(d.part_heads); a.seqlens = d.seqlens;
    a.c8 = (const uint8_t*)d.c_cache; a.kr8 = (const uint8_t*)d.kr_cache; a.scales = p.scales; a.qimg = d.qimg;
    a.seqinfo = d.seqinfo; a.part_o = d.part_o; a.part_ml = d.part_ml; a.status = d.status;
    a.failed = p.failed; a.n_absorb = d.n_kv * qdec_absorb_tiles(d.B, d.g) * kQdecAbsorbSplit;
    const dim3 grid((unsigned)d.n_hg, (unsigned)d.n_ranges);
    cudaError_t e;
    switch (d.part_heads / HT) {
      case 1: e = launch_dependent<qdecode_split_kernel<1>>(grid, Lay<1>::NT, Lay<1>::SMEM, s, tc, tr, a); break;
      case 2: e = launch_dependent<qdecode_split_kernel<2>>(grid, Lay<2>::NT, Lay<2>::SMEM, s, tc, tr, a); break;
      case 3: e = launch_dependent<qdecode_split_kernel<3>>(grid, Lay<3>::NT, Lay<3>::SMEM, s, tc, tr, a); break;
      default: return cudaErrorInvalidValue;
    }
    if (e != cudaSuccess) return e;
  }
  CUtensorMap tw;
  if (!w_map(&tw, d, 256)) return cudaErrorInvalidValue;
  CombineArgs a{};
  a.B = d.B; a.T_max = d.T_max; a.n_kv = d.n_kv; a.g = d.g; a.H_q = H_q; a.n_hg = d.n_hg; a.hpc = d.hpc;
  a.NH = d.part_heads; a.n_ranges = d.n_ranges; a.seqlens = d.seqlens; a.seqinfo = d.seqinfo; a.part_o = d.part_o; a.part_ml = d.part_ml;
  a.lam = d.lam; a.gate = reinterpret_cast<const __nv_bfloat16*>(d.gate);
  a.out = reinterpret_cast<__nv_bfloat16*>(d.out); a.status = d.status;
  // sequences per block: as few as fill one wave of blocks over the SMs, at most the 32 rows
  const int per_group = kQdecSMs / d.n_kv > 1 ? kQdecSMs / d.n_kv : 1;
  const int fill = (d.B + per_group - 1) / per_group, cap = CB_R / (d.g + 1);
  a.spb = fill < 1 ? 1 : (fill > cap ? cap : fill);
  return launch_dependent<qdecode_combine_kernel>(dim3((unsigned)d.n_kv, (unsigned)((d.B + a.spb - 1) / a.spb)), CB_T, CB_SMEM,
                                                  s, tw, a);
}

}  // namespace gdla
