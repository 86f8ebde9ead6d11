// HBM-bound kernels of the block: modulated RMSNorm, q/k RMSNorm + rotary pack, gated residual
// add, SiLU gate, and the small glue of a guided denoising step (sequence assembly, guidance +
// Euler update).  The MOSS-Image transformer page lists the first four as its hand-written kernels
// ("modulated RMSNorm, q/k norm and rotary into packed rows, situ [SiLU gate], gated add").
//
// All of them move 16-byte vectors (8 bf16) per thread, reduce in fp32 with a fixed shuffle
// order (so results repeat bit for bit), and round once to bf16 at the output.
#include <stdlib.h>

#include "mi_internal.h"
#include "ptx.cuh"

namespace mi {

namespace {

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x);
  f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z);
  f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ float silu_f(float g) { return g / (1.0f + __expf(-g)); }

// ------------------------------------------------------------------------------------ adaLN norm
// out[i] = x[in_row(i)] * rsqrt(mean(x^2) + eps) * (1 + scale[b]) + shift[b]; one warp per row.
// Row i of the output reads input row (i / out_seq) * in_seq + in_off + i % out_seq, which lets
// the final norm of a denoising step read only the image rows of each batch element.
//
// Each CTA (one per SM) takes a contiguous range of rows; its warps take every kNormWarps-th row
// of it.  A warp keeps `depth` of its rows in flight as bulk asynchronous copies into its own
// shared-memory slots (one mbarrier each), issued before any arithmetic: at the block's 4130 rows
// every row an SM handles is requested at the start, so the reads stream at full depth from the
// first microsecond instead of ramping up behind register-held loads.  A row is read from its slot
// twice (sum of squares, then the outputs, which go straight to global memory) and the slot is then
// refilled with the warp's row `depth` further on.  The launch is programmatic-dependent: the CTAs start (barrier set-up)
// while the previous kernel in the stream finishes and wait for its results before the first copy.
// The arithmetic and its order (per-lane fp32 sums on two packed lanes, then a fixed shuffle
// butterfly) are fixed: results repeat bit for bit.  NV = hidden / 256 (hidden <= 4096).
constexpr int kNormWarps = 16;
constexpr int kNormSlotBytes = 192 * 1024;        // shared memory for row slots per CTA
constexpr int kNormMaxDepth = 4;

template <int NV>
__global__ void __launch_bounds__(kNormWarps * 32, 1)
    mod_rmsnorm_kernel(const __nv_bfloat16* __restrict__ x, const __nv_bfloat16* __restrict__ shift,
                       const __nv_bfloat16* __restrict__ scale, int mod_bstride, __nv_bfloat16* __restrict__ out,
                       int rows, int out_seq, int in_seq, int in_off, int hidden, float eps, int depth, int* err,
                       int* zero, int zero_n) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  constexpr uint32_t kRowBytes = NV * 512;
  __shared__ uint64_t bars[kNormWarps * kNormMaxDepth];
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int r0 = (int)((long long)rows * blockIdx.x / gridDim.x);
  const int r1 = (int)((long long)rows * (blockIdx.x + 1) / gridDim.x);
  const int n_mine = (r1 - r0 - warp + kNormWarps - 1) / kNormWarps;  // rows r0 + warp + k * kNormWarps
  uint64_t* my_bars = bars + warp * kNormMaxDepth;
  uint8_t* my_slots = smem_raw + (size_t)warp * depth * kRowBytes;
  if (lane == 0) {
    for (int i = 0; i < depth; ++i) mbar_init(&my_bars[i], 1);
    if (warp == 0) abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  grid_dep_wait();  // x may be the previous kernel's output
  if (zero != nullptr)
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < zero_n; i += gridDim.x * blockDim.x) zero[i] = 0;

  auto issue = [&](int k) {  // lane 0: row k of this warp into slot k % depth
    const int r = r0 + warp + k * kNormWarps;
    const int in_row = (r / out_seq) * in_seq + in_off + r % out_seq;
    const int sl = k % depth;
    mbar_arrive_expect_tx(&my_bars[sl], kRowBytes);
    bulk_load(my_slots + (size_t)sl * kRowBytes, x + (size_t)in_row * hidden, kRowBytes, &my_bars[sl]);
  };
  int issued = n_mine < depth ? (n_mine > 0 ? n_mine : 0) : depth;
  if (lane == 0)
    for (int k = 0; k < issued; ++k) issue(k);
  grid_dep_launch();

  // Rows are taken two at a time when a warp has two left (they share one read of the modulation
  // vectors), else one at a time.
  auto row_rstd = [&](const uint4* src) {
    f32x2_t ss2 = 0ull;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint4 v = src[i * 32 + lane];
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f32x2_t f = f2_pack(bf16_lo(w[e]), bf16_hi(w[e]));
        ss2 = f2_fma(f, f, ss2);
      }
    }
    float ss_lo, ss_hi;
    f2_unpack(ss2, ss_lo, ss_hi);
    float ss = ss_lo + ss_hi;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    return rsqrtf(ss / (float)hidden + eps);
  };
  auto mod_piece = [&](uint4 v, uint4 vs, uint4 vc, f32x2_t rstd2) {
    const f32x2_t one2 = f2_pack(1.0f, 1.0f);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w}, ws[4] = {vs.x, vs.y, vs.z, vs.w}, wc[4] = {vc.x, vc.y, vc.z, vc.w};
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const f32x2_t t = f2_mul(f2_pack(bf16_lo(w[e]), bf16_hi(w[e])), rstd2);
      const f32x2_t c = f2_add(f2_pack(bf16_lo(wc[e]), bf16_hi(wc[e])), one2);
      float lo, hi;
      f2_unpack(f2_fma(t, c, f2_pack(bf16_lo(ws[e]), bf16_hi(ws[e]))), lo, hi);
      o[e] = pack_bf16x2(lo, hi);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  };
  int k = 0;
  while (k < n_mine) {
    const int take = (depth >= 2 && k + 1 < n_mine && (r0 + warp + k * kNormWarps) / out_seq ==
                                            (r0 + warp + (k + 1) * kNormWarps) / out_seq) ? 2 : 1;
    const int slA = k % depth, slB = (k + 1) % depth;
    if (!mbar_wait_warp(&my_bars[slA], (uint32_t)((k / depth) & 1), &abort_flag, err, DEV_TIMEOUT_NORM + 1)) break;
    if (take == 2 &&
        !mbar_wait_warp(&my_bars[slB], (uint32_t)(((k + 1) / depth) & 1), &abort_flag, err, DEV_TIMEOUT_NORM + 1))
      break;
    const uint4* srcA = reinterpret_cast<const uint4*>(my_slots + (size_t)slA * kRowBytes);
    const uint4* srcB = reinterpret_cast<const uint4*>(my_slots + (size_t)slB * kRowBytes);
    const int rowA = r0 + warp + k * kNormWarps;
    const int rowB = rowA + kNormWarps;
    const float rstdA = row_rstd(srcA);
    const float rstdB = take == 2 ? row_rstd(srcB) : 0.0f;
    const int b = rowA / out_seq;
    const uint4* sh = reinterpret_cast<const uint4*>(shift + (size_t)b * mod_bstride);
    const uint4* sc = reinterpret_cast<const uint4*>(scale + (size_t)b * mod_bstride);
    uint4* orowA = reinterpret_cast<uint4*>(out + (size_t)rowA * hidden);
    uint4* orowB = reinterpret_cast<uint4*>(out + (size_t)rowB * hidden);
    const f32x2_t rA = f2_pack(rstdA, rstdA), rB = f2_pack(rstdB, rstdB);
#pragma unroll
    for (int i = 0; i < NV; ++i) {  // each row read again from its slot; (x * rstd) * (1 + scale) + shift
      const uint4 vs = __ldg(sh + i * 32 + lane);
      const uint4 vc = __ldg(sc + i * 32 + lane);
      orowA[i * 32 + lane] = mod_piece(srcA[i * 32 + lane], vs, vc, rA);
      if (take == 2) orowB[i * 32 + lane] = mod_piece(srcB[i * 32 + lane], vs, vc, rB);
    }
    __syncwarp();  // every lane is done with the slots before they are refilled
    for (int t = 0; t < take; ++t) {
      if (k + depth < n_mine) {
        if (lane == 0) {
          fence_proxy_async_smem();
          issue(k + depth);
        }
        ++issued;
      }
      ++k;
    }
  }
  // after an abort: the copies still in flight land before the CTA's shared memory is released
  if (lane == 0)
    for (int j = k; j < issued; ++j)
      mbar_wait_drain(&my_bars[j % depth], (uint32_t)((j / depth) & 1), err, DEV_TIMEOUT_NORM + 2);
}

template <int NV>
cudaError_t mod_rmsnorm_launch_nv(const __nv_bfloat16* x, const __nv_bfloat16* shift, const __nv_bfloat16* scale,
                                  int mod_bstride, __nv_bfloat16* out, int rows, int out_seq, int in_seq, int in_off,
                                  int hidden, float eps, int* err, int num_sms, int dev, cudaStream_t s, int* zero,
                                  int zero_n) {
  constexpr int kRowBytes = NV * 512;
  const int depth_fit = kNormSlotBytes / (kNormWarps * kRowBytes);
  const int depth = depth_fit < kNormMaxDepth ? depth_fit : kNormMaxDepth;
  const int smem = kNormWarps * depth * kRowBytes;
  static bool attr_done[kMaxDevices] = {};
  if (!attr_done[dev]) {
    cudaError_t e = cudaFuncSetAttribute(mod_rmsnorm_kernel<NV>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    attr_done[dev] = true;
  }
  const int need = (rows + kNormWarps - 1) / kNormWarps;
  const int grid = need < num_sms ? need : num_sms;
  return launch_kernel(mod_rmsnorm_kernel<NV>, dim3(grid), dim3(kNormWarps * 32), smem, s, true, x, shift, scale,
                       mod_bstride, out, rows, out_seq, in_seq, in_off, hidden, eps, depth, err, zero, zero_n);
}

cudaError_t mod_rmsnorm_any(const __nv_bfloat16* x, const __nv_bfloat16* shift, const __nv_bfloat16* scale,
                            int mod_bstride, __nv_bfloat16* out, int rows, int out_seq, int in_seq, int in_off,
                            int hidden, float eps, int* err, cudaStream_t s, int* zero, int zero_n) {
  static int sms_cache[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (sms_cache[dev] == 0) {
    e = cudaDeviceGetAttribute(&sms_cache[dev], cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
  }
  if (rows <= 0) return cudaSuccess;
  switch (hidden >> 8) {
#define MI_NORM_CASE(n)                                                                                          \
  case n:                                                                                                        \
    return mod_rmsnorm_launch_nv<n>(x, shift, scale, mod_bstride, out, rows, out_seq, in_seq, in_off, hidden, eps, \
                                    err, sms_cache[dev], dev, s, zero, zero_n);
    MI_NORM_CASE(1) MI_NORM_CASE(2) MI_NORM_CASE(3) MI_NORM_CASE(4) MI_NORM_CASE(5) MI_NORM_CASE(6) MI_NORM_CASE(7)
    MI_NORM_CASE(8) MI_NORM_CASE(9) MI_NORM_CASE(10) MI_NORM_CASE(11) MI_NORM_CASE(12) MI_NORM_CASE(13)
    MI_NORM_CASE(14) MI_NORM_CASE(15) MI_NORM_CASE(16)
#undef MI_NORM_CASE
    default:
      return cudaErrorInvalidValue;
  }
}

// ------------------------------------------------------------------------------------ q/k pack
// One warp per (row, head): lanes 0-15 take q, lanes 16-31 take k, 8 consecutive elements each
// (4 rotary pairs).  RMSNorm over the 128 elements of the head, gain, then the rotation of the
// interleaved pairs (2p, 2p+1) by the table angle at (row, p).  Output rows are packed per head:
// qp/kp[(b * heads + h) * S + s][0..128).
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(const __nv_bfloat16* __restrict__ qkv,
                                                           const __nv_bfloat16* __restrict__ wq,
                                                           const __nv_bfloat16* __restrict__ wk,
                                                           const float* __restrict__ cosv,
                                                           const float* __restrict__ sinv, int rope_bstride,
                                                           __nv_bfloat16* __restrict__ qp,
                                                           __nv_bfloat16* __restrict__ kp, int batch, int seq,
                                                           int heads, float eps) {
  const long long item = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const long long total = (long long)batch * seq * heads;
  if (item >= total) return;
  const int h = (int)(item % heads);
  const long long row = item / heads;  // b * seq + s
  const int b = (int)(row / seq);
  const int s = (int)(row % seq);
  const int H = heads * kHeadDim;
  const int which = lane >> 4;  // 0: q, 1: k
  const int sub = lane & 15;
  const int e0 = sub * 8;
  const uint4 v = *reinterpret_cast<const uint4*>(qkv + (size_t)row * 3 * H + (size_t)which * H +
                                                  (size_t)h * kHeadDim + e0);
  float f[8];
  unpack8(v, f);
  float ss = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float rstd = rsqrtf(ss * (1.0f / kHeadDim) + eps);
  float g[8];
  unpack8(__ldg(reinterpret_cast<const uint4*>((which ? wk : wq) + e0)), g);
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = f[e] * rstd * g[e];
  const float* cr = cosv + (size_t)b * rope_bstride + (size_t)s * (kHeadDim / 2) + sub * 4;
  const float* sr = sinv + (size_t)b * rope_bstride + (size_t)s * (kHeadDim / 2) + sub * 4;
  const float4 c4 = __ldg(reinterpret_cast<const float4*>(cr));
  const float4 s4 = __ldg(reinterpret_cast<const float4*>(sr));
  const float cs[4] = {c4.x, c4.y, c4.z, c4.w};
  const float sn[4] = {s4.x, s4.y, s4.z, s4.w};
  float o[8];
#pragma unroll
  for (int pr = 0; pr < 4; ++pr) {
    const float a = f[2 * pr], bb = f[2 * pr + 1];
    o[2 * pr] = fmaf(a, cs[pr], -bb * sn[pr]);
    o[2 * pr + 1] = fmaf(a, sn[pr], bb * cs[pr]);
  }
  __nv_bfloat16* dst = (which ? kp : qp) + (((size_t)b * heads + h) * seq + s) * kHeadDim + e0;
  *reinterpret_cast<uint4*>(dst) = pack8(o);
}

// ------------------------------------------------------------------------------------ q/k gradient
// With n = x r, r = rsqrt(mean x^2 + eps), y = rotate(n gain): the gradient of y is rotated back (dz),
// dgain = sum of dz n over all rows and heads, and with t = dz gain, dx = r (t - n mean(t n)).
// HBM bound: 12 bytes per element of q and k (8260 rows x 24 heads: 52 us, 5.88 TB/s; with 2 CTAs per SM
// 59 us, with 2 heads at a time and 4 CTAs 58, and 3 heads 56).  A warp takes kQkHeads heads of a row at a time (lanes 0-15 q,
// lanes 16-31 k, 8 elements each), with all their loads in flight before the first is used, and one read
// of the row's angles for all of them.  dgain is summed in registers, then over the CTA's warps, then over
// the CTAs, each in a fixed order: by a second kernel, or (kCluster, few rows) over the one cluster of the
// launch through shared memory, which saves the second launch where launches are what a call costs.
// A head whose dy is zero in a row (a masked key's, or a row's without a valid key) has a zero gradient and
// adds nothing to dgain, whatever x holds; but zero times an infinity or NaN in a padded row is not zero.  Such
// a row leaves a sum that is not finite, and the warp then takes its items again, leaving such heads out (looked
// for head by head in the first place it costs every call 3 to 7 %; this way only calls with such rows pay: 118 instead of
// 53 us at 8260 rows x 24 heads when every warp has some).
constexpr int kQkBwdThreads = 256;
constexpr int kQkBwdWarps = kQkBwdThreads / 32;
constexpr int kQkHeads = 4;
constexpr int kQkCtas = 3;  // per SM
constexpr int kQkCluster = 8;

// One head of a row: adds to dg and returns dx of this lane's 8 elements.  live: false where x and r count as zero.
__device__ __forceinline__ uint4 qk_bwd_head(uint4 xv, uint4 yv, const float (&cs)[4], const float (&sn)[4], const float (&g)[8],
                                             float eps, bool live, float (&dg)[8]) {
  float x[8], y[8];
  unpack8(xv, x);
  unpack8(yv, y);
#pragma unroll
  for (int pr = 0; pr < 4; ++pr) {
    const float a = y[2 * pr], bb = y[2 * pr + 1];
    y[2 * pr] = fmaf(a, cs[pr], bb * sn[pr]);
    y[2 * pr + 1] = fmaf(bb, cs[pr], -a * sn[pr]);
  }
  float ss = 0.0f, tx = 0.0f;  // sums of x^2 and of t x
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    ss = fmaf(x[e], x[e], ss);
    tx = fmaf(y[e] * g[e], x[e], tx);
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    ss += __shfl_xor_sync(0xffffffffu, ss, o);
    tx += __shfl_xor_sync(0xffffffffu, tx, o);
  }
  const float r = live ? rsqrtf(ss * (1.0f / kHeadDim) + eps) : 0.0f;
  const float m = tx * r * r * (1.0f / kHeadDim);  // mean(t n) r
  float o[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    dg[e] = fmaf(y[e], x[e] * r, dg[e]);
    o[e] = r * fmaf(y[e], g[e], -x[e] * m);
  }
  return pack8(o);
}

// A warp's items again, a head at a time; heads whose dy is zero are left out of dgain and get zeros.
__device__ __forceinline__ void qk_bwd_again(const __nv_bfloat16* qkv, const __nv_bfloat16* gain, const float* cosv,
                                          const float* sinv, int rope_bstride, const __nv_bfloat16* dyp,
                                          __nv_bfloat16* dqkv, int batch, int seq, int heads, float eps, float* sum) {
  const int lane = threadIdx.x & 31;
  const int e0 = (lane & 15) * 8;
  const int H = heads * kHeadDim;
  const int groups = (heads + kQkHeads - 1) / kQkHeads;
  const long long total = (long long)batch * seq * groups;
  float g[8], dg[8] = {};
  unpack8(__ldg(reinterpret_cast<const uint4*>(gain + e0)), g);
  for (long long item = (long long)blockIdx.x * kQkBwdWarps + (threadIdx.x >> 5); item < total;
       item += (long long)gridDim.x * kQkBwdWarps) {
    const long long row = item / groups;
    const int b = (int)(row / seq), s = (int)(row % seq), h0 = (int)(item % groups) * kQkHeads;
    const size_t tab = (size_t)b * rope_bstride + (size_t)s * (kHeadDim / 2) + (lane & 15) * 4;
#pragma unroll 1
    for (int h = h0; h < h0 + kQkHeads && h < heads; ++h) {
      const size_t x_at = (size_t)row * 3 * H + (size_t)(lane >> 4) * H + (size_t)h * kHeadDim + e0;
      uint4 xv = __ldg(reinterpret_cast<const uint4*>(qkv + x_at));
      const uint4 yv = __ldg(reinterpret_cast<const uint4*>(dyp + (((size_t)b * heads + h) * seq + s) * kHeadDim + e0));
      const uint32_t bits = (yv.x | yv.y | yv.z | yv.w) & 0x7fff7fffu;  // (a zero of either sign)
      const bool live = ((__ballot_sync(0xffffffffu, bits != 0) >> (lane & 16)) & 0xffffu) != 0;
      if (!live) xv = make_uint4(0, 0, 0, 0);
      const float4 c4 = __ldg(reinterpret_cast<const float4*>(cosv + tab));
      const float4 s4 = __ldg(reinterpret_cast<const float4*>(sinv + tab));
      const float cs[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
      *reinterpret_cast<uint4*>(dqkv + x_at) = qk_bwd_head(xv, yv, cs, sn, g, eps, live, dg);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = dg[e];
}

template <bool kCluster>
__global__ void __launch_bounds__(kQkBwdThreads, kQkCtas)
    qk_norm_rope_bwd_kernel(const __nv_bfloat16* __restrict__ qkv, const __nv_bfloat16* __restrict__ wq,
                            const __nv_bfloat16* __restrict__ wk, const float* __restrict__ cosv,
                            const float* __restrict__ sinv, int rope_bstride, const __nv_bfloat16* __restrict__ dqp,
                            const __nv_bfloat16* __restrict__ dkp, __nv_bfloat16* __restrict__ dqkv,
                            float* __restrict__ partial, float* __restrict__ dwq, float* __restrict__ dwk, int batch,
                            int seq, int heads, float eps) {
  __shared__ float sums[kQkBwdWarps][256];
  __shared__ float cta_sum[256];
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int which = lane >> 4;  // 0: q, 1: k
  const int e0 = (lane & 15) * 8;
  const int H = heads * kHeadDim;
  const int groups = (heads + kQkHeads - 1) / kQkHeads;
  const long long total = (long long)batch * seq * groups;
  const long long stride = (long long)gridDim.x * kQkBwdWarps;
  float g[8], dg[8];
  unpack8(__ldg(reinterpret_cast<const uint4*>((which ? wk : wq) + e0)), g);
#pragma unroll
  for (int e = 0; e < 8; ++e) dg[e] = 0.0f;
  for (long long item = (long long)blockIdx.x * kQkBwdWarps + warp; item < total; item += stride) {
    const int h0 = (int)(item % groups) * kQkHeads;
    const long long row = item / groups;
    const int b = (int)(row / seq);
    const int s = (int)(row % seq);
    const size_t x_at = (size_t)row * 3 * H + (size_t)which * H + (size_t)h0 * kHeadDim + e0;
    const __nv_bfloat16* dy = (which ? dkp : dqp) + (((size_t)b * heads + h0) * seq + s) * kHeadDim + e0;
    uint4 xv[kQkHeads], yv[kQkHeads];
#pragma unroll
    for (int i = 0; i < kQkHeads; ++i) {
      if (h0 + i < heads) {
        xv[i] = __ldg(reinterpret_cast<const uint4*>(qkv + x_at + (size_t)i * kHeadDim));
        yv[i] = __ldg(reinterpret_cast<const uint4*>(dy + (size_t)i * seq * kHeadDim));
      } else {
        xv[i] = yv[i] = make_uint4(0, 0, 0, 0);
      }
    }
    const size_t tab = (size_t)b * rope_bstride + (size_t)s * (kHeadDim / 2) + (lane & 15) * 4;
    const float4 c4 = __ldg(reinterpret_cast<const float4*>(cosv + tab));
    const float4 s4 = __ldg(reinterpret_cast<const float4*>(sinv + tab));
    const float cs[4] = {c4.x, c4.y, c4.z, c4.w}, sn[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int i = 0; i < kQkHeads; ++i) {
      const uint4 dx = qk_bwd_head(xv[i], yv[i], cs, sn, g, eps, true, dg);
      if (h0 + i < heads) *reinterpret_cast<uint4*>(dqkv + x_at + (size_t)i * kHeadDim) = dx;
    }
  }
  bool finite = true;
#pragma unroll
  for (int e = 0; e < 8; ++e) finite &= fabsf(dg[e]) <= 3.402823466e38f;
  float* sum = &sums[warp][which * 128 + e0];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = dg[e];
  if (!__all_sync(0xffffffffu, finite))
    qk_bwd_again(qkv, which ? wk : wq, cosv, sinv, rope_bstride, which ? dkp : dqp, dqkv, batch, seq, heads, eps, sum);
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int w = 0; w < kQkBwdWarps; ++w) t += sums[w][threadIdx.x];
  if (!kCluster) {
    partial[(size_t)blockIdx.x * 256 + threadIdx.x] = t;
  } else {
    cta_sum[threadIdx.x] = t;
    cluster_sync();
    constexpr int kCols = 256 / kQkCluster;  // columns of this CTA
    if (threadIdx.x < kCols) {
      const int c = (int)cluster_rank() * kCols + (int)threadIdx.x;
      float v[kQkCluster];
#pragma unroll
      for (int i = 0; i < kQkCluster; ++i)
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[i]) : "r"(cluster_addr(&cta_sum[c], (uint32_t)i)) : "memory");
      float all = 0.0f;
#pragma unroll
      for (int i = 0; i < kQkCluster; ++i) all += v[i];
      (c < 128 ? dwq : dwk)[c & 127] = all;
    }
    cluster_sync();  // nobody leaves while its sums are being read
  }
}

// dgain[c] = sum of the CTAs' partial sums: a block takes 16 of the 256 columns, 16 groups of threads every
// 16th CTA each, and adds the groups in order.
__global__ void __launch_bounds__(256) qk_gain_sum_kernel(const float* partial, int n,
                                                          float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ float sums[16][17];
  grid_dep_wait();
  const int col = threadIdx.x & 15, grp = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + col;
  float t = 0.0f;
#pragma unroll 8
  for (int i = grp; i < n; i += 16) t += __ldcg(partial + (size_t)i * 256 + c);
  sums[grp][col] = t;
  __syncthreads();
  if (grp == 0) {
    float all = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) all += sums[i][col];
    (c < 128 ? dwq : dwk)[c & 127] = all;
  }
}

// ------------------------------------------------------------------------------------ gated add
// out = x + gate[b] * y (fp32 fma, one rounding); the same expression as the fused GEMM epilogue.
__global__ void __launch_bounds__(256) gated_add_kernel(const __nv_bfloat16* __restrict__ x,
                                                        const __nv_bfloat16* __restrict__ y,
                                                        const __nv_bfloat16* __restrict__ gate, int gate_bstride,
                                                        __nv_bfloat16* __restrict__ out, long long n_vec, int seq,
                                                        int hidden) {
  const int vpr = hidden >> 3;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n_vec;
       i += (long long)gridDim.x * blockDim.x) {
    const long long row = i / vpr;
    const int cv = (int)(i % vpr);
    const int b = (int)(row / seq);
    float fx[8], fy[8], fg[8];
    unpack8(reinterpret_cast<const uint4*>(x)[i], fx);
    unpack8(reinterpret_cast<const uint4*>(y)[i], fy);
    unpack8(__ldg(reinterpret_cast<const uint4*>(gate + (size_t)b * gate_bstride) + cv), fg);
#pragma unroll
    for (int e = 0; e < 8; ++e) fx[e] = fmaf(fg[e], fy[e], fx[e]);
    reinterpret_cast<uint4*>(out)[i] = pack8(fx);
  }
}

// ------------------------------------------------------------------------------------ SiLU gate
// m[r, j] = silu(gu[r, j]) * gu[r, I + j]; the same expression as the fused GEMM epilogue.
__global__ void __launch_bounds__(256) silu_gate_kernel(const __nv_bfloat16* __restrict__ gu,
                                                        __nv_bfloat16* __restrict__ m, long long n_vec, int inter) {
  const int vpr = inter >> 3;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n_vec;
       i += (long long)gridDim.x * blockDim.x) {
    const long long row = i / vpr;
    const int cv = (int)(i % vpr);
    const uint4* src = reinterpret_cast<const uint4*>(gu + (size_t)row * 2 * inter);
    float g[8], u[8];
    unpack8(src[cv], g);
    unpack8(src[vpr + cv], u);
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = silu_f(g[e]) * u[e];
    reinterpret_cast<uint4*>(m)[i] = pack8(g);
  }
}

// ------------------------------------------------------------------------------------ step glue
// x[b, t] = text[b, t] for t < T, x[b, T + n] = u[n] (the embedded latent is shared by the batch).
__global__ void __launch_bounds__(256) assemble_seq_kernel(const uint4* __restrict__ text, const uint4* __restrict__ u,
                                                           uint4* __restrict__ x, int batch, int text_pad,
                                                           int n_img, int vpr) {
  const long long S = text_pad + n_img;
  const long long total = (long long)batch * S * vpr;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += (long long)gridDim.x * blockDim.x) {
    const long long row = i / vpr;
    const int cv = (int)(i % vpr);
    const int b = (int)(row / S);
    const int s = (int)(row % S);
    x[i] = s < text_pad ? text[((long long)b * text_pad + s) * vpr + cv] : u[(long long)(s - text_pad) * vpr + cv];
  }
}

__global__ void __launch_bounds__(256) copy_vec_kernel(const uint4* __restrict__ src, uint4* __restrict__ dst,
                                                       long long n_vec) {
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n_vec;
       i += (long long)gridDim.x * blockDim.x)
    dst[i] = src[i];
}

// v = v_neg + g (v_pos - v_neg), latent <- latent + dt v, all fp32.  vel is [batch, N, C].
__global__ void __launch_bounds__(256) cfg_euler_kernel(const float* __restrict__ vel, float* __restrict__ latent,
                                                        long long n, float dt, float guidance, int batch) {
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (long long)gridDim.x * blockDim.x) {
    const float vp = vel[i];
    const float v = batch > 1 ? fmaf(guidance, vp - vel[n + i], vel[n + i]) : vp;
    latent[i] = fmaf(dt, v, latent[i]);
  }
}

__global__ void __launch_bounds__(256) f32_to_bf16_kernel(const float* __restrict__ src, __nv_bfloat16* __restrict__ dst,
                                                          long long n) {
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (long long)gridDim.x * blockDim.x)
    dst[i] = __float2bfloat16_rn(src[i]);
}

// ------------------------------------------------------------------------------------ builders
// Rotary tables on the device: row s, pair j turns by pos * theta^(-(j mod 32)/32) with pos the row
// position (pairs < 32) or column position (pairs >= 32) of the token; text row t has position t
// on both axes.  Angles in fp64, stored as fp32.
__global__ void __launch_bounds__(256) rope_table_kernel(float* __restrict__ cosv, float* __restrict__ sinv, int S,
                                                          int text_pad, int grid_w, double theta) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= S * 64) return;
  const int s = i >> 6;
  const int j = i & 63;
  double pos;
  if (s < text_pad) {
    pos = (double)s;
  } else {
    const int r = (s - text_pad) / grid_w;
    const int c = (s - text_pad) % grid_w;
    pos = (double)(j < 32 ? r : c);
  }
  const double ang = pos * pow(theta, -(double)(j & 31) / 32.0);
  cosv[i] = (float)cos(ang);
  sinv[i] = (float)sin(ang);
}

// Rotary tables from per-token positions: pair j of row r turns by pos[r, axis j] (hi_j + lo_j) full
// turns, hi + lo a frequency over 2 pi in 48 bits.  The product is formed in two fp32 parts (t, and what its
// rounding and lo leave: recovered by two fmas), whole and quarter turns are taken off t exactly, and the
// Taylor polynomials of sine and cosine see at most an eighth of a turn, where their first terms left out
// are below 2^-28: the angle is as exact as in 64 bits up to positions of 2^24.  The rest of a far position
// may itself be turns; taking those off keeps every entry a sine or cosine of some angle.
// 16 lanes take a row, 4 pairs each, and keep their frequencies in registers over the rows of a
// grid-stride loop (a warp's 16 different constants are read one by one: few CTAs, vector loads).
__global__ void __launch_bounds__(256) rope_axes_kernel(const float* __restrict__ pos, int rows, int n_axes,
                                                        const __grid_constant__ RopeAxes f, float* __restrict__ cosv,
                                                        float* __restrict__ sinv) {
  grid_dep_wait();
  grid_dep_launch();
  const int j0 = (threadIdx.x & 15) * 4;
  const float4 hi4 = *reinterpret_cast<const float4*>(f.hi + j0), lo4 = *reinterpret_cast<const float4*>(f.lo + j0);
  const uchar4 ax4 = *reinterpret_cast<const uchar4*>(f.axis + j0);
  const float hi[4] = {hi4.x, hi4.y, hi4.z, hi4.w}, lo[4] = {lo4.x, lo4.y, lo4.z, lo4.w};
  const int axis[4] = {ax4.x, ax4.y, ax4.z, ax4.w};
  const long long stride = (long long)gridDim.x * 16;
  long long r = (long long)blockIdx.x * 16 + (threadIdx.x >> 4);
  float next[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  auto read = [&](long long row) {
#pragma unroll
    for (int i = 0; i < 4; ++i) next[i] = __ldg(pos + row * n_axes + axis[i]);
  };
  if (r < rows) read(r);
  for (; r < rows; r += stride) {
    const float at[4] = {next[0], next[1], next[2], next[3]};
    if (r + stride < rows) read(r + stride);
    float c[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; i += 2) {  // two pairs at a time in packed arithmetic
      const f32x2_t p = f2_pack(at[i], at[i + 1]), h = f2_pack(hi[i], hi[i + 1]), l = f2_pack(lo[i], lo[i + 1]);
      const f32x2_t t = f2_mul(p, h);
      const f32x2_t left = f2_fma(p, l, f2_fma(p, h, f2_mul(t, f2_of(-1.0f))));
      float t0, t1, l0, l1;
      f2_unpack(t, t0, t1);
      f2_unpack(left, l0, l1);
      const f32x2_t frac = f2_add(t, f2_pack(-rintf(t0), -rintf(t1)));
      const f32x2_t rest = f2_add(left, f2_pack(-rintf(l0), -rintf(l1)));
      constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to a whole number in the low bits
      const f32x2_t nb = f2_fma(f2_add(frac, rest), f2_of(4.0f), f2_of(kMagic));
      const f32x2_t turn = f2_add(f2_fma(f2_add(nb, f2_of(-kMagic)), f2_of(-0.25f), frac), rest);
      const f32x2_t x = f2_mul(turn, f2_of(6.283185307179586f));
      const f32x2_t x2 = f2_mul(x, x);
      f32x2_t sp = f2_fma(x2, f2_of(2.75573192e-6f), f2_of(-1.98412698e-4f));  // 1/9!, -1/7!
      sp = f2_fma(x2, sp, f2_of(8.33333333e-3f));                               // 1/5!
      sp = f2_fma(x2, sp, f2_of(-1.66666667e-1f));                              // -1/3!
      sp = f2_fma(f2_mul(x, x2), sp, x);
      f32x2_t cp = f2_fma(x2, f2_of(-2.75573192e-7f), f2_of(2.48015873e-5f));   // -1/10!, 1/8!
      cp = f2_fma(x2, cp, f2_of(-1.38888889e-3f));                              // -1/6!
      cp = f2_fma(x2, cp, f2_of(4.16666667e-2f));                               // 1/4!
      cp = f2_fma(x2, cp, f2_of(-0.5f));
      cp = f2_fma(x2, cp, f2_of(1.0f));
      float sv[2], cv[2], nv[2];
      f2_unpack(sp, sv[0], sv[1]);
      f2_unpack(cp, cv[0], cv[1]);
      f2_unpack(nb, nv[0], nv[1]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {  // a quarter turn on: (c, s) -> (-s, c)
        const uint32_t quarter = __float_as_uint(nv[e]);
        const bool odd = quarter & 1u;
        const uint32_t cq = __float_as_uint(odd ? sv[e] : cv[e]), sq = __float_as_uint(odd ? cv[e] : sv[e]);
        c[i + e] = __uint_as_float(cq ^ (((quarter + 1u) & 2u) << 30));
        s[i + e] = __uint_as_float(sq ^ ((quarter & 2u) << 30));
      }
    }
    // evict-first: a table larger than the L2 cache does not push out what the consumers read next
    __stcs(reinterpret_cast<float4*>(cosv + r * 64 + j0), make_float4(c[0], c[1], c[2], c[3]));
    __stcs(reinterpret_cast<float4*>(sinv + r * 64 + j0), make_float4(s[0], s[1], s[2], s[3]));
  }
}

// Sinusoidal timestep embedding: out[b, k] = cos(scale t_b f_k), out[b, half + k] = sin(scale t_b f_k),
// f_k = max_period^(-k / half); fp64, rounded to bf16.
__global__ void __launch_bounds__(256) timestep_embedding_kernel(const float* __restrict__ t, __nv_bfloat16* __restrict__ out,
                                                                 int batch, int half, double scale, double max_period) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= batch * half) return;
  const int b = i / half;
  const int k = i % half;
  const double ang = scale * (double)t[b] * pow(max_period, -(double)k / (double)half);
  out[(size_t)b * 2 * half + k] = __float2bfloat16_rn((float)cos(ang));
  out[(size_t)b * 2 * half + half + k] = __float2bfloat16_rn((float)sin(ang));
}

__global__ void __launch_bounds__(256) silu_inplace_kernel(__nv_bfloat16* __restrict__ v, long long n) {
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x)
    v[i] = __float2bfloat16_rn(silu_f(__bfloat162float(v[i])));
}

// all[b, (6 i + k) H + c] -> mods[i, b, k, c]; all[b, (6 n + k) H + c] -> final[b, k, c].
__global__ void __launch_bounds__(256) modulation_split_kernel(const uint4* __restrict__ all, uint4* __restrict__ mods,
                                                               uint4* __restrict__ fin, int batch, int n_blocks,
                                                               int vpr /* H / 8 */) {
  const long long per_b = (long long)(6 * n_blocks + 2) * vpr;
  const long long total = per_b * batch;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total;
       i += (long long)gridDim.x * blockDim.x) {
    const int b = (int)(i / per_b);
    const long long r = i % per_b;
    const int vec = (int)(r / vpr);  // which H-wide vector
    const int c = (int)(r % vpr);
    if (vec < 6 * n_blocks) {
      const int blk = vec / 6, k = vec % 6;
      mods[(((long long)blk * batch + b) * 6 + k) * vpr + c] = all[i];
    } else {
      fin[((long long)b * 2 + (vec - 6 * n_blocks)) * vpr + c] = all[i];
    }
  }
}

__global__ void time_advance_kernel(float* __restrict__ t, int n, float dt) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) t[i] += dt;
}

int grid_for(long long work_items, int threads) {
  long long g = (work_items + threads - 1) / threads;
  const long long cap = 152LL * 16;  // enough resident blocks for a grid-stride loop
  if (g > cap) g = cap;
  if (g < 1) g = 1;
  return (int)g;
}

}  // namespace

bool pdl_enabled() {
  static const bool on = [] {
    const char* e = getenv("MI_PDL");
    return !(e && e[0] == '0');
  }();
  return on;
}

cudaError_t mod_rmsnorm_launch(const __nv_bfloat16* x, const __nv_bfloat16* shift, const __nv_bfloat16* scale,
                               int mod_bstride, __nv_bfloat16* out, int rows, int seq, int hidden, float eps, int* err,
                               cudaStream_t s, int* zero, int zero_n) {
  return mod_rmsnorm_any(x, shift, scale, mod_bstride, out, rows, seq, seq, 0, hidden, eps, err, s, zero, zero_n);
}

cudaError_t mod_rmsnorm_rows_launch(const __nv_bfloat16* x, const __nv_bfloat16* shift, const __nv_bfloat16* scale,
                                    int mod_bstride, __nv_bfloat16* out, int rows, int out_seq, int in_seq, int in_off,
                                    int hidden, float eps, int* err, cudaStream_t s) {
  return mod_rmsnorm_any(x, shift, scale, mod_bstride, out, rows, out_seq, in_seq, in_off, hidden, eps, err, s,
                         nullptr, 0);
}

cudaError_t qk_norm_rope_launch(const __nv_bfloat16* qkv, const __nv_bfloat16* wq, const __nv_bfloat16* wk,
                                const float* cos, const float* sin, int rope_bstride, __nv_bfloat16* qp,
                                __nv_bfloat16* kp, int batch, int seq, int n_heads, float eps, cudaStream_t s) {
  const long long warps = (long long)batch * seq * n_heads;
  if (warps <= 0) return cudaSuccess;
  const int threads = 256;
  const long long blocks = (warps * 32 + threads - 1) / threads;
  qk_norm_rope_kernel<<<(unsigned)blocks, threads, 0, s>>>(qkv, wq, wk, cos, sin, rope_bstride, qp, kp, batch, seq,
                                                           n_heads, eps);
  return cudaGetLastError();
}

static long long qk_bwd_items(int batch, int seq, int n_heads) {
  return (long long)batch * seq * ((n_heads + kQkHeads - 1) / kQkHeads);
}

// One cluster for up to 2 turns of its 64 warps; beyond, the whole GPU and a second kernel.  (Cluster against two
// kernels, replayed from a graph: 64 items 3.3 against 3.8 us, 96 items 4.5 against 3.8, 256 items 6.9 against 4.2.  Called
// in turn, where launches are what a call costs: 8.7 against 10.5 at all of these.  So a second turn still pays for
// calls, and costs a replay less than it saves them; a third and fourth do not.)
static bool qk_bwd_one_cluster(long long items) { return items <= 2LL * kQkCluster * kQkBwdWarps; }

int qk_norm_rope_bwd_grid(int batch, int seq, int n_heads, int num_sms) {
  const long long items = qk_bwd_items(batch, seq, n_heads);
  if (qk_bwd_one_cluster(items)) return kQkCluster;
  const long long need = (items + kQkBwdWarps - 1) / kQkBwdWarps;
  const long long cap = (long long)kQkCtas * num_sms;
  return (int)(need < cap ? need : cap);
}

cudaError_t qk_norm_rope_bwd_launch(const __nv_bfloat16* qkv, const __nv_bfloat16* wq, const __nv_bfloat16* wk,
                                    const float* cos, const float* sin, int rope_bstride, const __nv_bfloat16* dqp,
                                    const __nv_bfloat16* dkp, __nv_bfloat16* dqkv, float* dwq, float* dwk,
                                    float* partial, int batch, int seq, int n_heads, float eps, int num_sms,
                                    cudaStream_t s) {
  const int grid = qk_norm_rope_bwd_grid(batch, seq, n_heads, num_sms);
  if (qk_bwd_one_cluster(qk_bwd_items(batch, seq, n_heads)))
    return launch_kernel_cluster(qk_norm_rope_bwd_kernel<true>, dim3(grid), dim3(kQkBwdThreads), 0, kQkCluster, s, qkv, wq, wk,
                                 cos, sin, rope_bstride, dqp, dkp, dqkv, partial, dwq, dwk, batch, seq, n_heads, eps);
  // (Early whatever the number of CTAs, unlike launch_early: the attention's gradient, which it follows, does not let
  // the next kernel in before its end, so nothing piles up.  Both after 2 x 8 heads x 1000: 44.4 us, 44.6 without; this
  // kernel again and again 8.2, 8.4 without.  Behind the attention forward, which does let it in, it would lose 10 of
  // 223 us at 24 heads x 4130.)
  cudaError_t e = launch_kernel(qk_norm_rope_bwd_kernel<false>, dim3(grid), dim3(kQkBwdThreads), 0, s, true, qkv, wq, wk,
                                cos, sin, rope_bstride, dqp, dkp, dqkv, partial, dwq, dwk, batch, seq, n_heads, eps);
  if (e != cudaSuccess) return e;
  return launch_kernel(qk_gain_sum_kernel, dim3(16), dim3(256), 0, s, true, (const float*)partial, grid, dwq, dwk);
}

cudaError_t gated_add_launch(const __nv_bfloat16* x, const __nv_bfloat16* y, const __nv_bfloat16* gate,
                             int gate_bstride, __nv_bfloat16* out, int rows, int seq, int hidden, cudaStream_t s) {
  const long long n_vec = (long long)rows * hidden / 8;
  if (n_vec <= 0) return cudaSuccess;
  gated_add_kernel<<<grid_for(n_vec, 256), 256, 0, s>>>(x, y, gate, gate_bstride, out, n_vec, seq, hidden);
  return cudaGetLastError();
}

cudaError_t silu_gate_launch(const __nv_bfloat16* gu, __nv_bfloat16* m, int rows, int inter, cudaStream_t s) {
  const long long n_vec = (long long)rows * inter / 8;
  if (n_vec <= 0) return cudaSuccess;
  silu_gate_kernel<<<grid_for(n_vec, 256), 256, 0, s>>>(gu, m, n_vec, inter);
  return cudaGetLastError();
}

cudaError_t assemble_seq_launch(const __nv_bfloat16* text, const __nv_bfloat16* u, __nv_bfloat16* x, int batch,
                                int text_pad, int n_img, int hidden, cudaStream_t s) {
  const int vpr = hidden / 8;
  const long long total = (long long)batch * (text_pad + n_img) * vpr;
  if (total <= 0) return cudaSuccess;
  assemble_seq_kernel<<<grid_for(total, 256), 256, 0, s>>>(reinterpret_cast<const uint4*>(text),
                                                            reinterpret_cast<const uint4*>(u),
                                                            reinterpret_cast<uint4*>(x), batch, text_pad, n_img, vpr);
  return cudaGetLastError();
}

cudaError_t copy_rows_launch(const __nv_bfloat16* src, __nv_bfloat16* dst, size_t n_elems, cudaStream_t s) {
  const long long n_vec = (long long)(n_elems / 8);
  if (n_vec <= 0) return cudaSuccess;
  copy_vec_kernel<<<grid_for(n_vec, 256), 256, 0, s>>>(reinterpret_cast<const uint4*>(src),
                                                        reinterpret_cast<uint4*>(dst), n_vec);
  return cudaGetLastError();
}

cudaError_t cfg_euler_launch(const float* vel, float* latent, int n_img, int channels, float dt, float guidance,
                             int batch, cudaStream_t s) {
  const long long n = (long long)n_img * channels;
  if (n <= 0) return cudaSuccess;
  cfg_euler_kernel<<<grid_for(n, 256), 256, 0, s>>>(vel, latent, n, dt, guidance, batch);
  return cudaGetLastError();
}

cudaError_t rope_table_launch(float* cosv, float* sinv, int S, int text_pad, int grid_w, double theta, cudaStream_t s) {
  if (S <= 0) return cudaSuccess;
  rope_table_kernel<<<(S * 64 + 255) / 256, 256, 0, s>>>(cosv, sinv, S, text_pad, grid_w, theta);
  return cudaGetLastError();
}

cudaError_t rope_axes_launch(const float* pos, int rows, int n_axes, const RopeAxes& f, float* cosv, float* sinv,
                             int num_sms, cudaStream_t s) {
  const int need = (rows + 15) / 16;
  const int cap = 4 * num_sms;
  const int grid = need < cap ? need : cap;
  // (Early whatever the number of CTAs, unlike launch_early: alone 2.6 against 3.1 us at 3000 rows, 4.0 against 4.4 at
  // 9000, 8.8 against 9.3 at 75,826; behind an attention forward of 2 heads x 2 x 500 rows 13.4 against 13.6, 14.7
  // against 15.5, 19.7 against 20.1, and 0.2 us the other way behind one of 2 x 8 x 1000.)
  return launch_kernel(rope_axes_kernel, dim3(grid), dim3(256), 0, s, true, pos, rows, n_axes, f, cosv, sinv);
}

cudaError_t timestep_embedding_launch(const float* t, __nv_bfloat16* out, int batch, int dim, double scale,
                                      double max_period, cudaStream_t s) {
  const int half = dim / 2;
  timestep_embedding_kernel<<<(batch * half + 255) / 256, 256, 0, s>>>(t, out, batch, half, scale, max_period);
  return cudaGetLastError();
}

cudaError_t silu_inplace_launch(__nv_bfloat16* v, long long n, cudaStream_t s) {
  if (n <= 0) return cudaSuccess;
  silu_inplace_kernel<<<grid_for(n, 256), 256, 0, s>>>(v, n);
  return cudaGetLastError();
}

cudaError_t modulation_split_launch(const __nv_bfloat16* all, __nv_bfloat16* mods, __nv_bfloat16* fin, int batch,
                                    int n_blocks, int hidden, cudaStream_t s) {
  const long long total = (long long)batch * (6 * n_blocks + 2) * (hidden / 8);
  modulation_split_kernel<<<grid_for(total, 256), 256, 0, s>>>(reinterpret_cast<const uint4*>(all),
                                                               reinterpret_cast<uint4*>(mods),
                                                               reinterpret_cast<uint4*>(fin), batch, n_blocks,
                                                               hidden / 8);
  return cudaGetLastError();
}

cudaError_t time_advance_launch(float* t, int n, float dt, cudaStream_t s) {
  if (n <= 0) return cudaSuccess;
  time_advance_kernel<<<(n + 255) / 256, 256, 0, s>>>(t, n, dt);
  return cudaGetLastError();
}

cudaError_t f32_to_bf16_launch(const float* src, __nv_bfloat16* dst, size_t n, cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  f32_to_bf16_kernel<<<grid_for((long long)n, 256), 256, 0, s>>>(src, dst, (long long)n);
  return cudaGetLastError();
}

}  // namespace mi
