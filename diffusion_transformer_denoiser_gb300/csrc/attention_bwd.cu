// Gradient of the attention at head dim 128.  With s_ij = q_i k_j / sqrt(128) (masked keys -inf) and
// P = exp(s - lse), lse from the forward, the probabilities are recomputed tile by tile:
//   D_i = sum_d dO_id O_id        dP = dO V^T        dS = P (dP - D)
//   dV = P^T dO       dK = dS^T Q / sqrt(128)        dQ = dS K / sqrt(128)
// Two passes share the five products so that every sum runs inside one CTA, in a fixed order and in
// fp32, without atomics: one over the key tiles (dK, dV) and one over the query tiles (dQ).
#include "mi_internal.h"
#include "ptx.cuh"

namespace mi {

namespace {

constexpr int BT = 128;                    // rows of every tile
constexpr int kThreads = 256;
constexpr int TILE_BYTES = BT * kHeadDim * 2;
constexpr int HALF_BYTES = TILE_BYTES / 2;
constexpr int OFF_A = 0;                   // the CTA's own two tiles
constexpr int OFF_B = 2 * TILE_BYTES;      // the streamed two tiles
constexpr int OFF_STAT = 4 * TILE_BYTES;   // lse2, delta of 128 queries
constexpr int OFF_BAR = OFF_STAT + 2 * BT * 4;
constexpr int SMEM_TOTAL = OFF_BAR + 64 + 1024;
constexpr uint32_t TM_S = 0, TM_DP = 128, TM_ACC0 = 256, TM_ACC1 = 384, TM_COLS = 512;

__device__ __forceinline__ float inf() { return __int_as_float(0x7f800000); }

// One half-warp per row of one head: D_i and the base-2 log-sum-exp.  Rows without a valid key and
// the rows that fill the last tile get +inf, so that exp2(s - lse2) is zero for them.
__global__ void __launch_bounds__(256) attn_bwd_rows_kernel(const AttnBwdArgs p) {
  grid_dep_wait();
  const long long item = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 4;
  const int sub = threadIdx.x & 15;
  const long long total = (long long)p.batch * p.seq_pad * p.n_heads;
  if (item >= total) return;
  const int h = (int)(item % p.n_heads);
  const long long r = item / p.n_heads;
  const int s = (int)(r % p.seq_pad);
  const int b = (int)(r / p.seq_pad);
  const size_t at = ((size_t)b * p.n_heads + h) * p.seq_pad + s;
  float acc = 0.0f;
  if (s < p.seq) {
    const size_t off = ((size_t)b * p.seq + s) * p.n_heads * kHeadDim + (size_t)h * kHeadDim + sub * 8;
    const uint4 x = *reinterpret_cast<const uint4*>(p.o + off);
    const uint4 g = *reinterpret_cast<const uint4*>(p.d_o + off);
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, gs[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) acc += bf16_lo(xs[i]) * bf16_lo(gs[i]) + bf16_hi(xs[i]) * bf16_hi(gs[i]);
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o, 16);
  if (sub == 0) {
    float l = -inf();
    if (s < p.seq) l = p.lse[((size_t)b * p.n_heads + h) * p.seq + s];
    p.lse2[at] = l == -inf() ? inf() : l * 1.4426950408889634f;
    p.delta[at] = acc;
  }
}

// kKeys: the CTA holds a tile of keys (K, V) and walks the query tiles (Q, dO), with scores transposed
// (a TMEM lane is a key) so that P^T and dS^T are A operands of dV and dK in TMEM.  Otherwise it holds
// a tile of queries and walks the key tiles, a lane is a query, and dS is the A operand of dQ.
template <bool kKeys>
__global__ void __launch_bounds__(kThreads, 1)
    attn_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                    const AttnBwdArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + (kKeys ? OFF_B : OFF_A);
  uint8_t* sDO = sQ + TILE_BYTES;
  uint8_t* sK = smem + (kKeys ? OFF_A : OFF_B);
  uint8_t* sV = sK + TILE_BYTES;
  float* s_lse = reinterpret_cast<float*>(smem + OFF_STAT);
  float* s_delta = s_lse + BT;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint64_t* done = full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(full + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(full, 1);
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_wait();

  const int S = p.seq;
  const int n_tiles = p.seq_pad / BT;
  const int own = (int)(blockIdx.x % n_tiles);
  const int bh = (int)(blockIdx.x / n_tiles);
  const int b = bh / p.n_heads, h = bh % p.n_heads;
  const int half = warp >> 2;                  // column half of this thread
  const int r = (warp & 3) * 32 + lane;        // TMEM lane
  const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  const uint8_t* mask = p.key_mask != nullptr ? p.key_mask + (size_t)b * S : nullptr;
  const float* g_lse = p.lse2 + (size_t)bh * p.seq_pad;
  const float* g_delta = p.delta + (size_t)bh * p.seq_pad;
  constexpr uint32_t idesc_kk = idesc_bf16(128, 128, false, false);
  constexpr uint32_t idesc_mn = idesc_bf16(128, 128, false, true);
  bool key_ok = true;                          // kKeys: this lane's key may be attended to
  float l_own = 0.0f, d_own = 0.0f;            // !kKeys: this lane's row statistics
  if (kKeys) {
    key_ok = own * BT + r < S && (mask == nullptr || mask[own * BT + r] != 0);
  } else {
    l_own = g_lse[own * BT + r];
    d_own = g_delta[own * BT + r];
  }

  auto load_q = [&](int t) {
    tma_load_3d(sQ, &tmQ, full, 0, t * BT, bh);
    tma_load_3d(sQ + HALF_BYTES, &tmQ, full, 64, t * BT, bh);
    tma_load_4d(sDO, &tmDO, full, 0, h, t * BT, b);
    tma_load_4d(sDO + HALF_BYTES, &tmDO, full, 64, h, t * BT, b);
  };
  auto load_kv = [&](int t) {
    tma_load_3d(sK, &tmK, full, 0, t * BT, bh);
    tma_load_3d(sK + HALF_BYTES, &tmK, full, 64, t * BT, bh);
    tma_load_4d(sV, &tmV, full, 0, h, t * BT, b);
    tma_load_4d(sV + HALF_BYTES, &tmV, full, 64, h, t * BT, b);
  };
  auto mma_ss = [&](uint32_t d, uint8_t* a, uint8_t* bt) {  // D = A B^T, both row-major in d
    const uint64_t ad = sdesc_sw128(smem_u32(a), 16, 1024), bd = sdesc_sw128(smem_u32(bt), 16, 1024);
    for (int kk = 0; kk < 8; ++kk) {
      const uint32_t off = ((uint32_t)(kk >> 2) * HALF_BYTES + (uint32_t)(kk & 3) * 32u) >> 4;
      tc_mma_ss_warp(d, ad + off, bd + off, idesc_kk, kk > 0 ? 1u : 0u);
    }
  };
  auto mma_ts = [&](uint32_t d, uint32_t a, uint8_t* bt, bool first) {  // D (+)= A B, A in TMEM
    const uint64_t bd = sdesc_sw128(smem_u32(bt), HALF_BYTES, 1024);
    for (int kk = 0; kk < 8; ++kk)
      tc_mma_ts_warp(d, a + (uint32_t)(kk >> 2) * 64u + (uint32_t)(kk & 3) * 8u, bd + (uint32_t)kk * (2048u >> 4),
                     idesc_mn, (!first || kk > 0) ? 1u : 0u);
  };

  bool ok = true;
  uint32_t ph_done = 0;
  for (int t = 0; t < n_tiles; ++t) {
    if (threadIdx.x == 0) {
      mbar_arrive_expect_tx(full, (t == 0 ? 4 : 2) * TILE_BYTES);
      if (kKeys || t == 0) load_q(kKeys ? t : own);
      if (!kKeys || t == 0) load_kv(kKeys ? own : t);
    }
    if (kKeys && threadIdx.x < BT) {
      s_lse[threadIdx.x] = g_lse[t * BT + threadIdx.x];
      s_delta[threadIdx.x] = g_delta[t * BT + threadIdx.x];
    }
    ok = mbar_wait(full, (uint32_t)(t & 1), abort_flag, p.err, DEV_TIMEOUT_ATTN_BWD + 1);
    if (__syncthreads_or(!ok)) break;
    if (warp == 0) {
      if (!kKeys && mask != nullptr) zero_masked_rows(sK, mask, t * BT, S, lane);
      __syncwarp();
      tc_fence_after();
      mma_ss(tmem + TM_S, kKeys ? sK : sQ, kKeys ? sQ : sK);
      mma_ss(tmem + TM_DP, kKeys ? sV : sDO, kKeys ? sDO : sV);
      tc_commit_warp(done);
    }
    ok = mbar_wait(done, ph_done, abort_flag, p.err, DEV_TIMEOUT_ATTN_BWD + 2);
    ph_done ^= 1;
    if (__syncthreads_or(!ok)) break;
    tc_fence_after();
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
      uint32_t sr[32], dr[32];
      const int c0 = half * 64 + c * 32;
      tmem_ld32(t_lane + TM_S + c0, sr);
      tmem_ld32(t_lane + TM_DP + c0, dr);
      tmem_ld_wait();
      uint32_t valid = 0xffffffffu;
      if (!kKeys) {
        const int kc = t * BT + c0 + lane;
        valid = __ballot_sync(0xffffffffu, kc < S && (mask == nullptr || mask[kc < S ? kc : 0] != 0));
      } else if (!key_ok) {
        valid = 0;
      }
      float pv[32], dv[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float l = kKeys ? s_lse[c0 + i] : l_own, d = kKeys ? s_delta[c0 + i] : d_own;
        const float e = ex2_approx(fmaf(__uint_as_float(sr[i]), p.scale_log2, -l));
        const bool v = (valid >> i) & 1u;
        pv[i] = v ? e : 0.0f;
        dv[i] = v ? e * (__uint_as_float(dr[i]) - d) : 0.0f;
      }
      // bf16 pairs over the first 32 columns of this thread's own half
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        sr[i] = pack_bf16x2(pv[2 * i], pv[2 * i + 1]);
        dr[i] = pack_bf16x2(dv[2 * i], dv[2 * i + 1]);
      }
      if (kKeys) tmem_st16(t_lane + TM_S + half * 64 + c * 16, sr);
      tmem_st16(t_lane + TM_DP + half * 64 + c * 16, dr);
      tmem_st_wait();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
      tc_fence_after();
      if (kKeys) {
        mma_ts(tmem + TM_ACC0, tmem + TM_S, sDO, t == 0);
        mma_ts(tmem + TM_ACC1, tmem + TM_DP, sQ, t == 0);
      } else {
        mma_ts(tmem + TM_ACC0, tmem + TM_DP, sK, t == 0);
      }
      tc_commit_warp(done);
    }
    ok = mbar_wait(done, ph_done, abort_flag, p.err, DEV_TIMEOUT_ATTN_BWD + 3);
    ph_done ^= 1;
    if (__syncthreads_or(!ok)) break;
  }
  if (ok) {
    tc_fence_after();
    const int row = own * BT + r;
#pragma unroll 1
    for (int c = 0; c < (kKeys ? 4 : 2); ++c) {
      const bool second = c >= 2;
      uint32_t x[32];
      tmem_ld32(t_lane + (second ? TM_ACC1 : TM_ACC0) + half * 64 + (c & 1) * 32, x);
      tmem_ld_wait();
      const float f = kKeys && !second ? 1.0f : p.scale;
      __nv_bfloat16* dst = kKeys && !second ? p.dv + ((size_t)b * S + row) * 3 * p.n_heads * kHeadDim + (size_t)h * kHeadDim
                                            : (kKeys ? p.dkp : p.dqp) + ((size_t)bh * S + row) * kHeadDim;
      if (row < S) {
        uint4* d4 = reinterpret_cast<uint4*>(dst + half * 64 + (c & 1) * 32);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = pack_bf16x2(__uint_as_float(x[v * 8 + 2 * e]) * f, __uint_as_float(x[v * 8 + 2 * e + 1]) * f);
          d4[v] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, TM_COLS);
  }
}

template <bool kKeys>
cudaError_t pass_launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tdo,
                        const AttnBwdArgs& a, int dev, cudaStream_t s) {
  static bool attr_done[kMaxDevices] = {};
  if (!attr_done[dev]) {
    cudaError_t e = cudaFuncSetAttribute(attn_bwd_kernel<kKeys>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_TOTAL);
    if (e != cudaSuccess) return e;
    attr_done[dev] = true;
  }
  const unsigned grid = (unsigned)((long long)a.batch * a.n_heads * (a.seq_pad / BT));
  return launch_kernel(attn_bwd_kernel<kKeys>, dim3(grid), dim3(kThreads), SMEM_TOTAL, s, true, tq, tk, tv, tdo, a);
}

}  // namespace

cudaError_t attention_bwd_launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                 const CUtensorMap& tdo, const AttnBwdArgs& a, cudaStream_t s) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  const long long rows = (long long)a.batch * a.n_heads * a.seq_pad;
  e = launch_kernel(attn_bwd_rows_kernel, dim3((unsigned)((rows + 15) / 16)), dim3(256), 0, s, true, a);
  if (e != cudaSuccess) return e;
  e = pass_launch<true>(tq, tk, tv, tdo, a, dev, s);
  if (e != cudaSuccess) return e;
  return pass_launch<false>(tq, tk, tv, tdo, a, dev, s);
}

}  // namespace mi
