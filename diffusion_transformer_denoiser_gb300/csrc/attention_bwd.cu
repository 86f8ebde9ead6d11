// Gradient of the attention at head dim 128.  With s_ij = q_i k_j / sqrt(128) (masked keys -inf) and
// P = exp(s - lse), lse from the forward, the probabilities are recomputed tile by tile:
//   D_i = sum_d dO_id O_id        dP = dO V^T        dS = P (dP - D)
//   dV = P^T dO       dK = dS^T Q / sqrt(128)        dQ = dS K / sqrt(128)
//
// Two passes share the products so that every sum runs inside one CTA, in a fixed order and in fp32,
// without atomics: results repeat bit for bit.  The keys pass holds 128 keys (K, V) and walks the query
// tiles: S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q.  The queries pass holds 128 queries
// (Q, dO) and walks the key tiles: S, dP, dQ += dS K.  That is 7 products of 128 x 128 x 128 per pair of
// tiles where 5 are needed; the alternative, one pass that adds dQ tiles into memory, either gives up
// the fixed order or makes CTAs wait for one another, and moves 64 KB of fp32 sums per pair of tiles.
// One launch runs both: the CTAs of the keys pass come first, those of the (shorter) queries pass fill
// the SMs as they free up.
//
// In both passes a TMEM lane is a row of the tile the CTA holds, so P^T and dS^T (keys) or dS (queries)
// go back to TMEM as bf16 and are the A operand of the product that sums over the streamed rows; the
// streamed tiles serve both as the row-major operand of S and dP and, read along the other axis, as the
// B operand of the sums.  Roles (384 threads, one CTA per SM):
//   * warp 0: TMA producer: the CTA's own tiles, then the streamed tiles in rings of 2 or 3 stages.
//   * warp 1: issues the MMAs (convergent warp, one elected lane per instruction).
//       keys:    dV_n, S_{n+1} | dK_n, dP_{n+1}, each pair behind one wait: P_n (over S_n) and dS_n (over
//                dP_n) are in the columns that the next scores overwrite, and the MMAs of one thread
//                execute in order.  P is computed while dK_{n-1}, dP_n run, dS while dV_n, S_{n+1} do.
//       queries: S_{n+1} | dP_{n+1} | dQ_n.  With one accumulator less, Q is kept in TMEM (no shared-memory
//                reads for it: those bound the scores' products) and dS has columns of its own, so the
//                next scores wait only for the present ones to be in registers.
//   * warp 2: wait proxy: adds an arrival to the barriers above once the tile that the next product
//     streams has landed, so that the issuer waits once per pair of products; it also clears masked K
//     rows (queries pass): zero times an infinity or NaN in a padded row would not be zero.
//   * warps 4-11: two warpgroups, each half of the 128 streamed rows; one thread per lane.
// P and dS are rounded to bf16 once, as matrix operands; scores, D, sums and P in dS are fp32.
#include "mi_internal.h"
#include "ptx.cuh"

namespace mi {

namespace {

constexpr int BT = 128;                    // rows of every tile
constexpr int kThreads = 384;
// Register split as in the forward: the launch's pool (384 x 168), given to the compute warpgroups.
constexpr int kRegsLaunch = 168;
constexpr int kRegsControl = 104;
constexpr int kRegsCompute = 200;
static_assert(128 * kRegsControl + 256 * kRegsCompute <= kThreads * kRegsLaunch, "register split exceeds the launch pool");
constexpr int TILE_BYTES = BT * kHeadDim * 2;
constexpr int HALF_BYTES = TILE_BYTES / 2;
constexpr int STAT_BYTES = 2 * BT * 4;     // -lse2 and -delta of 128 queries

// Shared memory: seven tiles, keys pass K | V | Q ring of 3 | dO ring of 2 and the row statistics with it;
// queries pass dO | K ring of 3 | V ring of 3.  Then the statistics (keys) or one bit per key tile
// (queries pass with a mask), and the barriers.
constexpr int kRingX = 3;
constexpr int OFF_X_KEYS = 2 * TILE_BYTES, OFF_Y_KEYS = OFF_X_KEYS + kRingX * TILE_BYTES;
constexpr int OFF_X_QUERIES = TILE_BYTES, OFF_Y_QUERIES = OFF_X_QUERIES + kRingX * TILE_BYTES;
constexpr int OFF_STAT = 7 * TILE_BYTES;
constexpr int kTileWords = 256;                    // 8192 tiles = 2^20 keys
constexpr int OFF_BAR = OFF_STAT + 2 * STAT_BYTES;
static_assert(kTileWords * 4 <= 2 * STAT_BYTES, "the tile bits take the statistics' place");
constexpr int SMEM_TOTAL = OFF_BAR + 256;          // the tiles need a base at a multiple of 1024 bytes

constexpr uint32_t TM_COLS = 512;
constexpr uint32_t TM_S = 0, TM_DP = 128;
constexpr uint32_t TM_DV = 256, TM_DK = 384;               // keys pass
constexpr uint32_t TM_DQ = 256, TM_Q = 384, TM_DS = 448;   // queries pass

__device__ __forceinline__ float inf() { return __int_as_float(0x7f800000); }

// One half-warp per row of one head: -D_i and minus the base-2 log-sum-exp (negated: the passes add
// them).  Rows without a valid key and the rows that fill the last tile get -inf, so that
// exp2(s - lse2) is zero for them.
__global__ void __launch_bounds__(256) attn_bwd_rows_kernel(const AttnBwdArgs p) {
  grid_dep_wait();
  grid_dep_launch();
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
    p.nlse2[at] = l == -inf() ? -inf() : l * -1.4426950408889634f;
    p.ndelta[at] = -acc;
  }
}

struct Bars {
  uint64_t own_x, own_y;                   // the CTA's own tiles: K / V or (Q in TMEM) / dO
  uint64_t x_full[kRingX], x_empty[kRingX];  // streamed tiles: Q or K
  uint64_t y_full[kRingX], y_empty[kRingX];  // dO (2 stages) or V (3)
  uint64_t first;                          // queries pass: the first K tile has landed and is clean
  uint64_t s_full, dp_full;                // scores in TMEM
  uint64_t s_read, dp_read;                // queries pass: scores in registers, and the next K / V landed
  uint64_t p_full, ds_full;                // P, dS in TMEM; keys pass: and the next Q / dO landed
  uint64_t acc_done;
  uint32_t tmem_slot;
  int abort_flag;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

// Position in a ring of kStages: the stage and the parity of its phase.
template <int kStages>
struct Ring {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++st == kStages) {
      st = 0;
      ph ^= 1u;
    }
  }
};

constexpr uint32_t kTile16 = TILE_BYTES >> 4;  // descriptor start addresses count 16 bytes
constexpr uint32_t kIdescScores = idesc_bf16(128, 128, false, false);
constexpr uint32_t kIdescSum = idesc_bf16(128, 128, false, true);

// D = A B^T over d, both tiles row-major in shared memory.
__device__ __forceinline__ void scores_ss(uint32_t d, uint64_t a, uint64_t b) {
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const uint32_t off = ((uint32_t)(kk >> 2) * HALF_BYTES + (uint32_t)(kk & 3) * 32u) >> 4;
    tc_mma_ss_warp(d, a + off, b + off, kIdescScores, kk > 0 ? 1u : 0u);
  }
}

// The same with A in TMEM.
__device__ __forceinline__ void scores_ts(uint32_t d, uint32_t a, uint64_t b) {
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const uint32_t off = ((uint32_t)(kk >> 2) * HALF_BYTES + (uint32_t)(kk & 3) * 32u) >> 4;
    tc_mma_ts_warp(d, a + (uint32_t)kk * 8u, b + off, kIdescScores, kk > 0 ? 1u : 0u);
  }
}

// D (+)= A B over the 128 streamed rows, A (P or dS) in TMEM: the two warpgroups' halves `half_cols` columns
// apart, B read along its rows.
__device__ __forceinline__ void sum_ts(uint32_t d, uint32_t a, uint32_t half_cols, uint64_t b, bool first) {
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    tc_mma_ts_warp(d, a + (uint32_t)(kk >> 2) * half_cols + (uint32_t)(kk & 3) * 8u, b + (uint32_t)kk * (2048u >> 4),
                   kIdescSum, (!first || kk > 0) ? 1u : 0u);
}

// 32 accumulator columns of a row, scaled, as bf16; zeros when the CTA walked no tile.
__device__ __forceinline__ void store32(__nv_bfloat16* dst, uint32_t src, float f, bool any, bool in_range) {
  uint32_t x[32];
  if (any) {
    tmem_ld32(src, x);
    tmem_ld_wait();
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = 0u;
  }
  if (!in_range) return;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = pack_bf16x2(__uint_as_float(x[v * 8 + 2 * e]) * f, __uint_as_float(x[v * 8 + 2 * e + 1]) * f);
    reinterpret_cast<uint4*>(dst)[v] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

__device__ __forceinline__ f32x2_t pair_of(const uint32_t* x) { return f2_pack(__uint_as_float(x[0]), __uint_as_float(x[1])); }

// ------------------------------------------------------------------------------------ keys pass
// K and V of 128 keys stay; Q and dO of n_tiles query tiles are walked.
__device__ __forceinline__ void keys_pass(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                          const CUtensorMap& tmDO, const AttnBwdArgs& p, uint8_t* smem, Bars* bars,
                                          uint32_t tmem, int own, int bh, int n_tiles) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.seq;
  const int b = bh / p.n_heads, h = bh % p.n_heads;
  volatile int* abort_flag = &bars->abort_flag;
  int* err = p.err;
  uint8_t* sK = smem;
  uint8_t* sV = smem + TILE_BYTES;
  uint8_t* sQ = smem + OFF_X_KEYS;
  uint8_t* sDO = smem + OFF_Y_KEYS;
  float* sStat = reinterpret_cast<float*>(smem + OFF_STAT);

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    if (warp == 0) {
      if (lane == 0 && n_tiles > 0) {
        // ---------------------------------------------------------------- TMA producer
        const float* nl = p.nlse2 + (size_t)bh * p.seq_pad;
        const float* nd = p.ndelta + (size_t)bh * p.seq_pad;
        Ring<kRingX> x;
        Ring<2> y;
        int nx = 0, ny = 0;
        mbar_arrive_expect_tx(&bars->own_x, TILE_BYTES);
        tma_load_3d(sK, &tmK, &bars->own_x, 0, own * BT, bh);
        tma_load_3d(sK + HALF_BYTES, &tmK, &bars->own_x, 64, own * BT, bh);
        for (int t = 0; t < n_tiles; ++t) {
          if (nx >= kRingX && !mbar_wait(&bars->x_empty[x.st], x.ph ^ 1u, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 1)) break;
          uint8_t* dq = sQ + x.st * TILE_BYTES;
          mbar_arrive_expect_tx(&bars->x_full[x.st], TILE_BYTES);
          tma_load_3d(dq, &tmQ, &bars->x_full[x.st], 0, t * BT, bh);
          tma_load_3d(dq + HALF_BYTES, &tmQ, &bars->x_full[x.st], 64, t * BT, bh);
          ++nx;
          x.next();
          if (t == 0) {
            mbar_arrive_expect_tx(&bars->own_y, TILE_BYTES);
            tma_load_4d(sV, &tmV, &bars->own_y, 0, h, own * BT, b);
            tma_load_4d(sV + HALF_BYTES, &tmV, &bars->own_y, 64, h, own * BT, b);
          }
          if (ny >= 2 && !mbar_wait(&bars->y_empty[y.st], y.ph ^ 1u, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 1)) break;
          uint8_t* dd = sDO + y.st * TILE_BYTES;
          float* stat = sStat + y.st * (STAT_BYTES / 4);
          mbar_arrive_expect_tx(&bars->y_full[y.st], TILE_BYTES + STAT_BYTES);
          bulk_load(stat, nl + t * BT, BT * 4, &bars->y_full[y.st]);
          bulk_load(stat + BT, nd + t * BT, BT * 4, &bars->y_full[y.st]);
          tma_load_4d(dd, &tmDO, &bars->y_full[y.st], 0, h, t * BT, b);
          tma_load_4d(dd + HALF_BYTES, &tmDO, &bars->y_full[y.st], 64, h, t * BT, b);
          ++ny;
          y.next();
        }
        // drain the copies still in flight (the last use of each barrier phase)
        mbar_wait_drain(&bars->own_x, 0, err, DEV_TIMEOUT_ATTN_BWD + 2);
        mbar_wait_drain(&bars->own_y, 0, err, DEV_TIMEOUT_ATTN_BWD + 2);
        for (int j = nx - kRingX < 0 ? 0 : nx - kRingX; j < nx; ++j)
          mbar_wait_drain(&bars->x_full[j % kRingX], (uint32_t)((j / kRingX) & 1), err, DEV_TIMEOUT_ATTN_BWD + 2);
        for (int j = ny - 2 < 0 ? 0 : ny - 2; j < ny; ++j)
          mbar_wait_drain(&bars->y_full[j & 1], (uint32_t)((j >> 1) & 1), err, DEV_TIMEOUT_ATTN_BWD + 2);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------------ MMA issuer
      const uint64_t k_d = sdesc_sw128(smem_u32(sK), 16, 1024), v_d = sdesc_sw128(smem_u32(sV), 16, 1024);
      const uint64_t q_k = sdesc_sw128(smem_u32(sQ), 16, 1024), do_k = sdesc_sw128(smem_u32(sDO), 16, 1024);
      const uint64_t q_mn = sdesc_sw128(smem_u32(sQ), HALF_BYTES, 1024), do_mn = sdesc_sw128(smem_u32(sDO), HALF_BYTES, 1024);
      bool ok = true;
      if (n_tiles > 0) {
        ok = mbar_wait_warp(&bars->own_x, 0, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 3) &&
             mbar_wait_warp(&bars->x_full[0], 0, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 3);
        if (ok) {
          tc_fence_after();
          scores_ss(tmem + TM_S, k_d, q_k);
          tc_commit_warp(&bars->s_full);
          ok = mbar_wait_warp(&bars->own_y, 0, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 3) &&
               mbar_wait_warp(&bars->y_full[0], 0, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 3);
        }
        if (ok) {
          tc_fence_after();
          scores_ss(tmem + TM_DP, v_d, do_k);
          tc_commit_warp(&bars->dp_full);
        }
      }
      int xs = 0;
      for (int n = 0; ok && n < n_tiles; ++n) {
        const bool more = n + 1 < n_tiles;
        const int xn = xs + 1 == kRingX ? 0 : xs + 1;
        const int ys = n & 1;
        if (!mbar_wait_warp(&bars->p_full, (uint32_t)(n & 1), abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 4)) break;
        tc_fence_after();
        sum_ts(tmem + TM_DV, tmem + TM_S, 64, do_mn + ys * kTile16, n == 0);
        if (more) {
          scores_ss(tmem + TM_S, k_d, q_k + xn * kTile16);
          tc_commit_warp(&bars->s_full);
        }
        if (!mbar_wait_warp(&bars->ds_full, (uint32_t)(n & 1), abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 5)) break;
        tc_fence_after();
        sum_ts(tmem + TM_DK, tmem + TM_DP, 64, q_mn + xs * kTile16, n == 0);
        tc_commit_warp(&bars->x_empty[xs]);
        tc_commit_warp(&bars->y_empty[ys]);
        if (more) {
          scores_ss(tmem + TM_DP, v_d, do_k + (ys ^ 1) * kTile16);
          tc_commit_warp(&bars->dp_full);
        }
        xs = xn;
      }
      tc_commit_warp(&bars->acc_done);
      mbar_wait_drain(&bars->acc_done, 0, err, DEV_TIMEOUT_ATTN_BWD + 6);
    } else if (warp == 2) {
      // ------------------------------------------------------------------ wait proxy
      Ring<kRingX> x;
      Ring<2> y;
      for (int n = 0; n < n_tiles; ++n) {
        const bool more = n + 1 < n_tiles;
        x.next();
        y.next();
        // each arrival belongs to the barrier's phase n: phase n - 1 must be complete first
        const uint32_t prev = (uint32_t)((n - 1) & 1);
        if ((n > 0 && !mbar_wait_warp(&bars->p_full, prev, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 7)) ||
            (more && !mbar_wait_warp(&bars->x_full[x.st], x.ph, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 7)))
          break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full);
        if ((n > 0 && !mbar_wait_warp(&bars->ds_full, prev, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 8)) ||
            (more && !mbar_wait_warp(&bars->y_full[y.st], y.ph, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 8)))
          break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->ds_full);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsCompute));
    // ------------------------------------------------------------------ P and dS
    const int half = (warp - 4) >> 2;            // query half of this warpgroup
    const int r = (warp & 3) * 32 + lane;        // TMEM lane: key of the tile
    const uint32_t t_row = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t t_s = t_row + TM_S + (uint32_t)half * 64u, t_dp = t_row + TM_DP + (uint32_t)half * 64u;
    const int row = own * BT + r;
    const uint8_t* mask = p.key_mask != nullptr ? p.key_mask + (size_t)b * S : nullptr;
    const bool row_ok = row < S && (mask == nullptr || mask[row] != 0);
    const bool rows_ok = __all_sync(0xffffffffu, row_ok) != 0;
    const f32x2_t sl2x2 = f2_pack(p.scale_log2, p.scale_log2);
    bool ok = true;
    for (int n = 0; n < n_tiles; ++n) {
      const int st = n & 1;
      const uint32_t ph = (uint32_t)(n & 1);
      // the statistics land with dO, well before the scores are there
      if (!mbar_wait_warp(&bars->y_full[st], (uint32_t)((n >> 1) & 1), abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 9)) {
        ok = false;
        break;
      }
      const float4* stat = reinterpret_cast<const float4*>(sStat + st * (STAT_BYTES / 4) + half * 64);
      float4 nl[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) nl[i] = stat[i];
      if (!mbar_wait_warp(&bars->s_full, ph, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 10)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t pr[64], pk[32];
      tmem_ld32(t_s, pr);
      tmem_ld32(t_s + 32, pr + 32);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float z[4];
        f2_unpack(f2_fma(pair_of(pr + 4 * i), sl2x2, f2_pack(nl[i].x, nl[i].y)), z[0], z[1]);
        f2_unpack(f2_fma(pair_of(pr + 4 * i + 2), sl2x2, f2_pack(nl[i].z, nl[i].w)), z[2], z[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) pr[4 * i + e] = __float_as_uint(ex2_approx(z[e]));
      }
      if (!rows_ok) {  // a masked key's scores may be anything
#pragma unroll
        for (int i = 0; i < 64; ++i) pr[i] = row_ok ? pr[i] : 0u;
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) pk[i] = pack_bf16x2(__uint_as_float(pr[2 * i]), __uint_as_float(pr[2 * i + 1]));
      tmem_st32(t_s, pk);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->p_full);
      float4 nd[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) nd[i] = stat[32 + i];
      if (!mbar_wait_warp(&bars->dp_full, ph, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 11)) {
        ok = false;
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t dp[32];
        tmem_ld32(t_dp + 32 * c, dp);
        if (c == 1) {
#pragma unroll
          for (int i = 0; i < 8; ++i) nd[i] = stat[40 + i];
        }
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 d = nd[i];
          float z[4];
          f2_unpack(f2_mul(f2_add(pair_of(dp + 4 * i), f2_pack(d.x, d.y)), pair_of(pr + 32 * c + 4 * i)), z[0], z[1]);
          f2_unpack(f2_mul(f2_add(pair_of(dp + 4 * i + 2), f2_pack(d.z, d.w)), pair_of(pr + 32 * c + 4 * i + 2)), z[2], z[3]);
          if (!rows_ok) {
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = row_ok ? z[e] : 0.0f;
          }
          pk[16 * c + 2 * i] = pack_bf16x2(z[0], z[1]);
          pk[16 * c + 2 * i + 1] = pack_bf16x2(z[2], z[3]);
        }
      }
      tmem_st32(t_dp, pk);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->ds_full);
    }
    // warpgroup 0 stores dV, warpgroup 1 dK
    if (ok && n_tiles > 0) ok = mbar_wait_warp(&bars->acc_done, 0, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 12);
    if (ok) {
      tc_fence_after();
      __nv_bfloat16* dst = half == 0 ? p.dv + ((size_t)b * S + row) * 3 * p.n_heads * kHeadDim + (size_t)h * kHeadDim
                                     : p.dkp + ((size_t)bh * S + row) * kHeadDim;
      const uint32_t src = t_row + (half == 0 ? TM_DV : TM_DK);
#pragma unroll 1
      for (int c = 0; c < 4; ++c) store32(dst + c * 32, src + c * 32, half == 0 ? 1.0f : p.scale, n_tiles > 0, row < S);
      tc_fence_before();
    }
  }
}

// ------------------------------------------------------------------------------------ queries pass
// Q (in TMEM) and dO of 128 queries stay; K and V of the key tiles are walked, those without a valid key
// left out.
__device__ __forceinline__ void queries_pass(const CUtensorMap& tmK, const CUtensorMap& tmV, const CUtensorMap& tmDO,
                                             const AttnBwdArgs& p, uint8_t* smem, Bars* bars, uint32_t tmem, int own,
                                             int bh, int n_tiles) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.seq;
  const int b = bh / p.n_heads, h = bh % p.n_heads;
  const uint8_t* mask = p.key_mask != nullptr ? p.key_mask + (size_t)b * S : nullptr;
  volatile int* abort_flag = &bars->abort_flag;
  int* err = p.err;
  uint8_t* sDO = smem;
  uint8_t* sK = smem + OFF_X_QUERIES;
  uint8_t* sV = smem + OFF_Y_QUERIES;
  const uint32_t* tile_any = reinterpret_cast<const uint32_t*>(smem + OFF_STAT);
  auto next = [&](int t) {  // first tile from t on that is walked
    if (mask != nullptr)
      while (t < n_tiles && !((tile_any[t >> 5] >> (t & 31)) & 1u)) ++t;
    return t;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    if (warp == 0) {
      if (lane == 0 && next(0) < n_tiles) {
        // ---------------------------------------------------------------- TMA producer
        Ring<kRingX> x;
        int nx = 0, ny = 0;
        bool own_sent = false;
        for (int t = next(0); t < n_tiles; t = next(t + 1), x.next()) {
          if (nx >= kRingX && !mbar_wait(&bars->x_empty[x.st], x.ph ^ 1u, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 1)) break;
          uint8_t* dk = sK + x.st * TILE_BYTES;
          mbar_arrive_expect_tx(&bars->x_full[x.st], TILE_BYTES);
          tma_load_3d(dk, &tmK, &bars->x_full[x.st], 0, t * BT, bh);
          tma_load_3d(dk + HALF_BYTES, &tmK, &bars->x_full[x.st], 64, t * BT, bh);
          ++nx;
          if (!own_sent) {
            own_sent = true;
            mbar_arrive_expect_tx(&bars->own_y, TILE_BYTES);
            tma_load_4d(sDO, &tmDO, &bars->own_y, 0, h, own * BT, b);
            tma_load_4d(sDO + HALF_BYTES, &tmDO, &bars->own_y, 64, h, own * BT, b);
          }
          if (ny >= kRingX && !mbar_wait(&bars->y_empty[x.st], x.ph ^ 1u, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 1)) break;
          uint8_t* dv = sV + x.st * TILE_BYTES;
          mbar_arrive_expect_tx(&bars->y_full[x.st], TILE_BYTES);
          tma_load_4d(dv, &tmV, &bars->y_full[x.st], 0, h, t * BT, b);
          tma_load_4d(dv + HALF_BYTES, &tmV, &bars->y_full[x.st], 64, h, t * BT, b);
          ++ny;
        }
        mbar_wait_drain(&bars->own_y, 0, err, DEV_TIMEOUT_ATTN_BWD + 2);
        for (int j = nx - kRingX < 0 ? 0 : nx - kRingX; j < nx; ++j)
          mbar_wait_drain(&bars->x_full[j % kRingX], (uint32_t)((j / kRingX) & 1), err, DEV_TIMEOUT_ATTN_BWD + 2);
        for (int j = ny - kRingX < 0 ? 0 : ny - kRingX; j < ny; ++j)
          mbar_wait_drain(&bars->y_full[j % kRingX], (uint32_t)((j / kRingX) & 1), err, DEV_TIMEOUT_ATTN_BWD + 2);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------------ MMA issuer
      const uint64_t do_d = sdesc_sw128(smem_u32(sDO), 16, 1024);
      const uint64_t k_k = sdesc_sw128(smem_u32(sK), 16, 1024), v_k = sdesc_sw128(smem_u32(sV), 16, 1024);
      const uint64_t k_mn = sdesc_sw128(smem_u32(sK), HALF_BYTES, 1024);
      int t = next(0);
      bool ok = true;
      if (t < n_tiles) {
        ok = mbar_wait_warp(&bars->own_x, 0, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 3) &&
             mbar_wait_warp(&bars->first, 0, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 3);
        if (ok) {
          tc_fence_after();
          scores_ts(tmem + TM_S, tmem + TM_Q, k_k);
          tc_commit_warp(&bars->s_full);
          ok = mbar_wait_warp(&bars->own_y, 0, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 3) &&
               mbar_wait_warp(&bars->y_full[0], 0, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 3);
        }
        if (ok) {
          tc_fence_after();
          scores_ss(tmem + TM_DP, do_d, v_k);
          tc_commit_warp(&bars->dp_full);
          tc_commit_warp(&bars->y_empty[0]);
        }
      }
      int st = 0;
      for (int n = 0; ok && t < n_tiles; ++n) {
        const int t1 = next(t + 1);
        const bool more = t1 < n_tiles;
        const int sn = st + 1 == kRingX ? 0 : st + 1;
        const uint32_t ph = (uint32_t)(n & 1);
        if (more) {
          if (!mbar_wait_warp(&bars->s_read, ph, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 4)) break;
          tc_fence_after();
          scores_ts(tmem + TM_S, tmem + TM_Q, k_k + sn * kTile16);
          tc_commit_warp(&bars->s_full);
          if (!mbar_wait_warp(&bars->dp_read, ph, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 4)) break;
          tc_fence_after();
          scores_ss(tmem + TM_DP, do_d, v_k + sn * kTile16);
          tc_commit_warp(&bars->dp_full);
          tc_commit_warp(&bars->y_empty[sn]);
        }
        if (!mbar_wait_warp(&bars->ds_full, ph, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 5)) break;
        tc_fence_after();
        sum_ts(tmem + TM_DQ, tmem + TM_DS, 32, k_mn + st * kTile16, n == 0);
        tc_commit_warp(&bars->x_empty[st]);
        st = sn;
        t = t1;
      }
      tc_commit_warp(&bars->acc_done);
      mbar_wait_drain(&bars->acc_done, 0, err, DEV_TIMEOUT_ATTN_BWD + 6);
    } else if (warp == 2) {
      // ------------------------------------------------------------------ wait proxy, cleaner
      Ring<kRingX> x;
      int n = 0;
      for (int t = next(0); t < n_tiles; ++n, x.next()) {
        // K of this tile, clean, for S_n: an arrival of phase n - 1 of s_read (phase n - 2 complete)
        uint32_t bad[4] = {0, 0, 0, 0};
        if (mask != nullptr) masked_keys(mask, t * BT, S, lane, bad);
        if ((n > 1 && !mbar_wait_warp(&bars->s_read, (uint32_t)(n & 1), abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 7)) ||
            !mbar_wait_warp(&bars->x_full[x.st], x.ph, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 7))
          break;
        zero_rows(sK + x.st * TILE_BYTES, bad, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(n == 0 ? &bars->first : &bars->s_read);
        // V of this tile, for dP_n
        if (n > 0) {
          if ((n > 1 && !mbar_wait_warp(&bars->dp_read, (uint32_t)(n & 1), abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 8)) ||
              !mbar_wait_warp(&bars->y_full[x.st], x.ph, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 8))
            break;
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->dp_read);
        }
        t = next(t + 1);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsCompute));
    // ------------------------------------------------------------------ dS
    const int half = (warp - 4) >> 2;            // key half of this warpgroup
    const int r = (warp & 3) * 32 + lane;        // TMEM lane: query of the tile
    const uint32_t t_row = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t t_s = t_row + TM_S + (uint32_t)half * 64u, t_dp = t_row + TM_DP + (uint32_t)half * 64u;
    const uint32_t t_ds = t_row + TM_DS + (uint32_t)half * 32u;
    const int row = own * BT + r;
    const f32x2_t sl2x2 = f2_pack(p.scale_log2, p.scale_log2);
    {
      // this row's half of Q to TMEM: element d in column d / 2, as in memory
      uint32_t q[32];
      const uint4* src = reinterpret_cast<const uint4*>(p.qp + ((size_t)bh * S + (row < S ? row : 0)) * kHeadDim + half * 64);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 v = row < S ? src[i] : make_uint4(0, 0, 0, 0);
        q[4 * i] = v.x;
        q[4 * i + 1] = v.y;
        q[4 * i + 2] = v.z;
        q[4 * i + 3] = v.w;
      }
      tmem_st32(t_row + TM_Q + (uint32_t)half * 32u, q);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->own_x);
    }
    const float nl = p.nlse2[(size_t)bh * p.seq_pad + row], nd = p.ndelta[(size_t)bh * p.seq_pad + row];
    const f32x2_t nl2 = f2_pack(nl, nl), nd2 = f2_pack(nd, nd);
    // may this lane's two keys of the tile be attended to (read a tile ahead)
    bool key[2] = {true, true};
    auto read_mask = [&](int t) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int kc = t * BT + half * 64 + w * 32 + lane;
        key[w] = kc < S && (mask == nullptr || mask[kc < S ? kc : 0] != 0);
      }
    };
    bool ok = true;
    int n = 0;
    Ring<kRingX> before;  // stage and phase of the tile before this one
    int t = next(0);
    if (t < n_tiles) read_mask(t);
    for (int t1; t < n_tiles; t = t1, ++n) {
      const uint32_t ph = (uint32_t)(n & 1);
      t1 = next(t + 1);
      const uint32_t valid[2] = {__ballot_sync(0xffffffffu, key[0]), __ballot_sync(0xffffffffu, key[1])};
      if (t1 < n_tiles) read_mask(t1);
      if (!mbar_wait_warp(&bars->s_full, ph, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 10)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t pr[64], dp[64], pk[32];
      tmem_ld32(t_s, pr);
      tmem_ld32(t_s + 32, pr + 32);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->s_read);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        float z0, z1;
        f2_unpack(f2_fma(pair_of(pr + 2 * i), sl2x2, nl2), z0, z1);
        pr[2 * i] = __float_as_uint(ex2_approx(z0));
        pr[2 * i + 1] = __float_as_uint(ex2_approx(z1));
      }
      if (!mbar_wait_warp(&bars->dp_full, ph, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 11)) {
        ok = false;
        break;
      }
      tc_fence_after();
      tmem_ld32(t_dp, dp);
      tmem_ld32(t_dp + 32, dp + 32);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->dp_read);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        float z0, z1;
        f2_unpack(f2_mul(f2_add(pair_of(dp + 2 * i), nd2), pair_of(pr + 2 * i)), z0, z1);
        dp[2 * i] = __float_as_uint(z0);
        dp[2 * i + 1] = __float_as_uint(z1);
      }
      if ((valid[0] & valid[1]) != 0xffffffffu) {  // a masked key's dP may be anything
#pragma unroll
        for (int i = 0; i < 64; ++i) dp[i] = (valid[i >> 5] >> (i & 31)) & 1u ? dp[i] : 0u;
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) pk[i] = pack_bf16x2(__uint_as_float(dp[2 * i]), __uint_as_float(dp[2 * i + 1]));
      // dQ of the tile before has read its dS
      if (n > 0) {
        if (!mbar_wait_warp(&bars->x_empty[before.st], before.ph, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 9)) {
          ok = false;
          break;
        }
        before.next();
        tc_fence_after();
      }
      tmem_st32(t_ds, pk);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->ds_full);
    }
    if (ok && n > 0) ok = mbar_wait_warp(&bars->acc_done, 0, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 12);
    if (ok) {
      tc_fence_after();
      __nv_bfloat16* dst = p.dqp + ((size_t)bh * S + row) * kHeadDim + half * 64;
#pragma unroll 1
      for (int c = 0; c < 2; ++c)
        store32(dst + c * 32, t_row + TM_DQ + (uint32_t)(half * 64 + c * 32), p.scale, n > 0, row < S);
      tc_fence_before();
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    attn_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                    const AttnBwdArgs p) {
  // The swizzled tiles need a base at a multiple of 1024 bytes, which the window of dynamic shared memory
  // of a kernel without static shared memory has (checked: a launch elsewhere would report, not compute).
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicCAS(p.err, 0, DEV_TIMEOUT_ATTN_BWD);
    return;
  }
  Bars* bars = reinterpret_cast<Bars*>(smem + OFF_BAR);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_tiles = p.seq_pad / BT;
  const unsigned units = (unsigned)(p.batch * p.n_heads) * (unsigned)n_tiles;
  const bool keys = blockIdx.x < units;
  const unsigned unit = keys ? blockIdx.x : blockIdx.x - units;
  const int own = (int)(unit % n_tiles), bh = (int)(unit / n_tiles);
  if (threadIdx.x == 0) {
    mbar_init(&bars->own_x, keys ? 1 : 8);
    mbar_init(&bars->own_y, 1);
    for (int i = 0; i < kRingX; ++i) {
      mbar_init(&bars->x_full[i], 1);
      mbar_init(&bars->y_full[i], 1);
      mbar_init(&bars->x_empty[i], 1);
      mbar_init(&bars->y_empty[i], 1);
    }
    mbar_init(&bars->first, 1);
    mbar_init(&bars->s_full, 1);
    mbar_init(&bars->dp_full, 1);
    // 8 compute warps, and the wait proxy where it adds the next tile's landing
    mbar_init(&bars->s_read, 9);
    mbar_init(&bars->dp_read, 9);
    mbar_init(&bars->p_full, 9);
    mbar_init(&bars->ds_full, keys ? 9 : 8);
    mbar_init(&bars->acc_done, 1);
    bars->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_slot, TM_COLS);
    tmem_relinquish();
  }
  grid_dep_wait();
  grid_dep_launch();
  // With a mask: a tile of keys without a valid one has zero gradients (keys pass) and is not walked
  // (queries pass).
  const uint8_t* mask = p.key_mask != nullptr ? p.key_mask + (size_t)(bh / p.n_heads) * p.seq : nullptr;
  bool walk = true;
  if (keys && mask != nullptr) {
    const int key = own * BT + (int)threadIdx.x;
    walk = __syncthreads_or(threadIdx.x < BT && key < p.seq && mask[key < p.seq ? key : 0] != 0) != 0;
  } else if (mask != nullptr) {
    uint32_t* tile_any = reinterpret_cast<uint32_t*>(smem + OFF_STAT);
    for (int i = threadIdx.x; i < (n_tiles + 31) / 32; i += kThreads) tile_any[i] = 0;
    __syncthreads();
    for (int t = warp; t < n_tiles; t += kThreads / 32) {
      bool any = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int kc = t * BT + i * 32 + lane;
        any |= kc < p.seq && mask[kc < p.seq ? kc : 0] != 0;
      }
      if (__any_sync(0xffffffffu, any) && lane == 0) atomicOr(&tile_any[t >> 5], 1u << (t & 31));
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_slot;
  if (keys) {
    keys_pass(tmQ, tmK, tmV, tmDO, p, smem, bars, tmem, own, bh, walk ? n_tiles : 0);
  } else {
    queries_pass(tmK, tmV, tmDO, p, smem, bars, tmem, own, bh, n_tiles);
  }
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, TM_COLS);
  }
}

}  // namespace

cudaError_t attention_bwd_launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                 const CUtensorMap& tdo, const AttnBwdArgs& a, cudaStream_t s) {
  static bool attr_done[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!attr_done[dev]) {
    e = cudaFuncSetAttribute(attn_bwd_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_TOTAL);
    if (e != cudaSuccess) return e;
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, attn_bwd_kernel);
    if (e != cudaSuccess) return e;
    if (fa.numRegs * kThreads < 128 * kRegsControl + 256 * kRegsCompute) return cudaErrorInvalidConfiguration;
    attr_done[dev] = true;
  }
  const long long rows = (long long)a.batch * a.n_heads * a.seq_pad;
  e = launch_kernel(attn_bwd_rows_kernel, dim3((unsigned)((rows + 15) / 16)), dim3(256), 0, s, true, a);
  if (e != cudaSuccess) return e;
  return launch_kernel(attn_bwd_kernel, dim3((unsigned)(2 * rows / BT)), dim3(kThreads), SMEM_TOTAL, s, true, tq, tk, tv,
                       tdo, a);
}

}  // namespace mi
