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
// are written back over their scores as bf16 and are the A operand of the product that sums over the
// streamed rows; the streamed tiles serve both as the row-major operand of S and dP and, read along
// the other axis, as the B operand of the sums.  Roles (384 threads, one CTA per SM):
//   * warp 0: TMA producer.  The CTA's own two tiles, then the two streamed tiles in rings of 2 stages.
//   * warp 1: issues the MMAs, in an order that keeps the tensor core busy while the scores of a tile
//     are turned into P and dS:   keys:    dV_i, S_{i+1} | dK_i, dP_{i+1}
//                                 queries: S_{i+1} | dQ_i, dP_{i+1}
//     (S_{i+1} has a second buffer in the queries pass, which has one accumulator less).
//   * warp 2: clears masked K rows in shared memory (queries pass with a key mask): zero times an
//     infinity or NaN in a padded row would not be zero.
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

constexpr int OFF_OWN = 0;                         // K, V (keys pass) or Q, dO (queries pass)
constexpr int OFF_X = OFF_OWN + 2 * TILE_BYTES;    // 2 stages: Q (keys pass) or K (queries pass)
constexpr int OFF_Y = OFF_X + 2 * TILE_BYTES;      // 2 stages: dO or V
constexpr int OFF_STAT = OFF_Y + 2 * TILE_BYTES;   // 2 stages
constexpr int OFF_TILES = OFF_STAT + 2 * STAT_BYTES;  // queries pass with a mask: one bit per key tile
constexpr int kTileWords = 256;                    // 8192 tiles = 2^20 keys
constexpr int OFF_BAR = OFF_TILES + kTileWords * 4;
constexpr int SMEM_TOTAL = OFF_BAR + 256 + 1024;

constexpr uint32_t TM_COLS = 512;
constexpr uint32_t TM_S = 0, TM_DP = 128;
constexpr uint32_t TM_DV = 256, TM_DK = 384;   // keys pass
constexpr uint32_t TM_S1 = 256, TM_DQ = 384;   // queries pass: the second score buffer

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
  uint64_t own_x, own_y;           // the CTA's own tiles: K / V or Q / dO
  uint64_t x_full[2], y_full[2];   // streamed tiles
  uint64_t x_empty[2], y_empty[2];
  uint64_t x_clean[2];             // queries pass with a mask: masked rows of K are zero
  uint64_t s_full[2], dp_full;     // scores in TMEM (two buffers in the queries pass)
  uint64_t p_full[2], ds_full[2];  // first and second half of each warpgroup's columns written
  uint64_t acc_done;
  uint32_t tmem_slot;
  int abort_flag;
};
static_assert(sizeof(Bars) <= 256, "barrier block");

// 16 consecutive columns of one warpgroup's half: element j of `pk` holds columns 2 j and 2 j + 1.
__device__ __forceinline__ uint32_t a_column(int kk) {
  // K slice kk (16 streamed rows): warpgroup kk / 4 wrote it over the first half of its own columns
  return (uint32_t)(kk >> 2) * 64u + (uint32_t)(kk & 3) * 8u;
}

// One pass of one CTA: `own` is its tile, `bh` its batch element and head, n_tiles the tiles to walk.
template <bool kKeys>
__device__ __forceinline__ void bwd_pass(const CUtensorMap& tmX, const CUtensorMap& tmY, const CUtensorMap& tmOwnX,
                                         const CUtensorMap& tmOwnY, const AttnBwdArgs& p, uint8_t* smem, Bars* bars,
                                         uint32_t tmem, int own, int bh, int n_tiles) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.seq;
  const int b = bh / p.n_heads, h = bh % p.n_heads;
  const uint8_t* mask = p.key_mask != nullptr ? p.key_mask + (size_t)b * S : nullptr;
  volatile int* abort_flag = &bars->abort_flag;
  int* err = p.err;
  uint8_t* sOwnX = smem + OFF_OWN;
  uint8_t* sOwnY = sOwnX + TILE_BYTES;
  uint8_t* sX = smem + OFF_X;
  uint8_t* sY = smem + OFF_Y;
  float* sStat = reinterpret_cast<float*>(smem + OFF_STAT);
  uint32_t* tile_any = reinterpret_cast<uint32_t*>(smem + OFF_TILES);
  const bool skip = !kKeys && mask != nullptr;  // key tiles without a valid key are left out
  // first tile from t on that is walked
  auto next = [&](int t) {
    if (skip)
      while (t < n_tiles && !((tile_any[t >> 5] >> (t & 31)) & 1u)) ++t;
    return t;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    if (warp == 0) {
      if (lane == 0) {
        // ------------------------------------------------------------------ TMA producer
        // keys pass: x = Q (3-D map), y = dO (4-D), own = K (3-D), V (4-D);
        // queries pass: x = K (3-D), y = V (4-D), own = Q (3-D), dO (4-D)
        int t = next(0);
        int n = 0;
        bool ok = true;
        if (t < n_tiles) {
          mbar_arrive_expect_tx(&bars->own_x, TILE_BYTES);
          tma_load_3d(sOwnX, &tmOwnX, &bars->own_x, 0, own * BT, bh);
          tma_load_3d(sOwnX + HALF_BYTES, &tmOwnX, &bars->own_x, 64, own * BT, bh);
        }
        int y_n = 0;
        for (; t < n_tiles; t = next(t + 1), ++n) {
          const int st = n & 1;
          const uint32_t ph = (uint32_t)((n >> 1) & 1);
          if (n >= 2 && !mbar_wait(&bars->x_empty[st], ph ^ 1u, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 1)) {
            ok = false;
            break;
          }
          uint8_t* dx = sX + st * TILE_BYTES;
          mbar_arrive_expect_tx(&bars->x_full[st], TILE_BYTES + (kKeys ? STAT_BYTES : 0));
          tma_load_3d(dx, &tmX, &bars->x_full[st], 0, t * BT, bh);
          tma_load_3d(dx + HALF_BYTES, &tmX, &bars->x_full[st], 64, t * BT, bh);
          if (kKeys) {
            float* stat = sStat + st * (STAT_BYTES / 4);
            bulk_load(stat, p.nlse2 + (size_t)bh * p.seq_pad + t * BT, BT * 4, &bars->x_full[st]);
            bulk_load(stat + BT, p.ndelta + (size_t)bh * p.seq_pad + t * BT, BT * 4, &bars->x_full[st]);
          }
          if (n == 0) {
            mbar_arrive_expect_tx(&bars->own_y, TILE_BYTES);
            tma_load_4d(sOwnY, &tmOwnY, &bars->own_y, 0, h, own * BT, b);
            tma_load_4d(sOwnY + HALF_BYTES, &tmOwnY, &bars->own_y, 64, h, own * BT, b);
          }
          if (n >= 2 && !mbar_wait(&bars->y_empty[st], ph ^ 1u, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 1)) {
            ++n;
            ok = false;
            break;
          }
          uint8_t* dy = sY + st * TILE_BYTES;
          mbar_arrive_expect_tx(&bars->y_full[st], TILE_BYTES);
          tma_load_4d(dy, &tmY, &bars->y_full[st], 0, h, t * BT, b);
          tma_load_4d(dy + HALF_BYTES, &tmY, &bars->y_full[st], 64, h, t * BT, b);
          y_n = n + 1;
        }
        (void)ok;
        // drain the copies still in flight (the last use of each barrier phase)
        if (n > 0) {
          mbar_wait_drain(&bars->own_x, 0, err, DEV_TIMEOUT_ATTN_BWD + 2);
          mbar_wait_drain(&bars->own_y, 0, err, DEV_TIMEOUT_ATTN_BWD + 2);
        }
        for (int j = n - 2 < 0 ? 0 : n - 2; j < n; ++j)
          mbar_wait_drain(&bars->x_full[j & 1], (uint32_t)((j >> 1) & 1), err, DEV_TIMEOUT_ATTN_BWD + 2);
        for (int j = y_n - 2 < 0 ? 0 : y_n - 2; j < y_n; ++j)
          mbar_wait_drain(&bars->y_full[j & 1], (uint32_t)((j >> 1) & 1), err, DEV_TIMEOUT_ATTN_BWD + 2);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------------ MMA issuer
      constexpr uint32_t idesc_s = idesc_bf16(128, 128, false, false);
      constexpr uint32_t idesc_acc = idesc_bf16(128, 128, false, true);
      const uint64_t own_x = sdesc_sw128(smem_u32(sOwnX), 16, 1024), own_y = sdesc_sw128(smem_u32(sOwnY), 16, 1024);
      // streamed tiles as row-major (K-major) operand and, for the sums, along the other axis
      const uint64_t x_k = sdesc_sw128(smem_u32(sX), 16, 1024), y_k = sdesc_sw128(smem_u32(sY), 16, 1024);
      const uint64_t x_mn = sdesc_sw128(smem_u32(sX), HALF_BYTES, 1024), y_mn = sdesc_sw128(smem_u32(sY), HALF_BYTES, 1024);
      constexpr uint32_t kStage = TILE_BYTES >> 4;  // descriptor start addresses count 16 bytes
      auto issue_scores = [&](uint32_t d, uint64_t a, uint64_t bt) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = ((uint32_t)(kk >> 2) * HALF_BYTES + (uint32_t)(kk & 3) * 32u) >> 4;
          tc_mma_ss_warp(d, a + off, bt + off, idesc_s, kk > 0 ? 1u : 0u);
        }
      };
      // the K slices of column half c of both warpgroups
      auto issue_sum = [&](uint32_t d, uint32_t a, uint64_t bt, int c, bool first) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int kk = (j >> 1) * 4 + 2 * c + (j & 1);
          tc_mma_ts_warp(d, a + a_column(kk), bt + (uint32_t)kk * (2048u >> 4), idesc_acc, (!first || c > 0 || j > 0) ? 1u : 0u);
        }
      };
      uint64_t* x_ready = skip ? bars->x_clean : bars->x_full;
      int t = next(0);
      bool ok = true;
      if (t < n_tiles) {
        ok = mbar_wait_warp(&bars->own_x, 0, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 3) &&
             mbar_wait_warp(&x_ready[0], 0, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 3);
        if (ok) {
          tc_fence_after();
          issue_scores(tmem + TM_S, own_x, x_k);
          tc_commit_warp(&bars->s_full[0]);
          ok = mbar_wait_warp(&bars->own_y, 0, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 3) &&
               mbar_wait_warp(&bars->y_full[0], 0, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 3);
        }
        if (ok) {
          tc_fence_after();
          issue_scores(tmem + TM_DP, own_y, y_k);
          tc_commit_warp(&bars->dp_full);
          if (!kKeys) tc_commit_warp(&bars->y_empty[0]);
        }
      }
      for (int n = 0; ok && t < n_tiles; ++n) {
        const int t1 = next(t + 1);
        const bool more = t1 < n_tiles;
        const int st = n & 1, nst = st ^ 1;
        const uint32_t ph = (uint32_t)(n & 1), nph = (uint32_t)(((n + 1) >> 1) & 1);
        const bool first = n == 0;
        if (kKeys) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (!ok) break;
            ok = mbar_wait_warp(&bars->p_full[c], ph, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 4);
            if (ok) {
              tc_fence_after();
              issue_sum(tmem + TM_DV, tmem + TM_S, y_mn + st * kStage, c, first);
            }
          }
          if (!ok) break;
          tc_commit_warp(&bars->y_empty[st]);
          if (more) {  // P_i, in the same columns, has been read: the MMAs of one thread execute in order
            ok = mbar_wait_warp(&x_ready[nst], nph, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 5);
            if (!ok) break;
            tc_fence_after();
            issue_scores(tmem + TM_S, own_x, x_k + nst * kStage);
            tc_commit_warp(&bars->s_full[0]);
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (!ok) break;
            ok = mbar_wait_warp(&bars->ds_full[c], ph, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 6);
            if (ok) {
              tc_fence_after();
              issue_sum(tmem + TM_DK, tmem + TM_DP, x_mn + st * kStage, c, first);
            }
          }
          if (!ok) break;
          tc_commit_warp(&bars->x_empty[st]);
          if (more) {
            ok = mbar_wait_warp(&bars->y_full[nst], nph, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 7);
            if (!ok) break;
            tc_fence_after();
            issue_scores(tmem + TM_DP, own_y, y_k + nst * kStage);
            tc_commit_warp(&bars->dp_full);
          }
        } else {
          if (more) {  // S of the tile before this one has been read: its dS was waited for
            ok = mbar_wait_warp(&x_ready[nst], nph, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 5);
            if (!ok) break;
            tc_fence_after();
            issue_scores(tmem + (nst ? TM_S1 : TM_S), own_x, x_k + nst * kStage);
            tc_commit_warp(&bars->s_full[nst]);
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (!ok) break;
            ok = mbar_wait_warp(&bars->ds_full[c], ph, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 6);
            if (ok) {
              tc_fence_after();
              issue_sum(tmem + TM_DQ, tmem + TM_DP, x_mn + st * kStage, c, first);
            }
          }
          if (!ok) break;
          tc_commit_warp(&bars->x_empty[st]);
          if (more) {
            ok = mbar_wait_warp(&bars->y_full[nst], nph, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 7);
            if (!ok) break;
            tc_fence_after();
            issue_scores(tmem + TM_DP, own_y, y_k + nst * kStage);
            tc_commit_warp(&bars->dp_full);
            tc_commit_warp(&bars->y_empty[nst]);
          }
        }
        t = t1;
      }
      tc_commit_warp(&bars->acc_done);
      mbar_wait_drain(&bars->acc_done, 0, err, DEV_TIMEOUT_ATTN_BWD + 8);
    } else if (warp == 2 && skip) {
      // ------------------------------------------------------------------ cleaner of masked K rows
      int n = 0;
      for (int t = next(0); t < n_tiles; t = next(t + 1), ++n) {
        const int st = n & 1;
        uint32_t bad[4];
        masked_keys(mask, t * BT, S, lane, bad);
        if (!mbar_wait_warp(&bars->x_full[st], (uint32_t)((n >> 1) & 1), abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 9)) break;
        zero_rows(sX + st * TILE_BYTES, bad, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->x_clean[st]);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsCompute));
    // ------------------------------------------------------------------ P and dS
    const int half = (warp - 4) >> 2;            // column half of this warpgroup
    const int r = (warp & 3) * 32 + lane;        // TMEM lane: row of the CTA's own tile
    const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)half * 64u;
    const int row = own * BT + r;
    const f32x2_t sl2x2 = f2_pack(p.scale_log2, p.scale_log2);
    // keys pass: the lane's key; queries pass: the lane's row statistics
    bool row_ok = true, rows_ok = true;
    f32x2_t nl2 = 0ull, nd2 = 0ull;
    if (kKeys) {
      row_ok = row < S && (mask == nullptr || mask[row] != 0);
      rows_ok = __all_sync(0xffffffffu, row_ok) != 0;
    } else {
      const float nl = p.nlse2[(size_t)bh * p.seq_pad + row], nd = p.ndelta[(size_t)bh * p.seq_pad + row];
      nl2 = f2_pack(nl, nl);
      nd2 = f2_pack(nd, nd);
    }
    // queries pass: may this lane's two keys of the tile be attended to (read a tile ahead)
    bool key[2] = {true, true};
    auto read_mask = [&](int t) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int kc = t * BT + half * 64 + w * 32 + lane;
        key[w] = kc < S && (!skip || mask[kc < S ? kc : 0] != 0);
      }
    };
    bool ok = true;
    int n = 0;
    int t = next(0);
    if (!kKeys && t < n_tiles) read_mask(t);
    for (int t1; t < n_tiles; t = t1, ++n) {
      const int st = n & 1;
      t1 = next(t + 1);
      uint32_t valid[2] = {0xffffffffu, 0xffffffffu};
      if (!kKeys) {
        valid[0] = __ballot_sync(0xffffffffu, key[0]);
        valid[1] = __ballot_sync(0xffffffffu, key[1]);
        if (t1 < n_tiles) read_mask(t1);
      }
      const uint32_t t_s = t_lane + (!kKeys && st ? TM_S1 : TM_S);
      if (!mbar_wait_warp(&bars->s_full[kKeys ? 0 : st], (uint32_t)((kKeys ? n : n >> 1) & 1), abort_flag, err,
                          DEV_TIMEOUT_ATTN_BWD + 10) ||
          (kKeys && !mbar_wait_warp(&bars->x_full[st], (uint32_t)((n >> 1) & 1), abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 10))) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t pr[64];
      tmem_ld32(t_s, pr);
      tmem_ld32(t_s + 32, pr + 32);
      tmem_ld_wait();
      const float4* nl4 = reinterpret_cast<const float4*>(sStat + st * (STAT_BYTES / 4) + half * 64);
      const float4* nd4 = reinterpret_cast<const float4*>(sStat + st * (STAT_BYTES / 4) + BT + half * 64);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int q = 0; q < 8; ++q) {  // four columns
          const int i = c * 32 + q * 4;
          f32x2_t la = nl2, lb = nl2;
          if (kKeys) {
            const float4 l = nl4[c * 8 + q];
            la = f2_pack(l.x, l.y);
            lb = f2_pack(l.z, l.w);
          }
          float z[4];
          f2_unpack(f2_fma(f2_pack(__uint_as_float(pr[i]), __uint_as_float(pr[i + 1])), sl2x2, la), z[0], z[1]);
          f2_unpack(f2_fma(f2_pack(__uint_as_float(pr[i + 2]), __uint_as_float(pr[i + 3])), sl2x2, lb), z[2], z[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) pr[i + e] = __float_as_uint(ex2_approx(z[e]));
        }
        if (kKeys) {
          if (!rows_ok) {
#pragma unroll
            for (int i = 0; i < 32; ++i) pr[c * 32 + i] = row_ok ? pr[c * 32 + i] : 0u;
          }
#pragma unroll
          for (int i = 0; i < 16; ++i)
            pk[i] = pack_bf16x2(__uint_as_float(pr[c * 32 + 2 * i]), __uint_as_float(pr[c * 32 + 2 * i + 1]));
          tmem_st16(t_s + c * 16, pk);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->p_full[c]);
        }
      }
      if (!mbar_wait_warp(&bars->dp_full, (uint32_t)(n & 1), abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 11)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t dp[64];
      tmem_ld32(t_lane + TM_DP, dp);
      tmem_ld32(t_lane + TM_DP + 32, dp + 32);
      tmem_ld_wait();
      const bool all = kKeys ? rows_ok : (valid[0] & valid[1]) == 0xffffffffu;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int i = c * 32 + q * 4;
          f32x2_t da = nd2, db = nd2;
          if (kKeys) {
            const float4 d = nd4[c * 8 + q];
            da = f2_pack(d.x, d.y);
            db = f2_pack(d.z, d.w);
          }
          float z[4];
          f2_unpack(f2_mul(f2_add(f2_pack(__uint_as_float(dp[i]), __uint_as_float(dp[i + 1])), da),
                           f2_pack(__uint_as_float(pr[i]), __uint_as_float(pr[i + 1]))), z[0], z[1]);
          f2_unpack(f2_mul(f2_add(f2_pack(__uint_as_float(dp[i + 2]), __uint_as_float(dp[i + 3])), db),
                           f2_pack(__uint_as_float(pr[i + 2]), __uint_as_float(pr[i + 3]))), z[2], z[3]);
          if (!all) {  // a masked key's dP may be anything
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool keep = kKeys ? row_ok : (valid[c] >> (q * 4 + e)) & 1u;
              z[e] = keep ? z[e] : 0.0f;
            }
          }
          pk[q * 2] = pack_bf16x2(z[0], z[1]);
          pk[q * 2 + 1] = pack_bf16x2(z[2], z[3]);
        }
        tmem_st16(t_lane + TM_DP + c * 16, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->ds_full[c]);
      }
    }
    // ------------------------------------------------------------------ outputs
    // Warpgroup 0 stores dV (keys pass) or the first half of dQ, warpgroup 1 dK or the second half.
    // A CTA that walked no tile (all its keys masked, or no valid key for its queries) stores zeros.
    if (ok && n > 0) ok = mbar_wait_warp(&bars->acc_done, 0, abort_flag, err, DEV_TIMEOUT_ATTN_BWD + 12);
    if (ok) {
      tc_fence_after();
      const bool is_v = kKeys && half == 0;
      const float f = is_v ? 1.0f : p.scale;
      __nv_bfloat16* dst = is_v ? p.dv + ((size_t)b * S + row) * 3 * p.n_heads * kHeadDim + (size_t)h * kHeadDim
                                : (kKeys ? p.dkp : p.dqp + half * 64) + ((size_t)bh * S + row) * kHeadDim;
      const uint32_t src = (t_lane - (uint32_t)half * 64u) + (kKeys ? (half ? TM_DK : TM_DV) : TM_DQ + (uint32_t)half * 64u);
#pragma unroll 1
      for (int c = 0; c < (kKeys ? 4 : 2); ++c) {
        uint32_t x[32];
        if (n > 0) {
          tmem_ld32(src + c * 32, x);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = 0u;
        }
        if (row < S) {
          uint4* d4 = reinterpret_cast<uint4*>(dst + c * 32);
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
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    attn_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                    const AttnBwdArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + OFF_BAR);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_tiles = p.seq_pad / BT;
  const unsigned units = (unsigned)(p.batch * p.n_heads) * (unsigned)n_tiles;
  const bool keys = blockIdx.x < units;
  const unsigned unit = keys ? blockIdx.x : blockIdx.x - units;
  const int own = (int)(unit % n_tiles), bh = (int)(unit / n_tiles);
  if (threadIdx.x == 0) {
    mbar_init(&bars->own_x, 1);
    mbar_init(&bars->own_y, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->x_full[i], 1);
      mbar_init(&bars->y_full[i], 1);
      mbar_init(&bars->x_empty[i], 1);
      mbar_init(&bars->y_empty[i], 1);
      mbar_init(&bars->x_clean[i], 1);
      mbar_init(&bars->s_full[i], 1);
      mbar_init(&bars->p_full[i], 8);
      mbar_init(&bars->ds_full[i], 8);
    }
    mbar_init(&bars->dp_full, 1);
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
    uint32_t* tile_any = reinterpret_cast<uint32_t*>(smem + OFF_TILES);
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
    bwd_pass<true>(tmQ, tmDO, tmK, tmV, p, smem, bars, tmem, own, bh, walk ? n_tiles : 0);
  } else {
    bwd_pass<false>(tmK, tmV, tmQ, tmDO, p, smem, bars, tmem, own, bh, walk ? n_tiles : 0);
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
