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
// One persistent launch runs both: a CTA takes units (a tile of one head) of the keys pass until there are
// none, then units of the (shorter) queries pass.  The first unit follows from the CTA's index, the others
// come from a counter in the workspace; which CTA computes a unit does not change its result.  The tiles
// of successive units form one stream: while the last tile of a unit is worked on, the next unit's own
// tiles land and its first scores are computed, and its first P (keys) or dS (queries) is withheld until
// the accumulators of the unit before have been read out.
//
// In both passes a TMEM lane is a row of the tile the CTA holds, so P^T and dS^T (keys) or dS (queries)
// go back to TMEM as bf16 and are the A operand of the product that sums over the streamed rows; the
// streamed tiles serve both as the row-major operand of S and dP and, read along the other axis, as the
// B operand of the sums.  Roles (384 threads, one CTA per SM):
//   * warp 0: takes the units (one whose keys are all masked gets its zeros here and is left out) and is
//     the TMA producer: the CTA's own tiles, the streamed tiles in rings of 2 or 3 stages.
//   * warp 1: issues the MMAs (convergent warp, one elected lane).
//       keys:    dV_n, S_{n+1} | dK_n, dP_{n+1}, each pair behind one wait: P_n (over S_n) and dS_n (over
//                dP_n) are in the columns that the next scores overwrite, and the MMAs of one thread
//                execute in order.  P is computed while dK_{n-1}, dP_n run, dS while dV_n, S_{n+1} do.
//       queries: S_{n+1} | dP_{n+1} | dQ_n.  With one accumulator less, Q is kept in TMEM (no shared-memory
//                reads for it: those bound the scores' products) and dS has columns of its own, so the
//                next scores wait only for the present ones to be in registers.
//   * warp 2: wait proxy: adds an arrival to the barriers above once the tile that the next product
//     streams has landed, so that the issuer waits once per pair of products; it also clears masked K
//     rows (queries pass): zero times an infinity or NaN in a padded row would not be zero.
//   * warps 4-11: two warpgroups, each half of the 128 streamed rows; one thread per lane.  They also read
//     the accumulators out (queries pass: through shared memory, stored by TMA, a warp its own 32 rows).
// Both passes are bound by the latency from a tile's scores to its P or dS, and sensitive to the length of the
// code (the roles' loops share the SM's instruction cache).  Shorter code was what made them faster, for 24 heads
// x 4130 rows in bursts (at the power cap that a second of calls reaches, 6 to 9 % more):
//   * unit ends that are read and stored in rolled loops, and masks applied in one place to the packed words;
//     then 460 us
//   * one election for the 8 MMAs of a product, where each had its own: 447
//   * waits with a single poll in the code, and a vote on its answer, where a first test without a vote had
//     saved the vote: 432
//   * descriptors made from one word, the producers' loops not unrolled: 424
// and in the queries pass the loads of dP asked for before the exponentials of S: 418.  Slower: four warpgroups
// with a quarter of the columns each, MMAs issued from loops, scores read and P stored in halves.  Cutting units
// along the streamed rows, with fp32 parts that another kernel adds up, pays for a single head of 1000 rows or
// more (4130: 34 instead of 49 us) and costs from two heads on (2 x 4130: 60 instead of 48), so it is not done.
// P and dS are rounded to bf16 once, as matrix operands; scores, D, sums and P in dS are fp32.  D is a sum over the
// output as the forward stored it, in bf16: P dP, which has no such rounding, would have to be summed before the
// first dS of a row.  It shows where a row's weight sits on few keys and dP - D cancels: against 64 bits dQ and dK are
// off by 0.0024 of their norm for scores of variance 1 either way, and by 0.0040 instead of 0.0024 for variance 36.
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

// Shared memory: seven tiles, keys pass K | V | Q ring of 3 | dO ring of 2, queries pass dO | K ring of 3 |
// V ring of 2 | output staging; then the row statistics that come with dO (keys pass) and the barriers of
// either pass.  Q and K are asked for half a tile's time after the sum that frees their stage, so two stages
// of them leave the tensor core waiting for copies (a ring of 2 for Q: 7.23 against 6.92 ms at 16418 rows).
constexpr int kRingQ = 3, kRingDO = 2, kRingK = 3, kRingV = 2;
constexpr int OFF_Q = 2 * TILE_BYTES, OFF_DO = OFF_Q + kRingQ * TILE_BYTES;
constexpr int OFF_K = TILE_BYTES, OFF_V = OFF_K + kRingK * TILE_BYTES;
constexpr int OFF_OUT = 6 * TILE_BYTES;
constexpr int OFF_STAT = 7 * TILE_BYTES;
constexpr int OFF_BAR = OFF_STAT + kRingDO * STAT_BYTES;
constexpr int kBarBytes = 256;
constexpr int SMEM_TOTAL = OFF_BAR + 2 * kBarBytes;  // the tiles need a base at a multiple of 1024 bytes
static_assert(OFF_DO + kRingDO * TILE_BYTES == OFF_STAT && OFF_V + kRingV * TILE_BYTES == OFF_OUT, "seven tiles");
static_assert(SMEM_TOTAL <= 232448, "shared memory of one CTA");

constexpr uint32_t TM_COLS = 512;
constexpr uint32_t TM_S = 0, TM_DP = 128;
constexpr uint32_t TM_DV = 256, TM_DK = 384;               // keys pass
constexpr uint32_t TM_DQ = 256, TM_Q = 384, TM_DS = 448;   // queries pass

__device__ __forceinline__ float inf() { return __int_as_float(0x7f800000); }

// Prepares a call.  One half-warp per row of one head: -D_i and minus the base-2 log-sum-exp (negated: the
// passes add them).  Rows without a valid key and the rows that fill the last tile get -inf, so that
// exp2(s - lse2) is zero for them.  With a key mask, the first `batch` blocks list the key tiles of an element
// that hold a valid key.  The unit counters start at zero.
constexpr int kRowHeads = 4;

__global__ void __launch_bounds__(256) attn_bwd_rows_kernel(const AttnBwdArgs p, bool early) {
  __shared__ int n_listed;
  __shared__ int ballot_of[8];
  grid_dep_wait();
  if (early) grid_dep_launch();
  int block = blockIdx.x;
  if (block == 0 && threadIdx.x < 2) p.counters[threadIdx.x] = 0;
  if (p.key_mask != nullptr) {
    if (block < p.batch) {
      const int n_tiles = p.seq_pad / BT;
      const uint8_t* mask = p.key_mask + (size_t)block * p.seq;
      const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
      if (threadIdx.x == 0) n_listed = 0;
      for (int t0 = 0; t0 < n_tiles; t0 += 8) {  // eight tiles at a time, one per warp
        const int t = t0 + warp;
        bool any = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int kc = t * BT + i * 32 + lane;
          any |= kc < p.seq && mask[kc < p.seq ? kc : 0] != 0;
        }
        any = __any_sync(0xffffffffu, any) != 0;
        if (lane == 0) ballot_of[warp] = any;
        __syncthreads();
        if (any && lane == 0) {
          int at = n_listed;
          for (int w = 0; w < warp; ++w) at += ballot_of[w];
          p.tiles[(size_t)block * n_tiles + at] = t;
        }
        __syncthreads();
        if (threadIdx.x == 0)
          for (int w = 0; w < 8; ++w) n_listed += ballot_of[w];
        __syncthreads();
      }
      if (threadIdx.x == 0) p.n_listed[block] = n_listed;
      return;
    }
    block -= p.batch;
  }
  // kRowHeads heads of a row per half-warp, all their loads in flight
  const long long item = ((long long)block * blockDim.x + threadIdx.x) >> 4;
  const int sub = threadIdx.x & 15;
  const int groups = (p.n_heads + kRowHeads - 1) / kRowHeads;
  if (item >= (long long)p.batch * p.seq_pad * groups) return;
  const int h0 = (int)(item % groups) * kRowHeads;
  const long long r = item / groups;
  const int s = (int)(r % p.seq_pad);
  const int b = (int)(r / p.seq_pad);
  const bool in = s < p.seq;
  const size_t off = ((size_t)b * p.seq + (in ? s : 0)) * p.n_heads * kHeadDim + (size_t)h0 * kHeadDim + sub * 8;
  uint4 x[kRowHeads], g[kRowHeads];
  float l[kRowHeads];
#pragma unroll
  for (int i = 0; i < kRowHeads; ++i) {
    const bool on = in && h0 + i < p.n_heads;
    x[i] = on ? *reinterpret_cast<const uint4*>(p.o + off + i * kHeadDim) : make_uint4(0, 0, 0, 0);
    g[i] = on ? *reinterpret_cast<const uint4*>(p.d_o + off + i * kHeadDim) : make_uint4(0, 0, 0, 0);
    l[i] = on ? p.lse[((size_t)b * p.n_heads + h0 + i) * p.seq + s] : -inf();
  }
#pragma unroll
  for (int i = 0; i < kRowHeads; ++i) {
    const uint32_t xs[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, gs[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
    float acc = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc += bf16_lo(xs[e]) * bf16_lo(gs[e]) + bf16_hi(xs[e]) * bf16_hi(gs[e]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o, 16);
    if (sub == 0 && h0 + i < p.n_heads) {
      const size_t at = ((size_t)b * p.n_heads + h0 + i) * p.seq_pad + s;
      p.nlse2[at] = l[i] == -inf() ? -inf() : l[i] * -1.4426950408889634f;
      p.ndelta[at] = -acc;
    }
  }
}

struct Bars {
  uint64_t own_x, own_y;           // the CTA's own tiles: K / V or (first unit's Q in TMEM) / dO
  uint64_t own_x_empty, own_y_empty;
  uint64_t x_full[3], x_empty[3];  // streamed tiles: Q or K
  uint64_t y_full[2], y_empty[2];  // dO or V
  uint64_t first;                  // queries pass: the first K tile has landed and is clean
  uint64_t s_full, dp_full;        // scores in TMEM
  uint64_t s_read, dp_read;        // queries pass: scores in registers, and the next K / V landed
  uint64_t p_full, ds_full;        // P, dS in TMEM; keys pass: and the next Q / dO landed
  uint64_t acc_done;               // a unit's accumulators are complete
  uint64_t unit_full[4];
  int unit[4];                     // the CTA's units in order, -1 behind the last
  uint32_t tmem_slot;
  int abort_flag;
};
static_assert(sizeof(Bars) <= kBarBytes, "barrier block");

// What every role of a pass knows.
struct Pass {
  const AttnBwdArgs* p;
  uint8_t* smem;
  Bars* bars;
  volatile int* abort_flag;
  uint32_t tmem;
  int n_tiles;   // tiles of a sequence
  int warp, lane;

  // Bounded, by a whole warp: one poll in the code, with a vote on its answer.
  __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int code) const {
    const uint32_t at = smem_u32(bar);
#pragma unroll 1
    for (uint32_t it = 0; it < kWaitPolls; ++it) {
      if (__all_sync(0xffffffffu, mbar_try_wait<false>(at, parity))) return true;
      if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
    }
    *abort_flag = 1;
    atomicCAS(p->err, 0, DEV_TIMEOUT_ATTN_BWD + code);
    return false;
  }
  // The CTA's k-th unit (-1: none); -2 when the CTA was aborted.  The producer is at most two units ahead
  // of the slowest role, so four slots need no release.
  __device__ __forceinline__ int unit(int k) const {
    if (!wait(&bars->unit_full[k & 3], (uint32_t)((k >> 2) & 1), 1)) return -2;
    return __shfl_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&bars->unit[k & 3]), 0);
  }
  __device__ __forceinline__ void publish(int k, int id) const {
    if (lane == 0) {
      bars->unit[k & 3] = id;
      mbar_arrive(&bars->unit_full[k & 3]);
    }
    __syncwarp();
  }
  __device__ __forceinline__ int units() const { return p->batch * p->n_heads * n_tiles; }
  // The next unit of either pass that no CTA has (they may be past the last).  The first gridDim.x units of the
  // keys pass, and those of the queries pass that CTAs without a keys unit begin with, follow from the CTA's index.
  __device__ __forceinline__ int draw_keys() const {
    int id = 0;
    if (lane == 0) id = (int)gridDim.x + atomicAdd(p->counters, 1);
    return __shfl_sync(0xffffffffu, id, 0);
  }
  __device__ __forceinline__ int draw_queries() const {
    const int fixed = (int)gridDim.x > units() ? (int)gridDim.x - units() : 0;
    int id = 0;
    if (lane == 0) id = fixed + atomicAdd(p->counters + 1, 1);
    return __shfl_sync(0xffffffffu, id, 0);
  }
  // queries pass: key tiles walked for batch element b
  __device__ __forceinline__ int walked(int b) const { return p->key_mask != nullptr ? p->n_listed[b] : n_tiles; }
  __device__ __forceinline__ int tile(int b, int n) const {
    return p->key_mask != nullptr ? p->tiles[(size_t)b * n_tiles + n] : n;
  }
};

// Clears the output rows of tile `own` (zeros of a unit without a valid key), by one warp.
__device__ __forceinline__ void zero_out(__nv_bfloat16* rows, size_t stride, int first, int seq, int lane) {
#pragma unroll 1
  for (int r = first + (lane >> 4); r < first + BT && r < seq; r += 2)
    *reinterpret_cast<uint4*>(rows + (size_t)r * stride + (lane & 15) * 8) = make_uint4(0, 0, 0, 0);
}

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

// A tile's descriptor by its low word (address and leading offset); the high word is the same for all.
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_lo(uint32_t start, uint32_t lbo) {
  return ((start & 0x3FFFFu) >> 4) | (lbo >> 4) << 16;
}
__device__ __forceinline__ uint64_t desc(uint32_t lo) { return (uint64_t)kDescHi << 32 | lo; }

// The three products, 8 MMAs each behind one election, by a warp whose index and TMEM base the compiler knows to
// be the same in all lanes (the broadcasts where the kernel begins).  (With the broadcasts and an election for
// every MMA the kernel is slowest: 611 us at 24 heads x 4130, 490 without either.)  The ring's stage is made uniform
// before the branch too: 455 instead of 457 us there, 1.5 % in bursts at 16418 rows.

// D = A B^T over d, both tiles row-major in shared memory.
__device__ __forceinline__ void scores_ss(uint32_t d, uint32_t a, uint32_t b) {
  a = __shfl_sync(0xffffffffu, a, 0);
  b = __shfl_sync(0xffffffffu, b, 0);
  if (elect_one()) {
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      const uint32_t off = ((uint32_t)(kk >> 2) * HALF_BYTES + (uint32_t)(kk & 3) * 32u) >> 4;
      tc_mma_ss(d, desc(a + off), desc(b + off), kIdescScores, kk > 0 ? 1u : 0u);
    }
  }
  __syncwarp();
}

// The same with A in TMEM.
__device__ __forceinline__ void scores_ts(uint32_t d, uint32_t a, uint32_t b) {
  b = __shfl_sync(0xffffffffu, b, 0);
  if (elect_one()) {
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      const uint32_t off = ((uint32_t)(kk >> 2) * HALF_BYTES + (uint32_t)(kk & 3) * 32u) >> 4;
      tc_mma_ts(d, a + (uint32_t)kk * 8u, desc(b + off), kIdescScores, kk > 0 ? 1u : 0u);
    }
  }
  __syncwarp();
}

// D (+)= A B over the 128 streamed rows, A (P or dS) in TMEM: the two warpgroups' halves `half_cols` columns
// apart, B read along its rows.
__device__ __forceinline__ void sum_ts(uint32_t d, uint32_t a, uint32_t half_cols, uint32_t b, bool first) {
  b = __shfl_sync(0xffffffffu, b, 0);
  if (elect_one()) {
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
      tc_mma_ts(d, a + (uint32_t)(kk >> 2) * half_cols + (uint32_t)(kk & 3) * 8u, desc(b + (uint32_t)kk * (2048u >> 4)),
                kIdescSum, (!first || kk > 0) ? 1u : 0u);
  }
  __syncwarp();
}

// 64 accumulator columns of a warp's 32 rows, scaled, as bf16 into its 4 KB of the staging tile
// (128-byte rows, 16-byte pieces swizzled by the row as the TMA expects).
__device__ __forceinline__ void stage64(uint8_t* out, uint32_t src, float f, int lane) {
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    uint32_t x[32];
    tmem_ld32(src + c * 32, x);
    tmem_ld_wait();
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = pack_bf16x2(__uint_as_float(x[v * 8 + 2 * e]) * f, __uint_as_float(x[v * 8 + 2 * e + 1]) * f);
      *reinterpret_cast<uint4*>(out + lane * 128 + (((c * 4 + v) ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  fence_proxy_async_smem();
  __syncwarp();
}

__device__ __forceinline__ f32x2_t pair_of(const uint32_t* x) { return f2_pack(__uint_as_float(x[0]), __uint_as_float(x[1])); }

// ------------------------------------------------------------------------------------ keys pass
// A unit: K and V of 128 keys stay; Q and dO of all query tiles are walked.  The producer returns the CTA's
// first unit of the queries pass, drawn when the last of this one is known.
__device__ __forceinline__ int keys_producer(const Pass& c, const CUtensorMap& tmQ, const CUtensorMap& tmK,
                                             const CUtensorMap& tmV, const CUtensorMap& tmDO) {
  const AttnBwdArgs& p = *c.p;
  Bars* bars = c.bars;
  const int n_units = c.units();
  // the next unit that has a valid key
  auto settle = [&](int id) {
#pragma unroll 1
    while (id < n_units) {
      if (p.key_mask == nullptr) return id;
      const int own = id % c.n_tiles, bh = id / c.n_tiles, b = bh / p.n_heads;
      bool any = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = own * BT + i * 32 + c.lane;
        any |= key < p.seq && p.key_mask[(size_t)b * p.seq + (key < p.seq ? key : 0)] != 0;
      }
      if (__any_sync(0xffffffffu, any)) return id;
      zero_out(p.dkp + (size_t)bh * p.seq * kHeadDim, kHeadDim, own * BT, p.seq, c.lane);
      zero_out(p.dv + (size_t)b * p.seq * 3 * p.n_heads * kHeadDim + (size_t)(bh % p.n_heads) * kHeadDim,
               (size_t)3 * p.n_heads * kHeadDim, own * BT, p.seq, c.lane);
      id = c.draw_keys();
    }
    return -1;
  };
  Ring<kRingQ> x;
  Ring<kRingDO> y;
  int nx = 0, ny = 0, nown_x = 0, nown_y = 0;
  bool ok = true;
  int id = settle((int)blockIdx.x);
  c.publish(0, id);
  int query = id < 0 ? c.draw_queries() : -1;
#pragma unroll 1
  for (int k = 0; ok && id >= 0; ++k) {
    const int own = id % c.n_tiles, bh = id / c.n_tiles;
    const int b = bh / p.n_heads, h = bh % p.n_heads;
    const float* nl = p.nlse2 + (size_t)bh * p.seq_pad;
    const float* nd = p.ndelta + (size_t)bh * p.seq_pad;
    int next_id = -1;
    if (k > 0 && !c.wait(&bars->own_x_empty, (uint32_t)((k - 1) & 1), 2)) break;
    if (c.lane == 0) {
      mbar_arrive_expect_tx(&bars->own_x, TILE_BYTES);
      tma_load_3d(c.smem, &tmK, &bars->own_x, 0, own * BT, bh);
      tma_load_3d(c.smem + HALF_BYTES, &tmK, &bars->own_x, 64, own * BT, bh);
    }
    ++nown_x;
#pragma unroll 1
    for (int t = 0; t < c.n_tiles; ++t) {
      if (nx >= kRingQ && !c.wait(&bars->x_empty[x.st], x.ph ^ 1u, 2)) {
        ok = false;
        break;
      }
      if (c.lane == 0) {
        uint8_t* dq = c.smem + OFF_Q + x.st * TILE_BYTES;
        mbar_arrive_expect_tx(&bars->x_full[x.st], TILE_BYTES);
        tma_load_3d(dq, &tmQ, &bars->x_full[x.st], 0, t * BT, bh);
        tma_load_3d(dq + HALF_BYTES, &tmQ, &bars->x_full[x.st], 64, t * BT, bh);
      }
      ++nx;
      x.next();
      if (t == 0) {
        if (k > 0 && !c.wait(&bars->own_y_empty, (uint32_t)((k - 1) & 1), 2)) {
          ok = false;
          break;
        }
        if (c.lane == 0) {
          mbar_arrive_expect_tx(&bars->own_y, TILE_BYTES);
          tma_load_4d(c.smem + TILE_BYTES, &tmV, &bars->own_y, 0, h, own * BT, b);
          tma_load_4d(c.smem + TILE_BYTES + HALF_BYTES, &tmV, &bars->own_y, 64, h, own * BT, b);
        }
        ++nown_y;
      }
      if (ny >= kRingDO && !c.wait(&bars->y_empty[y.st], y.ph ^ 1u, 2)) {
        ok = false;
        break;
      }
      if (c.lane == 0) {
        uint8_t* dd = c.smem + OFF_DO + y.st * TILE_BYTES;
        float* stat = reinterpret_cast<float*>(c.smem + OFF_STAT + y.st * STAT_BYTES);
        mbar_arrive_expect_tx(&bars->y_full[y.st], TILE_BYTES + STAT_BYTES);
        bulk_load(stat, nl + t * BT, BT * 4, &bars->y_full[y.st]);
        bulk_load(stat + BT, nd + t * BT, BT * 4, &bars->y_full[y.st]);
        tma_load_4d(dd, &tmDO, &bars->y_full[y.st], 0, h, t * BT, b);
        tma_load_4d(dd + HALF_BYTES, &tmDO, &bars->y_full[y.st], 64, h, t * BT, b);
      }
      ++ny;
      y.next();
      if (t == (c.n_tiles > 1 ? 1 : 0)) {  // the next unit, before anyone asks for it
        next_id = settle(c.draw_keys());
        c.publish(k + 1, next_id);
        if (next_id < 0) query = c.draw_queries();
      }
    }
    id = next_id;
  }
  // drain the copies still in flight (the last use of each barrier phase)
  if (nown_x > 0) mbar_wait_drain(&bars->own_x, (uint32_t)((nown_x - 1) & 1), p.err, DEV_TIMEOUT_ATTN_BWD + 3);
  if (nown_y > 0) mbar_wait_drain(&bars->own_y, (uint32_t)((nown_y - 1) & 1), p.err, DEV_TIMEOUT_ATTN_BWD + 3);
#pragma unroll 1
  for (int j = nx - kRingQ < 0 ? 0 : nx - kRingQ; j < nx; ++j)
    mbar_wait_drain(&bars->x_full[j % kRingQ], (uint32_t)((j / kRingQ) & 1), p.err, DEV_TIMEOUT_ATTN_BWD + 3);
#pragma unroll 1
  for (int j = ny - kRingDO < 0 ? 0 : ny - kRingDO; j < ny; ++j)
    mbar_wait_drain(&bars->y_full[j % kRingDO], (uint32_t)((j / kRingDO) & 1), p.err, DEV_TIMEOUT_ATTN_BWD + 3);
  return query < 0 ? n_units : query;  // (an aborted CTA has none left)
}

__device__ __forceinline__ void keys_mma(const Pass& c) {
  Bars* bars = c.bars;
  const uint32_t tmem = c.tmem;
  const uint32_t sm = smem_u32(c.smem);
  const uint32_t k_d = desc_lo(sm, 16), v_d = desc_lo(sm + TILE_BYTES, 16);
  const uint32_t q_k = desc_lo(sm + OFF_Q, 16), do_k = desc_lo(sm + OFF_DO, 16);
  const uint32_t q_mn = desc_lo(sm + OFF_Q, HALF_BYTES), do_mn = desc_lo(sm + OFF_DO, HALF_BYTES);
  const int last = c.n_tiles - 1;
  int id = c.unit(0);
  bool ok = id >= 0;
  if (ok) {
    ok = c.wait(&bars->own_x, 0, 4) && c.wait(&bars->x_full[0], 0, 4);
    if (ok) {
      tc_fence_after();
      scores_ss(tmem + TM_S, k_d, q_k);
      tc_commit_warp(&bars->s_full);
      if (last == 0) tc_commit_warp(&bars->own_x_empty);
      ok = c.wait(&bars->own_y, 0, 4) && c.wait(&bars->y_full[0], 0, 4);
    }
    if (ok) {
      tc_fence_after();
      scores_ss(tmem + TM_DP, v_d, do_k);
      tc_commit_warp(&bars->dp_full);
      if (last == 0) tc_commit_warp(&bars->own_y_empty);
    }
  }
  uint32_t g = 0;  // tiles so far, over all units: phases, and the dO stage
  uint32_t qs = 0;  // Q stage
  for (int k = 0; ok && id >= 0; ++k) {
    for (int n = 0; n <= last; ++n, ++g) {
      if (n == last) {
        id = c.unit(k + 1);
        if (id == -2) {
          ok = false;
          break;
        }
      }
      const bool more = id >= 0;                                  // a tile follows
      const bool next_last = n == last ? last == 0 : n + 1 == last;  // and is the last of its unit
      const uint32_t st = g & 1u, ph = g & 1u;
      const uint32_t qn = qs + 1 == kRingQ ? 0 : qs + 1;
      // P of this tile, and Q of the next (and its K, for a new unit) landed; P of a unit's first tile is
      // released when the accumulators of the unit before have been read
      if (!c.wait(&bars->p_full, ph, 5)) {
        ok = false;
        break;
      }
      tc_fence_after();
      sum_ts(tmem + TM_DV, tmem + TM_S, 64, do_mn + st * kTile16, n == 0);
      if (more) {
        scores_ss(tmem + TM_S, k_d, q_k + qn * kTile16);
        tc_commit_warp(&bars->s_full);
        if (next_last) tc_commit_warp(&bars->own_x_empty);
      }
      if (!c.wait(&bars->ds_full, ph, 6)) {
        ok = false;
        break;
      }
      tc_fence_after();
      sum_ts(tmem + TM_DK, tmem + TM_DP, 64, q_mn + qs * kTile16, n == 0);
      tc_commit_warp(&bars->x_empty[qs]);
      tc_commit_warp(&bars->y_empty[st]);
      if (n == last) tc_commit_warp(&bars->acc_done);
      if (more) {
        scores_ss(tmem + TM_DP, v_d, do_k + (st ^ 1u) * kTile16);
        tc_commit_warp(&bars->dp_full);
        if (next_last) tc_commit_warp(&bars->own_y_empty);
      }
      qs = qn;
    }
  }
}

__device__ __forceinline__ void keys_proxy(const Pass& c) {
  Bars* bars = c.bars;
  int id = c.unit(0);
  bool ok = true;
  uint32_t g = 0;
  Ring<kRingQ> x;
  for (int k = 0; ok && id >= 0; ++k) {
    for (int n = 0; n < c.n_tiles; ++n, ++g) {
      x.next();
      const bool turn = n + 1 == c.n_tiles;  // the next tile is a new unit's
      if (turn) {
        id = c.unit(k + 1);
        if (id == -2) {
          ok = false;
          break;
        }
      }
      const bool more = id >= 0;
      const uint32_t st = (g + 1) & 1u, ph = ((g + 1) >> 1) & 1u;
      // each arrival belongs to the barrier's phase g: phase g - 1 must be complete first
      const uint32_t prev = (g - 1) & 1u;
      if ((g > 0 && !c.wait(&bars->p_full, prev, 7)) || (more && turn && !c.wait(&bars->own_x, (uint32_t)((k + 1) & 1), 7)) ||
          (more && !c.wait(&bars->x_full[x.st], x.ph, 7))) {
        ok = false;
        break;
      }
      __syncwarp();
      if (c.lane == 0) mbar_arrive(&bars->p_full);
      if ((g > 0 && !c.wait(&bars->ds_full, prev, 8)) || (more && turn && !c.wait(&bars->own_y, (uint32_t)((k + 1) & 1), 8)) ||
          (more && !c.wait(&bars->y_full[st], ph, 8))) {
        ok = false;
        break;
      }
      __syncwarp();
      if (c.lane == 0) mbar_arrive(&bars->ds_full);
    }
  }
}

// `wide`: dst is aligned to 32 bytes, else to 16.
__device__ __forceinline__ void store_32_bytes(void* dst, const uint32_t* w, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Warpgroup 0 stores dV, warpgroup 1 dK, 32 columns at a time.  A lane's row is a line of its own, and a store
// costs a request per line: 16 bytes per lane took 7300 cycles of a unit, 32 bytes 3750.  So two lanes
// exchange their pieces first and store 64 bytes of one row, then of the other (2600 cycles).
__device__ __forceinline__ void keys_store(const Pass& c, int id, int half, uint32_t src, float f) {
  const AttnBwdArgs& p = *c.p;
  const int row = (id % c.n_tiles) * BT + (c.warp & 3) * 32 + c.lane, bh = id / c.n_tiles;
  const size_t stride = half == 0 ? (size_t)3 * p.n_heads * kHeadDim : kHeadDim;
  __nv_bfloat16* base = half == 0 ? p.dv + (size_t)(bh / p.n_heads) * p.seq * stride + (size_t)(bh % p.n_heads) * kHeadDim
                                  : p.dkp + (size_t)bh * p.seq * kHeadDim;
  const bool odd = c.lane & 1, wide = (reinterpret_cast<uintptr_t>(base) & 31) == 0;
  const int even_row = row & ~1;
  __nv_bfloat16* even = base + (size_t)even_row * stride + (odd ? 16 : 0);
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    uint32_t x[32], a[8], b[8];
    tmem_ld32(src + i * 32, x);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t lo = pack_bf16x2(__uint_as_float(x[2 * e]) * f, __uint_as_float(x[2 * e + 1]) * f);
      const uint32_t hi = pack_bf16x2(__uint_as_float(x[16 + 2 * e]) * f, __uint_as_float(x[16 + 2 * e + 1]) * f);
      const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? lo : hi, 1);
      a[e] = odd ? got : lo;
      b[e] = odd ? hi : got;
    }
    if (even_row < p.seq) store_32_bytes(even + 32 * i, a, wide);
    if (even_row + 1 < p.seq) store_32_bytes(even + stride + 32 * i, b, wide);
  }
}

// Ends at the barrier between the passes.
__device__ __forceinline__ void keys_compute(const Pass& c) {
  const AttnBwdArgs& p = *c.p;
  Bars* bars = c.bars;
  const int half = (c.warp - 4) >> 2;          // query half of this warpgroup
  const int r = (c.warp & 3) * 32 + c.lane;    // TMEM lane: key of the tile
  const uint32_t t_row = c.tmem + ((uint32_t)((c.warp & 3) * 32) << 16);
  const uint32_t t_s = t_row + TM_S + (uint32_t)half * 64u, t_dp = t_row + TM_DP + (uint32_t)half * 64u;
  const uint32_t t_acc = t_row + (half == 0 ? TM_DV : TM_DK);
  const float f_acc = half == 0 ? 1.0f : p.scale;
  const f32x2_t sl2x2 = f2_pack(p.scale_log2, p.scale_log2);
  int before = -1;                             // the unit whose accumulators are still to be read
  bool ok = true;
  uint32_t g = 0;
  for (int k = 0; ok; ++k) {
    const int id = c.unit(k);
    if (id < 0) {
      ok = id != -2;
      break;
    }
    const int row = (id % c.n_tiles) * BT + r;
    // (read here, looked at when the first scores are there)
    uint32_t row_mask = row < p.seq;
    if (row < p.seq && p.key_mask != nullptr) row_mask = p.key_mask[(size_t)(id / c.n_tiles / p.n_heads) * p.seq + row];
    bool row_ok = true, rows_ok = true;
    for (int n = 0; n < c.n_tiles; ++n, ++g) {
      const uint32_t st = g & 1u, ph = g & 1u;
      // the statistics land with dO, well before the scores are there
      if (!c.wait(&bars->y_full[st], (g >> 1) & 1u, 9)) {
        ok = false;
        break;
      }
      const float4* stat = reinterpret_cast<const float4*>(c.smem + OFF_STAT + st * STAT_BYTES) + half * 16;
      float4 nl[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) nl[i] = stat[i];
      if (!c.wait(&bars->s_full, ph, 10)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t pr[64], pk[32];
      tmem_ld32(t_s, pr);
      tmem_ld32(t_s + 32, pr + 32);
      if (n == 0) {
        row_ok = row_mask != 0;
        rows_ok = __all_sync(0xffffffffu, row_ok) != 0;
      }
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float z[4];
        f2_unpack(f2_fma(pair_of(pr + 4 * i), sl2x2, f2_pack(nl[i].x, nl[i].y)), z[0], z[1]);
        f2_unpack(f2_fma(pair_of(pr + 4 * i + 2), sl2x2, f2_pack(nl[i].z, nl[i].w)), z[2], z[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) pr[4 * i + e] = __float_as_uint(ex2_approx(z[e]));
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) pk[i] = pack_bf16x2(__uint_as_float(pr[2 * i]), __uint_as_float(pr[2 * i + 1]));
      if (!rows_ok) {  // a masked key's scores may be anything
#pragma unroll
        for (int i = 0; i < 32; ++i) pk[i] = row_ok ? pk[i] : 0u;
      }
      tmem_st32(t_s, pk);
      tmem_st_wait();
      if (n == 0 && before >= 0) {
        if (!c.wait(&bars->acc_done, (uint32_t)((k - 1) & 1), 11)) {
          ok = false;
          break;
        }
        tc_fence_after();
        keys_store(c, before, half, t_acc, f_acc);
      }
      tc_fence_before();
      __syncwarp();
      if (c.lane == 0) mbar_arrive(&bars->p_full);
      float4 nd[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) nd[i] = stat[32 + i];
      if (!c.wait(&bars->dp_full, ph, 12)) {
        ok = false;
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t dp[32];
        tmem_ld32(t_dp + 32 * j, dp);
        if (j == 1) {
#pragma unroll
          for (int i = 0; i < 8; ++i) nd[i] = stat[40 + i];
        }
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float z[4];
          f2_unpack(f2_mul(f2_add(pair_of(dp + 4 * i), f2_pack(nd[i].x, nd[i].y)), pair_of(pr + 32 * j + 4 * i)), z[0], z[1]);
          f2_unpack(f2_mul(f2_add(pair_of(dp + 4 * i + 2), f2_pack(nd[i].z, nd[i].w)), pair_of(pr + 32 * j + 4 * i + 2)), z[2],
                    z[3]);
          pk[16 * j + 2 * i] = pack_bf16x2(z[0], z[1]);
          pk[16 * j + 2 * i + 1] = pack_bf16x2(z[2], z[3]);
        }
      }
      if (!rows_ok) {
#pragma unroll
        for (int i = 0; i < 32; ++i) pk[i] = row_ok ? pk[i] : 0u;
      }
      tmem_st32(t_dp, pk);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (c.lane == 0) mbar_arrive(&bars->ds_full);
    }
    before = id;
    if (!ok) break;
    // the last unit's accumulators (any other's are read behind the next unit's first scores)
    const int next_id = c.unit(k + 1);
    if (next_id < 0) {
      const bool done = next_id == -1 && c.wait(&bars->acc_done, (uint32_t)(k & 1), 13);
      if (done) {
        tc_fence_after();
        keys_store(c, id, half, t_acc, f_acc);
      }
      tc_fence_before();
      __syncthreads();
      return;
    }
  }
  tc_fence_before();
  __syncthreads();
}

// ------------------------------------------------------------------------------------ queries pass
// A unit: Q (in TMEM) and dO of 128 queries stay; K and V of the key tiles with a valid key are walked.
__device__ __forceinline__ void queries_producer(const Pass& c, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                                 const CUtensorMap& tmDO, int first) {
  const AttnBwdArgs& p = *c.p;
  Bars* bars = c.bars;
  const int n_units = c.units();
  auto settle = [&](int id) {
#pragma unroll 1
    while (id < n_units) {
      const int own = id % c.n_tiles, bh = id / c.n_tiles;
      if (c.walked(bh / p.n_heads) > 0) return id;
      zero_out(p.dqp + (size_t)bh * p.seq * kHeadDim, kHeadDim, own * BT, p.seq, c.lane);
      id = c.draw_queries();
    }
    return -1;
  };
  Ring<kRingK> x;
  Ring<kRingV> y;
  int nx = 0, ny = 0, nown = 0;
  bool ok = true;
  int id = settle(first);
  c.publish(0, id);
#pragma unroll 1
  for (int k = 0; ok && id >= 0; ++k) {
    const int own = id % c.n_tiles, bh = id / c.n_tiles;
    const int b = bh / p.n_heads, h = bh % p.n_heads;
    const int count = c.walked(b);
    int next_id = -1;
    int t1 = c.tile(b, 0);
#pragma unroll 1
    for (int n = 0; n < count; ++n) {
      const int t = t1;
      if (n + 1 < count) t1 = c.tile(b, n + 1);
      if (nx >= kRingK && !c.wait(&bars->x_empty[x.st], x.ph ^ 1u, 2)) {
        ok = false;
        break;
      }
      if (c.lane == 0) {
        uint8_t* dk = c.smem + OFF_K + x.st * TILE_BYTES;
        mbar_arrive_expect_tx(&bars->x_full[x.st], TILE_BYTES);
        tma_load_3d(dk, &tmK, &bars->x_full[x.st], 0, t * BT, bh);
        tma_load_3d(dk + HALF_BYTES, &tmK, &bars->x_full[x.st], 64, t * BT, bh);
      }
      ++nx;
      x.next();
      if (n == 0) {
        if (k > 0 && !c.wait(&bars->own_y_empty, (uint32_t)((k - 1) & 1), 2)) {
          ok = false;
          break;
        }
        if (c.lane == 0) {
          mbar_arrive_expect_tx(&bars->own_y, TILE_BYTES);
          tma_load_4d(c.smem, &tmDO, &bars->own_y, 0, h, own * BT, b);
          tma_load_4d(c.smem + HALF_BYTES, &tmDO, &bars->own_y, 64, h, own * BT, b);
        }
        ++nown;
      }
      if (ny >= kRingV && !c.wait(&bars->y_empty[y.st], y.ph ^ 1u, 2)) {
        ok = false;
        break;
      }
      if (c.lane == 0) {
        uint8_t* dv = c.smem + OFF_V + y.st * TILE_BYTES;
        mbar_arrive_expect_tx(&bars->y_full[y.st], TILE_BYTES);
        tma_load_4d(dv, &tmV, &bars->y_full[y.st], 0, h, t * BT, b);
        tma_load_4d(dv + HALF_BYTES, &tmV, &bars->y_full[y.st], 64, h, t * BT, b);
      }
      ++ny;
      y.next();
      if (n == (count > 1 ? 1 : 0)) {
        next_id = settle(c.draw_queries());
        c.publish(k + 1, next_id);
      }
    }
    id = next_id;
  }
  if (nown > 0) mbar_wait_drain(&bars->own_y, (uint32_t)((nown - 1) & 1), p.err, DEV_TIMEOUT_ATTN_BWD + 3);
#pragma unroll 1
  for (int j = nx - kRingK < 0 ? 0 : nx - kRingK; j < nx; ++j)
    mbar_wait_drain(&bars->x_full[j % kRingK], (uint32_t)((j / kRingK) & 1), p.err, DEV_TIMEOUT_ATTN_BWD + 3);
#pragma unroll 1
  for (int j = ny - kRingV < 0 ? 0 : ny - kRingV; j < ny; ++j)
    mbar_wait_drain(&bars->y_full[j % kRingV], (uint32_t)((j / kRingV) & 1), p.err, DEV_TIMEOUT_ATTN_BWD + 3);
}

__device__ __forceinline__ void queries_mma(const Pass& c) {
  Bars* bars = c.bars;
  const uint32_t tmem = c.tmem;
  const uint32_t sm = smem_u32(c.smem);
  const uint32_t do_d = desc_lo(sm, 16);
  const uint32_t k_k = desc_lo(sm + OFF_K, 16), v_k = desc_lo(sm + OFF_V, 16);
  const uint32_t k_mn = desc_lo(sm + OFF_K, HALF_BYTES);
  int id = c.unit(0);
  bool ok = id >= 0;
  int count = ok ? c.walked(id / c.n_tiles / c.p->n_heads) : 0;
  if (ok) {
    ok = c.wait(&bars->own_x, 0, 4) && c.wait(&bars->first, 0, 4);
    if (ok) {
      tc_fence_after();
      scores_ts(tmem + TM_S, tmem + TM_Q, k_k);
      tc_commit_warp(&bars->s_full);
      ok = c.wait(&bars->own_y, 0, 4) && c.wait(&bars->y_full[0], 0, 4);
    }
    if (ok) {
      tc_fence_after();
      scores_ss(tmem + TM_DP, do_d, v_k);
      tc_commit_warp(&bars->dp_full);
      tc_commit_warp(&bars->y_empty[0]);
      if (count == 1) tc_commit_warp(&bars->own_y_empty);
    }
  }
  uint32_t g = 0;
  int st = 0;
  for (int k = 0; ok && id >= 0; ++k) {
    const int here = count;
    for (int n = 0; n < here; ++n, ++g) {
      if (n + 1 == here) {
        id = c.unit(k + 1);
        if (id == -2) {
          ok = false;
          break;
        }
        if (id >= 0) count = c.walked(id / c.n_tiles / c.p->n_heads);
      }
      const bool next_last = n + 1 == here ? count == 1 : n + 2 == here;
      const int sn = st + 1 == kRingK ? 0 : st + 1;
      const uint32_t ph = g & 1u, vn = (g + 1) & 1u;
      if (id >= 0) {
        // the scores are in registers and K of the next tile has landed, clean (and its Q is in TMEM)
        if (!c.wait(&bars->s_read, ph, 5)) {
          ok = false;
          break;
        }
        tc_fence_after();
        scores_ts(tmem + TM_S, tmem + TM_Q, k_k + (uint32_t)sn * kTile16);
        tc_commit_warp(&bars->s_full);
        if (!c.wait(&bars->dp_read, ph, 5)) {  // and V (and dO)
          ok = false;
          break;
        }
        tc_fence_after();
        scores_ss(tmem + TM_DP, do_d, v_k + vn * kTile16);
        tc_commit_warp(&bars->dp_full);
        tc_commit_warp(&bars->y_empty[vn]);
        if (next_last) tc_commit_warp(&bars->own_y_empty);
      }
      // dS of a unit's first tile is released when dQ of the unit before has been read
      if (!c.wait(&bars->ds_full, ph, 6)) {
        ok = false;
        break;
      }
      tc_fence_after();
      sum_ts(tmem + TM_DQ, tmem + TM_DS, 32, k_mn + (uint32_t)st * kTile16, n == 0);
      tc_commit_warp(&bars->x_empty[st]);
      if (n + 1 == here) tc_commit_warp(&bars->acc_done);
      st = sn;
    }
  }
}

__device__ __forceinline__ void queries_proxy(const Pass& c) {
  const AttnBwdArgs& p = *c.p;
  Bars* bars = c.bars;
  Ring<kRingK> x;
  Ring<kRingV> y;
  uint32_t g = 0;
  bool ok = true;
  for (int k = 0; ok; ++k) {
    const int id = c.unit(k);
    if (id < 0) break;
    const int b = id / c.n_tiles / p.n_heads;
    const int count = c.walked(b);
    const uint8_t* mask = p.key_mask != nullptr ? p.key_mask + (size_t)b * p.seq : nullptr;
    // with a mask: which of this lane's keys of the next tile are masked, read a tile ahead
    bool off[4] = {false, false, false, false};
    auto read_mask = [&](int t) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int kc = t * BT + w * 32 + c.lane;
        off[w] = kc < p.seq && mask[kc < p.seq ? kc : 0] == 0;
      }
    };
    int t_ahead = 0;
    if (mask != nullptr) {
      read_mask(c.tile(b, 0));
      if (count > 1) t_ahead = c.tile(b, 1);
    }
    for (int n = 0; n < count; ++n, ++g, x.next(), y.next()) {
      // K of tile g, clean: an arrival of phase g - 1 of s_read (phase g - 2 complete)
      uint32_t bad[4] = {0, 0, 0, 0};
      if (mask != nullptr) {
#pragma unroll
        for (int w = 0; w < 4; ++w) bad[w] = __ballot_sync(0xffffffffu, off[w]);
        if (n + 1 < count) read_mask(t_ahead);
        if (n + 2 < count) t_ahead = c.tile(b, n + 2);
      }
      if ((g > 1 && !c.wait(&bars->s_read, g & 1u, 7)) || !c.wait(&bars->x_full[x.st], x.ph, 7)) {
        ok = false;
        break;
      }
      zero_rows(c.smem + OFF_K + x.st * TILE_BYTES, bad, c.lane);
      __syncwarp();
      if (c.lane == 0) mbar_arrive(g == 0 ? &bars->first : &bars->s_read);
      if (g == 0) continue;
      // V of tile g (and dO, for a new unit)
      if ((g > 1 && !c.wait(&bars->dp_read, g & 1u, 8)) || (n == 0 && !c.wait(&bars->own_y, (uint32_t)(k & 1), 8)) ||
          !c.wait(&bars->y_full[y.st], y.ph, 8)) {
        ok = false;
        break;
      }
      __syncwarp();
      if (c.lane == 0) mbar_arrive(&bars->dp_read);
    }
  }
}

// Each warpgroup stores its half of the columns of dQ.
__device__ __forceinline__ void queries_store(const Pass& c, const CUtensorMap& tmDQ, int id, int half, uint32_t t_row) {
  const AttnBwdArgs& p = *c.p;
  const int row = (id % c.n_tiles) * BT + (c.warp & 3) * 32;
  uint8_t* out = c.smem + OFF_OUT + (c.warp - 4) * 4096;
  if (c.lane == 0) bulk_wait_read();
  __syncwarp();
  stage64(out, t_row + TM_DQ + (uint32_t)half * 64u, p.scale, c.lane);
  if (c.lane == 0 && row < p.seq) {
    tma_store_3d(&tmDQ, out, half * 64, row, id / c.n_tiles);
    bulk_commit();
  }
}

__device__ __forceinline__ void queries_compute(const Pass& c, const CUtensorMap& tmDQ) {
  const AttnBwdArgs& p = *c.p;
  Bars* bars = c.bars;
  const int half = (c.warp - 4) >> 2;          // key half of this warpgroup
  const int r = (c.warp & 3) * 32 + c.lane;    // TMEM lane: query of the tile
  const uint32_t t_row = c.tmem + ((uint32_t)((c.warp & 3) * 32) << 16);
  const uint32_t t_s = t_row + TM_S + (uint32_t)half * 64u, t_dp = t_row + TM_DP + (uint32_t)half * 64u;
  const uint32_t t_ds = t_row + TM_DS + (uint32_t)half * 32u, t_q = t_row + TM_Q + (uint32_t)half * 32u;
  const f32x2_t sl2x2 = f2_pack(p.scale_log2, p.scale_log2);
  // a unit's row: its half of Q goes to TMEM (element d in column d / 2, as in memory)
  uint32_t q[32];
  float nl = 0.0f, nd = 0.0f;
  auto read_row = [&](int id) {
    const int row = (id % c.n_tiles) * BT + r, bh = id / c.n_tiles;
    const uint4* src = reinterpret_cast<const uint4*>(p.qp + ((size_t)bh * p.seq + (row < p.seq ? row : 0)) * kHeadDim + half * 64);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 v = row < p.seq ? src[i] : make_uint4(0, 0, 0, 0);
      q[4 * i] = v.x;
      q[4 * i + 1] = v.y;
      q[4 * i + 2] = v.z;
      q[4 * i + 3] = v.w;
    }
  };
  auto read_stats = [&](int id) {
    const size_t at = (size_t)(id / c.n_tiles) * p.seq_pad + (id % c.n_tiles) * BT + r;
    nl = p.nlse2[at];
    nd = p.ndelta[at];
  };
  bool ok = true;
  uint32_t g = 0;
  Ring<kRingK> last;  // stage and phase of the tile before
  int before = -1;
  int id = c.unit(0);
  if (id >= 0) {
    read_row(id);
    read_stats(id);
    tmem_st32(t_q, q);
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (c.lane == 0) mbar_arrive(&bars->own_x);
  }
  for (int k = 0; ok && id >= 0; ++k) {
    const int b = id / c.n_tiles / p.n_heads;
    const int count = c.walked(b);
    const uint8_t* mask = p.key_mask != nullptr ? p.key_mask + (size_t)b * p.seq : nullptr;
    const f32x2_t nl2 = f2_pack(nl, nl), nd2 = f2_pack(nd, nd);
    int next_id = -1;
    // may this lane's two keys of the tile be attended to (read a tile ahead)
    bool key[2];
    auto read_mask = [&](int t) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int kc = t * BT + half * 64 + w * 32 + c.lane;
        key[w] = kc < p.seq && (mask == nullptr || mask[kc < p.seq ? kc : 0] != 0);
      }
    };
    read_mask(c.tile(b, 0));
    int t_ahead = count > 1 ? c.tile(b, 1) : 0;
    for (int n = 0; n < count; ++n, ++g) {
      const uint32_t ph = g & 1u;
      const bool turn = n + 1 == count;  // the next tile is a new unit's
      const uint32_t valid[2] = {__ballot_sync(0xffffffffu, key[0]), __ballot_sync(0xffffffffu, key[1])};
      if (turn) {
        next_id = c.unit(k + 1);
        if (next_id >= 0) read_row(next_id);
        ok = next_id != -2;
      } else {
        read_mask(t_ahead);
        if (n + 2 < count) t_ahead = c.tile(b, n + 2);
      }
      if (!ok || !c.wait(&bars->s_full, ph, 10)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (turn && next_id >= 0) tmem_st32(t_q, q);  // the scores of this unit's last tile are done with Q
      uint32_t pr[64], dp[64], pk[32];
      tmem_ld32(t_s, pr);
      tmem_ld32(t_s + 32, pr + 32);
      tmem_ld_wait();
      if (turn) tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (c.lane == 0) mbar_arrive(&bars->s_read);
      if (!c.wait(&bars->dp_full, ph, 12)) {
        ok = false;
        break;
      }
      tc_fence_after();
      tmem_ld32(t_dp, dp);  // (on their way while the exponentials are taken: 205 us instead of 211 of this pass)
      tmem_ld32(t_dp + 32, dp + 32);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        float z0, z1;
        f2_unpack(f2_fma(pair_of(pr + 2 * i), sl2x2, nl2), z0, z1);
        pr[2 * i] = __float_as_uint(ex2_approx(z0));
        pr[2 * i + 1] = __float_as_uint(ex2_approx(z1));
      }
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (c.lane == 0) mbar_arrive(&bars->dp_read);
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
      if (g > 0) {
        if (!c.wait(&bars->x_empty[last.st], last.ph, 9)) {
          ok = false;
          break;
        }
        last.next();
        tc_fence_after();
      }
      tmem_st32(t_ds, pk);
      tmem_st_wait();
      if (n == 0 && before >= 0) {
        if (!c.wait(&bars->acc_done, (uint32_t)((k - 1) & 1), 11)) {
          ok = false;
          break;
        }
        tc_fence_after();
        queries_store(c, tmDQ, before, half, t_row);
      }
      tc_fence_before();
      __syncwarp();
      if (c.lane == 0) mbar_arrive(&bars->ds_full);
    }
    if (!ok) break;
    before = id;
    if (next_id < 0) {
      if (c.wait(&bars->acc_done, (uint32_t)(k & 1), 13)) {
        tc_fence_after();
        queries_store(c, tmDQ, id, half, t_row);
      }
      break;
    }
    id = next_id;
    read_stats(id);
  }
  tc_fence_before();
}

__device__ __forceinline__ void init_bars(Bars* bars, bool keys) {
  mbar_init(&bars->own_x, keys ? 1 : 8);
  mbar_init(&bars->own_y, 1);
  mbar_init(&bars->own_x_empty, 1);
  mbar_init(&bars->own_y_empty, 1);
  for (int i = 0; i < 3; ++i) {
    mbar_init(&bars->x_full[i], 1);
    mbar_init(&bars->x_empty[i], 1);
  }
  for (int i = 0; i < 2; ++i) {
    mbar_init(&bars->y_full[i], 1);
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
  for (int i = 0; i < 4; ++i) mbar_init(&bars->unit_full[i], 1);
}

__global__ void __launch_bounds__(kThreads, 1)
    attn_bwd_kernel(const __grid_constant__ AttnBwdMaps m, const __grid_constant__ AttnBwdArgs p) {
  // The swizzled tiles need a base at a multiple of 1024 bytes, which the window of dynamic shared memory
  // of a kernel without static shared memory has (checked: a launch elsewhere would report, not compute).
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicCAS(p.err, 0, DEV_TIMEOUT_ATTN_BWD);
    return;
  }
  Bars* bars = reinterpret_cast<Bars*>(smem + OFF_BAR);            // keys pass
  Bars* bars_q = reinterpret_cast<Bars*>(smem + OFF_BAR + kBarBytes);
  Pass c;
  c.p = &p;
  c.smem = smem;
  c.bars = bars;
  c.abort_flag = &bars->abort_flag;
  c.n_tiles = p.seq_pad / BT;
  c.warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);
  c.lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    init_bars(bars, true);
    init_bars(bars_q, false);
    bars->abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&m.q);
    tma_prefetch_desc(&m.k);
    tma_prefetch_desc(&m.v);
    tma_prefetch_desc(&m.d_o);
  }
  if (c.warp == 1) {
    tmem_alloc(&bars->tmem_slot, TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  c.tmem = __shfl_sync(0xffffffffu, bars->tmem_slot, 0);
  grid_dep_wait();
  // (No early launch of the next kernel: this one's CTAs end up to a unit apart, and whatever began to fill the
  // SMs that are done would have to stay there.)
  // Between the passes every role is done with the keys pass: its tiles and accumulators are free.
  const bool keys = (int)blockIdx.x < c.units();
  if (c.warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    int query = (int)blockIdx.x - c.units();
    if (keys) {
      if (c.warp == 0) query = keys_producer(c, m.q, m.k, m.v, m.d_o);
      if (c.warp == 1) {
        keys_mma(c);
        tc_commit_warp(&bars->first);  // (unused in this pass) every MMA has completed
        mbar_wait_drain(&bars->first, 0, p.err, DEV_TIMEOUT_ATTN_BWD + 14);
      }
      if (c.warp == 2) keys_proxy(c);
      tc_fence_before();
      __syncthreads();
      tc_fence_after();
    }
    c.bars = bars_q;
    if (c.warp == 0) queries_producer(c, m.k, m.v, m.d_o, query);
    if (c.warp == 1) {
      queries_mma(c);
      tc_commit_warp(&bars_q->own_x_empty);  // (unused in this pass)
      mbar_wait_drain(&bars_q->own_x_empty, 0, p.err, DEV_TIMEOUT_ATTN_BWD + 14);
    }
    if (c.warp == 2) queries_proxy(c);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsCompute));
    if (keys) {
      keys_compute(c);
      tc_fence_after();
    }
    c.bars = bars_q;
    queries_compute(c, m.dq);
    if (c.lane == 0) bulk_wait();  // the outputs are in memory
  }
  __syncthreads();
  if (c.warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(c.tmem, TM_COLS);
  }
}

}  // namespace

size_t attention_bwd_plan(AttnBwdArgs* a, uint8_t* base) {
  a->seq_pad = (a->seq + BT - 1) / BT * BT;
  const size_t rows = (size_t)a->batch * a->n_heads * a->seq_pad;
  const auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
  size_t at = 0;
  a->nlse2 = reinterpret_cast<float*>(base + at);
  at += up(rows * sizeof(float));
  a->ndelta = reinterpret_cast<float*>(base + at);
  at += up(rows * sizeof(float));
  a->counters = reinterpret_cast<int*>(base + at);
  at += 256;
  a->n_listed = reinterpret_cast<int*>(base + at);
  at += up((size_t)a->batch * sizeof(int));
  a->tiles = reinterpret_cast<int*>(base + at);
  at += up((size_t)a->batch * (a->seq_pad / BT) * sizeof(int));
  return at;
}

cudaError_t attention_bwd_launch(const AttnBwdMaps& m, const AttnBwdArgs& a, int num_sms, cudaStream_t s) {
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
  const long long units = (long long)a.batch * a.n_heads * (a.seq_pad / BT);
  const long long items = (long long)a.batch * a.seq_pad * ((a.n_heads + kRowHeads - 1) / kRowHeads);
  const long long row_ctas = (items + 15) / 16 + (a.key_mask != nullptr ? a.batch : 0);
  // Early launch, and leave for the next kernel to launch early, only while there are no more CTAs than SMs
  // (launch_early in mi_internal.h; 2 x 1000 rows x 8 heads, 256 CTAs: 46 us with both, 43 with the second, 37).
  const bool early = launch_early(row_ctas, num_sms);
  e = launch_kernel(attn_bwd_rows_kernel, dim3((unsigned)row_ctas), dim3(256), 0, s, early, a, early);
  if (e != cudaSuccess) return e;
  return launch_kernel(attn_bwd_kernel, dim3((unsigned)(2 * units < num_sms ? 2 * units : num_sms)), dim3(kThreads), SMEM_TOTAL,
                       s, true, m, a);
}

}  // namespace mi
