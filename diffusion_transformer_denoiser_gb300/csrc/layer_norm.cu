// Layer norm.  What it shares with the gradients, and what bounds it, is in norm_rows.cuh.
#include "norm_rows.cuh"

namespace mi {

namespace {

// f of the columns of a row by pairs, which v has one after the other.  Single words make one with the word before.
template <int V, typename L, typename F>
__device__ __forceinline__ void in_pairs(int c, L v, L& before, F f) {
  if constexpr (V > 1) f(v);
  else if (c % 2 == 1) f(f2_pack(before, v));
  before = v;
}

// A row's squares are taken around its mean, and what the mean's rounding leaves is taken off again: a row that is far from zero
// and hardly spread (100000.1 everywhere) is closer together than an fp32 mean is good.  A warp with n columns finds their
// mean m, the deviations d = x - m, which are what is kept of x, and the sums r of d (0 but for m's rounding) and q of d^2.
// Over the warps of a row, A = sum (n (m - m_0) + r) and B = sum (q + (m - m_0) (n (m - m_0) + 2 r)) are the sums of x - m_0 and of its
// square: the row's mean is m_0 + A / width, its squares are B - A^2 / width, its deviations d + (m - m_0) - A / width.  Only
// the mean that is stored is rounded at x's size.  (What the difference of the squares takes off is at most as many times what is
// left as there are warps, 16: the row's squares are at least n_0 (m_0 - mean)^2, its first warp's.  Where nothing but rounding is
// left it is not let below 0.)
//
// kRest: r is summed up, for rows of fp32.  In 16 bits it is sum(x) - n m, one fma, because the sum is exact where r counts: of at
// most 1024 columns whose values have 11 bits within 3 binades, or 8 bits within 6, and are multiples of max|x| / 2^14.  A row
// with smaller ones is spread from its largest |x| down to an eighth of it, and the sum's rounding is below 10^-4 of its deviation.
// (Summing up r there as well: 16418 x 4096 bf16 53.9 us, with the fma 44.9, without either 44.6.  fp32 9237 x 1155 19.0, without 18.6.)
//
// kBehind: a row's sums over its warps, and its outputs, are one turn behind the warps' own sums and run beside the next row's,
// which hides most of the shuffles' and the barrier's time (16418 x 4096 bf16 51.5 -> 45.5 us, 8260 x 2560 20.1 -> 19.0).  It takes the
// registers of a second row: single words and 32 columns a lane do not have them (9237 x 1155 fp32 21.2 -> 27.4 us), and rows of
// one warp have nothing to wait for (40000 x 256 10.5 -> 10.9).
template <typename T, int V, int E, int kDepth, int kWarps, bool kWide>
__global__ void __launch_bounds__(kWarps * 32, 1) layer_norm_kernel(const LayerNormArgs a, const Plan p) {
  using P = Piece<T, V>;
  using L = typename P::L;
  constexpr int C = E / V, N = P::N;
  using In = Reader<T, V, C, kWarps, kWide>;
  constexpr int kStage = In::kTurn;
  constexpr bool kBehind = kWide && V >= 4 && E == 16;
  constexpr bool kRest = sizeof(T) == 4;
  // 32 columns a lane: what is kept of x, the weights and the biases do not all fit in registers.  (4000 rows, us: odd rows read from
  // shared memory again, 10,007 columns bf16 84.9, in registers 95.1, fp32 75.7 and 78.4; vectors in registers, bf16 10,240 and
  // 16,384 columns 37.3 and 49.9, from shared memory 38.6 and 53.4; biases of fp32 vectors from L1, 12,288 columns 70.3, in
  // registers 74.1; of bf16, 10,240 and 16,384 columns, 41.0 and 48.1.)
  constexpr bool kHold = E <= 16 || V >= 4, kHoldBias = E <= 16 || V != 4;
  constexpr int H = kHold ? C : 1;
  // What a warp tells the others: m, q and r; or in fewer words its sum of x and q - r^2 / n.  (8260 x 2560 bf16 17.9 us, with three
  // words 18.2; but 32 columns a lane have no registers for what it takes: 4000 x 16384 bf16 49.9 with three, 59.3 with two.)
  constexpr bool kThree = kRest || (E == 32 && V == 8);
  using Part = typename std::conditional<kThree, float4, float2>::type;
  extern __shared__ __align__(128) uint8_t memory[];
  __shared__ Part parts[2][kWarps + 16];  // (read 16 from a group's first on)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Place<V, C, kWide> me(p);
  grid_dep_wait();
  const Share mine_of(a.rows, blockIdx.x, gridDim.x);
  const long long row0 = mine_of.first;
  const int rows = mine_of.count;
  const int apart = p.apart;
  int left = me.group < p.groups ? rows - me.group * p.batch : 0;  // rows from the group's next batch on
  long long row = row0 + me.group * p.batch + me.sub;
  uint32_t bytes[C];  // of the thread's pieces that are in the row
#pragma unroll
  for (int c = 0; c < C; ++c) bytes[c] = (uint32_t)min(max(a.width - me.column(c), 0), V) * sizeof(T);
  In x_in(a.x, a.x_stride, row, a.width, me);
  const uint32_t slot0 = In::place(smem_u32(memory), me);
  int to_ask = left - me.sub;  // rows of this thread
  auto ask = [&](uint32_t to) {
    x_in.ask(a.x, to, me, bytes, to_ask > 0, to_ask > apart, p.step[0]);
    to_ask -= apart;
    copy_commit();
  };
#pragma unroll
  for (int k = 0; k < kDepth - 1; ++k) ask(slot0 + k * kStage);
  grid_dep_launch();
  const float inv = 1.0f / (float)a.width;
  // Columns of a warp of the row: all full but the last one.
  const int last_warp = p.row_warps - 1;
  const float n_last = (float)(a.width - last_warp * 32 * E), inv_last = 1.0f / n_last;
  const float cols = me.row_warp < last_warp ? (float)(32 * E) : n_last, inv_cols = me.row_warp < last_warp ? 1.0f / (32 * E) : inv_last;
  L w[C][N], b[kHoldBias ? C : 1][N];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    load_param<T, V>(a.weight, a.param_dtype, a.param_vec, 0, me.column(c), a.width, 1.0f, 0.0f, w[c]);
    if constexpr (kHoldBias) load_param<T, V>(a.bias, a.param_dtype, a.param_vec, 0, me.column(c), a.width, 0.0f, 0.0f, b[c]);
  }
  uint8_t* out = static_cast<uint8_t*>(a.out) + (row * a.out_stride + me.first) * (long long)sizeof(T);
  const uint32_t last = slot0 + (kDepth - 1) * kStage;
  uint32_t stage = slot0, ahead = last;
  uint32_t here = slot0;  // where the row that has come is
  auto fetch = [&](L (&x)[H][N], float& s) {  // the row that has come, and the sum of this lane's columns
    if (V < 4) __syncwarp();  // (the warp has read what now makes room)
    ask(ahead);
    copy_wait<kDepth - 1>();
    if (V < 4) __syncwarp();
    f32x2_t t = 0;
    L before;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      L (&xc)[N] = x[kHold ? c : 0];
      x_in.load(stage, me, c, xc);
#pragma unroll
      for (int e = 0; e < N; ++e) in_pairs<V>(c, xc[e], before, [&](f32x2_t v) { t = f2_add(t, v); });
    }
    here = ahead = stage;
    stage = stage == last ? slot0 : stage + kStage;
    s = v_sum(t);
  };
  auto minus = [&](float m, int c) -> L {  // -m in the columns of piece c that are in the row
    const L none = 0;
    return bytes[c] == V * sizeof(T) ? v_of<L>(-m) : V == 2 && bytes[c] == sizeof(T) ? v_of2<L>(-m, 0.0f) : none;
  };
  // The sums of this lane's deviations' squares and (kRest) of the deviations, which take x's place.
  auto squares = [&](L (&x)[H][N], float m, float& rest) {
    f32x2_t t = 0, r = 0;
    L before;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      L (&xc)[N] = x[kHold ? c : 0];
      if constexpr (!kHold) x_in.load(here, me, c, xc);
      const L nm = minus(m, c);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        xc[e] = v_add(xc[e], nm);
        in_pairs<V>(c, xc[e], before, [&](f32x2_t d) {
          t = f2_fma(d, d, t);
          if constexpr (kRest) r = f2_add(d, r);
        });
      }
    }
    if constexpr (kRest) rest = v_sum(r);
    return v_sum(t);
  };
  // The lane's part of a row's sums over its warps (see above), from the turn's parts.  (The first warp of several is full.)
  float first = 0.0f;  // m_0
  auto joined = [&](int turn) {
    const Part* at = &parts[turn][me.group * p.row_warps];
    const Part part = at[lane & 15];
    const bool full = (lane & 15) < last_warp;
    const float n = full ? (float)(32 * E) : n_last;
    float v;
    if constexpr (kThree) {
      first = at[0].x;
      const float d = part.x - first, nd = fmaf(n, d, part.z);
      v = lane < 16 ? nd : fmaf(d, nd + part.z, part.y);
    } else {
      first = __fmul_rn(at[0].x, 1.0f / (32 * E));
      const float nd = fmaf(-n, first, part.x);
      v = lane < 16 ? nd : fmaf(nd * (full ? 1.0f / (32 * E) : inv_last), nd, part.y);
    }
    return (lane & 15) <= last_warp ? v : 0.0f;
  };
  auto share = [&](int turn, float s, float m, float q, float r) {  // q: this lane's; r: this lane's (kRest) or the warp's
    q = warp_sum(q);
    if constexpr (kRest) r = warp_sum(r);
    if constexpr (kThree) {
      if (lane == 0) parts[turn][warp] = Part{m, q, r, 0.0f};
    } else {
      q = fmaf(-r * inv_cols, r, q);
      if (lane == 0) parts[turn][warp] = Part{s, q};
    }
    group_sync(me.group, p.row_warps);
  };
  // x: the deviations from this warp's mean m; off: what is still to be added to them
  auto write = [&](const L (&x)[H][N], float m, float mean, float off, float square) {
    const float rstd = rsqrtf(fmaf(square < 0.0f ? 0.0f : square, inv, a.eps));
    const bool mine = me.sub < left;
    const L shift = v_of<L>(off), rs = v_of<L>(rstd);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      L d[N], o[N];
      if constexpr (!kHoldBias) load_param<T, V>(a.bias, a.param_dtype, a.param_vec, 0, me.column(c), a.width, 0.0f, 0.0f, b[0]);
      if constexpr (!kHold) x_in.load(here, me, c, d);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        d[e] = kHold ? x[kHold ? c : 0][e] : v_add(d[e], minus(m, c));
        o[e] = v_fma(v_mul(v_add(d[e], shift), rs), w[c][e], b[kHoldBias ? c : 0][e]);
      }
      P::store(out + c * me.apart() * (int)sizeof(T), mine ? bytes[c] : 0u, o);
    }
    if (me.first == 0 && mine) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    x_in.advance(p.step[0]);
    left -= apart;
    row += apart;
    out += p.step[3];
  };
  if constexpr (kBehind) {
    float m;  // this warp's mean of the row in x
    auto turn_of = [&](int turn, L (&x)[H][N], L (&next)[H][N]) {
      float s, r;
      fetch(next, s);
      float v = joined(turn);
      const float apart_by = m - first;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        if (o < 16) v += __shfl_xor_sync(0xffffffffu, v, o);
      }
      const float u = __shfl_xor_sync(0xffffffffu, v, 16);
      const float sum = lane < 16 ? v : u, more = lane < 16 ? u : v;
      m = __fmul_rn(s, inv_cols);
      r = fmaf(-cols, m, s);
      const float q = squares(next, m, r);
      write(x, m, fmaf(sum, inv, first), fmaf(-sum, inv, apart_by), fmaf(-sum * inv, sum, more));
      share(turn ^ 1, s, m, q, r);
    };
    L even[H][N], odd[H][N];
    if (left > 0) {
      float s;
      fetch(even, s);
      s = warp_sum(s);
      m = __fmul_rn(s, inv_cols);
      float r = fmaf(-cols, m, s);
      const float q = squares(even, m, r);
      share(0, s, m, q, r);
    }
    while (left > 0) {
      turn_of(0, even, odd);
      if (left <= 0) break;
      turn_of(1, odd, even);
    }
  } else {
    for (int turn = 0; left > 0; turn ^= 1) {
      L x[H][N];
      float s;
      fetch(x, s);
      s = kWide ? warp_sum(s) : lanes_sum(s, p.row_lanes);
      const float m = __fmul_rn(s, inv_cols);
      float r = fmaf(-cols, m, s);
      const float q = squares(x, m, r);
      if constexpr (kWide) {
        share(turn, s, m, q, r);
        const float2 both = warps_sum2(joined(turn));
        write(x, m, fmaf(both.x, inv, first), fmaf(-both.x, inv, m - first), fmaf(-both.x * inv, both.x, both.y));
      } else {
        const float2 both = make_float2(kRest ? lanes_sum(r, p.row_lanes) : r, lanes_sum(q, p.row_lanes));
        write(x, m, fmaf(both.x, inv, m), -both.x * inv, fmaf(-both.x * inv, both.x, both.y));
      }
    }
  }
  copy_wait<0>();
}

template <typename T, int V, int E, int kWarps, bool kWide>
cudaError_t layer_norm_start(const LayerNormArgs& a, const Plan& p, int grid, cudaStream_t s) {
  constexpr int kTurn = Reader<T, V, E / V, kWarps, kWide>::kTurn, kDepth = depth_of(1, kTurn);
  constexpr auto kKernel = layer_norm_kernel<T, V, E, kDepth, kWarps, kWide>;
  cudaError_t e = allow_ring<kKernel>();
  if (e != cudaSuccess) return e;
  return launch_kernel(kKernel, dim3(grid), dim3(kWarps * 32), (size_t)kDepth * kTurn, s, true, a, p);
}

template <typename T, int V, int E, int kWarps>
cudaError_t layer_norm_run(const LayerNormArgs& a, int num_sms, cudaStream_t s) {
  Plan p = make_plan(a.width, E, kWarps);
  p.step[0] = p.apart * a.x_stride * (long long)sizeof(T);
  p.step[3] = p.apart * a.out_stride * (long long)sizeof(T);
  const long long need = ((long long)a.rows + p.apart - 1) / p.apart;
  const int grid = need < num_sms ? (int)need : num_sms;
  if constexpr (E == 8 || (E == 16 && V >= 4))  // (wider pieces come with wide rows only)
    if (p.row_warps == 1) return layer_norm_start<T, V, E, kWarps, false>(a, p, grid, s);
  if (!wide_plan(p)) return cudaErrorInvalidConfiguration;
  return layer_norm_start<T, V, E, kWarps, true>(a, p, grid, s);
}

// Columns of a lane and warps of a CTA: 16 with 16 (40 M bf16 elements: 30 us at widths 256, 2560 and 4096; 8 with 24 warps, without the
// turn behind, 30, 39, 43).  Odd rows of 16 bits: 8 with 24 up to six warps of them (16 M: width 515 35 / 40 us, 1155 30 / 32,
// 1535 27 / 27); of fp32: up to three (515 33 / 36; 771 27 with 16 columns, 30 with 8; 1283 26 / 28).  32 where 16 warps of 16
// columns a lane do not hold a row.
template <typename T, int V>
cudaError_t layer_norm_any(const LayerNormArgs& a, int num_sms, cudaStream_t s) {
  if (a.width > 16 * 32 * 16) return layer_norm_run<T, V, 32, 16>(a, num_sms, s);
  if constexpr (V < 4)
    if (a.width <= (V == 1 ? 3 : 6) * 32 * 8) return layer_norm_run<T, V, 8, 24>(a, num_sms, s);
  return layer_norm_run<T, V, 16, 16>(a, num_sms, s);
}

template <typename T, int V>
cudaError_t layer_norm_type(LayerNormArgs a, int num_sms, cudaStream_t s) {
  a.param_vec = on16(a.weight, 0) && on16(a.bias, 0);
  const long long size = sizeof(T);
  if (a.width % V == 0 && on16(a.x, a.x_stride * size) && on16(a.out, a.out_stride * size))
    return layer_norm_any<T, V>(a, num_sms, s);
  return layer_norm_any<T, sizeof(T) == 4 ? 1 : 2>(a, num_sms, s);
}

}  // namespace

cudaError_t layer_norm_launch(const LayerNormArgs& a, int num_sms, cudaStream_t s) {
  if (a.rows <= 0) return cudaSuccess;
  if (a.dtype == MI_F32) return layer_norm_type<float, 4>(a, num_sms, s);
  if (a.dtype == MI_F16) return layer_norm_type<__half, 8>(a, num_sms, s);
  return layer_norm_type<__nv_bfloat16, 8>(a, num_sms, s);
}

}  // namespace mi
