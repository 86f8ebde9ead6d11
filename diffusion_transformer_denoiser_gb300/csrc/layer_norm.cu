// Layer norm.  What it shares with the gradients, and what bounds it, is in norm_rows.cuh.
#include "norm_rows.cuh"

namespace mi {

namespace {

// A row's sum of squares is taken around its mean, so a row far from zero loses nothing: a warp with n columns finds their
// mean m and the squares q around it.  Over the warps of a row, A = sum n (m - m_0) and B = sum (q + n (m - m_0)^2) give the
// row's mean m_0 + A / width and its squares B - A^2 / width.  (What that difference takes off is at most as many times what is
// left as there are warps, 16: the row's squares are at least n_0 (m_0 - mean)^2, its first warp's.)
//
// kBehind: a row's sums over its warps, and its outputs, are one turn behind the warps' own sums and run beside the next row's,
// which hides most of the shuffles' and the barrier's time (16418 x 4096 bf16 51.5 -> 45.5 us, 8260 x 2560 20.1 -> 19.0).  It takes the
// registers of a second row: single words and 32 columns a lane do not have them (9237 x 1155 fp32 21.2 -> 27.4 us), and rows of
// one warp have nothing to wait for (40000 x 256 10.5 -> 10.9).
template <typename T, int V, int E, int kDepth, int kWarps, bool kWide>
__global__ void __launch_bounds__(kWarps * 32, 1) layer_norm_kernel(const LayerNormArgs a, const Plan p) {
  using P = Piece<T, V>;
  using L = typename P::L;
  constexpr int C = E / V, N = P::N, kThreads = kWarps * 32;
  using In = Reader<T, V, C, kWarps, kWide>;
  constexpr int kStage = In::kTurn;
  constexpr bool kBehind = kWide && V >= 4 && E == 16;
  extern __shared__ __align__(128) uint8_t memory[];
  __shared__ float2 parts[2][kWarps + 16];  // a warp's mean and squares (read 16 from a group's first on)
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
  auto columns_of = [&](int w) {  // of warp w of a row
    int n = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) n += min(max(a.width - (w * C + c) * 32 * V, 0), 32 * V);
    return (float)n;
  };
  const float inv_cols = kWide ? 1.0f / fmaxf(columns_of(me.row_warp), 1.0f) : inv;
  const float n_of_lane = (lane & 15) < p.row_warps ? columns_of(lane & 15) : 0.0f;
  L w[C][N], b[C][N];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    load_param<T, V>(a.weight, a.param_dtype, a.param_vec, 0, me.column(c), a.width, 1.0f, 0.0f, w[c]);
    load_param<T, V>(a.bias, a.param_dtype, a.param_vec, 0, me.column(c), a.width, 0.0f, 0.0f, b[c]);
  }
  uint8_t* out = static_cast<uint8_t*>(a.out) + (row * a.out_stride + me.first) * (long long)sizeof(T);
  const uint32_t last = slot0 + (kDepth - 1) * kStage;
  uint32_t stage = slot0, ahead = last;
  auto fetch = [&](L (&x)[C][N], float& s) {  // the row that has come, and the sum of this lane's columns
    if (V < 4) __syncwarp();  // (the warp has read what now makes room)
    ask(ahead);
    copy_wait<kDepth - 1>();
    if (V < 4) __syncwarp();
    L t = v_of<L>(0.0f);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      x_in.load(stage, me, c, x[c]);
#pragma unroll
      for (int e = 0; e < N; ++e) t = v_add(t, x[c][e]);
    }
    x_in.advance(p.step[0]);
    ahead = stage;
    stage = stage == last ? slot0 : stage + kStage;
    s = v_sum(t);
  };
  auto squares = [&](const L (&x)[C][N], float m) {  // of this lane's columns around m
    L t = v_of<L>(0.0f);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const L nm = bytes[c] == V * sizeof(T) ? v_of<L>(-m) : V == 2 && bytes[c] == sizeof(T) ? v_of2<L>(-m, 0.0f) : v_of<L>(0.0f);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const L d = v_add(x[c][e], nm);
        t = v_fma(d, d, t);
      }
    }
    return v_sum(t);
  };
  // The lane's part of a row's sums over its warps (see above), from the turn's parts.
  float first = 0.0f;
  auto joined = [&](int turn) {
    first = parts[turn][me.group * p.row_warps].x;
    const float2 part = parts[turn][me.group * p.row_warps + (lane & 15)];
    const float d = part.x - first, nd = n_of_lane * d;
    const float v = lane < 16 ? nd : fmaf(nd, d, part.y);
    return (lane & 15) < p.row_warps ? v : 0.0f;
  };
  auto write = [&](const L (&x)[C][N], float mean, float square) {
    const float rstd = rsqrtf(fmaf(square, inv, a.eps));
    const bool mine = me.sub < left;
    const L nm = v_of<L>(-mean), rs = v_of<L>(rstd);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      L o[N];
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = v_fma(v_mul(v_add(x[c][e], nm), rs), w[c][e], b[c][e]);
      P::store(out + c * me.apart() * (int)sizeof(T), mine ? bytes[c] : 0u, o);
    }
    if (me.first == 0 && mine) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    left -= apart;
    row += apart;
    out += p.step[3];
  };
  float m, q;  // a row's, as this warp has it
  if constexpr (kBehind) {
    auto share = [&](int turn) {
      if (lane == 0) parts[turn][warp] = make_float2(m, q);
      group_sync(me.group, p.row_warps);
    };
    auto turn_of = [&](int turn, const L (&x)[C][N], L (&next)[C][N]) {
      float s;
      fetch(next, s);
      float v = joined(turn);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        s += __shfl_xor_sync(0xffffffffu, s, o);
        if (o < 16) v += __shfl_xor_sync(0xffffffffu, v, o);
      }
      const float u = __shfl_xor_sync(0xffffffffu, v, 16);
      const float sum = lane < 16 ? v : u, more = lane < 16 ? u : v;
      m = s * inv_cols;
      q = warp_sum(squares(next, m));
      write(x, fmaf(sum, inv, first), fmaf(-sum * inv, sum, more));
      share(turn ^ 1);
    };
    L even[C][N], odd[C][N];
    if (left > 0) {
      fetch(even, m);
      m = warp_sum(m) * inv_cols;
      q = warp_sum(squares(even, m));
      share(0);
    }
    while (left > 0) {
      turn_of(0, even, odd);
      if (left <= 0) break;
      turn_of(1, odd, even);
    }
  } else {
    for (int turn = 0; left > 0; turn ^= 1) {
      L x[C][N];
      float s;
      fetch(x, s);
      m = (kWide ? warp_sum(s) : lanes_sum(s, p.row_lanes)) * inv_cols;
      s = squares(x, m);
      q = kWide ? warp_sum(s) : lanes_sum(s, p.row_lanes);
      if constexpr (kWide) {
        if (lane == 0) parts[turn][warp] = make_float2(m, q);
        group_sync(me.group, p.row_warps);
        const float2 both = warps_sum2(joined(turn));
        m = fmaf(both.x, inv, first);
        q = fmaf(-both.x * inv, both.x, both.y);
      }
      write(x, m, q);
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
