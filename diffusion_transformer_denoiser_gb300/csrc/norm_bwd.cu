// Gradients of layer norm and of the modulated RMSNorm.  What they share with the forward, and what bounds them, is in
// norm_rows.cuh.
#include "norm_rows.cuh"

namespace mi {

namespace {

constexpr float kMax = 3.402823466e38f;
constexpr int kCluster = 8;       // CTAs that sum their rows up in one launch, where rows are few
// Turns of their groups up to which that is done.  (Width 256, us called in turn / replayed from a graph, against two kernels:
// 74 rows 9.3 / 5.4 against 11.2 / 6.2; 512, two turns, 9.4 / 6.9 against 11.0 / 6.6; 1024, four, 9.5 / 8.4 against 11.0 / 6.7.)
constexpr int kClusterTurns = 2;

// With g = dy w, n = (x - mean) rstd (rms: x rstd) and the row's sums of g and g (x - mean) (rms: of x^2 and g x):
//   dx = residual + rstd (g - mean(g) - n mean(g n))   (rms: without mean(g))
//   sums over rows: dweight += dy n, dbias += dy.
// A row whose sums or statistics are not finite, and with given statistics one whose two sums are both zero, is looked at
// again: if its dy is zero it counts as absent, so what padding holds reaches nothing.  (A dy of zeros gives sums of 0 or NaN.
// With finite x and statistics n may still overflow and dy n be NaN; an rms norm makes its own r, and x r stays finite.)
// Rows with a gradient pay two comparisons (8260 x 2560 bf16 with a residual 32.4 us on the device with and without them); a batch that
// is all padding 33.2 instead of 32.6, 4503 x 1283 fp16 18.9 instead of 17.7.
//
// Without the sums over rows the loop runs at 0.98 of the measured copy rate (33040 x 2560 with a residual 103 us, the copies'
// floor 101); adding them up costs 4 to 5 us a call.  A row's sums one turn behind, beside the next row's, as in the forward, gained
// nothing: the registers of a second row are not there, and reading the row from shared memory again costs as much as it
// hides (8260 x 2560 35.0 against 33.9 us; with 8 columns a lane 3 x 10571 x 1792 rms 69.3 against 65.0).
template <typename T, int V, int E, int kDepth, int kWarps, bool kWide, bool kRms, bool kResidual>
__global__ void __launch_bounds__(kWarps * 32, 1) norm_bwd_kernel(const NormBwdArgs a, const Plan p, int n_parts) {
  using P = Piece<T, V>;
  using L = typename P::L;
  constexpr int C = E / V, N = P::N, kInputs = kResidual ? 3 : 2, kThreads = kWarps * 32;
  constexpr bool kHold = E <= 16;  // a row in registers; wider rows are read from shared memory again, their weights from L1
  using In = Reader<T, V, C, kWarps, kWide>;
  constexpr int kStage = kInputs * In::kTurn;
  extern __shared__ __align__(128) uint8_t memory[];
  __shared__ float2 parts[2][kWarps + 16];  // a warp's sums (read 16 from a group's first on)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Place<V, C, kWide> me(p);
  grid_dep_wait();
  const int set = blockIdx.x / n_parts, part_of_set = blockIdx.x - set * n_parts;
  const Share mine_of(a.seq, part_of_set, n_parts);
  const long long row0 = (long long)set * a.seq + mine_of.first;
  const int rows = mine_of.count;
  const int apart = p.apart;
  int left = me.group < p.groups ? rows - me.group * p.batch : 0;  // rows from the group's next batch on
  long long row = row0 + me.group * p.batch + me.sub;
  uint32_t bytes[C];
#pragma unroll
  for (int c = 0; c < C; ++c) bytes[c] = (uint32_t)min(max(a.width - me.column(c), 0), V) * sizeof(T);
  In x_in(a.x, a.x_stride, row, a.width, me), y_in(a.dy, a.dy_stride, row, a.width, me), r_in(a.residual, a.residual_stride, row, a.width, me);
  const uint32_t slot0 = In::place(smem_u32(memory), me);
  int to_ask = left - me.sub;
  auto ask = [&](uint32_t to) {
    x_in.ask(a.x, to, me, bytes, to_ask > 0, to_ask > apart, p.step[0]);
    y_in.ask(a.dy, to + In::kTurn, me, bytes, to_ask > 0, to_ask > apart, p.step[1]);
    if (kResidual) r_in.ask(a.residual, to + 2 * In::kTurn, me, bytes, to_ask > 0, to_ask > apart, p.step[2]);
    to_ask -= apart;
    copy_commit();
  };
#pragma unroll
  for (int k = 0; k < kDepth - 1; ++k) ask(slot0 + k * kStage);
  grid_dep_launch();
  const float inv = 1.0f / (float)a.width;
  const long long w_at = set * a.weight_gstride;
  auto weights = [&](int c, L (&f)[N]) {
    load_param<T, V>(a.weight, a.param_dtype, a.param_vec, w_at, me.column(c), a.width, kRms ? 0.0f : 1.0f,
                     kRms ? 1.0f : 0.0f, f);
  };
  L w[kHold ? C : 1][N], aw[C][N], ab[C][N];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if constexpr (kHold) weights(c, w[c]);
#pragma unroll
    for (int e = 0; e < N; ++e) aw[c][e] = ab[c][e] = v_of<L>(0.0f);
  }
  uint8_t* out = static_cast<uint8_t*>(a.dx) + (row * a.dx_stride + me.first) * (long long)sizeof(T);
  float next_mean = 0.0f, next_rstd = 0.0f;
  if (!kRms && me.sub < left) {
    next_mean = a.mean[row];
    next_rstd = a.rstd[row];
  }
  const uint32_t last = slot0 + (kDepth - 1) * kStage;
  uint32_t stage = slot0, ahead = last;
  for (int turn = 0; left > 0; turn ^= 1) {
    if (V < 4) __syncwarp();  // (the warp has read what now makes room)
    ask(ahead);
    float mean = next_mean, rstd = next_rstd;
    if (!kRms && me.sub < left - apart) {
      next_mean = a.mean[row + apart];
      next_rstd = a.rstd[row + apart];
    }
    copy_wait<kDepth - 1>();
    if (V < 4) __syncwarp();
    const bool mine = me.sub < left;
    const L m = v_of<L>(-mean);
    L x[kHold ? C : 1][N], y[kHold ? C : 1][N];  // x: less its mean
    L t1 = v_of<L>(0.0f), t2 = v_of<L>(0.0f);
    auto load = [&](int c, L (&xc)[N], L (&yc)[N]) {
      x_in.load(stage, me, c, xc);
      y_in.load(stage + In::kTurn, me, c, yc);
    };
    auto add = [&](L (&xc)[N], const L (&yc)[N], const L (&wc)[N]) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const L g = v_mul(yc[e], wc[e]);
        if (kRms) {
          t1 = v_fma(xc[e], xc[e], t1);
        } else {
          xc[e] = v_add(xc[e], m);
          t1 = v_add(g, t1);
        }
        t2 = v_fma(g, xc[e], t2);
      }
    };
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if constexpr (kHold) {
        load(c, x[c], y[c]);
        add(x[c], y[c], w[c]);
      } else {
        L xc[N], yc[N], wc[N];
        load(c, xc, yc);
        weights(c, wc);
        add(xc, yc, wc);
      }
    }
    float s1 = v_sum(t1), s2 = v_sum(t2);
    if constexpr (kWide) {
      // both sums in one butterfly: the lower half of the warp goes on with s1, the upper with s2
      const bool upper = lane >= 16;
      float keep = upper ? s2 : s1;
      keep += __shfl_xor_sync(0xffffffffu, upper ? s1 : s2, 16);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) keep += __shfl_xor_sync(0xffffffffu, keep, o);
      if ((lane & 15) == 0) reinterpret_cast<float*>(&parts[turn][warp])[lane >> 4] = keep;
      group_sync(me.group, p.row_warps);
      const float2 part = parts[turn][me.group * p.row_warps + (lane & 15)];
      const float2 both = warps_sum2((lane & 15) < p.row_warps ? (upper ? part.y : part.x) : 0.0f);
      s1 = both.x;
      s2 = both.y;
    } else {
      s1 = lanes_sum(s1, p.row_lanes);
      s2 = lanes_sum(s2, p.row_lanes);
    }
    if (kRms) rstd = rsqrtf(fmaf(s1, inv, a.eps));
    float c1 = kRms ? 0.0f : s1 * inv, c2 = s2 * rstd * inv;
    bool gone = !(fabsf((c1 + c2) + (rstd + mean)) <= kMax) || (!kRms && s1 == 0.0f && s2 == 0.0f);
    if (kWide ? gone : (bool)__any_sync(0xffffffffu, gone)) {  // does the row have a gradient at all?
      bool any = false;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        L xc[N], yc[N];
        load(c, xc, yc);
#pragma unroll
        for (int e = 0; e < N; ++e) any |= v_any(yc[e]);
      }
      if constexpr (kWide) {
        gone = !group_any(any, me.group, p.row_warps);
      } else {
        const uint32_t lanes = __ballot_sync(0xffffffffu, any) >> (me.sub * p.row_lanes);
        gone = gone && (p.row_lanes == 32 ? lanes : lanes & ((1u << p.row_lanes) - 1u)) == 0;
      }
      if (gone) {
        rstd = c1 = c2 = 0.0f;
        if constexpr (kHold) {
#pragma unroll
          for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < N; ++e) x[c][e] = v_of<L>(0.0f);
        }
      }
    } else {
      gone = false;
    }
    const L rs = v_of<L>(rstd), nc1 = v_of<L>(-c1), nc2 = v_of<L>(-c2);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      L xc[N], yc[N], wc[N], o[N];
      if constexpr (kHold) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          xc[e] = x[c][e];
          yc[e] = y[c][e];
          wc[e] = w[c][e];
        }
      } else {
        load(c, xc, yc);
        weights(c, wc);
#pragma unroll
        for (int e = 0; e < N; ++e) xc[e] = gone ? v_of<L>(0.0f) : kRms ? xc[e] : v_add(xc[e], m);
      }
      if constexpr (kResidual) {
        r_in.load(stage + 2 * In::kTurn, me, c, o);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] = v_of<L>(0.0f);
      }
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const L xn = v_mul(xc[e], rs);
        aw[c][e] = v_fma(yc[e], xn, aw[c][e]);
        ab[c][e] = v_add(yc[e], ab[c][e]);
        const L g = kRms ? v_mul(yc[e], wc[e]) : v_fma(yc[e], wc[e], nc1);
        const L t = v_fma(xn, nc2, g);
        o[e] = kResidual ? v_fma(t, rs, o[e]) : v_mul(t, rs);
      }
      P::store(out + c * me.apart() * (int)sizeof(T), mine ? bytes[c] : 0u, o);
    }
    x_in.advance(p.step[0]);
    y_in.advance(p.step[1]);
    if (kResidual) r_in.advance(p.step[2]);
    left -= apart;
    row += apart;
    out += p.step[3];
    ahead = stage;
    stage = stage == last ? slot0 : stage + kStage;
  }
  copy_wait<0>();
  if (a.dweight == nullptr && a.dbias == nullptr) return;
  // The groups' sums, in place of the copies: [group][2][width].
  __syncthreads();
  if (p.batch > 1) {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < N; ++e)
#pragma unroll
        for (int o = 16; o >= 4; o >>= 1)
          if (o >= p.row_lanes) {
            aw[c][e] = v_add(aw[c][e], __shfl_xor_sync(0xffffffffu, aw[c][e], o));
            ab[c][e] = v_add(ab[c][e], __shfl_xor_sync(0xffffffffu, ab[c][e], o));
          }
  }
  float* sums = reinterpret_cast<float*>(memory);
  if (me.group < p.groups && me.sub == 0) {
    float* to = sums + (size_t)me.group * 2 * a.width;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int col = me.column(c);
      if constexpr (V >= 4) {  // whole vectors, at multiples of 16 bytes
        if (bytes[c] == 0) continue;
#pragma unroll
        for (int e = 0; e < N; e += 2) {
          float4 v;
          f2_unpack(aw[c][e], v.x, v.y);
          f2_unpack(aw[c][e + 1], v.z, v.w);
          *reinterpret_cast<float4*>(to + col + 2 * e) = v;
          f2_unpack(ab[c][e], v.x, v.y);
          f2_unpack(ab[c][e + 1], v.z, v.w);
          *reinterpret_cast<float4*>(to + a.width + col + 2 * e) = v;
        }
      } else if constexpr (V == 2) {
        float lo, hi;
        f2_unpack(aw[c][0], lo, hi);
        if (col < a.width) to[col] = lo;
        if (col + 1 < a.width) to[col + 1] = hi;
        f2_unpack(ab[c][0], lo, hi);
        if (col < a.width) to[a.width + col] = lo;
        if (col + 1 < a.width) to[a.width + col + 1] = hi;
      } else if (col < a.width) {
        to[col] = aw[c][0];
        to[a.width + col] = ab[c][0];
      }
    }
  }
  __syncthreads();
  float* to = p.cluster > 0 ? sums : a.partial + (long long)blockIdx.x * 2 * a.width;  // (in a cluster: the first group's place)
  if constexpr (V >= 4) {
    for (int c = threadIdx.x * 4; c < 2 * a.width; c += kThreads * 4) {
      float4 t = *reinterpret_cast<const float4*>(sums + c);
      for (int g = 1; g < p.groups; ++g) {
        const float4 v = *reinterpret_cast<const float4*>(sums + (size_t)g * 2 * a.width + c);
        t = make_float4(t.x + v.x, t.y + v.y, t.z + v.z, t.w + v.w);
      }
      *reinterpret_cast<float4*>(to + c) = t;
    }
  } else {
    for (int c = threadIdx.x; c < 2 * a.width; c += kThreads) {
      float t = sums[c];
      for (int g = 1; g < p.groups; ++g) t += sums[(size_t)g * 2 * a.width + c];
      to[c] = t;
    }
  }
  if (p.cluster == 0) return;
  // The cluster is all CTAs of the set: each adds up its share of the columns.
  cluster_sync();
  const int rank = (int)cluster_rank();
  const bool both = a.dweight == a.dbias;
  const long long at = set * a.sum_gstride;
  for (int c = rank * kThreads + threadIdx.x; c < a.width; c += p.cluster * kThreads) {
    float dw = 0.0f, db = 0.0f;
    for (int r = 0; r < p.cluster; ++r) {
      float v, u;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr(sums + c, (uint32_t)r)) : "memory");
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(u) : "r"(cluster_addr(sums + a.width + c, (uint32_t)r)) : "memory");
      dw += v;
      db += u;
    }
    if (both) {
      a.dweight[at + c] = dw + db;
    } else {
      if (a.dweight != nullptr) a.dweight[at + c] = dw;
      if (a.dbias != nullptr) a.dbias[at + c] = db;
    }
  }
  cluster_sync();  // nobody leaves while its sums are being read
}

// dweight and dbias: the sums of the CTAs' parts [set][part][2][width].  A CTA takes 32 of the 2 width columns, its 16 warps
// every 16th part each (with up to 160 parts all loads at once: the kernel is one trip to the L2 cache), and adds the warps up
// in order.  both: the two go to one row, added.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(kSumWarps * 32) norm_sum_kernel(const float* partial, int parts, int width,
                                                                  float* dweight, float* dbias, long long sum_gstride, int blocks) {
  __shared__ float sums[kSumWarps][33];
  const int set = blockIdx.x / blocks, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = (blockIdx.x - set * blocks) * 32 + lane;
  const bool both = dweight == dbias;
  const float* p = partial + ((long long)set * parts + warp) * 2 * width + c;
  float t = 0.0f;
  grid_dep_wait();
  grid_dep_launch();
  if (c < (both ? width : 2 * width)) {
    for (int i = warp; i < parts; i += 10 * kSumWarps, p += 10LL * kSumWarps * 2 * width) {
      float v[10], u[10];
#pragma unroll
      for (int k = 0; k < 10; ++k) {
        const bool in = i + k * kSumWarps < parts;
        v[k] = in ? __ldcg(p + (long long)k * kSumWarps * 2 * width) : 0.0f;
        u[k] = in && both ? __ldcg(p + (long long)k * kSumWarps * 2 * width + width) : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < 10; ++k) t += v[k] + u[k];
    }
  }
  sums[warp][lane] = t;
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int i = 1; i < kSumWarps; ++i) t += sums[i][lane];
  const long long at = set * sum_gstride;
  if (c < width) {
    if (dweight != nullptr) dweight[at + c] = t;
  } else if (c < 2 * width && dbias != nullptr && !both) {
    dbias[at + c - width] = t;
  }
}

int norm_bwd_parts(int groups, int seq, int num_sms) {
  const int most = num_sms / groups > 0 ? num_sms / groups : 1;
  return seq < most ? seq : most;
}

template <typename T, int V, int E, int kWarps, bool kWide, bool kRms, bool kResidual>
cudaError_t norm_bwd_start(const NormBwdArgs& a, const Plan& p, int parts, bool sums, cudaStream_t s) {
  constexpr int kInputs = kResidual ? 3 : 2, kTurn = Reader<T, V, E / V, kWarps, kWide>::kTurn, kDepth = depth_of(kInputs, kTurn);
  constexpr auto kKernel = norm_bwd_kernel<T, V, E, kDepth, kWarps, kWide, kRms, kResidual>;
  const size_t copies = (size_t)kDepth * kInputs * kTurn, rows = sums ? (size_t)p.groups * 2 * a.width * sizeof(float) : 0;
  const size_t memory = copies > rows ? copies : rows;
  cudaError_t e = allow_ring<kKernel>();
  if (e != cudaSuccess) return e;
  const dim3 grid(parts * a.groups), block(kWarps * 32);
  if (p.cluster > 0) return launch_kernel_cluster(kKernel, grid, block, memory, (unsigned)p.cluster, s, a, p, parts);
  return launch_kernel(kKernel, grid, block, memory, s, true, a, p, parts);
}

template <typename T, int V, int E, int kWarps, bool kRms, bool kResidual>
cudaError_t norm_bwd_width(const NormBwdArgs& a, const Plan& p, int parts, bool sums, cudaStream_t s) {
  if constexpr ((E == 8 && !kRms) || (E == 16 && V >= 4))  // (wider pieces come with wide rows only, and 8 columns with rms)
    if (p.row_warps == 1) return norm_bwd_start<T, V, E, kWarps, false, kRms, kResidual>(a, p, parts, sums, s);
  if (!wide_plan(p)) return cudaErrorInvalidConfiguration;
  return norm_bwd_start<T, V, E, kWarps, true, kRms, kResidual>(a, p, parts, sums, s);
}

template <typename T, int V, int E, int kWarps, bool kRms>
cudaError_t norm_bwd_run(const NormBwdArgs& a, int num_sms, cudaStream_t s) {
  int parts = norm_bwd_parts(a.groups, a.seq, num_sms);
  const bool sums = a.dweight != nullptr || a.dbias != nullptr;
  bool second = sums;
  if (parts > 0) {
    Plan p = make_plan(a.width, E, kWarps);
    const long long strides[4] = {a.x_stride, a.dy_stride, a.residual_stride, a.dx_stride};
    for (int i = 0; i < 4; ++i) p.step[i] = p.apart * strides[i] * (long long)sizeof(T);
    const int need = (a.seq - 1) / p.apart + 1;
    parts = need < parts ? need : parts;
    if (sums && need <= kCluster * kClusterTurns && a.groups * kCluster <= num_sms) {
      p.cluster = 1;
      while (p.cluster < kCluster && p.cluster < need) p.cluster *= 2;  // (a CTA may be left without rows)
      parts = p.cluster;
      second = false;
    }
    cudaError_t e = cudaErrorInvalidConfiguration;
    if (a.residual != nullptr) e = norm_bwd_width<T, V, E, kWarps, kRms, true>(a, p, parts, sums, s);
    else if constexpr (!(kRms && E == 8))  // (rms has 8 columns a lane with a residual only)
      e = norm_bwd_width<T, V, E, kWarps, kRms, false>(a, p, parts, sums, s);
    if (e != cudaSuccess) return e;
  }
  if (!second) return cudaSuccess;
  const int blocks = ((a.dweight == a.dbias ? 1 : 2) * a.width + 31) / 32;
  return launch_kernel(norm_sum_kernel, dim3(blocks * a.groups), dim3(kSumWarps * 32), 0, s, true, (const float*)a.partial, parts, a.width,
                       a.dweight, a.dbias, a.sum_gstride, blocks);
}

// Columns of a lane and warps of a CTA: 16 with 16, so that few warps meet for a row (40 M elements, us; layer norm with a
// residual: width 2560 55 against 72 for 8 with 16, 4096 56 / 62; rms without: 2560 43 against 49 for 8 with 24, 4096 44 / 55).
// rms: 8 with 24 where 16 would leave a quarter of the warps without a row and there is a residual's memory traffic to hide it
// (width 2816 60 / 64, 3072 55 / 57; without a residual 53 / 51, 47 / 45).  Odd rows of 16 bits: 8 up to three warps of them (16 M: width 515
// 47 / 49, with a residual 56 / 65), then 16 (769 37 / 44, 1283 36 / 45, with one 43 / 53); of fp32: 8 up to
// 4096 columns, whose copies leave room for a row or two on the way.  32 where these do not hold a row.
template <typename T, int V, bool kRms>
cudaError_t norm_bwd_any(const NormBwdArgs& a, int num_sms, cudaStream_t s) {
  if constexpr (kRms) {
    if (a.residual != nullptr && a.width > 5 * 32 * 16 && a.width <= 6 * 32 * 16)
      return norm_bwd_run<T, V, 8, 24, true>(a, num_sms, s);
    return norm_bwd_run<T, V, 16, 16, true>(a, num_sms, s);
  } else {
    if (a.width > 16 * 32 * 16) return norm_bwd_run<T, V, 32, 16, false>(a, num_sms, s);
    if constexpr (V < 4)
      if (a.width <= (V == 2 ? 3 : 16) * 32 * 8) return norm_bwd_run<T, V, 8, 16, false>(a, num_sms, s);
    return norm_bwd_run<T, V, 16, 16, false>(a, num_sms, s);
  }
}

template <typename T, int V>
cudaError_t norm_bwd_type(const NormBwdArgs& a, int num_sms, cudaStream_t s) {
  const long long size = sizeof(T);
  if (a.width % V == 0 && on16(a.x, a.x_stride * size) && on16(a.dy, a.dy_stride * size) && on16(a.dx, a.dx_stride * size) &&
      on16(a.residual, a.residual_stride * size))
    return norm_bwd_any<T, V, false>(a, num_sms, s);
  return norm_bwd_any<T, sizeof(T) == 4 ? 1 : 2, false>(a, num_sms, s);
}

}  // namespace

size_t norm_bwd_workspace(int groups, int seq, int width, int num_sms) {
  return (size_t)groups * norm_bwd_parts(groups, seq, num_sms) * 2 * width * sizeof(float);
}

cudaError_t norm_bwd_launch(const NormBwdArgs& given, int num_sms, cudaStream_t s) {
  NormBwdArgs a = given;
  a.param_vec = on16(a.weight, a.weight_gstride * (a.param_dtype == MI_F32 ? 4 : 2));
  if (a.rms) return norm_bwd_any<__nv_bfloat16, 8, true>(a, num_sms, s);
  if (a.dtype == MI_F32) return norm_bwd_type<float, 4>(a, num_sms, s);
  if (a.dtype == MI_F16) return norm_bwd_type<__half, 8>(a, num_sms, s);
  return norm_bwd_type<__nv_bfloat16, 8>(a, num_sms, s);
}

}  // namespace mi
