// Layer norm, its gradient, and the gradient of the modulated RMSNorm.
//
// All three need sums over a row before they can write it, and are bound by HBM (forward 2 values an element, backward 3, or
// 4 with a residual gradient).  They share one scheme.  A CTA per SM takes a contiguous part of the rows.  Groups of warps
// share a row (or a warp takes several short rows), a lane with the same E columns of every row, whose weights and, backward,
// sums over rows stay in its registers.  Every lane copies the elements that it will need asynchronously into shared memory
// of its own, some rows ahead, so the reads stream whatever the sums wait for, and nobody waits for another lane's copy;
// a group meets once a row, for the sums.
//
// Rows may begin anywhere.  Where every tensor's rows are on 16-byte boundaries a lane moves vectors of V elements = 16 bytes.
// Otherwise fp32 rows go element by element (V = 1) and 16-bit rows in pairs of columns (V = 2): a pair in a row that begins
// in the middle of a 4-byte word is put together from the two words that hold it.
//
// Sums are fp32 in a fixed order: a lane's columns, a butterfly over the warp, the row's warps; over rows a lane's
// rows, the CTA's lanes of the same columns, the CTAs.  Results repeat bit for bit.
//
#include <cuda_fp16.h>

#include <type_traits>

#include "../../include/mi_block.h"
#include "mi_internal.h"
#include "ptx.cuh"

namespace mi {

namespace {

constexpr int kRingBytes = 200 * 1024;   // of the 227 KB of shared memory that a CTA may have
constexpr float kMax = 3.402823466e38f;

// ------------------------------------------------------------------------------- element types
// One or two values in fp32: the kernels' arithmetic is written once for both.
__device__ __forceinline__ float v_add(float a, float b) { return a + b; }
__device__ __forceinline__ float v_mul(float a, float b) { return a * b; }
__device__ __forceinline__ float v_fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float v_sum(float a) { return a; }
__device__ __forceinline__ f32x2_t v_add(f32x2_t a, f32x2_t b) { return f2_add(a, b); }
__device__ __forceinline__ f32x2_t v_mul(f32x2_t a, f32x2_t b) { return f2_mul(a, b); }
__device__ __forceinline__ f32x2_t v_fma(f32x2_t a, f32x2_t b, f32x2_t c) { return f2_fma(a, b, c); }
__device__ __forceinline__ float v_sum(f32x2_t a) {
  float lo, hi;
  f2_unpack(a, lo, hi);
  return lo + hi;
}
__device__ __forceinline__ bool v_any(float a) { return a != 0.0f; }
__device__ __forceinline__ bool v_any(f32x2_t a) { return (a & 0x7fffffff7fffffffull) != 0; }
template <typename L> __device__ __forceinline__ L v_of(float a);
template <> __device__ __forceinline__ float v_of<float>(float a) { return a; }
template <> __device__ __forceinline__ f32x2_t v_of<f32x2_t>(float a) { return f2_of(a); }

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// Two 16-bit values in a word as fp32, and back (rounded once).
template <typename T> __device__ __forceinline__ f32x2_t unpack2(uint32_t w) {
  if constexpr (std::is_same<T, __half>::value) {
    const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w));
    return f2_pack(t.x, t.y);
  } else {
    return f2_pack(bf16_lo(w), bf16_hi(w));
  }
}
template <typename T> __device__ __forceinline__ uint32_t pack2(f32x2_t v) {
  float lo, hi;
  f2_unpack(v, lo, hi);
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return pack_bf16x2(lo, hi);
  }
}

// Copies the first `bytes` of kBytes and fills up with zeros (0: nothing is read).
template <int kBytes> __device__ __forceinline__ void copy_async(uint32_t dst, const uint8_t* src, uint32_t bytes) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }

__device__ __forceinline__ uint4 load_shared16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// A lane's V columns of a row: kSlot bytes of shared memory, N numbers of type L in fp32.
//   copy   asks for the elements at `src`; `bytes` of them are in the row (the others read as zeros)
//   load   gives them; `src`: the low bits of copy's
//   store  writes them to `dst`, where `bytes` (not 0) of them are in the row
template <typename T, int V> struct Piece;
template <> struct Piece<float, 1> {
  using L = float;
  static constexpr int N = 1, kSlot = 4;
  __device__ __forceinline__ static void copy(uint32_t slot, const uint8_t* src, uint32_t bytes) { copy_async<4>(slot, src, bytes); }
  __device__ __forceinline__ static void load(uint32_t slot, uint32_t, L (&f)[1]) {
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f[0]) : "r"(slot) : "memory");
  }
  __device__ __forceinline__ static void store(uint8_t* dst, uint32_t, const L (&f)[1]) { *reinterpret_cast<float*>(dst) = f[0]; }
};
template <> struct Piece<float, 4> {
  using L = f32x2_t;
  static constexpr int N = 2, kSlot = 16;
  __device__ __forceinline__ static void copy(uint32_t slot, const uint8_t* src, uint32_t bytes) { copy_async<16>(slot, src, bytes); }
  __device__ __forceinline__ static void load(uint32_t slot, uint32_t, L (&f)[2]) {
    const uint4 v = load_shared16(slot);
    f[0] = f2_pack(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = f2_pack(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  __device__ __forceinline__ static void store(uint8_t* dst, uint32_t, const L (&f)[2]) {
    float4 v;
    f2_unpack(f[0], v.x, v.y);
    f2_unpack(f[1], v.z, v.w);
    *reinterpret_cast<float4*>(dst) = v;
  }
};
template <typename T> struct Piece<T, 8> {
  using L = f32x2_t;
  static constexpr int N = 4, kSlot = 16;
  __device__ __forceinline__ static void copy(uint32_t slot, const uint8_t* src, uint32_t bytes) { copy_async<16>(slot, src, bytes); }
  __device__ __forceinline__ static void load(uint32_t slot, uint32_t, L (&f)[4]) {
    const uint4 v = load_shared16(slot);
    f[0] = unpack2<T>(v.x);
    f[1] = unpack2<T>(v.y);
    f[2] = unpack2<T>(v.z);
    f[3] = unpack2<T>(v.w);
  }
  __device__ __forceinline__ static void store(uint8_t* dst, uint32_t, const L (&f)[4]) {
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack2<T>(f[0]), pack2<T>(f[1]), pack2<T>(f[2]), pack2<T>(f[3]));
  }
};
template <typename T> struct Piece<T, 2> {
  using L = f32x2_t;
  static constexpr int N = 1, kSlot = 8;
  // The word that holds the first element, and where that is its upper half the next word, too.
  __device__ __forceinline__ static void copy(uint32_t slot, const uint8_t* src, uint32_t bytes) {
    const uint32_t off = (uint32_t)reinterpret_cast<uintptr_t>(src) & 2u;
    const uint8_t* word = src - off;
    copy_async<4>(slot, word, off == 0 || bytes == 0 ? bytes : 4u);
    copy_async<4>(slot + 4, word + (bytes == 0 ? 0 : 4), off != 0 && bytes == 4 ? 2u : 0u);
  }
  // The same where the tensor begins with that upper half: the element is copied alone.
  __device__ __forceinline__ static void copy_first(uint32_t slot, const uint8_t* src, uint32_t bytes) {
    const uint32_t v = *reinterpret_cast<const uint16_t*>(src);
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(slot), "r"(v << 16) : "memory");
    copy_async<4>(slot + 4, src + (bytes == 4 ? 2 : -2), bytes == 4 ? 2u : 0u);
  }
  __device__ __forceinline__ static void load(uint32_t slot, uint32_t src, L (&f)[1]) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(slot) : "memory");
    f[0] = unpack2<T>(__funnelshift_r(v.x, v.y, (src & 2u) * 8));
  }
  __device__ __forceinline__ static void store(uint8_t* dst, uint32_t bytes, const L (&f)[1]) {
    const uint32_t w = pack2<T>(f[0]);
    if ((reinterpret_cast<uintptr_t>(dst) & 2u) == 0 && bytes == 4) {
      *reinterpret_cast<uint32_t*>(dst) = w;
    } else {
      *reinterpret_cast<uint16_t*>(dst) = (uint16_t)w;
      if (bytes == 4) *reinterpret_cast<uint16_t*>(dst + 2) = (uint16_t)(w >> 16);
    }
  }
};

template <typename L> __device__ __forceinline__ L v_of2(float a, float b) {
  if constexpr (sizeof(L) == 8) return f2_pack(a, b);
  else return a;
}

// Entry i of a parameter of the given type; p null: `none`.
__device__ __forceinline__ float param_at(const void* p, int dtype, long long i, float none) {
  if (p == nullptr) return none;
  if (dtype == MI_F32) return static_cast<const float*>(p)[i];
  if (dtype == MI_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// A lane's V columns from col on of a parameter, `plus` added (zeros past the width).  T: the rows' type, which the
// parameter has unless it is fp32; aligned: the parameter is on a 16-byte boundary.
template <typename T, int V>
__device__ __forceinline__ void load_param(const void* p, int dtype, bool aligned, long long at, int col, int width, float none,
                                           float plus, typename Piece<T, V>::L (&w)[Piece<T, V>::N]) {
  using P = Piece<T, V>;
  using L = typename P::L;
  if constexpr (V >= 4) if (p != nullptr && aligned && col < width) {
    if (sizeof(T) == 4 || dtype == MI_F32) {
      const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at + col);
#pragma unroll
      for (int i = 0; i < P::N; i += 2) {
        const float4 v = f[i / 2];
        w[i] = v_of2<L>(v.x, v.y);
        w[i + 1] = v_of2<L>(v.z, v.w);
      }
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const T*>(p) + at + col);
      const uint32_t f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < P::N; ++i) w[i] = unpack2<T>(f[i % 4]);
    }
#pragma unroll
    for (int i = 0; i < P::N; ++i) w[i] = v_add(w[i], v_of<L>(plus));
    return;
  }
  float f[V];
#pragma unroll
  for (int e = 0; e < V; ++e) f[e] = col + e < width ? param_at(p, dtype, at + col + e, none) + plus : 0.0f;
#pragma unroll
  for (int i = 0; i < P::N; ++i) w[i] = V == 1 ? v_of<L>(f[0]) : v_of2<L>(f[(2 * i) % V], f[(2 * i + 1) % V]);
}

// ---------------------------------------------------------------------------------------------- rows
// How a launch spreads rows over lanes.
struct Plan {
  int pieces;                  // of V columns in a row (the last may be part of one: V = 2)
  int row_warps;               // warps that share a row
  int row_lanes;               // lanes of a row in a warp: 32, or fewer (a power of two) with several rows a warp
  int batch;                   // rows that a group takes at a time: 32 / row_lanes
  int groups;                  // of a CTA
  int apart;                   // rows between a group's batches
  long long step[4];           // and bytes: of x, dy, the residual; of the output
};

// This thread's place: which rows of the CTA it takes, and which columns.
struct Place {
  int group, row_warp, sub, pos, row_threads;
  __device__ __forceinline__ explicit Place(const Plan& p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    group = warp / p.row_warps;
    row_warp = warp - group * p.row_warps;
    row_threads = p.row_warps > 1 ? p.row_warps * 32 : p.row_lanes;
    sub = p.row_warps > 1 ? 0 : lane / p.row_lanes;
    pos = p.row_warps > 1 ? row_warp * 32 + lane : lane - sub * p.row_lanes;
  }
};

// One input's rows, as a thread reads them: it asks for its pieces of rows kDepth - 1 turns before it loads them.
template <typename T, int V, int C, int kDepth, int kThreads>
struct Reader {
  using P = Piece<T, V>;
  static constexpr int kPieces = C * kThreads * P::kSlot;  // shared memory of an input's turn
  const uint8_t* next;  // the thread's first piece in the row to be asked for next

  __device__ __forceinline__ Reader(const void* tensor, long long stride, long long row, const Place& at)
      : next(static_cast<const uint8_t*>(tensor) + (row * stride + at.pos * V) * (long long)sizeof(T)) {}
  // to: the thread's place in the turn's shared memory.  Without a row or a column nothing is read, and zeros come.
  __device__ __forceinline__ void ask(const void* tensor, uint32_t to, int chunk, const uint32_t (&bytes)[C], bool has, long long step) {
    const uint8_t* src = has ? next : static_cast<const uint8_t*>(tensor);
    const bool first = V == 2 && src == tensor && has && (reinterpret_cast<uintptr_t>(src) & 2u) != 0;
    if constexpr (V == 2)
      if (first) P::copy_first(to, src, bytes[0]);
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (c > 0 || !first)
        P::copy(to + c * kThreads * P::kSlot, bytes[c] == 0 ? src : src + c * chunk, has ? bytes[c] : 0u);
    next += step;
  }
  __device__ __forceinline__ void load(uint32_t from, int chunk, int c, long long step, typename P::L (&f)[P::N]) const {
    const uint32_t src = (uint32_t)reinterpret_cast<uintptr_t>(next) - kDepth * (uint32_t)step;  // (where the row came from)
    P::load(from + c * kThreads * P::kSlot, src + c * chunk, f);
  }
};

__device__ __forceinline__ void group_sync(int group, int warps) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(warps * 32) : "memory");
}

// Whether any thread of the group has p.
__device__ __forceinline__ bool group_any(bool p, int group, int warps) {
  int r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.or.pred q, %2, %3, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
               : "=r"(r) : "r"((int)p), "r"(group + 1), "r"(warps * 32) : "memory");
  return r != 0;
}

// Sum over the `lanes` lanes of a row (without a branch: one costs as much as a shuffle here).
__device__ __forceinline__ float lanes_sum(float v, int lanes) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v += o < lanes ? u : 0.0f;
  }
  return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums over the warps of a row, at most 16, of two values: lane i < 16 holds warp i's first one, lane 16 + i its second (zeros
// where there is no warp).  All lanes get both.
__device__ __forceinline__ float2 warps_sum2(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const float u = __shfl_xor_sync(0xffffffffu, v, 16);
  return (threadIdx.x & 16) != 0 ? make_float2(u, v) : make_float2(v, u);
}

// ------------------------------------------------------------------------------------------ forward
// A row's sum of squares is taken around its mean, so a row far from zero loses nothing: a warp with n columns finds their
// mean m and the squares q around it.  Over the warps of a row, A = sum n (m - m_0) and B = sum (q + n (m - m_0)^2) give the
// row's mean m_0 + A / width and its squares B - A^2 / width.  (What that difference takes off is at most as many times what is
// left as there are warps, 16: the row's squares are at least n_0 (m_0 - mean)^2, its first warp's.)
template <typename T, int V, int E, int kDepth, int kWarps>
__global__ void __launch_bounds__(kWarps * 32, 1) layer_norm_kernel(const LayerNormArgs a, const Plan p) {
  using P = Piece<T, V>;
  using L = typename P::L;
  constexpr int C = E / V, N = P::N, kThreads = kWarps * 32;
  using In = Reader<T, V, C, kDepth, kThreads>;
  constexpr int kStage = In::kPieces;
  extern __shared__ __align__(128) uint8_t memory[];
  __shared__ float2 parts[2][kWarps + 16];  // a warp's mean and squares (read 16 from a group's first on)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Place me(p);
  const bool wide = p.row_warps > 1;
  grid_dep_wait();
  const long long row0 = (long long)a.rows * blockIdx.x / gridDim.x;
  const int rows = (int)((long long)a.rows * (blockIdx.x + 1) / gridDim.x - row0);
  const int apart = p.apart, chunk = me.row_threads * V * (int)sizeof(T);
  int left = me.group < p.groups ? rows - me.group * p.batch : 0;  // rows from the group's next batch on
  long long row = row0 + me.group * p.batch + me.sub;
  uint32_t bytes[C];  // of the thread's pieces that are in the row
#pragma unroll
  for (int c = 0; c < C; ++c) bytes[c] = (uint32_t)min(max(a.width - (c * me.row_threads + me.pos) * V, 0), V) * sizeof(T);
  In x_in(a.x, a.x_stride, row, me);
  const uint32_t slot0 = smem_u32(memory) + threadIdx.x * P::kSlot;
  int to_ask = left - me.sub;  // rows of this thread
  auto ask = [&](uint32_t to) {
    x_in.ask(a.x, to, chunk, bytes, to_ask > 0, p.step[0]);
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
    for (int c = 0; c < C; ++c) n += min(max(a.width - (c * me.row_threads + w * 32) * V, 0), 32 * V);
    return (float)n;
  };
  const float inv_cols = wide ? 1.0f / fmaxf(columns_of(me.row_warp), 1.0f) : inv;
  const float n_of_lane = (lane & 15) < p.row_warps ? columns_of(lane & 15) : 0.0f;
  L w[C][N], b[C][N];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    load_param<T, V>(a.weight, a.param_dtype, a.param_vec, 0, (c * me.row_threads + me.pos) * V, a.width, 1.0f, 0.0f, w[c]);
    load_param<T, V>(a.bias, a.param_dtype, a.param_vec, 0, (c * me.row_threads + me.pos) * V, a.width, 0.0f, 0.0f, b[c]);
  }
  uint8_t* out = static_cast<uint8_t*>(a.out) + (row * a.out_stride + me.pos * V) * (long long)sizeof(T);
  const uint32_t last = slot0 + (kDepth - 1) * kStage;
  uint32_t stage = slot0, ahead = last;
  for (int turn = 0; left > 0; turn ^= 1) {
    ask(ahead);
    copy_wait<kDepth - 1>();
    L x[C][N];
    L t = v_of<L>(0.0f);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      x_in.load(stage, chunk, c, p.step[0], x[c]);
#pragma unroll
      for (int e = 0; e < N; ++e) t = v_add(t, x[c][e]);
    }
    const float s = wide ? warp_sum(v_sum(t)) : lanes_sum(v_sum(t), p.row_lanes);
    const float m = s * inv_cols;
    t = v_of<L>(0.0f);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const L nm = bytes[c] == V * sizeof(T) ? v_of<L>(-m) : V == 2 && bytes[c] == sizeof(T) ? v_of2<L>(-m, 0.0f) : v_of<L>(0.0f);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const L d = v_add(x[c][e], nm);
        t = v_fma(d, d, t);
      }
    }
    float mean = m, square = wide ? warp_sum(v_sum(t)) : lanes_sum(v_sum(t), p.row_lanes);
    if (wide) {
      if (lane == 0) parts[turn][warp] = make_float2(m, square);
      group_sync(me.group, p.row_warps);
      const float first = parts[turn][me.group * p.row_warps].x;
      const float2 part = parts[turn][me.group * p.row_warps + (lane & 15)];
      const float d = part.x - first, nd = n_of_lane * d;
      const float v = lane < 16 ? nd : fmaf(nd, d, part.y);
      const float2 both = warps_sum2((lane & 15) < p.row_warps ? v : 0.0f);
      mean = fmaf(both.x, inv, first);
      square = fmaf(-both.x * inv, both.x, both.y);
    }
    const float rstd = rsqrtf(fmaf(square, inv, a.eps));
    const bool mine = me.sub < left;
    const L nm = v_of<L>(-mean), rs = v_of<L>(rstd);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      L o[N];
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = v_fma(v_mul(v_add(x[c][e], nm), rs), w[c][e], b[c][e]);
      if (bytes[c] != 0 && mine) P::store(out + c * chunk, bytes[c], o);
    }
    if (me.pos == 0 && mine) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    left -= apart;
    row += apart;
    out += p.step[3];
    stage = stage == last ? slot0 : stage + kStage;
    ahead = ahead == last ? slot0 : ahead + kStage;
  }
  copy_wait<0>();
}

// ----------------------------------------------------------------------------------------- backward
// With g = dy w, n = (x - mean) rstd (rms: x rstd) and the row's sums of g and g (x - mean) (rms: of x^2 and g x):
//   dx = residual + rstd (g - mean(g) - n mean(g n))   (rms: without mean(g))
//   sums over rows: dweight += dy n, dbias += dy.
// A row whose sums or statistics are not finite is looked at again: if its dy is zero it counts as absent (so what
// padding holds reaches nothing), which costs rows that are finite nothing.
template <typename T, int V, int E, int kDepth, int kWarps, bool kRms, bool kResidual>
__global__ void __launch_bounds__(kWarps * 32, 1) norm_bwd_kernel(const NormBwdArgs a, const Plan p, int n_parts) {
  using P = Piece<T, V>;
  using L = typename P::L;
  constexpr int C = E / V, N = P::N, kInputs = kResidual ? 3 : 2, kThreads = kWarps * 32;
  constexpr bool kHold = E <= 16;  // a row in registers; wider rows are read from shared memory again, their weights from L1
  using In = Reader<T, V, C, kDepth, kThreads>;
  constexpr int kStage = kInputs * In::kPieces;
  extern __shared__ __align__(128) uint8_t memory[];
  __shared__ float2 parts[2][kWarps + 16];  // a warp's sums (read 16 from a group's first on)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Place me(p);
  const bool wide = p.row_warps > 1;
  grid_dep_wait();
  const int set = blockIdx.x / n_parts, part_of_set = blockIdx.x - set * n_parts;
  const long long row0 = (long long)set * a.seq + (long long)a.seq * part_of_set / n_parts;
  const int rows = (int)((long long)set * a.seq + (long long)a.seq * (part_of_set + 1) / n_parts - row0);
  const int apart = p.apart, chunk = me.row_threads * V * (int)sizeof(T);
  int left = me.group < p.groups ? rows - me.group * p.batch : 0;  // rows from the group's next batch on
  long long row = row0 + me.group * p.batch + me.sub;
  uint32_t bytes[C];
#pragma unroll
  for (int c = 0; c < C; ++c) bytes[c] = (uint32_t)min(max(a.width - (c * me.row_threads + me.pos) * V, 0), V) * sizeof(T);
  In x_in(a.x, a.x_stride, row, me), y_in(a.dy, a.dy_stride, row, me), r_in(a.residual, a.residual_stride, row, me);
  const uint32_t slot0 = smem_u32(memory) + threadIdx.x * P::kSlot;
  int to_ask = left - me.sub;
  auto ask = [&](uint32_t to) {
    x_in.ask(a.x, to, chunk, bytes, to_ask > 0, p.step[0]);
    y_in.ask(a.dy, to + In::kPieces, chunk, bytes, to_ask > 0, p.step[1]);
    if (kResidual) r_in.ask(a.residual, to + 2 * In::kPieces, chunk, bytes, to_ask > 0, p.step[2]);
    to_ask -= apart;
    copy_commit();
  };
#pragma unroll
  for (int k = 0; k < kDepth - 1; ++k) ask(slot0 + k * kStage);
  grid_dep_launch();
  const float inv = 1.0f / (float)a.width;
  const long long w_at = set * a.weight_gstride;
  auto weights = [&](int c, L (&f)[N]) {
    load_param<T, V>(a.weight, a.param_dtype, a.param_vec, w_at, (c * me.row_threads + me.pos) * V, a.width, kRms ? 0.0f : 1.0f,
                     kRms ? 1.0f : 0.0f, f);
  };
  L w[kHold ? C : 1][N], aw[C][N], ab[C][N];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if constexpr (kHold) weights(c, w[c]);
#pragma unroll
    for (int e = 0; e < N; ++e) aw[c][e] = ab[c][e] = v_of<L>(0.0f);
  }
  uint8_t* out = static_cast<uint8_t*>(a.dx) + (row * a.dx_stride + me.pos * V) * (long long)sizeof(T);
  float next_mean = 0.0f, next_rstd = 0.0f;
  if (!kRms && me.sub < left) {
    next_mean = __ldg(a.mean + row);
    next_rstd = __ldg(a.rstd + row);
  }
  const uint32_t last = slot0 + (kDepth - 1) * kStage;
  uint32_t stage = slot0, ahead = last;
  for (int turn = 0; left > 0; turn ^= 1) {
    ask(ahead);
    float mean = next_mean, rstd = next_rstd;
    if (!kRms && me.sub < left - apart) {
      next_mean = __ldg(a.mean + row + apart);
      next_rstd = __ldg(a.rstd + row + apart);
    }
    copy_wait<kDepth - 1>();
    const bool mine = me.sub < left;
    const L m = v_of<L>(-mean);
    L x[kHold ? C : 1][N], y[kHold ? C : 1][N];  // x: less its mean
    L t1 = v_of<L>(0.0f), t2 = v_of<L>(0.0f);
    auto load = [&](int c, L (&xc)[N], L (&yc)[N]) {
      x_in.load(stage, chunk, c, p.step[0], xc);
      y_in.load(stage + In::kPieces, chunk, c, p.step[1], yc);
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
    if (wide) {
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
    bool gone = !(fabsf((c1 + c2) + (rstd + mean)) <= kMax);
    if (wide ? gone : __any_sync(0xffffffffu, gone)) {  // does the row have a gradient at all?
      bool any = false;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        L xc[N], yc[N];
        load(c, xc, yc);
#pragma unroll
        for (int e = 0; e < N; ++e) any |= v_any(yc[e]);
      }
      if (wide) {
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
        r_in.load(stage + 2 * In::kPieces, chunk, c, p.step[2], o);
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
      if (bytes[c] != 0 && mine) P::store(out + c * chunk, bytes[c], o);
    }
    left -= apart;
    row += apart;
    out += p.step[3];
    stage = stage == last ? slot0 : stage + kStage;
    ahead = ahead == last ? slot0 : ahead + kStage;
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
      const int col = (c * me.row_threads + me.pos) * V;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        if constexpr (V == 1) {
          if (col < a.width) {
            to[col] = aw[c][e];
            to[a.width + col] = ab[c][e];
          }
        } else {
          const int at = col + 2 * e;
          float lo, hi;
          f2_unpack(aw[c][e], lo, hi);
          if (at < a.width) to[at] = lo;
          if (at + 1 < a.width) to[at + 1] = hi;
          f2_unpack(ab[c][e], lo, hi);
          if (at < a.width) to[a.width + at] = lo;
          if (at + 1 < a.width) to[a.width + at + 1] = hi;
        }
      }
    }
  }
  __syncthreads();
  float* to = a.partial + (long long)blockIdx.x * 2 * a.width;
  for (int c = threadIdx.x; c < 2 * a.width; c += kThreads) {
    float t = 0.0f;
    for (int g = 0; g < p.groups; ++g) t += sums[(size_t)g * 2 * a.width + c];
    to[c] = t;
  }
}

// dweight and dbias: the sums of the CTAs' parts [set][part][2][width].  A CTA takes 32 of the 2 width columns, its 8 warps
// every 8th part each, and adds the warps up in order.  both: the two go to one row, added.
__global__ void __launch_bounds__(256) norm_sum_kernel(const float* __restrict__ partial, int parts, int width, float* dweight,
                                                       float* dbias, long long sum_gstride, int blocks) {
  __shared__ float sums[8][33];
  grid_dep_wait();
  grid_dep_launch();
  const int set = blockIdx.x / blocks, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = (blockIdx.x - set * blocks) * 32 + lane;
  const bool both = dweight == dbias;
  float t = 0.0f;
  if (c < (both ? width : 2 * width)) {
    const float* p = partial + (long long)set * parts * 2 * width + c;
#pragma unroll 4
    for (int i = warp; i < parts; i += 8) {
      t += p[(long long)i * 2 * width];
      if (both) t += p[(long long)i * 2 * width + width];
    }
  }
  sums[warp][lane] = t;
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) t += sums[i][lane];
  const long long at = set * sum_gstride;
  if (c < width) {
    if (dweight != nullptr) dweight[at + c] = t;
  } else if (c < 2 * width && dbias != nullptr && !both) {
    dbias[at + c - width] = t;
  }
}

// ----------------------------------------------------------------------------------------- launches
int norm_bwd_parts(int groups, int seq, int num_sms) {
  const int most = num_sms / groups > 0 ? num_sms / groups : 1;
  return seq < most ? seq : most;
}

bool on16(const void* p, long long stride_bytes) { return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)stride_bytes) & 15u) == 0; }

Plan make_plan(int width, int v, int e, int warps) {
  Plan p = {};
  p.pieces = (width + v - 1) / v;
  const int threads = (p.pieces + e / v - 1) / (e / v);  // of a row
  p.row_warps = (threads + 31) / 32;
  p.row_lanes = 32;
  while (p.row_warps == 1 && p.row_lanes > 4 && p.row_lanes / 2 >= threads) p.row_lanes /= 2;
  p.batch = 32 / p.row_lanes;
  p.groups = warps / p.row_warps;
  p.apart = p.groups * p.batch;
  return p;
}

// Rows that a thread has on the way: as many as the shared memory holds, up to 8.
constexpr int depth_of(int inputs, int pieces, int slot, int warps) {
  const int fit = kRingBytes / (inputs * pieces * warps * 32 * slot);
  return fit < 8 ? fit : 8;
}

template <auto kKernel>
cudaError_t allow_ring() {
  static bool done[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
  done[dev] = e == cudaSuccess;
  return e;
}

template <typename T, int V, int E, int kWarps>
cudaError_t layer_norm_run(const LayerNormArgs& a, int num_sms, cudaStream_t s) {
  constexpr int kSlot = Piece<T, V>::kSlot, kDepth = depth_of(1, E / V, kSlot, kWarps);
  constexpr auto kKernel = layer_norm_kernel<T, V, E, kDepth, kWarps>;
  Plan p = make_plan(a.width, V, E, kWarps);
  p.step[0] = p.apart * a.x_stride * (long long)sizeof(T);
  p.step[3] = p.apart * a.out_stride * (long long)sizeof(T);
  const long long need = ((long long)a.rows + p.apart - 1) / p.apart;
  const int grid = need < num_sms ? (int)need : num_sms;
  cudaError_t e = allow_ring<kKernel>();
  if (e != cudaSuccess) return e;
  return launch_kernel(kKernel, dim3(grid), dim3(kWarps * 32), (size_t)kDepth * (E / V) * kWarps * 32 * kSlot, s, true, a, p);
}

// Columns of a lane: 16 (40 M bf16 elements: 31 us at width 256, 35 at 2560, 34 at 4096; with 8 and 24 warps 34, 43, 47), but 8
// in odd rows while a CTA of 24 warps holds two of them (20 M: 49 against 50 us at width 1023, 51 against 49 at 2047), and 32
// where 16 warps of 16 columns a lane do not hold a row.
template <typename T, int V>
cudaError_t layer_norm_any(const LayerNormArgs& a, int num_sms, cudaStream_t s) {
  if (a.width > 16 * 32 * 16) return layer_norm_run<T, V, 32, 16>(a, num_sms, s);
  if constexpr (V < 4)
    if (a.width <= 12 * 32 * 8 / 2) return layer_norm_run<T, V, 8, 24>(a, num_sms, s);
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

template <typename T, int V, int E, int kWarps, bool kRms, bool kResidual>
cudaError_t norm_bwd_launch_kernel(const NormBwdArgs& a, const Plan& p, int parts, bool sums, cudaStream_t s) {
  constexpr int kSlot = Piece<T, V>::kSlot, kInputs = kResidual ? 3 : 2, kDepth = depth_of(kInputs, E / V, kSlot, kWarps);
  constexpr auto kKernel = norm_bwd_kernel<T, V, E, kDepth, kWarps, kRms, kResidual>;
  const size_t copies = (size_t)kDepth * kInputs * (E / V) * kWarps * 32 * kSlot;
  const size_t rows = sums ? (size_t)p.groups * 2 * a.width * sizeof(float) : 0;
  cudaError_t e = allow_ring<kKernel>();
  if (e != cudaSuccess) return e;
  return launch_kernel(kKernel, dim3(parts * a.groups), dim3(kWarps * 32), copies > rows ? copies : rows, s, true, a, p, parts);
}

template <typename T, int V, int E, int kWarps, bool kRms>
cudaError_t norm_bwd_run(const NormBwdArgs& a, int num_sms, cudaStream_t s) {
  int parts = norm_bwd_parts(a.groups, a.seq, num_sms);
  const bool sums = a.dweight != nullptr || a.dbias != nullptr;
  if (parts > 0) {
    Plan p = make_plan(a.width, V, E, kWarps);
    const long long strides[4] = {a.x_stride, a.dy_stride, a.residual_stride, a.dx_stride};
    for (int i = 0; i < 4; ++i) p.step[i] = p.apart * strides[i] * (long long)sizeof(T);
    const int need = (a.seq - 1) / p.apart + 1;
    parts = need < parts ? need : parts;
    cudaError_t e = a.residual != nullptr ? norm_bwd_launch_kernel<T, V, E, kWarps, kRms, true>(a, p, parts, sums, s)
                                          : norm_bwd_launch_kernel<T, V, E, kWarps, kRms, false>(a, p, parts, sums, s);
    if (e != cudaSuccess) return e;
  }
  if (!sums) return cudaSuccess;
  const int blocks = ((a.dweight == a.dbias ? 1 : 2) * a.width + 31) / 32;
  return launch_kernel(norm_sum_kernel, dim3(blocks * a.groups), dim3(256), 0, s, true, (const float*)a.partial, parts, a.width,
                       a.dweight, a.dbias, a.sum_gstride, blocks);
}

// Columns of a lane: the fewer registers a row takes, the more warps there can be.  rms: 8 with 24 warps (40 M elements with a
// residual: 59 us at width 3072, 60 at 2560; with 16 and 16 warps 67, 66).  Layer norm: 16 (61 us at 2560, 62 at 4096; with 8
// 65, 71), in odd rows 8 (20 M, no residual: 70 us at width 1023; with 16 82).  32 where these do not hold a row.
template <typename T, int V, bool kRms>
cudaError_t norm_bwd_any(const NormBwdArgs& a, int num_sms, cudaStream_t s) {
  if constexpr (kRms) return norm_bwd_run<T, V, 8, 24, true>(a, num_sms, s);  // (at most 4096 columns: 16 warps)
  if (a.width > 16 * 32 * 16) return norm_bwd_run<T, V, 32, 16, kRms>(a, num_sms, s);
  if constexpr (V < 4)
    if (a.width <= 16 * 32 * 8) return norm_bwd_run<T, V, 8, 16, kRms>(a, num_sms, s);
  return norm_bwd_run<T, V, 16, 16, kRms>(a, num_sms, s);
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

cudaError_t layer_norm_launch(const LayerNormArgs& a, int num_sms, cudaStream_t s) {
  if (a.rows <= 0) return cudaSuccess;
  if (a.dtype == MI_F32) return layer_norm_type<float, 4>(a, num_sms, s);
  if (a.dtype == MI_F16) return layer_norm_type<__half, 8>(a, num_sms, s);
  return layer_norm_type<__nv_bfloat16, 8>(a, num_sms, s);
}

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
