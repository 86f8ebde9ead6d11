// What the kernels of layer norm, its gradient and the modulated RMSNorm's gradient (layer_norm.cu, norm_bwd.cu) share.
//
// All three need sums over a row before they can write it, and are bound by HBM (forward 2 values an element, backward 3, or
// 4 with a residual gradient).  They share one scheme.  A CTA per SM takes a contiguous part of the rows.  Groups of warps
// share a row (or a warp takes several short rows), a lane with the same E columns of every row, whose weights and, backward,
// sums over rows stay in its registers.  Rows are copied asynchronously into shared memory one to four turns ahead, so the reads
// stream whatever the sums wait for.  No warp waits for another warp's copies; a group meets once a row, for the sums.  (Where a turn's
// inputs fill the shared memory nothing is ahead, and HBM idles during a row's arithmetic: backward, fp32 rows above 8192 columns,
// and with a residual odd fp32 rows above 4096 and odd 16-bit rows above 8192.  4000 x 10007 fp32 451 us, with a residual 691, of a
// floor of 72 and 96.)
//
// Where every tensor's rows are on 16-byte boundaries, a lane copies and moves vectors of V elements = 16 bytes.  Rows that
// begin anywhere are copied by the 16-byte granules that hold a warp's columns, and read word by word: single columns of fp32
// (V = 1), pairs of 16-bit columns (V = 2, put together from two words where the row begins in the middle of one).
//
// Sums are fp32 in a fixed order: a lane's columns, a butterfly over the warp, the row's warps; over rows a lane's
// rows, the CTA's lanes of the same columns, the CTAs.  Results repeat bit for bit.
//
// Measured on the way (GB300, bf16; 8260 x 2560 backward with a residual / 16418 x 4096 forward, us): one row a CTA at a
// time from L1 368 / 141; rows by bulk copies of one thread a group into a ring with barriers 51 / 64 (the one thread's copies,
// and every branch, are on the row's chain of about 1400 cycles); sums and outputs as two phases over tiles of rows, each
// with its own mapping of threads, 56 / 67 (twice the instructions); a lane's own copies 39 / 51; fewer rows on the way and
// cheaper ends 34 / 46.
#pragma once

#include "../../include/mi_block.h"
#include "mi_internal.h"
#include "ptx.cuh"
#include "values.cuh"

namespace mi {

namespace {

constexpr int kRingBytes = 200 * 1024;   // of the 227 KB of shared memory that a CTA may have

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

// Copies `bytes` of 16 and fills up with zeros (0: nothing is read).
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }

__device__ __forceinline__ uint4 load_shared16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ void store_global16(uint8_t* at, uint32_t bytes, uint4 v) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t@p st.global.v4.b32 [%0], {%1, %2, %3, %4};\n\t}" ::"l"(at), "r"(v.x),
               "r"(v.y), "r"(v.z), "r"(v.w), "r"(bytes)
               : "memory");
}

// V columns of a row: N numbers of type L in fp32.
//   load   gives them from shared memory (words: `src` is the row's address in global memory, mod 2^32)
//   store  writes those of them to `dst` that are in the row, `bytes` (by predicates: a branch would cost more)
template <typename T, int V> struct Piece;
template <> struct Piece<float, 1> {
  using L = float;
  static constexpr int N = 1;
  __device__ __forceinline__ static void load(uint32_t at, uint32_t, L (&f)[1]) {
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f[0]) : "r"(at) : "memory");
  }
  __device__ __forceinline__ static void store(uint8_t* dst, uint32_t bytes, const L (&f)[1]) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t@p st.global.f32 [%0], %1;\n\t}" ::"l"(dst), "f"(f[0]), "r"(bytes) : "memory");
  }
};
template <> struct Piece<float, 4> {
  using L = f32x2_t;
  static constexpr int N = 2;
  __device__ __forceinline__ static void load(uint32_t at, L (&f)[2]) {
    const uint4 v = load_shared16(at);
    f[0] = f2_pack(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = f2_pack(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  __device__ __forceinline__ static void store(uint8_t* dst, uint32_t bytes, const L (&f)[2]) {
    float4 v;
    f2_unpack(f[0], v.x, v.y);
    f2_unpack(f[1], v.z, v.w);
    store_global16(dst, bytes, make_uint4(__float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z), __float_as_uint(v.w)));
  }
};
template <typename T> struct Piece<T, 8> {
  using L = f32x2_t;
  static constexpr int N = 4;
  __device__ __forceinline__ static void load(uint32_t at, L (&f)[4]) {
    const uint4 v = load_shared16(at);
    f[0] = unpack2<T>(v.x);
    f[1] = unpack2<T>(v.y);
    f[2] = unpack2<T>(v.z);
    f[3] = unpack2<T>(v.w);
  }
  __device__ __forceinline__ static void store(uint8_t* dst, uint32_t bytes, const L (&f)[4]) {
    store_global16(dst, bytes, make_uint4(pack2<T>(f[0]), pack2<T>(f[1]), pack2<T>(f[2]), pack2<T>(f[3])));
  }
};
template <typename T> struct Piece<T, 2> {
  using L = f32x2_t;
  static constexpr int N = 1;
  __device__ __forceinline__ static void load(uint32_t at, uint32_t src, L (&f)[1]) {
    uint32_t lo, hi;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(lo) : "r"(at) : "memory");
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(hi) : "r"(at + 4) : "memory");
    f[0] = unpack2<T>(__funnelshift_r(lo, hi, (src & 2u) * 8));
  }
  __device__ __forceinline__ static void store(uint8_t* dst, uint32_t bytes, const L (&f)[1]) {
    const uint32_t w = pack2<T>(f[0]), halves = ((uint32_t)reinterpret_cast<uintptr_t>(dst) & 2u) | (bytes ^ 4u);  // 0: the word at once
    asm volatile(
        "{\n\t.reg .pred word, lo, hi;\n\t.reg .b16 l, h;\n\tsetp.eq.u32 word, %2, 0;\n\tsetp.ne.u32 lo, %2, 0;\n\t"
        "setp.eq.and.u32 hi, %3, 4, lo;\n\tsetp.ne.and.u32 lo, %3, 0, lo;\n\tmov.b32 {l, h}, %1;\n\t"
        "@word st.global.b32 [%0], %1;\n\t@lo st.global.b16 [%0], l;\n\t@hi st.global.b16 [%0 + 2], h;\n\t}" ::"l"(dst),
        "r"(w), "r"(halves), "r"(bytes)
        : "memory");
  }
};

template <typename L> __device__ __forceinline__ L v_of2(float a, float b) {
  if constexpr (sizeof(L) == 8) return f2_pack(a, b);
  else return a;
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
  for (int e = 0; e < V; ++e) f[e] = col + e < width ? value_at(p, dtype, at + col + e, none) + plus : 0.0f;
#pragma unroll
  for (int i = 0; i < P::N; ++i) w[i] = V == 1 ? v_of<L>(f[0]) : v_of2<L>(f[(2 * i) % V], f[(2 * i + 1) % V]);
}

// ---------------------------------------------------------------------------------------------- rows
// How a launch spreads rows over lanes.
struct Plan {
  int row_warps;               // warps that share a row
  int row_lanes;               // lanes of a row in a warp: 32, or fewer (a power of two) with several rows a warp
  int batch;                   // rows that a group takes at a time: 32 / row_lanes
  int groups;                  // of a CTA
  int apart;                   // rows between a group's batches
  int cluster;                 // CTAs of a cluster that sum rows up together (backward; 0: a second kernel does)
  long long step[4];           // and bytes: of x, dy, the residual; of the output
};

// Rows [first, first + count) of n for the i-th of `parts` CTAs, each as many or one more.
struct Share {
  int first, count;
  __device__ __forceinline__ Share(int n, int i, int parts) {
    const int each = n / parts, more = n - each * parts;
    first = i * each + min(i, more);
    count = each + (i < more);
  }
};

// This thread's place: which rows of the CTA it takes, and which columns: piece c is columns [first + c apart, + V).
// kWide: warps share a row; otherwise rows share a warp, or have one each.
template <int V, int C, bool kWide>
struct Place {
  int group, row_warp, sub, lane, first;  // lane: of the row in this warp
  int lanes;
  __device__ __forceinline__ explicit Place(const Plan& p) {
    const int warp = threadIdx.x >> 5;
    lanes = p.row_lanes;
    group = kWide ? warp / p.row_warps : warp;
    row_warp = kWide ? warp - group * p.row_warps : 0;
    sub = kWide ? 0 : (threadIdx.x & 31) / p.row_lanes;
    lane = kWide ? threadIdx.x & 31 : (threadIdx.x & 31) - sub * p.row_lanes;
    first = (row_warp * C * 32 + lane) * V;
  }
  __device__ __forceinline__ int row_lanes() const { return kWide ? 32 : lanes; }
  __device__ __forceinline__ int apart() const { return row_lanes() * V; }
  __device__ __forceinline__ int column(int c) const { return first + c * apart(); }
};

// One input's rows, as a thread reads them: it asks for its part of rows kDepth - 1 turns before it loads them.  Columns and
// rows that are not there read as zeros.
template <typename T, int V, int C, int kWarps, bool kWide, bool kVectors = (V >= 4)>
struct Reader;

// Vectors: a lane copies its own pieces.
template <typename T, int V, int C, int kWarps, bool kWide>
struct Reader<T, V, C, kWarps, kWide, true> {
  using P = Piece<T, V>;
  using At = Place<V, C, kWide>;
  static constexpr int kTurn = C * kWarps * 32 * 16;  // shared memory of an input's turn
  const uint8_t* next;  // this thread's first piece in the row to be asked for next

  __device__ __forceinline__ Reader(const void* tensor, long long stride, long long row, int, const At& me)
      : next(static_cast<const uint8_t*>(tensor) + (row * stride + me.first) * (long long)sizeof(T)) {}
  __device__ __forceinline__ static uint32_t place(uint32_t memory, const At&) { return memory + threadIdx.x * 16; }
  // to: the turn's shared memory, this thread's place in it; has: there is such a row; more: and another one after it.
  __device__ __forceinline__ void ask(const void* tensor, uint32_t to, const At& me, const uint32_t (&bytes)[C], bool has, bool more,
                                      long long step) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t n = has ? bytes[c] : 0u;  // (0: the address is not read)
      copy_async(to + c * kWarps * 32 * 16, next + (c > 0 && bytes[c] == 0 ? 0 : c * me.apart() * (int)sizeof(T)), n);
    }
    if (more) next += step;
  }
  __device__ __forceinline__ void load(uint32_t from, const At&, int c, typename P::L (&f)[P::N]) const {
    P::load(from + c * kWarps * 32 * 16, f);
  }
  __device__ __forceinline__ void advance(long long) {}
};

// Words: the lanes of a row copy the granules of their C row_lanes columns or pairs of columns (and one more: they may begin in
// the middle of a granule); a lane reads other lanes' copies, so a warp meets (__syncwarp) between copies and reads.
template <typename T, int V, int C, int kWarps, bool kWide>
struct Reader<T, V, C, kWarps, kWide, false> {
  using P = Piece<T, V>;
  using At = Place<V, C, kWide>;
  static constexpr int kWarp = (8 * C + 8) * 16;  // a warp's: C / 4 granules a lane, and one more for each of up to 8 rows
  static constexpr int kTurn = kWarps * kWarp;
  const uint8_t* next;  // the warp's first column in the row to be asked for next
  uint32_t src;         // the same of the row to be loaded next, mod 2^32
  int left;             // bytes of a row from there on

  __device__ __forceinline__ Reader(const void* tensor, long long stride, long long row, int width, const At& me) {
    const int first = me.row_warp * C * 32 * V;
    next = static_cast<const uint8_t*>(tensor) + (row * stride + first) * (long long)sizeof(T);
    src = (uint32_t)reinterpret_cast<uintptr_t>(next);
    left = max(width - first, 0) * (int)sizeof(T);
  }
  __device__ __forceinline__ static uint32_t place(uint32_t memory, const At& me) {
    return memory + (threadIdx.x >> 5) * kWarp + me.sub * (me.row_lanes() * (C / 4) + 1) * 16;
  }
  __device__ __forceinline__ void ask(const void* tensor, uint32_t to, const At& me, const uint32_t (&)[C], bool has, bool more,
                                      long long step) {
    const int lead = (int)(reinterpret_cast<uintptr_t>(next) & 15u), n = has ? left + lead : 0;
    const uint8_t* start = next - lead;
    const bool front = has && start < tensor;  // the tensor's first row begins in the middle of a granule
#pragma unroll
    for (int k = 0; k <= C / 4; ++k) {
      const int g = k < C / 4 ? k * me.row_lanes() + me.lane : C / 4 * me.row_lanes();
      const int size = min(max(n - 16 * g, 0), 16);
      if ((k < C / 4 || me.lane == 0) && !(front && g == 0)) copy_async(to + 16 * g, start + (size > 0 ? 16 * g : 0), (uint32_t)size);
    }
    if (front && me.lane == 0) first_granule(tensor, to, start, n);
    if (more) next += step;
  }
  // Its elements of the row one by one, and zeros.
  __device__ __noinline__ static void first_granule(const void* tensor, uint32_t to, const uint8_t* start, int n) {
    for (int i = 0; i < 16; i += (int)sizeof(T)) {
      const bool in = start + i >= tensor && i < n;
      if constexpr (sizeof(T) == 4) {
        const uint32_t v = in ? *reinterpret_cast<const uint32_t*>(start + i) : 0u;
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + i), "r"(v) : "memory");
      } else {
        const uint16_t v = in ? *reinterpret_cast<const uint16_t*>(start + i) : (uint16_t)0;
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + i), "h"(v) : "memory");
      }
    }
  }
  __device__ __forceinline__ void load(uint32_t from, const At& me, int c, typename P::L (&f)[P::N]) const {
    P::load(from + (src & 12u) + (c * me.row_lanes() + me.lane) * 4, src, f);
  }
  __device__ __forceinline__ void advance(long long step) { src += (uint32_t)step; }
};

// The groups of a kernel with kWide meet at barriers 1 to groups, of 16 that there are: rows of one warp, which need none, have
// kernels without it.
constexpr int kBarriers = 16;

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

// ---------------------------------------------------------------------------------------------- host
inline bool on16(const void* p, long long stride_bytes) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)stride_bytes) & 15u) == 0;
}

// A row of `width` over lanes of e columns.
inline Plan make_plan(int width, int e, int warps) {
  Plan p = {};
  const int threads = (width + e - 1) / e;  // of a row
  p.row_warps = (threads + 31) / 32;
  p.row_lanes = 32;
  while (p.row_warps == 1 && p.row_lanes > 4 && p.row_lanes / 2 >= threads) p.row_lanes /= 2;
  p.batch = 32 / p.row_lanes;
  p.groups = warps / p.row_warps;
  p.apart = p.groups * p.batch;
  return p;
}

// Whether a kernel with kWide can run the plan.
inline bool wide_plan(const Plan& p) { return p.row_warps > 1 && p.row_warps <= 16 && p.groups > 0 && p.groups < kBarriers; }

// Turns in shared memory: as many as keep 48 KB on the way per SM.  What all SMs ask for at the start comes in any order, so
// more makes the first rows late and gains nothing later (us with 32, 48, 64, 96, 128 KB: 4130 x 2560 forward 12.1, 12.4, 12.6, 13.5,
// 14.0; 16418 x 4096 50.9, 51.5, 51.6, 52.8, 53.0; 3 x 10571 x 1792 rms backward, then with 8 columns a lane,
// 65.3, 65.2, 63.9, 64.7, 66.5).
constexpr int kFlight = 48 * 1024;
constexpr int depth_of(int inputs, int turn) {
  const int want = 1 + (kFlight + inputs * turn - 1) / (inputs * turn), fit = kRingBytes / (inputs * turn);
  return want < fit ? want : fit;
}

// Lets a kernel have that much shared memory, once a device.
template <auto kKernel>
cudaError_t allow_ring() {
  static bool done[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
  done[dev] = e == cudaSuccess;
  return e;
}

}  // namespace

}  // namespace mi
