// The norms on both sides of a block, with its gate and its residual:
//
//   n = y s_y v,  s_y = 1 / sqrt(mean(y^2) + eps)   (v the norm's weight after
//                                                    the block; without it n = y)
//   r = a x + b g n       (y the block's output, g its gate; without y, r = x)
//   h = r s_r w,  s_r = 1 / sqrt(mean(r^2) + eps)   (w the next block's norm's weight)
//
// and the gradients for upstream dr and dh:
//   t = dh w,  d = dr + s_r (t - r s_r mean(t r s_r)),  dw = sum_rows dh r s_r
//   dx = a d,  dg = sum_rows b d n,  q = b d g,  dv = sum_rows q y s_y
//   dy = s_y (q v - y s_y mean(q v y s_y))           (without v: dy = q)
//
// Every sum is in fp32 and every output is rounded once: h comes from the r
// that is not rounded yet, and the backward computes r again from x and y
// instead of reading the rounded one (the same bytes).
//
// The bytes bound both directions.  A row belongs to a row group of H / 8
// threads (whole warps; the backward's of H / 16), so that a row's quantities
// stay in registers between its sums; a block holds several row groups and is
// alone on its SM.  Each row group takes a range of consecutive rows and has a
// ring in shared memory that bulk copies keep full: the loads in flight do not
// depend on the registers, nor on the barriers of a row's sums.
// Consecutive rows keep the columns' sums of the backward in registers until
// the range ends, and a gate's group ends at most twice inside a range.
//
// Measured: 16384 x 7168 in bf16 with a gate for each 1024 rows 148 us forward
// (940 MB, 6.4 TB/s) and 195 backward with the sums (1.4 GB, 7.2 TB/s).  With
// both norms a row has two sums to wait for, and its bytes take less time than
// they do: 8191 x 2048, fp32 stream, 40 us forward (5.0 TB/s), 68 backward
// (4.5); instructions issue half of the time.
#include <algorithm>

#include "kernels.h"

namespace moe {

namespace {

constexpr int kNormMaxH = 8192;
constexpr int kNormBlocks = 152;        // GB300's SMs; fixed, as the order of the columns' sums goes by it
constexpr int kNormThreads = 1024;
constexpr int kNormSmem = 216 * 1024;   // of a block: the rings and the operands that rows share
constexpr int kNormMaxStages = 4;

// Eight columns of a thread (Columns), as four pairs for the packed fp32 instructions
// (two products, sums or fused ones an instruction, each rounded as alone).
struct F8 {
  float2 v[4];
};
__device__ __forceinline__ uint64_t bits(const float2& a) { return reinterpret_cast<const uint64_t&>(a); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
  return reinterpret_cast<float2&>(d);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return reinterpret_cast<float2&>(d);
}
__device__ __forceinline__ F8 fill8(float c) {
  F8 r;
#pragma unroll
  for (int k = 0; k < 4; ++k) r.v[k] = make_float2(c, c);
  return r;
}
__device__ __forceinline__ void mul8(F8& a, const F8& b) {
#pragma unroll
  for (int k = 0; k < 4; ++k) a.v[k] = mul2(a.v[k], b.v[k]);
}
__device__ __forceinline__ void mul8(F8& a, float b) { mul8(a, fill8(b)); }
// a b + c into c
__device__ __forceinline__ void fma8(const F8& a, const F8& b, F8& c) {
#pragma unroll
  for (int k = 0; k < 4; ++k) c.v[k] = fma2(a.v[k], b.v[k], c.v[k]);
}
__device__ __forceinline__ float dot8(const F8& a, const F8& b) {
  float2 s = mul2(a.v[0], b.v[0]);
#pragma unroll
  for (int k = 1; k < 4; ++k) s = fma2(a.v[k], b.v[k], s);
  return s.x + s.y;
}

// A warp has 256 consecutive columns, and a lane four of either half of them:
// 16-byte accesses of fp32 then lie side by side, in shared memory without
// bank conflicts and in global memory in whole sectors.
struct Columns {
  int a, b;          // the first of either four
  bool in_a, in_b;   // within the row
  __device__ __forceinline__ Columns() {}
  __device__ __forceinline__ Columns(int warp, int H) {
    a = 256 * warp + 4 * (threadIdx.x & 31);
    b = a + 128;
    in_a = a < H;
    in_b = b < H;
  }
};

__device__ __forceinline__ void load4(const float* p, float2* v) {
  const float4 q = *reinterpret_cast<const float4*>(p);
  v[0] = make_float2(q.x, q.y);
  v[1] = make_float2(q.z, q.w);
}
__device__ __forceinline__ void load4(const uint16_t* p, float2* v) {
  const uint2 q = *reinterpret_cast<const uint2*>(p);
  v[0] = make_float2(bf16_lo(q.x), bf16_hi(q.x));
  v[1] = make_float2(bf16_lo(q.y), bf16_hi(q.y));
}
__device__ __forceinline__ void store4(float* p, const float2* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
}
__device__ __forceinline__ void store4(uint16_t* p, const float2* v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y));
}
// A thread's columns of a row, zeros beyond it.
template <typename T>
__device__ __forceinline__ F8 load8(const T* row, const Columns& c) {
  F8 r = fill8(0.f);
  if (c.in_a) load4(row + c.a, r.v);
  if (c.in_b) load4(row + c.b, r.v + 2);
  return r;
}
template <typename T>
__device__ __forceinline__ void store8(T* row, const Columns& c, const F8& v) {
  if (c.in_a) store4(row + c.a, v.v);
  if (c.in_b) store4(row + c.b, v.v + 2);
}

// Vectors that rows share, fp32 or bf16.
struct Shared {
  const void* p;
  bool f32;
  __device__ __forceinline__ F8 load(int64_t at, const Columns& c) const {
    return f32 ? load8(static_cast<const float*>(p) + at, c) : load8(static_cast<const uint16_t*>(p) + at, c);
  }
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}

enum { kInGlobal, kAsGiven, kAsFp32 };   // the last two in shared memory

struct NormParams {
  const void* x;
  const uint16_t* y;
  const void *w, *v, *g;
  void* r;
  uint16_t* h;
  float* stats;           // [2, T]: s_r, s_y
  const uint16_t* dh;     // backward
  const void* dr;
  void* dx;
  uint16_t* dy;
  float* parts;           // [grid][sums][H], then [row groups][2][H] of the gate's groups
  void* dg;               // finished groups are written here
  void *dw, *dv;          // written by a launch of one block, as its only group's dg
  int64_t T;
  int H;
  int64_t gate_rows;      // rows of a gate's group
  int64_t groups;
  float a, b, eps;
  int w_f32, v_f32, g_f32;
  int n_sums;             // columns' sums over all rows: dw, dv, dg with one group
  int stages;
  int shared_params;      // where w, v and a single g are
  uint32_t* status;
  uint64_t wait_limit_ns;
};

// The first of row group v's rows, of n row groups.
__device__ __forceinline__ uint32_t norm_first_row(uint32_t T, uint32_t n, uint32_t v) {
  const uint32_t share = T / n, more = T - share * n;
  return v * share + min(v, more);
}
// The row group of a row.
__device__ __forceinline__ uint32_t norm_group_of(uint32_t T, uint32_t n, uint32_t row) {
  const uint32_t share = T / n, more = T - share * n;
  return row < more * (share + 1) ? row / (share + 1) : more + (row - more * (share + 1)) / share;
}

__device__ __noinline__ void norm_wait_more(uint32_t bar, uint32_t phase, volatile int* abort, uint64_t limit_ns, uint32_t* status) {
  mbar_wait_bounded(bar, phase, abort, limit_ns, status, 1, kKernNorm);
}

// A row group: its rows, its ring and its sums.
struct RowGroup {
  // the stream that this thread copies, if any: a thread of another warp for
  // each where the row group has as many, as all wait for the slowest
  const uint8_t* src;     // its first row of the range
  uint32_t bytes, offset; // of a row; in a stage
  uint8_t* ring;
  uint32_t row_bytes;     // of a stage
  uint32_t bar;
  int rows;
  float* buf;             // [2][32]: the warps' partial sums, then zeros
  int turn;
  volatile int* abort;

  __device__ __forceinline__ int warps() const { return blockDim.x >> 5; }
  __device__ __forceinline__ void sync() const {
    if (warps() == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.y), "r"((int)blockDim.x) : "memory");
  }
  // The sum over the row's threads.  Two buffers in turn: a thread writes one
  // again only after the barrier of the sum in between, which every thread
  // reaches after reading it.
  __device__ __forceinline__ float sum(float v) {
    v = warp_sum(v);
    const int n = warps();
    if (n == 1) return v;
    float* b = buf + turn * 32;
    if ((threadIdx.x & 31) == 0) b[threadIdx.x >> 5] = v;
    sync();
    turn ^= 1;
    if (n <= 8) {   // a few: in every thread, without shuffles
      const float4 q = *reinterpret_cast<const float4*>(b), r = *reinterpret_cast<const float4*>(b + 4);
      return ((q.x + q.y) + (q.z + q.w)) + ((r.x + r.y) + (r.z + r.w));
    }
    return warp_sum(b[threadIdx.x & 31]);
  }
  __device__ __forceinline__ void issue(int i, int stage) const {   // row i of the range
    if (!src) return;
    mbar_arrive_expect_tx(bar + 8 * stage, bytes);
    bulk_load(smem_u32(ring) + stage * row_bytes + offset, src + (int64_t)i * bytes, bytes, bar + 8 * stage);
  }
  // Row i has landed.  A wait that runs out is reported; the rows are then
  // undefined, and the kernel goes on to its end.
  __device__ __forceinline__ const uint8_t* wait(const NormParams& p, int stage, uint32_t phase) const {
    const uint32_t b = bar + 8 * stage;
    if (!mbar_try_wait(b, phase)) norm_wait_more(b, phase, abort, p.wait_limit_ns, p.status);
    return ring + stage * row_bytes;
  }
  // Between two barriers of row i, all of row i - 1's reads are done: its
  // stage takes the row `stages` after it.
  __device__ __forceinline__ void refill(const NormParams& p, int i, int stage) const {
    if (i > 0 && i - 1 + p.stages < rows) issue(i - 1 + p.stages, stage == 0 ? p.stages - 1 : stage - 1);
  }
};

struct NormSetup {
  RowGroup rg;
  Shared w, v, g;         // w, v and a single gate: in shared memory where they fit
};

// The block's shared memory: the row groups' rings, then w, v and a single g.
__device__ __forceinline__ NormSetup norm_setup(const NormParams& p, uint8_t* smem, const void* const (&src)[4],
                                                const int (&elem)[4], int64_t begin, int rows) {
  __shared__ uint64_t bars[32 * kNormMaxStages];
  __shared__ __align__(16) float sums[32 * 64];
  __shared__ int abort_flag;
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, ty = threadIdx.y;
  NormSetup s;
  RowGroup& g = s.rg;
  g.row_bytes = 0;
  g.src = nullptr;
  g.bytes = g.offset = 0;
  int n = 0, n_src = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) n_src += src[k] != nullptr;
  const int step = g.warps() >= n_src ? 32 : 1;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (src[k]) {
      const uint32_t bytes = (uint32_t)p.H * elem[k];
      if ((int)threadIdx.x == n * step) {
        g.src = static_cast<const uint8_t*>(src[k]) + begin * bytes;
        g.bytes = bytes;
        g.offset = g.row_bytes;
      }
      g.row_bytes += bytes;
      ++n;
    }
  g.rows = rows;
  g.bar = smem_u32(bars) + 8 * ty * p.stages;
  g.buf = sums + 64 * ty;
  g.turn = 0;
  g.abort = &abort_flag;
  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < (int)blockDim.y * p.stages; ++i) mbar_init(smem_u32(bars) + 8 * i, n_src);
    fence_mbar_init();
  }
  for (int i = tid; i < 32 * 64; i += blockDim.x * blockDim.y) sums[i] = 0.f;
  g.ring = smem + (size_t)ty * p.stages * g.row_bytes;
  uint8_t* at = smem + (size_t)blockDim.y * p.stages * g.row_bytes;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  for (int i = 0; i < p.stages && i < rows; ++i) g.issue(i, i);
  const int threads = blockDim.x * blockDim.y;
  auto share = [&](const void* from, int f32) {
    const Shared given{from, f32 != 0};
    if (!from || !p.shared_params) return given;
    uint8_t* to = at;
    if (p.shared_params == kAsFp32) {
      for (int i = tid * 4; i < p.H; i += threads * 4) {
        float2 v[2];
        if (given.f32) load4(static_cast<const float*>(from) + i, v);
        else load4(static_cast<const uint16_t*>(from) + i, v);
        store4(reinterpret_cast<float*>(to) + i, v);
      }
      at += p.H * 4;
      return Shared{to, true};
    }
    const int bytes = p.H * (f32 ? 4 : 2);
    for (int i = tid * 16; i < bytes; i += threads * 16)
      *reinterpret_cast<uint4*>(to + i) = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(from) + i));
    at += bytes;
    return Shared{to, given.f32};
  };
  s.w = share(p.w, p.w_f32);
  s.v = share(p.v, p.v_f32);
  s.g = p.groups > 1 ? Shared{p.g, p.g_f32 != 0} : share(p.g, p.g_f32);
  __syncthreads();
  return s;
}

// Where a row is among the gate's groups.
struct GatePlace {
  int group = 0, left = 0;   // its group, and the group's rows from it on
  __device__ __forceinline__ GatePlace(const NormParams& p, int64_t begin, int rows) {
    if (p.groups > 1 && rows > 0) {
      group = (int)(begin / p.gate_rows);
      left = (int)((group + 1) * p.gate_rows - begin);
    }
  }
  __device__ __forceinline__ bool ends() { return --left == 0; }
  __device__ __forceinline__ void next(const NormParams& p) {
    ++group;
    left = (int)p.gate_rows;
  }
  __device__ __forceinline__ int64_t first(const NormParams& p) const { return p.groups > 1 ? (int64_t)group * p.H : 0; }
};

// Groups of 8 columns of a thread of the forward: with two sums to wait for in
// a row of an fp32 stream, two, so that twice as many rows are under way (8191
// x 2048, both norms: 39.8 us, with one group 47.0; but of a bf16 stream 29.2,
// with one group 26.7, and with one norm 16384 x 7168 162, with one group 147).
constexpr __host__ __device__ int norm_groups(bool two_sums, bool x_f32) { return two_sums && x_f32 ? 2 : 1; }

// Y: there is a block's output (y); W, V, G: w, v, g.
template <typename X, bool Y, bool W, bool V, bool G>
__global__ void __launch_bounds__(kNormThreads, 1) block_norm_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(16) uint8_t norm_smem[];
  constexpr int N = norm_groups(V && W, sizeof(X) == 4);
  Columns c[N];
#pragma unroll
  for (int j = 0; j < N; ++j) c[j] = Columns((threadIdx.x + j * blockDim.x) >> 5, p.H);
  const uint32_t n = gridDim.x * blockDim.y, me = blockIdx.x * blockDim.y + threadIdx.y;
  const int64_t begin = norm_first_row((uint32_t)p.T, n, me);
  const int rows = (int)(norm_first_row((uint32_t)p.T, n, me + 1) - begin);
  NormSetup s = norm_setup(p, norm_smem, {p.x, p.y, nullptr, nullptr}, {(int)sizeof(X), 2, 0, 0}, begin, rows);
  RowGroup& rg = s.rg;
  const float inv = 1.f / (float)p.H;
  int stage = 0;
  uint32_t phase = 0;
  GatePlace gate(p, begin, G ? rows : 0);
  constexpr bool kKeepG = !V;   // a gate's row stays in registers
  F8 gate_row[N];
  auto next_gate = [&]() {
#pragma unroll
    for (int j = 0; j < N; ++j) gate_row[j] = s.g.load(gate.first(p), c[j]);
  };
  if (G && kKeepG && rows > 0) next_gate();
  X* out_r = static_cast<X*>(p.r) + begin * p.H;
  uint16_t* out_h = p.h + begin * p.H;
  auto squares = [](const F8 (&v)[N]) {
    float q = dot8(v[0], v[0]);
#pragma unroll
    for (int j = 1; j < N; ++j) q += dot8(v[j], v[j]);
    return q;
  };
  for (int i = 0; i < rows; ++i) {
    const uint8_t* row = rg.wait(p, stage, phase);
    F8 r[N], y[N];
    float sy = p.b;   // the factor of y, s_y among it
    if (Y) {
#pragma unroll
      for (int j = 0; j < N; ++j) y[j] = load8(reinterpret_cast<const uint16_t*>(row + p.H * sizeof(X)), c[j]);
    }
    if (V) {
      const float q = rsqrtf(rg.sum(squares(y)) * inv + p.eps);
      rg.refill(p, i, stage);
      if (p.stats && threadIdx.x == 0) p.stats[p.T + begin + i] = q;
      sy *= q;
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      r[j] = load8(reinterpret_cast<const X*>(row), c[j]);
      if (!Y) continue;
      if (V) mul8(y[j], s.v.load(0, c[j]));
      if (G) mul8(y[j], kKeepG ? gate_row[j] : s.g.load(gate.first(p), c[j]));
      mul8(r[j], p.a);
      fma8(y[j], fill8(sy), r[j]);
      store8(out_r, c[j], r[j]);
    }
    if (W) {
      const float sr = rsqrtf(rg.sum(squares(r)) * inv + p.eps);
      if (!V) rg.refill(p, i, stage);
      if (p.stats && threadIdx.x == 0) p.stats[begin + i] = sr;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        mul8(r[j], sr);
        mul8(r[j], s.w.load(0, c[j]));
        store8(out_h, c[j], r[j]);
      }
    }
    if (!V && !W) {
      rg.sync();
      rg.refill(p, i, stage);
    }
    if (G && p.groups > 1 && gate.ends()) {
      gate.next(p);
      if (kKeepG && i + 1 < rows) next_gate();
    }
    if (Y) out_r += p.H;
    if (W) out_h += p.H;
    if (++stage == p.stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
}

// A thread has two groups of 8 columns here, H / 16 threads to a row, and the
// block half the threads: the columns' sums and what is kept between a row's
// sums take up to 128 registers (with 8 columns and 64 registers the operands
// of a gate or of v spill: 135 us for 8191 x 2048 with all of them).
template <typename X, bool Y, bool W, bool V, bool G>
__global__ void __launch_bounds__(kNormThreads / 2, 1) block_norm_bwd_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(16) uint8_t norm_smem[];
  constexpr bool kKeepG = !V;   // a gate's row stays in registers
  const Columns c[2] = {Columns(threadIdx.x >> 5, p.H), Columns((threadIdx.x + blockDim.x) >> 5, p.H)};
  const uint32_t n = gridDim.x * blockDim.y, me = blockIdx.x * blockDim.y + threadIdx.y;
  const int64_t begin = norm_first_row((uint32_t)p.T, n, me);
  const int rows = (int)(norm_first_row((uint32_t)p.T, n, me + 1) - begin);
  NormSetup s = norm_setup(p, norm_smem, {p.x, p.y, p.dh, p.dr}, {(int)sizeof(X), 2, 2, (int)sizeof(X)}, begin, rows);
  RowGroup& rg = s.rg;
  const float inv = 1.f / (float)p.H;
  F8 dw[2], dv[2], dg[2], gate_row[2];
  int stage = 0;
  uint32_t phase = 0;
  GatePlace gate(p, begin, G ? rows : 0);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    dw[j] = dv[j] = dg[j] = gate_row[j] = fill8(0.f);
    if (G && kKeepG && rows > 0) gate_row[j] = s.g.load(gate.first(p), c[j]);
  }
  auto gate_of = [&](int j) { return kKeepG ? gate_row[j] : s.g.load(gate.first(p), c[j]); };
  float next_r = 0.f, next_y = 0.f;   // the next row's statistics
  auto stats = [&](int i) {
    if (i >= rows) return;
    if (W) next_r = p.stats[begin + i];
    if (V) next_y = p.stats[p.T + begin + i];
  };
  stats(0);
  X* out_x = static_cast<X*>(p.dx) + begin * p.H;
  uint16_t* out_y = p.dy + begin * p.H;
  const uint32_t at_y = p.H * sizeof(X), at_dh = at_y + (Y ? p.H * 2 : 0), at_dr = at_dh + (W ? p.H * 2 : 0);
  for (int i = 0; i < rows; ++i) {
    const float sr = next_r, sy = next_y;
    stats(i + 1);
    // Between the sums a thread keeps r and dh w alone, and reads the row's
    // other operands from shared memory again.
    const uint8_t* row = rg.wait(p, stage, phase);
    auto load_y = [&](int j) {   // normed, without v
      F8 y = load8(reinterpret_cast<const uint16_t*>(row + at_y), c[j]);
      if (V) mul8(y, sy);
      return y;
    };
    auto load_dr = [&](int j) {
      return p.dr ? load8(reinterpret_cast<const X*>(row + at_dr), c[j]) : fill8(0.f);
    };
    F8 d[2];
    if (W) {
      F8 r[2];
      float q = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {   // d: dh w
        r[j] = load8(reinterpret_cast<const X*>(row), c[j]);
        if (Y) {
          F8 y = load_y(j);
          if (V) mul8(y, s.v.load(0, c[j]));
          if (G) mul8(y, gate_of(j));
          mul8(y, p.b);
          fma8(fill8(p.a), r[j], y);
          r[j] = y;
        }
        mul8(r[j], sr);
        d[j] = load8(reinterpret_cast<const uint16_t*>(row + at_dh), c[j]);
        fma8(d[j], r[j], dw[j]);
        mul8(d[j], s.w.load(0, c[j]));
        q += dot8(d[j], r[j]);
      }
      q = rg.sum(q) * inv;
      rg.refill(p, i, stage);
#pragma unroll
      for (int j = 0; j < 2; ++j) {   // d = dr + s_r (dh w - r q)
        fma8(fill8(-q), r[j], d[j]);
        F8 o = load_dr(j);
        fma8(fill8(sr), d[j], o);
        d[j] = o;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) d[j] = load_dr(j);
    }
    float q = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      F8 o = d[j];
      mul8(o, p.a);
      store8(out_x, c[j], o);
      if (!Y) continue;
      mul8(d[j], p.b);
      if (!G && !V) continue;
      const F8 y = load_y(j);
      if (V) {
        const F8 v = s.v.load(0, c[j]);
        if (G) {
          F8 m = y;
          mul8(m, v);
          fma8(d[j], m, dg[j]);
          mul8(d[j], gate_of(j));
        }
        fma8(d[j], y, dv[j]);
        mul8(d[j], v);
        q += dot8(d[j], y);
      } else {
        fma8(d[j], y, dg[j]);
        mul8(d[j], gate_of(j));
      }
    }
    if (V) {
      q = rg.sum(q) * inv;
      if (!W) rg.refill(p, i, stage);
    }
    if (Y) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
          if (V) {
          fma8(fill8(-q), load_y(j), d[j]);
          mul8(d[j], sy);
        }
        store8(out_y, c[j], d[j]);
      }
    }
    if (!V && !W) {
      rg.sync();
      rg.refill(p, i, stage);
    }
    if (G && p.groups > 1) {
      const bool ends = gate.ends();
      if (ends || i + 1 == rows) {
        const int64_t first = gate.group * p.gate_rows, at = gate.first(p);
        gate.next(p);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
              if (ends && first >= begin) {
            if (p.g_f32) store8(static_cast<float*>(p.dg) + at, c[j], dg[j]);
            else store8(static_cast<uint16_t*>(p.dg) + at, c[j], dg[j]);
          } else {   // the range's first group, or its last
            store8(p.parts + ((int64_t)gridDim.x * p.n_sums + 2 * (int64_t)me + (first > begin)) * p.H, c[j], dg[j]);
          }
          dg[j] = fill8(0.f);
          if (kKeepG && i + 1 < rows) gate_row[j] = s.g.load(gate.first(p), c[j]);
        }
      }
    }
    out_x += p.H;
    if (Y) out_y += p.H;
    if (++stage == p.stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  // the block's sums, its row groups in order, through the rings' memory
  float* sums = reinterpret_cast<float*>(norm_smem);   // [row groups][H]
  int k = 0;
  auto add_up = [&](const F8 (&sum)[2], void* final, int f32) {
    float* out = p.parts + ((int64_t)blockIdx.x * p.n_sums + k++) * p.H;
    auto put = [&](int i, const float2 (&v)[2]) {   // four columns from i on
      if (gridDim.x > 1) store4(out + i, v);
      else if (f32) store4(static_cast<float*>(final) + i, v);
      else store4(static_cast<uint16_t*>(final) + i, v);
    };
    __syncthreads();   // the rows, or the sums before, have been read
#pragma unroll
    for (int j = 0; j < 2; ++j) store8(sums + threadIdx.y * p.H, c[j], sum[j]);
    __syncthreads();
    for (int i = 4 * (threadIdx.y * blockDim.x + threadIdx.x); i < p.H; i += 4 * blockDim.x * blockDim.y) {
      float2 q[2], r[2];
      load4(sums + i, q);
      for (int ty = 1; ty < (int)blockDim.y; ++ty) {
        load4(sums + ty * p.H + i, r);
        q[0].x += r[0].x; q[0].y += r[0].y; q[1].x += r[1].x; q[1].y += r[1].y;
      }
      put(i, q);
    }
  };
  if (W) add_up(dw, p.dw, p.w_f32);
  if (V) add_up(dv, p.dv, p.v_f32);
  if (G && p.groups == 1) add_up(dg, p.dg, p.g_f32);
}

struct NormSumParams {
  const float* parts;
  void* out[3];
  int f32[3];
  int n_sums, blocks;     // sums over all rows
  void* dg;
  int dg_f32;
  uint32_t T, groups, gate_rows, row_groups;
  int H;
};

// The sums of the parts: blockIdx.y < n_sums a sum over all rows; beyond, a
// gate's group that several ranges share: group blockIdx.y - n_sums where
// there are no more groups than ranges, else the one that range
// blockIdx.y - n_sums + 1 goes on with.
constexpr int kNormSumWarps = 16;
__global__ void __launch_bounds__(32 * kNormSumWarps) block_norm_sum_kernel(const __grid_constant__ NormSumParams p) {
  __shared__ float2 part[kNormSumWarps][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 64 + 2 * lane;
  const bool mine = c < p.H;
  const bool whole = (int)blockIdx.y < p.n_sums;
  const float* first = p.parts + (int64_t)blockIdx.y * p.H;   // of the first part; the others: `rest` + i * pitch
  const float* rest = first;
  int64_t pitch = (int64_t)p.n_sums * p.H;
  uint32_t n = p.blocks, group = 0;
  if (!whole) {
    const uint32_t y = blockIdx.y - p.n_sums;
    uint32_t from;
    if (p.groups <= p.row_groups) {
      group = y;
      from = norm_group_of(p.T, p.row_groups, group * p.gate_rows);
    } else {
      const uint32_t start = norm_first_row(p.T, p.row_groups, y + 1);
      group = start / p.gate_rows;
      if (start == group * p.gate_rows) return;
      from = norm_group_of(p.T, p.row_groups, group * p.gate_rows);
      if (from != y) return;
    }
    const uint32_t to = norm_group_of(p.T, p.row_groups, (group + 1) * p.gate_rows - 1);
    if (from == to) return;   // within one range, which wrote it
    n = to - from + 1;
    pitch = 2 * p.H;
    rest = p.parts + ((int64_t)p.blocks * p.n_sums + 2 * (int64_t)from) * p.H;
    first = rest + (norm_first_row(p.T, p.row_groups, from) < group * p.gate_rows ? p.H : 0);
  }
  float2 s = make_float2(0.f, 0.f);
  if (mine) {
    // all of a warp's parts in flight together (152 parts: ten)
    for (uint32_t i0 = warp; i0 < n; i0 += 10 * kNormSumWarps) {
      float2 q[10];
#pragma unroll
      for (int k = 0; k < 10; ++k) {
        const uint32_t i = i0 + k * kNormSumWarps;
        q[k] = make_float2(0.f, 0.f);
        if (i < n) q[k] = *reinterpret_cast<const float2*>((i == 0 ? first : rest + i * pitch) + c);
      }
#pragma unroll
      for (int k = 0; k < 10; ++k) {
        s.x += q[k].x; s.y += q[k].y;
      }
    }
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && mine) {
#pragma unroll
    for (int i = 1; i < kNormSumWarps; ++i) {
      const float2 q = part[i][lane];
      s.x += q.x; s.y += q.y;
    }
    void* out = whole ? p.out[blockIdx.y] : p.dg;
    const int64_t at = (int64_t)group * p.H + c;
    if (whole ? p.f32[blockIdx.y] : p.dg_f32) *reinterpret_cast<float2*>(static_cast<float*>(out) + at) = s;
    else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(out) + at) = pack_bf16x2(s.x, s.y);
  }
}

// A launch's shape.  row_bytes: of a row's streams; params, wide: of w, v and
// a single gate as given and as fp32.  They are kept as fp32 where two stages
// fit beside them (16384 x 7168, bf16, backward: 200 us, as given 212), else as
// given (4096 x 4096, fp32 stream, bf16 weights: 83 us, from global memory 94).
// one_block: as many rows as one block holds take one, which needs no sums of
// sums (forward and backward of 8 x 256 6.4 us, in blocks of a row 7.7).
struct NormShape {
  dim3 block;
  int grid, stages, shared_params;
  size_t smem;
};
NormShape norm_shape(int64_t T, int64_t H, int threads, int groups, size_t row_bytes, size_t params, size_t wide,   // of a block; of 8 columns
                     bool one_block) {
  NormShape s;
  const int tpr = (int)((H + 256 * groups - 1) / (256 * groups) * 32);
  int rows = threads / tpr;
  if (tpr > 32) rows = std::min(rows, 15);   // row groups' barriers 1 .. 15; a warp needs none
  rows = (int)std::max<size_t>(1, std::min<size_t>(rows, kNormSmem / (2 * row_bytes)));
  rows = one_block && T <= rows ? (int)T : (int)std::max<int64_t>(1, std::min<int64_t>(rows, (T + kNormBlocks - 1) / kNormBlocks));
  s.shared_params = 2 * rows * row_bytes + wide <= kNormSmem ? kAsFp32 : 2 * rows * row_bytes + params <= kNormSmem ? kAsGiven : kInGlobal;
  params = s.shared_params == kAsFp32 ? wide : s.shared_params == kAsGiven ? params : 0;
  const size_t room = kNormSmem - params;
  s.stages = (int)std::min<size_t>(kNormMaxStages, room / (rows * row_bytes));
  s.block = dim3(tpr, rows);
  s.grid = (int)std::min<int64_t>((T + rows - 1) / rows, kNormBlocks);
  s.smem = (size_t)rows * s.stages * row_bytes + params;
  return s;
}

size_t norm_wide_bytes(const BlockNorm& n) { return (size_t)n.H * 4 * ((n.w != nullptr) + (n.v != nullptr) + (n.groups == 1)); }
size_t norm_params_bytes(const BlockNorm& n) {
  return (size_t)n.H * ((n.w ? (n.w_f32 ? 4 : 2) : 0) + (n.v ? (n.v_f32 ? 4 : 2) : 0) + (n.groups == 1 ? (n.g_f32 ? 4 : 2) : 0));
}

NormParams norm_params(const BlockNorm& n, const NormShape& s, const DeviceInfo& dev) {
  NormParams p = {};
  p.x = n.x; p.y = n.y; p.w = n.w; p.v = n.v; p.g = n.g;
  p.T = n.T; p.H = (int)n.H; p.groups = n.groups; p.gate_rows = n.groups ? n.T / n.groups : n.T;
  p.a = n.a; p.b = n.b; p.eps = n.eps;
  p.w_f32 = n.w_f32; p.v_f32 = n.v_f32; p.g_f32 = n.g_f32;
  p.stages = s.stages;
  p.shared_params = s.shared_params;
  p.status = dev.status;
  p.wait_limit_ns = dev.wait_limit_ns;
  return p;
}

using NormKernel = void (*)(NormParams);

template <typename X>
NormKernel norm_kernel(bool bwd, const BlockNorm& n) {
  const int which = (n.w ? 1 : 0) | (n.v ? 2 : 0) | (n.g ? 4 : 0);
  if (!n.y) return bwd ? block_norm_bwd_kernel<X, false, true, false, false> : block_norm_kernel<X, false, true, false, false>;
#define MOE_NORM(i) \
  case i: return bwd ? block_norm_bwd_kernel<X, true, (i & 1) != 0, (i & 2) != 0, (i & 4) != 0> \
                     : block_norm_kernel<X, true, (i & 1) != 0, (i & 2) != 0, (i & 4) != 0>;
  switch (which) {
    MOE_NORM(0) MOE_NORM(1) MOE_NORM(2) MOE_NORM(3) MOE_NORM(4) MOE_NORM(5) MOE_NORM(6)
    default: MOE_NORM(7)
  }
#undef MOE_NORM
}

cudaError_t norm_launch(bool bwd, const BlockNorm& n, const NormShape& s, const NormParams& p, const DeviceInfo& dev,
                        cudaStream_t stream) {
  const NormKernel kernel = n.x_f32 ? norm_kernel<float>(bwd, n) : norm_kernel<uint16_t>(bwd, n);
  // per-device set-up, cached (a race between host threads only repeats it)
  static std::atomic<int> configured[kMaxDevices][2][2][9] = {};
  std::atomic<int>& done = configured[dev.ordinal][bwd][n.x_f32 != 0][n.y ? (n.w ? 1 : 0) | (n.v ? 2 : 0) | (n.g ? 4 : 0) : 8];
  if (!done.load()) {
    const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kNormSmem);
    if (e != cudaSuccess) return e;
    done.store(1);
  }
  return launch_pdl(kernel, dim3(s.grid), s.block, s.smem, stream, 1, p);
}

NormShape norm_bwd_shape(const BlockNorm& n, bool dr) {
  return norm_shape(n.T, n.H, kNormThreads / 2, 2, (size_t)n.H * ((n.x_f32 ? 4 : 2) * (dr ? 2 : 1) + (n.y ? 2 : 0) + (n.w ? 2 : 0)),
                    norm_params_bytes(n), norm_wide_bytes(n), n.groups <= 1 || n.groups == n.T);   // no gate's rows to join
}

}  // namespace

int64_t block_norm_max_width() { return kNormMaxH; }

cudaError_t launch_block_norm(const BlockNorm& n, void* r, uint16_t* h, float* stats, const DeviceInfo& dev,
                              cudaStream_t stream) {
  const NormShape s = norm_shape(n.T, n.H, kNormThreads, norm_groups(n.v && n.w, n.x_f32), (size_t)n.H * ((n.x_f32 ? 4 : 2) + (n.y ? 2 : 0)), norm_params_bytes(n),
                                 norm_wide_bytes(n), false);
  NormParams p = norm_params(n, s, dev);
  p.r = r; p.h = h; p.stats = stats;
  return norm_launch(false, n, s, p, dev, stream);
}

// The most that any types and any dr take: row groups are fewest bytes a row.
size_t block_norm_bwd_workspace_bytes(int64_t T, int64_t H, int64_t groups, bool w, bool v) {
  if (T == 0) return 0;
  const NormShape s = norm_shape(T, H, kNormThreads / 2, 2, (size_t)H * (w ? 4 : 2), 0, 0, true);
  const size_t n_sums = (w ? 1 : 0) + (v ? 1 : 0) + (groups == 1 ? 1 : 0);
  const size_t blocks = std::min<int64_t>(T, kNormBlocks);
  return sizeof(float) * (size_t)H * (blocks * n_sums + (groups > 1 ? 2 * blocks * s.block.y : 0));
}

cudaError_t launch_block_norm_bwd(const BlockNorm& n, const uint16_t* dh, const void* dr, const float* stats,
                                  const BlockNormGrads& d, void* ws, const DeviceInfo& dev, cudaStream_t stream) {
  if (n.T == 0) {   // sums over no rows
    const struct { void* out; int f32; int64_t rows; } zero[] = {{d.w, n.w_f32, 1}, {d.v, n.v_f32, 1}, {d.g, n.g_f32, n.groups}};
    for (const auto& z : zero)
      if (z.out) {
        const cudaError_t e = cudaMemsetAsync(z.out, 0, (size_t)(z.rows * n.H) * (z.f32 ? 4 : 2), stream);
        if (e != cudaSuccess) return e;
      }
    return cudaSuccess;
  }
  const NormShape s = norm_bwd_shape(n, dr != nullptr);
  NormParams p = norm_params(n, s, dev);
  p.stats = const_cast<float*>(stats);
  p.dh = dh; p.dr = dr; p.dx = d.x; p.dy = d.y; p.dg = d.g; p.dw = d.w; p.dv = d.v;
  p.parts = static_cast<float*>(ws);
  NormSumParams q = {};
  q.parts = p.parts;
  int k = 0;
  if (n.w) { q.out[k] = d.w; q.f32[k++] = n.w_f32; }
  if (n.v) { q.out[k] = d.v; q.f32[k++] = n.v_f32; }
  if (n.groups == 1) { q.out[k] = d.g; q.f32[k++] = n.g_f32; }
  p.n_sums = q.n_sums = k;
  const cudaError_t e = norm_launch(true, n, s, p, dev, stream);
  if (e != cudaSuccess) return e;
  q.blocks = s.grid;
  q.dg = d.g;
  q.dg_f32 = n.g_f32;
  q.T = (uint32_t)n.T; q.groups = (uint32_t)n.groups; q.gate_rows = (uint32_t)p.gate_rows; q.H = p.H;
  q.row_groups = (uint32_t)s.grid * s.block.y;
  const int64_t shared = n.groups > 1 && p.gate_rows > 1 ? (n.groups <= q.row_groups ? n.groups : (int64_t)q.row_groups - 1) : 0;
  if (s.grid == 1 || k + shared == 0) return cudaSuccess;
  return launch_pdl(block_norm_sum_kernel, dim3((unsigned)((n.H + 63) / 64), (unsigned)(k + shared)), dim3(32 * kNormSumWarps), 0, stream, 1, q);
}

}  // namespace moe
