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
// Rows that share v and g share K = b g v, one vector, and the backward needs
// one columns' sum for both: u = sum_rows d y s_y, dv = b g u, dg = b v u
// (8191 x 2048, fp32 stream, backward: 44 us, with a vector and a sum for each
// 67; 4096 x 7168 84, with each 158).
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
// Measured on inputs that come from HBM: 16384 x 7168 in bf16 with a gate for
// each 1024 rows 156 us forward (940 MB, 6.0 TB/s) and 224 backward with the sums
// (1.41 GB, 6.3 TB/s).  With both norms a row has two sums to wait for: 8191 x
// 2048, fp32 stream, 37.5 us forward (201 MB, 5.4 TB/s), 56.5 backward (302 MB,
// 5.3).  The figures beside the choices, above and below, compare variants on one
// set of inputs used again and again, which the L2 holds in part: they are lower.
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
  __device__ __forceinline__ void load4(int at, float2* v) const {
    if (f32) moe::load4(static_cast<const float*>(p) + at, v);
    else moe::load4(static_cast<const uint16_t*>(p) + at, v);
  }
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}

// What y is multiplied by: b alone; a vector that all rows share, K = b g v of
// v and a single gate, whichever there are; v and a gate for each group of
// rows; v and a row's own gate, which is one of its streams.
enum { kPlain, kVector, kGroups, kOwnGate };

// The columns' sums' way out: of sum_rows dh r s_r into dw; with kVector of
// u = sum_rows d y s_y into dv = b g u and dg = b v u, else of dv as it is.
struct SumsOut {
  void *dw, *dv, *dg;
  const void *v, *g;
  int w_f32, v_f32, g_f32;
  int vector;
  float b;
};
__device__ __forceinline__ float2 get2(const void* p, int f32, int64_t at) {
  if (f32) return *reinterpret_cast<const float2*>(static_cast<const float*>(p) + at);
  const uint32_t q = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p) + at);
  return make_float2(bf16_lo(q), bf16_hi(q));
}
__device__ __forceinline__ void put2(void* p, int f32, int64_t at, float2 v) {
  if (f32) *reinterpret_cast<float2*>(static_cast<float*>(p) + at) = v;
  else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p) + at) = pack_bf16x2(v.x, v.y);
}
__device__ __forceinline__ void sums_out(const SumsOut& o, bool of_w, int c, float2 u) {
  if (of_w) return put2(o.dw, o.w_f32, c, u);
  if (!o.vector) return put2(o.dv, o.v_f32, c, u);
  u = mul2(u, make_float2(o.b, o.b));
  if (o.v) put2(o.dv, o.v_f32, c, o.g ? mul2(u, get2(o.g, o.g_f32, c)) : u);
  if (o.g) put2(o.dg, o.g_f32, c, o.v ? mul2(u, get2(o.v, o.v_f32, c)) : u);
}

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
  float* parts;           // [grid][sums][H], then [row groups][norm_slots][H] of the gate's groups
  void* dg;               // finished groups are written here
  SumsOut out;            // for a launch of one block
  int64_t T;
  int H;
  int64_t gate_rows;      // rows of a gate's group
  float a, b, eps;
  int w_f32, v_f32, g_f32;
  int n_sums;             // columns' sums over all rows: w's, then v's or K's
  int stages;
  int vectors_shared;     // w and v are in shared memory (always but with a row's own gates)
  uint32_t* status;
  uint64_t wait_limit_ns;
  int stall;              // test hook: no copies of x
};

// Rows of the workspace for a range among several of a gate's groups: its first
// group's sum, its last one's, and dv's where there is one.
constexpr __host__ __device__ int norm_slots(bool v) { return v ? 3 : 2; }

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

__device__ __noinline__ bool norm_wait_more(uint32_t bar, uint32_t phase, volatile int* abort, uint64_t limit_ns, uint32_t* status) {
  return mbar_wait_bounded(bar, phase, abort, limit_ns, status, 1, kKernNorm);
}

// After a wait for row i that ran out, by a thread that copies a stream: its
// copies of rows i .. end - 1 are in flight, and nobody may write the ring or
// leave before them.  Bounded too: a phase lacks what other threads did not copy.
__device__ __noinline__ void norm_land(uint32_t bar, int i, int end, int stage, uint32_t phase, int stages, uint64_t limit_ns) {
  const uint64_t t0 = globaltimer_ns();
  for (; i < end; ++i) {
    while (!mbar_try_wait(bar + 8 * stage, phase) && globaltimer_ns() - t0 < limit_ns) {
    }
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
}

// A row group: its rows, its ring and its sums.
struct RowGroup {
  static constexpr uint32_t kPrefetch = 0xffffffffu, kGivenUp = 0xffffffffu;
  // the stream that this thread copies, if any: a thread of another warp for
  // each where the row group has as many, as all wait for the slowest
  const uint8_t* src;     // its first row of the range
  uint32_t bytes, offset; // of a row; in a stage (kPrefetch: into the L2 instead)
  uint8_t* ring;
  uint32_t row_bytes;     // of a stage
  uint32_t bar;           // kGivenUp: this thread's wait ran out
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
    if (offset == kPrefetch) {
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src + (int64_t)i * bytes), "r"(bytes) : "memory");
      return;
    }
    mbar_arrive_expect_tx(bar + 8 * stage, bytes);
    bulk_load(smem_u32(ring) + stage * row_bytes + offset, src + (int64_t)i * bytes, bytes, bar + 8 * stage);
  }
  // Row i has landed.  A thread whose wait runs out reports it, lets its copies
  // in flight land, and neither waits nor copies from then on: a stage whose
  // phase did not complete takes no further copy.  All threads go on through
  // the same barriers to the kernel's end, over rows that are undefined.
  __device__ __forceinline__ const uint8_t* wait(const NormParams& p, int i, int stage, uint32_t phase) {
    const uint32_t b = bar + 8 * stage;
    if (bar != kGivenUp && !mbar_try_wait(b, phase) && !norm_wait_more(b, phase, abort, p.wait_limit_ns, p.status)) {
      // refill() has issued the rows below i - 1 + stages
      if (src && offset != kPrefetch) norm_land(bar, i, min(rows, max(i - 1, 0) + p.stages), stage, phase, p.stages, p.wait_limit_ns);
      src = nullptr;
      bar = kGivenUp;
    }
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
  const float *w, *k;     // in shared memory, fp32: w; K or v
};

// A row's streams, in a stage's order; kGate: a gate of every row's own.
enum { kX, kY, kDh, kDr, kGate };

// The block's shared memory: the row groups' rings, then w and K or v.
__device__ __forceinline__ NormSetup norm_setup(const NormParams& p, uint8_t* smem, const void* const (&src)[5],
                                                const int (&elem)[5], int64_t begin, int rows, bool dr_staged, bool vector) {
  __shared__ uint64_t bars[32 * kNormMaxStages];
  __shared__ __align__(16) float sums[32 * 64];
  __shared__ int abort_flag;
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, ty = threadIdx.y;
  NormSetup s;
  RowGroup& g = s.rg;
  g.row_bytes = 0;
  g.src = nullptr;
  g.bytes = g.offset = 0;
  int n = 0, n_src = 0, n_staged = 0;
#pragma unroll
  for (int k = 0; k < 5; ++k) {
    n_src += src[k] != nullptr;
    n_staged += src[k] != nullptr && (k != kDr || dr_staged);
  }
  const int step = g.warps() >= n_src ? 32 : 1;
#pragma unroll
  for (int k = 0; k < 5; ++k)
    if (src[k]) {
      const uint32_t bytes = (uint32_t)p.H * elem[k];
      const bool staged = k != kDr || dr_staged;
      if ((int)threadIdx.x == n * step) {
        g.src = k == kX && p.stall ? nullptr : static_cast<const uint8_t*>(src[k]) + begin * bytes;
        g.bytes = bytes;
        g.offset = staged ? g.row_bytes : RowGroup::kPrefetch;
      }
      if (staged) g.row_bytes += bytes;
      ++n;
    }
  g.rows = rows;
  g.bar = smem_u32(bars) + 8 * ty * p.stages;
  g.buf = sums + 64 * ty;
  g.turn = 0;
  g.abort = &abort_flag;
  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < (int)blockDim.y * p.stages; ++i) mbar_init(smem_u32(bars) + 8 * i, n_staged);
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
  float* to = reinterpret_cast<float*>(at);
  auto share = [&](const void* from, int f32, const void* times, int times_f32, float b) {
    const float* given = to;
    const Shared v{from, f32 != 0}, g{times, times_f32 != 0};
    for (int i = tid * 4; i < p.H; i += threads * 4) {
      float2 q[2] = {make_float2(b, b), make_float2(b, b)}, t[2];
      const Shared* const both[2] = {&v, &g};
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (both[k]->p) {
          both[k]->load4(i, t);
          q[0] = mul2(q[0], t[0]);
          q[1] = mul2(q[1], t[1]);
        }
      store4(to + i, q);
    }
    to += p.H;
    return given;
  };
  s.w = s.k = nullptr;
  if (p.vectors_shared) {
    if (p.w) s.w = share(p.w, p.w_f32, nullptr, 0, 1.f);
    if (vector) s.k = share(p.v, p.v_f32, p.g, p.g_f32, p.b);
    else if (p.v) s.k = share(p.v, p.v_f32, nullptr, 0, 1.f);
  }
  __syncthreads();
  return s;
}

// Where a row is among the gate's groups.
struct GatePlace {
  int group = 0, left = 0;   // its group, and the group's rows from it on
  __device__ __forceinline__ GatePlace(const NormParams& p, int64_t begin, int rows) {
    if (rows > 0) {
      group = (int)(begin / p.gate_rows);
      left = (int)((group + 1) * p.gate_rows - begin);
    }
  }
  __device__ __forceinline__ bool ends() { return --left == 0; }
  __device__ __forceinline__ void next(const NormParams& p) {
    ++group;
    left = (int)p.gate_rows;
  }
  __device__ __forceinline__ int64_t first(const NormParams& p) const { return (int64_t)group * p.H; }
};

// Groups of 8 columns of a thread of the forward: with two sums to wait for in
// a row of an fp32 stream, two, so that twice as many rows are under way (8191
// x 2048, both norms: 36.7 us, with one group 37.4; but of a bf16 stream 29.2,
// with one group 26.7, and with one norm 16384 x 7168 162, with one group 147),
// unless a group's K takes the registers (4096 x 7168, 4 gates: 60, with two 77).
constexpr __host__ __device__ int norm_groups(bool two_sums, bool x_f32, int kind) {
  return two_sums && x_f32 && kind != kGroups ? 2 : 1;
}

// Y: there is a block's output (y); W, V, G: w, v, g.
template <typename X, bool Y, bool W, bool V, int G>
__global__ void __launch_bounds__(kNormThreads, 1) block_norm_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(16) uint8_t norm_smem[];
  constexpr int N = norm_groups(V && W, sizeof(X) == 4, G);
  Columns c[N];
#pragma unroll
  for (int j = 0; j < N; ++j) c[j] = Columns((threadIdx.x + j * blockDim.x) >> 5, p.H);
  const uint32_t n = gridDim.x * blockDim.y, me = blockIdx.x * blockDim.y + threadIdx.y;
  const int64_t begin = norm_first_row((uint32_t)p.T, n, me);
  const int rows = (int)(norm_first_row((uint32_t)p.T, n, me + 1) - begin);
  NormSetup s = norm_setup(p, norm_smem, {p.x, p.y, nullptr, nullptr, G == kOwnGate ? p.g : nullptr},
                           {(int)sizeof(X), 2, 0, 0, p.g_f32 ? 4 : 2}, begin, rows, true, G == kVector);
  RowGroup& rg = s.rg;
  const float inv = 1.f / (float)p.H;
  int stage = 0;
  uint32_t phase = 0;
  GatePlace gate(p, begin, G == kGroups ? rows : 0);
  F8 group_k[N];   // K of the group, in registers
  const bool shared = G != kOwnGate || p.vectors_shared;
  auto load_w = [&](int j) { return shared ? load8(s.w, c[j]) : Shared{p.w, p.w_f32 != 0}.load(0, c[j]); };
  auto load_v = [&](int j) { return shared ? load8(s.k, c[j]) : Shared{p.v, p.v_f32 != 0}.load(0, c[j]); };
  auto next_gate = [&]() {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      group_k[j] = Shared{p.g, p.g_f32 != 0}.load(gate.first(p), c[j]);
      if (V) mul8(group_k[j], load_v(j));
      mul8(group_k[j], p.b);
    }
  };
  if (G == kGroups && rows > 0) next_gate();
  X* out_r = static_cast<X*>(p.r) + begin * p.H;
  uint16_t* out_h = p.h + begin * p.H;
  auto squares = [](const F8 (&v)[N]) {
    float q = dot8(v[0], v[0]);
#pragma unroll
    for (int j = 1; j < N; ++j) q += dot8(v[j], v[j]);
    return q;
  };
  for (int i = 0; i < rows; ++i) {
    const uint8_t* row = rg.wait(p, i, stage, phase);
    const Shared own{row + p.H * (sizeof(X) + 2), p.g_f32 != 0};
    F8 r[N], y[N];
    float sy = G == kVector || G == kGroups ? 1.f : p.b;   // the factor of y, s_y among it
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
      if (G == kGroups) mul8(y[j], group_k[j]);
      else if (V || G == kVector) mul8(y[j], load_v(j));
      if (G == kOwnGate) mul8(y[j], own.load(0, c[j]));
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
        mul8(r[j], load_w(j));
        store8(out_h, c[j], r[j]);
      }
    }
    if (!V && !W) {
      rg.sync();
      rg.refill(p, i, stage);
    }
    if (G == kGroups && gate.ends()) {
      gate.next(p);
      if (i + 1 < rows) next_gate();
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
// sums take up to 128 registers (with 8 columns a thread and 64 registers they spill).
template <typename X, bool Y, bool W, bool V, int G, bool R>
__global__ void __launch_bounds__(kNormThreads / 2, 1) block_norm_bwd_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(16) uint8_t norm_smem[];
  const Columns c[2] = {Columns(threadIdx.x >> 5, p.H), Columns((threadIdx.x + blockDim.x) >> 5, p.H)};
  const uint32_t n = gridDim.x * blockDim.y, me = blockIdx.x * blockDim.y + threadIdx.y;
  const int64_t begin = norm_first_row((uint32_t)p.T, n, me);
  const int rows = (int)(norm_first_row((uint32_t)p.T, n, me + 1) - begin);
  NormSetup s = norm_setup(p, norm_smem, {p.x, p.y, p.dh, p.dr, G == kOwnGate ? p.g : nullptr},
                           {(int)sizeof(X), 2, 2, (int)sizeof(X), p.g_f32 ? 4 : 2}, begin, rows, R, G == kVector);
  RowGroup& rg = s.rg;
  const float inv = 1.f / (float)p.H;
  // Of several groups' gates dv is added up in the workspace, at the groups'
  // ends: its registers hold K (8192 x 2048 in bf16, 8 gates: 39 us; with dv
  // in registers too 60, with K from shared and global memory 58).
  auto slot = [&](int k) { return p.parts + ((int64_t)gridDim.x * p.n_sums + norm_slots(V) * (int64_t)me + k) * p.H; };
  F8 dw[2], dv[2], u[2], group_k[2];   // u: of all rows with K, else of the gate's group, whose K stays here
  const Shared gates{p.g, p.g_f32 != 0};
  const bool shared = G != kOwnGate || p.vectors_shared;
  auto load_w = [&](int j) { return shared ? load8(s.w, c[j]) : Shared{p.w, p.w_f32 != 0}.load(0, c[j]); };
  auto load_v = [&](int j) { return shared ? load8(s.k, c[j]) : Shared{p.v, p.v_f32 != 0}.load(0, c[j]); };
  int stage = 0;
  uint32_t phase = 0;
  GatePlace gate(p, begin, G == kGroups ? rows : 0);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    dw[j] = dv[j] = u[j] = fill8(0.f);
  }
  auto next_gate = [&](int j) {
    group_k[j] = gates.load(gate.first(p), c[j]);
    if (V) mul8(group_k[j], load_v(j));
    mul8(group_k[j], p.b);
  };
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (G == kGroups && rows > 0) next_gate(j);
  auto load_k = [&](int j) { return G == kGroups ? group_k[j] : load_v(j); };
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
  const uint32_t at_gate = at_dr + (R && p.dr ? p.H * sizeof(X) : 0);
  for (int i = 0; i < rows; ++i) {
    const float sr = next_r, sy = next_y;
    stats(i + 1);
    // Between the sums a thread keeps r and dh w alone, and reads the row's
    // other operands from shared memory again.
    const uint8_t* row = rg.wait(p, i, stage, phase);
    auto own_of = [&](int j) { return Shared{row + at_gate, p.g_f32 != 0}.load(0, c[j]); };
    auto load_y = [&](int j) {   // normed, without v
      F8 y = load8(reinterpret_cast<const uint16_t*>(row + at_y), c[j]);
      if (V) mul8(y, sy);
      return y;
    };
    auto load_dr = [&](int j) {
      if (!p.dr) return fill8(0.f);
      return R ? load8(reinterpret_cast<const X*>(row + at_dr), c[j])
               : load8(static_cast<const X*>(p.dr) + (begin + i) * p.H, c[j]);
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
          if (V || G == kVector || G == kGroups) mul8(y, load_k(j));
          if (G == kOwnGate) mul8(y, own_of(j));
          if (G == kPlain || G == kOwnGate) mul8(y, p.b);
          fma8(fill8(p.a), r[j], y);
          r[j] = y;
        }
        mul8(r[j], sr);
        d[j] = load8(reinterpret_cast<const uint16_t*>(row + at_dh), c[j]);
        fma8(d[j], r[j], dw[j]);
        mul8(d[j], load_w(j));
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
      if (G == kPlain || G == kOwnGate) mul8(d[j], p.b);
      if (G == kPlain) continue;
      const F8 y = load_y(j);
      if (G == kOwnGate) {   // dg of this row, b d times its n
        F8 m = y;
        mul8(m, d[j]);
        const F8 g = own_of(j);
        if (V) {
          const F8 v = load_v(j);
          fma8(m, g, dv[j]);
          mul8(m, v);
          mul8(d[j], v);
        }
        const int64_t at = (begin + i) * p.H;
        if (p.g_f32) store8(static_cast<float*>(p.dg) + at, c[j], m);
        else store8(static_cast<uint16_t*>(p.dg) + at, c[j], m);
        mul8(d[j], g);
      } else {
        fma8(d[j], y, u[j]);
        mul8(d[j], load_k(j));
      }
      if (V) q += dot8(d[j], y);
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
    if (G == kGroups) {   // dg = b v u, and g's part of dv
      const bool ends = gate.ends();
      if (ends || i + 1 == rows) {
        const int64_t first = gate.group * p.gate_rows, at = gate.first(p);
        gate.next(p);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          mul8(u[j], p.b);
          if (V) {
            F8 sum = first > begin ? load8(slot(2), c[j]) : fill8(0.f);
            fma8(u[j], gates.load(at, c[j]), sum);
            store8(slot(2), c[j], sum);
            mul8(u[j], load_v(j));
          }
          if (ends && first >= begin) {
            if (p.g_f32) store8(static_cast<float*>(p.dg) + at, c[j], u[j]);
            else store8(static_cast<uint16_t*>(p.dg) + at, c[j], u[j]);
          } else {   // the range's first group, or its last
            store8(slot(first > begin), c[j], u[j]);
          }
          u[j] = fill8(0.f);
          if (i + 1 < rows) next_gate(j);
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
  auto add_up = [&](const F8 (&sum)[2], bool of_w) {
    float* out = p.parts + ((int64_t)blockIdx.x * p.n_sums + k++) * p.H;
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
      if (gridDim.x > 1) {
        store4(out + i, q);
      } else {
        sums_out(p.out, of_w, i, q[0]);
        sums_out(p.out, of_w, i + 2, q[1]);
      }
    }
  };
  if (W) add_up(dw, true);
  if (G == kVector) add_up(u, false);
  else if (V) {
    if (G == kGroups && rows > 0) {
#pragma unroll
      for (int j = 0; j < 2; ++j) dv[j] = load8(slot(2), c[j]);
    }
    add_up(dv, false);
  }
}

struct NormSumParams {
  const float* parts;
  SumsOut out;
  int n_sums, blocks;     // sums over all rows
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
    pitch = norm_slots(p.out.v) * p.H;
    rest = p.parts + ((int64_t)p.blocks * p.n_sums + norm_slots(p.out.v) * (int64_t)from) * p.H;
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
    if (whole) sums_out(p.out, blockIdx.y == 0 && p.out.dw, c, s);
    else put2(p.out.dg, p.out.g_f32, (int64_t)group * p.H + c, s);
  }
}

// A launch's shape.  row_bytes: of a row's streams; vectors: of w and K or v
// as fp32, which stay in global memory where two stages of one row do not fit
// beside them (a row's own gates beyond H 6912).
// one_block: as many rows as one block holds take one, which needs no sums of
// sums (forward and backward of 8 x 256 6.4 us, in blocks of a row 7.7).
struct NormShape {
  dim3 block;
  int grid, stages, vectors_shared;
  size_t smem;
};
NormShape norm_shape(int64_t T, int64_t H, int threads, int groups, size_t row_bytes, size_t vectors, bool one_block) {   // groups of 8 columns
  NormShape s;
  const int tpr = (int)((H + 256 * groups - 1) / (256 * groups) * 32);
  s.vectors_shared = 2 * row_bytes + vectors <= kNormSmem;
  if (!s.vectors_shared) vectors = 0;
  const size_t room = kNormSmem - vectors;
  int rows = threads / tpr;
  if (tpr > 32) rows = std::min(rows, 15);   // row groups' barriers 1 .. 15; a warp needs none
  rows = (int)std::max<size_t>(1, std::min<size_t>(rows, room / (2 * row_bytes)));
  rows = one_block && T <= rows ? (int)T : (int)std::max<int64_t>(1, std::min<int64_t>(rows, (T + kNormBlocks - 1) / kNormBlocks));
  s.stages = (int)std::min<size_t>(kNormMaxStages, room / (rows * row_bytes));
  s.block = dim3(tpr, rows);
  s.grid = (int)std::min<int64_t>((T + rows - 1) / rows, kNormBlocks);
  s.smem = (size_t)rows * s.stages * row_bytes + vectors;
  return s;
}

size_t norm_vectors_bytes(const BlockNorm& n) { return (size_t)n.H * 4 * ((n.w != nullptr) + (n.v || n.groups == 1)); }
bool own_gate(const BlockNorm& n) { return n.groups > 1 && n.groups == n.T; }
size_t norm_gate_bytes(const BlockNorm& n) { return own_gate(n) ? (size_t)n.H * (n.g_f32 ? 4 : 2) : 0; }

NormParams norm_params(const BlockNorm& n, const NormShape& s, const DeviceInfo& dev) {
  NormParams p = {};
  p.x = n.x; p.y = n.y; p.w = n.w; p.v = n.v; p.g = n.g;
  p.T = n.T; p.H = (int)n.H; p.gate_rows = n.groups ? n.T / n.groups : n.T;
  p.a = n.a; p.b = n.b; p.eps = n.eps;
  p.w_f32 = n.w_f32; p.v_f32 = n.v_f32; p.g_f32 = n.g_f32;
  p.stages = s.stages;
  p.vectors_shared = s.vectors_shared;
  p.status = dev.status;
  p.wait_limit_ns = dev.wait_limit_ns;
  p.stall = dev.test_stall_producer;
  return p;
}

using NormKernel = void (*)(NormParams);

int norm_kind(const BlockNorm& n) { return own_gate(n) ? kOwnGate : n.groups > 1 ? kGroups : n.v || n.g ? kVector : kPlain; }

template <typename X, bool R, bool W, bool V, int G>
NormKernel norm_kernel(bool bwd) {
  return bwd ? block_norm_bwd_kernel<X, true, W, V, G, R> : block_norm_kernel<X, true, W, V, G>;
}
template <typename X, bool R>
NormKernel norm_kernel(bool bwd, const BlockNorm& n) {
  if (!n.y) return bwd ? block_norm_bwd_kernel<X, false, true, false, kPlain, R> : block_norm_kernel<X, false, true, false, kPlain>;
#define MOE_NORM(G) \
  case G: return n.w ? (n.v ? norm_kernel<X, R, true, true, G>(bwd) : norm_kernel<X, R, true, false, G>(bwd)) \
                     : (n.v ? norm_kernel<X, R, false, true, G>(bwd) : norm_kernel<X, R, false, false, G>(bwd));
  switch (norm_kind(n)) {
    MOE_NORM(kVector) MOE_NORM(kGroups) MOE_NORM(kOwnGate)
    default: return n.w ? norm_kernel<X, R, true, false, kPlain>(bwd) : norm_kernel<X, R, false, false, kPlain>(bwd);
  }
#undef MOE_NORM
}

cudaError_t norm_launch(bool bwd, bool dr_staged, const BlockNorm& n, const NormShape& s, const NormParams& p, const DeviceInfo& dev,
                        cudaStream_t stream) {
  const NormKernel kernel = n.x_f32 ? (dr_staged ? norm_kernel<float, true>(bwd, n) : norm_kernel<float, false>(bwd, n))
                                    : (dr_staged ? norm_kernel<uint16_t, true>(bwd, n) : norm_kernel<uint16_t, false>(bwd, n));
  // per-device set-up, cached (a race between host threads only repeats it)
  static std::atomic<int> configured[kMaxDevices][2][2][2][17] = {};
  std::atomic<int>& done = configured[dev.ordinal][bwd][dr_staged][n.x_f32 != 0]
                                       [n.y ? (n.w ? 1 : 0) | (n.v ? 2 : 0) | norm_kind(n) << 2 : 16];
  if (!done.load()) {
    const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kNormSmem);
    if (e != cudaSuccess) return e;
    done.store(1);
  }
  return launch_pdl(kernel, dim3(s.grid), s.block, s.smem, stream, 1, p);
}

// dr stays out of the ring where it leaves no room for two stages (the others
// take 12 bytes a column at most, 192 KB), for w and K or v, or for as many row
// groups.  Its rows are then prefetched into the L2 (4096 x 7168, fp32 stream,
// both norms: 80 us, with w and v read from global memory instead 97).
NormShape norm_bwd_shape(const BlockNorm& n, bool dr, bool* dr_staged) {
  const size_t dr_bytes = dr ? (size_t)n.H * (n.x_f32 ? 4 : 2) : 0;
  const size_t others = (size_t)n.H * ((n.x_f32 ? 4 : 2) + (n.y ? 2 : 0) + (n.w ? 2 : 0)) + norm_gate_bytes(n);
  const auto shape = [&](size_t row_bytes) {
    return norm_shape(n.T, n.H, kNormThreads / 2, 2, row_bytes, norm_vectors_bytes(n),
                      n.groups <= 1 || n.groups == n.T);   // no gate's rows to join
  };
  const NormShape with = shape(others + dr_bytes), without = shape(others);
  *dr_staged = with.stages >= 2 && with.vectors_shared == without.vectors_shared && with.block.y == without.block.y;
  return *dr_staged ? with : without;
}

}  // namespace

int64_t block_norm_max_width() { return kNormMaxH; }

cudaError_t launch_block_norm(const BlockNorm& n, void* r, uint16_t* h, float* stats, const DeviceInfo& dev,
                              cudaStream_t stream) {
  const NormShape s = norm_shape(n.T, n.H, kNormThreads, norm_groups(n.v && n.w, n.x_f32, norm_kind(n)),
                                 (size_t)n.H * ((n.x_f32 ? 4 : 2) + (n.y ? 2 : 0)) + norm_gate_bytes(n), norm_vectors_bytes(n), false);
  NormParams p = norm_params(n, s, dev);
  p.r = r; p.h = h; p.stats = stats;
  return norm_launch(false, true, n, s, p, dev, stream);
}

// The most that any types and any dr take: row groups are fewest bytes a row.
size_t block_norm_bwd_workspace_bytes(int64_t T, int64_t H, int64_t groups, bool w, bool v) {
  if (T == 0) return 0;
  const NormShape s = norm_shape(T, H, kNormThreads / 2, 2, (size_t)H * (w ? 4 : 2), 0, true);
  const size_t n_sums = (w ? 1 : 0) + (v || groups == 1 ? 1 : 0);
  const size_t blocks = std::min<int64_t>(T, kNormBlocks);
  return sizeof(float) * (size_t)H * (blocks * n_sums + (groups > 1 && groups != T ? norm_slots(v) * blocks * s.block.y : 0));
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
  bool dr_staged;
  const NormShape s = norm_bwd_shape(n, dr != nullptr, &dr_staged);
  NormParams p = norm_params(n, s, dev);
  p.stats = const_cast<float*>(stats);
  p.dh = dh; p.dr = dr; p.dx = d.x; p.dy = d.y; p.dg = d.g;
  p.out = {n.w ? d.w : nullptr, d.v, d.g, n.v, n.g, n.w_f32, n.v_f32, n.g_f32, norm_kind(n) == kVector, n.b};
  p.parts = static_cast<float*>(ws);
  NormSumParams q = {};
  q.parts = p.parts;
  q.out = p.out;
  const int k = (n.w ? 1 : 0) + (n.v || n.groups == 1 ? 1 : 0);
  p.n_sums = q.n_sums = k;
  const cudaError_t e = norm_launch(true, dr_staged, n, s, p, dev, stream);
  if (e != cudaSuccess) return e;
  q.blocks = s.grid;
  q.T = (uint32_t)n.T; q.groups = (uint32_t)n.groups; q.gate_rows = (uint32_t)p.gate_rows; q.H = p.H;
  q.row_groups = (uint32_t)s.grid * s.block.y;
  const int64_t shared = n.groups > 1 && p.gate_rows > 1 ? (n.groups <= q.row_groups ? n.groups : (int64_t)q.row_groups - 1) : 0;
  if (s.grid == 1 || k + shared == 0) return cudaSuccess;
  return launch_pdl(block_norm_sum_kernel, dim3((unsigned)((n.H + 63) / 64), (unsigned)(k + shared)), dim3(32 * kNormSumWarps), 0, stream, 1, q);
}

}  // namespace moe
