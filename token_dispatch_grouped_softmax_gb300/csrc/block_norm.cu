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
// A row belongs to TPR threads, each with 8 consecutive columns, and a block
// of up to 1024 threads holds several rows at a time.
#include <algorithm>

#include "kernels.h"

namespace moe {

namespace {

constexpr int kNormMaxH = 8192;
constexpr int kNormBlocks = 152;   // GB300's SMs; fixed, as the order of the columns' sums goes by it

__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const uint16_t* p, float* v) { unpack8(*reinterpret_cast<const uint4*>(p), v); }
__device__ __forceinline__ void store8(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(uint16_t* p, const float* v) { *reinterpret_cast<uint4*>(p) = pack8(v); }

// 8 values of an fp32 or bf16 vector.
__device__ __forceinline__ void load8(const void* p, bool f32, int64_t at, float* v) {
  if (f32) load8(static_cast<const float*>(p) + at, v);
  else load8(static_cast<const uint16_t*>(p) + at, v);
}
__device__ __forceinline__ void fill8(float* v, float c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = c;
}

// Sums over a row's threads.  Two buffers in turn: a thread writes a buffer
// again only after the barrier of the sum in between, which every thread
// reaches after reading it.
struct RowSum {
  float* buf;       // [2][warps of the block]
  int warps;        // of a row
  int warps_block;
  int turn = 0;

  __device__ __forceinline__ float operator()(float v) {
    v = warp_sum(v);
    if (warps == 1) return v;
    const int w = threadIdx.x >> 5;
    float* b = buf + turn * warps_block + threadIdx.y * warps;
    if ((threadIdx.x & 31) == 0) b[w] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.y), "r"(32 * warps) : "memory");
    turn ^= 1;
    float s = 0.f;
    for (int i = 0; i < warps; ++i) s += b[i];
    return s;
  }
};

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
  float* parts;           // [grid][sums][H], then [virtual blocks][2][H] of the gate's groups
  void* dg;               // finished groups are written here
  int64_t T;
  int H;
  int64_t gate_rows;      // rows of a gate's group
  int64_t groups;
  float a, b, eps;
  int w_f32, v_f32, g_f32;
  int n_sums;             // columns' sums over all rows: dw, dv, dg with one group
};

template <typename X>
__global__ void __launch_bounds__(1024) block_norm_kernel(const NormParams p) {
  __shared__ float sums[2 * 32];
  pdl_wait();
  pdl_trigger();
  const int c = threadIdx.x * 8;
  const bool mine = c < p.H;
  RowSum row_sum{sums, (int)blockDim.x >> 5, (int)(blockDim.x * blockDim.y) >> 5};
  float w[8], v[8], g[8];
  fill8(w, 1.f);
  fill8(v, 1.f);
  fill8(g, 1.f);
  if (mine) {
    if (p.w) load8(p.w, p.w_f32, c, w);
    if (p.v) load8(p.v, p.v_f32, c, v);
    if (p.groups == 1) load8(p.g, p.g_f32, c, g);
  }
  const X* x = static_cast<const X*>(p.x);
  const float inv = 1.f / (float)p.H;
  for (int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; t < p.T; t += (int64_t)gridDim.x * blockDim.y) {
    const int64_t at = t * p.H + c;
    float r[8], y[8];
    fill8(r, 0.f);
    fill8(y, 0.f);
    if (mine) {
      load8(x + at, r);
      if (p.y) load8(p.y + at, y);
    }
    if (p.y) {
      if (p.v) {
        float q = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) q = fmaf(y[i], y[i], q);
        const float s = rsqrtf(row_sum(q) * inv + p.eps);
        if (p.stats && threadIdx.x == 0) p.stats[p.T + t] = s;
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] *= s * v[i];
      }
      if (p.groups > 1 && mine) load8(p.g, p.g_f32, t / p.gate_rows * p.H + c, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = fmaf(p.a, r[i], p.b * (g[i] * y[i]));
      if (mine) store8(static_cast<X*>(p.r) + at, r);
    }
    if (p.w) {
      float q = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) q = fmaf(r[i], r[i], q);
      if (!mine) q = 0.f;
      const float s = rsqrtf(row_sum(q) * inv + p.eps);
      if (p.stats && threadIdx.x == 0) p.stats[t] = s;
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] *= s * w[i];
      if (mine) store8(p.h + at, r);
    }
  }
}

// A virtual block (one row's threads of a block) takes a range of consecutive
// rows, so that its columns' sums stay in registers and a gate's group ends
// at most twice inside a range.
__device__ __host__ __forceinline__ int64_t norm_first_row(int64_t T, int64_t n, int64_t v) {
  const int64_t share = T / n, more = T - share * n;
  return v * share + (v < more ? v : more);
}

template <typename X>
__global__ void __launch_bounds__(1024, 1) block_norm_bwd_kernel(const NormParams p) {
  __shared__ float sums[2 * 32];
  pdl_wait();
  pdl_trigger();
  const int c = threadIdx.x * 8;
  const bool mine = c < p.H;
  RowSum row_sum{sums, (int)blockDim.x >> 5, (int)(blockDim.x * blockDim.y) >> 5};
  const X* x = static_cast<const X*>(p.x);
  const float inv = 1.f / (float)p.H;
  float dw[8], dv[8], dg[8];
  fill8(dw, 0.f);
  fill8(dv, 0.f);
  fill8(dg, 0.f);
  const int64_t n = (int64_t)gridDim.x * blockDim.y, me = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int64_t begin = norm_first_row(p.T, n, me), end = norm_first_row(p.T, n, me + 1);
  for (int64_t t = begin; t < end; ++t) {
    const int64_t at = t * p.H + c;
    float r[8], y[8], g[8], d[8];
    fill8(r, 0.f);
    fill8(y, 0.f);
    fill8(g, 1.f);
    fill8(d, 0.f);
    float s_y = 1.f;
    if (mine) {
      load8(x + at, r);
      if (p.y) load8(p.y + at, y);
      if (p.dr) load8(static_cast<const X*>(p.dr) + at, d);
      if (p.g) load8(p.g, p.g_f32, (p.groups > 1 ? t / p.gate_rows * p.H : 0) + c, g);
    }
    float v[8];
    fill8(v, 1.f);
    if (p.v) {
      s_y = p.stats[p.T + t];
      if (mine) load8(p.v, p.v_f32, c, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] *= s_y;
    }
    if (p.y) {
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = fmaf(p.a, r[i], p.b * (g[i] * (y[i] * v[i])));
    }
    if (p.w) {
      float u[8], w[8];
      fill8(u, 0.f);
      fill8(w, 0.f);
      if (mine) {
        load8(p.dh + at, u);
        load8(p.w, p.w_f32, c, w);
      }
      const float s = p.stats[t];
      float q = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        r[i] *= s;
        dw[i] = fmaf(u[i], r[i], dw[i]);
        u[i] *= w[i];
        q = fmaf(u[i], r[i], q);
      }
      q = row_sum(q) * inv;
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] = fmaf(s, u[i] - r[i] * q, d[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = p.a * d[i];
    if (mine) store8(static_cast<X*>(p.dx) + at, r);
    if (p.y) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[i] *= p.b;
        dg[i] = fmaf(d[i], y[i] * v[i], dg[i]);
        d[i] *= g[i];
      }
      if (p.v) {
        float q = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dv[i] = fmaf(d[i], y[i], dv[i]);
          d[i] *= v[i];
          q = fmaf(d[i], y[i], q);
        }
        q = row_sum(q) * inv;
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = s_y * (d[i] - y[i] * q);
      }
      if (mine) store8(p.dy + at, d);
    }
    if (p.groups > 1 && ((t + 1) % p.gate_rows == 0 || t + 1 == end)) {
      const int64_t group = t / p.gate_rows;
      if (mine) {
        if (group * p.gate_rows >= begin && (group + 1) * p.gate_rows <= end) {
          if (p.g_f32) store8(static_cast<float*>(p.dg) + group * p.H + c, dg);
          else store8(static_cast<uint16_t*>(p.dg) + group * p.H + c, dg);
        } else {
          const int64_t slot = 2 * me + (group != begin / p.gate_rows);
          store8(p.parts + ((int64_t)gridDim.x * p.n_sums + slot) * p.H + c, dg);
        }
      }
      fill8(dg, 0.f);
    }
  }
  // the block's rows' sums, in the order of its rows' threads
  extern __shared__ float block_sums[];   // [H], with more than one row
  int k = 0;
  auto add_up = [&](const float (&sum)[8]) {
    for (int ty = 0; ty < (int)blockDim.y; ++ty) {
      if (blockDim.y > 1) __syncthreads();
      if ((int)threadIdx.y != ty || !mine) continue;
      float s[8];
      fill8(s, 0.f);
      if (ty > 0) load8(block_sums + c, s);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] += sum[i];
      if (ty + 1 < (int)blockDim.y) store8(block_sums + c, s);
      else store8(p.parts + ((int64_t)blockIdx.x * p.n_sums + k) * p.H + c, s);
    }
    ++k;
  };
  if (p.w) add_up(dw);
  if (p.v) add_up(dv);
  if (p.groups == 1) add_up(dg);
}

struct NormSumParams {
  const float* parts;
  void* out[3];
  int f32[3];
  int n_sums, blocks;     // sums over all rows
  void* dg;
  int dg_f32;
  int64_t T, groups, gate_rows, virtual_blocks;
  int H;
};

// The sums of the blocks' parts: blockIdx.y < n_sums a sum over all rows, and
// from there on the gate's group that the range of virtual block
// blockIdx.y - n_sums + 1 is the second to touch.
__global__ void __launch_bounds__(1024) block_norm_sum_kernel(const NormSumParams p) {
  __shared__ float4 part[32][32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 128 + 4 * lane;
  const bool mine = c < p.H;
  const float* first;
  int64_t n, pitch, group = 0;
  int64_t first_v = 0;
  const bool whole = (int)blockIdx.y < p.n_sums;
  if (whole) {
    first = p.parts + (int64_t)blockIdx.y * p.H;
    n = p.blocks;
    pitch = (int64_t)p.n_sums * p.H;
  } else {
    const int64_t vb = blockIdx.y - p.n_sums + 1, start = norm_first_row(p.T, p.virtual_blocks, vb);
    if (start >= p.T) return;
    group = start / p.gate_rows;
    const int64_t row0 = group * p.gate_rows;
    first_v = vb - 1;
    if (start == row0 || norm_first_row(p.T, p.virtual_blocks, first_v) > row0) return;   // no group spans here, or not its first two
    int64_t last = vb;
    while (last + 1 < p.virtual_blocks && norm_first_row(p.T, p.virtual_blocks, last + 1) < row0 + p.gate_rows) ++last;
    n = last - first_v + 1;
    first = p.parts + (int64_t)p.blocks * p.n_sums * p.H;
    pitch = 0;
  }
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (mine) {
    for (int64_t i = warp; i < n; i += 32) {
      const float* at = first + i * pitch + c;
      if (!whole) {
        const int64_t v = first_v + i;
        at = first + (2 * v + (norm_first_row(p.T, p.virtual_blocks, v) / p.gate_rows != group)) * p.H + c;
      }
      const float4 q = *reinterpret_cast<const float4*>(at);
      s.x += q.x; s.y += q.y; s.z += q.z; s.w += q.w;
    }
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && mine) {
    for (int i = 1; i < 32; ++i) {
      const float4 q = part[i][lane];
      s.x += q.x; s.y += q.y; s.z += q.z; s.w += q.w;
    }
    void* out = whole ? p.out[blockIdx.y] : p.dg;
    const int64_t at = (whole ? 0 : group * p.H) + c;
    if (whole ? p.f32[blockIdx.y] : p.dg_f32) *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = s;
    else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  }
}

dim3 norm_block(int64_t T, int64_t H, int sms, int max_threads) {
  const int tpr = (int)((H / 8 + 31) / 32 * 32);
  int rows = std::min(max_threads / tpr, 15);   // barriers 1 .. 15 belong to rows
  if (tpr == 32) rows = max_threads / tpr;      // a warp needs none
  rows = (int)std::max<int64_t>(1, std::min<int64_t>(rows, (T + sms - 1) / sms));
  return dim3(tpr, rows);
}

struct NormBwdShape {
  dim3 block;
  int grid, n_sums;
};
NormBwdShape norm_bwd_shape(int64_t T, int64_t H, int64_t groups, bool w, bool v) {
  NormBwdShape s;
  s.block = norm_block(T, H, kNormBlocks, 1024);
  s.grid = (int)std::min<int64_t>((T + s.block.y - 1) / s.block.y, kNormBlocks);
  s.n_sums = (w ? 1 : 0) + (v ? 1 : 0) + (groups == 1 ? 1 : 0);
  return s;
}

}  // namespace

int64_t block_norm_max_width() { return kNormMaxH; }

cudaError_t launch_block_norm(const BlockNorm& n, void* r, uint16_t* h, float* stats, cudaStream_t stream) {
  NormParams p = {};
  p.x = n.x; p.y = n.y; p.w = n.w; p.v = n.v; p.g = n.g;
  p.r = r; p.h = h; p.stats = stats;
  p.T = n.T; p.H = (int)n.H; p.groups = n.groups; p.gate_rows = n.groups ? n.T / n.groups : n.T;
  p.a = n.a; p.b = n.b; p.eps = n.eps;
  p.w_f32 = n.w_f32; p.v_f32 = n.v_f32; p.g_f32 = n.g_f32;
  const dim3 block = norm_block(n.T, n.H, 4 * kNormBlocks, 256);
  const int per_sm = 2048 / (int)(block.x * block.y);
  const unsigned grid = (unsigned)std::min<int64_t>((n.T + block.y - 1) / block.y, (int64_t)kNormBlocks * per_sm);
  return launch_pdl(n.x_f32 ? block_norm_kernel<float> : block_norm_kernel<uint16_t>, dim3(grid), block, 0, stream, 1, p);
}

size_t block_norm_bwd_workspace_bytes(int64_t T, int64_t H, int64_t groups, bool w, bool v) {
  const NormBwdShape s = norm_bwd_shape(T, H, groups, w, v);
  return sizeof(float) * (size_t)H * ((size_t)s.grid * s.n_sums + (groups > 1 ? (size_t)2 * s.grid * s.block.y : 0));
}

cudaError_t launch_block_norm_bwd(const BlockNorm& n, const uint16_t* dh, const void* dr, const float* stats,
                                  const BlockNormGrads& d, void* ws, cudaStream_t stream) {
  if (n.T == 0) {   // sums over no rows
    const struct { void* out; int f32; int64_t rows; } zero[] = {{d.w, n.w_f32, 1}, {d.v, n.v_f32, 1}, {d.g, n.g_f32, n.groups}};
    for (const auto& z : zero)
      if (z.out) {
        const cudaError_t e = cudaMemsetAsync(z.out, 0, (size_t)(z.rows * n.H) * (z.f32 ? 4 : 2), stream);
        if (e != cudaSuccess) return e;
      }
    return cudaSuccess;
  }
  NormParams p = {};
  p.x = n.x; p.y = n.y; p.w = n.w; p.v = n.v; p.g = n.g;
  p.stats = const_cast<float*>(stats);
  p.dh = dh; p.dr = dr; p.dx = d.x; p.dy = d.y; p.dg = d.g;
  p.parts = static_cast<float*>(ws);
  p.T = n.T; p.H = (int)n.H; p.groups = n.groups; p.gate_rows = n.groups ? n.T / n.groups : n.T;
  p.a = n.a; p.b = n.b; p.eps = n.eps;
  p.w_f32 = n.w_f32; p.v_f32 = n.v_f32; p.g_f32 = n.g_f32;
  const NormBwdShape s = norm_bwd_shape(n.T, n.H, n.groups, n.w, n.v);
  p.n_sums = s.n_sums;
  const size_t smem = s.block.y > 1 ? (size_t)n.H * sizeof(float) : 0;
  cudaError_t e = launch_pdl(n.x_f32 ? block_norm_bwd_kernel<float> : block_norm_bwd_kernel<uint16_t>, dim3(s.grid),
                             s.block, smem, stream, 1, p);
  if (e != cudaSuccess) return e;
  NormSumParams q = {};
  q.parts = p.parts;
  int k = 0;
  if (n.w) { q.out[k] = d.w; q.f32[k++] = n.w_f32; }
  if (n.v) { q.out[k] = d.v; q.f32[k++] = n.v_f32; }
  if (n.groups == 1) { q.out[k] = d.g; q.f32[k++] = n.g_f32; }
  q.n_sums = k;
  q.blocks = s.grid;
  q.dg = d.g;
  q.dg_f32 = n.g_f32;
  q.T = n.T; q.groups = n.groups; q.gate_rows = p.gate_rows; q.H = p.H;
  q.virtual_blocks = (int64_t)s.grid * s.block.y;
  const unsigned spans = n.groups > 1 && p.gate_rows > 1 ? (unsigned)(q.virtual_blocks - 1) : 0;
  if (k + spans == 0) return cudaSuccess;
  return launch_pdl(block_norm_sum_kernel, dim3((unsigned)((n.H + 127) / 128), k + spans), dim3(1024), 0, stream, 1, q);
}

}  // namespace moe
