// Experts' products of a decode batch with 4-bit weights and group scales.
//
//   W_e[k, n] = scale[k / G, n] * (q[k, n] - zero[k / G, n]),  q in 0..15
//   gate_up:  h[t, j] = silu(x_t . Wg_e) * (x_t . Wu_e),  e = ids[t, j]
//   down:     y[t] = sum_j w[t, j] (h[t, j] . Wd_e)  (+ y_shared[t])
//
// q is int32 [E*K/8, N]: the word of row r holds the codes of k = 8r .. 8r+7
// of one column, lowest nibble first.  A slot whose id is -1 is empty.
#include <algorithm>

#include "kernels.h"

namespace moe {

namespace {

constexpr int kW4Cols = 128;   // columns (threads) per block

struct W4View {
  const uint32_t* q;
  const uint16_t* scales;
  const uint8_t* zeros;
  int K, N, group;
};

// sum_k row[k] * W[k, n] of one column of expert e: the codes' integer
// products are summed per group in fp32 and scaled once per group.
__device__ __forceinline__ float w4_dot(const W4View& w, int e, int n, const float* row) {
  float acc = 0.f;
  const int words = w.group / 8;
  const uint32_t* q = w.q + (int64_t)e * (w.K / 8) * w.N + n;
  const int64_t g0 = (int64_t)e * (w.K / w.group);
  for (int g = 0; g < w.K / w.group; ++g) {
    const float zero = w.zeros ? (float)w.zeros[(g0 + g) * w.N + n] : 8.f;
    float part = 0.f;
    for (int r = 0; r < words; ++r) {
      const uint32_t word = q[(int64_t)(g * words + r) * w.N];
      const float* x = row + (g * words + r) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) part = fmaf((float)((word >> (4 * i)) & 15u) - zero, x[i], part);
    }
    acc = fmaf(__uint_as_float((uint32_t)w.scales[(g0 + g) * w.N + n] << 16), part, acc);
  }
  return acc;
}

// The expert of a slot: -1 when it is empty; ids NULL is one dense expert.
__device__ __forceinline__ int slot_expert(const int32_t* ids, int64_t slot, int E, uint32_t* status) {
  if (!ids) return 0;
  const int e = ids[slot];
  if (e < -1 || e >= E) {
    report_status(status, kStatusDevice, kKernW4, 1);
    return -1;
  }
  return e;
}

__global__ void __launch_bounds__(kW4Cols) w4_gate_up_kernel(const uint16_t* __restrict__ x,
                                                             const int32_t* __restrict__ ids, const W4View w, int E,
                                                             int k, int I, uint16_t* __restrict__ h,
                                                             uint32_t* status) {
  extern __shared__ float row[];
  pdl_wait();
  pdl_trigger();
  const int64_t slot = blockIdx.x;
  const int n = blockIdx.y * kW4Cols + threadIdx.x;
  const int e = slot_expert(ids, slot, E, status);
  for (int c = threadIdx.x; c < w.K; c += kW4Cols) row[c] = __uint_as_float((uint32_t)x[slot / k * w.K + c] << 16);
  __syncthreads();
  if (n >= I) return;
  float v = 0.f;
  if (e >= 0) {
    const float g = w4_dot(w, e, n, row), u = w4_dot(w, e, I + n, row);
    v = g / (1.f + expf(-g)) * u;
  }
  h[slot * I + n] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

__global__ void __launch_bounds__(kW4Cols) w4_down_kernel(const uint16_t* __restrict__ h,
                                                          const int32_t* __restrict__ ids,
                                                          const float* __restrict__ wt, const W4View w, int E, int k,
                                                          const uint16_t* __restrict__ y_shared,
                                                          uint16_t* __restrict__ y, uint32_t* status) {
  extern __shared__ float row[];
  pdl_wait();
  pdl_trigger();
  const int64_t t = blockIdx.x;
  const int n = blockIdx.y * kW4Cols + threadIdx.x;
  float acc = 0.f;
  for (int j = 0; j < k; ++j) {
    const int64_t slot = t * k + j;
    const int e = slot_expert(ids, slot, E, status);
    if (e < 0) continue;
    __syncthreads();
    for (int c = threadIdx.x; c < w.K; c += kW4Cols) row[c] = __uint_as_float((uint32_t)h[slot * w.K + c] << 16);
    __syncthreads();
    if (n < w.N) acc = fmaf(wt ? wt[slot] : 1.f, w4_dot(w, e, n, row), acc);
  }
  if (n >= w.N) return;
  if (y_shared) acc += __uint_as_float((uint32_t)y_shared[t * w.N + n] << 16);
  y[t * w.N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(acc));
}

// One thread per (group, column) of [rows, N] bf16 weights.
//   symmetric: scale = bf16(max|w| / 7), q = clamp(rint(w / scale) + 8, 0, 15)
//   zeros:     scale = bf16((max(w, 0) - min(w, 0)) / 15), zero = clamp(rint(-min(w, 0) / scale), 0, 15),
//              q = clamp(rint(w / scale) + zero, 0, 15)
// A group of zeros has scale 0 and q = zero.
__global__ void __launch_bounds__(256) w4_quantize_kernel(const uint16_t* __restrict__ w, int64_t groups, int N,
                                                          int group, uint32_t* __restrict__ q,
                                                          uint16_t* __restrict__ scales, uint8_t* __restrict__ zeros) {
  pdl_wait();
  pdl_trigger();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= groups * N) return;
  const int64_t g = i / N;
  const int n = (int)(i - g * N);
  const uint16_t* src = w + g * group * N + n;
  float lo = 0.f, hi = 0.f;
  for (int r = 0; r < group; ++r) {
    const float v = __uint_as_float((uint32_t)src[(int64_t)r * N] << 16);
    lo = fminf(lo, v);
    hi = fmaxf(hi, v);
  }
  const float want = zeros ? (hi - lo) / 15.f : fmaxf(hi, -lo) / 7.f;
  const __nv_bfloat16 sb = __float2bfloat16_rn(want);
  const float s = __bfloat162float(sb);
  const float zero = zeros ? (s > 0.f ? fminf(rintf(-lo / s), 15.f) : 0.f) : 8.f;
  scales[i] = __bfloat16_as_ushort(sb);
  if (zeros) zeros[i] = (uint8_t)zero;
  for (int r = 0; r < group; r += 8) {
    uint32_t word = 0;
    for (int b = 0; b < 8; ++b) {
      const float v = __uint_as_float((uint32_t)src[(int64_t)(r + b) * N] << 16);
      const float c = s > 0.f ? fminf(fmaxf(rintf(v / s) + zero, 0.f), 15.f) : zero;
      word |= (uint32_t)c << (4 * b);
    }
    q[(g * group + r) / 8 * N + n] = word;
  }
}

// One thread per word: scale * (q - zero) in fp32, rounded to bf16.
__global__ void __launch_bounds__(256) w4_dequantize_kernel(const uint32_t* __restrict__ q,
                                                            const uint16_t* __restrict__ scales,
                                                            const uint8_t* __restrict__ zeros, int64_t words, int N,
                                                            int group, uint16_t* __restrict__ w) {
  pdl_wait();
  pdl_trigger();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= words * N) return;
  const int64_t r = i / N;
  const int n = (int)(i - r * N);
  const int64_t sg = r * 8 / group * N + n;
  const float s = __uint_as_float((uint32_t)scales[sg] << 16);
  const float zero = zeros ? (float)zeros[sg] : 8.f;
  const uint32_t word = q[i];
#pragma unroll
  for (int b = 0; b < 8; ++b)
    w[(r * 8 + b) * N + n] = __bfloat16_as_ushort(__float2bfloat16_rn(s * ((float)((word >> (4 * b)) & 15u) - zero)));
}

}  // namespace

cudaError_t launch_w4_gate_up(const uint16_t* x, const int32_t* ids, const uint32_t* q, const uint16_t* scales,
                              const uint8_t* zeros, int64_t T, int64_t H, int64_t E, int64_t k, int64_t I,
                              int64_t group, uint16_t* h, const DeviceInfo& dev, cudaStream_t stream) {
  const W4View w{q, scales, zeros, (int)H, (int)(2 * I), (int)group};
  return launch_pdl(w4_gate_up_kernel, dim3((unsigned)(T * k), (unsigned)((I + kW4Cols - 1) / kW4Cols)),
                    dim3(kW4Cols), (size_t)H * 4, stream, 1, x, ids, w, (int)E, (int)k, (int)I, h, dev.status);
}

cudaError_t launch_w4_down(const uint16_t* h, const int32_t* ids, const float* wt, const uint32_t* q,
                           const uint16_t* scales, const uint8_t* zeros, const uint16_t* y_shared, int64_t T,
                           int64_t H, int64_t E, int64_t k, int64_t I, int64_t group, uint16_t* y,
                           const DeviceInfo& dev, cudaStream_t stream) {
  const W4View w{q, scales, zeros, (int)I, (int)H, (int)group};
  return launch_pdl(w4_down_kernel, dim3((unsigned)T, (unsigned)((H + kW4Cols - 1) / kW4Cols)), dim3(kW4Cols),
                    (size_t)I * 4, stream, 1, h, ids, wt, w, (int)E, (int)k, y_shared, y, dev.status);
}

cudaError_t launch_w4_quantize(const uint16_t* w, int64_t rows, int64_t N, int64_t group, uint32_t* q,
                               uint16_t* scales, uint8_t* zeros, cudaStream_t stream) {
  const int64_t n = rows / group * N;
  return launch_pdl(w4_quantize_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, 1, w, rows / group,
                    (int)N, (int)group, q, scales, zeros);
}

cudaError_t launch_w4_dequantize(const uint32_t* q, const uint16_t* scales, const uint8_t* zeros, int64_t rows,
                                 int64_t N, int64_t group, uint16_t* w, cudaStream_t stream) {
  const int64_t n = rows / 8 * N;
  return launch_pdl(w4_dequantize_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, 1, q, scales,
                    zeros, rows / 8, (int)N, (int)group, w);
}

}  // namespace moe
