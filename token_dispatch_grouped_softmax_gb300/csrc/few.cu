// The expert layer for a few tokens in bf16, rows in slot order:
//
//   h[t, j] = silu(x_t . Wg_e) * (x_t . Wu_e),  e = ids[t, j]
//   y_t = sum_j w[t, j] (h[t, j] . Wd_e)  (+ the shared expert's, weight 1)
//
// One thread to a column.  Sums are fp32 in increasing k and j.
#include <algorithm>

#include "kernels.h"

namespace moe {

namespace {

constexpr int kFewThreads = 128;

struct FewParams {
  const uint16_t* x;
  const int32_t* ids;
  const float* w;
  const uint16_t *gate_up, *down, *sh_gate_up, *sh_down;
  uint16_t* y;
  float* h;          // [T*k, I], then [T, I_s] of the shared expert
  uint32_t* status;
  int T, H, E, k, I, I_s;
};

__device__ __forceinline__ float bf16_value(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

__global__ void __launch_bounds__(kFewThreads) few_gate_up_kernel(const FewParams p) {
  pdl_wait();
  pdl_trigger();
  const int slot = blockIdx.y;
  const bool shared = slot >= p.T * p.k;
  const int t = shared ? slot - p.T * p.k : slot / p.k;
  const int I = shared ? p.I_s : p.I;
  const int c = blockIdx.x * kFewThreads + threadIdx.x;
  const uint16_t* W = p.sh_gate_up;
  if (!shared) {
    const int e = p.ids[slot];
    if (e < 0 || e >= p.E) {
      if (e != -1) report_status(p.status, kStatusDevice, kKernFew, 1);
      return;
    }
    W = p.gate_up + (int64_t)e * p.H * 2 * I;
  }
  if (c >= I) return;
  const uint16_t* x = p.x + (int64_t)t * p.H;
  float g = 0.f, u = 0.f;
#pragma unroll 8
  for (int i = 0; i < p.H; ++i) {
    const float xi = bf16_value(x[i]);
    const uint16_t* row = W + (int64_t)i * 2 * I + c;
    g = fmaf(xi, bf16_value(row[0]), g);
    u = fmaf(xi, bf16_value(row[I]), u);
  }
  float* h = shared ? p.h + (int64_t)p.T * p.k * p.I + (int64_t)t * I : p.h + (int64_t)slot * I;
  h[c] = g / (1.f + expf(-g)) * u;
}

__global__ void __launch_bounds__(kFewThreads) few_down_kernel(const FewParams p) {
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.y, c = blockIdx.x * kFewThreads + threadIdx.x;
  if (c >= p.H) return;
  float y = 0.f;
  for (int j = 0; j < p.k; ++j) {
    const int e = p.ids[t * p.k + j];
    if (e < 0 || e >= p.E) continue;
    const float* h = p.h + (int64_t)(t * p.k + j) * p.I;
    const uint16_t* W = p.down + (int64_t)e * p.I * p.H + c;
    float s = 0.f;
#pragma unroll 8
    for (int i = 0; i < p.I; ++i) s = fmaf(h[i], bf16_value(W[(int64_t)i * p.H]), s);
    y = fmaf(p.w[t * p.k + j], s, y);
  }
  if (p.I_s) {
    const float* h = p.h + (int64_t)p.T * p.k * p.I + (int64_t)t * p.I_s;
    float s = 0.f;
#pragma unroll 8
    for (int i = 0; i < p.I_s; ++i) s = fmaf(h[i], bf16_value(p.sh_down[(int64_t)i * p.H + c]), s);
    y += s;
  }
  p.y[(int64_t)t * p.H + c] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
}

}  // namespace

size_t few_experts_workspace_bytes(const FewShape& s) {
  return sizeof(float) * (size_t)(s.T * s.k * s.I + s.T * s.I_s);
}

cudaError_t launch_few_experts(const FewShape& s, const uint16_t* x, const int32_t* ids, const float* w,
                               const FewWeights& weights, uint16_t* y, void* ws, const DeviceInfo& dev,
                               cudaStream_t stream) {
  FewParams p = {};
  p.x = x; p.ids = ids; p.w = w; p.y = y;
  p.gate_up = weights.gate_up; p.down = weights.down;
  p.sh_gate_up = weights.sh_gate_up; p.sh_down = weights.sh_down;
  p.h = static_cast<float*>(ws);
  p.status = dev.status;
  p.T = (int)s.T; p.H = (int)s.H; p.E = (int)s.E; p.k = (int)s.k; p.I = (int)s.I; p.I_s = (int)s.I_s;
  const int64_t wide = std::max(s.I, s.I_s);
  const dim3 rows((unsigned)((wide + kFewThreads - 1) / kFewThreads), (unsigned)(s.T * s.k + (s.I_s ? s.T : 0)));
  const cudaError_t e = launch_pdl(few_gate_up_kernel, rows, dim3(kFewThreads), 0, stream, 1, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(few_down_kernel, dim3((unsigned)((s.H + kFewThreads - 1) / kFewThreads), (unsigned)s.T),
                    dim3(kFewThreads), 0, stream, 1, p);
}

}  // namespace moe
