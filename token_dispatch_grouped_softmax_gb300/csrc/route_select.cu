// Expert choice from logits: softmax or sigmoid scores, a balance bias that
// only chooses, groups of experts, top-k, renormalised and scaled weights;
// its gradient; and the update of the balance bias.
//
//   s_e = sigmoid(z_e)  or  softmax(z)_e
//   a_e = s_e + b_e, the choice value (z_e itself where no bias and no top2
//         group score needs s: s is increasing in z); -inf for a masked
//         expert (z_e = -inf)
//   A_g = the largest a_e of group g, or the sum of its two largest unmasked
//   ids = the k largest a_e of the top_groups largest A_g, equal values to
//         the lower index;  w_j = scale * s_j (/ sum_i s_i)
//
// One warp per token.  A group's experts lie in L = 32 / 2^ceil(log2 groups)
// consecutive lanes, so that all groups reduce at once by log2(L) butterfly
// steps.  Comparisons are on 32-bit order-preserving keys.
#include <algorithm>

#include "kernels.h"

namespace moe {

namespace {

constexpr int kSelWarps = 8;   // tokens per block

// Order-preserving key of a value: larger value, larger key; +0 and -0 are
// one key; every NaN is above +inf.  0 is below every value's key.
__device__ __forceinline__ uint32_t value_key(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(v + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

// 1 / (1 + exp(-z)), each step rounded to fp32.
__device__ __forceinline__ float sigmoid(float z) { return __frcp_rn(1.f + expf(-z)); }

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ void store_grad(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(uint16_t* p, float v) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// The experts of the k largest keys of the warp, equal keys to the lowest
// expert: slot j's in lane j.  A lane holds the keys of experts e0 + i * step.
// Each round takes the warp's largest leading key.  Up to 8 keys a lane sorts
// them once (stable adjacent exchanges: 28 of them at 8) and its leading key
// is key[0]; above that it scans its keys in each round (a sort grows with NV^2).
template <int NV>
__device__ __forceinline__ int choose(uint32_t (&key)[NV], int e0, int step, int k, int lane) {
  int chosen = 0;
  if constexpr (NV <= 8) {
    int at[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) at[i] = e0 + i * step;
#pragma unroll
    for (int a = 0; a < NV - 1; ++a)
#pragma unroll
      for (int b = NV - 1; b > a; --b) {
        const bool up = key[b] > key[b - 1];
        const uint32_t hi = max(key[b], key[b - 1]), lo = min(key[b], key[b - 1]);
        const int ahi = up ? at[b] : at[b - 1], alo = up ? at[b - 1] : at[b];
        key[b - 1] = hi;
        key[b] = lo;
        at[b - 1] = ahi;
        at[b] = alo;
      }
    for (int j = 0; j < k; ++j) {
      const uint32_t top = __reduce_max_sync(0xffffffffu, key[0]);
      const uint32_t low = __reduce_min_sync(0xffffffffu, key[0] == top ? (uint32_t)at[0] : 0xFFFFFFFFu);
      if ((uint32_t)at[0] == low) {   // this lane held it (experts are distinct)
#pragma unroll
        for (int i = 0; i < NV - 1; ++i) {
          key[i] = key[i + 1];
          at[i] = at[i + 1];
        }
        key[NV - 1] = 0;
        at[NV - 1] = -1;
      }
      if (lane == j) chosen = (int)low;
    }
  } else {
    for (int j = 0; j < k; ++j) {
      uint32_t best = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) best = max(best, key[i]);
      const uint32_t top = __reduce_max_sync(0xffffffffu, best);
      uint32_t mine = 0xFFFFFFFFu;
#pragma unroll
      for (int i = NV - 1; i >= 0; --i)
        if (key[i] == top) mine = (uint32_t)(e0 + i * step);
      const uint32_t low = __reduce_min_sync(0xffffffffu, mine);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if ((uint32_t)(e0 + i * step) == low) key[i] = 0;
      if (lane == j) chosen = (int)low;
    }
  }
  return chosen;
}

struct SelectParams {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* w;
  int T, E, k;
  int groups, top_groups, per_group;   // per_group = E / groups
  int lanes_log2;                      // log2 of the lanes of a group
  int sigmoid, top2, renorm;
  float scale;
};

// NV: values per lane (per_group <= NV << lanes_log2).
template <int NV, typename Z>
__global__ void __launch_bounds__(32 * kSelWarps) route_select_kernel(const SelectParams p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kSelWarps + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const Z* z = static_cast<const Z*>(p.logits) + (int64_t)t * p.E;
  const int L = 1 << p.lanes_log2;
  const int g = lane >> p.lanes_log2, l = lane & (L - 1);
  const float neg_inf = __uint_as_float(0xFF800000u);

  float v[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int r = l + i * L;
    v[i] = (g < p.groups && r < p.per_group) ? load_logit(z + g * p.per_group + r) : neg_inf;
  }
  // softmax statistics over the whole row
  const bool by_score = p.bias || (p.top2 && p.groups > 1);
  float zmax = 0.f, zsum = 1.f;
  if (!p.sigmoid && (by_score || !p.renorm)) {
    zmax = neg_inf;
#pragma unroll
    for (int i = 0; i < NV; ++i) zmax = fmaxf(zmax, v[i]);
    zmax = warp_max(zmax);
    zsum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) zsum += v[i] == neg_inf ? 0.f : expf(v[i] - zmax);
    zsum = warp_sum(zsum);
  }
  const int e0 = g * p.per_group + l;   // value i is expert e0 + i * L
  uint32_t key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    key[i] = 0;
    if (g < p.groups && l + i * L < p.per_group) {
      float a = v[i];
      if (by_score && a != neg_inf) {
        a = p.sigmoid ? sigmoid(a) : expf(a - zmax) / zsum;
        if (p.bias) a += p.bias[e0 + i * L];
      }
      key[i] = value_key(a);
    }
  }
  if (p.top_groups < p.groups) {
    uint32_t m1 = 0, m2 = 0;   // the lane's two largest
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      m2 = max(m2, min(m1, key[i]));
      m1 = max(m1, key[i]);
    }
    for (int o = 1; o < L; o <<= 1) {
      const uint32_t o1 = __shfl_xor_sync(0xffffffffu, m1, o), o2 = __shfl_xor_sync(0xffffffffu, m2, o);
      m2 = max(max(m2, o2), min(m1, o1));
      m1 = max(m1, o1);
    }
    uint32_t mine = m1;
    if (p.top2 && g < p.groups) {   // masked experts (-inf, or none) add nothing
      const uint32_t masked = value_key(neg_inf);
      if (m2 > masked) mine = value_key(key_value(m1) + key_value(m2));
    }
    int rank = 0;
    for (int q = 0; q < p.groups; ++q) {
      const uint32_t other = __shfl_sync(0xffffffffu, mine, q << p.lanes_log2);
      rank += other > mine || (other == mine && q < g);
    }
    if (rank >= p.top_groups) {
#pragma unroll
      for (int i = 0; i < NV; ++i) key[i] = 0;
    }
  }
  const int chosen = choose<NV>(key, e0, L, p.k, lane);
  // the chosen scores, from the logits again
  float s = 0.f;
  const float zc = lane < p.k ? load_logit(z + chosen) : neg_inf;
  if (p.sigmoid) {
    s = lane < p.k ? sigmoid(zc) : 0.f;
  } else {
    const float m = p.renorm ? warp_max(zc) : zmax;   // renormalised: the row's sum cancels
    s = zc == neg_inf ? 0.f : expf(zc - m) / (p.renorm ? 1.f : zsum);
  }
  if (p.renorm) {
    const float sum = warp_sum(s);
    s = sum == 0.f ? 0.f : s / sum;
  }
  if (lane < p.k) {
    p.ids[(int64_t)t * p.k + lane] = chosen;
    p.w[(int64_t)t * p.k + lane] = p.scale * s;
  }
}

struct SelectBwdParams {
  const float* dw_part;
  const int32_t* row_map;
  const void* logits;
  const int32_t* ids;
  void* d_logits;
  float* dw;
  uint32_t* status;
  int T, E, k, nparts;
  int sigmoid, renorm;
  float scale;
};

// One warp per token: lane j < k holds slot j.  The row is filled (zeros, or
// the dense part of the softmax without renormalisation), then the chosen
// elements are written over it.
template <typename Z>
__global__ void __launch_bounds__(32 * kSelWarps) route_select_bwd_kernel(const SelectBwdParams p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kSelWarps + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const Z* z = static_cast<const Z*>(p.logits) + (int64_t)t * p.E;
  Z* dz = static_cast<Z*>(p.d_logits) + (int64_t)t * p.E;
  const float neg_inf = __uint_as_float(0xFF800000u);
  float dwj = 0.f, zc = neg_inf;
  int e = -1;
  if (lane < p.k) {
    const int64_t i = (int64_t)t * p.k + lane;
    e = p.ids[i];
    if (e < 0 || e >= p.E) {   // no expert: report, and leave the slot out
      report_status(p.status, kStatusDevice, kKernRouteSelect, 1);
      e = -1;
    }
    int64_t row = i;
    if (p.row_map) {
      row = p.row_map[i];
      if (row < 0 || row >= (int64_t)p.T * p.k) {
        report_status(p.status, kStatusDevice, kKernRouteSelect, 2);
        row = 0;
      }
    }
    for (int n = 0; n < p.nparts; ++n) dwj += p.dw_part[row * p.nparts + n];   // fixed order
    if (p.dw) p.dw[i] = dwj;
    if (e >= 0) zc = load_logit(z + e);
  }
  float d = 0.f;        // the chosen element's gradient
  if (p.renorm || p.sigmoid) {
    for (int c = lane; c < p.E; c += 32) store_grad(dz + c, 0.f);
    float u;            // the slot's score, renormalised when asked
    if (p.sigmoid) {
      u = lane < p.k ? sigmoid(zc) : 0.f;
    } else {
      const float m = warp_max(zc);
      u = zc == neg_inf ? 0.f : expf(zc - m);
    }
    float mean = 0.f;
    if (p.renorm) {
      const float sum = warp_sum(u);
      u = sum == 0.f ? 0.f : u / sum;
      mean = warp_sum(u * dwj);
    }
    d = p.scale * u * (dwj - mean);
    if (p.sigmoid) d *= sigmoid(-zc);   // 1 - s without cancellation
  } else {
    float zmax = neg_inf;
    for (int c = lane; c < p.E; c += 32) zmax = fmaxf(zmax, load_logit(z + c));
    zmax = warp_max(zmax);
    float zsum = 0.f;
    for (int c = lane; c < p.E; c += 32) {
      const float v = load_logit(z + c);
      zsum += v == neg_inf ? 0.f : expf(v - zmax);
    }
    zsum = warp_sum(zsum);
    const float pj = zc == neg_inf ? 0.f : expf(zc - zmax) / zsum;
    const float mean = warp_sum(pj * dwj);
    for (int c = lane; c < p.E; c += 32) {
      const float v = load_logit(z + c);
      store_grad(dz + c, v == neg_inf ? 0.f : p.scale * (expf(v - zmax) / zsum) * -mean);
    }
    d = p.scale * pj * (dwj - mean);
  }
  __syncwarp();   // orders the row's fill before the chosen elements
  if (e >= 0) store_grad(dz + e, d);
}

// b_e += rate * sign(mean load - load_e), decided in integers: the sign of
// sum(counts) - E * counts_e.
__global__ void __launch_bounds__(kMaxExperts) route_balance_bias_kernel(const float* __restrict__ bias,
                                                                         const int32_t* __restrict__ counts, int E,
                                                                         float rate, float* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  __shared__ unsigned long long total;
  const int e = threadIdx.x;
  if (e == 0) total = 0;
  __syncthreads();
  const long long n = e < E ? counts[e] : 0;
  if (e < E) atomicAdd(&total, (unsigned long long)n);   // integers: the order does not matter
  __syncthreads();
  if (e < E) {
    const long long d = (long long)total - (long long)E * n;
    out[e] = bias[e] + (d > 0 ? rate : d < 0 ? -rate : 0.f);
  }
}

template <int NV>
cudaError_t launch_select_nv(const SelectParams& p, bool bf16, cudaStream_t stream) {
  const dim3 grid((unsigned)((p.T + kSelWarps - 1) / kSelWarps)), block(32 * kSelWarps);
  return bf16 ? launch_pdl(route_select_kernel<NV, uint16_t>, grid, block, 0, stream, 1, p)
              : launch_pdl(route_select_kernel<NV, float>, grid, block, 0, stream, 1, p);
}

}  // namespace

cudaError_t launch_route_select(const void* logits, bool bf16, const float* bias, int64_t T, int64_t E, int64_t k,
                                const RouteChoice& c, int32_t* ids, float* w, cudaStream_t stream) {
  SelectParams p;
  p.logits = logits;
  p.bias = bias;
  p.ids = ids;
  p.w = w;
  p.T = (int)T;
  p.E = (int)E;
  p.k = (int)k;
  p.groups = c.groups;
  p.top_groups = c.top_groups;
  p.per_group = (int)(E / c.groups);
  int span = 1;
  while (span < c.groups) span <<= 1;
  p.lanes_log2 = 0;
  while ((span << p.lanes_log2) < 32) ++p.lanes_log2;
  p.sigmoid = c.sigmoid;
  p.top2 = c.top2 && p.per_group > 1;
  p.renorm = c.renorm;
  p.scale = c.scale;
  const int nv = (p.per_group + (1 << p.lanes_log2) - 1) >> p.lanes_log2;
  if (nv <= 1) return launch_select_nv<1>(p, bf16, stream);
  if (nv <= 2) return launch_select_nv<2>(p, bf16, stream);
  if (nv <= 4) return launch_select_nv<4>(p, bf16, stream);
  if (nv <= 8) return launch_select_nv<8>(p, bf16, stream);
  if (nv <= 16) return launch_select_nv<16>(p, bf16, stream);
  if (nv <= 32) return launch_select_nv<32>(p, bf16, stream);
  return launch_select_nv<64>(p, bf16, stream);
}

cudaError_t launch_route_select_bwd(const float* dw_part, int nparts, const int32_t* row_map, const void* logits,
                                    bool bf16, const int32_t* ids, int64_t T, int64_t E, int64_t k,
                                    const RouteChoice& c, void* d_logits, float* dw, uint32_t* status,
                                    cudaStream_t stream) {
  const SelectBwdParams p{dw_part, row_map, logits, ids, d_logits, dw, status, (int)T, (int)E, (int)k, nparts,
                          c.sigmoid, c.renorm, c.scale};
  const dim3 grid((unsigned)((T + kSelWarps - 1) / kSelWarps)), block(32 * kSelWarps);
  return bf16 ? launch_pdl(route_select_bwd_kernel<uint16_t>, grid, block, 0, stream, 1, p)
              : launch_pdl(route_select_bwd_kernel<float>, grid, block, 0, stream, 1, p);
}

cudaError_t launch_route_balance_bias(const float* bias, const int32_t* counts, int64_t E, float rate, float* out,
                                      cudaStream_t stream) {
  return launch_pdl(route_balance_bias_kernel, dim3(1), dim3((unsigned)((E + 31) / 32 * 32)), 0, stream, 1, bias,
                    counts, (int)E, rate, out);
}

}  // namespace moe
