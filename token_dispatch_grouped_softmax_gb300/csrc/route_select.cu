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

// Order-preserving key of the result of an fp32 addition: larger value,
// larger key; NaN (an addition's NaN is positive) above +inf.  0 is below
// every value's key.
__device__ __forceinline__ uint32_t value_key(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

// 1 / d rounded to nearest, for 1 <= d < 2^120: a Newton step in fused
// multiply-adds from an approximation within a unit of the last place
// (Markstein, IBM J. Res. Dev. 34, 1990).  A GPU test compares it with the
// quotient for the d of every fp32 logit.
__device__ __forceinline__ float reciprocal(float d) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return fmaf(r, fmaf(-d, r, 1.f), r);
}

// 1 / (1 + exp(-z)), each step rounded to fp32.  NEAR: z >= kNearest.
constexpr float kNearest = -80.f;
template <bool NEAR = false>
__device__ __forceinline__ float sigmoid(float z) {
  const float d = 1.f + expf(-z);
  return NEAR || d <= 0x1p119f ? reciprocal(d) : __frcp_rn(d);
}

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ void store_grad(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(uint16_t* p, float v) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

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

// Four consecutive logits (16 or 8 bytes).
__device__ __forceinline__ void load_logits4(const float* p, float* v) {
  const float4 q = __ldg(reinterpret_cast<const float4*>(p));
  v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
}
__device__ __forceinline__ void load_logits4(const uint16_t* p, float* v) {
  const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
  v[0] = bf16_lo(q.x); v[1] = bf16_hi(q.x); v[2] = bf16_lo(q.y); v[3] = bf16_hi(q.y);
}

// Drops the keys of the groups that are out, finds the candidates and gathers
// up to 32 of them, (key, expert) in `out`; returns their number.
template <int NV, typename ExpertOf>
__device__ __forceinline__ int find_candidates(const SelectParams& p, uint32_t (&key)[NV], int g, int l, int lane,
                                               ExpertOf expert_of, uint2* out) {
  const int L = 1 << p.lanes_log2;
  const uint32_t masked = value_key(__uint_as_float(0xFF800000u));
  uint32_t lead = 0, next = 0;   // the lane's two largest
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    next = max(next, min(lead, key[i]));
    lead = max(lead, key[i]);
  }
  if (p.top_groups < p.groups) {
    uint32_t m1 = lead, m2 = next;   // the group's two largest
    for (int o = 1; o < L; o <<= 1) {
      const uint32_t o1 = __shfl_xor_sync(0xffffffffu, m1, o), o2 = __shfl_xor_sync(0xffffffffu, m2, o);
      m2 = max(max(m2, o2), min(m1, o1));
      m1 = max(m1, o1);
    }
    uint32_t mine = m1;
    if (p.top2 && g < p.groups && m2 > masked)   // masked experts (-inf, or none) add nothing
      mine = value_key(key_value(m1) + key_value(m2));
    int rank = 0;   // groups before this one: the group's lanes share the comparisons out
    for (int q0 = 0; q0 < p.groups; q0 += L) {
      const int q = min(q0 + l, p.groups - 1);
      const uint32_t other = __shfl_sync(0xffffffffu, mine, q << p.lanes_log2);
      rank += q == q0 + l && (other > mine || (other == mine && q < g));
    }
    for (int o = 1; o < L; o <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (rank >= p.top_groups) {
      lead = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) key[i] = 0;
    }
  }
  if (NV == 1) return 0;   // one candidate a lane as it is
  uint32_t tau = 1;
  for (int j = 0; j < p.k; ++j) {
    tau = max(__reduce_max_sync(0xffffffffu, lead), 1u);
    if (lead >= tau) lead = 0;
  }
  int n = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const bool in = key[i] >= tau;
    const uint32_t who = __ballot_sync(0xffffffffu, in);
    const int at = n + __popc(who & ((1u << lane) - 1u));
    if (in && at < 32) out[at] = make_uint2(key[i], expert_of(i));
    n += __popc(who);
  }
  __syncwarp();
  return n;
}

// NV values per lane, of the lane's group; value i is member l + i L of the
// group (l the lane's place among the group's L lanes), or with QUADS member
// 4 l + i % 4 + 4 L (i / 4): vectors of four.  Either way a lane's experts
// increase with i.
//
// The k best: the k-th largest of the lanes' largest keys is at most the k-th
// largest key, so only keys from it on can be chosen, little more than k of
// them.  They are gathered one to a lane, and k rounds of two warp reductions
// (the largest key, the lowest expert that has it) put them in order.  Where
// more than 32 pass (large k, many equal keys) the rounds scan every key.
// The instructions of a token bound it: 13.9 us for 16384 tokens at E = 256
// with 8 groups (15.6 with the library's reciprocal, 21.3 with a sort of each
// lane's 8 keys, 23.1 with approximate sigmoids to find the candidates), and
// 3.4 us for 4096 tokens of E = 128 by softmax.
enum { kByLogit, kBySigmoid, kBySoftmax };   // what chooses

template <int NV, bool QUADS, int MODE, typename Z>
__global__ void __launch_bounds__(32 * kSelWarps) route_select_kernel(const SelectParams p) {
  __shared__ uint2 gathered[kSelWarps][NV > 1 ? 32 : 1];   // (key, expert)
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kSelWarps + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const Z* z = static_cast<const Z*>(p.logits) + (int64_t)t * p.E;
  const int L = 1 << p.lanes_log2;
  const int g = lane >> p.lanes_log2, l = lane & (L - 1);
  const float neg_inf = __uint_as_float(0xFF800000u);
  const int first = g * p.per_group + (QUADS ? 4 * l : l);
  const int members = g < p.groups ? p.per_group - (QUADS ? 4 * l : l) : 0;   // of the group from `first` on
  auto step = [&](int i) { return QUADS ? (i >> 2) * 4 * L + (i & 3) : i * L; };   // of value i from `first`

  float v[NV];
  if (QUADS) {
#pragma unroll
    for (int i = 0; i < NV; i += 4) {
      v[i] = v[i + 1] = v[i + 2] = v[i + 3] = neg_inf;
      if (step(i) < members) load_logits4(z + first + step(i), v + i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = step(i) < members ? load_logit(z + first + step(i)) : neg_inf;
  }
  // softmax statistics over the whole row
  float zmax = 0.f, zsum = 1.f;
  if (MODE == kBySoftmax || (!p.sigmoid && !p.renorm)) {
    zmax = neg_inf;
#pragma unroll
    for (int i = 0; i < NV; ++i) zmax = fmaxf(zmax, v[i]);
    zmax = warp_max(zmax);
    zsum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) zsum += v[i] == neg_inf ? 0.f : expf(v[i] - zmax);
    zsum = warp_sum(zsum);
  }
  float b[NV];   // what is added to the score
#pragma unroll
  for (int i = 0; i < NV; ++i) b[i] = 0.f;
  if (MODE != kByLogit && p.bias) {
#pragma unroll
    for (int i = 0; i < NV; i += QUADS ? 4 : 1)
      if (step(i) < members) {
        if (QUADS) load_logits4(p.bias + first + step(i), b + i);
        else b[i] = __ldg(p.bias + first + step(i));
      }
  }
  // the key of the value that chooses
  auto choice_key = [&](float zi, float s, float bi) {
    if (MODE == kByLogit) return value_key(zi + 0.f);   // -0 to +0
    return zi == neg_inf ? value_key(neg_inf) : value_key(s + bi);
  };
  uint32_t key[NV];
  if (MODE == kBySigmoid) {
    float low = v[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) low = fminf(low, v[i]);
    if (__all_sync(0xffffffffu, low >= kNearest)) {   // no masked expert, nor a place without one
#pragma unroll
      for (int i = 0; i < NV; ++i) key[i] = value_key(sigmoid<true>(v[i]) + b[i]);
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) key[i] = step(i) < members ? choice_key(v[i], sigmoid(v[i]), b[i]) : 0u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) key[i] = step(i) < members ? choice_key(v[i], expf(v[i] - zmax) / zsum, b[i]) : 0u;
  }
  uint2* mine = gathered[threadIdx.x >> 5];
  const int total = find_candidates<NV>(p, key, g, l, lane, [&](int i) { return (uint32_t)(first + step(i)); }, mine);
  const bool gather = NV > 1 && total <= 32;
  uint32_t one = key[0], expert = (uint32_t)first;   // a lane's candidate
  if (gather) {
    one = 0;
    if (lane < total) {
      one = mine[lane].x;
      expert = mine[lane].y;
    }
  }
  // k rounds: the warp's largest key, equal keys to the lowest expert
  int chosen = 0;
  if (gather || NV == 1) {
    for (int j = 0; j < p.k; ++j) {
      const uint32_t top = __reduce_max_sync(0xffffffffu, one);
      const uint32_t low = __reduce_min_sync(0xffffffffu, one == top ? expert : 0xFFFFFFFFu);
      if (expert == low) one = 0;
      if (lane == j) chosen = (int)low;
    }
  } else {
    for (int j = 0; j < p.k; ++j) {
      uint32_t best = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) best = max(best, key[i]);
      const uint32_t top = __reduce_max_sync(0xffffffffu, best);
      uint32_t mine = 0xFFFFFFFFu;
#pragma unroll
      for (int i = NV - 1; i >= 0; --i)
        if (key[i] == top) mine = (uint32_t)(first + step(i));
      const uint32_t low = __reduce_min_sync(0xffffffffu, mine);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (mine == low && (uint32_t)(first + step(i)) == low) key[i] = 0;
      if (lane == j) chosen = (int)low;
    }
  }
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

// A lane's NV consecutive-by-vector elements of a row: element i of lane l is
// V (l + 32 (i / V)) + i % V, in vectors of V elements of 16 bytes; or, with
// V 1, l + 32 i.
template <int V>
__device__ __forceinline__ int row_element(int lane, int i) {
  return V * (lane + 32 * (i / V)) + i % V;
}
template <int V>
__device__ __forceinline__ void load_vec(const float* p, float* v) {
  if (V == 4) load_logits4(p, v);
  else v[0] = *p;
}
template <int V>
__device__ __forceinline__ void load_vec(const uint16_t* p, float* v) {
  if (V == 8) unpack8(__ldg(reinterpret_cast<const uint4*>(p)), v);
  else v[0] = load_logit(p);
}
template <int V>
__device__ __forceinline__ void store_vec(float* p, const float* v) {
  if (V == 4) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  else *p = v[0];
}
template <int V>
__device__ __forceinline__ void store_vec(uint16_t* p, const float* v) {
  if (V == 8) *reinterpret_cast<uint4*>(p) = pack8(v);
  else store_grad(p, v[0]);
}

// One warp per token: lane j < k holds slot j.  The row is filled (zeros, or
// the dense part of the softmax without renormalisation, whose row stays in
// registers between its maximum, its sum and its gradient), then the chosen
// elements are written over it: bound by the write of d_logits (8192 tokens
// of E 256, fp32: 5.8 us from cold caches, launch included; dense, 8191 of
// E 128 in bf16: 6.3).
// NV >= E / 32 elements a lane for the dense form; NV 0: the other forms.
template <int NV, int V, typename Z>
__global__ void __launch_bounds__(32 * kSelWarps) route_select_bwd_kernel(const SelectBwdParams p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kSelWarps + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const Z* z = static_cast<const Z*>(p.logits) + (int64_t)t * p.E;
  Z* dz = static_cast<Z*>(p.d_logits) + (int64_t)t * p.E;
  const float neg_inf = __uint_as_float(0xFF800000u);
  constexpr int N = NV > 0 ? NV : 1;
  float v[N];
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < N; i += V) {
#pragma unroll
      for (int c = 0; c < V; ++c) v[i + c] = neg_inf;
      if (row_element<V>(lane, i) < p.E) load_vec<V>(z + row_element<V>(lane, i), v + i);
    }
  } else {
    float zero[V];
#pragma unroll
    for (int c = 0; c < V; ++c) zero[c] = 0.f;
    for (int c = V * lane; c < p.E; c += 32 * V) store_vec<V>(dz + c, zero);
  }
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
  float d;        // the chosen element's gradient
  if constexpr (NV == 0) {
    float u;      // the slot's score, renormalised when asked
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
#pragma unroll
    for (int i = 0; i < N; ++i) zmax = fmaxf(zmax, v[i]);
    zmax = warp_max(zmax);
    float zsum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = v[i] == neg_inf ? 0.f : expf(v[i] - zmax);
      zsum += v[i];
    }
    zsum = warp_sum(zsum);
    const float pj = zc == neg_inf ? 0.f : expf(zc - zmax) / zsum;
    const float mean = warp_sum(pj * dwj);
    const float f = zsum == 0.f ? 0.f : p.scale * -mean / zsum;   // a row of masked experts: 0
#pragma unroll
    for (int i = 0; i < N; i += V) {
#pragma unroll
      for (int c = 0; c < V; ++c) v[i + c] *= f;
      if (row_element<V>(lane, i) < p.E) store_vec<V>(dz + row_element<V>(lane, i), v + i);
    }
    d = p.scale * pj * (dwj - mean);
  }
  __syncwarp();   // orders the row's fill before the chosen elements
  if (e >= 0) store_grad(dz + e, d);
}

// b_e += rate * sign(mean load - load_e), decided in integers: the sign of
// sum(counts) - E * counts_e.  A launch's latency (3.3 us from cold caches).
// out may be bias.
__global__ void __launch_bounds__(kMaxExperts) route_balance_bias_kernel(const float* bias,
                                                                         const int32_t* __restrict__ counts, int E,
                                                                         float rate, float* out) {
  pdl_wait();
  pdl_trigger();
  __shared__ long long part[32];
  const int e = threadIdx.x;
  const long long n = e < E ? counts[e] : 0;
  long long sum = n;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((e & 31) == 0) part[e >> 5] = sum;
  __syncthreads();
  if (e < E) {
    long long total = 0;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) total += part[w];
    const long long d = total - (long long)E * n;
    out[e] = bias[e] + (d > 0 ? rate : d < 0 ? -rate : 0.f);
  }
}

template <int NV, bool QUADS, int MODE>
cudaError_t launch_select_mode(const SelectParams& p, bool bf16, cudaStream_t stream) {
  const dim3 grid((unsigned)((p.T + kSelWarps - 1) / kSelWarps)), block(32 * kSelWarps);
  return bf16 ? launch_pdl(route_select_kernel<NV, QUADS, MODE, uint16_t>, grid, block, 0, stream, 1, p)
              : launch_pdl(route_select_kernel<NV, QUADS, MODE, float>, grid, block, 0, stream, 1, p);
}

template <int NV, bool QUADS>
cudaError_t launch_select_nv(const SelectParams& p, bool bf16, cudaStream_t stream) {
  if (!p.bias && !(p.top2 && p.groups > 1)) return launch_select_mode<NV, QUADS, kByLogit>(p, bf16, stream);
  return p.sigmoid ? launch_select_mode<NV, QUADS, kBySigmoid>(p, bf16, stream)
                   : launch_select_mode<NV, QUADS, kBySoftmax>(p, bf16, stream);
}

template <int V, typename Z>
cudaError_t launch_bwd_v(const SelectBwdParams& p, cudaStream_t stream) {
  const dim3 grid((unsigned)((p.T + kSelWarps - 1) / kSelWarps)), block(32 * kSelWarps);
  if (p.renorm || p.sigmoid) return launch_pdl(route_select_bwd_kernel<0, V, Z>, grid, block, 0, stream, 1, p);
  const int nv = (p.E + 32 * V - 1) / (32 * V) * V;
  if constexpr (V == 1) {
    if (nv <= 1) return launch_pdl(route_select_bwd_kernel<1, V, Z>, grid, block, 0, stream, 1, p);
    if (nv <= 2) return launch_pdl(route_select_bwd_kernel<2, V, Z>, grid, block, 0, stream, 1, p);
  }
  if constexpr (V <= 4)
    if (nv <= 4) return launch_pdl(route_select_bwd_kernel<4, V, Z>, grid, block, 0, stream, 1, p);
  if (nv <= 8) return launch_pdl(route_select_bwd_kernel<8, V, Z>, grid, block, 0, stream, 1, p);
  if (nv <= 16) return launch_pdl(route_select_bwd_kernel<16, V, Z>, grid, block, 0, stream, 1, p);
  return launch_pdl(route_select_bwd_kernel<32, V, Z>, grid, block, 0, stream, 1, p);
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
  // vectors of four where a group gives each of its lanes at least one, and
  // every row and group starts on one
  const int L = 1 << p.lanes_log2;
  if (p.per_group % 4 == 0 && p.per_group >= 4 * L) {
    const int quads = (p.per_group / 4 + L - 1) / L;
    if (quads <= 1) return launch_select_nv<4, true>(p, bf16, stream);
    if (quads <= 2) return launch_select_nv<8, true>(p, bf16, stream);
    if (quads <= 4) return launch_select_nv<16, true>(p, bf16, stream);
    if (quads <= 8) return launch_select_nv<32, true>(p, bf16, stream);
    return launch_select_nv<64, true>(p, bf16, stream);
  }
  const int nv = (p.per_group + L - 1) / L;
  if (nv <= 1) return launch_select_nv<1, false>(p, bf16, stream);
  if (nv <= 2) return launch_select_nv<2, false>(p, bf16, stream);
  if (nv <= 4) return launch_select_nv<4, false>(p, bf16, stream);
  if (nv <= 8) return launch_select_nv<8, false>(p, bf16, stream);
  if (nv <= 16) return launch_select_nv<16, false>(p, bf16, stream);
  if (nv <= 32) return launch_select_nv<32, false>(p, bf16, stream);
  return launch_select_nv<64, false>(p, bf16, stream);
}

cudaError_t launch_route_select_bwd(const float* dw_part, int nparts, const int32_t* row_map, const void* logits,
                                    bool bf16, const int32_t* ids, int64_t T, int64_t E, int64_t k,
                                    const RouteChoice& c, void* d_logits, float* dw, uint32_t* status,
                                    cudaStream_t stream) {
  const SelectBwdParams p{dw_part, row_map, logits, ids, d_logits, dw, status, (int)T, (int)E, (int)k, nparts,
                          c.sigmoid, c.renorm, c.scale};
  // rows in 16-byte vectors where every row starts on one
  if (bf16) return E % 8 == 0 ? launch_bwd_v<8, uint16_t>(p, stream) : launch_bwd_v<1, uint16_t>(p, stream);
  return E % 4 == 0 ? launch_bwd_v<4, float>(p, stream) : launch_bwd_v<1, float>(p, stream);
}

cudaError_t launch_route_balance_bias(const float* bias, const int32_t* counts, int64_t E, float rate, float* out,
                                      cudaStream_t stream) {
  return launch_pdl(route_balance_bias_kernel, dim3(1), dim3((unsigned)((E + 31) / 32 * 32)), 0, stream, 1, bias,
                    counts, (int)E, rate, out);
}

}  // namespace moe
