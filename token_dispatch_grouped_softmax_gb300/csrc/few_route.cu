// The router of a few tokens in one launch: logits, choice and weights.
//
//   z_t = x_t . W_r (+ bias),  then the choice of route_select.cu on z_t
//
// A cluster of 16 blocks takes up to 8 tokens.  Each block reads its share of
// W_r's rows once (fp32, as it lies) and holds the tokens' partial logits;
// the block that chooses for a token adds the 16 parts through distributed
// shared memory.  W_r's bytes and a few dependent
// steps bound it: with one cluster 16 SMs read W_r.  Of 5.6 us for one token of
// H 2048, E 128, 1.8 pass until W_r and x are there, 1.8 in the sums over the
// block and the cluster, 2 in the choice; 8 tokens take 7.7.  Products are fp32 FMAs:
// 8 tokens a read of W_r leave them far below the loads.
#include <algorithm>

#include "kernels.h"
#include "route_choice.cuh"

namespace moe {

namespace {

constexpr int kRouteThreads = 512;
constexpr int kRouteCluster = 16;
constexpr int kRouteRows = 512;     // rows of x in shared memory at a time
constexpr int kRouteBatch = 8;      // rows of W_r a thread has in flight

struct FewRouteParams {
  const uint16_t* x;
  const float* w_router;
  const float *bias, *balance;
  int32_t* ids;
  float* w;
  uint32_t* zero;      // words to clear for the experts' launch
  int zero_words;
  int T, H, E, k;
  int rows;            // of W_r a block reads
  int x_floats;        // room of x's rows, and of a token's logits after them
  int groups, top_groups, per_group;
  int sigmoid, top2, renorm, by_logit;
  float scale;
};

// The k best of a token's experts, by the whole block: every expert counts the
// ones before it.  (One warp that takes the best k times runs through four
// times the code once, and fetching that cost 5 us of the launch's 9.)
// z: the logits; keys: room for the experts' keys, [E] and three more.
__device__ __forceinline__ void choose(const FewRouteParams& p, const float* z, uint32_t* keys, int t) {
  __shared__ uint32_t strength[32];   // of the groups
  __shared__ int chosen_at[32];
  const int tid = threadIdx.x, lane = tid & 31;
  const float neg_inf = __uint_as_float(0xFF800000u);
  const bool grouped = p.top_groups < p.groups;
  float zmax = neg_inf, zsum = 1.f;
  if (!p.sigmoid && !(p.renorm && p.by_logit)) {   // every warp for itself
#pragma unroll 1
    for (int e = lane; e < p.E; e += 32) zmax = fmaxf(zmax, z[e]);
    zmax = warp_max(zmax);
    zsum = 0.f;
#pragma unroll 1
    for (int e = lane; e < p.E; e += 32) zsum += z[e] == neg_inf ? 0.f : expf(z[e] - zmax);
    zsum = warp_sum(zsum);
  }
#pragma unroll 1
  for (int e = tid; e < ((p.E + 3) & ~3); e += kRouteThreads) {
    float v = neg_inf;
    if (e < p.E) {
      v = z[e] + 0.f;   // -0 to +0
      if (!p.by_logit && v != neg_inf)
        v = (p.sigmoid ? sigmoid(v) : expf(v - zmax) / zsum) + (p.balance ? p.balance[e] : 0.f);
    }
    keys[e] = e < p.E ? value_key(v) : 0u;
  }
  __syncthreads();
  if (grouped) {
    if (tid < p.groups) {
      uint32_t m1 = 0, m2 = 0;   // the group's two largest
#pragma unroll 4
      for (int e = tid * p.per_group; e < (tid + 1) * p.per_group; ++e) {
        const uint32_t key = keys[e];
        m2 = max(m2, min(m1, key));
        m1 = max(m1, key);
      }
      strength[tid] = p.top2 && m2 > value_key(neg_inf) ? value_key(key_value(m1) + key_value(m2)) : m1;
    }
    __syncthreads();
#pragma unroll 1
    for (int e = tid; e < p.E; e += kRouteThreads) {
      const int group = e / p.per_group;
      const uint32_t mine = strength[group];
      int before = 0;
#pragma unroll 1
      for (int g = 0; g < p.groups; ++g) before += strength[g] > mine || (strength[g] == mine && g < group);
      if (before >= p.top_groups) keys[e] = 0;
    }
    __syncthreads();
  }
#pragma unroll 1
  for (int e = tid; e < p.E; e += kRouteThreads) {
    const uint32_t key = keys[e];
    if (key == 0) continue;      // of a group that is out
    int before = 0;              // equal keys go to the lower expert
#pragma unroll 2
    for (int i = 0; i < p.E; i += 4) {
      const uint4 q = *reinterpret_cast<const uint4*>(keys + i);
      before += (q.x > key - (i < e)) + (q.y > key - (i + 1 < e)) + (q.z > key - (i + 2 < e)) + (q.w > key - (i + 3 < e));
    }
    if (before < p.k) chosen_at[before] = e;
  }
  __syncthreads();
  if (tid >= 32) return;
  const int chosen = lane < p.k ? chosen_at[lane] : 0;
  float s = 0.f;
  const float zc = lane < p.k ? z[chosen] : neg_inf;
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

// TT tokens a cluster; V consecutive experts a thread (4: E % 4 == 0).
template <int TT, int V>
__global__ void __launch_bounds__(kRouteThreads) few_route_kernel(const __grid_constant__ FewRouteParams p) {
  extern __shared__ float few_route_smem[];
  float* xs = few_route_smem;                    // [rows][TT]
  float* part = xs + p.x_floats;                 // [row groups][TT][E]; the first of them: the block's sums
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, rank = (int)cluster_ctarank();
  const int t0 = (int)(blockIdx.x / kRouteCluster) * TT;
  for (int64_t i = (int64_t)blockIdx.x * kRouteThreads + tid; i < p.zero_words; i += (int64_t)gridDim.x * kRouteThreads) p.zero[i] = 0;
  const int begin = min(rank * p.rows, p.H), end = min(begin + p.rows, p.H);
  const int per_row = (p.E + V - 1) / V;         // threads that read a row (more experts than threads: in turns)
  const int row_groups = max(1, kRouteThreads / per_row);
  const int rg = tid / per_row, c0 = (tid - rg * per_row) * V;
  const int turns = (per_row + kRouteThreads - 1) / kRouteThreads;
  for (int turn = 0; turn < turns; ++turn) {
    const int c = (turns > 1 ? tid * V + turn * kRouteThreads * V : c0);
    const bool mine = c < p.E && (turns > 1 || rg < row_groups);
    float acc[TT][V];
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int v = 0; v < V; ++v) acc[t][v] = 0.f;
    for (int r0 = begin; r0 < end; r0 += kRouteRows) {
      const int n = min(kRouteRows, end - r0);   // multiples of 8
      const float* W = p.w_router + (int64_t)r0 * p.E + c;
      const int first = turns > 1 ? 0 : rg;
      float wv[kRouteBatch][V];
      auto load = [&](int r) {   // rows r, r + row_groups, ..; zeros beyond the share
#pragma unroll
        for (int b = 0; b < kRouteBatch; ++b) {
          const bool in = mine && r + b * row_groups < n;
          if (V == 4) {
            const float4 q = in ? __ldg(reinterpret_cast<const float4*>(W + (int64_t)(r + b * row_groups) * p.E)) : make_float4(0.f, 0.f, 0.f, 0.f);
            wv[b][0] = q.x; wv[b][V > 1 ? 1 : 0] = q.y; wv[b][V > 2 ? 2 : 0] = q.z; wv[b][V > 3 ? 3 : 0] = q.w;
          } else {
            wv[b][0] = in ? __ldg(W + (int64_t)(r + b * row_groups) * p.E) : 0.f;
          }
        }
      };
      load(first);               // on the way while x is laid out
      __syncthreads();
      for (int i = tid; i < n / 8 * TT; i += kRouteThreads) {
        const int t = i / (n / 8), r = (i - t * (n / 8)) * 8;
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = 0.f;
        if (t0 + t < p.T) unpack8(__ldg(reinterpret_cast<const uint4*>(p.x + (int64_t)(t0 + t) * p.H + r0 + r)), v);
#pragma unroll
        for (int q = 0; q < 8; ++q) xs[(r + q) * TT + t] = v[q];
      }
      __syncthreads();
#pragma unroll 1
      for (int r = first; r < n; r += kRouteBatch * row_groups) {
        if (r != first) load(r);
#pragma unroll
        for (int b = 0; b < kRouteBatch; ++b) {
          if (r + b * row_groups >= n) break;
          const float* xr = xs + (r + b * row_groups) * TT;
#pragma unroll
          for (int t = 0; t < TT; ++t)
#pragma unroll
            for (int v = 0; v < V; ++v) acc[t][v] = fmaf(xr[t], wv[b][v], acc[t][v]);
        }
      }
    }
    if (mine) {
      float* out = part + (turns > 1 ? 0 : rg) * TT * p.E + c;
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int v = 0; v < V; ++v) out[t * p.E + v] = acc[t][v];
    }
  }
  __syncthreads();
  for (int i = tid; i < TT * p.E; i += kRouteThreads) {
    float s = part[i];
    for (int g = 1; g < row_groups; ++g) s += part[g * TT * p.E + i];
    part[i] = s;
  }
  cluster_sync_all();
  // token t0 + rank's logits from the cluster's blocks, in order
  const int t = t0 + rank;
  float* z = xs;                                 // [E]; the rows of x are done with
  const bool chooses = rank < TT && t < p.T;
  if (chooses) {
    const uint32_t from = smem_u32(part + rank * p.E);
    for (int e = tid; e < p.E; e += kRouteThreads) {
      float v[kRouteCluster];
#pragma unroll
      for (int r = 0; r < kRouteCluster; ++r) v[r] = ld_shared_cluster_f32(mapa_shared(from + 4 * e, r));
      float s = p.bias ? p.bias[e] : 0.f;
      float sum = v[0];
#pragma unroll
      for (int r = 1; r < kRouteCluster; ++r) sum += v[r];
      z[e] = sum + s;
    }
  }
  cluster_sync_all();   // no block leaves while its sums are read; z is complete too
  if (chooses) choose(p, z, reinterpret_cast<uint32_t*>(part), t);
}

template <int TT, int V>
cudaError_t launch(FewRouteParams p, const DeviceInfo& dev, cudaStream_t stream) {
  const int per_row = (p.E + V - 1) / V, row_groups = std::max(1, kRouteThreads / per_row);
  p.x_floats = std::max(kRouteRows * TT, (p.E + 3) / 4 * 4);
  const size_t smem = sizeof(float) * ((size_t)p.x_floats + (size_t)row_groups * TT * p.E + 4);   // the keys' last four pad
  static std::atomic<int> configured[kMaxDevices] = {};
  if (!configured[dev.ordinal].load()) {
    cudaError_t e = cudaFuncSetAttribute(few_route_kernel<TT, V>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(few_route_kernel<TT, V>, cudaFuncAttributeMaxDynamicSharedMemorySize, 98304);
    if (e != cudaSuccess) return e;
    configured[dev.ordinal].store(1);
  }
  const unsigned clusters = (unsigned)((p.T + TT - 1) / TT);
  return launch_pdl(few_route_kernel<TT, V>, dim3(clusters * kRouteCluster), dim3(kRouteThreads), smem, stream, kRouteCluster, p);
}

template <int TT>
cudaError_t launch(const FewRouteParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  return p.E % 4 == 0 ? launch<TT, 4>(p, dev, stream) : launch<TT, 1>(p, dev, stream);
}

}  // namespace

cudaError_t launch_few_route(const FewShape& s, const uint16_t* x, const float* w_router, const float* bias,
                             const float* balance, const RouteChoice& c, int32_t* ids, float* w, uint32_t* zero,
                             int64_t zero_words, const DeviceInfo& dev, cudaStream_t stream) {
  FewRouteParams p;
  p.x = x; p.w_router = w_router; p.bias = bias; p.balance = balance;
  p.ids = ids; p.w = w; p.zero = zero; p.zero_words = (int)zero_words;
  p.T = (int)s.T; p.H = (int)s.H; p.E = (int)s.E; p.k = (int)s.k;
  p.rows = (int)((s.H / 8 + kRouteCluster - 1) / kRouteCluster * 8);
  p.groups = c.groups; p.top_groups = c.top_groups; p.per_group = (int)(s.E / c.groups);
  p.sigmoid = c.sigmoid; p.renorm = c.renorm; p.scale = c.scale;
  p.top2 = c.top2 && p.per_group > 1;
  p.by_logit = !balance && (c.groups == 1 || !p.top2);   // as moe_route_select: the scores order the experts as the logits do
  if (s.T == 1) return launch<1>(p, dev, stream);
  if (s.T <= 4) return launch<4>(p, dev, stream);
  return launch<8>(p, dev, stream);
}

}  // namespace moe
