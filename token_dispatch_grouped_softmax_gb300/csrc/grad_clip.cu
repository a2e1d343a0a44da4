// The 2-norm over a list of gradients, and the gradients scaled so that it is
// at most max_norm:
//
//   norm = sqrt(sum_i sum_e g_i[e]^2),  out_i = g_i min(1, max_norm / (norm + eps))
//
// The tensors are cut into chunks of 2^14 elements that the blocks take in
// turn, whatever tensor they belong to: one launch for a list of hundreds.
// A thread sums the squares of its 64 elements of a chunk in fp32 and adds
// the sum to a double; where that sum leaves the range in which fp32 squares
// lose nothing that counts (values beyond 2^63, or all of them below 2^-40 or
// so), it squares its elements again in double.  The blocks' sums add up in
// a fixed order.
//
// The bytes bound both kernels, read once for the norm and once more to be
// scaled: 604 M elements in bf16, 1.2 GB, 175 us for the norm (6.9 TB/s) and
// 372 to scale (6.5 TB/s).  The chunks go to the blocks in turn, so that all of
// them work in one region (a range to each block: 437 us to scale).
#include <algorithm>

#include "kernels.h"

namespace moe {

namespace {

constexpr int kClipThreads = 256;
constexpr int kClipChunk = 1 << 14;      // elements
constexpr int kClipTensors = 512;        // of one launch: 17 KB of parameters
constexpr int kClipBlocks = 8 * 152;     // eight to an SM of GB300; fixed, as the order of the sums goes by it

struct ClipList {
  const void* src[kClipTensors];
  void* dst[kClipTensors];
  int64_t size[kClipTensors];            // elements; fp32 tensors as ~size
  int first_chunk[kClipTensors + 1];
  // the tensor of a block's first chunk, from where it walks on (a search among
  // the parameters is a chain of misses in the constant cache: 97 small tensors
  // took 11 us to scale)
  uint16_t start[kClipBlocks];
  int n;
};

struct ClipChunk {
  int tensor;
  int64_t begin, end;    // elements
  bool f32;
};

// A tensor's elements before its first 16-byte boundary.
__device__ __host__ __forceinline__ int clip_head(const void* p, bool f32) {
  return (int)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (f32 ? 4 : 2);
}

// Chunk `at` of the list, of tensor `tensor`: chunk i of a tensor holds
// elements head + 2^14 i on, and the first the head too, so that every chunk's
// vectors are aligned.
__device__ __forceinline__ ClipChunk clip_chunk(const ClipList& list, int tensor, int at) {
  ClipChunk c;
  c.tensor = tensor;
  int64_t size = list.size[tensor];
  c.f32 = size < 0;
  if (c.f32) size = ~size;
  const int i = at - list.first_chunk[tensor];
  const int head = clip_head(list.src[tensor], c.f32);
  c.begin = i == 0 ? 0 : head + (int64_t)i * kClipChunk;
  c.end = min(head + (int64_t)(i + 1) * kClipChunk, size);
  return c;
}

__device__ __forceinline__ void square(float v, float& sum, uint32_t& bits) {
  sum = fmaf(v, v, sum);
  bits |= __float_as_uint(v) & 0x7FFFFFFFu;
}

__device__ __forceinline__ float element(const void* p, bool f32, int64_t i) {
  return f32 ? static_cast<const float*>(p)[i] : __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
}

// Calls f(i) for the thread's elements before the chunk's first and after its
// last whole vector of V elements, and vec(i) for its vectors.
template <int V, typename F, typename Vec>
__device__ __forceinline__ void clip_visit(const ClipChunk& c, int head, F f, Vec vec) {
  int64_t begin = c.begin;
  if (begin == 0) {
    begin = min((int64_t)head, c.end);
    if ((int64_t)threadIdx.x < begin) f((int64_t)threadIdx.x);
  }
  const int vectors = (int)((c.end - begin) / V);
#pragma unroll 4
  for (int i = threadIdx.x; i < vectors; i += kClipThreads) vec(begin + (int64_t)i * V);
  const int64_t tail = begin + (int64_t)vectors * V + threadIdx.x;
  if (tail < c.end) f(tail);
}

__global__ void __launch_bounds__(kClipThreads) grad_norm_kernel(const __grid_constant__ ClipList list, double* parts) {
  __shared__ double warps[kClipThreads / 32];
  pdl_wait();
  pdl_trigger();
  double total = 0.0;
  const int chunks = list.first_chunk[list.n];
  int tensor = list.start[blockIdx.x];
  for (int at = blockIdx.x; at < chunks; at += gridDim.x) {
    while (at >= list.first_chunk[tensor + 1]) ++tensor;
    const ClipChunk c = clip_chunk(list, tensor, at);
    const void* src = list.src[c.tensor];
    const int head = clip_head(src, c.f32);
    float s = 0.f;
    uint32_t bits = 0;
    auto one = [&](int64_t i) { square(element(src, c.f32, i), s, bits); };
    if (c.f32) {
      clip_visit<4>(c, head, one, [&](int64_t i) {
        const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(src) + i));
        square(v.x, s, bits); square(v.y, s, bits); square(v.z, s, bits); square(v.w, s, bits);
      });
    } else {
      clip_visit<8>(c, head, one, [&](int64_t i) {
        float v[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(src) + i)), v);
#pragma unroll
        for (int k = 0; k < 8; ++k) square(v[k], s, bits);
      });
    }
    if (bits != 0 && !(s >= 0x1p-80f && s < 0x1p127f)) {   // NaN too
      double d = 0.0;
      auto again = [&](int64_t i) {
        const double v = element(src, c.f32, i);
        d += v * v;
      };
      if (c.f32) clip_visit<4>(c, head, again, [&](int64_t i) { for (int k = 0; k < 4; ++k) again(i + k); });
      else clip_visit<8>(c, head, again, [&](int64_t i) { for (int k = 0; k < 8; ++k) again(i + k); });
      total += d;
    } else {
      total += s;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = total;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kClipThreads / 32; ++i) total += warps[i];
    parts[blockIdx.x] = total;
  }
}

// The sum of the blocks' sums, the same bits in every block that computes it.
__device__ __forceinline__ double clip_sum(const double* parts, int n) {
  __shared__ double warps[kClipThreads / 32];
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kClipThreads) s += parts[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0.0;
  for (int i = 0; i < kClipThreads / 32; ++i) s += warps[i];
  return s;
}

__global__ void __launch_bounds__(kClipThreads) grad_norm_sum_kernel(const double* parts, int n, float* norm) {
  pdl_wait();
  pdl_trigger();
  const double s = clip_sum(parts, n);
  if (threadIdx.x == 0) *norm = (float)sqrt(s);
}

__global__ void __launch_bounds__(kClipThreads) grad_scale_kernel(const __grid_constant__ ClipList list, const double* parts,
                                                                  int n, float max_norm, float eps, float* norm) {
  pdl_wait();
  pdl_trigger();
  __shared__ float2 scale_step;
  const double sum = clip_sum(parts, n);
  if (threadIdx.x == 0) {
    const double total = sqrt(sum);
    if (norm && blockIdx.x == 0) *norm = (float)total;
    double factor = max_norm / (total + eps);
    if (factor > 1.0) factor = 1.0;   // NaN stays
    // a factor below fp32's normal range, of gradients near the range's end, in two steps
    scale_step = factor < 0x1p-64 ? make_float2((float)(factor * 0x1p64), 0x1p-64f) : make_float2((float)factor, 1.f);
  }
  __syncthreads();
  const float scale = scale_step.x, step = scale_step.y;
  auto scaled = [&](float v) { return v * scale * step; };
  int tensor = list.start[blockIdx.x];
  // from the last chunk on: those are the ones that the L2 still holds
  for (int at = list.first_chunk[list.n] - 1 - blockIdx.x; at >= 0; at -= gridDim.x) {
    while (at < list.first_chunk[tensor]) --tensor;
    const ClipChunk c = clip_chunk(list, tensor, at);
    const void* src = list.src[c.tensor];
    void* dst = list.dst[c.tensor];
    if (scale == 1.f && step == 1.f && src == dst) continue;
    const int head = clip_head(src, c.f32);
    const bool aligned = clip_head(dst, c.f32) == head;
    if (c.f32) {
      auto one = [&](int64_t i) { static_cast<float*>(dst)[i] = scaled(static_cast<const float*>(src)[i]); };
      clip_visit<4>(c, head, one, [&](int64_t i) {
        if (!aligned) {
          for (int k = 0; k < 4; ++k) one(i + k);
          return;
        }
        const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(src) + i);
        *reinterpret_cast<float4*>(static_cast<float*>(dst) + i) = make_float4(scaled(v.x), scaled(v.y), scaled(v.z), scaled(v.w));
      });
    } else {
      auto one = [&](int64_t i) {
        static_cast<uint16_t*>(dst)[i] = __bfloat16_as_ushort(__float2bfloat16_rn(scaled(element(src, false, i))));
      };
      clip_visit<8>(c, head, one, [&](int64_t i) {
        if (!aligned) {
          for (int k = 0; k < 8; ++k) one(i + k);
          return;
        }
        float v[8];
        unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(src) + i), v);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = scaled(v[k]);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dst) + i) = pack8(v);
      });
    }
  }
}

int64_t clip_chunks(const void* p, int64_t size, bool f32) {
  if (size == 0) return 0;
  return std::max<int64_t>(1, (size - clip_head(p, f32) + kClipChunk - 1) / kClipChunk);
}

// The list's launches: tensors [first, first + n) in `chunks` chunks.
struct ClipLaunch {
  int64_t first;
  int n, grid;
};
ClipLaunch clip_launch(const GradList& g, int64_t first, bool backward, ClipList* list) {   // chunks from the last on
  ClipLaunch l{first, (int)std::min<int64_t>(kClipTensors, g.n - first), 0};
  int64_t chunks = 0;
  for (int i = 0; i < l.n; ++i) {
    const bool f32 = g.f32[first + i] != 0;
    const int64_t more = clip_chunks(g.src[first + i], g.size[first + i], f32);
    if (i > 0 && chunks + more > 2147483647) {
      l.n = i;
      break;
    }
    if (list) {
      list->src[i] = g.src[first + i];
      list->dst[i] = g.dst ? g.dst[first + i] : nullptr;
      list->size[i] = f32 ? ~g.size[first + i] : g.size[first + i];
      list->first_chunk[i] = (int)chunks;
    }
    chunks += more;
  }
  if (list) {
    list->first_chunk[l.n] = (int)chunks;
    list->n = l.n;
  }
  l.grid = (int)std::min<int64_t>(chunks, (int64_t)kClipBlocks);
  if (list && !backward)
    for (int b = 0, i = 0; b < l.grid; ++b) {
      while (b >= list->first_chunk[i + 1]) ++i;
      list->start[b] = (uint16_t)i;
    }
  if (list && backward)
    for (int b = 0, i = l.n - 1; b < l.grid; ++b) {
      while ((int)chunks - 1 - b < list->first_chunk[i]) --i;
      list->start[b] = (uint16_t)i;
    }
  return l;
}

}  // namespace

size_t grad_norm_workspace_bytes(const GradList& g) {
  size_t parts = 0;
  for (int64_t at = 0; at < g.n;) {
    const ClipLaunch l = clip_launch(g, at, false, nullptr);
    parts += l.grid;
    at += l.n;
  }
  return parts * sizeof(double);
}

cudaError_t launch_grad_clip(const GradList& g, float max_norm, float eps, float* norm, void* ws, cudaStream_t stream) {
  ClipList list;
  double* parts = static_cast<double*>(ws);
  int n = 0;
  for (int64_t at = 0; at < g.n;) {
    const ClipLaunch l = clip_launch(g, at, false, &list);
    if (l.grid > 0) {
      const cudaError_t e = launch_pdl(grad_norm_kernel, dim3(l.grid), dim3(kClipThreads), 0, stream, 1, list, parts + n);
      if (e != cudaSuccess) return e;
      n += l.grid;
    }
    at += l.n;
  }
  if (!g.dst || n == 0)
    return launch_pdl(grad_norm_sum_kernel, dim3(1), dim3(kClipThreads), 0, stream, 1, (const double*)parts, n, norm);
  for (int64_t at = 0; at < g.n;) {
    const ClipLaunch l = clip_launch(g, at, true, &list);
    if (l.grid > 0) {
      const cudaError_t e = launch_pdl(grad_scale_kernel, dim3(l.grid), dim3(kClipThreads), 0, stream, 1, list,
                                       (const double*)parts, n, max_norm, eps, norm);
      if (e != cudaSuccess) return e;
      norm = nullptr;   // the first launch writes it
    }
    at += l.n;
  }
  return cudaSuccess;
}

}  // namespace moe
