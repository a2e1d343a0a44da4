// What the 4-bit experts' kernels share: their arguments, the lists of the
// experts in use and their slots, and the codes' decoding.
#pragma once

#include "kernels.h"

namespace moe {

struct W4Params {
  CUtensorMap tm_q;        // codes as [E*K/8 rows][2 halves of the columns][N/2], boxes of 16 x 2 x 32 words
  CUtensorMap tm_scale;    // scales the same way, boxes of (128 / group) x 2 x 32
  CUtensorMap tm_zero;
  const uint16_t* rows;    // gate_up: x [T, K]; down: h [slots, K]
  const int32_t* ids;      // [slots], NULL: one dense expert
  uint16_t* h;             // gate_up's output [slots, N / 2]
  float* part;             // down's products [slots, N]
  uint32_t* status;
  uint64_t wait_limit_ns;
  int K, N, E, k;
  int slots, slots_per_row;
  int parts_log2;          // a sum over K is 2^parts_log2 partial sums
  int blocks;              // column blocks: columns 32 b .. 32 b + 31 of both halves
};

// The kernel for many rows an expert (w4_wide.cu).
cudaError_t launch_w4_wide(W4Params& p, bool gate_up, int64_t group, bool zeros, const DeviceInfo& dev,
                           cudaStream_t stream);

// An expert in use: its rows are list[row0 .. row0 + rows), cut into chunks
// (of 8 or 64) numbered from chunk0.
struct W4Active {
  int expert, row0, rows, chunk0;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int32_t c0, int32_t c1, int32_t c2,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// Codes i and i + 4 of a word plus 128, as two bf16: 128 + code is 0x4300 |
// code.  One lop3 with the shift before it: (a & b) | c is table 0xEA.
__device__ __forceinline__ uint32_t w4_pair(uint32_t word, int i) {
  uint32_t v;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(word >> (4 * i)), "r"(0x000F000Fu), "r"(0x43004300u));
  return v;
}

// The experts of the slots of this launch row, and each expert's slots in
// increasing order (every block sorts for itself and must find the same
// chunks).  bits is scratch, [E] rows of w4_bit_row(slots) words: bit i of row
// e says that slot i is expert e's, so a slot's place is a count of the bits
// before it, whatever order they were set in; the row's last word is the
// expert's first place.  Behind them, 16 bits for each word: the bits set in
// the row's words before it.  Returns the numbers of chunks (low 32 bits) and
// of experts in use.  (Counting with __match_any_sync took 6900 cycles for
// 360 slots of 128 experts, most of it in that instruction.)
__host__ __device__ constexpr int w4_bit_row(int slots) { return ((slots + 31) / 32 + 1) | 1; }   // odd: no bank conflicts

// Slots that a launch row can take: at most `most`, whole tokens, and the
// sort's scratch in `bytes`.
__host__ __device__ constexpr int w4_row_slots(int E, int k, int most, int bytes) {
  int slots = most;
  while (E * w4_bit_row(slots) * 6 > bytes) slots -= 32;
  return slots / k * k;
}

// ROWS: rows of a chunk.  SLOTS: the most slots of a launch row.  By the
// first THREADS threads of the block, which takes part in the barriers;
// warp_sums holds one word a warp of them.
template <int ROWS, int THREADS, int SLOTS>
__device__ __forceinline__ uint64_t w4_lists(const W4Params& p, int slot0, int slots, uint32_t* bits, W4Active* act,
                                             uint16_t* list, uint64_t* warp_sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int words = (slots + 31) / 32, stride = w4_bit_row(slots);
  uint16_t* before_word = reinterpret_cast<uint16_t*>(bits + p.E * stride);
  int e_of[SLOTS / THREADS];
#pragma unroll
  for (int j = 0; j < SLOTS / THREADS; ++j) {
    const int i = j * THREADS + tid;
    e_of[j] = -1;
    if (tid < THREADS && i < slots) {
      const int e = p.ids ? p.ids[slot0 + i] : 0;
      if (e >= 0 && e < p.E) e_of[j] = e;
      else if (e != -1 && blockIdx.x == 0) report_status(p.status, kStatusDevice, kKernW4, 1);
    }
  }
  for (int i = tid; i < p.E * stride; i += blockDim.x) bits[i] = 0;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < SLOTS / THREADS; ++j)
    if (e_of[j] >= 0) atomicOr(&bits[e_of[j] * stride + j * (THREADS / 32) + warp], 1u << lane);
  __syncthreads();
  // thread i: experts [i * per, (i + 1) * per); prefix of (rows, experts, chunks)
  const int per = (p.E + THREADS - 1) / THREADS;
  auto packed = [](int n) { return (uint64_t)n | 1ull << 20 | (uint64_t)((n + ROWS - 1) / ROWS) << 40; };
  auto rows_of = [&](int e) {
    int n = 0;
    for (int w = 0; w < words; ++w) {
      before_word[e * stride + w] = (uint16_t)n;
      n += __popc(bits[e * stride + w]);
    }
    return n;
  };
  int n_of[kMaxExperts / THREADS];
  uint64_t sum = 0;
#pragma unroll
  for (int q = 0; q < kMaxExperts / THREADS; ++q) {
    const int e = tid * per + q;
    n_of[q] = q < per && e < p.E ? rows_of(e) : 0;
    if (n_of[q]) sum += packed(n_of[q]);
  }
  uint64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31 && tid < THREADS) warp_sums[warp] = incl;
  __syncthreads();
  uint64_t before = incl - sum, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const uint64_t s = warp_sums[w];
    if (w < warp) before += s;
    total += s;
  }
#pragma unroll
  for (int q = 0; q < kMaxExperts / THREADS; ++q) {
    const int e = tid * per + q;
    if (n_of[q]) {
      act[(int)(before >> 20 & 0xFFFFF)] = W4Active{e, (int)(before & 0xFFFFF), n_of[q], (int)(before >> 40)};
      bits[e * stride + stride - 1] = (uint32_t)(before & 0xFFFFF);
      before += packed(n_of[q]);
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < SLOTS / THREADS; ++j)
    if (e_of[j] >= 0) {
      const uint32_t* row = bits + e_of[j] * stride;
      const int at = j * (THREADS / 32) + warp;   // the word of slot j * THREADS + tid
      const int place = (int)row[stride - 1] + before_word[e_of[j] * stride + at] + __popc(row[at] & ((1u << lane) - 1u));
      list[place] = (uint16_t)(j * THREADS + tid);
    }
  return (total >> 40) | (total >> 20 & 0xFFFFF) << 32;
}

// The same for at most 32 slots, by one warp: experts in the order of their
// first slot.
template <int ROWS>
__device__ __forceinline__ uint64_t w4_lists_small(const W4Params& p, int slots, W4Active* act, uint16_t* list,
                                                   uint64_t* result) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int e = -1;
    if (lane < slots) {
      e = p.ids ? p.ids[lane] : 0;
      if (e < 0 || e >= p.E) {
        if (e != -1 && blockIdx.x == 0) report_status(p.status, kStatusDevice, kKernW4, 1);
        e = -1;
      }
    }
    uint32_t peers = 0;
#pragma unroll 8
    for (int j = 0; j < slots; ++j) peers |= (uint32_t)(__shfl_sync(0xffffffffu, e, j) == e) << j;
    const int n = __popc(peers), first = __ffs(peers) - 1;
    const bool leads = e >= 0 && lane == first;
    const int mine = leads ? n | (n + ROWS - 1) / ROWS << 16 : 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const int before = incl - mine;
    const uint32_t leaders = __ballot_sync(0xffffffffu, leads);
    if (leads) act[__popc(leaders & ((1u << lane) - 1u))] = W4Active{e, before & 0xFFFF, n, before >> 16};
    const int row0 = __shfl_sync(0xffffffffu, before & 0xFFFF, first & 31);
    if (e >= 0) list[row0 + __popc(peers & ((1u << lane) - 1u))] = (uint16_t)lane;
    if (lane == 31) *result = (uint64_t)(incl >> 16) | (uint64_t)__popc(leaders) << 32;
  }
  __syncthreads();
  return *result;
}

// Zero rows of h for the empty slots, shared out over the blocks.
__device__ __forceinline__ void w4_zero_rows(const W4Params& p, int slot0, int slots) {
  const int I = p.N / 2;
  for (int i = blockIdx.x; i < slots; i += gridDim.x) {
    const int e = p.ids[slot0 + i];
    if (e >= 0 && e < p.E) continue;
    for (int c = threadIdx.x; c < I / 8; c += blockDim.x)
      reinterpret_cast<uint4*>(p.h + (int64_t)(slot0 + i) * I)[c] = make_uint4(0, 0, 0, 0);
  }
}

__device__ __forceinline__ float w4_swiglu(float g, float u) { return g / (1.f + expf(-g)) * u; }

}  // namespace moe
