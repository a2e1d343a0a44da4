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

constexpr int kW4Warps = 8;
constexpr int kW4Threads = 32 * kW4Warps;
constexpr int kW4MaxSlots = 2048;   // slots of one launch row (shared-memory lists)

struct W4Params {
  CUtensorMap tm_q;        // codes as [E*K/8 rows][2 halves of the columns][N/2], boxes of 8 x 2 x 32 words
  CUtensorMap tm_scale;    // scales the same way, boxes of (64 / group, or 1) x 2 x 32
  CUtensorMap tm_zero;
  const uint16_t* rows;    // gate_up: x [T, K]; down: h [slots, K]
  const int32_t* ids;      // [slots], NULL: one dense expert
  uint16_t* h;             // gate_up's output [slots, N / 2]
  float* part;             // down's products [slots, N]
  uint32_t* status;
  uint64_t wait_limit_ns;
  int K, N, E, k;
  int slots, slots_per_row;
  int has_zeros;
  int split_log2;          // 2^split_log2 warps share a column block's K
  int blocks;              // column blocks: columns 32 b .. 32 b + 31 of both halves
  int block_items;         // items of one chunk: blocks / (8 >> split_log2), rounded up
};

// A stage of a warp's ring: a unit of 64 k of 2 x 32 columns (two swizzled
// 8 x 128-byte atoms), and the columns' scales and zeros (two groups where a
// group is 32).
template <int NT, int GROUP>
struct W4Ring {
  static constexpr int kRows = GROUP == 32 ? 2 : 1;   // group rows of a unit
  static constexpr int kQ = 2048, kScale = 128 * kRows, kZero = 128;   // TMA destinations are 128-byte aligned
  static constexpr int kDepth = NT == 1 ? 3 : 4;
  static constexpr int kRed = 16 * NT * 33;   // floats of one warp's partial sums
  static constexpr int kBlocksPerSm = NT == 1 ? 3 : 2;
};
static_assert(kW4Warps * kMaxExperts * 4 <= kW4Warps * W4Ring<1, 128>::kDepth * W4Ring<1, 128>::kQ,
              "the sort's counts fit the rings");

// An expert in use: its rows are list[row0 .. row0 + rows), cut into chunks
// of 8 NT rows numbered from chunk0.
struct W4Active {
  int expert, row0, rows, chunk0;
};

template <int NT, int GROUP>
__host__ __device__ constexpr int w4_smem(int E, int slots, bool zeros) {
  using R = W4Ring<NT, GROUP>;
  return 1024 + kW4Warps * (R::kDepth * (R::kQ + R::kScale + (zeros ? R::kZero : 0) + 8) + R::kRed * 4) +
         (E < slots ? E : slots) * (int)sizeof(W4Active) + (slots * 2 + 15) / 16 * 16 + 128;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int32_t c0, int32_t c1, int32_t c2,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// D += A B, A 16 x 16 and B 16 x 8 bf16, fp32 accumulators.
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// D = A B.
__device__ __forceinline__ void mma_16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Codes i and i + 4 of a word plus 128, as two bf16: 128 + code is 0x4300 |
// code.  One lop3 with the shift before it: (a & b) | c is table 0xEA.
__device__ __forceinline__ uint32_t w4_pair(uint32_t word, int i) {
  uint32_t v;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(word >> (4 * i)), "r"(0x000F000Fu), "r"(0x43004300u));
  return v;
}

// The experts of the slots of this launch row, and each expert's slots in
// increasing order: a stable counting sort in shared memory (every block
// sorts for itself and must find the same chunks).  Warp w counts and places
// its eighth of the slots; cnt is [8][E] scratch.  Returns the number of
// chunks.
template <int NT>
__device__ __forceinline__ int w4_lists(const W4Params& p, int slot0, int slots, int* cnt, W4Active* act,
                                        uint16_t* list, uint64_t* warp_sum64) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kW4Warps * p.E; i += kW4Threads) cnt[i] = 0;
  __syncthreads();
  const int s_begin = slots * warp / kW4Warps, s_end = slots * (warp + 1) / kW4Warps;
  int* mine = cnt + warp * p.E;
  auto expert_of = [&](int i) {   // -1: an empty slot, or none
    if (i >= s_end) return -1;
    const int e = p.ids ? p.ids[slot0 + i] : 0;
    if (e >= 0 && e < p.E) return e;
    if (e != -1 && blockIdx.x == 0) report_status(p.status, kStatusDevice, kKernW4, 1);
    return -1;
  };
  for (int i0 = s_begin; i0 < s_end; i0 += 32) {
    const int e = expert_of(i0 + lane);
    const uint32_t peers = __match_any_sync(0xffffffffu, e);
    if (e >= 0 && lane == __ffs(peers) - 1) mine[e] += __popc(peers);
    __syncwarp();
  }
  __syncthreads();
  // thread i: experts [i * per, (i + 1) * per); prefix of (rows, experts, chunks)
  const int per = (p.E + kW4Threads - 1) / kW4Threads;
  auto packed = [](int n) { return (uint64_t)n | 1ull << 20 | (uint64_t)((n + 8 * NT - 1) / (8 * NT)) << 40; };
  uint64_t sum = 0;
  for (int q = 0; q < per; ++q) {
    const int e = tid * per + q;
    if (e >= p.E) break;
    int n = 0;
    for (int w = 0; w < kW4Warps; ++w) n += cnt[w * p.E + e];
    if (n) sum += packed(n);
  }
  uint64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) warp_sum64[warp] = incl;
  __syncthreads();
  uint64_t before = incl - sum, total = 0;
  for (int w = 0; w < kW4Warps; ++w) {
    const uint64_t s = warp_sum64[w];
    if (w < warp) before += s;
    total += s;
  }
  for (int q = 0; q < per; ++q) {
    const int e = tid * per + q;
    if (e >= p.E) break;
    const int row0 = (int)(before & 0xFFFFF);
    int n = 0;
    for (int w = 0; w < kW4Warps; ++w) {   // counts to first places
      const int c = cnt[w * p.E + e];
      cnt[w * p.E + e] = row0 + n;
      n += c;
    }
    if (n) {
      act[(int)(before >> 20 & 0xFFFFF)] = W4Active{e, row0, n, (int)(before >> 40)};
      before += packed(n);
    }
  }
  __syncthreads();
  for (int i0 = s_begin; i0 < s_end; i0 += 32) {
    const int e = expert_of(i0 + lane);
    const uint32_t peers = __match_any_sync(0xffffffffu, e);
    int place = 0;
    if (e >= 0) {
      place = mine[e] + __popc(peers & ((1u << lane) - 1u));
      list[place] = (uint16_t)(i0 + lane);
    }
    __syncwarp();
    if (e >= 0 && lane == __ffs(peers) - 1) mine[e] = place + __popc(peers);
    __syncwarp();
  }
  __syncthreads();
  return (int)(total >> 40);
}

// The same for at most 32 slots, by one warp: experts in the order of their
// first slot.
template <int NT>
__device__ __forceinline__ int w4_lists_small(const W4Params& p, int slots, W4Active* act, uint16_t* list, int* chunks) {
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
    const uint32_t peers = __match_any_sync(0xffffffffu, e);
    const int n = __popc(peers), first = __ffs(peers) - 1;
    const bool leads = e >= 0 && lane == first;
    const int mine = leads ? n | (n + 8 * NT - 1) / (8 * NT) << 16 : 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const int before = incl - mine;
    const uint32_t leaders = __ballot_sync(0xffffffffu, leads);
    if (leads) act[__popc(leaders & ((1u << lane) - 1u))] = W4Active{e, before & 0xFFFF, n, before >> 16};
    const int row0 = __shfl_sync(0xffffffffu, before & 0xFFFF, first);
    if (e >= 0) list[row0 + __popc(peers & ((1u << lane) - 1u))] = (uint16_t)lane;
    if (lane == 31) *chunks = incl >> 16;
  }
  __syncthreads();
  return *chunks;
}

// Persistent: a block takes consecutive items (chunk of an expert's rows,
// column blocks).  2^split_log2 of its 8 warps share a column block, each
// with its part of K, and their sums are added in that order; a warp streams
// 64-k units through a ring of its own, filled by TMA.
//
// Per 32 k a lane holds one 16-byte vector of codes per half: columns 4g ..
// 4g+3, k = 8t .. 8t+7 (g = lane / 4, t = lane % 4).  In the ring these are
// 128-byte lines (row, half) in the 128-byte swizzle, read without bank
// conflicts.  The k order inside an mma is free as long as A and B agree:
// step s takes codes (2s, 2s+4) and (2s+1, 2s+5) of the word, and the same of
// x.  A rows are weight columns (two tiles a half), B columns the expert's
// rows.
//
// The codes go into the mma as 128 + q, an or with no subtraction; the sum
// over the group of (128 + zero) x, from one more mma with a tile of ones, is
// taken off before the scale: sum (q - zero) x = sum (128 + q) x - (128 +
// zero) sum x.  Every product is exact; the fp32 sums round at 128 + q
// instead of q - zero, some 2^-19 of the terms, 2^10 below the bf16 result.
template <int NT, bool GATE_UP, int GROUP>
__global__ void __launch_bounds__(kW4Threads, W4Ring<NT, GROUP>::kBlocksPerSm)
    w4_kernel(const __grid_constant__ W4Params p) {
  using Ring = W4Ring<NT, GROUP>;
  extern __shared__ uint8_t w4_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(w4_smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int n_act = min(p.E, min(p.slots_per_row, p.slots));
  // rings | scale rings | zero rings | sums of the warps | experts in use | slot lists
  uint8_t* ring = smem + warp * (Ring::kDepth * Ring::kQ);
  uint8_t* scales = smem + kW4Warps * Ring::kDepth * Ring::kQ;
  uint8_t* zeros = scales + kW4Warps * Ring::kDepth * Ring::kScale;
  float* red = reinterpret_cast<float*>(zeros + (p.has_zeros ? kW4Warps * Ring::kDepth * Ring::kZero : 0));
  W4Active* act = reinterpret_cast<W4Active*>(red + kW4Warps * Ring::kRed);
  uint64_t* sums = reinterpret_cast<uint64_t*>(act + n_act);
  uint64_t* bars = sums + kW4Warps;
  int* abort_flag = reinterpret_cast<int*>(bars + kW4Warps * Ring::kDepth);
  uint16_t* list = reinterpret_cast<uint16_t*>(abort_flag + 2);
  int* cnt = reinterpret_cast<int*>(smem);   // [8][E] over the rings, before they are used
  scales += warp * (Ring::kDepth * Ring::kScale);
  zeros += warp * (Ring::kDepth * Ring::kZero);
  const uint32_t bar0 = smem_u32(bars + warp * Ring::kDepth);
  if (lane == 0) {
    for (int d = 0; d < Ring::kDepth; ++d) mbar_init(bar0 + 8 * d, 1);
    if (warp == 0) *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tm_q);
    tma_prefetch_desc(&p.tm_scale);
  }
  pdl_wait();
  pdl_trigger();
  const int slot0 = blockIdx.y * p.slots_per_row;
  const int slots = min(p.slots_per_row, p.slots - slot0);
  const int chunks = p.slots <= 32 ? w4_lists_small<NT>(p, slots, act, list, reinterpret_cast<int*>(sums))
                                   : w4_lists<NT>(p, slot0, slots, cnt, act, list, sums);
  const int half = p.N / 2;
  if (GATE_UP && p.ids) {                    // empty slots: zero rows
    for (int i = blockIdx.x; i < slots; i += gridDim.x) {
      const int e = p.ids[slot0 + i];
      if (e < 0 || e >= p.E)
        for (int c = tid; c < half / 8; c += kW4Threads)
          reinterpret_cast<uint4*>(p.h + (int64_t)(slot0 + i) * half)[c] = make_uint4(0, 0, 0, 0);
    }
  }
  const int64_t items = (int64_t)chunks * p.block_items;
  const int begin = (int)(items * blockIdx.x / gridDim.x), end = (int)(items * (blockIdx.x + 1) / gridDim.x);
  if (begin >= end) return;
  fence_proxy_async_smem();   // the sort's writes into the rings, before TMA's
  __syncthreads();
  const int split = 1 << p.split_log2, wide = kW4Warps >> p.split_log2;   // warps of a block, blocks of an item
  const int part = warp & (split - 1), sub = warp >> p.split_log2;
  const int units = p.K / 64;
  const int u0 = units * part / split, u1 = units * (part + 1) / split;
  auto chunks_of = [](const W4Active& a) { return (a.rows + 8 * NT - 1) / (8 * NT); };

  // the loader: item (lchunk, lblock), unit lu of the next copies, and their
  // coordinates; only items with a column block for this warp take stages
  int litem = begin, lchunk = begin / p.block_items, lblock = begin - lchunk * p.block_items;
  int la = 0, lu = u0, lstage = 0;
  while (lchunk >= act[la].chunk0 + chunks_of(act[la])) ++la;
  int ca = la, cchunk = lchunk, cblock = lblock;   // the same of the item being computed
  int lcol = 0, lqrow = 0, lsrow = 0;
  auto next_item = [&]() {   // litem, or the next one with a column block for this warp
    for (; litem < end; ++litem, ++lblock) {
      if (lblock == p.block_items) {
        lblock = 0;
        ++lchunk;
      }
      if (lblock * wide + sub < p.blocks) break;
    }
    if (litem >= end) return;
    if (lchunk >= act[la].chunk0 + chunks_of(act[la])) ++la;   // chunks come one after another
    const int expert = act[la].expert;
    lcol = (lblock * wide + sub) * 32;
    lqrow = expert * (p.K / 8);
    lsrow = expert * (p.K / GROUP);
  };
  next_item();
  auto issue = [&]() {
    if (litem >= end) return;
    if (lane == 0) {
      const uint32_t bar = bar0 + 8 * lstage;
      const bool sc = GROUP <= 64 || lu == u0 || (lu & 1) == 0;
      const uint32_t bytes = Ring::kQ + (sc ? Ring::kRows * (p.has_zeros ? 192 : 128) : 0);
      mbar_arrive_expect_tx(bar, bytes);
      tma_load_3d(smem_u32(ring + lstage * Ring::kQ), &p.tm_q, lcol, 0, lqrow + lu * 8, bar);
      if (sc) {
        const int row = lsrow + (GROUP <= 64 ? lu * Ring::kRows : lu >> 1);
        tma_load_3d(smem_u32(scales + lstage * Ring::kScale), &p.tm_scale, lcol, 0, row, bar);
        if (p.has_zeros) tma_load_3d(smem_u32(zeros + lstage * Ring::kZero), &p.tm_zero, lcol, 0, row, bar);
      }
    }
    if (++lstage == Ring::kDepth) lstage = 0;
    if (++lu == u1) {
      lu = u0;
      ++litem;
      ++lblock;
      next_item();
    }
  };
#pragma unroll 1
  for (int d = 0; d < Ring::kDepth; ++d) issue();
  const uint32_t q_at = t * 256 + ((g ^ 2 * t) << 4);   // line 2t; the second half's line is the next, its chunk ^ 1

  // this lane's rows of the chunk, and their vectors of the next unit: loaded a
  // unit ahead (the first unit's again at an item's end, for the next block)
  const uint16_t* x[NT];
  uint4 xn[NT][2];
  int stage = 0;
  uint32_t phase = 0;
  bool ok = true;
#pragma unroll 1
  for (int item = begin; item < end; ++item) {
    if (cchunk >= act[ca].chunk0 + chunks_of(act[ca])) ++ca;
    const W4Active a = act[ca];
    const int row_first = (cchunk - a.chunk0) * 8 * NT;
    if (cblock == 0 || item == begin) {   // another chunk: its rows
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int r = row_first + n * 8 + g;
        x[n] = nullptr;
        xn[n][0] = xn[n][1] = make_uint4(0, 0, 0, 0);
        if (r < a.rows) {
          const int slot = slot0 + list[a.row0 + r];
          x[n] = p.rows + (int64_t)(GATE_UP ? slot / p.k : slot) * p.K + u0 * 64 + 8 * t;
          xn[n][0] = __ldg(reinterpret_cast<const uint4*>(x[n]));
          xn[n][1] = __ldg(reinterpret_cast<const uint4*>(x[n] + 32));
        }
      }
    }
    float tot[2][2][NT][4];
#pragma unroll
    for (int i = 0; i < 16 * NT; ++i) (&tot[0][0][0][0])[i] = 0.f;
    if (cblock * wide + sub < p.blocks && ok) {
      float acc[2][2][NT][4], sum[NT][4];
      if (GROUP == 128) {
#pragma unroll
        for (int i = 0; i < 16 * NT; ++i) (&acc[0][0][0][0])[i] = 0.f;
#pragma unroll
        for (int i = 0; i < 4 * NT; ++i) (&sum[0][0])[i] = 0.f;
      }
      uint2 sraw[2];
      uint32_t zraw[2] = {0x08080808u, 0x08080808u};
#pragma unroll 1
      for (int u = u0; u < u1; ++u) {
        if (!mbar_wait_warp(bar0 + 8 * stage, phase, abort_flag, p.wait_limit_ns, p.status, 2, kKernW4)) {
          ok = false;
          break;
        }
        const uint8_t* s = ring + stage * Ring::kQ;
        auto read_scales = [&](int row) {
#pragma unroll
          for (int set = 0; set < 2; ++set) {
            sraw[set] = *reinterpret_cast<const uint2*>(scales + stage * Ring::kScale + (row * 2 + set) * 64 + g * 8);
            if (p.has_zeros)
              zraw[set] = *reinterpret_cast<const uint32_t*>(zeros + stage * Ring::kZero + (row * 2 + set) * 32 + g * 4);
          }
        };
        if (GROUP == 128 && (u == u0 || (u & 1) == 0)) read_scales(0);
        uint32_t b[2][NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 v = xn[n][i];
            b[i][n][0] = __byte_perm(v.x, v.z, 0x5410);   // x0 x4
            b[i][n][1] = __byte_perm(v.x, v.z, 0x7632);   // x1 x5
            b[i][n][2] = __byte_perm(v.y, v.w, 0x5410);   // x2 x6
            b[i][n][3] = __byte_perm(v.y, v.w, 0x7632);   // x3 x7
          }
          if (x[n]) {
            const uint16_t* next = x[n] + (u + 1 < u1 ? (u + 1 - u0) * 64 : 0);
            xn[n][0] = __ldg(reinterpret_cast<const uint4*>(next));
            xn[n][1] = __ldg(reinterpret_cast<const uint4*>(next + 32));
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {   // 32 k each
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint32_t ones[4] = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
            if (GROUP == 32 || (GROUP == 64 && i == 0)) mma_16816_first(sum[n], ones, b[i][n][0], b[i][n][1]);
            else mma_16816(sum[n], ones, b[i][n][0], b[i][n][1]);
            mma_16816(sum[n], ones, b[i][n][2], b[i][n][3]);
          }
#pragma unroll
          for (int set = 0; set < 2; ++set) {
            const uint4 v = *reinterpret_cast<const uint4*>(s + i * 1024 + (set ? (q_at ^ 16) + 128 : q_at));
            const uint32_t word[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
              for (int st = 0; st < 2; ++st) {
                const uint32_t w[4] = {w4_pair(word[2 * hf], 2 * st), w4_pair(word[2 * hf + 1], 2 * st),
                                       w4_pair(word[2 * hf], 2 * st + 1), w4_pair(word[2 * hf + 1], 2 * st + 1)};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  if (st == 0 && (GROUP == 32 || (GROUP == 64 && i == 0)))
                    mma_16816_first(acc[set][hf][n], w, b[i][n][0], b[i][n][1]);
                  else
                    mma_16816(acc[set][hf][n], w, b[i][n][2 * st], b[i][n][2 * st + 1]);
                }
              }
          }
          if (GROUP == 32 || (i == 1 && (GROUP == 64 || u + 1 == u1 || (u & 1) != 0))) {
            if (GROUP <= 64) read_scales(GROUP == 32 ? i : 0);
#pragma unroll
            for (int set = 0; set < 2; ++set)
#pragma unroll
              for (int c = 0; c < 4; ++c) {   // the lane's four columns
                const uint32_t sp = c < 2 ? sraw[set].x : sraw[set].y;
                const float scale = (c & 1) ? bf16_hi(sp) : bf16_lo(sp);
                const float zero = __uint_as_float(0x43000000u | ((zraw[set] >> (8 * c)) & 15u) << 16);   // 128 + zero
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                  for (int r = 0; r < 2; ++r) {
                    float& v = acc[set][c >> 1][n][(c & 1) * 2 + r];
                    float& o = tot[set][c >> 1][n][(c & 1) * 2 + r];
                    o = fmaf(scale, fmaf(-zero, sum[n][r], v), o);
                    if (GROUP == 128) v = 0.f;
                  }
              }
            if (GROUP == 128) {
#pragma unroll
              for (int i2 = 0; i2 < 4 * NT; ++i2) (&sum[0][0])[i2] = 0.f;
            }
          }
        }
        __syncwarp();   // every lane has read the stage
        issue();        // into the same stage
        if (++stage == Ring::kDepth) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // join the warps' sums: value (set, column, row) of lane (column / 4, row / 2)
    float* mine = red + warp * Ring::kRed;
#pragma unroll
    for (int set = 0; set < 2; ++set)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            mine[((set * NT + n) * 8 + (r & 1) * 4 + 2 * hf + (r >> 1)) * 33 + lane] = tot[set][hf][n][r];
    __syncthreads();
    const int at = ((warp & 1) * 4 + (lane & 3)) * 33 + (lane >> 2) * 4 + (warp >> 1);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = row_first + n * 8 + warp;   // this warp's row
      if (r >= a.rows) continue;
      const int64_t slot = slot0 + list[a.row0 + r];
      for (int b = 0; b < wide; ++b) {
        const int block = cblock * wide + b;
        if (block >= p.blocks) break;
        const float* from = red + b * split * Ring::kRed + n * 8 * 33 + at;
        float v[2] = {0.f, 0.f};
#pragma unroll 4
        for (int w = 0; w < split; ++w)
#pragma unroll
          for (int set = 0; set < 2; ++set) v[set] += from[w * Ring::kRed + set * NT * 8 * 33];
        if (GATE_UP) {
          const float y = v[0] / (1.f + expf(-v[0])) * v[1];
          p.h[slot * half + block * 32 + lane] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
        } else {
          p.part[slot * p.N + block * 32 + lane] = v[0];
          p.part[slot * p.N + half + block * 32 + lane] = v[1];
        }
      }
    }
    __syncthreads();
    if (++cblock == p.block_items) {
      cblock = 0;
      ++cchunk;
    }
  }
  if (!ok && lane == 0) {   // stopped early: the copies in flight land (bounded) before the block's memory goes
    for (int d = 0; d < Ring::kDepth; ++d) {
      const uint64_t t0 = globaltimer_ns();
      const uint32_t par = d < stage ? phase ^ 1u : phase;
      while (!mbar_try_wait(bar0 + 8 * d, par) && globaltimer_ns() - t0 < p.wait_limit_ns) {
      }
    }
  }
}

constexpr int kW4CombineThreads = 64;   // small blocks: one token's columns spread over several SMs

// y[t] = sum_j w[t, j] part[t, j] (+ y_shared[t]) over the slots in use, 8
// columns per thread.
__global__ void __launch_bounds__(kW4CombineThreads) w4_combine_kernel(const float* __restrict__ part,
                                                         const int32_t* __restrict__ ids,
                                                         const float* __restrict__ wt,
                                                         const uint16_t* __restrict__ y_shared, int64_t T, int E, int k,
                                                         int H, uint16_t* __restrict__ y) {
  pdl_wait();
  pdl_trigger();
  const int64_t i = (int64_t)blockIdx.x * kW4CombineThreads + threadIdx.x;
  const int nch = H / 8;
  const int64_t t = i / nch;
  const int c = (int)(i - t * nch) * 8;
  if (t >= T) return;
  float acc[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) acc[q] = 0.f;
  for (int j0 = 0; j0 < k; j0 += 8) {   // eight slots' loads in flight
    float w[8];
    bool on[8];
    float4 v[8][2];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int64_t slot = t * k + j0 + q;
      on[q] = j0 + q < k;
      if (on[q]) {
        const int e = ids ? ids[slot] : 0;
        w[q] = wt ? wt[slot] : 1.f;
        const float4* src = reinterpret_cast<const float4*>(part + slot * H + c);
        v[q][0] = src[0];   // of an empty slot: whatever the workspace holds, not used
        v[q][1] = src[1];
        on[q] = e >= 0 && e < E;
      }
    }
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (on[q]) {
        acc[0] = fmaf(w[q], v[q][0].x, acc[0]); acc[1] = fmaf(w[q], v[q][0].y, acc[1]);
        acc[2] = fmaf(w[q], v[q][0].z, acc[2]); acc[3] = fmaf(w[q], v[q][0].w, acc[3]);
        acc[4] = fmaf(w[q], v[q][1].x, acc[4]); acc[5] = fmaf(w[q], v[q][1].y, acc[5]);
        acc[6] = fmaf(w[q], v[q][1].z, acc[6]); acc[7] = fmaf(w[q], v[q][1].w, acc[7]);
      }
  }
  if (y_shared) {
    float f[8];
    unpack8(*reinterpret_cast<const uint4*>(y_shared + t * H + c), f);
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] += f[q];
  }
  *reinterpret_cast<uint4*>(y + t * H + c) = pack8(acc);
}

template <int NT, bool GATE_UP, int GROUP>
cudaError_t launch_w4(const W4Params& p, const DeviceInfo& dev, cudaStream_t stream) {
  using Ring = W4Ring<NT, GROUP>;
  static std::atomic<int> configured[kMaxDevices] = {};   // per device (a race only repeats the set-up)
  if (!configured[dev.ordinal].load()) {
    const cudaError_t err = cudaFuncSetAttribute(w4_kernel<NT, GATE_UP, GROUP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 w4_smem<NT, GROUP>(kMaxExperts, kW4MaxSlots, true));
    if (err != cudaSuccess) return err;
    configured[dev.ordinal].store(1);
  }
  const int row_slots = std::min(p.slots_per_row, p.slots);
  const int rows = (p.slots + p.slots_per_row - 1) / p.slots_per_row;
  const int64_t most = (int64_t)row_slots * p.block_items;   // every slot its own chunk
  return launch_pdl(w4_kernel<NT, GATE_UP, GROUP>,
                    dim3((unsigned)std::min<int64_t>(most, Ring::kBlocksPerSm * dev.num_sms), (unsigned)rows),
                    dim3(kW4Threads), w4_smem<NT, GROUP>(p.E, row_slots, p.has_zeros), stream, 1, p);
}

template <bool GATE_UP, int GROUP>
cudaError_t launch_w4_rows(const W4Params& p, const DeviceInfo& dev, cudaStream_t stream) {
  // 8 rows a chunk while the experts in use hold few rows each, else 16
  return (int64_t)p.slots <= (int64_t)4 * p.E || p.slots <= 8 * p.k ? launch_w4<1, GATE_UP, GROUP>(p, dev, stream)
                                                                   : launch_w4<2, GATE_UP, GROUP>(p, dev, stream);
}

// K's split over warps and the launch of the group's kernel.  The split is
// a rule on K alone, so that a row's sums do not depend on the batch: the
// most warps (8 at most) whose shares of K's 64-k units are equal, or nearly
// (at least 16 units a warp).
template <bool GATE_UP>
cudaError_t launch_w4_group(W4Params& p, const uint32_t* q, const uint16_t* scales, const uint8_t* zeros,
                            int64_t group, const DeviceInfo& dev, cudaStream_t stream) {
  const cuuint64_t half = p.N / 2, rows = (cuuint64_t)p.E * p.K;
  auto encode = [&](CUtensorMap* map, CUtensorMapDataType type, cuuint64_t bytes, const void* base, cuuint64_t n,
                    cuuint32_t box_rows, CUtensorMapSwizzle swizzle) {
    const cuuint64_t dims[3] = {half, 2, n}, strides[2] = {half * bytes, (cuuint64_t)p.N * bytes};
    const cuuint32_t box[3] = {32, 2, box_rows};
    return encode_tensor_map_3d(map, type, base, dims, strides, box, swizzle);
  };
  const cuuint32_t box_rows = group == 32 ? 2 : 1;
  if (!encode(&p.tm_q, CU_TENSOR_MAP_DATA_TYPE_INT32, 4, q, rows / 8, 8, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode(&p.tm_scale, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, scales, rows / group, box_rows, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  p.has_zeros = zeros != nullptr;
  if (zeros && !encode(&p.tm_zero, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, zeros, rows / group, box_rows, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  p.status = dev.status;
  p.wait_limit_ns = dev.wait_limit_ns;
  p.slots_per_row = kW4MaxSlots / p.k * p.k;
  p.blocks = (int)(half / 32);
  const int units = p.K / 64;
  p.split_log2 = 3;
  while (p.split_log2 > 0 && units % (1 << p.split_log2) != 0 && units < (16 << p.split_log2)) --p.split_log2;
  const int wide = kW4Warps >> p.split_log2;
  p.block_items = (p.blocks + wide - 1) / wide;
  if (group == 32) return launch_w4_rows<GATE_UP, 32>(p, dev, stream);
  if (group == 64) return launch_w4_rows<GATE_UP, 64>(p, dev, stream);
  return launch_w4_rows<GATE_UP, 128>(p, dev, stream);
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
  W4Params p{};
  p.rows = x;
  p.ids = ids;
  p.h = h;
  p.K = (int)H;
  p.N = (int)(2 * I);
  p.E = (int)E;
  p.k = (int)k;
  p.slots = (int)(T * k);
  return launch_w4_group<true>(p, q, scales, zeros, group, dev, stream);
}

size_t w4_down_workspace_bytes(int64_t T, int64_t k, int64_t H) { return (size_t)(T * k * H * 4); }

cudaError_t launch_w4_down(const uint16_t* h, const int32_t* ids, const float* wt, const uint32_t* q,
                           const uint16_t* scales, const uint8_t* zeros, const uint16_t* y_shared, int64_t T,
                           int64_t H, int64_t E, int64_t k, int64_t I, int64_t group, uint16_t* y, void* ws,
                           const DeviceInfo& dev, cudaStream_t stream) {
  W4Params p{};
  p.rows = h;
  p.ids = ids;
  p.part = static_cast<float*>(ws);
  p.K = (int)I;
  p.N = (int)H;
  p.E = (int)E;
  p.k = (int)k;
  p.slots = (int)(T * k);
  const cudaError_t err = launch_w4_group<false>(p, q, scales, zeros, group, dev, stream);
  if (err != cudaSuccess) return err;
  return launch_pdl(w4_combine_kernel, dim3((unsigned)((T * (H / 8) + kW4CombineThreads - 1) / kW4CombineThreads)),
                    dim3(kW4CombineThreads), 0, stream, 1, static_cast<const float*>(ws), ids, wt, y_shared, T, (int)E, (int)k, (int)H, y);
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
