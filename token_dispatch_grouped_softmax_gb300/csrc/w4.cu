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
constexpr int kW4Rows = 8;          // rows of a chunk: the columns of an mma
constexpr int kW4MaxSlots = 2048;   // slots of one launch row (shared-memory lists)

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
  int stall;               // test hook: issue no copies
  int parts_log2;          // a sum over K is 2^parts_log2 partial sums
  uint32_t blocks_magic, grid_magic;   // 2^32 / blocks and / the grid's blocks
  int blocks;              // column blocks: columns 32 b .. 32 b + 31 of both halves
};

// An expert in use: its rows are list[row0 .. row0 + rows), cut into chunks
// of kW4Rows numbered from chunk0.
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

// Codes i and i + 4 of a word less their zero, as two bf16: 128 + code is
// 0x4300 | code (one lop3 with the shift before it: (a & b) | c is table
// 0xEA), and `offset`, 128 + zero twice, comes off exactly.
__device__ __forceinline__ uint32_t w4_pair(uint32_t word, int i, uint32_t offset) {
  uint32_t v;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(word >> (4 * i)), "r"(0x000F000Fu), "r"(0x43004300u));
  asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(v) : "r"(offset));
  return v;
}

// n / d with magic = floor((2^32 - 1) / d): at most one too small before the fix.
__device__ __forceinline__ uint32_t w4_div(uint32_t n, uint32_t d, uint32_t magic) {
  const uint32_t q = __umulhi(n, magic);
  return q + (n - q * d >= d);
}

// The experts of the slots of this launch row, and each expert's slots in
// increasing order (every block sorts for itself and must find the same
// chunks).  bits is scratch, zeroed, [E] rows of w4_bit_row(slots) words: bit i of row
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

__device__ __forceinline__ uint64_t w4_lists(const W4Params& p, int slot0, int slots, uint32_t* bits, W4Active* act,
                                             uint16_t* list, uint64_t* warp_sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int words = (slots + 31) / 32, stride = w4_bit_row(slots);
  uint16_t* before_word = reinterpret_cast<uint16_t*>(bits + p.E * stride);
  int e_of[kW4MaxSlots / kW4Threads];
#pragma unroll
  for (int j = 0; j < kW4MaxSlots / kW4Threads; ++j) {   // all the loads in flight
    const int i = j * kW4Threads + tid;
    e_of[j] = -1;
    if (i < slots) e_of[j] = p.ids ? __ldg(p.ids + slot0 + i) : 0;
  }
#pragma unroll
  for (int j = 0; j < kW4MaxSlots / kW4Threads; ++j)
    if (e_of[j] < 0 || e_of[j] >= p.E) {
      if (e_of[j] != -1 && blockIdx.x == 0) report_status(p.status, kStatusDevice, kKernW4, 1);
      e_of[j] = -1;
    }
#pragma unroll
  for (int j = 0; j < kW4MaxSlots / kW4Threads; ++j)
    if (e_of[j] >= 0) atomicOr(&bits[e_of[j] * stride + j * (kW4Warps) + warp], 1u << lane);
  __syncthreads();
  // thread i: experts [i * per, (i + 1) * per); prefix of (rows, experts, chunks)
  const int per = (p.E + kW4Threads - 1) / kW4Threads;
  auto packed = [](int n) { return (uint64_t)n | 1ull << 20 | (uint64_t)((n + kW4Rows - 1) / kW4Rows) << 40; };
  auto rows_of = [&](int e) {
    int n = 0;
    for (int w0 = 0; w0 < words; w0 += 8) {   // eight loads in flight
      uint32_t word[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) word[i] = w0 + i < words ? bits[e * stride + w0 + i] : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (w0 + i < words) before_word[e * stride + w0 + i] = (uint16_t)n;
        n += __popc(word[i]);
      }
    }
    return n;
  };
  int n_of[kMaxExperts / kW4Threads];
  uint64_t sum = 0;
#pragma unroll
  for (int q = 0; q < kMaxExperts / kW4Threads; ++q) {
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
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  uint64_t before = incl - sum, total = 0;
#pragma unroll
  for (int w = 0; w < kW4Warps; ++w) {
    const uint64_t s = warp_sums[w];
    if (w < warp) before += s;
    total += s;
  }
#pragma unroll
  for (int q = 0; q < kMaxExperts / kW4Threads; ++q) {
    const int e = tid * per + q;
    if (n_of[q]) {
      act[(int)(before >> 20 & 0xFFFFF)] = W4Active{e, (int)(before & 0xFFFFF), n_of[q], (int)(before >> 40)};
      bits[e * stride + stride - 1] = (uint32_t)(before & 0xFFFFF);
      before += packed(n_of[q]);
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kW4MaxSlots / kW4Threads; ++j)
    if (e_of[j] >= 0) {
      const uint32_t* row = bits + e_of[j] * stride;
      const int at = j * (kW4Warps) + warp;   // the word of slot j * kW4Threads + tid
      const int place = (int)row[stride - 1] + before_word[e_of[j] * stride + at] + __popc(row[at] & ((1u << lane) - 1u));
      list[place] = (uint16_t)(j * kW4Threads + tid);
    }
  return (total >> 40) | (total >> 20 & 0xFFFFF) << 32;
}

// The same for at most 32 slots, by one warp: experts in the order of their
// first slot.
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
    const int mine = leads ? n | (n + kW4Rows - 1) / kW4Rows << 16 : 0;
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
    for (int c = threadIdx.x; c < I / 8; c += kW4Threads)
      reinterpret_cast<uint4*>(p.h + (int64_t)(slot0 + i) * I)[c] = make_uint4(0, 0, 0, 0);
  }
}

__device__ __forceinline__ float w4_swiglu(float g, float u) { return g / (1.f + expf(-g)) * u; }

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

// Persistent: a block takes consecutive items (a chunk of an expert's rows, a
// column block of 32 columns in each half), and every sum over K is a sum of
// 2^parts_log2 partial sums added in order, whoever computes them, so that a
// row's result does not depend on the batch.  While a block has eight items
// or more, each warp takes a whole item (its partial sums pass through shared
// memory of its own, no barrier) and the warps' neighbouring column blocks
// read whole DRAM pages of a row together.  The items left over (all of them
// in a small batch) are shared: a warp to each part of an item's K, joined in
// shared memory.  A unit of the stream is 128 k, filled by TMA into a ring of
// the warp's own, two units deep; every group ends at a place known at
// compile time.
//
// Per 32 k a lane holds one 16-byte vector of codes per half: columns 4g ..
// 4g+3, k = 8t .. 8t+7 (g = lane / 4, t = lane % 4).  In the ring these are
// 128-byte lines (row, half) in the 128-byte swizzle, read without bank
// conflicts.  The k order inside an mma is free as long as A and B agree:
// step s takes codes (2s, 2s+4) and (2s+1, 2s+5) of the word, and the same of
// x.  A rows are weight columns (two tiles a half), B columns the expert's
// rows.
//
// The codes go into the mma as q - zero, exact in bf16: every product is
// exact, and the fp32 sums round at the size of the formula's own terms.
// (128 + q in the mma, an or with no subtraction, and (128 + zero) sum x taken
// off a group's sum rounds at 136 |x|, also where q equals the zero; one large
// x there loses the rest.)
//
// Bound by the stream of the codes where it is long: 32 tokens, top-8 of 256,
// H 7168, I 2048, groups of 128: gate_up 459 us (5.39 TB/s), down 232 (5.32).
// 45 tokens, top-8 of 128, H 2048, I 768, groups of 64 with zeros: 50 us (4.1)
// and 35 (2.9) with start, end and latency: 16 warps an SM, ALU pipe 57 %.
template <int GROUP, bool ZEROS>
struct W4Ring {
  static constexpr int kRows = 128 / GROUP;   // group rows of a unit
  static constexpr int kQ = 4096, kScale = 128 * kRows, kZero = ZEROS ? (64 * kRows + 127) / 128 * 128 : 0;
  static constexpr int kDepth = 2;
  static constexpr int kBytes = kW4Warps * kDepth * (kQ + kScale + kZero);
  static constexpr int kPart = 16 * 32;   // floats of a warp's partial sums
};
static_assert(w4_row_slots(kMaxExperts, 32, kW4MaxSlots, W4Ring<128, false>::kBytes) >= 32, "a token's slots fit one launch row");

template <int GROUP, bool ZEROS>
__host__ __device__ constexpr int w4_smem(int E, int slots) {
  using Ring = W4Ring<GROUP, ZEROS>;
  return 1024 + Ring::kBytes + kW4Warps * (Ring::kPart * 4 + Ring::kDepth * 8) +
         (E < slots ? E : slots) * (int)sizeof(W4Active) + (slots * 2 + 15) / 16 * 16 + 128;
}

// One unit: tot += its 128 k's products.  xn holds the lane's vectors of x's
// next 64 k and is loaded a step ahead, from next_k on; past the end the
// first, for the next item.  q_at, scales, zeros: the lane's place in the
// stage; of SETS halves of the columns (two: lines of both halves in turn).
template <int GROUP, bool ZEROS, int SETS>
__device__ __forceinline__ void w4_unit(float (&tot)[SETS][2][4], uint4 (&xn)[2], const uint16_t* x, int& next_k, int K, int k0,
                                        uint32_t q_at, const uint8_t* scales, const uint8_t* zeros) {
  float acc[SETS][2][4];
#pragma unroll
  for (int j = 0; j < 2; ++j) {   // 64 k each; K may end after the first
    if (j == 1 && k0 + 64 >= K) break;
    uint32_t b[2][4];
    if (next_k >= K) next_k = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 v = xn[i];
      b[i][0] = __byte_perm(v.x, v.z, 0x5410);   // x0 x4
      b[i][1] = __byte_perm(v.x, v.z, 0x7632);   // x1 x5
      b[i][2] = __byte_perm(v.y, v.w, 0x5410);   // x2 x6
      b[i][3] = __byte_perm(v.y, v.w, 0x7632);   // x3 x7
    }
    if (x) {
      xn[0] = __ldg(reinterpret_cast<const uint4*>(x + next_k));
      xn[1] = __ldg(reinterpret_cast<const uint4*>(x + next_k + 32));
    }
    next_k += 64;
#pragma unroll
    for (int i = 0; i < 2; ++i) {   // 32 k each
      const bool first = GROUP == 32 || (GROUP == 64 && i == 0) || (GROUP == 128 && i == 0 && j == 0);
      const bool last = GROUP == 32 || (GROUP == 64 && i == 1) || (GROUP == 128 && i == 1 && j == 1);
      const int row = GROUP == 32 ? 2 * j + i : GROUP == 64 ? j : 0;
#pragma unroll
      for (int set = 0; set < SETS; ++set) {
        const uint32_t at = SETS == 2 ? (set ? (q_at ^ 16) + 128 : q_at) + (2 * j + i) * 1024 : (q_at ^ i << 6) + (2 * j + i) * 512;
        uint32_t word[4];
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(word[0]), "=r"(word[1]), "=r"(word[2]), "=r"(word[3])
                     : "r"(at));
        uint32_t off[4] = {0x43084308u, 0x43084308u, 0x43084308u, 0x43084308u};   // of the lane's four columns
        if (ZEROS) {
          const uint32_t zr = *reinterpret_cast<const uint32_t*>(zeros + (row * SETS + set) * 32);
#pragma unroll
          for (int c = 0; c < 4; ++c) off[c] = __byte_perm(zr, 0x43u, 0x4040 | c << 8 | c);
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            const uint32_t w[4] = {w4_pair(word[2 * hf], 2 * st, off[2 * hf]), w4_pair(word[2 * hf + 1], 2 * st, off[2 * hf + 1]),
                                   w4_pair(word[2 * hf], 2 * st + 1, off[2 * hf]),
                                   w4_pair(word[2 * hf + 1], 2 * st + 1, off[2 * hf + 1])};
            if (st == 0 && first) mma_16816_first(acc[set][hf], w, b[i][0], b[i][1]);
            else mma_16816(acc[set][hf], w, b[i][2 * st], b[i][2 * st + 1]);
          }
      }
      if (last) {
#pragma unroll
        for (int set = 0; set < SETS; ++set) {
          const uint2 sr = *reinterpret_cast<const uint2*>(scales + (row * SETS + set) * 64);
#pragma unroll
          for (int c = 0; c < 4; ++c) {   // the lane's four columns
            const uint32_t sp = c < 2 ? sr.x : sr.y;
            const float scale = (c & 1) ? bf16_hi(sp) : bf16_lo(sp);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float& o = tot[set][c >> 1][(c & 1) * 2 + r];
              o = fmaf(scale, acc[set][c >> 1][(c & 1) * 2 + r], o);
            }
          }
        }
      }
    }
  }
}

// Stopped early: the copies in flight land (bounded) before the block's
// memory goes.
__device__ __forceinline__ void w4_land(uint32_t bar0, int depth, int stage, uint32_t phase, uint64_t limit_ns) {
  for (int d = 0; d < depth; ++d) {
    const uint64_t t0 = globaltimer_ns();
    const uint32_t par = d < stage ? phase ^ 1u : phase;
    while (!mbar_try_wait(bar0 + 8 * d, par) && globaltimer_ns() - t0 < limit_ns) {
    }
  }
}

template <bool GATE_UP, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(kW4Threads, 2) w4_kernel(const __grid_constant__ W4Params p) {
  using Ring = W4Ring<GROUP, ZEROS>;
  extern __shared__ uint8_t w4_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(w4_smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int n_act = min(p.E, min(p.slots_per_row, p.slots));
  uint8_t* ring = smem + warp * (Ring::kDepth * Ring::kQ);
  uint8_t* scales = smem + kW4Warps * Ring::kDepth * Ring::kQ + warp * (Ring::kDepth * Ring::kScale);
  uint8_t* zeros = smem + kW4Warps * Ring::kDepth * (Ring::kQ + Ring::kScale) + warp * (Ring::kDepth * Ring::kZero);
  float* sums_of_parts = reinterpret_cast<float*>(smem + Ring::kBytes);   // [8 warps][16 values][32 lanes]
  W4Active* act = reinterpret_cast<W4Active*>(sums_of_parts + kW4Warps * Ring::kPart);
  uint64_t* scratch = reinterpret_cast<uint64_t*>(act + n_act);
  uint64_t* bars = scratch + kW4Warps;
  int* abort_flag = reinterpret_cast<int*>(bars + kW4Warps * Ring::kDepth);
  int* first_act = abort_flag + 1;
  uint16_t* list = reinterpret_cast<uint16_t*>(abort_flag + 2);
  uint32_t* bits = reinterpret_cast<uint32_t*>(smem);   // over the rings, before they are used
  const uint32_t bar0 = smem_u32(bars + warp * Ring::kDepth);
  if (lane == 0) {
    for (int d = 0; d < Ring::kDepth; ++d) mbar_init(bar0 + 8 * d, 1);
    if (warp == 0) *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tm_q);
    tma_prefetch_desc(&p.tm_scale);
  }
  const int slot0 = blockIdx.y * p.slots_per_row;
  const int slots = min(p.slots_per_row, p.slots - slot0);
  if (p.slots > 32)   // the sort's bits
    for (int i = tid; i < p.E * w4_bit_row(slots); i += kW4Threads) bits[i] = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const uint64_t found = p.slots <= 32 ? w4_lists_small(p, slots, act, list, scratch)
                                       : w4_lists(p, slot0, slots, bits, act, list, scratch);
  const uint32_t chunks = (uint32_t)found;
  const int half = p.N / 2;
  if (GATE_UP && p.ids) w4_zero_rows(p, slot0, slots);
  // this block's items: an even share, the first blocks one more
  const uint32_t items = chunks * (uint32_t)p.blocks, share = w4_div(items, gridDim.x, p.grid_magic), more = items - share * gridDim.x;
  const int begin = (int)(blockIdx.x * share + min(blockIdx.x, more));
  const int end = begin + (int)share + (blockIdx.x < more ? 1 : 0);
  if (begin >= end) return;
  // the expert of its first chunk
  const int first_chunk = (int)w4_div(begin, p.blocks, p.blocks_magic);
  for (int i = tid; i < (int)(found >> 32); i += kW4Threads)
    if (first_chunk >= act[i].chunk0 && first_chunk < act[i].chunk0 + (act[i].rows + kW4Rows - 1) / kW4Rows) *first_act = i;
  fence_proxy_async_smem();   // the sort's writes into the rings, before TMA's
  __syncthreads();
  const int units = (p.K + 127) / 128;
  auto chunks_of = [](const W4Active& a) { return (a.rows + kW4Rows - 1) / kW4Rows; };

  // The warp's runs: run s < whole is an item of its own over the whole of K,
  // then one part of a shared item in each pass.
  const int parts = 1 << p.parts_log2, together = kW4Warps >> p.parts_log2;   // items shared at once
  int left = (end - begin) & (kW4Warps - 1), passes = (left + together - 1) >> (3 - p.parts_log2);
  if (passes >= parts) left = passes = 0;   // sharing would take as long: one more round of whole items
  const int whole = (end - left - begin + kW4Warps - 1) / kW4Warps;
  const int runs = whole + passes;
  const int part = warp & (parts - 1);                                        // of the shared items
  const int part_u0 = units * part >> p.parts_log2, part_u1 = units * (part + 1) >> p.parts_log2;
  auto item_of = [&](int s) {   // end or more: none
    if (s >= whole) return end - left + (s - whole) * together + (warp >> p.parts_log2);
    const int item = begin + warp + s * kW4Warps;
    return item < end - left ? item : end;
  };

  // the loader: run, the next unit's coordinates, and the stage
  int lrun = -1, lu = 0, lu_end = 0, lstage = 0, la = *first_act;
  int lcol = 0, lqrow = 0, lsrow = 0;
  auto next_run = [&]() {   // the next run that has an item
    while (++lrun < runs) {
      const int item = item_of(lrun);
      if (item >= end) continue;
      lu = lrun < whole ? 0 : part_u0;
      lu_end = lrun < whole ? units : part_u1;
      const int chunk = (int)w4_div(item, p.blocks, p.blocks_magic);
      while (chunk >= act[la].chunk0 + chunks_of(act[la])) ++la;
      const int expert = act[la].expert;
      lcol = (item - chunk * p.blocks) * 32;
      lqrow = expert * (p.K / 8) + lu * 16;
      lsrow = expert * (p.K / GROUP) + lu * Ring::kRows;
      return;
    }
  };
  auto issue = [&]() {
    if (lu == lu_end) {
      if (lrun >= runs) return;
      next_run();
      if (lrun >= runs) return;
    }
    if (lane == 0 && !p.stall) {
      const uint32_t bar = bar0 + 8 * lstage;
      mbar_arrive_expect_tx(bar, Ring::kQ + Ring::kRows * (ZEROS ? 192 : 128));
      tma_load_3d(smem_u32(ring) + lstage * Ring::kQ, &p.tm_q, lcol, 0, lqrow, bar);
      tma_load_3d(smem_u32(scales) + lstage * Ring::kScale, &p.tm_scale, lcol, 0, lsrow, bar);
      if (ZEROS) tma_load_3d(smem_u32(zeros) + lstage * Ring::kZero, &p.tm_zero, lcol, 0, lsrow, bar);
    }
    lqrow += 16;
    lsrow += Ring::kRows;
    lstage ^= 1;
    ++lu;
  };
  issue();
  issue();
  const uint32_t q_at = smem_u32(ring) + t * 256 + ((g ^ 2 * t) << 4);   // line 2t; the second half's line is the next, its chunk ^ 1

  const uint16_t* x;  // this lane's row of the chunk, if it has one
  uint4 xn[2];       // its vectors of the next 64 k
  int x_chunk = -1;  // the chunk that x is of
  int ca = *first_act, stage = 0;
  uint32_t phase = 0;
  bool ok = true;
  W4Active a = act[0];
  float* mine = sums_of_parts + warp * Ring::kPart + lane;
#pragma unroll 1
  for (int run = 0; run < runs; ++run) {
    const int item = item_of(run);
    const bool shared = run >= whole;
    const int u0 = shared ? part_u0 : 0, u1 = shared ? part_u1 : units;
    int block = 0, row_first = 0;
    float tot[2][2][4];
#pragma unroll
    for (int i = 0; i < 16; ++i) (&tot[0][0][0])[i] = 0.f;
    if (item < end) {
      const int chunk = (int)w4_div(item, p.blocks, p.blocks_magic);
      block = item - chunk * p.blocks;
      while (chunk >= act[ca].chunk0 + chunks_of(act[ca])) ++ca;
      a = act[ca];
      row_first = (chunk - a.chunk0) * kW4Rows;
      if (chunk != x_chunk || shared) {
        x_chunk = chunk;
        x = nullptr;
        xn[0] = xn[1] = make_uint4(0, 0, 0, 0);
        if (row_first + g < a.rows) {
          const int slot = slot0 + list[a.row0 + row_first + g];
          x = p.rows + (int64_t)(GATE_UP ? slot / p.k : slot) * p.K + 8 * t;
          xn[0] = __ldg(reinterpret_cast<const uint4*>(x + u0 * 128));
          xn[1] = __ldg(reinterpret_cast<const uint4*>(x + u0 * 128 + 32));
          // The rest of the run's row into L1, 128 bytes a lane: the loads 64 k ahead would each wait for L2.
          for (int c = u0 * 128 + 64 * (t + 1); c < min(u1 * 128, p.K); c += 256)
            asm volatile("prefetch.global.L1 [%0];" ::"l"(x - 8 * t + c));
        }
      }
    }
    if (item < end && ok) {
      int next_k = u0 * 128 + 64;   // the 64 k to load ahead; past the end the first, for the next item
      int part_end = shared ? u1 : units >> p.parts_log2, parts_done = 0;
#pragma unroll 1
      for (int u = u0; u < u1; ++u) {
        if (u == part_end) {   // the parts' sums in order, through this lane's shared memory
          if (parts_done > 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) (&tot[0][0][0])[i] += mine[i * 32];
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            mine[i * 32] = (&tot[0][0][0])[i];
            (&tot[0][0][0])[i] = 0.f;
          }
          ++parts_done;
          part_end = units * (parts_done + 1) >> p.parts_log2;
        }
        if (!mbar_wait_warp(bar0 + 8 * stage, phase, abort_flag, p.wait_limit_ns, p.status, 2, kKernW4)) {
          ok = false;
          break;
        }
        w4_unit<GROUP, ZEROS, 2>(tot, xn, x, next_k, p.K, u * 128, q_at + stage * Ring::kQ, scales + stage * Ring::kScale + g * 8,
                                 zeros + stage * Ring::kZero + g * 4);
        __syncwarp();   // every lane has read the stage
        issue();        // into the same stage
        stage ^= 1;
        phase ^= stage == 0;
      }
    }
    if (!shared) {
      if (item >= end) continue;
      if (parts > 1) {
#pragma unroll
        for (int i = 0; i < 16; ++i) (&tot[0][0][0])[i] += mine[i * 32];
      }
      // columns 4g .. 4g+3 of rows 2t, 2t+1 are this lane's
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = row_first + 2 * t + r;
        if (row >= a.rows) continue;
        const int64_t slot = slot0 + list[a.row0 + row];
        float v[2][4];
#pragma unroll
        for (int set = 0; set < 2; ++set)
#pragma unroll
          for (int c = 0; c < 4; ++c) v[set][c] = tot[set][c >> 1][(c & 1) * 2 + r];
        if (GATE_UP) {
#pragma unroll
          for (int c = 0; c < 4; ++c) v[0][c] = w4_swiglu(v[0][c], v[1][c]);
          *reinterpret_cast<uint2*>(p.h + slot * half + block * 32 + 4 * g) =
              make_uint2(pack_bf16x2(v[0][0], v[0][1]), pack_bf16x2(v[0][2], v[0][3]));
        } else {
#pragma unroll
          for (int set = 0; set < 2; ++set)
            *reinterpret_cast<float4*>(p.part + slot * p.N + set * half + block * 32 + 4 * g) =
                make_float4(v[set][0], v[set][1], v[set][2], v[set][3]);
        }
      }
      continue;
    }
    // a shared item: its parts' sums meet in shared memory, and its warps
    // share the values out: value i of the first half and of the second
#pragma unroll
    for (int i = 0; i < 16; ++i) mine[i * 32] = (&tot[0][0][0])[i];
    __syncthreads();
    if (item < end) {
      const float* from = sums_of_parts + (warp - part) * Ring::kPart + lane;
      for (int i = part; i < 8; i += parts) {   // i = hf * 4 + r
        const int r = i & 3, hf = i >> 2;
        const int row = row_first + 2 * t + (r & 1);
        if (row >= a.rows) continue;
        float v0 = from[i * 32], v1 = from[(8 + i) * 32];
        for (int w = 1; w < parts; ++w) {
          v0 += from[w * Ring::kPart + i * 32];
          v1 += from[w * Ring::kPart + (8 + i) * 32];
        }
        const int64_t slot = slot0 + list[a.row0 + row];
        const int col = block * 32 + 4 * g + 2 * hf + (r >> 1);
        if (GATE_UP) {
          p.h[slot * half + col] = __bfloat16_as_ushort(__float2bfloat16_rn(w4_swiglu(v0, v1)));
        } else {
          p.part[slot * p.N + col] = v0;
          p.part[slot * p.N + half + col] = v1;
        }
      }
    }
    __syncthreads();
  }
  if (!ok && lane == 0 && !p.stall) w4_land(bar0, Ring::kDepth, stage, phase, p.wait_limit_ns);
}

// The products of a few slots, all blocks at once on the GPU: a cluster takes
// a slot (gate_up) or a token's slots (down, with the combine) and a column
// block, a warp one part of a slot's sum over K, of one half of the columns
// (gate_up) or both (down).  The sums meet in the first block's shared memory
// and its first warp adds them in the order of the other kernels: the same
// bits.  No lists, and one launch for down: one token, top-8 of 128 experts,
// H 2048, I 768, down takes 6.1 us instead of 7.4 (4 tokens 11.3 instead of
// 13.3); one token, top-2 of 16, H 2048, I 1408, gate_up 5.1 instead of 6.7.
// Halves of the columns for down too took 7.3: clusters of eight blocks.
template <bool GATE_UP, int GROUP, bool ZEROS>
struct W4SlotRing {
  static constexpr int kSets = GATE_UP ? 1 : 2;   // halves of a warp's sum
  static constexpr int kRows = 128 / GROUP;       // group rows of a unit
  static constexpr int kQ = 2048 * kSets, kScale = (64 * kSets * kRows + 127) / 128 * 128;
  static constexpr int kZero = ZEROS ? (32 * kSets * kRows + 127) / 128 * 128 : 0;
  static constexpr int kDepth = 4 / kSets;
  static constexpr int kBytes = kW4Warps * kDepth * (kQ + kScale + kZero);
};

template <bool GATE_UP, int GROUP, bool ZEROS>
__host__ __device__ constexpr int w4_slots_smem(int sums) {
  using Ring = W4SlotRing<GATE_UP, GROUP, ZEROS>;
  return 1024 + Ring::kBytes + sums * Ring::kSets * 32 * 4 + kW4Warps * Ring::kDepth * 8 + 16;
}

struct W4SlotArgs {
  int per;            // slots of a cluster: 1, or k and their combine
  int cluster_log2;   // blocks of a cluster
  const float* wt;
  const uint16_t* y_shared;
  uint16_t* y;
};

template <bool GATE_UP, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(kW4Threads, 2) w4_slots_kernel(const __grid_constant__ W4Params p, const W4SlotArgs s) {
  using Ring = W4SlotRing<GATE_UP, GROUP, ZEROS>;
  constexpr int kSets = Ring::kSets, kSplit = 2 - kSets;   // kSplit: bits of a sum's number for its half
  extern __shared__ uint8_t w4_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(w4_smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int parts = 1 << p.parts_log2, slot_shift = p.parts_log2 + kSplit;
  const int sums = s.per << slot_shift;   // sum n: slot, part, half
  uint8_t* ring = smem + warp * (Ring::kDepth * Ring::kQ);
  uint8_t* scales = smem + kW4Warps * Ring::kDepth * Ring::kQ + warp * (Ring::kDepth * Ring::kScale);
  uint8_t* zeros = smem + kW4Warps * Ring::kDepth * (Ring::kQ + Ring::kScale) + warp * (Ring::kDepth * Ring::kZero);
  float* met = reinterpret_cast<float*>(smem + Ring::kBytes);   // [sums][kSets][32 columns], of the cluster's first block
  uint64_t* bars = reinterpret_cast<uint64_t*>(met + sums * kSets * 32);
  int* abort_flag = reinterpret_cast<int*>(bars + kW4Warps * Ring::kDepth);
  const uint32_t bar0 = smem_u32(bars + warp * Ring::kDepth);
  if (lane == 0) {
    for (int d = 0; d < Ring::kDepth; ++d) mbar_init(bar0 + 8 * d, 1);
    if (warp == 0) *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tm_q);
    tma_prefetch_desc(&p.tm_scale);
  }
  __syncthreads();
  cluster_arrive_release();   // this block runs: its shared memory may be written
  pdl_wait();
  pdl_trigger();
  const int rank = blockIdx.x & ((1 << s.cluster_log2) - 1), block = blockIdx.x >> s.cluster_log2;
  const int slot0 = blockIdx.y * s.per, half = p.N / 2;
  int expert = -1;   // of slot slot0 + lane
  float weight = 1.f;
  if (lane < s.per) {
    expert = p.ids ? p.ids[slot0 + lane] : 0;
    if (!GATE_UP && s.wt) weight = s.wt[slot0 + lane];
    if (expert < 0 || expert >= p.E) {
      if (expert != -1 && blockIdx.x == 0 && warp == 0) report_status(p.status, kStatusDevice, kKernW4, 1);
      expert = -1;
    }
  }
  const int units = (p.K + 127) / 128, stride = kW4Warps << s.cluster_log2;
  auto next_sum = [&](int n) {   // from n on, the first of the warp's sums whose slot has an expert
    while (n < sums && __shfl_sync(0xffffffffu, expert, n >> slot_shift) < 0) n += stride;
    return n;
  };
  const int first = next_sum(rank * kW4Warps + warp);

  // the loader: the sum, the next unit's coordinates, and the stage
  int ln = first, lu = 0, lu_end = 0, lstage = 0, lqrow = 0, lsrow = 0;
  auto open = [&]() {
    if (ln >= sums) return;
    const int part = ln >> kSplit & (parts - 1), e = __shfl_sync(0xffffffffu, expert, ln >> slot_shift);
    lu = units * part >> p.parts_log2;
    lu_end = units * (part + 1) >> p.parts_log2;
    lqrow = e * (p.K / 8) + lu * 16;
    lsrow = e * (p.K / GROUP) + lu * Ring::kRows;
  };
  auto issue = [&]() {
    if (ln >= sums) return;
    if (lane == 0 && !p.stall) {
      const uint32_t bar = bar0 + 8 * lstage;
      mbar_arrive_expect_tx(bar, Ring::kQ + Ring::kRows * kSets * (ZEROS ? 96 : 64));
      tma_load_3d(smem_u32(ring) + lstage * Ring::kQ, &p.tm_q, block * 32, ln & kSplit, lqrow, bar);
      tma_load_3d(smem_u32(scales) + lstage * Ring::kScale, &p.tm_scale, block * 32, ln & kSplit, lsrow, bar);
      if (ZEROS) tma_load_3d(smem_u32(zeros) + lstage * Ring::kZero, &p.tm_zero, block * 32, ln & kSplit, lsrow, bar);
    }
    lqrow += 16;
    lsrow += Ring::kRows;
    lstage = (lstage + 1) & (Ring::kDepth - 1);
    if (++lu == lu_end) {
      ln = next_sum(ln + stride);
      open();
    }
  };
  open();
  for (int d = 0; d < Ring::kDepth; ++d) issue();
  // Columns 4 c4 .. 4 c4 + 3 are the lane's: with one half, and c4 = g, the
  // lanes of a quarter warp, two g and four t, would read the same banks.
  const int c4 = kSets == 2 ? g : g >> 1 | (g & 1) << 2;
  const uint32_t q_at = smem_u32(ring) + t * (128 * kSets) + ((c4 ^ kSets * t) << 4);
  const uint32_t met_at = mapa_shared(smem_u32(met), 0);
  __syncwarp();
  cluster_wait_acquire();
  int stage = 0;
  uint32_t phase = 0;
  bool ok = true;
#pragma unroll 1
  for (int n = first; n < sums && ok; n = next_sum(n + stride)) {
    const int part = n >> kSplit & (parts - 1), slot = slot0 + (n >> slot_shift);
    const int u0 = units * part >> p.parts_log2, u1 = units * (part + 1) >> p.parts_log2;
    float tot[kSets][2][4];
#pragma unroll
    for (int i = 0; i < 8 * kSets; ++i) (&tot[0][0][0])[i] = 0.f;
    const uint16_t* x = nullptr;   // the mma's other rows are zero
    uint4 xn[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (g == 0) {
      x = p.rows + (int64_t)(GATE_UP ? slot / p.k : slot) * p.K + 8 * t;
      xn[0] = __ldg(reinterpret_cast<const uint4*>(x + u0 * 128));
      xn[1] = __ldg(reinterpret_cast<const uint4*>(x + u0 * 128 + 32));
      for (int c = u0 * 128 + 64 * (t + 1); c < min(u1 * 128, p.K); c += 256)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(x - 8 * t + c));
    }
    int next_k = u0 * 128 + 64;
#pragma unroll 1
    for (int u = u0; u < u1; ++u) {
      if (!mbar_wait_warp(bar0 + 8 * stage, phase, abort_flag, p.wait_limit_ns, p.status, 2, kKernW4)) {
        ok = false;
        break;
      }
      w4_unit<GROUP, ZEROS, kSets>(tot, xn, x, next_k, p.K, u * 128, q_at + stage * Ring::kQ, scales + stage * Ring::kScale + c4 * 8,
                               zeros + stage * Ring::kZero + c4 * 4);
      __syncwarp();   // every lane has read the stage
      issue();        // into the same stage
      stage = (stage + 1) & (Ring::kDepth - 1);
      phase ^= stage == 0;
    }
    if (t == 0) {   // row 0: the lane's four columns
#pragma unroll
      for (int set = 0; set < kSets; ++set)
        st_shared_cluster_f32x4(met_at + (uint32_t)((n * kSets + set) * 32 + 4 * c4) * 4,
                                make_float4(tot[set][0][0], tot[set][0][2], tot[set][1][0], tot[set][1][2]));
    }
  }
  const bool adds = rank == 0 && warp == 0;
  // down: the lane's two columns are of the first half, or of the second
  const int64_t at = (int64_t)blockIdx.y * p.N + (lane < 16 ? 0 : half) + block * 32 + 2 * (lane & 15);
  uint32_t extra = 0;
  if (!GATE_UP && adds && s.y_shared) extra = *reinterpret_cast<const uint32_t*>(s.y_shared + at);
  __syncwarp();
  cluster_sync_all();
  if (adds && GATE_UP) {
    float v[2] = {0.f, 0.f};
    const bool used = __shfl_sync(0xffffffffu, expert, 0) >= 0;
    if (used) {
      v[0] = met[lane];
      v[1] = met[32 + lane];
      for (int q = 1; q < parts; ++q) {
        v[0] += met[q * 64 + lane];
        v[1] += met[q * 64 + 32 + lane];
      }
    }
    p.h[(int64_t)slot0 * half + block * 32 + lane] = used ? __bfloat16_as_ushort(__float2bfloat16_rn(w4_swiglu(v[0], v[1]))) : 0;
  }
  if (adds && !GATE_UP) {
    float acc[2] = {0.f, 0.f};
    for (int j = 0; j < s.per; ++j) {
      const float w = __shfl_sync(0xffffffffu, weight, j);
      if (__shfl_sync(0xffffffffu, expert, j) < 0) continue;
      const float* from = met + j * parts * 64 + 2 * lane;   // the halves' columns lie together
      float2 v = *reinterpret_cast<const float2*>(from);
      for (int q = 1; q < parts; ++q) {
        const float2 o = *reinterpret_cast<const float2*>(from + q * 64);
        v.x += o.x;
        v.y += o.y;
      }
      acc[0] = fmaf(w, v.x, acc[0]);
      acc[1] = fmaf(w, v.y, acc[1]);
    }
    if (s.y_shared) {
      acc[0] += bf16_lo(extra);
      acc[1] += bf16_hi(extra);
    }
    *reinterpret_cast<uint32_t*>(s.y + at) = pack_bf16x2(acc[0], acc[1]);
  }
  if (!ok && lane == 0 && !p.stall) w4_land(bar0, Ring::kDepth, stage, phase, p.wait_limit_ns);
}

constexpr int kW4CombineThreads = 64;   // small blocks: one token's columns spread over several SMs

// y[t] = sum_j w[t, j] part[t, j] (+ y_shared[t]) over the slots in use, 8
// columns per thread.  Latency of two dependent loads: 4 us for 45 tokens,
// top-8, H 2048.
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

template <bool GATE_UP, int GROUP, bool ZEROS>
cudaError_t launch_w4_slots(const W4Params& p, const W4SlotArgs& s, const DeviceInfo& dev, cudaStream_t stream) {
  static std::atomic<int> configured[kMaxDevices] = {};   // per device (a race only repeats the set-up)
  if (!configured[dev.ordinal].load()) {
    const cudaError_t err = cudaFuncSetAttribute(w4_slots_kernel<GATE_UP, GROUP, ZEROS>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 w4_slots_smem<GATE_UP, GROUP, ZEROS>(16 * kW4Warps));
    if (err != cudaSuccess) return err;
    configured[dev.ordinal].store(1);
  }
  return launch_pdl(w4_slots_kernel<GATE_UP, GROUP, ZEROS>, dim3((unsigned)(p.blocks << s.cluster_log2), (unsigned)(p.slots / s.per)),
                    dim3(kW4Threads), w4_slots_smem<GATE_UP, GROUP, ZEROS>(s.per << (p.parts_log2 + GATE_UP)), stream, 1u << s.cluster_log2, p, s);
}

template <bool GATE_UP, int GROUP, bool ZEROS>
cudaError_t launch_w4(const W4Params& p, const W4SlotArgs& s, const DeviceInfo& dev, cudaStream_t stream) {
  if (s.per) return launch_w4_slots<GATE_UP, GROUP, ZEROS>(p, s, dev, stream);
  static std::atomic<int> configured[kMaxDevices] = {};   // per device (a race only repeats the set-up)
  if (!configured[dev.ordinal].load()) {
    const cudaError_t err = cudaFuncSetAttribute(w4_kernel<GATE_UP, GROUP, ZEROS>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 w4_smem<GROUP, ZEROS>(kMaxExperts, kW4MaxSlots));
    if (err != cudaSuccess) return err;
    configured[dev.ordinal].store(1);
  }
  const int row_slots = std::min(p.slots_per_row, p.slots);
  const int rows = (p.slots + p.slots_per_row - 1) / p.slots_per_row;
  const int64_t most = (int64_t)row_slots * p.blocks;   // every slot its own chunk
  W4Params q = p;
  const unsigned grid = (unsigned)std::min<int64_t>(most, 2 * dev.num_sms);
  q.grid_magic = 0xFFFFFFFFu / grid;
  q.blocks_magic = 0xFFFFFFFFu / (uint32_t)p.blocks;
  return launch_pdl(w4_kernel<GATE_UP, GROUP, ZEROS>, dim3(grid, (unsigned)rows), dim3(kW4Threads),
                    w4_smem<GROUP, ZEROS>(p.E, row_slots), stream, 1, q);
}

// How w4_slots_kernel would run the call, per 0: not.  Its blocks must all be
// on the GPU at once, two an SM, with a warp for every two sums: beyond that
// the tokens' common experts are read again and again (down at H 2048, I 768,
// top-8 of 128: 4 tokens with two sums a warp 11.3 us, with a warp each, in
// two waves, 14.1, by w4_kernel 13.3; 8 tokens 22.4, by w4_kernel 21.5).
template <bool GATE_UP>
W4SlotArgs w4_slot_plan(const W4Params& p, const DeviceInfo& dev) {
  W4SlotArgs s{};
  const int per = GATE_UP ? 1 : p.k, sums = per << (p.parts_log2 + GATE_UP);
  const int64_t clusters = (int64_t)p.blocks * (p.slots / per);
  int c = 0;
  while (c < 3 && kW4Warps << c < sums && clusters << (c + 1) <= 2 * dev.num_sms) ++c;
  s.cluster_log2 = c;
  s.per = clusters << c <= 2 * dev.num_sms && sums <= 2 * kW4Warps << c ? per : 0;
  return s;
}

// The tensor maps and the launch of the group's kernel.
template <bool GATE_UP>
cudaError_t launch_w4_group(W4Params& p, const W4SlotArgs& s, const uint32_t* q, const uint16_t* scales, const uint8_t* zeros,
                            int64_t group, const DeviceInfo& dev, cudaStream_t stream) {
  const cuuint64_t half = p.N / 2, rows = (cuuint64_t)p.E * p.K;
  auto encode = [&](CUtensorMap* map, CUtensorMapDataType type, cuuint64_t bytes, const void* base, cuuint64_t n,
                    int box_rows, CUtensorMapSwizzle swizzle) {
    const cuuint64_t dims[3] = {half, 2, n}, strides[2] = {half * bytes, (cuuint64_t)p.N * bytes};
    const cuuint32_t box[3] = {32, GATE_UP && s.per ? 1u : 2u, (cuuint32_t)box_rows};
    return encode_tensor_map_3d(map, type, base, dims, strides, box, swizzle);
  };
  const int group_rows = (int)(128 / group);
  if (!encode(&p.tm_q, CU_TENSOR_MAP_DATA_TYPE_INT32, 4, q, rows / 8, 16, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode(&p.tm_scale, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, scales, rows / group, group_rows, CU_TENSOR_MAP_SWIZZLE_NONE) ||
      (zeros && !encode(&p.tm_zero, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, zeros, rows / group, group_rows, CU_TENSOR_MAP_SWIZZLE_NONE)))
    return cudaErrorInvalidValue;
  if (group == 32)
    return zeros ? launch_w4<GATE_UP, 32, true>(p, s, dev, stream) : launch_w4<GATE_UP, 32, false>(p, s, dev, stream);
  if (group == 64)
    return zeros ? launch_w4<GATE_UP, 64, true>(p, s, dev, stream) : launch_w4<GATE_UP, 64, false>(p, s, dev, stream);
  return zeros ? launch_w4<GATE_UP, 128, true>(p, s, dev, stream) : launch_w4<GATE_UP, 128, false>(p, s, dev, stream);
}

int w4_slots_per_row(int E, int k) { return w4_row_slots(E, k, kW4MaxSlots, W4Ring<128, false>::kBytes); }

// The call's sizes, K's parts, and the device.
W4Params w4_params(const uint16_t* rows, const int32_t* ids, int64_t T, int64_t K, int64_t N, int64_t E, int64_t k,
                   const DeviceInfo& dev) {
  W4Params p{};
  p.rows = rows;
  p.ids = ids;
  p.K = (int)K;
  p.N = (int)N;
  p.E = (int)E;
  p.k = (int)k;
  p.slots = (int)(T * k);
  p.status = dev.status;
  p.wait_limit_ns = dev.wait_limit_ns;
  p.stall = dev.test_stall_producer;
  p.slots_per_row = w4_slots_per_row(p.E, p.k);
  p.blocks = (int)(N / 64);
  const int units = (p.K + 127) / 128;
  p.parts_log2 = units >= 32 ? 3 : units >= 4 ? 2 : units >= 2 ? 1 : 0;
  return p;
}

// One thread per group and 2 columns of [rows, N] bf16 weights.
//   symmetric: scale = bf16(max|w| / 7), q = clamp(rint(w / scale) + 8, 0, 15)
//   zeros:     scale = bf16((max(w, 0) - min(w, 0)) / 15), zero = min(rint(-min(w, 0) / scale), 15),
//              q = clamp(rint(w / scale) + zero, 0, 15)
// A group of zeros has scale 0 and q = zero.  Two passes over the group, the
// second from cache: 550 us for 0.4 G weights (0.8 GB, 1.5 TB/s).
__global__ void __launch_bounds__(256) w4_quantize_kernel(const uint16_t* __restrict__ w, int64_t groups, int N,
                                                          int group, uint32_t* __restrict__ q,
                                                          uint16_t* __restrict__ scales, uint8_t* __restrict__ zeros) {
  pdl_wait();
  pdl_trigger();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int nv = N / 2;
  if (i >= groups * nv) return;
  const int64_t g = i / nv;
  const int n = (int)(i - g * nv) * 2;
  const uint16_t* src = w + g * group * N + n;
  float lo[2] = {0.f, 0.f}, hi[2] = {0.f, 0.f}, s[2], zero[2];
#pragma unroll 16
  for (int r = 0; r < group; ++r) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(src + (int64_t)r * N);
    lo[0] = fminf(lo[0], bf16_lo(v));
    hi[0] = fmaxf(hi[0], bf16_lo(v));
    lo[1] = fminf(lo[1], bf16_hi(v));
    hi[1] = fmaxf(hi[1], bf16_hi(v));
  }
  uint32_t sbits = 0, zbits = 0;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const float want = zeros ? (hi[c] - lo[c]) / 15.f : fmaxf(hi[c], -lo[c]) / 7.f;
    const __nv_bfloat16 sb = __float2bfloat16_rn(want);
    s[c] = __bfloat162float(sb);
    zero[c] = zeros ? (s[c] > 0.f ? fminf(rintf(-lo[c] / s[c]), 15.f) : 0.f) : 8.f;
    sbits |= (uint32_t)__bfloat16_as_ushort(sb) << (16 * c);
    zbits |= (uint32_t)zero[c] << (8 * c);
  }
  *reinterpret_cast<uint32_t*>(scales + g * N + n) = sbits;
  if (zeros) *reinterpret_cast<uint16_t*>(zeros + g * N + n) = (uint16_t)zbits;
  for (int r = 0; r < group; r += 8) {
    uint32_t word[2] = {0, 0};
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const uint32_t v = *reinterpret_cast<const uint32_t*>(src + (int64_t)(r + b) * N);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float code = s[c] > 0.f ? fminf(fmaxf(rintf((c ? bf16_hi(v) : bf16_lo(v)) / s[c]) + zero[c], 0.f), 15.f) : zero[c];
        word[c] |= (uint32_t)code << (4 * b);
      }
    }
    *reinterpret_cast<uint2*>(q + (g * group + r) / 8 * N + n) = make_uint2(word[0], word[1]);
  }
}

// One thread per word row and 8 columns: scale * (q - zero) in fp32, rounded
// to bf16, written as 8 vectors of 16 bytes.  Bound by the writes: 148 us for
// 0.4 G weights (1.0 GB moved, 6.8 TB/s).
__global__ void __launch_bounds__(256) w4_dequantize_kernel(const uint32_t* __restrict__ q,
                                                            const uint16_t* __restrict__ scales,
                                                            const uint8_t* __restrict__ zeros, int64_t words, int N,
                                                            int group, uint16_t* __restrict__ w) {
  pdl_wait();
  pdl_trigger();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int nv = N / 8;
  if (i >= words * nv) return;
  const int64_t r = i / nv;
  const int n = (int)(i - r * nv) * 8;
  const int64_t sg = r * 8 / group * N + n;
  const uint4* src = reinterpret_cast<const uint4*>(q + r * N + n);
  const uint4 a = src[0], b = src[1];
  const uint32_t word[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  float s[8], zero[8];
  unpack8(*reinterpret_cast<const uint4*>(scales + sg), s);
  const uint2 z = zeros ? *reinterpret_cast<const uint2*>(zeros + sg) : make_uint2(0x08080808u, 0x08080808u);
#pragma unroll
  for (int c = 0; c < 8; ++c) zero[c] = (float)(((c < 4 ? z.x : z.y) >> (8 * (c & 3))) & 255u);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float v[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = s[c] * ((float)((word[c] >> (4 * k)) & 15u) - zero[c]);
    *reinterpret_cast<uint4*>(w + (r * 8 + k) * N + n) = pack8(v);
  }
}

}  // namespace

int64_t w4_max_slots(int64_t E, int64_t k) { return 65535ll * w4_slots_per_row((int)E, (int)k); }   // launch rows of a grid

cudaError_t launch_w4_gate_up(const uint16_t* x, const int32_t* ids, const uint32_t* q, const uint16_t* scales,
                              const uint8_t* zeros, int64_t T, int64_t H, int64_t E, int64_t k, int64_t I,
                              int64_t group, uint16_t* h, const DeviceInfo& dev, cudaStream_t stream) {
  W4Params p = w4_params(x, ids, T, H, 2 * I, E, k, dev);
  p.h = h;
  return launch_w4_group<true>(p, w4_slot_plan<true>(p, dev), q, scales, zeros, group, dev, stream);
}

size_t w4_down_workspace_bytes(int64_t T, int64_t k, int64_t H) { return (size_t)(T * k * H * 4); }

cudaError_t launch_w4_down(const uint16_t* h, const int32_t* ids, const float* wt, const uint32_t* q,
                           const uint16_t* scales, const uint8_t* zeros, const uint16_t* y_shared, int64_t T,
                           int64_t H, int64_t E, int64_t k, int64_t I, int64_t group, uint16_t* y, void* ws,
                           const DeviceInfo& dev, cudaStream_t stream) {
  W4Params p = w4_params(h, ids, T, I, H, E, k, dev);
  p.part = static_cast<float*>(ws);
  W4SlotArgs s = w4_slot_plan<false>(p, dev);
  s.wt = wt;
  s.y_shared = y_shared;
  s.y = y;
  const cudaError_t err = launch_w4_group<false>(p, s, q, scales, zeros, group, dev, stream);
  if (err != cudaSuccess || s.per) return err;
  return launch_pdl(w4_combine_kernel, dim3((unsigned)((T * (H / 8) + kW4CombineThreads - 1) / kW4CombineThreads)),
                    dim3(kW4CombineThreads), 0, stream, 1, static_cast<const float*>(ws), ids, wt, y_shared, T, (int)E, (int)k, (int)H, y);
}

cudaError_t launch_w4_quantize(const uint16_t* w, int64_t rows, int64_t N, int64_t group, uint32_t* q,
                               uint16_t* scales, uint8_t* zeros, cudaStream_t stream) {
  const int64_t n = rows / group * (N / 2);
  return launch_pdl(w4_quantize_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, 1, w, rows / group,
                    (int)N, (int)group, q, scales, zeros);
}

cudaError_t launch_w4_dequantize(const uint32_t* q, const uint16_t* scales, const uint8_t* zeros, int64_t rows,
                                 int64_t N, int64_t group, uint16_t* w, cudaStream_t stream) {
  const int64_t n = rows / 8 * (N / 8);
  return launch_pdl(w4_dequantize_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, 1, q, scales,
                    zeros, rows / 8, (int)N, (int)group, w);
}

}  // namespace moe
