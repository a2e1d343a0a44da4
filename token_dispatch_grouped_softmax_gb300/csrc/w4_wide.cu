// The 4-bit experts' products where experts hold many rows (chunks of up to
// 64): the codes are decoded once for all of them and go to the 5th-generation
// tensor cores (tcgen05), whose time does not show beside the decoding.
//
//   D[m, n] = sum over a group's k of (q[k, m] - zero[m]) x[n, k]   (TMEM, fp32)
//   total[m, n] += scale[m] D[m, n]                                 (registers, fp32)
//
// m: 64 columns of the first half of N and the same of the second (gate and
// up), 128 in all; n: the chunk's rows.  Codes less zeros are exact in bf16.
#include <algorithm>

#include "w4.cuh"

namespace moe {

namespace {

constexpr int kWideRows = 64;
constexpr int kWideThreads = 896;     // warp 0 TMA, 1 MMA, 4..11 totals, 12..27 decoders
constexpr int kListThreads = 512;     // of them in the sort of the slots
constexpr int kTotalWarps = 8;        // four of the tile's 128 columns, for each half of the rows
constexpr int kWideMaxSlots = 4096;   // slots of one launch row
constexpr int kDecoders = 8;          // warps of a decoder group; two groups take the steps in turn
constexpr int kQStages = 4, kAbStages = 3, kDBuffers = 4;
constexpr int kABytes = 128 * 128 * 2, kBBytes = kWideRows * 128 * 2;   // a step: 128 k

// The MMA and the commit by one elected lane of the converged warp.  (The
// same lane issues both: a commit follows the MMAs of its own thread.)
__device__ __forceinline__ void mma_elected(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n elect.sync _|q, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit_elected(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar)
      : "memory");
}

template <int GROUP, bool ZEROS>
struct WideRing {
  static constexpr int kSubs = 128 / GROUP;   // groups of a step
  static constexpr int kQ = 8192, kScale = 2 * 128 * kSubs;
  static constexpr int kZeroBox = ZEROS ? (64 * kSubs + 127) / 128 * 128 : 0, kZero = 2 * kZeroBox;
  static constexpr int kBytes = kAbStages * (kABytes + kBBytes) + kQStages * (kQ + kScale + kZero);
};
constexpr int kSortBytes = kAbStages * (kABytes + kBBytes) + kQStages * 8192;   // the sort's scratch: under the rings
static_assert(w4_row_slots(kMaxExperts, 32, kWideMaxSlots, kSortBytes) >= 32, "a token's slots fit one launch row");

template <int GROUP, bool ZEROS>
__host__ __device__ constexpr int wide_smem(int E, int slots) {
  return 1024 + WideRing<GROUP, ZEROS>::kBytes + kWideRows * 64 * 4 + (E < slots ? E : slots) * (int)sizeof(W4Active) +
         (slots * 2 + 15) / 16 * 16 + 512;
}

// No memory clobber, so that a run of them and the loads around them overlap:
// ordered by the proxy fence that follows (an asm with a memory clobber).
__device__ __forceinline__ void st_shared16(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d));
}

// Codes i and i + 4 of a word less the zero, as two bf16 (exact: 128 + code
// less 128 + zero, zero2 the latter in both halves).
__device__ __forceinline__ uint32_t w4_less_zero(uint32_t word, int i, uint32_t zero2) {
  const uint32_t v = w4_pair(word, i);
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                   *reinterpret_cast<const __nv_bfloat162*>(&zero2));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// Persistent, warp-specialised, one block per SM; an item is (chunk, 64
// columns of each half), streamed over K in steps of 128:
//   TMA      codes, scales and zeros of the step, four stages deep
//   decoders codes -> A [128 columns][128 k] and x rows -> B [rows][128 k],
//            both K-major in the 128-byte swizzle; within 8 k the order is
//            k0 k4 k1 k5 k2 k6 k3 k7, as the codes come apart.  A step is some
//            1300 cycles of waits, loads and conversions one after another to
//            its warps: two groups of them take the steps in turn
//   MMA      a group's products into a fresh TMEM buffer (four of 64 columns)
//   totals   buffer -> registers, a lane to a column: one scale for all rows
// Every wait is bounded (MOE_ERR_TIMEOUT in the status word).
template <bool GATE_UP, int GROUP, bool ZEROS>
__global__ void __launch_bounds__(kWideThreads, 1) w4_wide_kernel(const __grid_constant__ W4Params p) {
  using Ring = WideRing<GROUP, ZEROS>;
  extern __shared__ uint8_t wide_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(wide_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n_act = min(p.E, min(p.slots_per_row, p.slots));
  const uint32_t ab = smem_u32(smem);                                          // [stage][A | B]
  uint8_t* codes = smem + kAbStages * (kABytes + kBBytes);                     // [stage][8192]
  uint8_t* scales = codes + kQStages * Ring::kQ;
  uint8_t* zeros = scales + kQStages * Ring::kScale;
  float* exchange = reinterpret_cast<float*>(smem + Ring::kBytes);             // [row][64 columns]
  W4Active* act = reinterpret_cast<W4Active*>(exchange + kWideRows * 64);
  uint64_t* scratch = reinterpret_cast<uint64_t*>(act + n_act);                // 16 warps' sums
  uint64_t* bars = scratch + 16;
  constexpr int kBars = 2 * (kQStages + kAbStages + kDBuffers) + 3;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kBars);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  int* first_act = abort_flag + 1;
  uint16_t* list = reinterpret_cast<uint16_t*>(first_act + 2);
  const uint32_t bar0 = smem_u32(bars);
  auto full_q = [&](int s) { return bar0 + 8u * s; };
  auto empty_q = [&](int s) { return bar0 + 8u * (kQStages + s); };
  auto full_ab = [&](int s) { return bar0 + 8u * (2 * kQStages + s); };
  auto empty_ab = [&](int s) { return bar0 + 8u * (2 * kQStages + kAbStages + s); };
  auto full_d = [&](int s) { return bar0 + 8u * (2 * (kQStages + kAbStages) + s); };
  auto empty_d = [&](int s) { return bar0 + 8u * (2 * (kQStages + kAbStages) + kDBuffers + s); };
  const uint32_t exch_full = bar0 + 8u * (kBars - 3), exch_empty = bar0 + 8u * (kBars - 2), drain = bar0 + 8u * (kBars - 1);
  if (tid == 0) {
    for (int s = 0; s < kQStages; ++s) {
      mbar_init(full_q(s), 1);
      mbar_init(empty_q(s), kDecoders + kTotalWarps);
    }
    for (int s = 0; s < kAbStages; ++s) {
      mbar_init(full_ab(s), kDecoders);
      mbar_init(empty_ab(s), 1);
    }
    for (int s = 0; s < kDBuffers; ++s) {
      mbar_init(full_d(s), 1);
      mbar_init(empty_d(s), kTotalWarps);
    }
    mbar_init(exch_full, kTotalWarps / 2);
    mbar_init(exch_empty, kTotalWarps / 2);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tm_q);
    tma_prefetch_desc(&p.tm_scale);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kDBuffers * 64);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  const int slot0 = blockIdx.y * p.slots_per_row;
  const int slots = min(p.slots_per_row, p.slots - slot0);
  uint32_t* bits = reinterpret_cast<uint32_t*>(smem);   // over the rings, before they are used
  const uint64_t found = w4_lists<kWideRows, kListThreads, kWideMaxSlots>(p, slot0, slots, bits, act, list, scratch);
  const uint32_t chunks = (uint32_t)found;
  const int half = p.N / 2;
  if (GATE_UP && p.ids) w4_zero_rows(p, slot0, slots);
  const uint32_t items = chunks * (uint32_t)p.blocks, share = items / gridDim.x, more = items - share * gridDim.x;
  const int begin = (int)(blockIdx.x * share + min(blockIdx.x, more));
  const int end = begin + (int)share + (blockIdx.x < more ? 1 : 0);
  auto chunks_of = [](const W4Active& a) { return (a.rows + kWideRows - 1) / kWideRows; };
  if (begin < end) {
    const int first_chunk = begin / p.blocks;
    for (int i = tid; i < (int)(found >> 32); i += kWideThreads)
      if (first_chunk >= act[i].chunk0 && first_chunk < act[i].chunk0 + chunks_of(act[i])) *first_act = i;
  }
  fence_proxy_async_smem();   // the sort's writes into the rings, before TMA's
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int steps = (p.K + 127) / 128;

  // the roles' common walk over the items
  struct Item {
    W4Active a;
    int block, row_first, rows;   // rows of this chunk
  };
  int at_act = begin < end ? *first_act : 0;
  auto item_at = [&](int item) {
    const int chunk = item / p.blocks;
    while (chunk >= act[at_act].chunk0 + chunks_of(act[at_act])) ++at_act;
    Item it;
    it.a = act[at_act];
    it.block = item - chunk * p.blocks;
    it.row_first = (chunk - it.a.chunk0) * kWideRows;
    it.rows = min(kWideRows, it.a.rows - it.row_first);
    return it;
  };
  auto subs_of = [&](int step) { return min(Ring::kSubs, (p.K - step * 128) / GROUP); };   // groups of a step
  auto wait = [&](uint32_t bar, uint32_t parity, uint32_t site) {
    return mbar_wait_warp(bar, parity, abort_flag, p.wait_limit_ns, p.status, site, kKernW4);
  };

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    int stage = 0;
    uint32_t phase = 0, issued = 0, last = 0;
    bool ok = true;
    for (int item = begin; item < end && ok; ++item) {
      const Item it = item_at(item);
      for (int st = 0; st < steps; ++st) {
        if (!(ok = wait(empty_q(stage), phase ^ 1u, 8))) break;
        if (lane == 0) {
          const uint32_t bar = full_q(stage);
          mbar_arrive_expect_tx(bar, Ring::kQ + 2 * Ring::kSubs * (ZEROS ? 192 : 128));
          const int qrow = it.a.expert * (p.K / 8) + st * 16, srow = it.a.expert * (p.K / GROUP) + st * Ring::kSubs;
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int col = it.block * 64 + b * 32;   // past the half's end: zeros
            tma_load_3d(smem_u32(codes + stage * Ring::kQ + b * 4096), &p.tm_q, col, 0, qrow, bar);
            tma_load_3d(smem_u32(scales + stage * Ring::kScale + b * 128 * Ring::kSubs), &p.tm_scale, col, 0, srow, bar);
            if (ZEROS) tma_load_3d(smem_u32(zeros + stage * Ring::kZero + b * Ring::kZeroBox), &p.tm_zero, col, 0, srow, bar);
          }
        }
        __syncwarp();
        issued |= 1u << stage;
        last = (last & ~(1u << stage)) | (phase << stage);
        if (++stage == kQStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) {   // stopped early: wait (bounded) for the copies in flight
      for (int s = 0; s < kQStages; ++s)
        if (issued & (1u << s)) {
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(full_q(s), (last >> s) & 1u) && globaltimer_ns() - t0 < p.wait_limit_ns) {
          }
        }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------- MMA issuer
    // The warp stays converged and an elected lane issues: the descriptors
    // are then uniform registers.
    int stage = 0, buf = 0;
    uint32_t phase = 0, dphase = 0;
    bool ok = true, issued_any = false;
    const uint64_t desc = umma_desc(0, 16, 1024);   // addresses are added in units of 16 bytes
    for (int item = begin; item < end && ok; ++item) {
      const Item it = item_at(item);
      const int cols = (it.rows + 15) & ~15;
      // D fp32, A and B bf16 K-major, M = 128, N = cols
      const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(cols >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
      for (int st = 0; st < steps && ok; ++st) {
        if (!(ok = wait(full_ab(stage), phase, 9))) break;
        tc_fence_after();
        const uint64_t da = desc + ((ab + stage * (kABytes + kBBytes)) >> 4), db = da + (kABytes >> 4);
        const int subs = subs_of(st);
#pragma unroll
        for (int sub = 0; sub < Ring::kSubs; ++sub) {
          if (sub >= subs) break;
          if (!(ok = wait(empty_d(buf), dphase ^ 1u, 10))) break;
          tc_fence_after();
          const uint32_t d = tmem_base + 64u * (uint32_t)buf;
#pragma unroll
          for (int i = 0; i < GROUP / 16; ++i) {
            const int kk = sub * (GROUP / 16) + i;   // 16 k: panel kk / 4, 32 bytes kk % 4
            mma_elected(d, da + (kk >> 2) * 1024 + (kk & 3) * 2, db + (kk >> 2) * (kWideRows * 8) + (kk & 3) * 2, idesc,
                        i != 0 ? 1u : 0u);
          }
          commit_elected(full_d(buf));
          issued_any = true;
          if (++buf == kDBuffers) {
            buf = 0;
            dphase ^= 1u;
          }
        }
        if (!ok) break;
        commit_elected(empty_ab(stage));
        if (++stage == kAbStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (issued_any) {   // every MMA has finished before the tensor memory is freed
      commit_elected(drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < p.wait_limit_ns) {
      }
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 4 + kTotalWarps) {
    // --------------------- totals: a lane to a column, a half of the rows
    constexpr int kRows = kWideRows / 2;
    const int row0 = ((warp - 4) >> 2) * kRows;
    const int m = (warp & 3) * 32 + lane, set = m >> 6, c = m & 63;   // column c of half `set`
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    int stage = 0, buf = 0;
    uint32_t phase = 0, dphase = 0, xphase = 0;
    bool ok = true;
    for (int item = begin; item < end && ok; ++item) {
      const Item it = item_at(item);
      const int rows = it.rows - row0;   // of this half, may be none
      float tot[kRows];
#pragma unroll
      for (int n = 0; n < kRows; ++n) tot[n] = 0.f;
      for (int st = 0; st < steps && ok; ++st) {
        if (!(ok = wait(full_q(stage), phase, 11))) break;
        const int subs = subs_of(st);
        const uint8_t* sc = scales + stage * Ring::kScale + (c >> 5) * 128 * Ring::kSubs + set * 64 + (c & 31) * 2;
        for (int sub = 0; sub < subs; ++sub) {
          const float scale = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(sc + sub * 128) << 16);
          if (!(ok = wait(full_d(buf), dphase, 12))) break;
          tc_fence_after();
#pragma unroll
          for (int n0 = 0; n0 < kRows; n0 += 16)
            if (n0 < rows) {
              float d[16];
              tmem_ld16(tmem_base + lanes + 64u * buf + row0 + n0, d);
#pragma unroll
              for (int n = 0; n < 16; ++n) tot[n0 + n] = fmaf(scale, d[n], tot[n0 + n]);
            }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(empty_d(buf));
          if (++buf == kDBuffers) {
            buf = 0;
            dphase ^= 1u;
          }
        }
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(empty_q(stage));
        if (++stage == kQStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      const int col = it.block * 64 + c;
      if (GATE_UP) {
        // the up columns' totals go to the gate columns' lanes through shared memory
        if (set == 1) {
          if (!(ok = wait(exch_empty, xphase ^ 1u, 13))) break;
#pragma unroll
          for (int n = 0; n < kRows; ++n)
            if (n < rows) exchange[(row0 + n) * 64 + c] = tot[n];
          __syncwarp();
          if (lane == 0) mbar_arrive(exch_full);
        } else {
          if (!(ok = wait(exch_full, xphase, 14))) break;
#pragma unroll
          for (int n = 0; n < kRows; ++n)
            if (n < rows && col < half) {
              const int64_t slot = slot0 + list[it.a.row0 + it.row_first + row0 + n];
              p.h[slot * half + col] = __bfloat16_as_ushort(__float2bfloat16_rn(w4_swiglu(tot[n], exchange[(row0 + n) * 64 + c])));
            }
          __syncwarp();
          if (lane == 0) mbar_arrive(exch_empty);
        }
        xphase ^= 1u;
      } else {
#pragma unroll
        for (int n = 0; n < kRows; ++n)
          if (n < rows && col < half) {
            const int64_t slot = slot0 + list[it.a.row0 + it.row_first + row0 + n];
            p.part[slot * p.N + set * half + col] = tot[n];
          }
      }
    }
  } else if (warp >= 4 + kTotalWarps) {
    // -------------------------------------------------------- decoders
    const int dw = (warp - 4 - kTotalWarps) % kDecoders, group = (warp - 4 - kTotalWarps) / kDecoders;
    const int dtid = dw * 32 + lane;
    const int g = lane >> 2, t = lane & 3;
    const int xrow = dtid >> 4, xchunk = dtid & 15;   // rows xrow + 16 j, 16-byte chunk of the step's 128 k
    // step s of the block (over all its items) is group s % 2's, in code
    // stage s % kQStages and A, B stage s % kAbStages
    int stage = group, astage = group, turn = group;   // turn: this group's next step of the item
    uint32_t phase = 0, aphase = 0;
    bool ok = true;
    for (int item = begin; item < end && ok; ++item, turn -= steps) {
      const Item it = item_at(item);
      const uint16_t* x[4];
      uint4 xn[4];
      auto load_x = [&](int st) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          xn[j] = make_uint4(0, 0, 0, 0);   // rows past the chunk's, k past K
          if (x[j] && st * 128 + xchunk * 8 < p.K) xn[j] = __ldg(reinterpret_cast<const uint4*>(x[j] + st * 128 + xchunk * 8));
        }
      };
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = xrow + 16 * j;
        x[j] = nullptr;
        if (r < it.rows) {
          const int slot = slot0 + list[it.a.row0 + it.row_first + r];
          x[j] = p.rows + (int64_t)(GATE_UP ? slot / p.k : slot) * p.K;
        }
      }
      load_x(turn);
      for (; turn < steps; turn += 2) {
        if (!(ok = wait(empty_ab(astage), aphase ^ 1u, 15))) break;
        const uint32_t sA = ab + astage * (kABytes + kBBytes), sB = sA + kABytes;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (16 * j < it.rows) {   // the MMA reads rows up to the next multiple of 16
            const int r = xrow + 16 * j;
            const uint4 v = xn[j];
            st_shared16(sB + (xchunk >> 3) * (kWideRows * 128) + r * 128 + (((xchunk & 7) ^ (r & 7)) << 4),
                        __byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                        __byte_perm(v.y, v.w, 0x7632));
          }
        load_x(turn + 2);   // past K: zeros
        if (!(ok = wait(full_q(stage), phase, 16))) break;
        // two pieces of 32 columns of a half x 4 word rows
        uint4 v[2];
        uint32_t zr[2] = {0x08080808u, 0x08080808u};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int sub = dw * 2 + q, b = sub >> 3, set = (sub >> 2) & 1, rq = sub & 3;
          const int line = (rq * 4 + t) * 2 + set;
          v[q] = *reinterpret_cast<const uint4*>(codes + stage * Ring::kQ + b * 4096 + line * 128 + ((g ^ (line & 7)) << 4));
          if (ZEROS)
            zr[q] = *reinterpret_cast<const uint32_t*>(zeros + stage * Ring::kZero + b * Ring::kZeroBox + ((rq * 32 / GROUP) * 2 + set) * 32 + g * 4);
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int sub = dw * 2 + q, b = sub >> 3, set = (sub >> 2) & 1, rq = sub & 3;
          const uint32_t word[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
          const int r = rq * 4 + t;   // word row: 16-byte chunk r of the column's 128 k
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t zero2 = 0x43004300u + ((zr[q] >> (8 * j)) & 255u) * 0x00010001u;
            const int row = set * 64 + b * 32 + g * 4 + j;
            st_shared16(sA + (r >> 3) * 16384 + row * 128 + (((r & 7) ^ (row & 7)) << 4), w4_less_zero(word[j], 0, zero2),
                        w4_less_zero(word[j], 1, zero2), w4_less_zero(word[j], 2, zero2), w4_less_zero(word[j], 3, zero2));
          }
        }
        fence_proxy_async_smem();   // A and B, before the tensor cores read them
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(full_ab(astage));
          mbar_arrive(empty_q(stage));
        }
        if ((stage += 2) >= kQStages) {
          stage -= kQStages;
          phase ^= 1u;
        }
        if ((astage += 2) >= kAbStages) {
          astage -= kAbStages;
          aphase ^= 1u;
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kDBuffers * 64);
  }
}

template <bool GATE_UP, int GROUP, bool ZEROS>
cudaError_t launch_wide(const W4Params& p, const DeviceInfo& dev, cudaStream_t stream) {
  const int row_slots = std::min(p.slots_per_row, p.slots);
  const int bytes = wide_smem<GROUP, ZEROS>(p.E, row_slots);
  static std::atomic<int> configured[kMaxDevices] = {};   // per device (a race only repeats the set-up)
  if (!configured[dev.ordinal].load()) {
    const cudaError_t err = cudaFuncSetAttribute(w4_wide_kernel<GATE_UP, GROUP, ZEROS>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 wide_smem<GROUP, ZEROS>(kMaxExperts, kWideMaxSlots));
    if (err != cudaSuccess) return err;
    configured[dev.ordinal].store(1);
  }
  const int rows = (p.slots + p.slots_per_row - 1) / p.slots_per_row;
  const int64_t most = (int64_t)row_slots * p.blocks;
  return launch_pdl(w4_wide_kernel<GATE_UP, GROUP, ZEROS>,
                    dim3((unsigned)std::min<int64_t>(most, dev.num_sms), (unsigned)rows), dim3(kWideThreads), bytes, stream,
                    1, p);
}

template <bool GATE_UP>
cudaError_t launch_wide_group(W4Params& p, int64_t group, bool zeros, const DeviceInfo& dev, cudaStream_t stream) {
  p.slots_per_row = w4_row_slots(p.E, p.k, kWideMaxSlots, kSortBytes);
  p.blocks = (p.N / 2 + 63) / 64;
  if (group == 32) return zeros ? launch_wide<GATE_UP, 32, true>(p, dev, stream) : launch_wide<GATE_UP, 32, false>(p, dev, stream);
  if (group == 64) return zeros ? launch_wide<GATE_UP, 64, true>(p, dev, stream) : launch_wide<GATE_UP, 64, false>(p, dev, stream);
  return zeros ? launch_wide<GATE_UP, 128, true>(p, dev, stream) : launch_wide<GATE_UP, 128, false>(p, dev, stream);
}

}  // namespace

cudaError_t launch_w4_wide(W4Params& p, bool gate_up, int64_t group, bool zeros, const DeviceInfo& dev,
                           cudaStream_t stream) {
  return gate_up ? launch_wide_group<true>(p, group, zeros, dev, stream)
                 : launch_wide_group<false>(p, group, zeros, dev, stream);
}

}  // namespace moe
