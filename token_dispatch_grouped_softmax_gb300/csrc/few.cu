// The expert layer for a few tokens in bf16, rows in slot order:
//
//   h[t, j] = silu(x_t . Wg_e) * (x_t . Wu_e),  e = ids[t, j]
//   y_t = sum_j w[t, j] (h[t, j] . Wd_e)  (+ the shared expert's, weight 1)
//
// With few rows an expert the weights' bytes are the cost: each weight of the
// experts in use has to come from HBM once.  One launch streams them all.  A
// unit of work is 128 columns of one expert's weight (64 gate and the 64 up
// columns beside them, or 128 of down) by a part of its K rows, for up to 32
// rows of that expert; gate_up's units come before down's.  Blocks draw units
// by tickets in that order, so that a block that waits for an expert's h
// waits only for units that running blocks have drawn: no block has to be
// resident for another to go on.
//
//   warp 3        draws the units, little ahead of the loads.
//   warp 0        keeps a ring of 128 x 128 tiles of the weights full by TMA.  It waits for nothing but free stages:
//                 while h is not ready, down's weights already arrive.
//   warp 1        gathers the rows' 128 values of K for each tile (TMA
//                 gather4), for down once the expert's h is complete.
//   warp 2        issues tcgen05.mma, the weights as A (M = 128 columns,
//                 MN-major as they lie) and the rows as B (N = 32): the
//                 accumulator has a column of the weight in each TMEM lane.
//   warps 4..19   four groups take the units in turn: TMEM to the unit's fp32
//                 partial sums in the workspace; whoever adds the last part
//                 of a tile sums the parts in order and writes h, and of a
//                 token's columns y.
//
// The parts of K depend on K alone, so a token's sums have one order and its
// result does not depend on the batch.
#include <algorithm>

#include "kernels.h"

namespace moe {

namespace {

constexpr int kFewGroups = 4;                  // of the epilogue, four warps each
constexpr int kFewThreads = 128 + 128 * kFewGroups;
constexpr int kFewRows = 32;                   // rows of a unit, N of an MMA
constexpr int kFewK = 128;                     // K rows of a stage
constexpr int kFewTile = kFewK * 128 * 2;      // its weights: 128 columns
constexpr int kFewHalf = kFewRows * 128;       // its rows' first 64 values of K
constexpr int kFewStage = kFewTile + 2 * kFewHalf;
constexpr int kFewMaxStages = 5;
constexpr int kFewParts = 8;                   // of K, at most
constexpr int kFewAcc = 8;                     // accumulators in TMEM
constexpr int kFewQueue = 16;                  // units between warp 3 and the epilogue
constexpr int kFewAhead = 2;                   // units that warp 3 has drawn beyond warp 0's
constexpr int kFewSmem = 232448;               // what a block may have (227 KB)
constexpr int kPrepThreads = 1024;

enum : uint32_t { kFewSitePrep = 1, kFewSiteTile = 2, kFewSiteRows = 3, kFewSiteMma = 4, kFewSiteEpi = 5, kFewSiteHidden = 6, kFewSiteUnits = 7 };

// One of an expert's two products: K rows in parts of part_k, N columns in tiles.
struct FewProduct {
  int K, parts, part_k, tiles;
};

struct FewEntry {       // an expert in use
  int expert, row0, rows, chunk0;    // its rows in the list, its first chunk of 32 rows
};

struct FewUnit {
  int kind;             // kGateUp, kDown or kEnd
  int shared;
  int entry;
  int row0, rows;       // in the list (shared: tokens)
  int chunk;
  int tile, part;
  int halves;           // 64 K rows each; a stage holds two, the last perhaps one
  int w_row, k0;        // first K row: of the weight matrix, of the part
};
enum { kGateUp, kDown, kEnd };

struct FewParams {      // 64-byte aligned through its CUtensorMap members
  CUtensorMap tm_gate_up, tm_down, tm_sh_gate_up, tm_sh_down, tm_x, tm_h, tm_sh_h;
  const int32_t* ids;
  const float* w;
  uint16_t* y;
  // workspace
  uint32_t* ticket;
  uint32_t* done;       // [entries + 1] finished tiles of h of each entry, the shared expert's last
  uint32_t* hidden;     // [chunks + shared chunks][tiles] parts of a gate_up tile that are there
  uint32_t* arrived;    // [tiles of down][T] slots' parts of a token's columns that are there
  int* head;            // entries, chunks
  FewEntry* entries;
  uint16_t* list;       // slots by expert
  uint16_t* of_chunk;   // entry of a chunk
  uint8_t* valid;       // slots of a token that name an expert
  float *part_gu, *part_sh_gu, *part_dn, *part_sh_dn;
  uint16_t *h, *sh_h;
  uint32_t* status;
  uint64_t wait_limit_ns;
  FewProduct gu, dn, sh_gu, sh_dn;
  int T, H, E, k, I, I_s;
  int max_entries, max_chunks, sh_chunks;
  int zero_words;       // counters from `ticket` on
  int stages;
  int stall;
};

// --------------------------------------------------------------- the lists

// One block: clears the counters and sorts the slots by expert (stable).
__global__ void __launch_bounds__(kPrepThreads) few_prep_kernel(const __grid_constant__ FewParams p) {
  extern __shared__ int few_prep_smem[];
  int* ids = few_prep_smem;                    // [S]
  int* first = ids + p.T * p.k;                // [E] counts, then the first place
  __shared__ int warp_sums[2][32];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slots = p.T * p.k;
  for (int i = tid; i < p.zero_words; i += kPrepThreads) p.ticket[i] = 0;
  for (int e = tid; e < p.E; e += kPrepThreads) first[e] = 0;
  bool bad = false;
  for (int i = tid; i < slots; i += kPrepThreads) {
    int e = p.ids[i];
    if (e < 0 || e >= p.E) {
      bad |= e != -1;
      e = -1;
    }
    ids[i] = e;
  }
  if (bad) report_status(p.status, kStatusDevice, kKernFew, kFewSitePrep);
  __syncthreads();
  int rank[4];                                 // slots <= 4096
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int i = tid + q * kPrepThreads;
    rank[q] = -1;
    if (i < slots && ids[i] >= 0) {
      int r = 0;
      for (int j = 0; j < i; ++j) r += ids[j] == ids[i];
      rank[q] = r;
      atomicAdd(&first[ids[i]], 1);
    }
  }
  for (int t = tid; t < p.T; t += kPrepThreads) {
    int n = 0;
    for (int j = 0; j < p.k; ++j) n += ids[t * p.k + j] >= 0;
    p.valid[t] = (uint8_t)n;
  }
  __syncthreads();
  // experts in order: rows, chunks and entries before each (E <= 1024: one a thread)
  const int rows = tid < p.E ? first[tid] : 0;
  const int chunks = (rows + kFewRows - 1) / kFewRows;
  int a = rows, b = chunks << 16 | (rows > 0);   // inclusive sums: rows; chunks and entries
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a += x;
      b += y;
    }
  }
  if (lane == 31) {
    warp_sums[0][warp] = a;
    warp_sums[1][warp] = b;
  }
  __syncthreads();
  int all = 0;
  for (int i = 0; i < kPrepThreads / 32; ++i) {
    if (i < warp) {
      a += warp_sums[0][i];
      b += warp_sums[1][i];
    }
    all += warp_sums[1][i];
  }
  const int row0 = a - rows, chunk0 = (b >> 16) - chunks, entry = (b & 0xFFFF) - (rows > 0);
  if (tid < p.E) first[tid] = row0;
  if (rows > 0) {
    p.entries[entry] = FewEntry{tid, row0, rows, chunk0};
    for (int c = 0; c < chunks; ++c) p.of_chunk[chunk0 + c] = (uint16_t)entry;
  }
  if (tid == 0) {
    p.head[0] = all & 0xFFFF;
    p.head[1] = all >> 16;
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (rank[q] >= 0) p.list[first[ids[tid + q * kPrepThreads]] + rank[q]] = (uint16_t)(tid + q * kPrepThreads);
}

// --------------------------------------------------------------- the units

// Unit `u` of the launch; the entries in shared memory.
__device__ __forceinline__ FewUnit few_unit(const FewParams& p, const FewEntry* entries, const uint16_t* of_chunk, int chunks,
                                            uint32_t u) {
  FewUnit x;
  x.kind = kEnd;
  FewProduct f;
  // the products in the order of their units; false: u is beyond this one's
  auto in = [&](const FewProduct& product, int n, int kind, int shared) {
    const uint32_t units = (uint32_t)n * (product.tiles * product.parts);
    if (u >= units) {
      u -= units;
      return false;
    }
    f = product;
    x.kind = kind;
    x.shared = shared;
    return true;
  };
  if (!(in(p.sh_gu, p.sh_chunks, kGateUp, 1) || in(p.gu, chunks, kGateUp, 0) || in(p.sh_dn, p.sh_chunks, kDown, 1) ||
        in(p.dn, chunks, kDown, 0)))
    return x;
  const uint32_t per = f.tiles * f.parts;
  int entry = 0, chunk0 = 0, n_chunks = p.sh_chunks, rows = p.T, row0 = 0, expert = 0;
  if (!x.shared) {
    entry = of_chunk[u / per];
    const FewEntry e = entries[entry];
    chunk0 = e.chunk0;
    rows = e.rows;
    row0 = e.row0;
    expert = e.expert;
    n_chunks = (rows + kFewRows - 1) / kFewRows;
  }
  // an expert's chunks read the same weights one after another, then come the
  // tiles, whose columns lie side by side, then the parts
  const uint32_t local = u - chunk0 * per;
  const int c = local % n_chunks;
  const uint32_t at = local / n_chunks;
  x.entry = x.shared ? p.max_entries : entry;
  x.chunk = (x.shared ? p.max_chunks : chunk0) + c;
  x.row0 = row0 + c * kFewRows;
  x.rows = min(kFewRows, rows - c * kFewRows);
  x.tile = at % f.tiles;
  x.part = at / f.tiles;
  x.k0 = x.part * f.part_k;
  x.halves = min(f.part_k, f.K - x.k0) / 64;
  x.w_row = expert * f.K + x.k0;
  return x;
}

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// A barrier of a group's 128 threads that says whether `ok` holds on all of them.
__device__ __forceinline__ bool group_all(int group, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
      " barrier.cta.red.and.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)ok), "r"(1 + group)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int group) { asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory"); }

__device__ __forceinline__ void gather4(uint32_t dst, const CUtensorMap* map, int k, const int (&row)[4], uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(k), "r"(row[0]), "r"(row[1]), "r"(row[2]), "r"(row[3]), "r"(bar)
      : "memory");
}

constexpr size_t few_tables_bytes(int64_t entries, int64_t chunks, int64_t slots) {
  return (size_t)(entries * sizeof(FewEntry) + (chunks + slots) * sizeof(uint16_t) + 15) & ~(size_t)15;
}
constexpr int kFewBars = 3 * kFewMaxStages + 2 * kFewAcc + 2 * kFewQueue + kFewAhead + 1;
constexpr size_t kFewFixed = kFewBars * 8 + kFewQueue * sizeof(FewUnit) + 64;

__global__ void __launch_bounds__(kFewThreads, 1) few_kernel(const __grid_constant__ FewParams p) {
  extern __shared__ uint8_t few_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(few_smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.stages * kFewStage);
  FewUnit* queue = reinterpret_cast<FewUnit*>(bars + kFewBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(queue + kFewQueue);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* group_word = tmem_slot + 2;        // [groups]
  FewEntry* entries = reinterpret_cast<FewEntry*>(smem + p.stages * kFewStage + kFewFixed);
  uint16_t* of_chunk = reinterpret_cast<uint16_t*>(entries + p.max_entries);
  uint16_t* list = of_chunk + p.max_chunks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t ring = smem_u32(smem), bar0 = smem_u32(bars);
  const int S = p.stages;
  auto tile_bar = [&](int s) { return bar0 + 8u * s; };                                  // a stage's weights are there
  auto rows_bar = [&](int s) { return bar0 + 8u * (kFewMaxStages + s); };                // its rows are
  auto free_bar = [&](int s) { return bar0 + 8u * (2 * kFewMaxStages + s); };            // it may be filled
  auto acc_bar = [&](int a) { return bar0 + 8u * (3 * kFewMaxStages + a); };             // an accumulator is complete
  auto read_bar = [&](int a) { return bar0 + 8u * (3 * kFewMaxStages + kFewAcc + a); };  // it has been read
  auto unit_bar = [&](int q) { return bar0 + 8u * (3 * kFewMaxStages + 2 * kFewAcc + q); };
  auto seen_bar = [&](int q) { return bar0 + 8u * (3 * kFewMaxStages + 2 * kFewAcc + kFewQueue + q); };
  auto begun_bar = [&](int i) { return bar0 + 8u * (3 * kFewMaxStages + 2 * kFewAcc + 2 * kFewQueue + i); };   // warp 0 has taken a unit
  const uint32_t drain_bar = bar0 + 8u * (kFewBars - 1);

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(tile_bar(s), 1);
      mbar_init(rows_bar(s), 1);
      mbar_init(free_bar(s), 1);
    }
    for (int a = 0; a < kFewAcc; ++a) {
      mbar_init(acc_bar(a), 1);
      mbar_init(read_bar(a), 4);
    }
    for (int q = 0; q < kFewQueue; ++q) {
      mbar_init(unit_bar(q), 1);
      mbar_init(seen_bar(q), 7);   // warps 0 to 2, four warps of a group
    }
    for (int i = 0; i < kFewAhead; ++i) mbar_init(begun_bar(i), 1);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tm_gate_up);
    tma_prefetch_desc(&p.tm_down);
    tma_prefetch_desc(&p.tm_x);
    tma_prefetch_desc(&p.tm_h);
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(tmem_slot), kFewAcc * kFewRows);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  const int n_entries = p.head[0], n_chunks = p.head[1];
  for (int i = tid; i < n_entries; i += kFewThreads) entries[i] = p.entries[i];
  for (int i = tid; i < n_chunks; i += kFewThreads) of_chunk[i] = p.of_chunk[i];
  for (int i = tid; i < p.T * p.k; i += kFewThreads) list[i] = p.list[i];
  for (int t = blockIdx.x; t < p.T; t += gridDim.x)   // tokens without an expert
    if (p.valid[t] == 0 && p.I_s == 0)
      for (int c = tid * 8; c < p.H; c += kFewThreads * 8)
        *reinterpret_cast<uint4*>(p.y + (int64_t)t * p.H + c) = make_uint4(0, 0, 0, 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](uint32_t bar, uint32_t parity, uint32_t site) {
    return mbar_wait_bounded(bar, parity, abort_flag, p.wait_limit_ns, p.status, site, kKernFew);
  };
  auto wait_warp = [&](uint32_t bar, uint32_t parity, uint32_t site) {
    return mbar_wait_warp(bar, parity, abort_flag, p.wait_limit_ns, p.status, site, kKernFew);
  };
  // after an early stop: a stage's copies have landed (bounded)
  auto land = [&](uint32_t bar, uint32_t parity) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t0 < p.wait_limit_ns) {
    }
  };

  if (warp == 3) {
    if (lane == 0) {
      uint32_t next = atomicAdd(p.ticket, 1u);
      for (int i = 0, ends = 0; ends < kFewGroups; ++i) {
        const FewUnit x = few_unit(p, entries, of_chunk, n_chunks, next);
        const int q = i % kFewQueue;
        // no further ahead of the loads, so that the blocks draw evenly
        if (i >= kFewAhead && x.kind != kEnd && !wait(begun_bar(i % kFewAhead), (i / kFewAhead - 1) & 1, kFewSiteUnits)) break;
        if (!wait(seen_bar(q), (i / kFewQueue & 1) ^ 1u, kFewSiteUnits)) break;
        queue[q] = x;
        mbar_arrive(unit_bar(q));
        if (x.kind == kEnd) {   // one for each group
          ++ends;
          continue;
        }
        next = atomicAdd(p.ticket, 1u);
      }
    }
  } else if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued = 0, parity = 0;   // bits of the stages
      bool ok = true;
      for (int i = 0; ok; ++i) {
        const int q = i % kFewQueue;
        ok = wait(unit_bar(q), i / kFewQueue & 1, kFewSiteTile);
        if (!ok) break;
        const FewUnit x = queue[q];
        mbar_arrive(seen_bar(q));
        mbar_arrive(begun_bar(i % kFewAhead));
        if (x.kind == kEnd) break;
        const CUtensorMap* map = x.kind == kGateUp ? (x.shared ? &p.tm_sh_gate_up : &p.tm_gate_up)
                                                   : (x.shared ? &p.tm_sh_down : &p.tm_down);
        const int c0 = x.kind == kGateUp ? 64 * x.tile : 128 * x.tile;
        const int c1 = x.kind == kGateUp ? (x.shared ? p.I_s : p.I) + c0 : c0 + 64;
        const bool both = x.kind == kGateUp || c1 < p.H;
        for (int s = 0; s < x.halves; s += 2) {
          ok = wait(free_bar(stage), phase ^ 1u, kFewSiteTile);
          if (!ok) break;
          if (!p.stall) {
            const uint32_t dst = ring + stage * kFewStage;
            mbar_arrive_expect_tx(tile_bar(stage), both ? kFewTile : kFewTile / 2);
            tma_load_2d(dst, map, c0, x.w_row + 64 * s, tile_bar(stage));
            if (both) tma_load_2d(dst + kFewTile / 2, map, c1, x.w_row + 64 * s, tile_bar(stage));
            issued |= 1u << stage;
            parity = (parity & ~(1u << stage)) | phase << stage;
          }
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok)
        for (int s = 0; s < S; ++s)
          if (issued >> s & 1u) land(tile_bar(s), parity >> s & 1u);
    }
  } else if (warp == 1) {
    int stage = 0, ready = -1;   // the entry whose h is known to be complete
    uint32_t phase = 0, issued = 0, parity = 0;
    bool ok = true;
    for (int i = 0; ok; ++i) {
      const int q = i % kFewQueue;
      ok = wait_warp(unit_bar(q), i / kFewQueue & 1, kFewSiteRows);
      if (!ok) break;
      const FewUnit x = queue[q];
      __syncwarp();
      if (lane == 0) mbar_arrive(seen_bar(q));
      if (x.kind == kEnd) break;
      int row[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int at = x.row0 + min(4 * lane + r, x.rows - 1);
        row[r] = x.shared ? at : x.kind == kDown ? list[at] : list[at] / p.k;
      }
      const CUtensorMap* map = x.kind == kGateUp ? &p.tm_x : x.shared ? &p.tm_sh_h : &p.tm_h;
      const int groups = (x.rows + 3) / 4;
      if (x.kind == kDown && ready != x.entry) {
        const FewProduct& f = x.shared ? p.sh_gu : p.gu;
        const int chunks = x.shared ? p.sh_chunks : (entries[x.entry].rows + kFewRows - 1) / kFewRows;
        const uint32_t need = (uint32_t)(chunks * f.tiles);
        if (ld_acquire(p.done + x.entry) < need) {
          const uint64_t t0 = globaltimer_ns();
          for (uint32_t n = 1; ld_acquire(p.done + x.entry) < need; ++n) {
            if ((n & 15u) != 0) continue;
            if (*abort_flag) ok = false;
            else if (globaltimer_ns() - t0 > p.wait_limit_ns) {
              *abort_flag = 1;
              report_status(p.status, kStatusTimeout, kKernFew, kFewSiteHidden);
              ok = false;
            }
            if (!ok) break;
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        fence_proxy_async_all();   // h was written by ordinary stores
        ready = x.entry;
      }
      for (int s = 0; s < x.halves; s += 2) {
        ok = wait_warp(free_bar(stage), phase ^ 1u, kFewSiteRows);
        if (!ok) break;
        const int halves = min(2, x.halves - s);
        if (lane == 0) mbar_arrive_expect_tx(rows_bar(stage), halves * groups * 512);
        __syncwarp();
        if (lane < groups) {
          const uint32_t dst = ring + stage * kFewStage + kFewTile + lane * 512;
          gather4(dst, map, x.k0 + 64 * s, row, rows_bar(stage));
          if (halves == 2) gather4(dst + kFewHalf, map, x.k0 + 64 * s + 64, row, rows_bar(stage));
        }
        issued |= 1u << stage;
        parity = (parity & ~(1u << stage)) | phase << stage;
        if (++stage == S) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && lane == 0)
      for (int s = 0; s < S; ++s)
        if (issued >> s & 1u) land(rows_bar(s), parity >> s & 1u);
  } else if (warp == 2) {
    if (lane == 0) {
      // D fp32, A and B bf16, A MN-major, N = 32, M = 128
      const uint32_t idesc = 1u << 4 | 1u << 7 | 1u << 10 | 1u << 15 | (uint32_t)(kFewRows >> 3) << 17 | 8u << 24;
      const uint64_t a0 = umma_desc(ring, kFewTile / 2, 1024), b0 = umma_desc(ring + kFewTile, 16, 1024);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true, issued = false;
      for (int i = 0; ok; ++i) {
        const int q = i % kFewQueue, a = i % kFewAcc;
        ok = wait(unit_bar(q), i / kFewQueue & 1, kFewSiteMma);
        if (!ok) break;
        const int kind = queue[q].kind, halves = queue[q].halves;
        mbar_arrive(seen_bar(q));
        if (kind == kEnd) break;
        ok = wait(read_bar(a), (i / kFewAcc & 1) ^ 1u, kFewSiteMma);
        if (!ok) break;
        tc_fence_after();
        for (int s = 0; s < halves; s += 2) {
          ok = wait(tile_bar(stage), phase, kFewSiteMma) && wait(rows_bar(stage), phase, kFewSiteMma);
          if (!ok) break;
          tc_fence_after();
          const uint64_t at = (uint64_t)(stage * kFewStage) >> 4;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            if (kk < 4 || s + 1 < halves)
              tc_mma_bf16(tmem + a * kFewRows, a0 + at + kk * (2048 >> 4), b0 + at + ((kk >> 2) * kFewHalf + (kk & 3) * 32 >> 4), idesc,
                          (s | kk) != 0);
          tc_commit(free_bar(stage));
          issued = true;
          if (++stage == S) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (ok) tc_commit(acc_bar(a));
      }
      if (!ok && issued) {
        tc_commit(drain_bar);
        land(drain_bar, 0);
      }
    }
  } else if (warp >= 4) {
    const int group = (warp - 4) >> 2, m = tid & 127;   // m: the column of the tile, and the TMEM lane
    for (int i = group;; i += kFewGroups) {
      const int q = i % kFewQueue, a = i % kFewAcc;
      FewUnit x;
      x.kind = kEnd;
      bool ok = wait_warp(unit_bar(q), i / kFewQueue & 1, kFewSiteEpi);
      if (ok) x = queue[q];
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(seen_bar(q));
      if (ok && x.kind != kEnd) ok = wait_warp(acc_bar(a), i / kFewAcc & 1, kFewSiteEpi);
      ok = group_all(group, ok);
      if (!ok || x.kind == kEnd) break;
      tc_fence_after();
      float v[kFewRows];
      tmem_ld32(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + a * kFewRows, v);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(read_bar(a));
      const bool gate_up = x.kind == kGateUp;
      const int I = x.shared ? p.I_s : p.I;
      const FewProduct& f = gate_up ? (x.shared ? p.sh_gu : p.gu) : (x.shared ? p.sh_dn : p.dn);
      float* part = gate_up ? (x.shared ? p.part_sh_gu : p.part_gu) : (x.shared ? p.part_sh_dn : p.part_dn);
      const int width = gate_up ? 2 * I : p.H;
      const int c = gate_up ? (m < 64 ? 64 * x.tile + m : I + 64 * x.tile + m - 64) : 128 * x.tile + m;
      if (c < width) {
#pragma unroll
        for (int r = 0; r < kFewRows; ++r) {
          if (r < x.rows) {
            const int row = x.shared ? x.row0 + r : list[x.row0 + r];
            __stcg(part + ((int64_t)row * f.parts + x.part) * width + c, v[r]);
          }
        }
      }
      group_sync(group);
      if (m < 32) __threadfence();   // the group's stores, before the counts
      if (gate_up) {
        if (m == 0) group_word[group] = atomicAdd(p.hidden + (x.shared ? (int64_t)p.max_chunks * p.gu.tiles + (int64_t)(x.chunk - p.max_chunks) * f.tiles
                                                                       : (int64_t)x.chunk * f.tiles) + x.tile, 1u);
        group_sync(group);
        if (group_word[group] + 1 != (uint32_t)f.parts) continue;
        __threadfence();
        uint16_t* h = x.shared ? p.sh_h : p.h;
        const int n = 64 * x.tile + (m & 63);
        for (int r = m >> 6; r < x.rows; r += 2) {
          const int row = x.shared ? x.row0 + r : list[x.row0 + r];
          const float* from = part + (int64_t)row * f.parts * width + n;
          float g = 0.f, u = 0.f;
#pragma unroll
          for (int j = 0; j < kFewParts; ++j)
            if (j < f.parts) {
              g += __ldcg(from + (int64_t)j * width);
              u += __ldcg(from + (int64_t)j * width + I);
            }
          // rounded as the grouped GEMMs round it: an operand of the tensor cores
          h[(int64_t)row * I + n] = __bfloat16_as_ushort(__float2bfloat16_rn(__fdividef(g, 1.0f + __expf(-g)) * u));
        }
        fence_proxy_async_all();   // h is read by TMA
        group_sync(group);
        if (m == 0) {
          __threadfence();
          atomicAdd(p.done + x.entry, 1u);
        }
      } else {
        if (m < 32) {   // the rows' tokens whose columns are complete
          int t = 0;
          bool last = false;
          if (m < x.rows) {
            t = x.shared ? x.row0 + m : list[x.row0 + m] / p.k;
            const uint32_t all = (uint32_t)p.valid[t] * p.dn.parts + (p.I_s ? p.sh_dn.parts : 0);
            last = atomicAdd(p.arrived + (int64_t)x.tile * p.T + t, 1u) + 1 == all;
          }
          const uint32_t mask = __ballot_sync(0xffffffffu, last);
          if (m == 0) group_word[group] = mask;
        }
        group_sync(group);
        uint32_t mask = group_word[group];
        if (mask) __threadfence();
        while (mask) {
          const int r = __ffs(mask) - 1;
          mask &= mask - 1;
          if (c >= p.H) continue;
          const int t = x.shared ? x.row0 + r : list[x.row0 + r] / p.k;
          float y = 0.f;
          for (int j0 = 0; j0 < p.k; j0 += 4) {   // four slots' parts in flight
            float s[4], wt[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int slot = t * p.k + j0 + j;
              const bool in = j0 + j < p.k && (uint32_t)p.ids[slot] < (uint32_t)p.E;
              wt[j] = in ? p.w[slot] : 0.f;
              s[j] = 0.f;
              const float* from = p.part_dn + (int64_t)slot * p.dn.parts * p.H + c;
#pragma unroll
              for (int l = 0; l < kFewParts; ++l)
                if (in && l < p.dn.parts) s[j] += __ldcg(from + (int64_t)l * p.H);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) y = fmaf(wt[j], s[j], y);
          }
          if (p.I_s) {
            const float* from = p.part_sh_dn + (int64_t)t * p.sh_dn.parts * p.H + c;
            float s = 0.f;
#pragma unroll
            for (int l = 0; l < kFewParts; ++l)
              if (l < p.sh_dn.parts) s += __ldcg(from + (int64_t)l * p.H);
            y += s;
          }
          p.y[(int64_t)t * p.H + c] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) tmem_dealloc(tmem, kFewAcc * kFewRows);
}

// K in at most 8 parts of at least 256 rows, whole stages.
FewProduct few_product(int64_t K, int64_t tiles) {
  FewProduct f;
  f.K = (int)K;
  f.tiles = (int)tiles;
  const int64_t parts = std::min<int64_t>(kFewParts, std::max<int64_t>(1, K / 256)), stages = (K + kFewK - 1) / kFewK;
  f.part_k = (int)((stages + parts - 1) / parts * kFewK);
  f.parts = K ? (int)((K + f.part_k - 1) / f.part_k) : 0;
  return f;
}

// Everything of a call but its pointers: the products, and where the
// workspace's pieces begin.
struct FewPlan {
  FewProduct gu, dn, sh_gu, sh_dn;
  int64_t slots, max_entries, max_chunks, sh_chunks, zero_words;
  size_t done, hidden, arrived, head, entries, list, of_chunk, valid, part_gu, part_sh_gu, part_dn, part_sh_dn, h, sh_h, bytes;
};

FewPlan few_plan(const FewShape& s) {
  FewPlan f;
  f.gu = few_product(s.H, s.I / 64);
  f.dn = few_product(s.I, (s.H + 127) / 128);
  f.sh_gu = few_product(s.I_s ? s.H : 0, s.I_s / 64);
  f.sh_dn = few_product(s.I_s, s.I_s ? (s.H + 127) / 128 : 0);
  f.slots = s.T * s.k;
  f.max_entries = std::min(s.E, f.slots);
  f.max_chunks = std::min(f.slots, f.max_entries + f.slots / kFewRows);
  f.sh_chunks = s.I_s ? (s.T + kFewRows - 1) / kFewRows : 0;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = (at + bytes + 15) & ~(size_t)15;
    return here;
  };
  take(16);   // the ticket
  f.done = take((f.max_entries + 1) * 4);
  f.hidden = take((f.max_chunks * f.gu.tiles + f.sh_chunks * f.sh_gu.tiles) * 4);
  f.arrived = take(f.dn.tiles * s.T * 4);
  f.zero_words = at / 4;
  f.head = take(8);
  f.entries = take(f.max_entries * sizeof(FewEntry));
  f.list = take(f.slots * 2);
  f.of_chunk = take(f.max_chunks * 2);
  f.valid = take(s.T);
  at = (at + 255) & ~(size_t)255;
  f.part_gu = take((size_t)f.slots * f.gu.parts * 2 * s.I * 4);
  f.part_sh_gu = take((size_t)s.T * f.sh_gu.parts * 2 * s.I_s * 4);
  f.part_dn = take((size_t)f.slots * f.dn.parts * s.H * 4);
  f.part_sh_dn = take((size_t)s.T * f.sh_dn.parts * s.H * 4);
  f.h = take((size_t)f.slots * s.I * 2);
  f.sh_h = take((size_t)s.T * s.I_s * 2);
  f.bytes = at;
  return f;
}

bool few_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(cols * 2)};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return encode_tensor_map_2d_bf16(map, base, dims, strides, box, estr);
}

}  // namespace

size_t few_experts_workspace_bytes(const FewShape& s) { return few_plan(s).bytes; }

int launch_few_experts(const FewShape& s, const uint16_t* x, const int32_t* ids, const float* w, const FewWeights& weights,
                       uint16_t* y, void* ws, const DeviceInfo& dev, cudaStream_t stream) {
  const FewPlan f = few_plan(s);
  uint8_t* base = static_cast<uint8_t*>(ws);
  FewParams p;
  p.ids = ids; p.w = w; p.y = y;
  p.ticket = reinterpret_cast<uint32_t*>(base);
  p.done = reinterpret_cast<uint32_t*>(base + f.done);
  p.hidden = reinterpret_cast<uint32_t*>(base + f.hidden);
  p.arrived = reinterpret_cast<uint32_t*>(base + f.arrived);
  p.head = reinterpret_cast<int*>(base + f.head);
  p.entries = reinterpret_cast<FewEntry*>(base + f.entries);
  p.list = reinterpret_cast<uint16_t*>(base + f.list);
  p.of_chunk = reinterpret_cast<uint16_t*>(base + f.of_chunk);
  p.valid = base + f.valid;
  p.part_gu = reinterpret_cast<float*>(base + f.part_gu);
  p.part_sh_gu = reinterpret_cast<float*>(base + f.part_sh_gu);
  p.part_dn = reinterpret_cast<float*>(base + f.part_dn);
  p.part_sh_dn = reinterpret_cast<float*>(base + f.part_sh_dn);
  p.h = reinterpret_cast<uint16_t*>(base + f.h);
  p.sh_h = reinterpret_cast<uint16_t*>(base + f.sh_h);
  p.status = dev.status;
  p.wait_limit_ns = dev.wait_limit_ns;
  p.stall = dev.test_stall_producer;
  p.gu = f.gu; p.dn = f.dn; p.sh_gu = f.sh_gu; p.sh_dn = f.sh_dn;
  p.T = (int)s.T; p.H = (int)s.H; p.E = (int)s.E; p.k = (int)s.k; p.I = (int)s.I; p.I_s = (int)s.I_s;
  p.max_entries = (int)f.max_entries; p.max_chunks = (int)f.max_chunks; p.sh_chunks = (int)f.sh_chunks;
  p.zero_words = (int)f.zero_words;
  const size_t tables = few_tables_bytes(f.max_entries, f.max_chunks, f.slots);
  p.stages = (int)std::min<size_t>(kFewMaxStages, (kFewSmem - 1024 - kFewFixed - tables) / kFewStage);
  if (!few_map(&p.tm_gate_up, weights.gate_up, s.E * s.H, 2 * s.I, kFewK) || !few_map(&p.tm_down, weights.down, s.E * s.I, s.H, kFewK) ||
      !few_map(&p.tm_x, x, s.T, s.H, 1) || !few_map(&p.tm_h, p.h, f.slots, s.I, 1))
    return -1;
  if (s.I_s && (!few_map(&p.tm_sh_gate_up, weights.sh_gate_up, s.H, 2 * s.I_s, kFewK) ||
                !few_map(&p.tm_sh_down, weights.sh_down, s.I_s, s.H, kFewK) || !few_map(&p.tm_sh_h, p.sh_h, s.T, s.I_s, 1)))
    return -1;
  static std::atomic<int> configured[kMaxDevices] = {};
  if (!configured[dev.ordinal].load()) {
    if (cudaFuncSetAttribute(few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem) != cudaSuccess) return 1;
    configured[dev.ordinal].store(1);
  }
  const size_t prep_smem = (size_t)(f.slots + s.E) * sizeof(int);
  if (launch_pdl(few_prep_kernel, dim3(1), dim3(kPrepThreads), prep_smem, stream, 1, p) != cudaSuccess) return 1;
  const size_t smem = 1024 + (size_t)p.stages * kFewStage + kFewFixed + tables;
  return launch_pdl(few_kernel, dim3((unsigned)dev.num_sms), dim3(kFewThreads), smem, stream, 1, p) == cudaSuccess ? 0 : 1;
}

}  // namespace moe
