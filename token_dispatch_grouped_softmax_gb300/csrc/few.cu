// The expert layer for a few tokens in bf16, rows in slot order:
//
//   h[t, j] = silu(x_t . Wg_e) * (x_t . Wu_e),  e = ids[t, j]
//   y_t = sum_j w[t, j] (h[t, j] . Wd_e)  (+ the shared expert's, weight 1)
//
// With few rows an expert the weights' bytes are the cost: each weight of the
// experts in use has to come from HBM once (an expert of more than 32 rows loads
// it again for every 32, one after another, out of the L2).  One launch streams them all.  A
// unit of work is 128 columns of one expert's weight (64 gate and the 64 up
// columns beside them, or 128 of down) by the whole of its K rows or a part,
// for up to 32 rows of that expert; gate_up's units come before down's.  Blocks draw units
// by tickets in that order, so that a block that waits for an expert's h
// waits only for units that running blocks have drawn: no block has to be
// resident for another to go on.
//
//   warp 3        draws the units, one ahead of the loads.
//   warp 0        keeps a ring of 128 x 128 tiles of the weights full by TMA.
//                 It waits for nothing but free stages: while h is not ready,
//                 down's weights already arrive.
//   warp 1        gathers the rows' 128 values of K for each tile (TMA
//                 gather4), for down once the expert's h is complete.
//   warp 2        issues tcgen05.mma, the weights as A (M = 128 columns,
//                 MN-major as they lie) and the rows as B (N = 32): the
//                 accumulator has a column of the weight in each TMEM lane.
//   warps 4..19   four groups take the units in turn, from TMEM.  gate_up over
//                 the whole of K becomes h at once; other sums go to the
//                 workspace in fp32, and whoever adds the last part of a tile
//                 sums the parts in order and writes h, or of a token's
//                 columns y.
//
// The parts of K depend on the shape alone, so a token's sums have one order
// and its result does not depend on the batch.
//
// Measured (device time, weights from HBM): 16 tokens of H 2048, top-8 of 128,
// I 768 126 us for 777 MB (82 experts in use), 6.2 TB/s (the copy rate is 6.7); 64
// tokens 192, 128 tokens 222, both for 1.2 GB; one
// token 27 us for 75 MB: there the dependent steps count (the lists 1 us, the
// first tile 3, h to down 4, down's rows and the sum 6), and 96 blocks read
// gate_up's 512 KB each in 10 us.  Beyond 32 slots a slot's place in the
// lists is counted over the slots before it, by every block and before the first
// load: a call with weights of next to nothing (H 64, I 64, E 128) takes 19 us with
// 128 slots, 29 with 512, 50 with 1024, 156 with 2048 and 373 with 4096 (128 tokens,
// top-32; with H 2048, I 768 713).  The tensor pipe is 5 to 9 % busy
// whether the weights are A or B: MMAs of 32 rows or of 16, four accumulators
// in turn instead of one, and weights as B with N = 128 all took the same time.
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
constexpr uint32_t kFewTmem = kFewAcc * kFewRows;   // columns
constexpr int kFewQueue = 16;                  // units between warp 3 and the epilogue
constexpr int kFewSmem = 232448 - 256;         // what a block may have (227 KB) but for its static variables

enum : uint32_t { kFewSiteIds = 1, kFewSiteTile = 2, kFewSiteRows = 3, kFewSiteMma = 4, kFewSiteEpi = 5, kFewSiteHidden = 6, kFewSiteUnits = 7 };

// One of an expert's two products: K rows in parts of part_k, N columns in tiles.
struct FewProduct {
  int K, parts, part_k, tiles;
  uint32_t units_magic, tiles_magic;   // of tiles * parts, and of tiles (div_by)
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
  uint32_t* hidden;     // [chunks, shared chunks][tiles] parts of a gate_up tile that are there, of a product in parts
  uint32_t* arrived;    // [tiles of down][T] slots' parts of a token's columns that are there
  float *part_gu, *part_sh_gu, *part_dn, *part_sh_dn;
  uint16_t *h, *sh_h;
  uint32_t* status;
  uint64_t wait_limit_ns;
  FewProduct gu, dn, sh_gu, sh_dn;
  int T, H, E, k, I, I_s;
  uint32_t k_magic;
  int max_entries, max_chunks, sh_chunks;
  int stages;
  int stall;
};

// --------------------------------------------------------------- the lists

// What every block makes of the ids for itself (a launch of its own would take
// longer): the slots grouped by expert, in an order that the ids fix, so that
// every block's are the same: experts in increasing order, or with up to 32
// slots as they first appear.
struct FewLists {
  FewEntry* entries;
  uint16_t* of_chunk;   // entry of a chunk
  uint16_t* list;       // slots by expert
  uint32_t* valid;      // which slots of a token name an expert
  float* w;             // [S]
  int* chunks;          // their number
};

// room: [S + E] ints that are free.
__device__ __forceinline__ void few_lists(const FewParams& p, const FewLists& out, int* room) {
  __shared__ int warp_sums[2][kFewThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, slots = p.T * p.k;
  if (slots <= 32) {   // one warp, a slot to a lane: no barriers
    if (warp > 0) return;
    int e = -1;
    if (lane < slots) {
      e = p.ids[lane];
      out.w[lane] = p.w[lane];
      if (e < 0 || e >= p.E) {
        if (e != -1) report_status(p.status, kStatusDevice, kKernFew, kFewSiteIds);
        e = -1;
      }
    }
    const uint32_t used = __ballot_sync(0xffffffffu, e >= 0), same = __match_any_sync(0xffffffffu, e), below = (1u << lane) - 1u;
    const bool leads = e >= 0 && (same & below) == 0;
    const uint32_t leaders = __ballot_sync(0xffffffffu, leads);
    int end = leads ? __popc(same) : 0;   // of the expert's rows in the list
    const int rows = end;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += x;
    }
    const int row0 = __shfl_sync(0xffffffffu, end - rows, __ffs(same) - 1), entry = __popc(leaders & below);
    if (leads) {
      out.entries[entry] = FewEntry{e, row0, rows, entry};   // at most 32 rows: one chunk
      out.of_chunk[entry] = (uint16_t)entry;
    }
    if (e >= 0) out.list[row0 + __popc(same & below)] = (uint16_t)lane;
    if (lane < p.T) out.valid[lane] = used >> lane * p.k & (0xFFFFFFFFu >> (32 - p.k));
    if (lane == 0) *out.chunks = __popc(leaders);
    return;
  }
  int *ids = room, *first = room + (slots + 3) / 4 * 4;
  for (int e = tid; e < p.E; e += kFewThreads) first[e] = 0;
  bool bad = false;
  for (int i = tid; i < slots; i += kFewThreads) {
    int e = p.ids[i];
    if (e < 0 || e >= p.E) {
      bad |= e != -1;
      e = -1;
    }
    ids[i] = e;
    out.w[i] = p.w[i];
  }
  if (bad) report_status(p.status, kStatusDevice, kKernFew, kFewSiteIds);
  __syncthreads();
  for (int i = tid; i < slots; i += kFewThreads)
    if (ids[i] >= 0) atomicAdd(&first[ids[i]], 1);
  if (tid < p.T) {
    uint32_t n = 0;
    for (int j = 0; j < p.k; ++j) n |= (uint32_t)(ids[tid * p.k + j] >= 0) << j;
    out.valid[tid] = n;
  }
  __syncthreads();
  // rows, chunks and entries before each expert, two experts a thread
  static_assert(2 * kFewThreads >= kMaxExperts, "every expert has a thread");
  int rows[2], chunks[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    rows[i] = 2 * tid + i < p.E ? first[2 * tid + i] : 0;
    chunks[i] = (rows[i] + kFewRows - 1) / kFewRows;
  }
  int a = rows[0] + rows[1], b = (chunks[0] + chunks[1]) << 16 | ((rows[0] > 0) + (rows[1] > 0));   // inclusive sums
  const int a0 = a, b0 = b;
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
#pragma unroll
  for (int i = 0; i < kFewThreads / 32; ++i) {
    const int n = warp_sums[1][i];
    if (i < warp) {
      a += warp_sums[0][i];
      b += n;
    }
    all += n;
  }
  int row0 = a - a0, chunk0 = (b - b0) >> 16, entry = (b - b0) & 0xFFFF;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = 2 * tid + i;
    if (e < p.E) first[e] = row0;
    if (rows[i] > 0) {
      out.entries[entry] = FewEntry{e, row0, rows[i], chunk0};
      for (int c = 0; c < chunks[i]; ++c) out.of_chunk[chunk0 + c] = (uint16_t)entry;
      ++entry;
    }
    row0 += rows[i];
    chunk0 += chunks[i];
  }
  __syncthreads();
#pragma unroll 1
  for (int i = tid; i < slots; i += kFewThreads) {
    const int e = ids[i];
    if (e < 0) continue;
    int at = first[e], j = 0;   // and the expert's slots before this one
#pragma unroll 1
    for (; j + 4 <= i; j += 4) {
      const int4 o = *reinterpret_cast<const int4*>(ids + j);
      at += (o.x == e) + (o.y == e) + (o.z == e) + (o.w == e);
    }
    for (; j < i; ++j) at += ids[j] == e;
    out.list[at] = (uint16_t)i;
  }
  if (tid == 0) *out.chunks = all >> 16;
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
    entry = of_chunk[div_by(u, per, f.units_magic)];
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
  const uint32_t at = n_chunks == 1 ? local : local / n_chunks;
  const int c = (int)(local - at * n_chunks);
  x.entry = x.shared ? p.max_entries : entry;
  x.chunk = (x.shared ? p.max_chunks : chunk0) + c;
  x.row0 = row0 + c * kFewRows;
  x.rows = min(kFewRows, rows - c * kFewRows);
  x.part = (int)div_by(at, f.tiles, f.tiles_magic);
  x.tile = (int)at - x.part * f.tiles;
  x.k0 = x.part * f.part_k;
  x.halves = min(f.part_k, f.K - x.k0) / 64;
  x.w_row = expert * f.K + x.k0;
  return x;
}

// A bounded wait whose first try is in line.  With few tokens a block runs
// most of its code once, so that fetching it counts: it is kept short.
struct FewWait {
  volatile int* abort;
  uint64_t limit_ns;
  uint32_t* status;
};
__device__ __noinline__ bool few_wait_more(uint32_t bar, uint32_t parity, const FewWait& w, uint32_t site) {
  return mbar_wait_bounded(bar, parity, w.abort, w.limit_ns, w.status, site, kKernFew);
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

constexpr size_t few_tables_bytes(int64_t entries, int64_t chunks, int64_t slots, int64_t T) {
  return (size_t)(entries * sizeof(FewEntry) + (T + slots) * 4 + (chunks + slots) * sizeof(uint16_t) + 15) & ~(size_t)15;
}
constexpr int kFewBars = 3 * kFewMaxStages + 2 * kFewAcc + 2 * kFewQueue + 2;
constexpr int kFewSwap = 8 * 128;              // floats of a group: eight rows of its unit
constexpr size_t kFewFixed = (kFewBars * 8 + kFewQueue * sizeof(FewUnit) + 64 + kFewGroups * kFewSwap * 4 + 15) & ~15;

__global__ void __launch_bounds__(kFewThreads, 1) few_kernel(const __grid_constant__ FewParams p) {
  extern __shared__ uint8_t few_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(few_smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + p.stages * kFewStage);
  FewUnit* queue = reinterpret_cast<FewUnit*>(bars + kFewBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(queue + kFewQueue);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* group_word = tmem_slot + 2;        // [groups]
  int* n_chunks = reinterpret_cast<int*>(tmem_slot + 2 + kFewGroups);
  float* swap = reinterpret_cast<float*>(tmem_slot + 16);
  FewEntry* entries = reinterpret_cast<FewEntry*>(smem + p.stages * kFewStage + kFewFixed);
  uint32_t* valid = reinterpret_cast<uint32_t*>(entries + p.max_entries);
  float* w = reinterpret_cast<float*>(valid + p.T);
  uint16_t* of_chunk = reinterpret_cast<uint16_t*>(w + p.T * p.k);
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
  const uint32_t issued_bar = bar0 + 8u * (kFewBars - 2);   // a unit's last loads are being issued
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
    mbar_init(issued_bar, 1);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.tm_gate_up);
    tma_prefetch_desc(&p.tm_down);
    tma_prefetch_desc(&p.tm_x);
    tma_prefetch_desc(&p.tm_h);
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(tmem_slot), kFewTmem);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  uint32_t next = 0;
  if (tid == 96) next = atomicAdd(p.ticket, 1u);   // warp 3's first, while the slots are sorted
  few_lists(p, FewLists{entries, of_chunk, list, valid, w, n_chunks}, reinterpret_cast<int*>(smem));
  fence_proxy_async_smem();   // the sort's writes into the ring, before TMA's
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  for (int t = blockIdx.x; t < p.T; t += gridDim.x)   // tokens without an expert
    if (valid[t] == 0 && p.I_s == 0)
      for (int c = tid * 8; c < p.H; c += kFewThreads * 8)
        *reinterpret_cast<uint4*>(p.y + (int64_t)t * p.H + c) = make_uint4(0, 0, 0, 0);
  const FewWait bounds{abort_flag, p.wait_limit_ns, p.status};
  auto wait = [&](uint32_t bar, uint32_t parity, uint32_t site) {
    return mbar_try_wait(bar, parity) || few_wait_more(bar, parity, bounds, site);
  };
  auto wait_warp = [&](uint32_t bar, uint32_t parity, uint32_t site) {   // every lane acquires the phase itself
    return __all_sync(0xffffffffu, wait(bar, parity, site));
  };
  // after an early stop: a stage's copies have landed (bounded)
  auto land = [&](uint32_t bar, uint32_t parity) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t0 < p.wait_limit_ns) {
    }
  };

  if (warp == 3) {
    if (lane == 0) {
      for (int i = 0, ends = 0; ends < kFewGroups; ++i) {
        const FewUnit x = few_unit(p, entries, of_chunk, *n_chunks, next);
        const int q = i % kFewQueue;
        if (!wait(seen_bar(q), (i / kFewQueue & 1) ^ 1u, kFewSiteUnits)) break;
        queue[q] = x;
        mbar_arrive(unit_bar(q));
        if (x.kind == kEnd) {   // one for each group
          ++ends;
          continue;
        }
        // the next only once this one's loads are out, so that the blocks draw
        // evenly; the ring's loads in flight cover the draw
        if (!wait(issued_bar, i & 1, kFewSiteUnits)) break;
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
        if (x.kind == kEnd) break;
        const CUtensorMap* map = x.kind == kGateUp ? (x.shared ? &p.tm_sh_gate_up : &p.tm_gate_up)
                                                   : (x.shared ? &p.tm_sh_down : &p.tm_down);
        const int c0 = x.kind == kGateUp ? 64 * x.tile : 128 * x.tile;
        const int c1 = x.kind == kGateUp ? (x.shared ? p.I_s : p.I) + c0 : c0 + 64;
        const bool both = x.kind == kGateUp || c1 < p.H;
        for (int s = 0; s < x.halves; s += 2) {
          ok = wait(free_bar(stage), phase ^ 1u, kFewSiteTile);
          if (!ok) break;
          if (s + 2 >= x.halves) mbar_arrive(issued_bar);
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
        row[r] = x.shared ? at : x.kind == kDown ? list[at] : (int)div_by(list[at], p.k, p.k_magic);
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
      auto row_of = [&](int r) { return x.shared ? x.row0 + r : (int)list[x.row0 + r]; };   // a slot, or the token
      uint16_t* h = (x.shared ? p.sh_h : p.h) + 64 * x.tile + (m & 63);
      // h is rounded as the grouped GEMMs round it: an operand of the tensor cores
      auto store_h = [&](int r, float g, float u) {
        h[(int64_t)row_of(r) * I] = __bfloat16_as_ushort(__float2bfloat16_rn(__fdividef(g, 1.0f + __expf(-g)) * u));
      };
      float* part = gate_up ? (x.shared ? p.part_sh_gu : p.part_gu) : (x.shared ? p.part_sh_dn : p.part_dn);
      const int width = gate_up ? 2 * I : p.H;
      const int c = gate_up ? (m < 64 ? 64 * x.tile + m : I + 64 * x.tile + m - 64) : 128 * x.tile + m;
      const bool whole = gate_up && f.parts == 1;
      float* rows = swap + group * kFewSwap;   // [8][128]
#pragma unroll
      for (int r0 = 0; r0 < kFewRows; r0 += 8) {
        if (r0 >= x.rows) break;
#pragma unroll
        for (int r = 0; r < 8; ++r) rows[128 * r + m] = v[r0 + r];
        const int n = min(8, x.rows - r0);
        if (whole) {   // gate in lanes 0..63, up in 64..127
          group_sync(group);
#pragma unroll 1
          for (int r = m >> 6; r < n; r += 2) store_h(r0 + r, rows[128 * r + (m & 63)], rows[128 * r + 64 + (m & 63)]);
          group_sync(group);
        } else if (c < width) {
#pragma unroll 1
          for (int r = 0; r < n; ++r) __stcg(part + ((int64_t)row_of(r0 + r) * f.parts + x.part) * width + c, rows[128 * r + m]);
        }
      }
      if (!whole) {
        group_sync(group);
        if (m < 32) {
          __threadfence();   // the group's stores, before the counts
          uint32_t answer = 0;
          if (gate_up) {
            if (m == 0) {
              const int64_t at = x.shared ? (int64_t)p.max_chunks * (p.gu.parts > 1 ? p.gu.tiles : 0) + (int64_t)(x.chunk - p.max_chunks) * f.tiles
                                          : (int64_t)x.chunk * f.tiles;
              answer = atomicAdd(p.hidden + at + x.tile, 1u) + 1 == (uint32_t)f.parts;
            }
          } else {           // the rows' tokens whose columns are complete
            bool last = false;
            if (m < x.rows) {
              const int t = x.shared ? x.row0 + m : (int)div_by(list[x.row0 + m], p.k, p.k_magic);
              const uint32_t all = (uint32_t)__popc(valid[t]) * p.dn.parts + (p.I_s ? p.sh_dn.parts : 0);
              last = atomicAdd(p.arrived + (int64_t)x.tile * p.T + t, 1u) + 1 == all;
            }
            answer = __ballot_sync(0xffffffffu, last);
          }
          // the counts, before the group's loads of the parts: by the lanes that
          // counted, so that the barrier carries it to the others
          __threadfence();
          if (m == 0) group_word[group] = answer;
        }
        group_sync(group);
        uint32_t mask = group_word[group];
        if (mask == 0) continue;
        if (gate_up) {
          for (int r = m >> 6; r < x.rows; r += 2) {
            const float* from = part + (int64_t)row_of(r) * f.parts * width + 64 * x.tile + (m & 63);
            float g = 0.f, u = 0.f;
#pragma unroll 4
            for (int j = 0; j < f.parts; ++j) {
              g += __ldcg(from + (int64_t)j * width);
              u += __ldcg(from + (int64_t)j * width + I);
            }
            store_h(r, g, u);
          }
        } else {
          if (c >= p.H) continue;
          for (; mask; mask &= mask - 1) {
            const int r = __ffs(mask) - 1;
            const int t = x.shared ? x.row0 + r : (int)div_by(list[x.row0 + r], p.k, p.k_magic);
            const uint32_t used = valid[t];
            float y = 0.f;
            if (p.dn.parts == 1) {
              const float* from = p.part_dn + (int64_t)t * p.k * p.H + c;
#pragma unroll 1
              for (int j0 = 0; j0 < p.k; j0 += 8) {   // eight slots' loads in flight
                float s[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) s[j] = used >> j0 >> j & 1u ? __ldcg(from + (int64_t)(j0 + j) * p.H) : 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  if (used >> j0 >> j & 1u) y = fmaf(w[t * p.k + j0 + j], s[j], y);
              }
            } else {
#pragma unroll 1
              for (int j = 0; j < p.k; ++j) {
                if (!(used >> j & 1u)) continue;
                const float* from = p.part_dn + (int64_t)(t * p.k + j) * p.dn.parts * p.H + c;
                float s = 0.f;
#pragma unroll 4
                for (int l = 0; l < p.dn.parts; ++l) s += __ldcg(from + (int64_t)l * p.H);
                y = fmaf(w[t * p.k + j], s, y);
              }
            }
            if (p.I_s) {
              const float* from = p.part_sh_dn + (int64_t)t * p.sh_dn.parts * p.H + c;
              float s = 0.f;
#pragma unroll 4
              for (int l = 0; l < p.sh_dn.parts; ++l) s += __ldcg(from + (int64_t)l * p.H);
              y += s;
            }
            p.y[(int64_t)t * p.H + c] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
          }
        }
        if (!gate_up) continue;
      }
      fence_proxy_async_all();   // h is read by TMA
      group_sync(group);
      if (m == 0) {
        __threadfence();
        atomicAdd(p.done + x.entry, 1u);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) tmem_dealloc(tmem, kFewTmem);
}

// A unit takes the whole of K where one token's slots make kFewUnits units of
// a product, so that a decoded token keeps most SMs busy: its sums stay in
// TMEM, and h needs no partial sums through memory.  With fewer units K is
// split: in at most 8 parts of at least 256 rows, whole stages.  K, the tiles
// and k alone decide, so that a token's sums do not depend on the batch.
// Measured with 48 and with 96: 7 tokens of H 1600, top-5 of 60, I 704 (55
// units of gate_up) 43 and 50 us; 4 tokens of H 4096, top-2 of 8, I 1024 (32)
// 42 and 44; one token of it 30.7 and 29.6.
constexpr int64_t kFewUnits = 48;
FewProduct few_product(int64_t K, int64_t tiles, int64_t slots) {
  FewProduct f = {};
  if (K == 0 || tiles == 0) return f;
  f.K = (int)K;
  f.tiles = (int)tiles;
  const int64_t stages = (K + kFewK - 1) / kFewK, wanted = (kFewUnits + tiles * slots - 1) / (tiles * slots);
  const int64_t parts = std::min({(int64_t)kFewParts, std::max<int64_t>(1, K / 256), wanted});
  f.part_k = (int)((stages + parts - 1) / parts * kFewK);
  f.parts = (int)((K + f.part_k - 1) / f.part_k);
  f.units_magic = 0xFFFFFFFFu / (uint32_t)(f.tiles * f.parts);
  f.tiles_magic = 0xFFFFFFFFu / (uint32_t)f.tiles;
  return f;
}

// Everything of a call but its pointers: the products, and where the
// workspace's pieces begin.
struct FewPlan {
  FewProduct gu, dn, sh_gu, sh_dn;
  int64_t slots, max_entries, max_chunks, sh_chunks, zero_words;
  size_t done, hidden, arrived, part_gu, part_sh_gu, part_dn, part_sh_dn, h, sh_h, bytes;
};

FewPlan few_plan(const FewShape& s) {
  FewPlan f;
  f.gu = few_product(s.H, s.I / 64, s.k);
  f.dn = few_product(s.I, (s.H + 127) / 128, s.k);
  f.sh_gu = few_product(s.H, s.I_s / 64, 1);
  f.sh_dn = few_product(s.I_s, (s.H + 127) / 128, 1);
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
  f.hidden = take((f.max_chunks * (f.gu.parts > 1 ? f.gu.tiles : 0) + f.sh_chunks * (f.sh_gu.parts > 1 ? f.sh_gu.tiles : 0)) * 4);
  f.arrived = take(f.dn.tiles * s.T * 4);
  f.zero_words = at / 4;
  at = (at + 255) & ~(size_t)255;
  f.part_gu = take(f.gu.parts > 1 ? (size_t)f.slots * f.gu.parts * 2 * s.I * 4 : 0);
  f.part_sh_gu = take(f.sh_gu.parts > 1 ? (size_t)s.T * f.sh_gu.parts * 2 * s.I_s * 4 : 0);
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
int64_t few_experts_counters(const FewShape& s) { return few_plan(s).zero_words; }

int launch_few_experts(const FewShape& s, const uint16_t* x, const int32_t* ids, const float* w, const FewWeights& weights,
                       uint16_t* y, void* ws, bool counters_clear, const DeviceInfo& dev, cudaStream_t stream) {
  const FewPlan f = few_plan(s);
  uint8_t* base = static_cast<uint8_t*>(ws);
  FewParams p;
  p.ids = ids; p.w = w; p.y = y;
  p.ticket = reinterpret_cast<uint32_t*>(base);
  p.done = reinterpret_cast<uint32_t*>(base + f.done);
  p.hidden = reinterpret_cast<uint32_t*>(base + f.hidden);
  p.arrived = reinterpret_cast<uint32_t*>(base + f.arrived);
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
  p.k_magic = 0xFFFFFFFFu / (uint32_t)s.k;
  p.max_entries = (int)f.max_entries; p.max_chunks = (int)f.max_chunks; p.sh_chunks = (int)f.sh_chunks;
  const size_t tables = few_tables_bytes(f.max_entries, f.max_chunks, f.slots, s.T);
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
  if (!counters_clear && cudaMemsetAsync(ws, 0, f.zero_words * 4, stream) != cudaSuccess) return 1;
  const size_t smem = 1024 + (size_t)p.stages * kFewStage + kFewFixed + tables;
  return launch_pdl(few_kernel, dim3((unsigned)dev.num_sms), dim3(kFewThreads), smem, stream, 1, p) == cudaSuccess ? 0 : 1;
}

}  // namespace moe
