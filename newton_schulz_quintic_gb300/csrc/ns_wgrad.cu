// ns_wgrad.cu -- weight gradients from an input held in 8 bits
// (include/ns.h): G[e] (+)= dY[e]^T X[e] over the rows of each group.
//
// A GEMM whose contraction runs over rows (tokens): both operands are
// MN-major as they lie in memory, and the tensor cores read them so. A value
// of X is q * 2^(E - 133) with |q| <= 127, exact in bf16, so the product runs
// at the bf16 rate with no rounding of X.
//
// X is widened to bf16 in scratch, once. Widening on the way to shared memory
// was built and measured: every tile of X is then widened again for each tile
// row of G (32 times at 8192 x 6144), which took 2400 warp instructions and
// 570 cycles of shared-memory traffic per 64 rows next to the 512 cycles of
// MMA, 767 us at 8192 x 8192 x 6144. There are two forms, to the same bits:
//   in the product's launch (ns_wgrad_kernel<true>, when TMA reads dY as it
//     lies): four more warps per CTA widen pieces of 64 x 256 in the order in
//     which the tiles need them and count them; a tile is handed out once its
//     part of X is counted. The launch is cooperative, since CTAs wait for one
//     another's pieces.
//   in a launch of its own before (ns_wgrad_prepare_kernel; the product sets
//     itself up meanwhile), which also makes dY's slices.
// The first form hides the widening behind the product, but the pieces that
// the first tiles wait for come at a lower rate than with all threads: 8192 rows,
// 8192 x 6144: 513 us against 522; 38912 rows in 76 groups, 2048 x 6144: 848 against
// 880; 4096 rows, 4096 x 4096: 96 against 104; 64 rows, 64 x 64: 12.8 against 16; but
// 16384 rows, 512 x 512, where the first tiles need all: 40 against 38. So it is
// taken when what the first tiles need, counted one and a half times, is no more
// than all pieces and one per CTA (the second launch).
//
// The product is one persistent kernel of CTA pairs (clusters of 2), one 256 x
// 256 tile of one group's G at a time (tcgen05.mma.cta_group::2, M = 256, N =
// 256, K = 16). CTA rank r holds rows (n_out) r*128.. and columns (n_in)
// r*128.. of the operands. Warps of a CTA:
//   0       TMA: 64 rows of its share of dY and X (two 64 x 64 boxes each,
//           128-byte swizzle) into a 6-stage ring
//   1       TMEM (two accumulators of 256 columns); in the leader the MMAs
//   2       passes a landed stage on to the MMAs. Where a group ends inside the
//           stage it first clears the rows beyond, in both operands, so that
//           nothing of the next group (infinities, NaN) takes part.
//   3       looks the pair's tiles up (place, group, rows) a few ahead and
//           hands them to the other warps through a small queue
//   4..7    (first form) X to bf16
//   last 8  sums: every kChunk k-blocks the accumulator is added to fp32
//           registers (128 columns x 1 row per thread) while the MMAs go on in
//           the other one; the tile is written at its end. The tensor cores'
//           own accumulation loses up to a unit in the last place per
//           instruction; 32 instructions between two drains keep that near
//           2^-21 of the sum for any number of rows.
// The tile leaves through TMA where G's rows are 16-byte aligned: overwritten,
// or (fp32) added in place, which is one rounding of old + sum; else
// element by element.
//
// fp32 dY is held as three bf16 slices (the h + m + l of ns_tc.cu) and the
// k-loop runs over the slices too, smallest first; X needs no slices. A bf16
// dY that TMA cannot address (pitch or base not on 16 bytes) is copied to a
// padded buffer the same way. When there are fewer tiles than CTA pairs the
// rows are split and the parts, fp32 in scratch, are added in order by a
// second kernel.
//
// One elected lane issues the copies and the MMAs (elect.sync, which tells the
// compiler that one lane runs there: with a test for lane 0 the MMAs of the same
// loop were issued 4 % slower at 8192 rows, 8192 x 6144, 7 % with the registers divided).
//
// Bound by the tensor pipe: 8192 rows, 8192 x 6144 bf16 in 500 to 525 us, 1.57 to
// 1.65 PFLOP/s at power-capped clocks; 4096 x 4096 x 4096 in 96 us. 76 experts of 512
// rows on average, 2048 x 6144: 848 us, of which G's stores take 150 (their
// staging shares the shared memory that the operands already fill).
// Every wait is bounded (mbar_wait): on a timeout the status word is set, the
// CTA waits for its own copies and MMAs, frees TMEM and exits.
#include <algorithm>

#include "../../include/ns.h"
#include "ns_rows.cuh"

namespace ns {

namespace {

constexpr int kBK = 64;                          // rows per k-block
constexpr int kStages = 6;
constexpr int kShare = 128 * kBK * 2;            // one operand's share of a stage: 16 KB
constexpr int kBoxBytes = 64 * kBK * 2;          // one TMA box
constexpr int kChunk = 8;                        // k-blocks between two drains of an accumulator
constexpr int kIssueWarps = 4, kWidenWarps = 4, kSumWarps = 8;
constexpr int threads_of(bool widen) { return 32 * (kIssueWarps + (widen ? kWidenWarps : 0) + kSumWarps); }
// Registers a thread: the block is launched with one number for all (168 or
// 128), which its warpgroups then divide again. The built kernel is checked for
// it before its first launch: a share beyond what the launch holds would never
// be granted. Without the division the sums spill: bf16 sums added to 4096 x 4096 in
// 143 us against 148.
template <bool kWiden>
struct Regs {
  static constexpr int kIssue = 56, kWidening = 80, kSum = 176;
  static constexpr int kTotal = 128 * (kIssue + (kWiden ? kWidening : 0) + 2 * kSum);
};
constexpr int kUnitRows = 64, kUnitCols = 256;   // piece of X that four warps widen at a time
constexpr int kBlockRows = 512;                  // rows of X that one counter stands for
constexpr int kTmemCols = 512;
constexpr int kPatch = 32 * 32 * 4;              // staging of a block of 32 rows x 128 bytes per sum warp

enum Store : int { kStoreTma, kStoreTmaAdd, kStorePlain };

struct WgradParams {
  CUtensorMap tm_dy;       // bf16 {n_out, rows, slices}, box {64, 64, 1}
  CUtensorMap tm_x;        // bf16 {n_in, rows}, box {64, 64}
  CUtensorMap tm_out;      // G, or the parts when splits > 1: {n_in, n_out, matrices}, box of 128 bytes x 32 rows
  const int32_t *offsets;  // nullptr: one group of all rows
  void *grad;              // groups x n_out x n_in
  float *parts;            // splits x groups x n_out x part_pitch when splits > 1
  int rows, n_out, n_in, groups;
  int part_pitch;
  int slices;              // bf16 slices of dY (1 or 3)
  int splits;              // parts of a group's rows
  int tn, tk, items;       // tiles along n_out and n_in; groups * tn * tk * splits
  int accumulate, gdtype, store;
  int *status;
  uint64_t wait_limit_ns;
  // X as the caller holds it, when the kernel widens it itself (units > 0)
  const int8_t *q;
  const uint8_t *s;
  __nv_bfloat16 *x;        // rows x pitch
  int pitch, scale_pitch;
  int units;               // pieces of X, the last bands' empty ones counted
  int band_units;          // pieces of kUnitRows rows in a band of rows
  int *widened;            // per kBlockRows rows and kUnitCols columns: pieces in place
  int *left;               // CTAs that have ended
};

// One tile of the pair's list as warp 3 hands it out.
struct alignas(16) WTile {
  int n0, k0;  // its first row and column in G
  int e, z;    // its group; its matrix in the output map
  int lo, hi;  // its rows of dY and X; lo < 0: no more tiles
  int pad[2];
  __device__ __forceinline__ int blocks() const { return (hi - lo + kBK - 1) / kBK; }
};
constexpr int kQueue = 4;

struct WgradBarriers {
  WTile queue[kQueue];
  uint64_t qfull[kQueue];    // a slot holds the next tile
  uint64_t qempty[kQueue];   // every consumer of this CTA has read it

  uint64_t full[kStages];    // this CTA's boxes of a stage landed
  uint64_t ready[kStages];   // leader: both CTAs' operands of a stage are in place
  uint64_t empty[kStages];   // each CTA: the MMAs are done with a stage
  uint64_t tfull[2];         // each CTA: an accumulator holds a chunk
  uint64_t tempty[2];        // leader: both CTAs have drained an accumulator
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};
constexpr int kBarBytes = (static_cast<int>(sizeof(WgradBarriers)) + 127) / 128 * 128;
constexpr int kSmem = 1024 + kStages * 2 * kShare + kSumWarps * kPatch + kBarBytes;
static_assert(kSmem <= 227 * 1024, "shared memory of the weight-gradient kernel");

// Tiles go in groups of 8 along n_out, column by column within a group, so the
// tiles in flight share a few panels of each operand.
__device__ __forceinline__ WTile look_up(const WgradParams &p, int item) {
  WTile t;
  const int per = p.tn * p.tk;
  const int split = item % p.splits, g = item / p.splits;
  t.e = g / per;
  t.z = split * p.groups + t.e;
  const int tile = g - t.e * per;
  const int band = tile / (8 * p.tk), first = band * 8;
  const int height = min(8, p.tn - first), in = tile - band * 8 * p.tk;
  t.n0 = (first + in % height) * 256;
  t.k0 = in / height * 256;
  t.lo = 0;
  t.hi = p.rows;
  if (p.offsets) {
    t.lo = min(max(__ldg(p.offsets + t.e), 0), p.rows);
    t.hi = min(max(__ldg(p.offsets + t.e + 1), t.lo), p.rows);
  }
  if (p.splits > 1) {  // whole k-blocks per part
    const int64_t nb = t.blocks();
    const int a = static_cast<int>(nb * split / p.splits), b = static_cast<int>(nb * (split + 1) / p.splits);
    t.hi = min(t.hi, t.lo + b * kBK);
    t.lo = min(t.lo + a * kBK, t.hi);
  }
  return t;
}

// A consumer's place in the queue. One lane takes a tile with take(); a warp
// with take_warp(). False: no more tiles, or a wait gave up.
struct TileReader {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void step() {
    if (++slot == kQueue) {
      slot = 0;
      parity ^= 1u;
    }
  }
  __device__ __forceinline__ bool take(WgradBarriers *bar, WTile &t, const Waiter &w) {
    if (!mbar_wait(&bar->qfull[slot], parity, w)) return false;
    t = bar->queue[slot];
    mbar_arrive(&bar->qempty[slot]);
    step();
    return t.lo >= 0;
  }
  __device__ __forceinline__ bool take_warp(WgradBarriers *bar, WTile &t, const Waiter &w) {
    if (!warp_mbar_wait<false>(&bar->qfull[slot], parity, w)) return false;
    __syncwarp();
    t = bar->queue[slot];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&bar->qempty[slot]);
    step();
    return t.lo >= 0;
  }
};

// 16 values of X in bf16, exactly. e: their block's exponent.
__device__ __forceinline__ Pack<kBF16, 16> widen16(const uint4 &w, int e) {
  const float unit = e == 255 ? __int_as_float(0x7fc00000) : __int_as_float((max(e, 7) - 6) << 23);
  const int8_t *q = reinterpret_cast<const int8_t *>(&w);
  Pack<kBF16, 16> v;
#pragma unroll
  for (int u = 0; u < 16; ++u) v.set(u, static_cast<float>(q[u]) * unit);
  return v;
}

// This CTA's pieces of X, in the order in which the tiles need them: bands of
// rows (all of them for one group, else about a group's), in a band column by
// column. thread: 0..127.
__device__ __forceinline__ void widen(const WgradParams &p, int thread) {
  constexpr int kAcross = kUnitCols / 16, kStep = kWidenWarps * 32 / kAcross, kLoads = kUnitRows / kStep;
  const size_t size = static_cast<size_t>(p.rows) * p.pitch * 2;
  const int per_band = p.band_units * p.tk;
  for (int u = blockIdx.x; u < p.units; u += gridDim.x) {
    const int band = u / per_band, in = u - band * per_band;
    const int col = in / p.band_units, piece = band * p.band_units + in - col * p.band_units;
    const int row0 = piece * kUnitRows, c = col * kUnitCols + thread % kAcross * 16, r0 = row0 + thread / kAcross;
    if (row0 >= p.rows) continue;
    if (c < p.pitch) {
      uint4 w[kLoads];
      int e[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = r0 + i * kStep;
        if (r < p.rows) {
          w[i] = __ldcs(reinterpret_cast<const uint4 *>(p.q + static_cast<int64_t>(r) * p.pitch + c));
          e[i] = p.s[static_cast<int64_t>(r) * p.scale_pitch + c / 32];
        }
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = r0 + i * kStep;
        if (r < p.rows) widen16(w[i], e[i]).store(p.x + static_cast<int64_t>(r) * p.pitch + c, p.x, size, p.status);
      }
    }
    fence_proxy_async_global();  // TMA reads it
    asm volatile("bar.sync 1, %0;" ::"n"(kWidenWarps * 32) : "memory");
    if (thread == 0) red_release_gpu_add(p.widened + row0 / kBlockRows * p.tk + col, 1);
  }
}

// Whether tile t's part of X is in place; the whole warp waits for it.
__device__ __forceinline__ bool wait_widened(const WgradParams &p, const WTile &t, const Waiter &w) {
  int ok = 1;
  if (t.lo < t.hi)
    for (int b = t.lo / kBlockRows + (threadIdx.x & 31); b <= (t.hi - 1) / kBlockRows; b += 32) {
      const int pieces = min(kBlockRows / kUnitRows, (p.rows - b * kBlockRows + kUnitRows - 1) / kUnitRows);
      ok = ok && wait_count(p.widened + b * p.tk + t.k0 / kUnitCols, pieces, w);
    }
  return __all_sync(0xffffffffu, ok);
}

// The k-blocks of a tile in order: chunks of kChunk blocks, in each the
// slices of dY from smallest to largest, in each slice the chunk's blocks.
template <typename F>
__device__ __forceinline__ bool for_blocks(const WTile &t, int slices, F &&f) {
  const int nb = t.blocks();
  for (int c = 0; c < nb; c += kChunk)
    for (int z = slices - 1; z >= 0; --z)
      for (int b = c; b < min(c + kChunk, nb); ++b)
        if (!f(b, z)) return false;
  return true;
}

// The sums of one thread (row row0 + lane, 128 columns from col0) by TMA: 32
// rows x 128 bytes at a time through the warp's staging block, in the swizzled
// layout of the map (16-byte pieces XOR the row modulo 8), which also spreads
// a quarter-warp's 16-byte stores over all banks.
template <bool kAdd, bool kHalf>
__device__ __forceinline__ void store_tma(const WgradParams &p, int z, int row0, int col0, const float (&acc)[128],
                                          uint8_t *patch) {
  constexpr int kCols = kHalf ? 64 : 32;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = 0; h < 128 / kCols; ++h) {
    if (col0 + h * kCols >= p.n_in) break;
    if (lane == 0) bulk_read_wait();
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      uint32_t v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (kHalf) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(acc[h * kCols + 8 * k + 2 * u], acc[h * kCols + 8 * k + 2 * u + 1]);
          v[u] = *reinterpret_cast<const uint32_t *>(&b);
        } else {
          v[u] = __float_as_uint(acc[h * kCols + 4 * k + u]);
        }
      }
      *reinterpret_cast<uint4 *>(patch + lane * 128 + ((k ^ (lane & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
    }
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) tma_store_3d<kAdd>(&p.tm_out, col0 + h * kCols, row0, z, patch);
  }
}

// n <= kRowsAhead rows of a staging block of 32 x 32 sums, one column per lane;
// what is added to is read for all of them first. Returns the next row's place.
constexpr int kRowsAhead = 8;
template <int GT, bool ADD>
__device__ __forceinline__ typename Elem<GT>::T *store_rows(const WgradParams &p, typename Elem<GT>::T *g,
                                                            const float *patch, int r0, int n, size_t size) {
  using G = typename Elem<GT>::T;
  const int lane = threadIdx.x & 31;
  G old[kRowsAhead];
  if (ADD) {
    const G *at = g;
#pragma unroll
    for (int r = 0; r < kRowsAhead; ++r, at += p.n_in)
      if (r < n) old[r] = *at;
  }
#pragma unroll
  for (int r = 0; r < kRowsAhead; ++r, g += p.n_in)
    if (r < n && in_bounds(g, sizeof(G), p.grad, size, p.status)) {
      const float v = patch[(r0 + r) * 32 + (lane ^ (r0 + r))];
      *g = Elem<GT>::from_f(ADD ? Elem<GT>::to_f(old[r]) + v : v);
    }
  return g;
}

// The same element by element (rows that TMA cannot address, bf16 sums that
// are added to what is there): a store instruction covers one row's 32
// consecutive columns. Two sum warps share a scheduler, so instructions count: with
// whole blocks of rows taken without a test a row, 3 x 5505 x 5671 bf16 take 93 us
// against 135, bf16 sums added to 4096 x 4096 117 against 134. Lines of 128 aligned bytes
// with a test per column write fewer sectors in part, but took 370 to 540 us.
template <int GT, bool ADD>
__device__ __forceinline__ void store_plain(const WgradParams &p, int e, int row0, int col0, const float (&acc)[128],
                                            float *patch) {
  using G = typename Elem<GT>::T;
  const int lane = threadIdx.x & 31;
  const size_t size = static_cast<size_t>(p.groups) * p.n_out * p.n_in * sizeof(G);
  const int rows = min(32, p.n_out - row0);
  G *to = static_cast<G *>(p.grad) + (static_cast<int64_t>(e) * p.n_out + row0) * p.n_in + col0 + lane;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    __syncwarp();
    // row lane, column c at word (c ^ lane): no bank conflict either way
#pragma unroll
    for (int c = 0; c < 32; ++c) patch[lane * 32 + (c ^ lane)] = acc[32 * k + c];
    __syncwarp();
    if (col0 + 32 * k + lane >= p.n_in) continue;
    G *g = to + 32 * k;
    if (rows == 32) {
#pragma unroll 1
      for (int r0 = 0; r0 < 32; r0 += kRowsAhead)
        g = store_rows<GT, ADD>(p, g, patch, r0, kRowsAhead, size);
    } else {
      for (int r0 = 0; r0 < rows; r0 += kRowsAhead)
        g = store_rows<GT, ADD>(p, g, patch, r0, min(kRowsAhead, rows - r0), size);
    }
  }
}

template <bool kWiden>
__global__ void __launch_bounds__(threads_of(kWiden), 1) ns_wgrad_kernel(const __grid_constant__ WgradParams p) {
  constexpr int kSum0 = kIssueWarps + (kWiden ? kWidenWarps : 0);
  extern __shared__ uint8_t smem_raw[];
  // 1024-byte aligned, by an offset so that accesses stay in the shared window
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *sA = smem, *sB = smem + kStages * kShare, *patches = sB + kStages * kShare;
  WgradBarriers *bar = reinterpret_cast<WgradBarriers *>(patches + kSumWarps * kPatch);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x / 2, npairs = gridDim.x / 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bar->full[s], 1);
      mbar_init(&bar->ready[s], 2);
      mbar_init(&bar->empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&bar->tfull[a], 1);
      mbar_init(&bar->tempty[a], 2 * kSumWarps);
    }
    for (int q = 0; q < kQueue; ++q) {
      mbar_init(&bar->qfull[q], 1);
      mbar_init(&bar->qempty[q], 2 + kSumWarps + (leader ? 1 : 0));
    }
    mbar_init(&bar->drain, 1);
    bar->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&bar->tmem_base, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = bar->tmem_base;
  // the launch before this one prepares the operands; what is above ran beside it
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const bool tmem_ok = ld_shared_cluster_u32(mapa_shared(smem_u32(&bar->tmem_base), rank ^ 1u)) == tmem;
  if (!tmem_ok && threadIdx.x == 0) set_status(p.status, kStatusTmemMismatch);
  volatile int *abort = &bar->abort;
  const Waiter w{abort, p.status, p.wait_limit_ns};

  if (warp < kIssueWarps)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<kWiden>::kIssue));
  if (tmem_ok && warp == 0) {
    // ---------------------------------------------------- operands by TMA, issued by one lane
    if (elect_one()) {
      int stage = 0;
      uint32_t parity = 0;
      uint32_t issued = 0, last = 0;  // per stage: whether copies were issued, the parity of the last
      const int x = static_cast<int>(rank) * 128;
      TileReader tiles;
      WTile t;
      while (tiles.take(bar, t, w)) {
        const bool ok = for_blocks(t, p.slices, [&](int block, int z) {
          if (!mbar_wait<true>(&bar->empty[stage], parity ^ 1u, w)) return false;
          mbar_arrive_expect_tx(&bar->full[stage], 2 * kShare);
          if (kWiden && block == 0) fence_proxy_async_global();  // X was written by this launch's threads
          const int y = t.lo + block * kBK;
          uint8_t *a = sA + stage * kShare, *b = sB + stage * kShare;
          tma_load_3d(a, &p.tm_dy, t.n0 + x, y, z, &bar->full[stage]);
          tma_load_3d(a + kBoxBytes, &p.tm_dy, t.n0 + x + 64, y, z, &bar->full[stage]);
          tma_load_2d(b, &p.tm_x, t.k0 + x, y, &bar->full[stage]);
          tma_load_2d(b + kBoxBytes, &p.tm_x, t.k0 + x + 64, y, &bar->full[stage]);
          issued |= 1u << stage;
          last = (last & ~(1u << stage)) | (parity << stage);
          if (++stage == kStages) {
            stage = 0;
            parity ^= 1u;
          }
          return true;
        });
        if (!ok) break;
      }
      if (*abort)
        for (int s = 0; s < kStages; ++s)
          if ((issued >> s) & 1u) drain_wait(&bar->full[s], (last >> s) & 1u, w.limit_ns);
    }
  } else if (tmem_ok && warp == 1 && leader) {
    // ---------------------------------------------------- MMAs, issued by one lane
    if (elect_one()) {
      constexpr uint32_t idesc = umma_idesc_bf16(256, 256, 1, 1);
      const uint64_t desc_a = sw128_mnmajor_desc(smem_u32(sA)), desc_b = sw128_mnmajor_desc(smem_u32(sB));
      int stage = 0, acc = 0;
      uint32_t parity = 0, acc_parity = 0;
      bool ok = true, seen = false;  // seen: the next stage is known to be ready
      TileReader tiles;
      WTile t;
      while (ok && tiles.take(bar, t, w)) {
        const int nb = t.blocks();
        for (int c = 0; ok && c < nb; c += kChunk) {
          if (!(ok = mbar_wait<true>(&bar->tempty[acc], acc_parity ^ 1u, w))) break;
          const uint32_t d = tmem + static_cast<uint32_t>(acc * 256);
          const int n = min(kChunk, nb - c) * p.slices;
          for (int i = 0; i < n; ++i) {
            if (!seen && !(ok = mbar_wait<true>(&bar->ready[stage], parity, w))) break;
            tc_fence_after();
            const uint64_t at = static_cast<uint64_t>(stage * (kShare >> 4));  // addresses are in 16-byte units
            uint64_t *const empty = &bar->empty[stage];
            if (++stage == kStages) {
              stage = 0;
              parity ^= 1u;
            }
            umma_bf16_pair(d, desc_a + at, desc_b + at, idesc, i > 0);
            umma_bf16_pair(d, desc_a + at + 128u, desc_b + at + 128u, idesc, 1);
            // look at the next stage while these run, so that its first MMA follows the last one here at once
            seen = mbar_try_wait_cluster(&bar->ready[stage], parity);
            umma_bf16_pair(d, desc_a + at + 256u, desc_b + at + 256u, idesc, 1);
            umma_bf16_pair(d, desc_a + at + 384u, desc_b + at + 384u, idesc, 1);
            umma_commit_pair_multicast(empty, 3u);
          }
          if (!ok) break;
          umma_commit_pair_multicast(&bar->tfull[acc], 3u);
          if (++acc == 2) {
            acc = 0;
            acc_parity ^= 1u;
          }
        }
      }
      umma_commit_pair_multicast(&bar->drain, 1u);
      drain_wait(&bar->drain, 0, w.limit_ns);
    }
  } else if (tmem_ok && warp == 2) {
    // ---------------------------------------------------- landed stages
    int stage = 0;
    uint32_t parity = 0;
    TileReader tiles;
    WTile t;
    while (tiles.take_warp(bar, t, w)) {
      const bool ok = for_blocks(t, p.slices, [&](int block, int) {
        if (!warp_mbar_wait<true>(&bar->full[stage], parity, w)) return false;
        const int left = t.hi - t.lo - block * kBK;
        if (left < kBK) {  // rows left.. of both boxes of both operands, 8 pieces of 16 bytes each
          uint8_t *a = sA + stage * kShare, *b = sB + stage * kShare;
          for (int i = left * 8 + lane; i < kBK * 8; i += 32) {
            const uint4 zero = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4 *>(a + i * 16) = zero;
            *reinterpret_cast<uint4 *>(a + kBoxBytes + i * 16) = zero;
            *reinterpret_cast<uint4 *>(b + i * 16) = zero;
            *reinterpret_cast<uint4 *>(b + kBoxBytes + i * 16) = zero;
          }
          fence_proxy_async_shared();
          __syncwarp();
        }
        if (lane == 0) arrive_pair_shared(mapa_shared(smem_u32(&bar->ready[stage]), 0));
        if (++stage == kStages) {
          stage = 0;
          parity ^= 1u;
        }
        return true;
      });
      if (!ok) break;
    }
  } else if (tmem_ok && warp == 3) {
    // ---------------------------------------------------- the pair's tiles, looked up ahead
    int slot = 0;
    uint32_t parity = 0;
    bool more = true;
    for (int item = pair; more; item += npairs) {
      WTile t;
      more = item < p.items;
      if (more)
        t = look_up(p, item);
      else
        t.lo = -1;
      if (kWiden && more && !wait_widened(p, t, w)) break;
      __syncwarp();  // orders the other lanes' looks at the counters before lane 0's arrival
      if (!warp_mbar_wait<false>(&bar->qempty[slot], parity ^ 1u, w)) break;
      if (lane == 0) {
        bar->queue[slot] = t;
        mbar_arrive(&bar->qfull[slot]);
      }
      if (++slot == kQueue) {
        slot = 0;
        parity ^= 1u;
      }
    }
  } else if (kWiden && warp >= kIssueWarps && warp < kSum0) {
    // ---------------------------------------------------- X to bf16
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<kWiden>::kWidening));
    widen(p, threadIdx.x - kIssueWarps * 32);
  } else if (tmem_ok && warp >= kSum0) {
    // ---------------------------------------------------- sums and the tile's store
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Regs<kWiden>::kSum));
    const int e = warp - kSum0, quarter = warp & 3, half = e >> 2;
    uint8_t *patch = patches + e * kPatch;
    int acc = 0;
    uint32_t acc_parity = 0;
    bool ok = true;
    TileReader tiles;
    WTile t;
    while (ok && tiles.take_warp(bar, t, w)) {
      const int nb = t.blocks();
      if (nb == 0 && p.accumulate && p.splits == 1) continue;
      float sum[128];
#pragma unroll
      for (int c = 0; c < 128; ++c) sum[c] = 0.f;
      for (int c = 0; c < nb; c += kChunk) {
        if (!warp_mbar_wait<true>(&bar->tfull[acc], acc_parity, w)) {
          ok = false;
          break;
        }
        __syncwarp();
        tc_fence_after();
        const uint32_t src = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * 256 + half * 128);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t v[16];
          tmem_ld16(src + 16 * k, v);
#pragma unroll
          for (int u = 0; u < 16; ++u) sum[16 * k + u] += __uint_as_float(v[u]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_pair(mapa_shared(smem_u32(&bar->tempty[acc]), 0));
        if (++acc == 2) {
          acc = 0;
          acc_parity ^= 1u;
        }
      }
      if (!ok) break;
      const int row0 = t.n0 + static_cast<int>(rank) * 128 + quarter * 32, col0 = t.k0 + half * 128;
      if (row0 >= p.n_out) continue;
      if (p.store == kStorePlain) {
        float *words = reinterpret_cast<float *>(patch);
        if (p.gdtype == kF32) {
          if (p.accumulate)
            store_plain<kF32, true>(p, t.e, row0, col0, sum, words);
          else
            store_plain<kF32, false>(p, t.e, row0, col0, sum, words);
        } else if (p.accumulate) {
          store_plain<kBF16, true>(p, t.e, row0, col0, sum, words);
        } else {
          store_plain<kBF16, false>(p, t.e, row0, col0, sum, words);
        }
      } else if (p.splits > 1 || (p.gdtype == kF32 && p.store == kStoreTma))
        store_tma<false, false>(p, t.z, row0, col0, sum, patch);
      else if (p.store == kStoreTmaAdd)
        store_tma<true, false>(p, t.z, row0, col0, sum, patch);
      else
        store_tma<false, true>(p, t.z, row0, col0, sum, patch);
    }
    if (lane == 0) bulk_wait();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, kTmemCols);
  if (kWiden && warp == 2) {  // the last CTA leaves the counters at 0 for the next call
    int n = 0;
    if (lane == 0) {
      __threadfence();  // this CTA's counting is done before it counts itself
      n = atomicAdd(p.left, 1);
      __threadfence();
    }
    if (__shfl_sync(0xffffffffu, n, 0) == static_cast<int>(gridDim.x) - 1) {
      const int counters = (p.rows + kBlockRows - 1) / kBlockRows * p.tk;
      for (int i = lane; i < counters; i += 32) p.widened[i] = 0;
      if (lane == 0) *p.left = 0;
    }
  }
}

// ------------------------------------------------------------------ around the product
struct PrepareParams {
  const int8_t *q;
  const uint8_t *s;
  __nv_bfloat16 *x;    // rows x pitch
  const void *dy;      // nullptr: the product reads dY itself
  __nv_bfloat16 *out;  // slices x rows x out_pitch
  int64_t ld;
  int rows, n_in, pitch, scale_pitch, n_out, out_pitch, slices;
  int *status;
};

// fp32 (or bf16 that TMA cannot address) as bf16 slices: the first is the
// value rounded, each further one what the ones before leave out.
__device__ __forceinline__ float next_slice(float &left) {
  __nv_bfloat16 b = __float2bfloat16_rn(left);
  if (__hisinf(b) && !isinf(left))  // beyond bf16's largest value: that one, the rest in the next slice
    b = __ushort_as_bfloat16(static_cast<uint16_t>(__float_as_uint(left) >> 16));
  const float f = __bfloat162float(b);
  left = isinf(f) || isnan(f) ? 0.f : left - f;  // an infinity or NaN stays in the first slice alone
  return f;
}

// X widened to bf16 (16 values per thread: its pitch is a multiple of 16),
// and dY as TMA can address it: bf16 rows of out_pitch elements (a multiple of
// 8), one slice, or three whose sum is the fp32 value to 2^-24 of it. A thread
// takes 8 values of dY: consecutive ones where its rows allow 16-byte
// accesses, else four pairs 64 apart, so that a warp's accesses stay coalesced.
template <int DT, bool WIDE>
__global__ void __launch_bounds__(256) ns_wgrad_prepare_kernel(const __grid_constant__ PrepareParams p) {
  using E = typename Elem<DT>::T;
  asm volatile("griddepcontrol.launch_dependents;");  // the product may set itself up meanwhile
  const int64_t per_row = p.pitch / 16, nx = p.rows * per_row;
  const int64_t dy_row = WIDE ? p.out_pitch / 8 : (p.out_pitch + 255) / 256 * 32, ny = p.dy ? p.rows * dy_row : 0;
  const int64_t slice = static_cast<int64_t>(p.rows) * p.out_pitch;
  const size_t xsize = static_cast<size_t>(p.rows) * p.pitch * 2, ysize = static_cast<size_t>(slice) * p.slices * 2;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < nx + ny; i += static_cast<int64_t>(gridDim.x) * 256) {
    if (i < nx) {
      const int64_t r = i / per_row;
      const int c = static_cast<int>(i - r * per_row) * 16;
      const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(p.q + r * p.pitch + c));
      widen16(w, p.s[r * p.scale_pitch + c / 32]).store(p.x + r * p.pitch + c, p.x, xsize, p.status);
      continue;
    }
    const int64_t k = i - nx, r = k / dy_row;
    const int j = static_cast<int>(k - r * dy_row);
    const E *row = static_cast<const E *>(p.dy) + r * p.ld;
    __nv_bfloat16 *out = p.out + r * p.out_pitch;
    float v[8];
    if constexpr (WIDE) {
      Pack<DT, 8> x;
      x.load_stream(row + j * 8);
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = x.get(u);
      for (int z = 0; z < p.slices; ++z) {
        Pack<kBF16, 8> h;
#pragma unroll
        for (int u = 0; u < 8; ++u) h.set(u, next_slice(v[u]));
        h.store(out + z * slice + j * 8, p.out, ysize, p.status);
      }
    } else {
      const int c0 = (j / 32) * 256 + (j % 32) * 2;  // pairs at c0, c0 + 64, ...
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int c = c0 + (u / 2) * 64 + u % 2;
        v[u] = c < p.n_out ? Elem<DT>::to_f(row[c]) : 0.f;
      }
      for (int z = 0; z < p.slices; ++z) {
#pragma unroll
        for (int u = 0; u < 8; u += 2) {
          const int c = c0 + u * 32;
          Pack<kBF16, 2> h;
          h.set(0, next_slice(v[u]));
          h.set(1, next_slice(v[u + 1]));
          if (c < p.out_pitch) h.store(out + z * slice + c, p.out, ysize, p.status);
        }
      }
    }
  }
}

// G (+)= the parts of a split contraction, added in order.
template <int GT>
__global__ void __launch_bounds__(256) ns_wgrad_join_kernel(const __grid_constant__ WgradParams p) {
  using G = typename Elem<GT>::T;
  const int64_t mats = static_cast<int64_t>(p.groups) * p.n_out, n = mats * p.n_in, part = mats * p.part_pitch;
  G *g = static_cast<G *>(p.grad);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t r = i / p.n_in, at = r * p.part_pitch + (i - r * p.n_in);
    float v = p.parts[at];
    for (int s = 1; s < p.splits; ++s) v += p.parts[s * part + at];
    if (p.accumulate) v += Elem<GT>::to_f(g[i]);
    if (in_bounds(g + i, sizeof(G), g, static_cast<size_t>(n) * sizeof(G), p.status)) g[i] = Elem<GT>::from_f(v);
  }
}

int run_prepare(const PrepareParams &p, int dtype, int sms, cudaStream_t s) {
  const bool wide = p.dy && p.n_out % 8 == 0 && rows_aligned(p.dy, p.ld, dtype == NS_BF16 ? 2 : 4, 8);
  const int64_t dy_row = wide ? p.out_pitch / 8 : (p.out_pitch + 255) / 256 * 32;
  const int64_t n = static_cast<int64_t>(p.rows) * (p.pitch / 16 + (p.dy ? dy_row : 0));
  const int grid = static_cast<int>(std::min<int64_t>((n + 255) / 256, static_cast<int64_t>(sms) * 16));
  if (dtype == NS_BF16)  // a bf16 dY with aligned rows is read as it is
    ns_wgrad_prepare_kernel<kBF16, false><<<grid, 256, 0, s>>>(p);
  else if (wide)
    ns_wgrad_prepare_kernel<kF32, true><<<grid, 256, 0, s>>>(p);
  else
    ns_wgrad_prepare_kernel<kF32, false><<<grid, 256, 0, s>>>(p);
  count_launch();
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

// CTA pairs that can be resident at once on this device (one CTA per SM).
template <bool kWiden>
int resident_pairs(int dev, int sms, cudaLaunchConfig_t &cfg) {
  static int cached[64] = {};
  int &n = cached[dev & 63];
  if (n == 0) {
    static SmemOptIn opt_in;
    if (opt_in.ensure(reinterpret_cast<const void *>(ns_wgrad_kernel<kWiden>), kSmem)) return 0;
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, ns_wgrad_kernel<kWiden>) != cudaSuccess ||
        attr.numRegs * threads_of(kWiden) < Regs<kWiden>::kTotal) {
      cudaGetLastError();
      return 0;
    }
    cfg.gridDim = dim3(sms / 2 * 2, 1, 1);
    cfg.blockDim = dim3(threads_of(kWiden), 1, 1);
    if (cudaOccupancyMaxActiveClusters(&n, ns_wgrad_kernel<kWiden>, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = 0;
    }
  }
  return n;
}

// Pieces of X that the first `pairs` tiles of the list need.
int64_t first_wave_pieces(const WgradParams &p, int pairs) {
  const int64_t wave = std::min(pairs, p.items), per_group = static_cast<int64_t>(p.tn) * p.tk * p.splits;
  if (wave > per_group) return (wave + per_group - 1) / per_group * p.band_units * p.tk;
  const int64_t column = static_cast<int64_t>(std::min(p.tn, 8)) * p.splits;  // tiles of one column of a band
  return std::min<int64_t>(p.tk, (wave + column - 1) / column) * p.band_units;
}

int run_join(const WgradParams &p, int sms, cudaStream_t s) {
  const int64_t n = static_cast<int64_t>(p.groups) * p.n_out * p.n_in;
  const int grid = static_cast<int>(std::min<int64_t>((n + 255) / 256, static_cast<int64_t>(sms) * 16));
  if (p.gdtype == kBF16)
    ns_wgrad_join_kernel<kBF16><<<grid, 256, 0, s>>>(p);
  else
    ns_wgrad_join_kernel<kF32><<<grid, 256, 0, s>>>(p);
  count_launch();
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace
}  // namespace ns

using namespace ns;

extern "C" int ns_ckpt_wgrad(const void *dy, int64_t ld_dy, int64_t rows, int64_t n_out, const void *q,
                             const void *scales, int64_t n_in, const int32_t *offsets, int groups, void *grad,
                             int dtype, int grad_dtype, int accumulate, void *stream) {
  if ((dtype != NS_F32 && dtype != NS_BF16) || (grad_dtype != NS_F32 && grad_dtype != NS_BF16) ||
      (accumulate != 0 && accumulate != 1) || groups < 0)
    return NS_EINVAL;
  if (bad_shape(rows, n_out, ld_dy) || bad_shape(n_out, n_in, n_in) || n_out > (1 << 30) || n_in > (1 << 30) ||
      rows > (1 << 30))
    return NS_EINVAL;
  if (!offsets && groups != 1) return NS_EINVAL;
  if (groups > 0 && n_out * n_in > (int64_t(1) << 42) / groups) return NS_EINVAL;
  if (groups == 0 || n_out == 0 || n_in == 0 || (rows == 0 && accumulate)) return NS_OK;
  if (!grad || (rows > 0 && (!dy || !q || !scales))) return NS_EINVAL;
  const int elt = dtype == NS_BF16 ? 2 : 4, gelt = grad_dtype == NS_BF16 ? 2 : 4;
  if (misaligned(dy, elt) || misaligned(grad, gelt) || misaligned(q, 16) || misaligned(scales, 16) ||
      misaligned(offsets, 4))
    return NS_EALIGN;
  WgradParams p{};
  const int64_t q_pitch = ns_ckpt_pitch(n_in);
  const int64_t scale_pitch = ns_ckpt_scale_pitch(n_in);
  const Range rg(grad, static_cast<int64_t>(groups) * n_out, n_in, n_in, gelt);
  if (rg.overlaps(Range(dy, rows, n_out, ld_dy, elt)) || rg.overlaps(Range(q, rows, q_pitch, q_pitch, 1)) ||
      rg.overlaps(Range(scales, rows, scale_pitch, scale_pitch, 1)) ||
      rg.overlaps(Range(offsets, 1, groups + int64_t(1), groups + int64_t(1), 4)))
    return NS_EINVAL;
  OpCall call(stream);
  if (call.rc) return call.rc;
  WgradParams &k = p;
  k.offsets = offsets;
  k.grad = grad;
  k.rows = static_cast<int>(rows);
  k.n_out = static_cast<int>(n_out);
  k.n_in = static_cast<int>(n_in);
  k.groups = groups;
  k.slices = dtype == NS_F32 ? 3 : 1;
  k.tn = static_cast<int>((n_out + 255) / 256);
  k.tk = static_cast<int>((n_in + 255) / 256);
  k.accumulate = accumulate;
  k.gdtype = grad_dtype;
  k.status = call.status;
  k.wait_limit_ns = kWaitLimitNs;

  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  // it starts while the preparation still runs and waits for it (griddepcontrol)
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = call.s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int pairs = std::min(resident_pairs<false>(call.dev, call.sms, cfg), resident_pairs<true>(call.dev, call.sms, cfg));
  if (pairs <= 0) return NS_ECUDA;
  const int64_t tiles = static_cast<int64_t>(groups) * k.tn * k.tk;
  // Fewer tiles than half the pairs: parts of the rows, of one drain interval
  // (kChunk k-blocks) or more, until every pair has one.
  k.splits = 1;
  if (tiles * 2 <= pairs) {
    const int64_t depth = (rows / groups + kChunk * kBK - 1) / (kChunk * kBK);
    k.splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(pairs / tiles, depth)));
  }
  if (tiles * k.splits > INT32_MAX) return NS_EINVAL;
  k.items = static_cast<int>(tiles * k.splits);
  k.part_pitch = static_cast<int>((n_in + 3) / 4 * 4);
  // TMA writes what it can address; it adds in fp32 only (bf16 would round the
  // sum before adding it). Debug builds store where every store is checked.
  const bool out_rows = !misaligned(grad, 16) && n_in * gelt % 16 == 0;
  k.store = k.splits > 1                         ? kStoreTma
            : kDebugBounds || !out_rows          ? kStorePlain
            : !accumulate                        ? kStoreTma
            : grad_dtype == NS_F32               ? kStoreTmaAdd
                                                 : kStorePlain;

  // scratch: X in bf16, dY's slices (fp32, or bf16 that TMA cannot address), the parts of a split
  const bool direct = dtype == NS_BF16 && !misaligned(dy, 16) && ld_dy % 8 == 0;
  const int64_t pitch = (n_out + 7) / 8 * 8;
  auto up = [](size_t v) { return (v + 1023) / 1024 * 1024; };
  const size_t x_bytes = up(static_cast<size_t>(rows) * q_pitch * 2);
  const size_t dy_bytes = direct ? 0 : up(static_cast<size_t>(k.slices) * rows * pitch * 2);
  const size_t part_bytes = k.splits > 1 ? static_cast<size_t>(k.splits) * groups * n_out * k.part_pitch * 4 : 0;
  uint8_t *ws = nullptr;
  int rc = call.workspace(kSlotWgrad, x_bytes + dy_bytes + part_bytes, &ws);
  if (rc) return rc;
  k.parts = reinterpret_cast<float *>(ws + x_bytes + dy_bytes);
  if (rows > 0) {
    const int64_t use = direct ? ld_dy : pitch;
    const int64_t dims[3] = {n_out, rows, k.slices}, strides[2] = {use * 2, use * 2 * rows};
    const int box[3] = {64, kBK, 1};
    if ((rc = call.tensor_map(&k.tm_dy, 2, direct ? dy : ws + x_bytes, 3, dims, strides, box))) return rc;
    const int64_t xdims[2] = {n_in, rows}, xstride[1] = {q_pitch * 2};
    if ((rc = call.tensor_map(&k.tm_x, 2, ws, 2, xdims, xstride, box))) return rc;
    k.q = static_cast<const int8_t *>(q);
    k.s = static_cast<const uint8_t *>(scales);
    k.x = reinterpret_cast<__nv_bfloat16 *>(ws);
    k.pitch = static_cast<int>(q_pitch);
    k.scale_pitch = static_cast<int>(scale_pitch);
    const int64_t pieces = (rows + kUnitRows - 1) / kUnitRows;
    k.band_units = static_cast<int>(std::max<int64_t>(1, pieces / groups));
    const int64_t units = (pieces + k.band_units - 1) / k.band_units * k.band_units * k.tk;
    if (direct && units <= INT32_MAX / 2 && 3 * first_wave_pieces(k, pairs) <= 2 * (units + 2ll * pairs)) {
      k.units = static_cast<int>(units);
      uint8_t *sync = nullptr;  // counters that every call leaves at 0
      const size_t bytes = 256 + static_cast<size_t>((rows + kBlockRows - 1) / kBlockRows) * k.tk * 4;
      if ((rc = call.workspace(kSlotWgradSync, bytes, &sync, bytes))) return rc;
      k.left = reinterpret_cast<int *>(sync);
      k.widened = reinterpret_cast<int *>(sync + 256);
    }
    PrepareParams pp{static_cast<const int8_t *>(q), static_cast<const uint8_t *>(scales),
                     reinterpret_cast<__nv_bfloat16 *>(ws), direct ? nullptr : dy,
                     reinterpret_cast<__nv_bfloat16 *>(ws + x_bytes), ld_dy, k.rows, k.n_in, static_cast<int>(q_pitch),
                     static_cast<int>(scale_pitch), k.n_out, static_cast<int>(pitch), k.slices, k.status};
    if (k.units == 0 && (rc = call.launch(kOpWgrad, [&] { return run_prepare(pp, dtype, call.sms, call.s); }))) return rc;
  }
  if (k.store != kStorePlain) {
    const bool f32 = k.splits > 1 || grad_dtype == NS_F32;
    const int64_t row_bytes = k.splits > 1 ? k.part_pitch * 4ll : n_in * gelt;
    const int64_t dims[3] = {n_in, n_out, static_cast<int64_t>(groups) * k.splits}, strides[2] = {row_bytes, row_bytes * n_out};
    const int box[3] = {f32 ? 32 : 64, 32, 1};
    if ((rc = call.tensor_map(&k.tm_out, f32 ? 4 : 2, k.splits > 1 ? static_cast<void *>(k.parts) : grad, 3, dims, strides, box)))
      return rc;
  }
  if (k.units > 0) {  // CTAs that wait for one another's pieces of X: all resident at once
    attr[1].id = cudaLaunchAttributeCooperative;
    attr[1].val.cooperative = 1;
  }
  cfg.gridDim = dim3(2 * static_cast<unsigned>(std::min<int64_t>(pairs, std::max(k.items, (k.units + 1) / 2))), 1, 1);
  cfg.numAttrs = rows > 0 ? 2 : 1;
  cfg.blockDim = dim3(threads_of(k.units > 0), 1, 1);
  rc = call.launch(kOpWgrad, [&] {
    if (cudaLaunchKernelEx(&cfg, k.units > 0 ? ns_wgrad_kernel<true> : ns_wgrad_kernel<false>, k) != cudaSuccess) {
      cudaGetLastError();
      return -1;
    }
    count_launch();
    return 0;
  });
  if (rc || k.splits == 1) return rc;
  return call.launch(kOpWgrad, [&] { return run_join(k, call.sms, call.s); });
}
