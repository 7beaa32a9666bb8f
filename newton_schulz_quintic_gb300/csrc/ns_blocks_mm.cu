// ns_blocks_mm.cu -- products of matrices held in e4m3 with a scale for each
// block of 128 (include/ns.h): Out = A W^T over groups of rows, or A W.
//
// A scale belongs to 128 values of the contraction, so a k-block is 128 deep:
// the tensor cores multiply it (tcgen05.mma kind::f8f6f4, fp32 accumulators in
// TMEM) and its sum is multiplied by the two scales, one power of two, and
// added to fp32 registers while the next k-block runs in the other accumulator.
//
// One persistent kernel of CTA pairs (clusters of 2), one 256 x 256 tile of Out
// at a time (cta_group::2, M = 256, N = 256, K = 32). CTA rank r holds rows
// r*128.. of A's and r*128.. of W's share. W is K-major as it lies for A W^T and
// MN-major for A W; the tensor cores read both. Warps of a CTA:
//   0      TMA: 128 rows x 128 values of A and of W (16 KB each, 128-byte
//          swizzle) into a 6-stage ring
//   1      TMEM (two accumulators of 256 columns); in the leader the MMAs
//   2      passes a landed stage on to the leader's MMAs
//   3      looks the pair's tiles up (place, group, rows) a few ahead
//   4..11  sums: 32 rows x 128 columns each
// Rows of other groups that a tile loads give rows of the tile that are not
// stored.
// Every wait is bounded (mbar_wait): on a timeout the status word is set, the
// CTA waits for its own copies and MMAs, frees TMEM and exits.
#include <algorithm>

#include "../../include/ns.h"
#include "ns_rows.cuh"

namespace ns {

namespace {

constexpr int kBK = 128;                         // depth of a k-block: one scale
constexpr int kStages = 6;
constexpr int kShare = 128 * kBK;                // one operand's share of a stage: 16 KB
constexpr int kIssueWarps = 4, kSumWarps = 8;
constexpr int kThreads = 32 * (kIssueWarps + kSumWarps);
// Registers a thread after the warpgroups have divided what the launch holds (168 each).
constexpr int kIssueRegs = 72, kSumRegs = 208;
constexpr int kTmemCols = 512;
constexpr int kPatch = 32 * 32 * 4;              // staging of 32 rows x 128 bytes per sum warp
constexpr int kMaxGroups = 1 << 20;

enum Store : int { kStoreTma, kStorePlain };

struct BmmParams {
  CUtensorMap tm_a;        // {K, rows}, box {128, 128}
  CUtensorMap tm_w;        // {columns, rows of one matrix, groups}, box {128, 128, 1}
  CUtensorMap tm_out;      // Out: {N, rows}, box of 128 bytes x 32 rows
  const uint8_t *sa, *sw;  // scales
  const int32_t *offsets;  // nullptr: one group of all rows
  void *out;
  int64_t ld_out;
  int rows, n, k, groups;
  int sa_pitch, sw_pitch;
  int sw_rows;             // rows of scales of one matrix of W
  int nb;                  // k-blocks
  int tn;                  // tiles along N
  int back;                // 1: Out = A W, W is K x N
  int odtype, store;
  int *status;
  uint64_t wait_limit_ns;
};

// One tile of the pair's list as warp 3 hands it out.
struct alignas(16) MTile {
  int m0, n0;  // its first row and column of Out
  int hi;      // rows of its group end here; < 0: no more tiles
  int e;       // its group; < 0: rows of no group, all zeros
};
constexpr int kQueue = 4;

struct BmmBarriers {
  MTile queue[kQueue];
  uint64_t qfull[kQueue];    // a slot holds the next tile
  uint64_t qempty[kQueue];   // every consumer of this CTA has read it
  uint64_t full[kStages];    // this CTA's boxes of a stage landed
  uint64_t ready[kStages];   // leader: both CTAs' operands of a stage are in place
  uint64_t empty[kStages];   // each CTA: the MMAs are done with a stage
  uint64_t tfull[2];         // each CTA: an accumulator holds a k-block
  uint64_t tempty[2];        // leader: both CTAs have drained an accumulator
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};
constexpr int kBarBytes = (static_cast<int>(sizeof(BmmBarriers)) + 127) / 128 * 128;
constexpr int kSmem = 1024 + kStages * 2 * kShare + kSumWarps * kPatch + kBarBytes;
static_assert(kSmem <= 227 * 1024, "shared memory of the product kernel");

struct MTileReader {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void step() {
    if (++slot == kQueue) {
      slot = 0;
      parity ^= 1u;
    }
  }
  __device__ __forceinline__ bool take(BmmBarriers *bar, MTile &t, const Waiter &w) {
    if (!mbar_wait(&bar->qfull[slot], parity, w)) return false;
    t = bar->queue[slot];
    mbar_arrive(&bar->qempty[slot]);
    step();
    return t.hi >= 0;
  }
  __device__ __forceinline__ bool take_warp(BmmBarriers *bar, MTile &t, const Waiter &w) {
    if (!warp_mbar_wait<false>(&bar->qfull[slot], parity, w)) return false;
    __syncwarp();
    t = bar->queue[slot];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&bar->qempty[slot]);
    step();
    return t.hi >= 0;
  }
};

// Rows [lo, hi) of part e: the groups in order, then (with offsets) the rows before the first and behind the last.
__device__ __forceinline__ void part_rows(const BmmParams &p, int e, int &lo, int &hi) {
  lo = 0;
  hi = p.rows;
  if (!p.offsets) return;
  if (e < p.groups) {
    lo = min(max(__ldg(p.offsets + e), 0), p.rows);
    hi = min(max(__ldg(p.offsets + e + 1), lo), p.rows);
  } else if (e == p.groups) {
    hi = min(max(__ldg(p.offsets), 0), p.rows);
  } else {
    lo = min(max(__ldg(p.offsets + p.groups), 0), p.rows);
  }
}

// The pair's tiles in order, found by a whole warp that walks over the parts 32 at a time.
struct TileWalk {
  int e0 = 0;          // first part of the 32 in hand
  int64_t base = 0;    // tiles before them
  int64_t incl = 0;    // this lane's part and those before it in the 32
  int lo = 0, hi = 0;  // this lane's part's rows
  int parts;
  __device__ __forceinline__ void load(const BmmParams &p) {
    const int lane = threadIdx.x & 31, e = e0 + lane;
    lo = hi = 0;
    if (e < parts) part_rows(p, e, lo, hi);
    incl = static_cast<int64_t>((hi - lo + 255) / 256) * p.tn;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
  }
  __device__ __forceinline__ void start(const BmmParams &p) {
    parts = p.groups + (p.offsets ? 2 : 0);
    load(p);
  }
  // Tile `item`; items ascend from call to call.
  __device__ __forceinline__ bool find(const BmmParams &p, int64_t item, MTile &t) {
    for (;;) {
      const uint32_t in = __ballot_sync(0xffffffffu, item < base + incl);
      if (in) {
        const int l = __ffs(in) - 1;
        const int64_t before = __shfl_sync(0xffffffffu, incl, l > 0 ? l - 1 : 0);
        const int first = __shfl_sync(0xffffffffu, lo, l), end = __shfl_sync(0xffffffffu, hi, l);
        const int tile = static_cast<int>(item - base - (l > 0 ? before : 0));
        // bands of 8 tiles of rows, column by column, so that the tiles in flight share a few panels
        const int tm = (end - first + 255) / 256, band = tile / (8 * p.tn), row = band * 8;
        const int height = min(8, tm - row), rest = tile - band * 8 * p.tn;
        t.m0 = first + (row + rest % height) * 256;
        t.n0 = rest / height * 256;
        t.hi = end;
        t.e = e0 + l < p.groups ? e0 + l : -1;
        return true;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
      e0 += 32;
      if (e0 >= parts) return false;
      load(p);
    }
  }
};

// Instruction descriptor of kind::f8f6f4: D fp32, A and B e4m3; b_mn selects an MN-major B operand.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, int a_mn, int b_mn) {
  return (1u << 4)                                    // D format: f32
         | (0u << 7) | (0u << 10)                     // A and B format: e4m3
         | (static_cast<uint32_t>(a_mn & 1) << 15) | (static_cast<uint32_t>(b_mn & 1) << 16)
         | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// Operand of 128 rows x 128 bytes written by TMA with the 128-byte swizzle. K-major: a row is one M or N index, a step
// of 32 along K is 32 bytes. MN-major: a row is one K index and holds 128 M or N indices, a step of 32 along K is 32
// rows; there is one such chunk, so the leading offset is not used.
__device__ __forceinline__ uint64_t e4m3_desc(uint32_t smem_addr) { return sw128_kmajor_desc(smem_addr); }

__device__ __forceinline__ void umma_e4m3_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 2^(a + b - 254) of two scale bytes, NaN for a block with infinities or NaN. In range: a normal or subnormal float.
__device__ __forceinline__ float pow2_of(int e) {  // 2^e, e in [-149, 127]
  return e >= -126 ? __int_as_float((e + 127) << 23) : __int_as_float(1 << (e + 149));
}

// The sums of one thread (row row0 + lane, 128 columns from col0) by TMA, 32
// rows x 128 bytes at a time through the warp's staging block, in the swizzled layout of the map.
template <bool kHalf>
__device__ __forceinline__ void put_tma(const BmmParams &p, int row0, int col0, const float (&acc)[128], uint8_t *patch) {
  constexpr int kCols = kHalf ? 64 : 32;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = 0; h < 128 / kCols; ++h) {
    if (col0 + h * kCols >= p.n) break;
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
    if (lane == 0) tma_store_2d(&p.tm_out, col0 + h * kCols, row0, patch);
  }
}

// The same element by element: the first `rows` of the 32 rows, for rows that
// TMA cannot address and tiles in which a group ends. A store covers 32 columns of a row.
template <int OT>
__device__ __forceinline__ void put_plain(const BmmParams &p, int row0, int rows, int col0, const float (&acc)[128], float *patch) {
  using O = typename Elem<OT>::T;
  const int lane = threadIdx.x & 31;
  const size_t size = static_cast<size_t>((p.rows - 1) * p.ld_out + p.n) * sizeof(O);
  O *to = static_cast<O *>(p.out) + static_cast<int64_t>(row0) * p.ld_out + col0 + lane;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    __syncwarp();
    // row lane, column c at word (c ^ lane): no bank conflict either way
#pragma unroll
    for (int c = 0; c < 32; ++c) patch[lane * 32 + (c ^ lane)] = acc[32 * k + c];
    __syncwarp();
    if (col0 + 32 * k + lane >= p.n) continue;
    O *g = to + 32 * k;
#pragma unroll 4
    for (int r = 0; r < rows; ++r, g += p.ld_out)
      if (in_bounds(g, sizeof(O), p.out, size, p.status)) *g = Elem<OT>::from_f(patch[r * 32 + (lane ^ r)]);
  }
}

template <bool kBack>
__global__ void __launch_bounds__(kThreads, 1) ns_blocks_mm_kernel(const __grid_constant__ BmmParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *sA = smem, *sB = smem + kStages * kShare, *patches = sB + kStages * kShare;
  BmmBarriers *bar = reinterpret_cast<BmmBarriers *>(patches + kSumWarps * kPatch);
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
  const bool tmem_ok = ld_shared_cluster_u32(mapa_shared(smem_u32(&bar->tmem_base), rank ^ 1u)) == tmem;
  if (!tmem_ok && threadIdx.x == 0) set_status(p.status, kStatusTmemMismatch);
  volatile int *abort = &bar->abort;
  const Waiter w{abort, p.status, p.wait_limit_ns};

  if (warp < kIssueWarps)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
  if (tmem_ok && warp == 0) {
    // ---------------------------------------------------- operands by TMA, issued by one lane
    if (elect_one()) {
      int stage = 0;
      uint32_t parity = 0;
      uint32_t issued = 0, last = 0;  // per stage: whether copies were issued, the parity of the last
      const int r = static_cast<int>(rank) * 128;
      MTileReader tiles;
      MTile t;
      bool ok = true;
      while (ok && tiles.take(bar, t, w)) {
        if (t.e < 0) continue;
        for (int b = 0; b < p.nb; ++b) {
          if (!(ok = mbar_wait<true>(&bar->empty[stage], parity ^ 1u, w))) break;
          mbar_arrive_expect_tx(&bar->full[stage], 2 * kShare);
          tma_load_2d(sA + stage * kShare, &p.tm_a, b * kBK, t.m0 + r, &bar->full[stage]);
          if (kBack)
            tma_load_3d(sB + stage * kShare, &p.tm_w, t.n0 + r, b * kBK, t.e, &bar->full[stage]);
          else
            tma_load_3d(sB + stage * kShare, &p.tm_w, b * kBK, t.n0 + r, t.e, &bar->full[stage]);
          issued |= 1u << stage;
          last = (last & ~(1u << stage)) | (parity << stage);
          if (++stage == kStages) {
            stage = 0;
            parity ^= 1u;
          }
        }
      }
      if (*abort)
        for (int s = 0; s < kStages; ++s)
          if ((issued >> s) & 1u) drain_wait(&bar->full[s], (last >> s) & 1u, w.limit_ns);
    }
  } else if (tmem_ok && warp == 1 && leader) {
    // ---------------------------------------------------- MMAs, issued by one lane
    if (elect_one()) {
      constexpr uint32_t idesc = idesc_e4m3(256, 256, 0, kBack ? 1 : 0);
      constexpr uint64_t kStepB = kBack ? 32 * 128 / 16 : 32 / 16;  // 32 along K, in 16-byte units
      const uint64_t desc_a = e4m3_desc(smem_u32(sA)), desc_b = e4m3_desc(smem_u32(sB));
      int stage = 0, acc = 0;
      uint32_t parity = 0, acc_parity = 0;
      bool ok = true, seen = false;  // seen: the next stage is known to be ready
      MTileReader tiles;
      MTile t;
      while (ok && tiles.take(bar, t, w)) {
        if (t.e < 0) continue;
        for (int b = 0; b < p.nb; ++b) {
          if (!(ok = mbar_wait<true>(&bar->tempty[acc], acc_parity ^ 1u, w))) break;
          if (!seen && !(ok = mbar_wait<true>(&bar->ready[stage], parity, w))) break;
          tc_fence_after();
          const uint32_t d = tmem + static_cast<uint32_t>(acc * 256);
          const uint64_t at = static_cast<uint64_t>(stage * (kShare >> 4));
          uint64_t *const empty = &bar->empty[stage];
          if (++stage == kStages) {
            stage = 0;
            parity ^= 1u;
          }
          umma_e4m3_pair(d, desc_a + at, desc_b + at, idesc, 0);
          umma_e4m3_pair(d, desc_a + at + 2u, desc_b + at + kStepB, idesc, 1);
          // look at the next stage while these run, so that its first MMA follows the last one here at once
          seen = mbar_try_wait_cluster(&bar->ready[stage], parity);
          umma_e4m3_pair(d, desc_a + at + 4u, desc_b + at + 2 * kStepB, idesc, 1);
          umma_e4m3_pair(d, desc_a + at + 6u, desc_b + at + 3 * kStepB, idesc, 1);
          umma_commit_pair_multicast(empty, 3u);
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
    if (elect_one()) {
      int stage = 0;
      uint32_t parity = 0;
      MTileReader tiles;
      MTile t;
      bool ok = true;
      while (ok && tiles.take(bar, t, w)) {
        if (t.e < 0) continue;
        for (int b = 0; b < p.nb; ++b) {
          if (!(ok = mbar_wait<true>(&bar->full[stage], parity, w))) break;
          arrive_pair(mapa_shared(smem_u32(&bar->ready[stage]), 0));
          if (++stage == kStages) {
            stage = 0;
            parity ^= 1u;
          }
        }
      }
    }
  } else if (tmem_ok && warp == 3) {
    // ---------------------------------------------------- the pair's tiles, looked up ahead
    int slot = 0;
    uint32_t parity = 0;
    bool more = true;
    TileWalk walk;
    walk.start(p);
    for (int64_t item = pair; more; item += npairs) {
      MTile t;
      more = walk.find(p, item, t);
      if (!more) t.hi = -1;
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
  } else if (tmem_ok && warp >= kIssueWarps) {
    // ---------------------------------------------------- sums and the tile's store
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
    const int e = warp - kIssueWarps, quarter = warp & 3, half = e >> 2;
    uint8_t *patch = patches + e * kPatch;
    int acc = 0;
    uint32_t acc_parity = 0;
    bool ok = true;
    MTileReader tiles;
    MTile t;
    while (ok && tiles.take_warp(bar, t, w)) {
      float sum[128];
#pragma unroll
      for (int c = 0; c < 128; ++c) sum[c] = 0.f;
      const int row0 = t.m0 + static_cast<int>(rank) * 128 + quarter * 32, col0 = t.n0 + half * 128;
      const uint8_t *sa = p.sa + static_cast<int64_t>(min(row0 + lane, p.rows - 1)) * p.sa_pitch;
      const uint8_t *sw = p.sw + static_cast<int64_t>(max(t.e, 0)) * p.sw_rows * p.sw_pitch;
      // the 128 columns' block: along K in a row of the scales (A W^T) or in a column of them (A W)
      const int nblock = min(col0, p.n - 1) / 128;
      sw += kBack ? nblock : static_cast<int64_t>(nblock) * p.sw_pitch;
      const int sw_step = kBack ? p.sw_pitch : 1;
      const int nb = t.e < 0 ? 0 : p.nb;
      int ea = 0, ew = 0;
      if (nb > 0) {
        ea = __ldg(sa);
        ew = __ldg(sw);
      }
      for (int b = 0; b < nb; ++b) {
        const int ca = ea, cw = ew;
        if (b + 1 < nb) {  // the next block's scales
          ea = __ldg(sa + b + 1);
          ew = __ldg(sw + (b + 1) * sw_step);
        }
        if (!warp_mbar_wait<true>(&bar->tfull[acc], acc_parity, w)) {
          ok = false;
          break;
        }
        __syncwarp();
        tc_fence_after();
        const uint32_t src = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * 256 + half * 128);
        const int ex = max(ca, 1) + max(cw, 1) - 254;
        const bool nan = ca == 255 || cw == 255;
        // one factor where both scales' product is a float; else one after the other (values near the type's ends)
        const bool split = !nan && (ex < -149 || ex > 127);
        const float f = nan ? __int_as_float(0x7fc00000) : split ? 0.f : pow2_of(ex);
        if (!__any_sync(0xffffffffu, split)) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            uint32_t v[16];
            tmem_ld16(src + 16 * k, v);
#pragma unroll
            for (int u = 0; u < 16; ++u) sum[16 * k + u] = fmaf(__uint_as_float(v[u]), f, sum[16 * k + u]);
          }
        } else {
          const float fa = ca == 255 ? __int_as_float(0x7fc00000) : pow2_of(max(ca, 1) - 127);
          const float fw = cw == 255 ? __int_as_float(0x7fc00000) : pow2_of(max(cw, 1) - 127);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            uint32_t v[16];
            tmem_ld16(src + 16 * k, v);
#pragma unroll
            for (int u = 0; u < 16; ++u) sum[16 * k + u] = fmaf(__uint_as_float(v[u]) * fa, fw, sum[16 * k + u]);
          }
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
      const int rows = min(32, t.hi - row0);
      if (rows <= 0 || col0 >= p.n) continue;
      if (p.store == kStorePlain || rows < 32) {
        if (lane == 0) bulk_read_wait();
        if (p.odtype == kBF16)
          put_plain<kBF16>(p, row0, rows, col0, sum, reinterpret_cast<float *>(patch));
        else
          put_plain<kF32>(p, row0, rows, col0, sum, reinterpret_cast<float *>(patch));
        __syncwarp();
      } else if (p.odtype == kBF16) {
        put_tma<true>(p, row0, col0, sum, patch);
      } else {
        put_tma<false>(p, row0, col0, sum, patch);
      }
    }
    if (lane == 0) bulk_wait();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, kTmemCols);
}

// CTA pairs that can be resident at once on this device (one CTA per SM).
template <bool kBack>
int resident_pairs(int dev, int sms, cudaLaunchConfig_t &cfg) {
  static int cached[64] = {};
  int &n = cached[dev & 63];
  if (n == 0) {
    static SmemOptIn opt_in;
    if (opt_in.ensure(reinterpret_cast<const void *>(ns_blocks_mm_kernel<kBack>), kSmem)) return 0;
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, ns_blocks_mm_kernel<kBack>) != cudaSuccess ||
        attr.numRegs * kThreads < 128 * (kIssueRegs + 2 * kSumRegs)) {  // a share beyond it would never be granted
      cudaGetLastError();
      return 0;
    }
    cfg.gridDim = dim3(sms / 2 * 2, 1, 1);
    if (cudaOccupancyMaxActiveClusters(&n, ns_blocks_mm_kernel<kBack>, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = 0;
    }
  }
  return n;
}

template <bool kBack>
int run_mm(const BmmParams &p, const OpCall &call) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = call.s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(kThreads, 1, 1);
  const int pairs = resident_pairs<kBack>(call.dev, call.sms, cfg);
  if (pairs <= 0) return -1;
  // at most this many tiles: each group may end inside one, and so may the rows before and behind them
  const int64_t parts = p.offsets ? p.groups + 2 : 1;
  const int64_t tiles = (std::min<int64_t>(p.rows, p.rows / 256 + parts)) * p.tn;
  cfg.gridDim = dim3(2 * static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(pairs, tiles))), 1, 1);
  if (cudaLaunchKernelEx(&cfg, ns_blocks_mm_kernel<kBack>, p) != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  count_launch();
  return 0;
}

}  // namespace
}  // namespace ns

using namespace ns;

extern "C" int ns_blocks_matmul(const void *qa, const void *sa, int64_t rows, int64_t k, const void *qw, const void *sw,
                                int64_t n, int back, const int32_t *offsets, int groups, void *out, int64_t ld_out,
                                int dtype, void *stream) {
  if ((dtype != NS_F32 && dtype != NS_BF16) || (back != 0 && back != 1) || groups < 0 || groups > kMaxGroups) return NS_EINVAL;
  if (!offsets && groups != 1) return NS_EINVAL;
  const int64_t w_rows = back ? k : n, w_cols = back ? n : k;
  if (bad_shape(rows, k, k) || bad_shape(rows, n, ld_out) || bad_shape(w_rows, w_cols, w_cols) || rows > (1 << 30) ||
      n > (1 << 30) || k > (1 << 30))
    return NS_EINVAL;
  if (groups > 0 && w_rows > 0 && w_cols > (int64_t(1) << 42) / w_rows / groups) return NS_EINVAL;
  if (rows == 0 || n == 0) return NS_OK;
  if (!out || (k > 0 && (!qa || !sa || (groups > 0 && (!qw || !sw))))) return NS_EINVAL;
  const int elt = dtype == NS_BF16 ? 2 : 4;
  if (misaligned(qa, 16) || misaligned(sa, 16) || misaligned(qw, 16) || misaligned(sw, 16) || misaligned(offsets, 4) ||
      misaligned(out, elt))
    return NS_EALIGN;
  const int64_t pa = ns_blocks_pitch(k), spa = ns_blocks_scale_pitch(k), pw = ns_blocks_pitch(w_cols), spw = ns_blocks_scale_pitch(w_cols);
  const int64_t sw_rows = (w_rows + 127) / 128, all = groups * w_rows, bands = groups * sw_rows;
  const Range ro(out, rows, n, ld_out, elt);
  if (ro.overlaps(Range(qa, rows, pa, pa, 1)) || ro.overlaps(Range(sa, rows, spa, spa, 1)) || ro.overlaps(Range(qw, all, pw, pw, 1)) ||
      ro.overlaps(Range(sw, bands, spw, spw, 1)) || ro.overlaps(Range(offsets, 1, groups + int64_t(1), groups + int64_t(1), 4)))
    return NS_EINVAL;
  OpCall call(stream);
  if (call.rc) return call.rc;
  BmmParams p{};
  p.sa = static_cast<const uint8_t *>(sa);
  p.sw = static_cast<const uint8_t *>(sw);
  p.offsets = offsets;
  p.out = out;
  p.ld_out = ld_out;
  p.rows = static_cast<int>(rows);
  p.n = static_cast<int>(n);
  p.k = static_cast<int>(k);
  p.groups = groups;
  p.sa_pitch = static_cast<int>(spa);
  p.sw_pitch = static_cast<int>(spw);
  p.sw_rows = static_cast<int>(sw_rows);
  p.nb = groups > 0 ? static_cast<int>((k + kBK - 1) / kBK) : 0;
  p.tn = static_cast<int>((n + 255) / 256);
  p.back = back;
  p.odtype = dtype;
  p.status = call.status;
  p.wait_limit_ns = kWaitLimitNs;
  // TMA writes what it can address. Debug builds store where every store is checked.
  p.store = kDebugBounds || misaligned(out, 16) || ld_out * elt % 16 != 0 ? kStorePlain : kStoreTma;
  int rc;
  if (p.nb > 0) {
    const int box[3] = {128, 128, 1};
    const int64_t adims[2] = {k, rows}, astride[1] = {pa};
    if ((rc = call.tensor_map(&p.tm_a, 1, qa, 2, adims, astride, box))) return rc;
    const int64_t wdims[3] = {w_cols, w_rows, groups}, wstride[2] = {pw, pw * w_rows};
    if ((rc = call.tensor_map(&p.tm_w, 1, qw, 3, wdims, wstride, box))) return rc;
  }
  if (p.store == kStoreTma) {
    const int64_t dims[2] = {n, rows}, stride[1] = {ld_out * elt};
    const int box[2] = {elt == 4 ? 32 : 64, 32};
    if ((rc = call.tensor_map(&p.tm_out, elt, out, 2, dims, stride, box))) return rc;
  }
  return call.launch(kOpBlocksMatmul, [&] { return back ? run_mm<true>(p, call) : run_mm<false>(p, call); });
}
