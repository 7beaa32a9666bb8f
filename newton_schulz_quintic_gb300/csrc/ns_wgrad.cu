// ns_wgrad.cu -- weight gradients from an input held in 8 bits
// (include/ns.h): G[e] (+)= dY[e]^T X[e] over the rows of each group.
//
// A GEMM whose contraction runs over rows (tokens): both operands are
// MN-major as they lie in memory. A value of X is q * 2^(E - 133) with |q| <=
// 127, exact in bf16, so X is turned into bf16 on its way into shared memory
// and the product runs at the bf16 rate of the tensor cores with no rounding
// of X; HBM and L2 move one byte per value of X instead of two.
//
// One persistent kernel of CTA pairs (clusters of 2), one 256 x 256 tile of one
// group's G at a time (tcgen05.mma.cta_group::2, M = 256, N = 256, K = 16).
// CTA rank r holds rows (n_out) r*128.. and columns (n_in) r*128.. of the
// operands. Warps of a CTA:
//   0       TMA of dY: its 128 columns x 64 rows of a k-block (two 64 x 64
//           boxes, 128-byte swizzle) into a 5-stage ring
//   1       TMEM (two accumulators of 256 columns); in the leader the MMAs
//   2       X as it is held: q by TMA, the rows' scales by cp.async, into a
//           ring of their own, up to 4 k-blocks ahead
//   3       passes on to the MMA warp that dY has landed
//   4..11   X made bf16 (see widen4), from that ring to where the MMA reads
//           it, in the swizzled layout, two groups of four warps taking
//           k-blocks in turn: what a warp spends on a k-block is mostly
//           latency. They also clear the rows beyond the group's end in both
//           operands, so nothing of the next group (infinities, NaN) takes part.
//   12..19  sums: every kChunk k-blocks the accumulator is added to fp32
//           registers (128 columns x 1 row per thread) while the MMAs go on in
//           the other one; the tile is written at its end. The tensor cores'
//           own accumulation loses up to a unit in the last place per
//           instruction; 32 instructions between two drains keep that near
//           2^-21 of the sum for any number of rows.
// X goes through shared memory twice because loads into registers do not
// stay in flight here: the proxy fence and the release of a stage wait for
// them (measured: 6600 cycles per k-block against 512 of MMA).
// Registers are split by warpgroup with setmaxnreg: 160 for the sums, 48
// elsewhere, together no more than the 96 x 640 the CTA is launched with.
//
// fp32 dY is held as three bf16 slices (the h + m + l of ns_tc.cu) and the
// k-loop runs over the slices too, smallest first; X needs no slices. A dY that
// TMA cannot address (pitch or base not on 16 bytes) is copied to a padded
// buffer first. When there are fewer tiles than CTA pairs the rows are split
// and the parts, fp32 in scratch, are added in order by a second kernel.
// Every wait is bounded (mbar_wait): on a timeout the status word is set, the
// CTA waits for its own copies and MMAs, frees TMEM and exits.
#include <algorithm>

#include "../../include/ns.h"
#include "ns_rows.cuh"

namespace ns {

namespace {

constexpr int kBK = 64;                          // rows per k-block
constexpr int kStages = 5;
constexpr int kRawStages = 4;                    // k-blocks of X as it is held
constexpr int kRaw = 128 * kBK;                  // q of this CTA's 128 columns: 8 KB
constexpr int kRawScales = 4 * kBK;              // and their scales
constexpr int kShare = 128 * kBK * 2;            // one operand's share of a stage: 16 KB
constexpr int kBoxBytes = 64 * kBK * 2;          // one TMA box
constexpr int kChunk = 8;                        // k-blocks between two drains of an accumulator
constexpr int kThreads = 640;
constexpr int kConvWarps = 4, kConvGroups = 2, kSumWarps = 8;
constexpr int kConv0 = 4, kSum0 = kConv0 + kConvWarps * kConvGroups;  // first warps of the roles
constexpr int kTmemCols = 512;
constexpr int kPatch = 32 * 32 * 4;              // staging of one 32 x 32 block per sum warp

struct WgradParams {
  CUtensorMap tm_dy;       // bf16 {n_out, rows, slices}, box {64, 64, 1}
  CUtensorMap tm_q;        // bytes {n_in, rows}, box {128, 64}
  const uint8_t *s;
  const int32_t *offsets;  // nullptr: one group of all rows
  void *grad;              // groups x n_out x n_in
  float *parts;            // splits x groups x n_out x n_in when splits > 1
  int rows, n_out, n_in, scale_pitch, groups;
  int slices;              // bf16 slices of dY (1 or 3)
  int splits;              // parts of a group's rows
  int tn, tk, items;       // tiles along n_out and n_in; groups * tn * tk * splits
  int accumulate, gdtype;
  int *status;
  uint64_t wait_limit_ns;
};

struct WgradBarriers {
  uint64_t afull[kStages];   // this CTA's dY boxes landed
  uint64_t ready[kStages];   // leader: both CTAs' operands of a stage are in place
  uint64_t empty[kStages];   // each CTA: the MMAs are done with a stage
  uint64_t rawfull[kRawStages];   // a k-block of q and scales landed
  uint64_t rawempty[kRawStages];  // the converters have read it
  uint64_t tfull[2];         // each CTA: an accumulator holds a chunk
  uint64_t tempty[2];        // leader: both CTAs have drained an accumulator
  uint64_t drain;
  int left[kRawStages];      // rows of the group in this k-block and after; -1: no more
  uint32_t tmem_base;
  int abort;
};
constexpr int kBarBytes = (static_cast<int>(sizeof(WgradBarriers)) + 127) / 128 * 128;
constexpr int kSmem = 1024 + kStages * 2 * kShare + kRawStages * (kRaw + kRawScales) + kBarBytes + kSumWarps * kPatch;
static_assert(kSmem <= 227 * 1024, "shared memory of the weight-gradient kernel");

// One tile of the work list: its place and its rows [lo, hi), split into k-blocks.
struct WTile {
  int e, n0, k0, split;
  int lo, hi;
  __device__ __forceinline__ int blocks() const { return (hi - lo + kBK - 1) / kBK; }
};

// Tiles in groups of 8 along n_out, column by column within a group, so the
// tiles in flight share a few panels of each operand.
__device__ __forceinline__ WTile wtile(const WgradParams &p, int item) {
  WTile t;
  const int per = p.tn * p.tk;
  t.split = item % p.splits;
  const int g = item / p.splits;
  t.e = g / per;
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
    const int a = static_cast<int>(nb * t.split / p.splits), b = static_cast<int>(nb * (t.split + 1) / p.splits);
    t.hi = min(t.hi, t.lo + b * kBK);
    t.lo += a * kBK;
    if (t.hi < t.lo) t.hi = t.lo;
  }
  return t;
}

__device__ __forceinline__ void tma_bytes(void *dst, const void *map, int x, int y, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}
// 4 bytes to shared memory, zeros when !inside.
__device__ __forceinline__ void copy4(void *dst, const void *src, bool inside) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(inside ? 4 : 0) : "memory");
}
// One of the barrier's expected arrivals, made when this thread's copies so far have landed.
__device__ __forceinline__ void arrive_after_copies(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma_box(void *dst, const void *map, int x, int y, int z, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
// Arrive on a barrier of either CTA of the pair once this CTA's operands are
// in place. What it orders lies in this CTA's own shared memory and has passed
// the proxy fence, so the release is at CTA scope: at cluster scope it would
// wait for every outstanding access of the warp, the loads ahead included.
__device__ __forceinline__ void arrive_pair(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}
// 32 lanes x 16 columns of TMEM words, complete on return.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void fence_proxy_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Four int8 (bytes 0..3 of w) to two bf16 pairs, times a power of two. With l
// the low 7 bits of a byte and s its sign bit, q = l - 128 s; the bf16 0x4300 |
// l is 128 + l and 0xC300 | (s << 7) is -(128 + 128 s), so their sum is q,
// exact in bf16 (as is the product: no bits are added, and units are at least
// 2^-126). Even bytes make the first pair, odd ones the second, which
// saves the byte shuffles: the second and third column of every four change
// places in shared memory and in the accumulator, and the store puts them back
// (true_column).
__device__ __forceinline__ void widen4(uint32_t w, __nv_bfloat162 unit, uint32_t &even, uint32_t &odd) {
  const uint32_t v = w >> 8;
  const uint32_t a0 = (w & 0x007f007fu) | 0x43004300u, b0 = (w & 0x00800080u) | 0xC300C300u;
  const uint32_t a1 = (v & 0x007f007fu) | 0x43004300u, b1 = (v & 0x00800080u) | 0xC300C300u;
  auto two = [](const uint32_t &x) { return *reinterpret_cast<const __nv_bfloat162 *>(&x); };
  const __nv_bfloat162 r0 = __hmul2(__hadd2(two(a0), two(b0)), unit);
  const __nv_bfloat162 r1 = __hmul2(__hadd2(two(a1), two(b1)), unit);
  even = *reinterpret_cast<const uint32_t *>(&r0);
  odd = *reinterpret_cast<const uint32_t *>(&r1);
}
// accumulator column of matrix column c (and back)
__device__ constexpr int true_column(int c) { return (c & 3) == 1 ? c + 1 : (c & 3) == 2 ? c - 1 : c; }
// 2^(e - 133) twice as bf16 (e below 7 reads as 7; 255 as NaN)
__device__ __forceinline__ __nv_bfloat162 unit_pair(uint32_t e) {
  const uint32_t u = e == 255u ? 0x7fc0u : (max(e, 7u) - 6u) << 7;
  const uint32_t v = u | (u << 16);
  return *reinterpret_cast<const __nv_bfloat162 *>(&v);
}

// A wait of a whole warp that is over as a rule: every lane polls once, and
// only if that fails lane 0 goes on polling for all.
template <bool kCluster>
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const Waiter &w) {
  const bool ok = kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
  if (__all_sync(0xffffffffu, ok)) return true;
  return warp_mbar_wait<kCluster>(bar, parity, w);
}

// The k-blocks of a pair's whole work list in order: tile by tile, a tile's
// chunks of kChunk blocks, in each the slices of dY from smallest to largest,
// in each slice the chunk's blocks.
struct BlockWalk {
  WTile t;
  int item, c, z, b;  // current block: chunk start, slice, block
  bool done;
  __device__ __forceinline__ void open(const WgradParams &p, int npairs) {
    for (; item < p.items; item += npairs) {
      t = wtile(p, item);
      if (t.blocks() > 0) {
        c = 0;
        b = 0;
        z = p.slices - 1;
        return;
      }
    }
    done = true;
  }
  __device__ __forceinline__ void start(const WgradParams &p, int pair, int npairs) {
    item = pair;
    done = false;
    open(p, npairs);
  }
  __device__ __forceinline__ void next(const WgradParams &p, int npairs) {
    const int nb = t.blocks();
    if (++b < min(c + kChunk, nb)) return;
    if (--z >= 0) {
      b = c;
      return;
    }
    c += kChunk;
    if (c < nb) {
      b = c;
      z = p.slices - 1;
      return;
    }
    item += npairs;
    open(p, npairs);
  }
};

// Bounded wait for an already issued copy or MMA after an abort.
__device__ __forceinline__ void drain_wait(uint64_t *bar, uint32_t parity, uint64_t limit_ns) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer_ns() - t0 > limit_ns) return;
}

// The sums of one thread (row r of the tile's half in this CTA, 128 columns
// from c0) written through the warp's staging block, so that a store
// instruction covers one row's 32 consecutive columns.
__device__ __forceinline__ void store_tile(const WgradParams &p, const WTile &t, int row0, int col0, const float (&acc)[128],
                                           float *patch) {
  const int lane = threadIdx.x & 31;
  const int64_t mat = static_cast<int64_t>(p.n_out) * p.n_in;
  const bool part = p.splits > 1;
  const int64_t base = (part ? static_cast<int64_t>(t.split) * p.groups * mat : 0) + t.e * mat;
  const size_t count = static_cast<size_t>(p.groups) * mat;
  const int rows = min(32, p.n_out - row0);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    __syncwarp();
    // row lane, column c at word (c ^ lane): no bank conflict either way
#pragma unroll
    for (int c = 0; c < 32; ++c) patch[lane * 32 + (c ^ lane)] = acc[32 * k + true_column(c)];
    __syncwarp();
    const int col = col0 + 32 * k + lane;
    if (col >= p.n_in) continue;
    for (int r = 0; r < rows; ++r) {
      const float v = patch[r * 32 + (lane ^ r)];
      const int64_t at = base + static_cast<int64_t>(row0 + r) * p.n_in + col;
      if (part) {
        if (in_bounds(p.parts + at, 4, p.parts, count * p.splits * 4, p.status)) p.parts[at] = v;
      } else if (p.gdtype == kF32) {
        float *g = static_cast<float *>(p.grad) + at;
        if (in_bounds(g, 4, p.grad, count * 4, p.status)) *g = p.accumulate ? *g + v : v;
      } else {
        __nv_bfloat16 *g = static_cast<__nv_bfloat16 *>(p.grad) + at;
        if (in_bounds(g, 2, p.grad, count * 2, p.status))
          *g = __float2bfloat16_rn(p.accumulate ? __bfloat162float(*g) + v : v);
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads, 1) ns_wgrad_kernel(const __grid_constant__ WgradParams p) {
  extern __shared__ uint8_t smem_raw[];
  // 1024-byte aligned, by an offset so that accesses stay in the shared window
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *sA = smem, *sB = smem + kStages * kShare;
  uint8_t *sQ = smem + 2 * kStages * kShare, *sS = sQ + kRawStages * kRaw;
  WgradBarriers *bar = reinterpret_cast<WgradBarriers *>(sS + kRawStages * kRawScales);
  float *patches = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(bar) + kBarBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x / 2, npairs = gridDim.x / 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bar->afull[s], 1);
      mbar_init(&bar->ready[s], 2 * (kConvWarps + 1));
      mbar_init(&bar->empty[s], 1);
    }
    for (int s = 0; s < kRawStages; ++s) {
      mbar_init(&bar->rawfull[s], 1 + 32);
      mbar_init(&bar->rawempty[s], kConvWarps);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&bar->tfull[a], 1);
      mbar_init(&bar->tempty[a], 2 * kSumWarps);
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

  if (warp < kConv0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (tmem_ok && warp == 0) {
      // -------------------------------------------------- dY by TMA
      if (lane == 0) {
        int stage = 0;
        uint32_t parity = 0;
        uint32_t issued = 0, last = 0;  // per stage: whether copies were issued, the parity of the last
        BlockWalk k;
        for (k.start(p, pair, npairs); !k.done; k.next(p, npairs)) {
          if (!mbar_wait<true, 40>(&bar->empty[stage], parity ^ 1u, w)) break;
          mbar_arrive_expect_tx(&bar->afull[stage], kShare);
          const int x = k.t.n0 + static_cast<int>(rank) * 128, y = k.t.lo + k.b * kBK;
          tma_box(sA + stage * kShare, &p.tm_dy, x, y, k.z, &bar->afull[stage]);
          tma_box(sA + stage * kShare + kBoxBytes, &p.tm_dy, x + 64, y, k.z, &bar->afull[stage]);
          issued |= 1u << stage;
          last = (last & ~(1u << stage)) | (parity << stage);
          if (++stage == kStages) {
            stage = 0;
            parity ^= 1u;
          }
        }
        if (*abort)
          for (int s = 0; s < kStages; ++s)
            if ((issued >> s) & 1u) drain_wait(&bar->afull[s], (last >> s) & 1u, w.limit_ns);
      }
    } else if (tmem_ok && warp == 2) {
      // -------------------------------------------------- X as it is held
      int raw = 0;
      uint32_t parity = 0;
      uint32_t issued = 0, last = 0;
      int end = 0;  // end marks published, one for each converter group
      BlockWalk k;
      k.start(p, pair, npairs);
      while (end < kConvGroups) {
        if (!warp_mbar_wait<false, 40>(&bar->rawempty[raw], parity ^ 1u, w)) break;
        if (k.done) {
          if (lane == 0) {
            bar->left[raw] = -1;
            mbar_arrive(&bar->rawfull[raw]);
          }
          mbar_arrive(&bar->rawfull[raw]);
          ++end;
        } else {
          const int col0 = k.t.k0 + static_cast<int>(rank) * 128, row0 = k.t.lo + k.b * kBK;
          if (lane == 0) {
            bar->left[raw] = k.t.hi - row0;
            mbar_arrive_expect_tx(&bar->rawfull[raw], kRaw);
            tma_bytes(sQ + raw * kRaw, &p.tm_q, col0, row0, &bar->rawfull[raw]);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = row0 + h * 32 + lane;
            const bool inside = row < k.t.hi && col0 / 32 < p.scale_pitch;
            copy4(sS + raw * kRawScales + 4 * (h * 32 + lane),
                  inside ? p.s + static_cast<int64_t>(row) * p.scale_pitch + col0 / 32 : p.s, inside);
          }
          arrive_after_copies(&bar->rawfull[raw]);
          issued |= 1u << raw;
          last = (last & ~(1u << raw)) | (parity << raw);
          k.next(p, npairs);
        }
        if (++raw == kRawStages) {
          raw = 0;
          parity ^= 1u;
        }
      }
      if (*abort)
        for (int s = 0; s < kRawStages; ++s)
          if ((issued >> s) & 1u) drain_wait(&bar->rawfull[s], (last >> s) & 1u, w.limit_ns);
    } else if (tmem_ok && warp == 3) {
      // -------------------------------------------------- dY landed
      if (lane == 0) {
        int stage = 0;
        uint32_t parity = 0;
        BlockWalk k;
        for (k.start(p, pair, npairs); !k.done; k.next(p, npairs)) {
          if (!mbar_wait<true, 20>(&bar->afull[stage], parity, w)) break;
          arrive_pair(mapa_shared(smem_u32(&bar->ready[stage]), 0));
          if (++stage == kStages) {
            stage = 0;
            parity ^= 1u;
          }
        }
      }
    } else if (tmem_ok && warp == 1 && leader) {
      // -------------------------------------------------- MMAs, issued by one lane
      if (lane == 0) {
        constexpr uint32_t idesc = umma_idesc_bf16(256, 256, 1, 1);
        const uint64_t desc_a = sw128_mnmajor_desc(smem_u32(sA)), desc_b = sw128_mnmajor_desc(smem_u32(sB));
        int stage = 0, acc = 0;
        uint32_t parity = 0, acc_parity = 0;
        bool ok = true;
        for (int item = pair; ok && item < p.items; item += npairs) {
          const int nb = wtile(p, item).blocks();
          for (int c = 0; ok && c < nb; c += kChunk) {
            if (!(ok = mbar_wait<true>(&bar->tempty[acc], acc_parity ^ 1u, w))) break;
            tc_fence_after();
            const uint32_t d = tmem + static_cast<uint32_t>(acc * 256);
            const int n = min(kChunk, nb - c) * p.slices;
            for (int i = 0; i < n; ++i) {
              if (!(ok = mbar_wait<true>(&bar->ready[stage], parity, w))) break;
              tc_fence_after();
              const uint64_t at = static_cast<uint64_t>(stage * (kShare >> 4));  // addresses are in 16-byte units
#pragma unroll
              for (int k = 0; k < kBK / 16; ++k)
                umma_bf16_pair(d, desc_a + at + k * 128u, desc_b + at + k * 128u, idesc, i > 0 || k > 0);
              umma_commit_pair_multicast(&bar->empty[stage], 3u);
              if (++stage == kStages) {
                stage = 0;
                parity ^= 1u;
              }
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
    }
  } else if (warp < kSum0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    if (tmem_ok) {
      // -------------------------------------------------- X to bf16
      const int group = (warp - kConv0) / kConvWarps, part = (warp - kConv0) % kConvWarps;
      const int j = lane & 7, row_in = part * 4 + (lane >> 3);
      // 16 values are two 16-byte pieces of a 64-column box row. Half of the
      // lanes take their second piece first: the 8 lanes that store one row
      // then cover all banks, and so do the 16 that read two rows. The
      // swizzle depends on the row modulo 8, the same for a lane's four rows.
      const int swap = ((j >> 2) ^ row_in) & 1;
      const int out0 = (j >> 2) * kBoxBytes + row_in * 128 + (((2 * (j & 3) + swap) ^ (row_in & 7)) << 4);
      const int out1 = out0 ^ 16, in = row_in * 128 + j * 16 + 8 * swap, in_scale = 4 * row_in + (j >> 1);
      int stage = group, raw = group;  // k-blocks group, group + kConvGroups, ...
      uint32_t parity = 0, raw_parity = 0;
      for (;;) {
        if (!warp_wait<false>(&bar->rawfull[raw], raw_parity, w)) break;
        const int left = bar->left[raw];
        if (left < 0) break;
        uint2 q0[4], q1[4];
        uint32_t sc[4];
        const uint8_t *src0 = sQ + raw * kRaw + in, *src1 = sQ + raw * kRaw + (in ^ 8);
        const uint8_t *scales = sS + raw * kRawScales + in_scale;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          q0[i] = *reinterpret_cast<const uint2 *>(src0 + i * 2048);
          q1[i] = *reinterpret_cast<const uint2 *>(src1 + i * 2048);
          sc[i] = scales[i * 64];
        }
        if (left < kBK) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i * 16 + row_in >= left) q0[i] = q1[i] = make_uint2(0, 0);  // and its scale is 0: the value is 0
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar->rawempty[raw]);
        if ((raw += kConvGroups) >= kRawStages) {
          raw -= kRawStages;
          raw_parity ^= 1u;
        }
        if (!warp_wait<true>(&bar->empty[stage], parity ^ 1u, w)) break;
        uint8_t *dst0 = sB + stage * kShare + out0, *dst1 = sB + stage * kShare + out1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 unit = unit_pair(sc[i]);
          uint4 a;
          widen4(q0[i].x, unit, a.x, a.y);
          widen4(q0[i].y, unit, a.z, a.w);
          *reinterpret_cast<uint4 *>(dst0 + i * 2048) = a;
          widen4(q1[i].x, unit, a.x, a.y);
          widen4(q1[i].y, unit, a.z, a.w);
          *reinterpret_cast<uint4 *>(dst1 + i * 2048) = a;
        }
        if (left < kBK) {  // clear dY beyond the group's end: 64 rows of 8 pieces in each box
          if (!warp_mbar_wait<true>(&bar->afull[stage], parity, w)) break;
          for (int i = part * 32 + lane; i < 2 * kBK * 8; i += 32 * kConvWarps) {
            const int r = (i >> 3) & (kBK - 1);
            if (r >= left)
              *reinterpret_cast<uint4 *>(sA + stage * kShare + (i >> 9) * kBoxBytes + r * 128 + (i & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) arrive_pair(mapa_shared(smem_u32(&bar->ready[stage]), 0));
        if ((stage += kConvGroups) >= kStages) {
          stage -= kStages;
          parity ^= 1u;
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
    if (tmem_ok) {
      // -------------------------------------------------- sums and the tile's store
      const int e = warp - kSum0, quarter = warp & 3, half = e >> 2;
      float *patch = patches + e * (kPatch / 4);
      int acc = 0;
      uint32_t acc_parity = 0;
      bool ok = true;
      for (int item = pair; ok && item < p.items; item += npairs) {
        const WTile t = wtile(p, item);
        const int nb = t.blocks();
        if (nb == 0 && p.accumulate && p.splits == 1) continue;
        float sum[128];
#pragma unroll
        for (int c = 0; c < 128; ++c) sum[c] = 0.f;
        for (int c = 0; c < nb; c += kChunk) {
          if (!warp_mbar_wait<true, 100>(&bar->tfull[acc], acc_parity, w)) {
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
          if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&bar->tempty[acc]), 0));
          if (++acc == 2) {
            acc = 0;
            acc_parity ^= 1u;
          }
        }
        if (!ok) break;
        const int row0 = t.n0 + static_cast<int>(rank) * 128 + quarter * 32;
        if (row0 < p.n_out) store_tile(p, t, row0, t.k0 + half * 128, sum, patch);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, kTmemCols);
}

// ------------------------------------------------------------------ around the product
struct SliceParams {
  const void *dy;
  __nv_bfloat16 *out;  // slices x rows x pitch
  int64_t ld;
  int rows, n_out, pitch, slices;
  int *status;
};

// dY as TMA can address it: bf16 rows of `pitch` elements (a multiple of 8),
// one slice, or three whose sum is the fp32 value to 2^-24 of it.
template <int DT>
__global__ void __launch_bounds__(256) ns_wgrad_slice_kernel(const __grid_constant__ SliceParams p) {
  using E = typename Elem<DT>::T;
  const int64_t slice = static_cast<int64_t>(p.rows) * p.pitch;
  const size_t size = static_cast<size_t>(slice) * p.slices * 2;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < slice; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t r = i / p.pitch;
    const int c = static_cast<int>(i - r * p.pitch);
    float v = c < p.n_out ? Elem<DT>::to_f(static_cast<const E *>(p.dy)[r * p.ld + c]) : 0.f;
    for (int z = 0; z < p.slices; ++z) {
      __nv_bfloat16 h = __float2bfloat16_rn(v);
      if (__hisinf(h) && !isinf(v))  // beyond bf16's largest value: that one, the rest in the next slice
        h = __ushort_as_bfloat16(static_cast<uint16_t>(__float_as_uint(v) >> 16));
      if (in_bounds(p.out + z * slice + i, 2, p.out, size, p.status)) p.out[z * slice + i] = h;
      const float f = __bfloat162float(h);
      v = isinf(f) || isnan(f) ? 0.f : v - f;  // an infinity or NaN stays in the first slice alone
    }
  }
}

// G (+)= the parts of a split contraction, added in order.
template <int GT>
__global__ void __launch_bounds__(256) ns_wgrad_join_kernel(const __grid_constant__ WgradParams p) {
  using G = typename Elem<GT>::T;
  const int64_t n = static_cast<int64_t>(p.groups) * p.n_out * p.n_in;
  G *g = static_cast<G *>(p.grad);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
    float v = p.parts[i];
    for (int s = 1; s < p.splits; ++s) v += p.parts[s * n + i];
    if (p.accumulate) v += Elem<GT>::to_f(g[i]);
    if (in_bounds(g + i, sizeof(G), g, static_cast<size_t>(n) * sizeof(G), p.status)) g[i] = Elem<GT>::from_f(v);
  }
}

int run_slice(const SliceParams &p, int dtype, int sms, cudaStream_t s) {
  const int64_t n = static_cast<int64_t>(p.rows) * p.pitch;
  const int grid = static_cast<int>(std::min<int64_t>((n + 255) / 256, static_cast<int64_t>(sms) * 16));
  if (dtype == NS_BF16)
    ns_wgrad_slice_kernel<kBF16><<<grid, 256, 0, s>>>(p);
  else
    ns_wgrad_slice_kernel<kF32><<<grid, 256, 0, s>>>(p);
  count_launch();
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

// CTA pairs that can be resident at once on this device (one CTA per SM).
int resident_pairs(int dev, int sms, cudaLaunchConfig_t &cfg) {
  static int cached[64] = {};
  int &n = cached[dev & 63];
  if (n == 0) {
    static SmemOptIn opt_in;
    if (opt_in.ensure(reinterpret_cast<const void *>(ns_wgrad_kernel), kSmem)) return 0;
    cfg.gridDim = dim3(sms / 2 * 2, 1, 1);
    if (cudaOccupancyMaxActiveClusters(&n, ns_wgrad_kernel, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = 0;
    }
  }
  return n;
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
  p.scale_pitch = static_cast<int>(ns_ckpt_scale_pitch(n_in));
  const Range rg(grad, static_cast<int64_t>(groups) * n_out, n_in, n_in, gelt);
  if (rg.overlaps(Range(dy, rows, n_out, ld_dy, elt)) || rg.overlaps(Range(q, rows, q_pitch, q_pitch, 1)) ||
      rg.overlaps(Range(scales, rows, p.scale_pitch, p.scale_pitch, 1)) ||
      rg.overlaps(Range(offsets, 1, groups + int64_t(1), groups + int64_t(1), 4)))
    return NS_EINVAL;
  OpCall call(stream);
  if (call.rc) return call.rc;
  WgradParams &k = p;
  k.s = static_cast<const uint8_t *>(scales);
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
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = call.s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int pairs = resident_pairs(call.dev, call.sms, cfg);
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

  // scratch: dY's slices (fp32, or bf16 that TMA cannot address), the parts of a split
  const bool direct = dtype == NS_BF16 && rows > 0 && !misaligned(dy, 16) && ld_dy % 8 == 0;
  const int64_t pitch = (n_out + 7) / 8 * 8;
  const size_t slice_bytes = direct ? 0 : (static_cast<size_t>(k.slices) * rows * pitch * 2 + 1023) / 1024 * 1024;
  const size_t part_bytes = k.splits > 1 ? static_cast<size_t>(k.splits) * groups * n_out * n_in * 4 : 0;
  uint8_t *ws = nullptr;
  int rc = NS_OK;
  if (slice_bytes + part_bytes && (rc = call.workspace(kSlotWgrad, slice_bytes + part_bytes, &ws))) return rc;
  k.parts = reinterpret_cast<float *>(ws + slice_bytes);
  const int64_t use = direct ? ld_dy : pitch;
  const int64_t dims[3] = {n_out, rows, k.slices}, strides[2] = {use * 2, use * 2 * std::max<int64_t>(rows, 1)};
  const int box[3] = {64, kBK, 1};
  // a map wants an address even when no row will be read through it
  const void *src = direct ? dy : slice_bytes ? ws : grad;
  if (rows > 0) {
    if ((rc = call.tensor_map(&k.tm_dy, 2, src, 3, dims, strides, box))) return rc;
    const int64_t qdims[2] = {n_in, rows}, qstride[1] = {q_pitch};
    const int qbox[2] = {128, kBK};
    if ((rc = call.tensor_map(&k.tm_q, 1, q, 2, qdims, qstride, qbox))) return rc;
  }
  if (!direct && rows > 0) {
    SliceParams sp{dy, reinterpret_cast<__nv_bfloat16 *>(ws), ld_dy, k.rows, k.n_out, static_cast<int>(pitch), k.slices, k.status};
    if ((rc = call.launch(kOpWgrad, [&] { return run_slice(sp, dtype, call.sms, call.s); }))) return rc;
  }
  cfg.gridDim = dim3(2 * static_cast<unsigned>(std::min<int64_t>(pairs, k.items)), 1, 1);
  rc = call.launch(kOpWgrad, [&] {
    if (cudaLaunchKernelEx(&cfg, ns_wgrad_kernel, k) != cudaSuccess) {
      cudaGetLastError();
      return -1;
    }
    count_launch();
    return 0;
  });
  if (rc || k.splits == 1) return rc;
  return call.launch(kOpWgrad, [&] { return run_join(k, call.sms, call.s); });
}
