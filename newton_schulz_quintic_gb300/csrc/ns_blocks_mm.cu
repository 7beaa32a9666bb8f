// ns_blocks_mm.cu -- products of matrices held in e4m3 with a scale for each
// block of 128 (include/ns.h): Out = A W^T over groups of rows, or A W.
//
// The scales are powers of two, which the tensor cores apply themselves
// (tcgen05.mma kind::mxf8f6f4.block_scale: one E8M0 scale per 32 values along the
// contraction and row, read from TMEM), so a block's scale is used by the four
// MMAs of its 128 values. Applying the scales in the registers instead, where
// each k-block's sums are drained from TMEM (256 x 256 tiles, kind::f8f6f4), took
// 392 us at 8192 x 8192 x 6144, against 227 us for the MMAs without their drains.
//
// W is the operand of M, the rows of A that of N: a tile is 256 columns of Out by
// TN rows, so a group's ragged rows cost what they are short of TN, W fits its
// 128-row boxes whichever way it lies (K-major for A W^T, MN-major for A W; the
// tensor cores read both), and a few rows of a decoding step run the same way
// with a small TN.
//
// One persistent kernel of CTA pairs (cta_group::2, M = 256, N = TN, K = 32). CTA
// rank r holds columns r*128.. of Out (rows of W's share) and rows r*TN/2.. of
// A's. Warps of a CTA:
//   0       TMA: 128 values of W and TN/2 of A, two k-blocks deep, into a ring of stages
//           (one a stage: the threads that hand stages on take about 500 cycles for each,
//           more than its MMAs)
//   1       TMEM (two accumulators, sets of scales); in the leader the MMAs
//   2       passes a landed stage on to the leader's MMAs (copies that count on the leader's
//           barrier themselves: 254 us at 8192 x 8192 x 6144 against 249)
//   3       looks the pair's tiles up (place, group, rows) a few ahead
//   4..7    scales: for four k-blocks at a time the 32-bit words as they lie in
//           memory, a byte a k-block, to TMEM (every warp to its own 32 lanes)
//   8..15   sums: every kChunk k-blocks the accumulator is added to fp32 registers
//           (32 columns of Out x TN/2 rows a warp) while the MMAs go on in the
//           other one. The tensor cores' own accumulation loses up to a unit in
//           the last place per instruction, over the 32 between two drains less
//           than 2^-17 of the sum of magnitudes at any depth. Measured, products of
//           one sign: 2^-21 at most; against 64 bits 1.2e-7 in the norm at a depth of 6144
//           (a plain product in fp32: 2.7e-7) and 1.3e-7 at 1024 (5.4e-8). Drains
//           every 4 k-blocks give 7.4e-8 and 6.5e-8 and cost 5 to 9 %.
// A tile leaves by plain stores: a lane holds one column of Out, a warp 32
// neighbours, so any pitch and alignment will do and rows are masked one by one.
//
// Where there are too few tiles for the pairs, the depth is split over the pairs
// of a cluster: each leaves its sums in its own shared memory, and every CTA adds
// and stores a share of the rows, in order.
//
// Bound by the tensor pipe: 8192 rows, W of 8192 x 6144 in 242 to 254 us, 3.3 PFLOP/s (its input's gradient 260 to 280);
// 76 experts of 2048 x 6144 over 38912 rows in 342 to 381 us, where a group's last tile is on average half full. Few rows:
// 7 of them with W of 8192 x 6144 in 16 us, twice the time of W's bytes; one row for each of 56 experts among 76 of 2048 x
// 6144 in 104 us, the time of those experts' bytes.
//
// Every wait is bounded (mbar_wait): on a timeout the status word is set, the
// CTA waits for its own copies and MMAs, frees TMEM and exits.
#include <algorithm>
#include <cmath>

#include "../../include/ns.h"
#include "ns_rows.cuh"

namespace ns {

namespace {

constexpr int kBK = 128;                         // depth of a k-block: one scale
constexpr int kChunk = 8;                        // k-blocks between two drains of an accumulator
constexpr int kIssueWarps = 4, kScaleWarps = 4, kSumWarps = 8;
constexpr int kThreads = 32 * (kIssueWarps + kScaleWarps + kSumWarps);
// Registers a thread after the warpgroups have divided what the launch holds (128 each).
constexpr int kOtherRegs = 80, kSumRegs = 168;
constexpr int kTmemCols = 512;
constexpr int kScaleCols = 12;                   // of a set: 4 for W's 128 rows, 8 for up to 256 rows of A
constexpr int kMaxGroups = 1 << 20;
constexpr int kMaxSplits = 4;  // a cluster of 8

template <int TN>
struct Shape {
  static constexpr int kW = 128 * kBK, kA = TN / 2 * kBK;  // bytes of a CTA's operands in a k-block
  static constexpr int kStageBytes = 2 * (kW + kA);
  static constexpr int kStages = 224 * 1024 / kStageBytes;
  static constexpr int kScaleAt = 2 * TN;                  // columns of TMEM behind the accumulators
  // A set of scales is used again once its MMAs are done and the scale warps of both CTAs have been told, have written
  // and have told the leader: with two sets that took longer than the four k-blocks of the other (337 us at 8192 x 8192 x
  // 6144 against 328 with eight; both before the arrival below was relaxed).
  static constexpr int kSets = (kTmemCols - kScaleAt) / kScaleCols < 8 ? (kTmemCols - kScaleAt) / kScaleCols : 8;
  static_assert(kStages * kStageBytes >= TN * 128 * 4, "a tile's sums fit the ring");
};

struct BmmParams {
  CUtensorMap tm_a;        // {K, rows}, box {128, TN / 2}
  CUtensorMap tm_w;        // {columns, rows of one matrix, groups}, box {128, 128, 1}
  const uint8_t *sa, *sw;  // scales
  const int32_t *offsets;  // nullptr: one group of all rows
  void *out;
  int64_t ld_out;
  int rows, n, groups;
  int sa_pitch, sw_pitch;
  int sw_rows;             // rows of scales of one matrix of W
  int nb;                  // k-blocks
  int tn;                  // tiles along Out's columns
  int splits;              // pairs that share a tile's depth
  int odtype;
  int *status;
  uint64_t wait_limit_ns;
};

// One tile of the pair's list as warp 3 hands it out.
struct alignas(16) MTile {
  int m0, n0;  // its first row and column of Out
  int hi;      // rows of its group end here; < 0: no more tiles
  int e;       // its group; < 0: rows of no group, all zeros
  int b0, b1;  // its k-blocks; b0 is a multiple of 4
  int pad[2];
};
constexpr int kQueue = 4;

template <int STAGES, int SETS>
struct BmmBarriers {
  MTile queue[kQueue];
  uint64_t qfull[kQueue];    // a slot holds the next tile
  uint64_t qempty[kQueue];   // every consumer of this CTA has read it
  uint64_t full[STAGES];     // this CTA's boxes of a stage landed
  uint64_t ready[STAGES];    // leader: both CTAs' operands of a stage are in place
  uint64_t empty[STAGES];    // each CTA: the MMAs are done with a stage
  uint64_t sfull[SETS];      // leader: both CTAs' scales of four k-blocks are in place
  uint64_t sempty[SETS];     // each CTA: the MMAs are done with them
  uint64_t tfull[2];         // each CTA: an accumulator holds a chunk
  uint64_t tempty[2];        // leader: both CTAs have drained an accumulator
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};
template <int TN>
constexpr int smem_of() {
  return 1024 + Shape<TN>::kStages * Shape<TN>::kStageBytes + static_cast<int>(sizeof(BmmBarriers<Shape<TN>::kStages, Shape<TN>::kSets>)) + 64;
}

template <typename B>
struct MTileReader {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void step() {
    if (++slot == kQueue) {
      slot = 0;
      parity ^= 1u;
    }
  }
  __device__ __forceinline__ bool take(B *bar, MTile &t, const Waiter &w) {
    if (!mbar_wait(&bar->qfull[slot], parity, w)) return false;
    t = bar->queue[slot];
    mbar_arrive(&bar->qempty[slot]);
    step();
    return t.hi >= 0;
  }
  __device__ __forceinline__ bool take_warp(B *bar, MTile &t, const Waiter &w) {
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

// The tiles in order, found by a whole warp that walks over the parts 32 at a time.
template <int TN>
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
    incl = static_cast<int64_t>((hi - lo + TN - 1) / TN) * p.tn;
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
        const int tm = (end - first + TN - 1) / TN, band = tile / (8 * p.tn), row = band * 8;
        const int height = min(8, tm - row), rest = tile - band * 8 * p.tn;
        t.m0 = first + (row + rest % height) * TN;
        t.n0 = rest / height * 256;
        t.hi = end;
        t.e = e0 + l < p.groups ? e0 + l : -1;
        t.b0 = 0;
        t.b1 = t.e < 0 ? 0 : p.nb;
        return true;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
      e0 += 32;
      if (e0 >= parts) return false;
      load(p);
    }
  }
};

// Instruction descriptor of kind::mxf8f6f4: A and B e4m3, scales E8M0; a_mn selects an MN-major A operand. The byte of
// the scales' words that an MMA uses is added by scale_byte_of.
__host__ __device__ constexpr uint32_t idesc_mx(int M, int N, int a_mn) {
  return (0u << 7) | (0u << 10)                       // A and B format: e4m3
         | (static_cast<uint32_t>(a_mn & 1) << 15)    // A major-ness (B is K-major)
         | (static_cast<uint32_t>(N >> 3) << 17)
         | (1u << 23)                                 // scales: E8M0
         | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t scale_byte_of(int i) {
  return static_cast<uint32_t>(i) << 29 | static_cast<uint32_t>(i) << 4;  // A's, B's
}

// Operands of 128-byte rows written by TMA with the 128-byte swizzle, in the shared-memory descriptor of
// sw128_kmajor_desc. K-major: a row is one M or N index, a step of 32 along K is 32 bytes. MN-major: a row is one K index
// and holds 128 M indices, a step of 32 along K is 32 rows; there is one such chunk, so the leading offset is not used.
__device__ __forceinline__ void umma_mx_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t sf_a, uint32_t sf_b, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sf_a), "r"(sf_b), "r"(accumulate)
      : "memory");
}

// 32 lanes x 4 columns of words to TMEM (this warp's lanes); complete after tmem_st_wait.
__device__ __forceinline__ void tmem_st4(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 lanes x 8 columns of TMEM words, complete on return.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}

// The sums of one thread: one column of Out, N rows.
template <int N>
struct Sums {
  float2 v[N / 2];
  __device__ __forceinline__ float operator[](int c) const { return c & 1 ? v[c / 2].y : v[c / 2].x; }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int c = 0; c < N / 2; ++c) v[c] = make_float2(0.f, 0.f);
  }
  template <int M>
  __device__ __forceinline__ void add(int c, const uint32_t (&x)[M]) {
#pragma unroll
    for (int u = 0; u < M / 2; ++u)
      v[c / 2 + u] = __fadd2_rn(v[c / 2 + u], make_float2(__uint_as_float(x[2 * u]), __uint_as_float(x[2 * u + 1])));
  }
  // an accumulator's N columns from `src` on
  __device__ __forceinline__ void drain(uint32_t src) {
    if constexpr (N % 16 == 0) {
#pragma unroll
      for (int k = 0; k < N / 16; ++k) {
        uint32_t x[16];
        tmem_ld16(src + 16 * k, x);
        add(16 * k, x);
      }
    } else {
#pragma unroll
      for (int k = 0; k < N / 8; ++k) {
        uint32_t x[8];
        tmem_ld8(src + 8 * k, x);
        add(8 * k, x);
      }
    }
  }
};

__device__ __forceinline__ void put_one(const BmmParams &p, int64_t row, int col, float v, size_t size) {
  if (p.odtype == kBF16) {
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + row * p.ld_out + col;
    if (in_bounds(o, 2, p.out, size, p.status)) *o = __float2bfloat16_rn(v);
  } else {
    float *o = static_cast<float *>(p.out) + row * p.ld_out + col;
    if (in_bounds(o, 4, p.out, size, p.status)) *o = v;
  }
}
__device__ __forceinline__ size_t out_bytes(const BmmParams &p) {
  return static_cast<size_t>((p.rows - 1) * p.ld_out + p.n) * (p.odtype == kBF16 ? 2 : 4);
}

// Column `col` of Out, rows row0.. below hi.
template <int OT, int N>
__device__ __forceinline__ void put_column(const BmmParams &p, int row0, int hi, int col, const Sums<N> &sum, size_t size) {
  using O = typename Elem<OT>::T;
  O *to = static_cast<O *>(p.out) + static_cast<int64_t>(row0) * p.ld_out + col;
  if (row0 + N <= hi) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (in_bounds(to + j * p.ld_out, sizeof(O), p.out, size, p.status)) to[j * p.ld_out] = Elem<OT>::from_f(sum[j]);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (row0 + j < hi && in_bounds(to + j * p.ld_out, sizeof(O), p.out, size, p.status)) to[j * p.ld_out] = Elem<OT>::from_f(sum[j]);
  }
}

template <bool kBack, int TN>
__global__ void __launch_bounds__(kThreads, 1) ns_blocks_mm_kernel(const __grid_constant__ BmmParams p) {
  using S = Shape<TN>;
  using Bar = BmmBarriers<S::kStages, S::kSets>;
  constexpr int kStages = S::kStages, kRing = kStages * S::kStageBytes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *sW = smem, *sA = smem + kStages * 2 * S::kW;
  Bar *bar = reinterpret_cast<Bar *>(smem + kRing);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank(), rank = crank & 1u, lead = crank & ~1u;  // the pair's leader in the cluster
  const int split = static_cast<int>(crank >> 1);
  const bool leader = rank == 0;
  const int width = 2 * p.splits;  // CTAs of a cluster
  const int cluster = blockIdx.x / width, nclusters = gridDim.x / width;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bar->full[s], 1);
      mbar_init(&bar->ready[s], 2);
      mbar_init(&bar->empty[s], 1);
    }
    for (int a = 0; a < S::kSets; ++a) {
      mbar_init(&bar->sfull[a], 2 * kScaleWarps);
      mbar_init(&bar->sempty[a], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&bar->tfull[a], 1);
      mbar_init(&bar->tempty[a], 2 * kSumWarps);
    }
    for (int q = 0; q < kQueue; ++q) {
      mbar_init(&bar->qfull[q], 1);
      mbar_init(&bar->qempty[q], 2 + kScaleWarps + kSumWarps + (leader ? 1 : 0));
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
  asm volatile("griddepcontrol.wait;" ::: "memory");  // what is above ran beside the end of the launch before
  const bool tmem_ok = ld_shared_cluster_u32(mapa_shared(smem_u32(&bar->tmem_base), crank ^ 1u)) == tmem;
  if (!tmem_ok && threadIdx.x == 0) set_status(p.status, kStatusTmemMismatch);
  volatile int *abort = &bar->abort;
  const Waiter w{abort, p.status, p.wait_limit_ns};
  const uint16_t both = static_cast<uint16_t>(3u << lead);

  MTile done;  // a split tile, whose sums are joined at the end
  done.hi = -1;
  if (warp < kIssueWarps + kScaleWarps)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
  if (tmem_ok && warp == 0) {
    // ---------------------------------------------------- operands by TMA, issued by one lane
    if (elect_one()) {
      int stage = 0;
      uint32_t parity = 0;
      uint32_t issued = 0, last = 0;  // per stage: whether copies were issued, the parity of the last
      const int r = static_cast<int>(rank);
      MTileReader<Bar> tiles;
      MTile t;
      bool ok = true;
      while (ok && tiles.take(bar, t, w)) {
        const int w0 = t.n0 + r * 128, a0 = t.m0 + r * (TN / 2);
        for (int b = t.b0; b < t.b1; b += 2) {
          if (!(ok = mbar_wait<true>(&bar->empty[stage], parity ^ 1u, w))) break;
          const bool two = b + 1 < t.b1;
          mbar_arrive_expect_tx(&bar->full[stage], two ? S::kStageBytes : S::kStageBytes / 2);
          uint8_t *dw = sW + stage * (2 * S::kW), *da = sA + stage * (2 * S::kA);
          tma_load_3d(dw, &p.tm_w, kBack ? w0 : b * kBK, kBack ? b * kBK : w0, t.e, &bar->full[stage]);
          tma_load_2d(da, &p.tm_a, b * kBK, a0, &bar->full[stage]);
          if (two) {
            tma_load_3d(dw + S::kW, &p.tm_w, kBack ? w0 : (b + 1) * kBK, kBack ? (b + 1) * kBK : w0, t.e, &bar->full[stage]);
            tma_load_2d(da + S::kA, &p.tm_a, (b + 1) * kBK, a0, &bar->full[stage]);
          }
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
      constexpr uint32_t idesc = idesc_mx(256, TN, kBack ? 1 : 0);
      constexpr uint64_t kStepW = kBack ? 32 * 128 / 16 : 32 / 16;  // 32 along K, in 16-byte units
      const uint64_t desc_w = sw128_kmajor_desc(smem_u32(sW)), desc_a = sw128_kmajor_desc(smem_u32(sA));
      int stage = 0, acc = 0, set = 0;
      uint32_t parity = 0, acc_parity = 0, set_parity = 0;
      bool ok = true, seen = false;  // seen: the next stage is known to be ready
      MTileReader<Bar> tiles;
      MTile t;
      while (ok && tiles.take(bar, t, w)) {
        const int n = t.b1 - t.b0;
        for (int i = 0; i < n; i += 2) {
          if (i % kChunk == 0 && !(ok = mbar_wait<true>(&bar->tempty[acc], acc_parity ^ 1u, w))) break;
          if (i % 4 == 0 && !(ok = mbar_wait<true>(&bar->sfull[set], set_parity, w))) break;
          if (!seen && !(ok = mbar_wait<true>(&bar->ready[stage], parity, w))) break;
          tc_fence_after();
          const uint32_t d = tmem + static_cast<uint32_t>(acc * TN);
          const uint32_t sfw = tmem + static_cast<uint32_t>(S::kScaleAt + set * kScaleCols), sfa = sfw + 4u;
          uint32_t id = idesc | scale_byte_of(i % 4);
          uint64_t dw = desc_w + static_cast<uint64_t>(stage * (2 * S::kW >> 4));
          uint64_t da = desc_a + static_cast<uint64_t>(stage * (2 * S::kA >> 4));
          uint64_t *const empty = &bar->empty[stage];
          if (++stage == kStages) {
            stage = 0;
            parity ^= 1u;
          }
          umma_mx_pair(d, dw, da, id, sfw, sfa, i % kChunk != 0);
          umma_mx_pair(d, dw + kStepW, da + 2u, id, sfw, sfa, 1);
          umma_mx_pair(d, dw + 2 * kStepW, da + 4u, id, sfw, sfa, 1);
          umma_mx_pair(d, dw + 3 * kStepW, da + 6u, id, sfw, sfa, 1);
          // look at the next stage while these run, so that its first MMA follows the last one here at once
          seen = mbar_try_wait_cluster(&bar->ready[stage], parity);
          if (i + 1 < n) {
            id += scale_byte_of(1);
            dw += S::kW >> 4;
            da += S::kA >> 4;
            umma_mx_pair(d, dw, da, id, sfw, sfa, 1);
            umma_mx_pair(d, dw + kStepW, da + 2u, id, sfw, sfa, 1);
            umma_mx_pair(d, dw + 2 * kStepW, da + 4u, id, sfw, sfa, 1);
            umma_mx_pair(d, dw + 3 * kStepW, da + 6u, id, sfw, sfa, 1);
          }
          umma_commit_pair_multicast(empty, both);
          const bool last = i + 2 >= n;
          if (i % 4 == 2 || last) {
            umma_commit_pair_multicast(&bar->sempty[set], both);
            if (++set == S::kSets) {
              set = 0;
              set_parity ^= 1u;
            }
          }
          if (i % kChunk == kChunk - 2 || last) {
            umma_commit_pair_multicast(&bar->tfull[acc], both);
            if (++acc == 2) {
              acc = 0;
              acc_parity ^= 1u;
            }
          }
        }
      }
      umma_commit_pair_multicast(&bar->drain, static_cast<uint16_t>(1u << lead));
      drain_wait(&bar->drain, 0, w.limit_ns);
    }
  } else if (tmem_ok && warp == 2) {
    // ---------------------------------------------------- landed stages
    if (elect_one()) {
      int stage = 0;
      uint32_t parity = 0;
      MTileReader<Bar> tiles;
      MTile t;
      bool ok = true;
      while (ok && tiles.take(bar, t, w)) {
        for (int b = t.b0; b < t.b1; b += 2) {
          if (!(ok = mbar_wait(&bar->full[stage], parity, w))) break;
          arrive_pair_shared(mapa_shared(smem_u32(&bar->ready[stage]), lead));
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
    TileWalk<TN> walk;
    walk.start(p);
    for (int64_t item = cluster; more; item += nclusters) {
      MTile t;
      more = walk.find(p, item, t);
      if (!more) t.hi = -1;
      if (more && p.splits > 1) {  // whole sets of scales per part
        const int sets = (t.b1 - t.b0 + 3) / 4;
        t.b0 = min(t.b1, sets * split / p.splits * 4);
        t.b1 = min(t.b1, sets * (split + 1) / p.splits * 4);
      }
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
  } else if (tmem_ok && warp >= kIssueWarps && warp < kIssueWarps + kScaleWarps) {
    // ---------------------------------------------------- scales
    constexpr int kAhead = 4, kWords = (TN + 31) / 32;  // of a lane: rows lane, lane + 32, ... of A's
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int set = 0;
    uint32_t set_parity = 0;
    bool ok = true;
    MTileReader<Bar> tiles;
    MTile t;
    while (ok && tiles.take_warp(bar, t, w)) {
      const uint8_t *sw = p.sw + static_cast<int64_t>(max(t.e, 0)) * p.sw_rows * p.sw_pitch;
      const int nblock = min(t.n0 / 128 + static_cast<int>(rank), (p.n - 1) / 128);
      // The words of kAhead sets are read at once: one set at a time, with the next one's words under way, a set took as
      // long as a read from L2, 1 us or five k-blocks.
      for (int b = t.b0; ok && b < t.b1; b += 4 * kAhead) {
        uint32_t ww[kAhead], wa[kAhead][kWords];
#pragma unroll
        for (int s = 0; s < kAhead; ++s) {
          const int k = b + 4 * s;
          ww[s] = 0;
          if (k < t.b1) {
            if (kBack) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (k + j < t.b1) ww[s] |= static_cast<uint32_t>(__ldg(sw + static_cast<int64_t>(k + j) * p.sw_pitch + nblock)) << (8 * j);
            } else {
              ww[s] = __ldg(reinterpret_cast<const uint32_t *>(sw + static_cast<int64_t>(nblock) * p.sw_pitch + k));
            }
          }
#pragma unroll
          for (int j = 0; j < kWords; ++j)
            wa[s][j] = k < t.b1 ? __ldg(reinterpret_cast<const uint32_t *>(
                                      p.sa + static_cast<int64_t>(min(t.m0 + j * 32 + lane, p.rows - 1)) * p.sa_pitch + k))
                                : 0u;
        }
#pragma unroll
        for (int s = 0; s < kAhead; ++s) {
          if (!ok || b + 4 * s >= t.b1) continue;
          if (!warp_mbar_wait<true>(&bar->sempty[set], set_parity ^ 1u, w)) {
            ok = false;
            continue;
          }
          __syncwarp();
          tc_fence_after();
          const uint32_t at = tmem + lanes + static_cast<uint32_t>(S::kScaleAt + set * kScaleCols);
          auto word = [&](int j) { return j < kWords ? wa[s][j < kWords ? j : 0] : 0u; };
          tmem_st4(at, ww[s], ww[s], ww[s], ww[s]);
          tmem_st4(at + 4, word(0), word(1), word(2), word(3));
          if (kWords > 4) tmem_st4(at + 8, word(4), word(5), word(6), word(7));
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          // (a release at cluster scope took 1400 cycles here)
          if (lane == 0) arrive_pair(mapa_shared(smem_u32(&bar->sfull[set]), lead));
          if (++set == S::kSets) {
            set = 0;
            set_parity ^= 1u;
          }
        }
      }
    }
  } else if (tmem_ok && warp >= kIssueWarps + kScaleWarps) {
    // ---------------------------------------------------- sums and the tile's store
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
    const int quarter = warp & 3, half = (warp - kIssueWarps - kScaleWarps) >> 2;
    const size_t size = out_bytes(p);
    int acc = 0;
    uint32_t acc_parity = 0;
    bool ok = true;
    MTileReader<Bar> tiles;
    MTile t;
    while (ok && tiles.take_warp(bar, t, w)) {
      Sums<TN / 2> sum;
      sum.clear();
      for (int i = 0; i < t.b1 - t.b0; i += kChunk) {
        if (!warp_mbar_wait<true>(&bar->tfull[acc], acc_parity, w)) {
          ok = false;
          break;
        }
        __syncwarp();
        tc_fence_after();
        sum.drain(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * TN + half * (TN / 2)));
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_pair(mapa_shared(smem_u32(&bar->tempty[acc]), lead));
        if (++acc == 2) {
          acc = 0;
          acc_parity ^= 1u;
        }
      }
      if (!ok) break;
      if (p.splits > 1) {  // one tile a cluster: its MMAs are done, so the ring is free and takes the sums, [row][column]
        float *mine = reinterpret_cast<float *>(smem) + half * (TN / 2) * 128 + quarter * 32 + lane;
#pragma unroll
        for (int j = 0; j < TN / 2; ++j) mine[j * 128] = sum[j];
        done = t;
        continue;
      }
      const int col = t.n0 + static_cast<int>(rank) * 128 + quarter * 32 + lane, row0 = t.m0 + half * (TN / 2);
      if (col >= p.n || row0 >= t.hi) continue;
      if (p.odtype == kBF16)
        put_column<kBF16, TN / 2>(p, row0, t.hi, col, sum, size);
      else
        put_column<kF32, TN / 2>(p, row0, t.hi, col, sum, size);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (p.splits > 1) {
    // every CTA adds a share of the rows of its 128 columns, the parts in order
    constexpr int kFirst = (kIssueWarps + kScaleWarps) * 32;
    const float *mine = reinterpret_cast<const float *>(smem);
    if (threadIdx.x >= kFirst && done.hi >= 0 && !*abort) {
      const int thread = threadIdx.x - kFirst, c = thread & 127, col = done.n0 + static_cast<int>(rank) * 128 + c;
      const int j0 = TN * split / p.splits, j1 = min(TN * (split + 1) / p.splits, done.hi - done.m0);
      const size_t size = out_bytes(p);
      if (col < p.n)
        for (int j = j0 + (thread >> 7); j < j1; j += 2) {
          float s = 0.f;
          for (int k = 0; k < p.splits; ++k)
            s += __uint_as_float(ld_shared_cluster_u32(mapa_shared(smem_u32(mine + j * 128 + c), static_cast<uint32_t>(2 * k) + rank)));
          put_one(p, done.m0 + j, col, s, size);
        }
    }
    cluster_sync();
  }
  if (warp == 1) tmem_dealloc_pair(tmem, kTmemCols);
}

// Clusters of 2 * splits CTAs that can be resident at once on this device (one CTA per SM).
template <bool kBack, int TN>
int resident_clusters(int dev, int sms, int splits) {
  static int cached[64][kMaxSplits + 1] = {};
  int &n = cached[dev & 63][splits];
  if (n == 0) {
    static SmemOptIn opt_in;
    if (opt_in.ensure(reinterpret_cast<const void *>(ns_blocks_mm_kernel<kBack, TN>), smem_of<TN>())) return 0;
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, ns_blocks_mm_kernel<kBack, TN>) != cudaSuccess ||
        attr.numRegs * kThreads < 256 * (kOtherRegs + kSumRegs)) {  // a share beyond it would never be granted
      cudaGetLastError();
      return 0;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = static_cast<unsigned>(2 * splits);
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    cfg.dynamicSmemBytes = smem_of<TN>();
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.gridDim = dim3(sms / (2 * splits) * (2 * splits), 1, 1);
    if (cudaOccupancyMaxActiveClusters(&n, ns_blocks_mm_kernel<kBack, TN>, &cfg) != cudaSuccess || n <= 0) {
      cudaGetLastError();
      n = 0;
    }
  }
  return n;
}

// Tiles of a call at most: each group may end inside one, and so may the rows before and behind them.
int64_t most_tiles(const BmmParams &p, int tn) {
  const int64_t parts = p.offsets ? p.groups + int64_t(2) : 1;
  return std::min<int64_t>(p.rows, p.rows / tn + parts) * p.tn;
}

template <bool kBack, int TN>
int run_mm(BmmParams &p, const void *qa, int64_t k, int64_t pa, int splits, OpCall &call) {
  const int n = resident_clusters<kBack, TN>(call.dev, call.sms, splits);
  if (n <= 0) return NS_ECUDA;
  const int box[2] = {128, TN / 2};
  const int64_t dims[2] = {k, p.rows}, stride[1] = {pa};
  if (p.nb > 0)
    if (const int rc = call.tensor_map(&p.tm_a, 1, qa, 2, dims, stride, box)) return rc;
  p.splits = splits;
  const int64_t tiles = std::max<int64_t>(1, most_tiles(p, TN));
  const int64_t clusters = splits > 1 ? tiles : std::min<int64_t>(n, tiles);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(2 * splits);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.dynamicSmemBytes = smem_of<TN>();
  cfg.stream = call.s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.gridDim = dim3(static_cast<unsigned>(2 * splits * clusters), 1, 1);
  return call.launch(kOpBlocksMatmul, [&] {
    if (cudaLaunchKernelEx(&cfg, ns_blocks_mm_kernel<kBack, TN>, p) != cudaSuccess) {
      cudaGetLastError();
      return -1;
    }
    count_launch();
    return 0;
  });
}

// Rows of a tile and pairs that share a tile's depth. A k-block takes a pair about 150 + 0.35 TN ns (few rows: W's 32 KB
// from L2; many: the MMAs), so TN is the one with the least of that times the rounds of tiles. Measured for W of 8192 x
// 6144, TN = 16 / 64 / 128 / 192: 7 rows 14.7 / - / - / -, 128 rows 32.6 / 16.5 / 18.5 / 19.9 us, 512 rows 98.9 / 35.7 /
// 26.5 / 30.0, 2048 rows - / 107 / 73 / 68. The depth is split in four where that still leaves every tile's parts room at
// once: W of 2048 x 6144, 7 rows: 10.2 us against 13.6, 64 rows 10.8 against 12.8; but 4096 x 4096 (16 tiles), two or
// three parts: 9.9 and 9.6 against 10.3.
template <bool kBack>
int choose_mm(BmmParams &p, const void *qa, int64_t k, int64_t pa, OpCall &call) {
  const int64_t pairs = call.sms / 2;
  int tn = 0;
  double best = 0;
  for (int t : {16, 32, 64, 128, 192}) {
    const double in_group = static_cast<double>(p.rows) / std::max(1, p.groups);
    const double tiles = std::max(1., p.offsets ? in_group / t + 0.5 : std::ceil(in_group / t)) * std::max(1, p.groups) * p.tn;
    const double cost = std::max(1., p.offsets ? tiles / pairs : std::ceil(tiles / pairs)) * (150 + 0.35 * t);
    if (tn == 0 || cost < best) {
      tn = t;
      best = cost;
    }
  }
  const int splits = p.nb >= 32 && most_tiles(p, tn) * kMaxSplits <= pairs ? kMaxSplits : 1;
  switch (tn) {
    case 16: return run_mm<kBack, 16>(p, qa, k, pa, splits, call);
    case 32: return run_mm<kBack, 32>(p, qa, k, pa, splits, call);
    case 64: return run_mm<kBack, 64>(p, qa, k, pa, splits, call);
    case 128: return run_mm<kBack, 128>(p, qa, k, pa, splits, call);
    default: return run_mm<kBack, 192>(p, qa, k, pa, splits, call);
  }
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
  p.groups = groups;
  p.sa_pitch = static_cast<int>(spa);
  p.sw_pitch = static_cast<int>(spw);
  p.sw_rows = static_cast<int>(sw_rows);
  p.nb = groups > 0 ? static_cast<int>((k + kBK - 1) / kBK) : 0;
  p.tn = static_cast<int>((n + 255) / 256);
  p.odtype = dtype;
  p.status = call.status;
  p.wait_limit_ns = kWaitLimitNs;
  if (p.nb > 0) {
    const int box[3] = {128, 128, 1};
    const int64_t wdims[3] = {w_cols, w_rows, groups}, wstride[2] = {pw, pw * w_rows};
    if (const int rc = call.tensor_map(&p.tm_w, 1, qw, 3, wdims, wstride, box)) return rc;
  }
  return back ? choose_mm<true>(p, qa, k, pa, call) : choose_mm<false>(p, qa, k, pa, call);
}
