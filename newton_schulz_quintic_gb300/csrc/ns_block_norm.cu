// ns_block_norm.cu -- the norms after and before a block, fused with the
// block's gate and the residual scale (include/ns.h), and their backward pass.
//
//     u = y * rsqrt(mean y^2 + eps) * post,  r = a x + b g u,  z = r * rsqrt(mean r^2 + eps) * pre
//
// Bound by HBM: forward reads x and y and writes r and z, backward reads the
// two gradients, x and y and writes two gradients (r is formed again, in fp32,
// from the kept 1 / rms of y). A row is held in the registers of its threads
// between the sums over it. So that memory stays busy while threads wait for
// one another at those sums, rows come through a ring in shared memory that a
// warp of its own keeps full: by bulk copies where rows are 16-byte aligned,
// else by four warps, element by element. (With reads straight into registers,
// rows of 8192 bf16 took 268 us forward and 603 back at 16384 rows.)
// The weights' gradients are sums over rows: a CTA walks over rows and adds in
// fp32, each thread its own columns, and a second launch adds the CTAs' parts in
// order.
#include <algorithm>
#include <cmath>

#include "../../include/ns.h"
#include "ns_rows.cuh"

namespace ns {

namespace {

enum Gate : int { kGateNone, kGateCols, kGateRows, kGateFull };
constexpr int kMaxCols = 16384;
constexpr int kMaxParts = 304;  // CTAs of a backward call: what the scratch holds

struct NormParams {
  const void *x, *y, *gate, *post, *pre;
  void *r, *z;              // forward
  float *post_rstd, *pre_rstd;
  const void *dr, *dz;      // backward
  void *dx, *dy, *dgate;
  float *parts;             // CTAs x 2 x cols: sums of dz * rh, and of the gate's (none, cols: drt * yh; else: g * drt * yh)
  int64_t ld_x, ld_y, ld_gate, ld_r, ld_z, ld_dr, ld_dz, ld_dx, ld_dy, ld_dgate;
  int64_t rows;
  int cols, gate_form, gate_type, weight_type;
  float a, b, eps;
  int *status;
  uint64_t wait_limit_ns;
};

// Value e of 8 that a thread holds from column c on: consecutive where rows allow packs (WIDE), else every 32nd.
template <bool WIDE>
__device__ __forceinline__ int col_of(int c, int e) { return WIDE ? c + e : c + 32 * e; }

template <int DT, bool WIDE>
__device__ __forceinline__ void load8(const void *row, int c, int cols, Pack<DT, 8> &v) {
  using E = typename Elem<DT>::T;
  const E *p = static_cast<const E *>(row);
  if constexpr (WIDE) {
    if (c < cols) {
      v.load(p + c);
      return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v.set(e, 0.f);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) reinterpret_cast<E *>(v.w)[e] = c + 32 * e < cols ? p[c + 32 * e] : Elem<DT>::from_f(0.f);
  }
}
template <int DT, bool WIDE>
__device__ __forceinline__ void store8(void *row, int c, int cols, const float (&f)[8], const void *base, size_t size, int *status) {
  using E = typename Elem<DT>::T;
  E *p = static_cast<E *>(row);
  Pack<DT, 8> v;
#pragma unroll
  for (int e = 0; e < 8; ++e) v.set(e, f[e]);
  if constexpr (WIDE) {
    if (c < cols) v.store_stream(p + c, base, size, status);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + 32 * e < cols && in_bounds(p + c + 32 * e, sizeof(E), base, size, status)) __stcs(p + c + 32 * e, reinterpret_cast<const E *>(v.w)[e]);
  }
}
// 8 values of either type as floats; 1 where there are none
template <bool WIDE>
__device__ __forceinline__ void load_any(const void *row, int type, int c, int cols, float (&f)[8]) {
  if (!row) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 1.f;
  } else if (type == kBF16) {
    Pack<kBF16, 8> v;
    load8<kBF16, WIDE>(row, c, cols, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = v.get(e);
  } else {
    Pack<kF32, 8> v;
    load8<kF32, WIDE>(row, c, cols, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = v.get(e);
  }
}
__device__ __forceinline__ const void *at_row(const void *p, int64_t row, int64_t ld, int type) {
  return static_cast<const uint8_t *>(p) + row * ld * (type == kBF16 ? 2 : 4);
}
__device__ __forceinline__ float one_of(const void *p, int64_t i, int type) {
  return type == kBF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]) : static_cast<const float *>(p)[i];
}

// Sum over the threads of a row, the same on all, in a fixed order. red: 2 x threads / 32 floats of the row's threads,
// used in turn, so one barrier a sum is enough.
struct RowSum {
  float *red;
  int threads, id, turn, thread;
  __device__ __forceinline__ float operator()(float v) {
    v = warp_sum(v);
    if (threads == 32) return v;
    float *at = red + turn * (threads / 32);
    turn ^= 1;
    if ((thread & 31) == 0) at[thread / 32] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
    float s = 0.f;
    for (int k = 0; k < threads / 32; ++k) s += at[k];
    return s;
  }
};

// ------------------------------------------------------------------ the ring of rows
constexpr int kMaxSlots = 8;
constexpr int kStreams = 3;  // x, y and (backward) dz
struct RingBarriers {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  int abort;
};
// What a CTA's ring holds: `slots` batches of `height` rows of each stream.
struct RingShape {
  const void *src[kStreams];
  int64_t ld_bytes[kStreams];
  int row_bytes[kStreams];  // as they lie in a slot, a multiple of 16; 0: no such stream
  int copy_bytes[kStreams];
  int elt[kStreams];
  int slot_bytes, slots, height, threads;  // threads of a row
};

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Copies n elements by `threads` threads, coalesced, several in flight each.
template <typename E>
__device__ __forceinline__ void copy_elements(E *dst, const E *src, int n, int thread, int threads) {
  constexpr int kDeep = 8;
  for (int i = thread; i < n; i += kDeep * threads) {
    E v[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k)
      if (i + k * threads < n) v[k] = __ldcs(src + i + k * threads);
#pragma unroll
    for (int k = 0; k < kDeep; ++k)
      if (i + k * threads < n) dst[i + k * threads] = v[k];
  }
}

constexpr int kFillWarps = 4;  // of rows without 16-byte access
template <bool WIDE>
constexpr int kFillThreads = WIDE ? 0 : kFillWarps * 32;
// 128 registers a thread where 512 threads do: a row's, or 384 and the four warps that copy
template <bool WIDE, int NP>
constexpr int kMaxThreads = WIDE || NP <= 2 ? 512 : 640;

// Rows that allow 16-byte access: the CTA's first warp issues the bulk copies of a batch itself, once every warp has left
// the slot (a warp of its own for it would leave the others 96 registers a thread instead of 128).
struct BulkFiller {
  uint32_t issued = 0, last = 0;  // per slot: whether copies were issued, the parity of the last
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void fill(const RingShape &ring, RingBarriers *bar, uint8_t *slots, int64_t rows, int64_t b,
                                       const Waiter &w) {
    if (b * ring.height >= rows) return;
    if (!warp_mbar_wait<false>(&bar->empty[slot], parity ^ 1u, w)) return;
    __syncwarp();
    const int lane = threadIdx.x & 31;
    const int n = static_cast<int>(min(static_cast<int64_t>(ring.height), rows - b * ring.height));
    int bytes = 0;
#pragma unroll
    for (int q = 0; q < kStreams; ++q) bytes += ring.row_bytes[q] ? ring.copy_bytes[q] : 0;
    if (lane == 0) mbar_arrive_expect_tx(&bar->full[slot], static_cast<uint32_t>(bytes * n));
    __syncwarp();
    if (lane < n) {
      uint8_t *to = slots + slot * ring.slot_bytes;
#pragma unroll
      for (int q = 0; q < kStreams; ++q)
        if (ring.row_bytes[q]) {
          bulk_load(to + lane * ring.row_bytes[q],
                    static_cast<const uint8_t *>(ring.src[q]) + (b * ring.height + lane) * ring.ld_bytes[q],
                    static_cast<uint32_t>(ring.copy_bytes[q]), &bar->full[slot]);
          to += ring.height * ring.row_bytes[q];
        }
    }
    issued |= 1u << slot;
    last = (last & ~(1u << slot)) | (parity << slot);
    if (++slot == ring.slots) {
      slot = 0;
      parity ^= 1u;
    }
  }
  __device__ __forceinline__ void first(const RingShape &ring, RingBarriers *bar, uint8_t *slots, int64_t rows, const Waiter &w) {
    for (int s = 0; s < ring.slots; ++s) fill(ring, bar, slots, rows, blockIdx.x + static_cast<int64_t>(s) * gridDim.x, w);
  }
  // after an abort: what was issued lands before the CTA ends
  __device__ __forceinline__ void end(const RingShape &ring, RingBarriers *bar, const Waiter &w) {
    if ((threadIdx.x & 31) == 0 && *w.abort)
      for (int s = 0; s < ring.slots; ++s)
        if ((issued >> s) & 1u) drain_wait(&bar->full[s], (last >> s) & 1u, w.limit_ns);
  }
};

// Other rows: four warps copy batches blockIdx.x, + gridDim.x, ... thread: 0.. of theirs.
__device__ __forceinline__ void copy_to_ring(const RingShape &ring, RingBarriers *bar, uint8_t *slots, int64_t rows, int thread,
                                             const Waiter &w) {
  int slot = 0;
  uint32_t parity = 0;
  for (int64_t b = blockIdx.x; b * ring.height < rows; b += gridDim.x) {
    if (!warp_mbar_wait<false>(&bar->empty[slot], parity ^ 1u, w)) break;
    __syncwarp();
    uint8_t *at = slots + slot * ring.slot_bytes;
    const int n = static_cast<int>(min(static_cast<int64_t>(ring.height), rows - b * ring.height));
    for (int q = 0; q < kStreams; ++q) {
      if (!ring.row_bytes[q]) continue;
      for (int r = 0; r < n; ++r) {
        const uint8_t *from = static_cast<const uint8_t *>(ring.src[q]) + (b * ring.height + r) * ring.ld_bytes[q];
        uint8_t *to = at + r * ring.row_bytes[q];
        if (ring.elt[q] == 2)
          copy_elements(reinterpret_cast<uint16_t *>(to), reinterpret_cast<const uint16_t *>(from), ring.copy_bytes[q] / 2, thread, kFillWarps * 32);
        else
          copy_elements(reinterpret_cast<uint32_t *>(to), reinterpret_cast<const uint32_t *>(from), ring.copy_bytes[q] / 4, thread, kFillWarps * 32);
      }
      at += ring.height * ring.row_bytes[q];
    }
    __syncwarp();
    if ((thread & 31) == 0) mbar_arrive(&bar->full[slot]);
    if (++slot == ring.slots) {
      slot = 0;
      parity ^= 1u;
    }
  }
}

// A consumer's place in the ring.
struct RowReader {
  int slot = 0;
  uint32_t parity = 0;
  // The slot's start once the batch is there. After a wait that gave up the caller goes on without storing, so that
  // the barriers of the other threads of a row are still met.
  __device__ __forceinline__ const uint8_t *wait(const RingShape &ring, RingBarriers *bar, const uint8_t *slots, const Waiter &w, bool &ok) {
    if (!mbar_wait(&bar->full[slot], parity, w)) ok = false;
    return slots + slot * ring.slot_bytes;
  }
  __device__ __forceinline__ void release(const RingShape &ring, RingBarriers *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&bar->empty[slot]);
    if (++slot == ring.slots) {
      slot = 0;
      parity ^= 1u;
    }
  }
};

__device__ __forceinline__ RingBarriers *start_ring(const RingShape &ring, uint8_t *smem, bool wide) {
  RingBarriers *bar = reinterpret_cast<RingBarriers *>(smem);
  if (threadIdx.x == 0) {
    for (int s = 0; s < ring.slots; ++s) {
      mbar_init(&bar->full[s], wide ? 1 : kFillWarps);
      mbar_init(&bar->empty[s], ring.threads * ring.height / 32);
    }
    bar->abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  return bar;
}
constexpr int kRingHead = (static_cast<int>(sizeof(RingBarriers)) + 127) / 128 * 128;

template <int XT, int YT, bool WIDE, int NP>
__global__ void __launch_bounds__(kMaxThreads<WIDE, NP>) ns_block_norm_kernel(const __grid_constant__ NormParams p,
                                                                                  const __grid_constant__ RingShape ring) {
  using X = typename Elem<XT>::T;
  using Y = typename Elem<YT>::T;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float reds[8][32];
  RingBarriers *bar = start_ring(ring, smem, WIDE);
  uint8_t *slots = smem + kRingHead;
  const Waiter w{&bar->abort, p.status, p.wait_limit_ns};
  const int consumers = ring.threads * ring.height;
  if (!WIDE && static_cast<int>(threadIdx.x) >= consumers) {
    copy_to_ring(ring, bar, slots, p.rows, threadIdx.x - consumers, w);
    return;
  }
  BulkFiller filler;
  const bool fills = WIDE && threadIdx.x < 32;
  if (fills) filler.first(ring, bar, slots, p.rows, w);
  const int group = threadIdx.x / ring.threads, thread = threadIdx.x - group * ring.threads;
  RowSum sum{reds[group], ring.threads, 1 + group, 0, thread};
  const size_t rsize = static_cast<size_t>((p.rows - 1) * p.ld_r + p.cols) * sizeof(X);
  const size_t zsize = static_cast<size_t>((p.rows - 1) * p.ld_z + p.cols) * sizeof(Y);
  const float n = static_cast<float>(p.cols);
  int c[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i)
    c[i] = WIDE ? (i * ring.threads + thread) * 8 : (i * ring.threads + (thread & ~31)) * 8 + (thread & 31);
  // the weights of this thread's columns, where there is room for them (else they are read again for each row)
  constexpr bool kHold = NP <= 2;
  float wp[kHold ? NP : 1][8], wz[kHold ? NP : 1][8];
  auto block_weight = [&](int i, float (&f)[8]) {  // b * post * gate of the columns
    load_any<WIDE>(p.post, p.weight_type, c[i], p.cols, f);
    if (p.gate_form == kGateCols) {
      float g[8];
      load_any<WIDE>(p.gate, p.gate_type, c[i], p.cols, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= g[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= p.b;
  };
  if constexpr (kHold) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if (p.y) block_weight(i, wp[i]);
      if (p.pre) load_any<WIDE>(p.pre, p.weight_type, c[i], p.cols, wz[i]);
    }
  }
  RowReader reader;
  bool ok = true;
  for (int64_t b = blockIdx.x; b * ring.height < p.rows; b += gridDim.x) {
    const uint8_t *at = reader.wait(ring, bar, slots, w, ok);
    const int64_t t = b * ring.height + group, ahead = b + static_cast<int64_t>(ring.slots) * gridDim.x;
    if (t >= p.rows) {  // (not the first warp: the batch's last rows)
      reader.release(ring, bar);
      continue;
    }
    const void *xs = at + group * ring.row_bytes[0], *ys = at + ring.height * ring.row_bytes[0] + group * ring.row_bytes[1];
    Pack<XT, 8> x[NP];
    Pack<YT, 8> y[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      load8<XT, WIDE>(xs, c[i], p.cols, x[i]);
      if (p.y) load8<YT, WIDE>(ys, c[i], p.cols, y[i]);
    }
    reader.release(ring, bar);
    float r[NP][8];
    if (p.y) {
      float k = p.gate_form == kGateRows ? one_of(p.gate, t * p.ld_gate, p.gate_type) : 1.f;
      if (p.post) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) s = fmaf(y[i].get(e), y[i].get(e), s);
        const float ry = rsqrtf(sum(s) / n + p.eps);
        if (thread == 0 && ok) p.post_rstd[t] = ry;
        k *= ry;
      }
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        float f[8];
        if constexpr (kHold) {
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = wp[i][e];
        } else {
          block_weight(i, f);
        }
        if (p.gate_form == kGateFull) {
          float g[8];
          load_any<WIDE>(at_row(p.gate, t, p.ld_gate, p.gate_type), p.gate_type, c[i], p.cols, g);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] *= g[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) r[i][e] = fmaf(y[i].get(e) * k, f[e], p.a * x[i].get(e));
      }
    } else {
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) r[i][e] = p.a * x[i].get(e);
    }
    if (fills) filler.fill(ring, bar, slots, p.rows, ahead, w);
    X *to = static_cast<X *>(p.r) + t * p.ld_r;
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (ok) store8<XT, WIDE>(to, c[i], p.cols, r[i], p.r, rsize, p.status);
    if (p.pre) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(r[i][e], r[i][e], s);
      const float rr = rsqrtf(sum(s) / n + p.eps);
      if (thread == 0 && ok) p.pre_rstd[t] = rr;
      Y *zt = static_cast<Y *>(p.z) + t * p.ld_z;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        float f[8];
        if constexpr (kHold) {
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = wz[i][e];
        } else {
          load_any<WIDE>(p.pre, p.weight_type, c[i], p.cols, f);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= r[i][e] * rr;
        if (ok) store8<YT, WIDE>(zt, c[i], p.cols, f, p.z, zsize, p.status);
      }
    }
  }
  if (fills) filler.end(ring, bar, w);
}

// Backward. The columns' sums are in registers, or for rows of more than 2 packs a thread in shared memory behind the
// ring ([2][NP][8][threads of a row] floats for each row of the CTA, every thread its own).
template <int XT, int YT, bool WIDE, int NP>
__global__ void __launch_bounds__(kMaxThreads<WIDE, NP>) ns_block_norm_backward_kernel(const __grid_constant__ NormParams p,
                                                                                           const __grid_constant__ RingShape ring) {
  using X = typename Elem<XT>::T;
  using Y = typename Elem<YT>::T;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float reds[8][32];
  RingBarriers *bar = start_ring(ring, smem, WIDE);
  uint8_t *slots = smem + kRingHead;
  const Waiter w{&bar->abort, p.status, p.wait_limit_ns};
  const int consumers = ring.threads * ring.height;
  const bool producer = !WIDE && static_cast<int>(threadIdx.x) >= consumers;
  const int group = producer ? 0 : threadIdx.x / ring.threads, thread = producer ? 0 : threadIdx.x - group * ring.threads;
  constexpr bool kHold = NP <= 2;
  const int step = ring.threads;
  float *sums = reinterpret_cast<float *>(kHold ? slots : slots + ring.slots * ring.slot_bytes);
  float *acc = sums + group * (2 * NP * 8 * step) + thread;
  int c[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i)
    c[i] = WIDE ? (i * ring.threads + thread) * 8 : (i * ring.threads + (thread & ~31)) * 8 + (thread & 31);
  if (producer) {
    copy_to_ring(ring, bar, slots, p.rows, threadIdx.x - consumers, w);
  } else {
    BulkFiller filler;
    const bool fills = WIDE && threadIdx.x < 32;
    if (fills) filler.first(ring, bar, slots, p.rows, w);
    RowSum sum{reds[group], ring.threads, 1 + group, 0, thread};
    const size_t xsize = static_cast<size_t>((p.rows - 1) * p.ld_dx + p.cols) * sizeof(X);
    const size_t ysize = static_cast<size_t>((p.rows - 1) * p.ld_dy + p.cols) * sizeof(Y);
    const float n = static_cast<float>(p.cols);
    float held[2][kHold ? NP : 1][8];
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (kHold) {
          held[0][i][e] = held[1][i][e] = 0.f;
        } else {
          acc[(i * 8 + e) * step] = acc[((NP + i) * 8 + e) * step] = 0.f;
        }
      }
    auto add = [&](int k, int i, int e, float v) {
      if constexpr (kHold)
        held[k][i][e] += v;
      else
        acc[((k * NP + i) * 8 + e) * step] += v;
    };
    // post * gate of the columns (a full gate's own)
    auto block_weight = [&](int i, int64_t t, float (&f)[8]) {
      load_any<WIDE>(p.y ? p.post : nullptr, p.weight_type, c[i], p.cols, f);
      if (p.gate_form == kGateCols || p.gate_form == kGateFull) {
        float g[8];
        load_any<WIDE>(p.gate_form == kGateFull ? at_row(p.gate, t, p.ld_gate, p.gate_type) : p.gate, p.gate_type, c[i], p.cols, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= g[e];
      }
    };
    RowReader reader;
    bool ok = true;
    for (int64_t b = blockIdx.x; b * ring.height < p.rows; b += gridDim.x) {
      const int64_t t = b * ring.height + group;
      const bool here = t < p.rows;
      Pack<XT, 8> dr[NP];
      if (p.dr && here) {  // used after the first sum: read past the ring
#pragma unroll
        for (int i = 0; i < NP; ++i) load8<XT, WIDE>(at_row(p.dr, t, p.ld_dr, XT), c[i], p.cols, dr[i]);
      }
      const float ry = here && p.y && p.post ? p.post_rstd[t] : 1.f, rr = here && p.pre ? p.pre_rstd[t] : 0.f;
      const float grow = here && p.gate_form == kGateRows ? one_of(p.gate, t * p.ld_gate, p.gate_type) : 1.f;
      const uint8_t *at = reader.wait(ring, bar, slots, w, ok);
      if (!here) {
        reader.release(ring, bar);
        continue;
      }
      // a stream that the ring has no room for is read where it lies
      const void *rows_at[kStreams];
#pragma unroll
      for (int q = 0; q < kStreams; ++q) {
        rows_at[q] = ring.row_bytes[q] ? at + group * ring.row_bytes[q] : static_cast<const uint8_t *>(ring.src[q]) + t * ring.ld_bytes[q];
        at += ring.height * ring.row_bytes[q];
      }
      const void *xs = rows_at[0], *ys = rows_at[1], *zs = rows_at[2];
      Pack<YT, 8> y[NP];
      float d[NP][8];  // the gradient of r
      if (p.pre) {
        float rh[NP][8], s = 0.f;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          Pack<XT, 8> x;
          load8<XT, WIDE>(xs, c[i], p.cols, x);
          if (p.y) {
            load8<YT, WIDE>(ys, c[i], p.cols, y[i]);
            float f[8];
            block_weight(i, t, f);
            const float k = p.b * ry * grow;
#pragma unroll
            for (int e = 0; e < 8; ++e) rh[i][e] = fmaf(y[i].get(e) * k, f[e], p.a * x.get(e)) * rr;
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) rh[i][e] = p.a * x.get(e) * rr;
          }
          Pack<YT, 8> dz;
          load8<YT, WIDE>(zs, c[i], p.cols, dz);
          float f[8];
          load_any<WIDE>(p.pre, p.weight_type, c[i], p.cols, f);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float z = dz.get(e);
            add(0, i, e, z * rh[i][e]);
            d[i][e] = z * f[e];
            s = fmaf(d[i][e], rh[i][e], s);
          }
        }
        reader.release(ring, bar);
        s = sum(s) / n;
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) d[i][e] = fmaf(rr, d[i][e] - rh[i][e] * s, p.dr ? dr[i].get(e) : 0.f);
      } else {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          if (p.y) load8<YT, WIDE>(ys, c[i], p.cols, y[i]);
#pragma unroll
          for (int e = 0; e < 8; ++e) d[i][e] = p.dr ? dr[i].get(e) : 0.f;
        }
        reader.release(ring, bar);
      }
      if (fills) filler.fill(ring, bar, slots, p.rows, b + static_cast<int64_t>(ring.slots) * gridDim.x, w);
      X *to = static_cast<X *>(p.dx) + t * p.ld_dx;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = p.a * d[i][e];
        if (ok) store8<XT, WIDE>(to, c[i], p.cols, o, p.dx, xsize, p.status);
      }
      if (!p.y) continue;
      // through the gate: d * yh enters the sums (with a row's or a full gate's factor; the columns' comes at their end);
      // the gradient of y's norm is b gate post d
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        float f[8];
        if (p.gate_form == kGateFull) {
          float g[8], og[8];
          load_any<WIDE>(p.post, p.weight_type, c[i], p.cols, f);
          load_any<WIDE>(at_row(p.gate, t, p.ld_gate, p.gate_type), p.gate_type, c[i], p.cols, g);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            og[e] = p.b * f[e] * d[i][e] * (y[i].get(e) * ry);
            d[i][e] *= g[e];
          }
          const size_t gsize = static_cast<size_t>((p.rows - 1) * p.ld_dgate + p.cols) * (p.gate_type == kBF16 ? 2 : 4);
          void *gt = const_cast<void *>(at_row(p.dgate, t, p.ld_dgate, p.gate_type));
          if (ok && p.gate_type == kBF16)
            store8<kBF16, WIDE>(gt, c[i], p.cols, og, p.dgate, gsize, p.status);
          else if (ok)
            store8<kF32, WIDE>(gt, c[i], p.cols, og, p.dgate, gsize, p.status);
        } else {
          block_weight(i, t, f);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float dyh = d[i][e] * (y[i].get(e) * ry);
          add(1, i, e, grow * dyh);
          s = fmaf(p.b * f[e], dyh, s);
          d[i][e] *= p.b * grow * f[e];
        }
      }
      s = p.post || p.gate_form == kGateRows ? sum(s) : 0.f;
      if (p.gate_form == kGateRows && thread == 0 && ok) {
        if (p.gate_type == kBF16)
          static_cast<__nv_bfloat16 *>(p.dgate)[t * p.ld_dgate] = __float2bfloat16_rn(s);
        else
          static_cast<float *>(p.dgate)[t * p.ld_dgate] = s;
      }
      const float k = p.post ? s * grow / n : 0.f;
      Y *yt = static_cast<Y *>(p.dy) + t * p.ld_dy;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = ry * (d[i][e] - y[i].get(e) * ry * k);
        if (ok) store8<YT, WIDE>(yt, c[i], p.cols, o, p.dy, ysize, p.status);
      }
    }
    if (fills) filler.end(ring, bar, w);
    if constexpr (kHold) {
      // the ring is done with once every thread is here: it takes the sums
      asm volatile("bar.sync 15, %0;" ::"r"(consumers) : "memory");
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[((k * NP + i) * 8 + e) * step] = held[k][i][e];
    }
    asm volatile("bar.sync 15, %0;" ::"r"(consumers) : "memory");
    // the CTA's rows added in order, to its part
    if (group == 0) {
      float *part = p.parts + static_cast<int64_t>(blockIdx.x) * 2 * p.cols;
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int at = (k * NP + i) * 8 + e, col = col_of<WIDE>(c[i], e);
            float v = acc[at * step];
            for (int j = 1; j < ring.height; ++j) v += acc[at * step + j * (2 * NP * 8 * step)];
            if (col < p.cols) part[k * p.cols + col] = v;
          }
    }
  }
}

struct JoinParams {
  const float *parts;
  int count, cols, gate_form, gate_type, weight_type;
  const void *gate, *post;
  void *dgate, *dpost, *dpre;
  float b;
  int *status;
};

// Weights' gradients from the CTAs' parts: 32 columns a CTA, its warps take parts in turn.
__global__ void __launch_bounds__(512) ns_block_norm_join_kernel(const __grid_constant__ JoinParams p) {
  __shared__ float red[2][16][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float s0 = 0.f, s1 = 0.f;
  if (col < p.cols)
#pragma unroll 4
    for (int k = warp; k < p.count; k += 16) {
      s0 += p.parts[(static_cast<int64_t>(k) * 2) * p.cols + col];
      s1 += p.parts[(static_cast<int64_t>(k) * 2 + 1) * p.cols + col];
    }
  red[0][warp][lane] = s0;
  red[1][warp][lane] = s1;
  __syncthreads();
  if (warp != 0 || col >= p.cols) return;
  for (int k = 1; k < 16; ++k) {
    s0 += red[0][k][lane];
    s1 += red[1][k][lane];
  }
  auto write = [&](void *out, int type, float v) {
    const size_t size = static_cast<size_t>(p.cols) * (type == kBF16 ? 2 : 4);
    if (type == kBF16) {
      __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(out) + col;
      if (in_bounds(to, 2, out, size, p.status)) *to = __float2bfloat16_rn(v);
    } else {
      float *to = static_cast<float *>(out) + col;
      if (in_bounds(to, 4, out, size, p.status)) *to = v;
    }
  };
  if (p.dpre) write(p.dpre, p.weight_type, s0);
  const float post = p.post ? one_of(p.post, col, p.weight_type) : 1.f;
  if (p.dpost) write(p.dpost, p.weight_type, p.b * s1 * (p.gate_form == kGateCols ? one_of(p.gate, col, p.gate_type) : 1.f));
  if (p.gate_form == kGateCols) write(p.dgate, p.gate_type, p.b * s1 * post);
}

// Threads of a row, packs a thread, rows of a CTA of about 256 threads, and the ring: as many slots as leave room for
// `per_sm` CTAs on an SM, two at least where that is possible at all.
struct Shape {
  int threads, packs, rows, per_sm, smem;
  RingShape ring{};
  Shape(const NormParams &p, bool backward, bool wide, int xt, int yt) {
    const int lanes = (p.cols + 7) / 8;
    packs = lanes <= 256 ? 1 : lanes <= (wide ? 1024 : 768) ? 2 : 4;
    threads = ((lanes + packs - 1) / packs + 31) / 32 * 32;
    rows = threads >= 256 ? 1 : std::min(8, 256 / threads);
    ring.height = rows;
    ring.threads = threads;
    const void *src[kStreams] = {p.x, p.y, backward && p.pre ? p.dz : nullptr};
    const int64_t ld[kStreams] = {p.ld_x, p.ld_y, p.ld_dz};
    const int elt[kStreams] = {xt == kBF16 ? 2 : 4, yt == kBF16 ? 2 : 4, yt == kBF16 ? 2 : 4};
    int bytes[kStreams];
    for (int q = 0; q < kStreams; ++q) {
      ring.src[q] = src[q];
      ring.ld_bytes[q] = ld[q] * elt[q];
      ring.copy_bytes[q] = p.cols * elt[q];
      ring.elt[q] = elt[q];
      bytes[q] = src[q] ? (p.cols * elt[q] + 15) / 16 * 16 : 0;
    }
    const int sums = backward ? 2 * packs * 8 * threads * rows * 4 : 0;
    const int room = 224 * 1024 - kRingHead - 4096;  // with the kernel's own
    const int beside = packs <= 2 ? 0 : sums;        // sums that the ring cannot take at the end
    int streams = kStreams;
    auto slot_of = [&](int n) {
      int v = 0;
      for (int q = 0; q < n; ++q) v += bytes[q] * rows;
      return v;
    };
    while (streams > 1 && slot_of(streams) + beside > room) --streams;
    for (int q = 0; q < streams; ++q) ring.row_bytes[q] = bytes[q];
    ring.slot_bytes = slot_of(streams);
    for (per_sm = backward ? 2 : std::max(1, std::min(4, 1024 / (threads * rows))); per_sm > 1; --per_sm)
      if ((room / per_sm - kRingHead - 4096 - beside) / ring.slot_bytes >= 2) break;
    const int mine = per_sm == 1 ? room : room / per_sm - kRingHead - 4096;
    ring.slots = std::max(1, std::min(kMaxSlots, (mine - beside) / ring.slot_bytes));
    smem = kRingHead + std::max(ring.slots * ring.slot_bytes + beside, sums);
  }
  int block(bool wide) const { return threads * rows + (wide ? 0 : kFillWarps * 32); }
  int64_t batches(int64_t n) const { return (n + rows - 1) / rows; }
};

template <typename F>
int by_packs(int packs, F &&f) {
  return packs == 1 ? f(std::integral_constant<int, 1>{}) : packs == 2 ? f(std::integral_constant<int, 2>{}) : f(std::integral_constant<int, 4>{});
}
template <typename F>
int by_types(int xt, int yt, bool wide, F &&f) {
  using B = std::integral_constant<int, kBF16>;
  using S = std::integral_constant<int, kF32>;
  if (xt == kBF16) return wide ? f(B{}, B{}, std::true_type{}) : f(B{}, B{}, std::false_type{});
  if (yt == kBF16) return wide ? f(S{}, B{}, std::true_type{}) : f(S{}, B{}, std::false_type{});
  return wide ? f(S{}, S{}, std::true_type{}) : f(S{}, S{}, std::false_type{});
}

bool bad_type(int t) { return t != NS_F32 && t != NS_BF16; }
int size_of(int t) { return t == NS_BF16 ? 2 : 4; }
// The checks that both directions share; fills p. `written`: ranges of the outputs to come are checked by the caller.
int check(NormParams &p, const void *x, int64_t ld_x, const void *y, int64_t ld_y, const void *gate, int gate_form,
          int64_t ld_gate, const void *post, const void *pre, int64_t rows, int64_t cols, float a, float b, int dtype,
          int block_dtype, int weight_dtype, int gate_dtype) {
  if (bad_type(dtype) || bad_type(block_dtype) || bad_type(weight_dtype) || bad_type(gate_dtype)) return NS_EINVAL;
  if (dtype == NS_BF16 && block_dtype == NS_F32) return NS_EINVAL;  // a residual narrower than the block's output
  if (bad_shape(rows, cols, ld_x) || cols > kMaxCols || gate_form < kGateNone || gate_form > kGateFull) return NS_EINVAL;
  if (!std::isfinite(a) || !std::isfinite(b)) return NS_EINVAL;
  if (y && bad_shape(rows, cols, ld_y)) return NS_EINVAL;
  if (!y && (gate_form != kGateNone || post)) return NS_EINVAL;
  if (!y && !pre && rows > 0) return NS_EINVAL;  // nothing to do
  if ((gate_form != kGateNone) != (gate != nullptr) && rows > 0) return NS_EINVAL;
  if (gate_form == kGateFull && bad_shape(rows, cols, ld_gate)) return NS_EINVAL;
  if (gate_form == kGateRows && bad_shape(rows, 1, ld_gate)) return NS_EINVAL;
  if (misaligned(x, size_of(dtype)) || misaligned(y, size_of(block_dtype)) || misaligned(gate, size_of(gate_dtype)) ||
      misaligned(post, size_of(weight_dtype)) || misaligned(pre, size_of(weight_dtype)))
    return NS_EALIGN;
  p.x = x;
  p.y = y;
  p.gate = gate;
  p.post = post;
  p.pre = pre;
  p.ld_x = ld_x;
  p.ld_y = ld_y;
  p.ld_gate = ld_gate;
  p.rows = rows;
  p.cols = static_cast<int>(cols);
  p.gate_form = gate_form;
  p.gate_type = gate_dtype;
  p.weight_type = weight_dtype;
  p.a = a;
  p.b = b;
  return NS_OK;
}
// Whether every operand that is read in packs allows it.
bool packs_fit(const NormParams &p, int dtype, int block_dtype) {
  return p.cols % 8 == 0 && rows_aligned(p.x, p.ld_x, size_of(dtype), 8) && rows_aligned(p.y, p.ld_y, size_of(block_dtype), 8) &&
         !misaligned(p.post, 16) && !misaligned(p.pre, 16) &&
         (p.gate_form == kGateCols ? !misaligned(p.gate, 16)
                                   : p.gate_form != kGateFull || rows_aligned(p.gate, p.ld_gate, size_of(p.gate_type), 8));
}
Range gate_range(const void *gate, int form, int64_t rows, int64_t cols, int64_t ld, int type) {
  return form == kGateCols   ? Range(gate, 1, cols, cols, size_of(type))
         : form == kGateRows ? Range(gate, rows, 1, ld, size_of(type))
         : form == kGateFull ? Range(gate, rows, cols, ld, size_of(type))
                             : Range(nullptr, 0, 0, 0, 1);
}

}  // namespace
}  // namespace ns

using namespace ns;

extern "C" int64_t ns_block_norm_workspace(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || cols > kMaxCols) return -1;
  return std::max<int64_t>(1, std::min<int64_t>(rows, kMaxParts)) * 2 * cols * 4;
}

extern "C" int ns_block_norm(const void *x, int64_t ld_x, const void *y, int64_t ld_y, const void *gate, int gate_form,
                             int64_t ld_gate, const void *post, const void *pre, int64_t rows, int64_t cols, float a,
                             float b, float eps, void *residual, int64_t ld_r, void *normed, int64_t ld_z,
                             float *post_rstd, float *pre_rstd, int dtype, int block_dtype, int weight_dtype,
                             int gate_dtype, void *stream) {
  NormParams p{};
  if (int rc = check(p, x, ld_x, y, ld_y, gate, gate_form, ld_gate, post, pre, rows, cols, a, b, dtype, block_dtype,
                     weight_dtype, gate_dtype))
    return rc;
  if (!(eps >= 0.f) || !std::isfinite(eps) || bad_shape(rows, cols, ld_r) || (pre && bad_shape(rows, cols, ld_z))) return NS_EINVAL;
  if (rows == 0 || cols == 0) return NS_OK;
  if (!x || !residual || (pre && (!normed || !pre_rstd)) || (post && !post_rstd)) return NS_EINVAL;
  const int xe = size_of(dtype), ye = size_of(block_dtype), we = size_of(weight_dtype);
  if (misaligned(residual, xe) || misaligned(normed, ye) || misaligned(post_rstd, 4) || misaligned(pre_rstd, 4)) return NS_EALIGN;
  const Range in[] = {Range(x, rows, cols, ld_x, xe), Range(y, rows, cols, ld_y, ye),
                      gate_range(gate, gate_form, rows, cols, ld_gate, gate_dtype), Range(post, 1, cols, cols, we),
                      Range(pre, 1, cols, cols, we)};
  const Range out[] = {Range(residual, rows, cols, ld_r, xe), Range(pre ? normed : nullptr, rows, cols, ld_z, ye),
                       Range(post ? post_rstd : nullptr, 1, rows, rows, 4), Range(pre ? pre_rstd : nullptr, 1, rows, rows, 4)};
  // a thread reads its part of a row before it writes there: residual may be x, normed may be y
  const bool over_x = residual == x && ld_r == ld_x, over_y = normed == y && ld_z == ld_y;
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 5; ++i)
      if (!(o == 0 && i == 0 && over_x) && !(o == 1 && i == 1 && over_y) && out[o].overlaps(in[i])) return NS_EINVAL;
    for (int k = 0; k < o; ++k)
      if (out[o].overlaps(out[k])) return NS_EINVAL;
  }
  OpCall call(stream);
  if (call.rc) return call.rc;
  p.r = residual;
  p.z = normed;
  p.ld_r = ld_r;
  p.ld_z = ld_z;
  p.post_rstd = post_rstd;
  p.pre_rstd = pre_rstd;
  p.eps = eps;
  p.status = call.status;
  p.wait_limit_ns = kWaitLimitNs;
  const bool wide = packs_fit(p, dtype, block_dtype) && rows_aligned(residual, ld_r, xe, 8) && (!pre || rows_aligned(normed, ld_z, ye, 8));
  const Shape sh(p, false, wide, dtype, block_dtype);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(sh.batches(rows), static_cast<int64_t>(call.sms) * sh.per_sm));
  return call.launch(kOpBlockNorm, [&] {
    const int rc = by_types(dtype, block_dtype, wide, [&](auto xt, auto yt, auto w) {
      return by_packs(sh.packs, [&](auto np) {
        auto *kernel = ns_block_norm_kernel<decltype(xt)::value, decltype(yt)::value, decltype(w)::value, decltype(np)::value>;
        static SmemOptIn opt_in;
        if (opt_in.ensure(reinterpret_cast<const void *>(kernel), sh.smem)) return -1;
        kernel<<<grid, sh.block(wide), sh.smem, call.s>>>(p, sh.ring);
        return 0;
      });
    });
    if (rc) return rc;
    count_launch();
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
  });
}

extern "C" int ns_block_norm_backward(const void *dresidual, int64_t ld_dr, const void *dnormed, int64_t ld_dz,
                                      const void *x, int64_t ld_x, const void *y, int64_t ld_y, const void *gate,
                                      int gate_form, int64_t ld_gate, const void *post, const void *pre,
                                      const float *post_rstd, const float *pre_rstd, int64_t rows, int64_t cols, float a,
                                      float b, void *dx, int64_t ld_dx, void *dy, int64_t ld_dy, void *dgate,
                                      int64_t ld_dgate, void *dpost, void *dpre, void *workspace,
                                      size_t workspace_bytes, int dtype, int block_dtype, int weight_dtype,
                                      int gate_dtype, void *stream) {
  NormParams p{};
  if (int rc = check(p, x, ld_x, y, ld_y, gate, gate_form, ld_gate, post, pre, rows, cols, a, b, dtype, block_dtype,
                     weight_dtype, gate_dtype))
    return rc;
  if ((dresidual && bad_shape(rows, cols, ld_dr)) || (pre && bad_shape(rows, cols, ld_dz)) || bad_shape(rows, cols, ld_dx) ||
      (y && bad_shape(rows, cols, ld_dy)) || (gate_form == kGateFull && bad_shape(rows, cols, ld_dgate)) ||
      (gate_form == kGateRows && bad_shape(rows, 1, ld_dgate)))
    return NS_EINVAL;
  if (cols == 0) return NS_OK;
  if ((post && !dpost) || (pre && !dpre) || (gate_form == kGateCols && !dgate) || !workspace) return NS_EINVAL;
  if (rows > 0 && (!x || !dx || (y && !dy) || (pre && (!dnormed || !pre_rstd)) || (post && !post_rstd) ||
                   (gate_form != kGateNone && !dgate) || (!dresidual && !pre)))
    return NS_EINVAL;
  if (workspace_bytes < static_cast<size_t>(ns_block_norm_workspace(rows, cols))) return NS_ENOMEM;
  const int xe = size_of(dtype), ye = size_of(block_dtype), we = size_of(weight_dtype), ge = size_of(gate_dtype);
  if (misaligned(dresidual, xe) || misaligned(dnormed, ye) || misaligned(dx, xe) || misaligned(dy, ye) || misaligned(dgate, ge) ||
      misaligned(dpost, we) || misaligned(dpre, we) || misaligned(post_rstd, 4) || misaligned(pre_rstd, 4) || misaligned(workspace, 4))
    return NS_EALIGN;
  const Range in[] = {Range(dresidual, rows, cols, ld_dr, xe), Range(pre ? dnormed : nullptr, rows, cols, ld_dz, ye),
                      Range(x, rows, cols, ld_x, xe), Range(y, rows, cols, ld_y, ye),
                      gate_range(gate, gate_form, rows, cols, ld_gate, gate_dtype), Range(post, 1, cols, cols, we),
                      Range(pre, 1, cols, cols, we), Range(post ? post_rstd : nullptr, 1, rows, rows, 4),
                      Range(pre ? pre_rstd : nullptr, 1, rows, rows, 4)};
  const Range out[] = {Range(dx, rows, cols, ld_dx, xe), Range(y ? dy : nullptr, rows, cols, ld_dy, ye),
                       gate_range(dgate, gate_form, rows, cols, ld_dgate, gate_dtype),
                       Range(post ? dpost : nullptr, 1, cols, cols, we), Range(pre ? dpre : nullptr, 1, cols, cols, we),
                       Range(workspace, 1, static_cast<int64_t>(workspace_bytes), static_cast<int64_t>(workspace_bytes), 1)};
  const bool over_r = dx == dresidual && ld_dx == ld_dr, over_z = dy == dnormed && ld_dy == ld_dz;
  for (int o = 0; o < 6; ++o) {
    for (int i = 0; i < 9; ++i)
      if (!(o == 0 && i == 0 && over_r) && !(o == 1 && i == 1 && over_z) && out[o].overlaps(in[i])) return NS_EINVAL;
    for (int k = 0; k < o; ++k)
      if (out[o].overlaps(out[k])) return NS_EINVAL;
  }
  OpCall call(stream);
  if (call.rc) return call.rc;
  p.dr = dresidual;
  p.dz = dnormed;
  p.dx = dx;
  p.dy = dy;
  p.dgate = dgate;
  p.ld_dr = ld_dr;
  p.ld_dz = ld_dz;
  p.ld_dx = ld_dx;
  p.ld_dy = ld_dy;
  p.ld_dgate = ld_dgate;
  p.post_rstd = const_cast<float *>(post_rstd);
  p.pre_rstd = const_cast<float *>(pre_rstd);
  p.parts = static_cast<float *>(workspace);
  p.status = call.status;
  p.wait_limit_ns = kWaitLimitNs;
  const bool wide = packs_fit(p, dtype, block_dtype) && rows_aligned(dresidual, ld_dr, xe, 8) && rows_aligned(dnormed, ld_dz, ye, 8) &&
                    rows_aligned(dx, ld_dx, xe, 8) && rows_aligned(dy, ld_dy, ye, 8) &&
                    (gate_form != kGateFull || rows_aligned(dgate, ld_dgate, ge, 8));
  const Shape sh(p, true, wide, dtype, block_dtype);
  const int grid = static_cast<int>(std::min<int64_t>({sh.batches(rows), static_cast<int64_t>(call.sms) * sh.per_sm, kMaxParts}));
  const JoinParams j{p.parts, grid, p.cols, gate_form, gate_dtype, weight_dtype, gate, post, dgate, post ? dpost : nullptr,
                     pre ? dpre : nullptr, b, call.status};
  return call.launch(kOpBlockNorm, [&] {
    int rc = 0;
    if (grid > 0) {
      rc = by_types(dtype, block_dtype, wide, [&](auto xt, auto yt, auto w) {
        return by_packs(sh.packs, [&](auto np) {
          auto *kernel = ns_block_norm_backward_kernel<decltype(xt)::value, decltype(yt)::value, decltype(w)::value, decltype(np)::value>;
          static SmemOptIn opt_in;
          if (opt_in.ensure(reinterpret_cast<const void *>(kernel), sh.smem)) return -1;
          kernel<<<grid, sh.block(wide), sh.smem, call.s>>>(p, sh.ring);
          return 0;
        });
      });
      if (rc) return rc;
      count_launch();
    }
    if (j.dpre || j.dpost || gate_form == kGateCols) {
      ns_block_norm_join_kernel<<<(p.cols + 31) / 32, 512, 0, call.s>>>(j);
      count_launch();
    }
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
  });
}
