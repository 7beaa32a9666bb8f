// ns_block_norm.cuh -- what the two directions of the block norms share: element access, the ring of rows, the shape of
// a launch and the checks of arguments.
#pragma once

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "../../include/ns.h"
#include "ns_rows.cuh"

namespace ns {
namespace block_norm {

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
  size_t parts_size;        // bytes of the scratch they are in
  int64_t ld_x, ld_y, ld_gate, ld_r, ld_z, ld_dr, ld_dz, ld_dx, ld_dy, ld_dgate;
  int64_t rows;
  int cols, gate_form, gate_type, weight_type;
  float a, b, eps;
  int *status;
  uint64_t wait_limit_ns;
  int hold;                 // the columns' weights are kept in shared memory
};

// The 8 columns of a pack that starts at column c, in pairs: consecutive where rows allow packs (WIDE), else every 32nd.
template <bool WIDE>
__device__ __forceinline__ int col_of(int c, int e) { return WIDE ? c + e : c + 32 * e; }
struct Eight2 {
  float2 v[4];
  __device__ __forceinline__ float get(int e) const { return e & 1 ? v[e / 2].y : v[e / 2].x; }
  __device__ __forceinline__ void fill(float f) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = make_float2(f, f);
  }
};
__device__ __forceinline__ float2 both(float f) { return make_float2(f, f); }

// Columns of a row at `row`, in shared memory or global (16-byte aligned where WIDE); zeros beyond it. PADDED: zeros lie
// behind the row.
template <int DT, bool WIDE, bool PADDED = false>
__device__ __forceinline__ void load8(const void *row, int c, int cols, Eight2 &o) {
  using E = typename Elem<DT>::T;
  const E *p = static_cast<const E *>(row);
  if constexpr (WIDE) {
    if (PADDED || c < cols) {
      if constexpr (DT == kBF16) {
        const uint4 w = *reinterpret_cast<const uint4 *>(p + c);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) o.v[j] = make_float2(__uint_as_float(u[j] << 16), __uint_as_float(u[j] & 0xffff0000u));
      } else {
        const float4 l = *reinterpret_cast<const float4 *>(p + c), h = *reinterpret_cast<const float4 *>(p + c + 4);
        o.v[0] = make_float2(l.x, l.y);
        o.v[1] = make_float2(l.z, l.w);
        o.v[2] = make_float2(h.x, h.y);
        o.v[3] = make_float2(h.z, h.w);
      }
    } else {
      o.fill(0.f);
    }
  } else {  // (what lies behind a ragged row is left from others)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o.v[j] = make_float2(c + 64 * j < cols ? Elem<DT>::to_f(p[c + 64 * j]) : 0.f,
                           c + 64 * j + 32 < cols ? Elem<DT>::to_f(p[c + 64 * j + 32]) : 0.f);
  }
}
template <int DT, bool WIDE>
__device__ __forceinline__ void store8(void *row, int c, int cols, const Eight2 &f, const void *base, size_t size, int *status) {
  using E = typename Elem<DT>::T;
  E *p = static_cast<E *>(row);
  if constexpr (WIDE) {
    Pack<DT, 8> v;
    if constexpr (DT == kBF16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __float22bfloat162_rn(f.v[j]);
        reinterpret_cast<uint32_t *>(v.w)[j] = *reinterpret_cast<const uint32_t *>(&h);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v.set(e, f.get(e));
    }
    if (c < cols) v.store_stream(p + c, base, size, status);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + 32 * e < cols && in_bounds(p + c + 32 * e, sizeof(E), base, size, status)) __stcs(p + c + 32 * e, Elem<DT>::from_f(f.get(e)));
  }
}
// 8 values of either type; 1 where there are none
template <bool WIDE>
__device__ __forceinline__ void load_any(const void *row, int type, int c, int cols, Eight2 &f) {
  if (!row)
    f.fill(1.f);
  else if (type == kBF16)
    load8<kBF16, WIDE>(row, c, cols, f);
  else
    load8<kF32, WIDE>(row, c, cols, f);
}
__device__ __forceinline__ const void *at_row(const void *p, int64_t row, int64_t ld, int type) {
  return static_cast<const uint8_t *>(p) + row * ld * (type == kBF16 ? 2 : 4);
}
__device__ __forceinline__ float one_of(const void *p, int64_t i, int type) {
  return type == kBF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]) : static_cast<const float *>(p)[i];
}

// Sum over the threads of a row, the same on all, in a fixed order. red: 2 x 16 floats of the row's threads, 0 where
// there is no warp, used in turn, so one barrier a sum is enough.
struct RowSum {
  float *red;
  int threads, id, turn, thread;
  __device__ __forceinline__ float operator()(float v) {
    v = warp_sum(v);
    if (threads == 32) return v;
    float *at = red + turn * 16;
    turn ^= 1;
    if ((thread & 31) == 0) at[thread / 32] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 q = reinterpret_cast<const float4 *>(at)[k];
      s = __fadd2_rn(s, __fadd2_rn(make_float2(q.x, q.y), make_float2(q.z, q.w)));
    }
    return s.x + s.y;
  }
};
constexpr int kMaxHeight = 8;  // rows of a batch: their streams are a warp's lanes
struct alignas(16) RowSums {
  float red[kMaxHeight][32];
  __device__ __forceinline__ void clear() {
    for (int i = threadIdx.x; i < kMaxHeight * 32; i += blockDim.x) red[i / 32][i % 32] = 0.f;
  }
};

// ------------------------------------------------------------------ the ring of rows
constexpr int kMaxSlots = 8;
constexpr int kStreams = 4;  // x, y and (backward) dz, dr
struct RingBarriers {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  int abort;
};
// What a CTA's ring holds: `slots` batches of `height` rows of each stream. A row lies as many bytes behind a 16-byte
// boundary as it does in memory.
struct RingShape {
  const uint8_t *src[kStreams];
  int64_t ld_bytes[kStreams];
  int row_bytes[kStreams];  // as they lie in a slot, a multiple of 16; 0: not in the ring
  int copy_bytes[kStreams];
  int elt[kStreams];
  int slot_bytes, slots, height, threads;  // threads of a row
  int padded;               // zeros follow a row up to the columns of all its threads
};

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}
// Bytes that a row lies behind a 16-byte boundary, and of it: before the first boundary, and behind the last.
__device__ __forceinline__ int offset_of(const uint8_t *p) { return static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u); }
struct Ends {
  int head, body;
  __device__ __forceinline__ Ends(int offset, int bytes) {
    head = min(bytes, (16 - offset) & 15);
    body = (bytes - head) & ~15;
  }
};

// Fills the ring, a warp's work: batches blockIdx.x, + gridDim.x, ... in turn. What lies between 16-byte boundaries goes by
// bulk copies, a lane for each row of each stream. WIDE: that is all, and the CTA's first warp does it beside its rows, once
// every warp has left the slot (a warp of its own for it would leave the others 96 registers a thread instead of 128).
// Else the rows' ends follow by single elements, which is waited for, so a warp of its own does it.
template <bool WIDE>
struct Filler {
  uint32_t issued = 0, last = 0;  // per slot: whether copies were issued, the parity of the last
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ bool fill(const RingShape &ring, RingBarriers *bar, uint8_t *slots, int64_t rows, int64_t b,
                                       const Waiter &w) {
    if (b * ring.height >= rows) return false;
    if (!warp_mbar_wait<false>(&bar->empty[slot], parity ^ 1u, w)) return false;
    __syncwarp();
    const int lane = threadIdx.x & 31;
    const int n = static_cast<int>(min(static_cast<int64_t>(ring.height), rows - b * ring.height));
    uint8_t *to = slots + slot * ring.slot_bytes;
    uint32_t bytes = 0;
    if (lane < n) {
#pragma unroll
      for (int q = 0; q < kStreams; ++q)
        if (ring.row_bytes[q]) {
          if constexpr (WIDE)
            bytes += ring.copy_bytes[q];
          else
            bytes += Ends(offset_of(ring.src[q] + (b * ring.height + lane) * ring.ld_bytes[q]), ring.copy_bytes[q]).body;
        }
    }
    bytes = __reduce_add_sync(0xffffffffu, bytes);
    if constexpr (!WIDE) {
      // the ends: 16 lanes a row and stream, those before and those behind
      uint8_t *row = to;
#pragma unroll
      for (int q = 0; q < kStreams; ++q) {
        if (!ring.row_bytes[q]) continue;
        for (int r0 = 0; r0 < n; r0 += 2) {
          const int r = r0 + lane / 16, l = lane & 15, elt = ring.elt[q];
          if (r < n) {
            const uint8_t *from = ring.src[q] + (b * ring.height + r) * ring.ld_bytes[q];
            const int offset = offset_of(from);
            const Ends ends(offset, ring.copy_bytes[q]);
            const int at = l < 8 ? l * elt : ends.head + ends.body + (l - 8) * elt;
            uint8_t *dst = row + r * ring.row_bytes[q] + offset + at;
            if (l < 8 ? at < ends.head : at < ring.copy_bytes[q]) {
              if (elt == 2)
                *reinterpret_cast<uint16_t *>(dst) = *reinterpret_cast<const uint16_t *>(from + at);
              else
                *reinterpret_cast<uint32_t *>(dst) = *reinterpret_cast<const uint32_t *>(from + at);
            }
          }
        }
        row += ring.height * ring.row_bytes[q];
      }
      // rows start at other places of a 16-byte word when a slot is used again: copies may fall on ends written for its last rows
      fence_proxy_async_shared();
      __syncwarp();
    }
    if (lane == 0) mbar_arrive_expect_tx(&bar->full[slot], bytes);
    __syncwarp();
    // a lane for each row of each stream
    const int q = lane % kStreams, r = lane / kStreams;
    if (r < n && ring.row_bytes[q]) {
      const uint8_t *from = ring.src[q] + (b * ring.height + r) * ring.ld_bytes[q];
      uint8_t *dst = to + r * ring.row_bytes[q];
#pragma unroll
      for (int k = 0; k < kStreams; ++k)
        if (k < q) dst += ring.height * ring.row_bytes[k];
      if constexpr (WIDE) {
        bulk_load(dst, from, static_cast<uint32_t>(ring.copy_bytes[q]), &bar->full[slot]);
      } else {
        const int offset = offset_of(from);
        const Ends ends(offset, ring.copy_bytes[q]);
        if (ends.body) bulk_load(dst + offset + ends.head, from + ends.head, static_cast<uint32_t>(ends.body), &bar->full[slot]);
      }
    }
    issued |= 1u << slot;
    last = (last & ~(1u << slot)) | (parity << slot);
    if (++slot == ring.slots) {
      slot = 0;
      parity ^= 1u;
    }
    return true;
  }
  __device__ __forceinline__ void first(const RingShape &ring, RingBarriers *bar, uint8_t *slots, int64_t rows, const Waiter &w) {
    for (int s = 0; s < ring.slots; ++s) fill(ring, bar, slots, rows, blockIdx.x + static_cast<int64_t>(s) * gridDim.x, w);
  }
  __device__ __forceinline__ void all(const RingShape &ring, RingBarriers *bar, uint8_t *slots, int64_t rows, const Waiter &w) {
    for (int64_t b = blockIdx.x; fill(ring, bar, slots, rows, b, w);) b += gridDim.x;
    end(ring, bar, w);
  }
  // after an abort: what was issued lands before the CTA ends
  __device__ __forceinline__ void end(const RingShape &ring, RingBarriers *bar, const Waiter &w) {
    if ((threadIdx.x & 31) == 0 && *w.abort)
      for (int s = 0; s < ring.slots; ++s)
        if ((issued >> s) & 1u) drain_wait(&bar->full[s], (last >> s) & 1u, w.limit_ns);
  }
};
// 16 warps at most, so that a thread has 128 registers (96 for ragged rows of more than 2 packs a thread)
constexpr int kRowThreads = 512, kRaggedRowThreads = 480;
template <bool WIDE, int NP> constexpr int kMostThreads = WIDE || NP <= 2 ? 512 : 544;

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
// One stream's row of this thread: in the slot at `at`, or in memory where the ring has no room for the stream. WIDE rows
// in the ring are followed by zeros up to the columns of all threads.
template <int DT, bool WIDE, int Q>
struct StreamRow {
  int place;  // in a slot
  __device__ __forceinline__ StreamRow(const RingShape &ring, int group) {
    place = group * ring.row_bytes[Q];
#pragma unroll
    for (int k = 0; k < Q; ++k) place += ring.height * ring.row_bytes[k];
  }
  __device__ __forceinline__ void load(const RingShape &ring, const uint8_t *at, uint32_t t, int c, int cols, Eight2 &o) const {
    const uint8_t *src = ring.src[Q] + t * ring.ld_bytes[Q];
    if (!ring.row_bytes[Q])
      load8<DT, WIDE>(src, c, cols, o);
    else
      load8<DT, WIDE, true>(at + place + (WIDE ? 0 : offset_of(src)), c, cols, o);
  }
};

__device__ __forceinline__ RingBarriers *start_ring(const RingShape &ring, uint8_t *smem) {
  RingBarriers *bar = reinterpret_cast<RingBarriers *>(smem);
  if (ring.padded) {  // the zeros behind rows, where copies never write
    uint8_t *slots = smem + (static_cast<int>(sizeof(RingBarriers)) + 127) / 128 * 128;
    for (int s = 0; s < ring.slots; ++s) {
      uint8_t *row = slots + s * ring.slot_bytes;
      for (int q = 0; q < kStreams; ++q)
        for (int r = 0; r < ring.height && ring.row_bytes[q]; ++r, row += ring.row_bytes[q])
          for (int i = ring.copy_bytes[q] + static_cast<int>(threadIdx.x) * 16; i < ring.row_bytes[q]; i += blockDim.x * 16)
            *reinterpret_cast<uint4 *>(row + i) = make_uint4(0, 0, 0, 0);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // bulk copies follow
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < ring.slots; ++s) {
      mbar_init(&bar->full[s], 1);
      mbar_init(&bar->empty[s], ring.threads * ring.height / 32);
    }
    bar->abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  return bar;
}
constexpr int kRingHead = (static_cast<int>(sizeof(RingBarriers)) + 127) / 128 * 128;

// The columns' weights, [2][NP][2][threads of a row] float4 in shared memory: post * gate of the columns, pre.
template <bool WIDE, int NP>
struct ColumnWeights {
  float4 *at;
  int threads;
  __device__ __forceinline__ void keep(const NormParams &p, const int (&c)[NP]) const {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      Eight2 f, g;
      load_any<WIDE>(p.post, p.weight_type, c[i], p.cols, f);
      load_any<WIDE>(p.gate_form == kGateCols ? p.gate : nullptr, p.gate_type, c[i], p.cols, g);
#pragma unroll
      for (int j = 0; j < 4; ++j) f.v[j] = __fmul2_rn(f.v[j], g.v[j]);
      put(0, i, f);
      load_any<WIDE>(p.pre, p.weight_type, c[i], p.cols, f);
      put(1, i, f);
    }
  }
  __device__ __forceinline__ void put(int k, int i, const Eight2 &f) const {
    float4 *to = at + (k * NP + i) * 2 * threads;
    to[0] = make_float4(f.v[0].x, f.v[0].y, f.v[1].x, f.v[1].y);
    to[threads] = make_float4(f.v[2].x, f.v[2].y, f.v[3].x, f.v[3].y);
  }
  __device__ __forceinline__ void get(int k, int i, Eight2 &f) const {
    const float4 *from = at + (k * NP + i) * 2 * threads;
    const float4 l = from[0], h = from[threads];
    f.v[0] = make_float2(l.x, l.y);
    f.v[1] = make_float2(l.z, l.w);
    f.v[2] = make_float2(h.x, h.y);
    f.v[3] = make_float2(h.z, h.w);
  }
};
// Where shared memory has no room for them they are read again for each row.
template <bool WIDE, int NP>
__device__ __forceinline__ void weights_of(const NormParams &p, const ColumnWeights<WIDE, NP> &held, int k, int i, int c, Eight2 &f) {
  if (p.hold) {
    held.get(k, i, f);
  } else if (k == 1) {
    load_any<WIDE>(p.pre, p.weight_type, c, p.cols, f);
  } else {
    Eight2 g;
    load_any<WIDE>(p.post, p.weight_type, c, p.cols, f);
    load_any<WIDE>(p.gate_form == kGateCols ? p.gate : nullptr, p.gate_type, c, p.cols, g);
#pragma unroll
    for (int j = 0; j < 4; ++j) f.v[j] = __fmul2_rn(f.v[j], g.v[j]);
  }
}

// Threads of a row, packs a thread, rows that a CTA has in hand at once (so that some compute while others wait for their
// sums), and the ring: as many slots as leave room for `per_sm` CTAs on an SM, two at least where that is possible. dr is
// left out where the others then get two slots; a stream for which there is no room at all is read past the ring.
struct Shape {
  int threads, packs, rows, per_sm, smem, hold;
  RingShape ring{};
  Shape(const NormParams &p, bool backward, bool wide, int xt, int yt, int sms) {
    const int lanes = (p.cols + 7) / 8, most = wide ? kRowThreads : kRaggedRowThreads;
    // backward has registers for the columns' sums of 2 packs; forward, ragged rows of 4 packs spill (4001 x 4099 bf16:
    // 74 us against 62 for 2 packs; 1171 x 7001, fp32 block: 42 against 27)
    packs = lanes <= 256 ? 1 : lanes <= (backward || !wide ? 2 * most : 512) ? 2 : 4;
    threads = ((lanes + packs - 1) / packs + 31) / 32 * 32;
    rows = std::max(1, std::min(kMaxHeight, most / threads));
    // narrow rows: CTAs of half the threads that an SM has registers for, so that two stay
    if (packs == 1) rows = std::max(1, std::min(rows, (wide ? 256 : 224) / threads));
    ring.height = rows;
    ring.threads = threads;
    // backward reads X for the norm of r alone
    const void *src[kStreams] = {backward && !p.pre ? nullptr : p.x, p.y, backward && p.pre ? p.dz : nullptr, backward ? p.dr : nullptr};
    const int64_t ld[kStreams] = {p.ld_x, p.ld_y, p.ld_dz, p.ld_dr};
    const int xe = xt == kBF16 ? 2 : 4, ye = yt == kBF16 ? 2 : 4, elt[kStreams] = {xe, ye, ye, xe};
    int bytes[kStreams];
    for (int q = 0; q < kStreams; ++q) {
      ring.src[q] = static_cast<const uint8_t *>(src[q]);
      ring.ld_bytes[q] = ld[q] * elt[q];
      ring.copy_bytes[q] = p.cols * elt[q];
      ring.elt[q] = elt[q];
      bytes[q] = !src[q] ? 0 : wide ? threads * packs * 8 * elt[q] : (p.cols * elt[q] + 31) / 16 * 16;
    }
    const int sums = backward ? 2 * packs * 8 * threads * rows * 4 : 0;
    const int weights = 2 * packs * 8 * threads * 4, extra = backward && packs > 2 ? sums : 0;
    const int room = 224 * 1024 - kRingHead - 2048;  // with the kernel's own
    auto slot_of = [&](int n) {
      int v = 0;
      for (int q = 0; q < n; ++q) v += bytes[q] * rows;
      return v;
    };
    // a call of no rows may have no stream at all (their pointers are null), and one stream may be read past the ring: slots
    // are empty then, but there is no dividing by 0
    auto slots_in = [](int space, int slot) { return space / std::max(1, slot); };
    // weights that a CTA uses for one batch or two are as well read where they lie
    hold = slot_of(2) + weights + extra <= room && p.rows > 2 * static_cast<int64_t>(rows) * sms ? 1 : 0;
    const int beside = extra + hold * weights;
    int streams = kStreams;
    if (slots_in(room - beside, slot_of(4)) < 2 && slots_in(room - beside, slot_of(3)) >= 2) streams = 3;
    while (streams > 1 && slot_of(streams) + beside > room) --streams;
    for (int q = 0; q < streams; ++q) ring.row_bytes[q] = bytes[q];
    ring.slot_bytes = slot_of(streams);
    ring.padded = wide && p.cols < threads * packs * 8;
    for (per_sm = packs == 1 ? 4 : 2; per_sm > 1; --per_sm)
      if (slots_in(room / per_sm - kRingHead - 2048 - beside, ring.slot_bytes) >= 2) break;
    // backward takes up to 128 registers a thread, forward less for one pack
    per_sm = std::max(1, std::min(per_sm, (backward ? 512 : packs == 1 ? 1024 : 512) / block(wide)));
    const int mine = per_sm == 1 ? room : room / per_sm - kRingHead - 2048;
    ring.slots = std::max(1, std::min(kMaxSlots, slots_in(mine - beside, ring.slot_bytes)));
    smem = kRingHead + std::max(ring.slots * ring.slot_bytes + beside, sums);
  }
  int block(bool wide) const { return threads * rows + (wide ? 0 : 32); }
  int64_t batches(int64_t n) const { return (n + rows - 1) / rows; }
};

template <typename F>
int by_packs(int packs, F &&f) {
  return packs == 1 ? f(std::integral_constant<int, 1>{}) : packs == 2 ? f(std::integral_constant<int, 2>{})
                      : f(std::integral_constant<int, 4>{});
}
template <typename F>
int by_types(int xt, int yt, bool wide, F &&f) {
  using B = std::integral_constant<int, kBF16>;
  using S = std::integral_constant<int, kF32>;
  if (xt == kBF16) return wide ? f(B{}, B{}, std::true_type{}) : f(B{}, B{}, std::false_type{});
  if (yt == kBF16) return wide ? f(S{}, B{}, std::true_type{}) : f(S{}, B{}, std::false_type{});
  return wide ? f(S{}, S{}, std::true_type{}) : f(S{}, S{}, std::false_type{});
}

inline bool bad_type(int t) { return t != NS_F32 && t != NS_BF16; }
inline int size_of(int t) { return t == NS_BF16 ? 2 : 4; }
// The checks that both directions share; fills p. `written`: ranges of the outputs to come are checked by the caller.
inline int check(NormParams &p, const void *x, int64_t ld_x, const void *y, int64_t ld_y, const void *gate, int gate_form,
          int64_t ld_gate, const void *post, const void *pre, int64_t rows, int64_t cols, float a, float b, int dtype,
          int block_dtype, int weight_dtype, int gate_dtype) {
  if (bad_type(dtype) || bad_type(block_dtype) || bad_type(weight_dtype) || bad_type(gate_dtype)) return NS_EINVAL;
  if (dtype == NS_BF16 && block_dtype == NS_F32) return NS_EINVAL;  // a residual narrower than the block's output
  if (bad_shape(rows, cols, ld_x) || cols > kMaxCols || gate_form < kGateNone || gate_form > kGateFull) return NS_EINVAL;
  if (!std::isfinite(a) || !std::isfinite(b)) return NS_EINVAL;
  if (y && bad_shape(rows, cols, ld_y)) return NS_EINVAL;
  if (rows > 0 && cols > 0) {  // (a null pointer may stand for what is empty)
    if (!y && (gate_form != kGateNone || post)) return NS_EINVAL;
    if (!y && !pre) return NS_EINVAL;  // nothing to do
    if ((gate_form != kGateNone) != (gate != nullptr)) return NS_EINVAL;
  }
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
inline bool packs_fit(const NormParams &p, int dtype, int block_dtype) {
  return p.cols % 8 == 0 && rows_aligned(p.x, p.ld_x, size_of(dtype), 8) && rows_aligned(p.y, p.ld_y, size_of(block_dtype), 8) &&
         !misaligned(p.post, 16) && !misaligned(p.pre, 16) &&
         (p.gate_form == kGateCols ? !misaligned(p.gate, 16)
                                   : p.gate_form != kGateFull || rows_aligned(p.gate, p.ld_gate, size_of(p.gate_type), 8));
}
inline Range gate_range(const void *gate, int form, int64_t rows, int64_t cols, int64_t ld, int type) {
  return form == kGateCols   ? Range(gate, 1, cols, cols, size_of(type))
         : form == kGateRows ? Range(gate, rows, 1, ld, size_of(type))
         : form == kGateFull ? Range(gate, rows, cols, ld, size_of(type))
                             : Range(nullptr, 0, 0, 0, 1);
}

}  // namespace block_norm
}  // namespace ns
