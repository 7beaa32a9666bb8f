// ns_rows.cuh -- row access shared by the training operators (ns_embed.cu,
// ns_policy.cu, ns_ckpt.cu): packs of VEC consecutive elements, loaded and
// stored as one access of up to 16 bytes and held as floats, and token ids of
// either integer type.
#pragma once

#include "ns_device.cuh"

namespace ns {

// One value to `at`, in the buffer of `size` bytes at `base` (debug builds check that).
template <typename T>
__device__ __forceinline__ void put(void *at, T v, const void *base, size_t size, int *status) {
  if (in_bounds(at, sizeof(T), base, size, status)) *static_cast<T *>(at) = v;
}

template <int BYTES> struct Word;
template <> struct Word<2> { using T = uint16_t; };
template <> struct Word<4> { using T = uint32_t; };
template <> struct Word<8> { using T = uint2; };
template <> struct Word<16> { using T = uint4; };

// VEC elements of type DT at p, which is aligned to their size (at most 16
// bytes per access; a wider pack is several accesses).
template <int DT, int VEC>
struct Pack {
  using E = typename Elem<DT>::T;
  static constexpr int kBytes = VEC * static_cast<int>(sizeof(E));
  static constexpr int kAcc = kBytes < 16 ? kBytes : 16;
  static constexpr int kN = kBytes / kAcc;
  using W = typename Word<kAcc>::T;
  W w[kN];

  // read once: keep it out of the way of what is re-read
  __device__ __forceinline__ void load_stream(const E *p) {
#pragma unroll
    for (int i = 0; i < kN; ++i) w[i] = __ldcs(reinterpret_cast<const W *>(p) + i);
  }
  __device__ __forceinline__ void load(const E *p) {
#pragma unroll
    for (int i = 0; i < kN; ++i) w[i] = reinterpret_cast<const W *>(p)[i];
  }
  __device__ __forceinline__ float get(int e) const {
    return Elem<DT>::to_f(reinterpret_cast<const E *>(w)[e]);
  }
  __device__ __forceinline__ void set(int e, float v) { reinterpret_cast<E *>(w)[e] = Elem<DT>::from_f(v); }
  // base, size: the buffer of p (debug builds check the store against it)
  __device__ __forceinline__ void store(E *p, const void *base, size_t size, int *status) const {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (in_bounds(reinterpret_cast<const W *>(p) + i, kAcc, base, size, status)) reinterpret_cast<W *>(p)[i] = w[i];
  }
  // written once and not read again here: first to leave the caches
  __device__ __forceinline__ void store_stream(E *p, const void *base, size_t size, int *status) const {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (in_bounds(reinterpret_cast<const W *>(p) + i, kAcc, base, size, status)) __stcs(reinterpret_cast<W *>(p) + i, w[i]);
  }
};

// The columns of a row that a thread holds, kN of them from its column c on:
// consecutive ones where rows allow packed accesses (WIDE), else every 32nd,
// so that a warp's accesses stay coalesced; beyond the row nothing is read or
// written. first() is c of a thread, for threads numbered along the row.
template <int DT, bool WIDE>
struct RowPart {
  static constexpr int kN = DT == kBF16 ? 8 : 4;
  using E = typename Elem<DT>::T;
  Pack<DT, kN> v;
  static __device__ __forceinline__ int first(int thread) { return WIDE ? thread * kN : (thread / 32) * (32 * kN) + thread % 32; }
  static __device__ __forceinline__ int at(int c, int e) { return WIDE ? c + e : c + 32 * e; }
  // ONCE: not read again, first to leave the caches
  template <bool ONCE>
  __device__ __forceinline__ void load(const E *row, int c, int cols) {
    if constexpr (WIDE) {
      if (ONCE)
        v.load_stream(row + c);
      else
        v.load(row + c);
    } else {
#pragma unroll
      for (int e = 0; e < kN; ++e)
        reinterpret_cast<E *>(v.w)[e] =
            c + 32 * e < cols ? (ONCE ? __ldcs(row + c + 32 * e) : row[c + 32 * e]) : Elem<DT>::from_f(0.f);
    }
  }
  __device__ __forceinline__ float get(int e) const { return v.get(e); }
  __device__ __forceinline__ void set(int e, float x) { v.set(e, x); }
  __device__ __forceinline__ void store(E *row, int c, int cols, const void *base, size_t size, int *status) const {
    if constexpr (WIDE) {
      v.store_stream(row + c, base, size, status);
    } else {
#pragma unroll
      for (int e = 0; e < kN; ++e)
        if (c + 32 * e < cols && in_bounds(row + c + 32 * e, sizeof(E), base, size, status))
          __stcs(row + c + 32 * e, reinterpret_cast<const E *>(v.w)[e]);
    }
  }
};

// Eight consecutive columns of a row per lane, for element-wise kernels whose lanes need neighbours. WIDE: rows that
// allow packs of 8 (whole packs lie in the row or outside). Else a warp's 256 columns from c0 on are read and written
// lane by lane, coalesced, and exchanged through the warp's piece of shared memory, kStage 16-byte words.
template <int DT, bool WIDE>
struct Eight {
  using E = typename Elem<DT>::T;
  static constexpr int kStage = 32 * 8 * static_cast<int>(sizeof(E)) / 16;
  Pack<DT, 8> v;
  // here: the row is to be read (its other columns read as zeros); all lanes of the warp call these
  __device__ __forceinline__ void load(const E *row, int c, int cols, bool here) {
    if constexpr (WIDE) {
      if (here && c < cols) {
        v.load_stream(row + c);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v.set(e, 0.f);
      }
    } else {
      const int lane = threadIdx.x & 31, first = c - lane * 8 + lane;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        reinterpret_cast<E *>(v.w)[e] = here && first + e * 32 < cols ? __ldcs(row + first + e * 32) : Elem<DT>::from_f(0.f);
    }
  }
  __device__ __forceinline__ void settle(uint4 *stage) {
    if constexpr (!WIDE) {
      const int lane = threadIdx.x & 31;
      E *s = reinterpret_cast<E *>(stage);
      constexpr int kW = sizeof(v.w) / 16;
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e * 32 + lane] = reinterpret_cast<const E *>(v.w)[e];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kW; ++i) reinterpret_cast<uint4 *>(v.w)[i] = stage[lane * kW + i];
    }
  }
  __device__ __forceinline__ float get(int e) const { return v.get(e); }
  __device__ __forceinline__ void set(int e, float x) { v.set(e, x); }
  __device__ __forceinline__ void store(E *row, int c, int cols, bool here, uint4 *stage, const void *base, size_t size,
                                        int *status) const {
    if constexpr (WIDE) {
      if (here && c < cols) v.store_stream(row + c, base, size, status);
    } else {
      const int lane = threadIdx.x & 31, first = c - lane * 8 + lane;
      constexpr int kW = sizeof(v.w) / 16;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kW; ++i) stage[lane * kW + i] = reinterpret_cast<const uint4 *>(v.w)[i];
      __syncwarp();
      const E *s = reinterpret_cast<const E *>(stage) + lane;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (here && first + e * 32 < cols && in_bounds(row + first + e * 32, sizeof(E), base, size, status))
          __stcs(row + first + e * 32, s[e * 32]);
    }
  }
};

// How a block of kThreads threads covers rows of 8-column packs: lanes 1 << lanes_log2 to a row (at least
// 1 << least_log2, whole warps where lanes exchange values), kThreads >> lanes_log2 rows at a time, further columns
// by blockIdx.x, walking down the rows by gridDim.y.
struct EightGrid {
  int lanes_log2;
  dim3 grid;
  EightGrid(int64_t rows, int64_t extent, int threads, bool wide, int least_log2, int sms, int per_sm) {
    const int64_t lanes = (extent + 7) / 8;
    lanes_log2 = wide ? least_log2 : 5;
    while ((2 << lanes_log2) <= threads && (1 << lanes_log2) < lanes) ++lanes_log2;
    const int64_t gx = (lanes + (1 << lanes_log2) - 1) >> lanes_log2;
    const int64_t height = threads >> lanes_log2, want = (rows + height - 1) / height;
    int64_t most = static_cast<int64_t>(sms) * per_sm / gx;
    most = most < 1 ? 1 : most > 65535 ? 65535 : most;
    grid = dim3(static_cast<unsigned>(gx), static_cast<unsigned>(want < most ? want : most), 1);
  }
};

// Token ids: int32 or int64; anything outside [0, vocab) becomes -1.
struct Ids {
  const void *p;
  int wide;
  int vocab;
  __device__ __forceinline__ int get(int64_t i) const {
    const long long v = wide ? static_cast<const long long *>(p)[i] : static_cast<const int *>(p)[i];
    return v >= 0 && v < vocab ? static_cast<int>(v) : -1;
  }
};

// Whether rows of `ld` elements of `elt` bytes starting at p can be accessed
// in packs of `vec` elements (packs above 16 bytes take several accesses).
inline bool rows_aligned(const void *p, int64_t ld, int elt, int vec) {
  const int b = elt * vec < 16 ? elt * vec : 16;
  return reinterpret_cast<uintptr_t>(p) % b == 0 && (ld * elt) % b == 0;
}

}  // namespace ns
