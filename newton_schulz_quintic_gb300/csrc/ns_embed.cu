// ns_embed.cu -- token embedding of the training operators (include/ns.h):
// ns_embed_lookup and the table's gradient ns_embed_grad.
//
// The gradient is a sum over positions grouped by token id. Atomic adds into
// the table would make the sums depend on the schedule (and serialise on the
// few very frequent ids of real text), so each id's rows are added in the
// order of their positions.
//   few positions (kDirect): one launch. A CTA per position and column range
//     finds the positions with the same id in the list itself; the first of
//     them adds them all.
//   else: sort      one cluster of 8 CTAs, a stable radix sort of (id,
//                   position); padding ids sort to the end;
//         segments  the sorted list in equal pieces of positions, one
//                   piece and column range per CTA, whatever the ids are: a
//                   run of equal ids inside a piece is written to the table,
//                   the parts of a run that crosses piece borders go to
//                   scratch as fp32 sums;
//         joins     adds the parts of each crossing run in piece order.
// Not accumulating, the rows that no id points to are cleared by the other
// CTAs of the first launch, which find them from the ids directly (a bitmap of
// their rows): most of the bytes of a large vocabulary, written while the sort
// (25 us for 32768 ids) runs beside them.
//
// Bound by HBM for long batches. 32768 ids of a 131072 x 4096 bf16 table: lookup
// 60 us, 6.0 TB/s (91 % of the copy rate); gradient 238 us, 5.6 TB/s (launches of
// 157, 54 and 15 us; sort, segments, joins and clearing one after the other:
// 290). 509 ids: 10 us, by latency.
#include <algorithm>

#include "../../include/ns.h"
#include "ns_rows.cuh"

namespace ns {

namespace {

// ------------------------------------------------------------------ lookup
struct LookupParams {
  const void *table;
  void *out;
  Ids ids;
  int64_t count, ld_table, ld_out;
  int dim;
  float scale;
  int *status;
};

constexpr int kLookupPacks = 4;  // packs a lane has in flight

// One warp per (row, stretch of 32 * kLookupPacks packs).
template <int DT, bool WIDE>
__global__ void __launch_bounds__(256) ns_embed_lookup_kernel(const __grid_constant__ LookupParams p) {
  using R = RowPart<DT, WIDE>;
  using E = typename R::E;
  constexpr int kSpan = 32 * kLookupPacks * R::kN;
  const int per_row = (p.dim + kSpan - 1) / kSpan;
  const int64_t items = p.count * per_row;
  const size_t size = static_cast<size_t>((p.count - 1) * p.ld_out + p.dim) * sizeof(E);
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); it < items;
       it += static_cast<int64_t>(gridDim.x) * 8) {
    const int64_t t = it / per_row;
    const int c0 = static_cast<int>(it - t * per_row) * kSpan + R::first(threadIdx.x & 31);
    const int id = p.ids.get(t);
    const E *src = static_cast<const E *>(p.table) + static_cast<int64_t>(id < 0 ? 0 : id) * p.ld_table;
    E *dst = static_cast<E *>(p.out) + t * p.ld_out;
    R v[kLookupPacks];
#pragma unroll
    for (int k = 0; k < kLookupPacks; ++k) {
      const int c = c0 + k * 32 * R::kN;
      if (id >= 0 && c < p.dim) v[k].template load<false>(src, c, p.dim);
    }
#pragma unroll
    for (int k = 0; k < kLookupPacks; ++k) {
      const int c = c0 + k * 32 * R::kN;
      if (c >= p.dim) continue;
#pragma unroll
      for (int e = 0; e < R::kN; ++e) v[k].set(e, id >= 0 ? v[k].get(e) * p.scale : 0.f);
      v[k].store(dst, c, p.dim, p.out, size, p.status);
    }
  }
}

// ------------------------------------------------------------------ absent rows
struct ZeroParams {
  Ids ids;
  int n;
  uint8_t *grad;
  int64_t ld_bytes;
  int row_bytes;
  size_t size;
  int *status;
};

constexpr int kZeroRows = 16384;  // rows of a bitmap
struct Bitmap {
  uint32_t w[kZeroRows / 32];
};

// The calling CTA, `part` of `parts`, clears those rows of its share of the
// table that no id points to.
__device__ __forceinline__ void zero_absent(const ZeroParams &p, Bitmap &seen, int part, int parts) {
  // lanes per row: a 16-byte word each as far as a row goes, 4 to 32
  int lanes = 4;
  while (lanes < 32 && lanes * 16 < p.row_bytes) lanes *= 2;
  const int lane = threadIdx.x & (lanes - 1);
  const int64_t vocab = p.ids.vocab;
  const int64_t r0 = vocab * part / parts, r1 = vocab * (part + 1) / parts;
  for (int64_t a = r0; a < r1; a += kZeroRows) {
    const int rows = static_cast<int>(min(static_cast<int64_t>(kZeroRows), r1 - a));
    for (int i = threadIdx.x; i < kZeroRows / 32; i += blockDim.x) seen.w[i] = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = threadIdx.x; i < p.n; i += blockDim.x) {
      const int64_t d = p.ids.get(i) - a;
      if (d >= 0 && d < rows) atomicOr(&seen.w[d >> 5], 1u << (d & 31));
    }
    __syncthreads();
    for (int r = threadIdx.x / lanes; r < rows; r += blockDim.x / lanes) {
      if ((seen.w[r >> 5] >> (r & 31)) & 1u) continue;
      // 2- or 4-byte elements up to a 16-byte boundary, whole 16-byte words, the rest
      uint8_t *row = p.grad + (a + r) * p.ld_bytes, *end = row + p.row_bytes;
      uint8_t *lo = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(row) + 15) & ~uintptr_t(15));
      uint8_t *hi = reinterpret_cast<uint8_t *>(reinterpret_cast<uintptr_t>(end) & ~uintptr_t(15));
      if (lo > hi) lo = hi = end;
      for (uint8_t *at = lo + lane * 16; at < hi; at += lanes * 16)
        if (in_bounds(at, 16, p.grad, p.size, p.status)) __stcs(reinterpret_cast<uint4 *>(at), make_uint4(0, 0, 0, 0));
      for (uint8_t *at = row + lane * 2; at < lo; at += lanes * 2)
        if (in_bounds(at, 2, p.grad, p.size, p.status)) *reinterpret_cast<uint16_t *>(at) = 0;
      for (uint8_t *at = hi + lane * 2; at < end; at += lanes * 2)
        if (in_bounds(at, 2, p.grad, p.size, p.status)) *reinterpret_cast<uint16_t *>(at) = 0;
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ sort
constexpr int kSortCluster = 8;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortRounds = 4;                                 // keys per thread and tile
constexpr int kSortTile = kSortThreads * kSortRounds;
constexpr int kSortBins = 512;                                 // 9 bits a pass at most

struct SortParams {
  Ids ids;
  int n;
  int bits, passes;      // digit width and number of passes
  int *keys[2], *pos[2];  // ping-pong; the last pass writes [0]
  int *status;
};

// Stable least-significant-digit radix sort by one cluster. Each CTA owns a
// contiguous share of the list. Per pass: every CTA counts its share's
// digits; the counts are exchanged through distributed shared memory, which
// gives each CTA where its keys of each digit go; then the share is ranked
// tile by tile: within a warp by matching digits, across warps by a prefix
// over the warps' counts, so equal digits keep their order.
// The clusters behind the first one clear the absent rows.
__global__ void __launch_bounds__(kSortThreads)
    ns_embed_sort_kernel(const __grid_constant__ SortParams p, const __grid_constant__ ZeroParams zero) {
  if (blockIdx.x >= kSortCluster) {
    __shared__ Bitmap seen;
    zero_absent(zero, seen, blockIdx.x - kSortCluster, gridDim.x - kSortCluster);
    return;
  }
  __shared__ int hist[kSortBins];
  __shared__ int base[kSortBins];
  __shared__ int wsum[kSortWarps];
  __shared__ uint16_t wcount[kSortWarps][kSortBins];
  const int rank = static_cast<int>(cluster_ctarank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int share = (p.n + kSortCluster - 1) / kSortCluster;
  const int lo = min(p.n, rank * share), hi = min(p.n, lo + share);
  const int bins = 1 << p.bits;
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.bits;
    const int to = (p.passes - 1 - pass) & 1, from = to ^ 1;
    auto key_at = [&](int i) {
      if (pass) return __ldcg(p.keys[from] + i);
      const int id = p.ids.get(i);
      return id < 0 ? p.ids.vocab : id;
    };
    for (int d = threadIdx.x; d < kSortBins; d += kSortThreads) hist[d] = 0;
    __syncthreads();
    for (int i = lo + threadIdx.x; i < hi; i += kSortThreads) atomicAdd(&hist[(key_at(i) >> shift) & (bins - 1)], 1);
    cluster_sync();
    // base[d] = keys of smaller digits anywhere + keys of digit d in lower shares
    int total = 0, before = 0;
    if (threadIdx.x < bins) {
#pragma unroll
      for (int c = 0; c < kSortCluster; ++c) {
        const int v = static_cast<int>(ld_shared_cluster_u32(mapa_shared(smem_u32(&hist[threadIdx.x]), c)));
        total += v;
        before += c < rank ? v : 0;
      }
    }
    int scan = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += v;
    }
    if (lane == 31) wsum[warp] = scan;
    __syncthreads();
    if (warp == 0) {
      int v = wsum[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      wsum[lane] = v;
    }
    __syncthreads();
    if (threadIdx.x < bins) base[threadIdx.x] = scan - total + (warp ? wsum[warp - 1] : 0) + before;
    for (int t0 = lo; t0 < hi; t0 += kSortTile) {
      __syncthreads();
      for (int i = threadIdx.x; i < kSortWarps * kSortBins / 2; i += kSortThreads)
        reinterpret_cast<uint32_t *>(&wcount[0][0])[i] = 0;
      __syncthreads();
      int key[kSortRounds], at[kSortRounds], loc[kSortRounds];
#pragma unroll
      for (int r = 0; r < kSortRounds; ++r) {
        const int i = t0 + warp * (32 * kSortRounds) + r * 32 + lane;
        key[r] = i < hi ? key_at(i) : -1;
        at[r] = i < hi ? (pass ? __ldcg(p.pos[from] + i) : i) : 0;
      }
#pragma unroll
      for (int r = 0; r < kSortRounds; ++r) {
        const bool live = key[r] >= 0;
        const int d = (key[r] >> shift) & (bins - 1);
        const uint32_t peers = __match_any_sync(0xffffffffu, live ? d : -1);
        const int seen = live ? wcount[warp][d] : 0;
        loc[r] = seen + __popc(peers & ((1u << lane) - 1));
        __syncwarp();
        if (live && (peers >> lane) == 1u) wcount[warp][d] = static_cast<uint16_t>(seen + __popc(peers));
        __syncwarp();
      }
      __syncthreads();
      int tile_total = 0;
      if (threadIdx.x < bins) {
        for (int w = 0; w < kSortWarps; ++w) {
          const int v = wcount[w][threadIdx.x];
          wcount[w][threadIdx.x] = static_cast<uint16_t>(tile_total);
          tile_total += v;
        }
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < kSortRounds; ++r) {
        if (key[r] < 0) continue;
        const int d = (key[r] >> shift) & (bins - 1);
        const int dst = base[d] + wcount[warp][d] + loc[r];
        if (in_bounds(p.keys[to] + dst, 4, p.keys[to], static_cast<size_t>(p.n) * 4, p.status)) {
          p.keys[to][dst] = key[r];
          p.pos[to][dst] = at[r];
        }
      }
      __syncthreads();
      if (threadIdx.x < bins) base[threadIdx.x] += tile_total;
    }
    cluster_sync();  // the pass's output is complete and every histogram read
  }
}

// ------------------------------------------------------------------ segment sums
constexpr int kSegMost = 64;     // sorted positions per piece at most, and
constexpr int kSegLeast = 16;    // at least (see run_segments)
constexpr int kSegThreads = 128;
constexpr int kSegAhead = 8;     // rows in flight per thread
constexpr int kJoinAhead = 16;   // parts in flight per thread

// CTAs that cover a row, with packs of vec elements per thread.
inline int chunks_of(int dim, int vec) { return (dim + kSegThreads * vec - 1) / (kSegThreads * vec); }

struct GradParams {
  const void *dout;
  void *grad;
  const int *keys, *pos;  // sorted; keys == vocab is padding
  float *parts;           // [piece][2][dim_pad]: the piece's share of the run that enters it / leaves it
  int64_t ld_dout, ld_grad;
  int n, vocab, dim, dim_pad, pieces;
  int seg;                // sorted positions per piece
  int chunks;             // column ranges per piece (one CTA each)
  float scale;
  int accumulate;
  int *status;
};

// The sums of a thread's columns into row id of the table; the columns are
// those of RowPart<DT, WIDE>, of kN sums, whatever the table's type is.
template <int GT, bool WIDE, int N>
__device__ __forceinline__ void write_row(const GradParams &p, int id, int c, const float (&sum)[N]) {
  using G = typename Elem<GT>::T;
  G *row = static_cast<G *>(p.grad) + static_cast<int64_t>(id) * p.ld_grad;
  const size_t size = static_cast<size_t>((p.vocab - 1) * p.ld_grad + p.dim) * sizeof(G);
  if constexpr (WIDE) {
    Pack<GT, N> v;
    if (p.accumulate) v.load(row + c);
#pragma unroll
    for (int e = 0; e < N; ++e) v.set(e, p.accumulate ? fmaf(p.scale, sum[e], v.get(e)) : p.scale * sum[e]);
    v.store(row + c, p.grad, size, p.status);
  } else {
    G old[N];
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (p.accumulate && c + 32 * e < p.dim) old[e] = row[c + 32 * e];
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (c + 32 * e < p.dim && in_bounds(row + c + 32 * e, sizeof(G), p.grad, size, p.status))
        row[c + 32 * e] = Elem<GT>::from_f(p.accumulate ? fmaf(p.scale, sum[e], Elem<GT>::to_f(old[e])) : p.scale * sum[e]);
  }
}

template <int DT, int GT, bool WIDE>
__global__ void __launch_bounds__(kSegThreads) ns_embed_segments_kernel(const __grid_constant__ GradParams p) {
  using R = RowPart<DT, WIDE>;
  using E = typename R::E;
  constexpr int kN = R::kN;
  __shared__ int key[kSegMost + 2];  // with the neighbours on either side
  __shared__ int at[kSegMost];
  const int piece = blockIdx.x / p.chunks, chunk = blockIdx.x - piece * p.chunks;
  const int i0 = piece * p.seg;
  const int len = min(p.seg, p.n - i0);
  if (threadIdx.x < p.seg + 2) {
    const int i = i0 - 1 + static_cast<int>(threadIdx.x);
    key[threadIdx.x] = i >= 0 && i < p.n ? p.keys[i] : -1;
    if (threadIdx.x < len) at[threadIdx.x] = p.pos[i0 + threadIdx.x];
  }
  __syncthreads();
  const int c = R::first(chunk * kSegThreads + threadIdx.x);
  if (c >= p.dim) return;
  float sum[kN];
#pragma unroll
  for (int e = 0; e < kN; ++e) sum[e] = 0.f;
  const E *src = static_cast<const E *>(p.dout);
  float *parts = p.parts + static_cast<int64_t>(piece) * 2 * p.dim_pad;
  bool entered = key[0] == key[1];  // the current run began in an earlier piece
  for (int k0 = 0; k0 < len; k0 += kSegAhead) {
    R v[kSegAhead];
#pragma unroll
    for (int k = 0; k < kSegAhead; ++k)
      if (k0 + k < len && key[k0 + k + 1] < p.vocab) v[k].template load<true>(src + static_cast<int64_t>(at[k0 + k]) * p.ld_dout, c, p.dim);
#pragma unroll
    for (int k = 0; k < kSegAhead; ++k) {
      const int i = k0 + k;
      if (i >= len) break;
      const int id = key[i + 1];
      if (id >= p.vocab) break;  // padding: the rest of the list
#pragma unroll
      for (int e = 0; e < kN; ++e) sum[e] += v[k].get(e);
      const bool ends = key[i + 2] != id;
      if (ends || i == len - 1) {
        if (ends && !entered) {
          write_row<GT, WIDE>(p, id, c, sum);
        } else {
          float *to = parts + (entered ? 0 : p.dim_pad);
#pragma unroll
          for (int e = 0; e < kN; ++e) {
            float *at_e = to + R::at(c, e);
            if (R::at(c, e) < p.dim && in_bounds(at_e, 4, p.parts, static_cast<size_t>(p.pieces) * 2 * p.dim_pad * 4, p.status))
              *at_e = sum[e];
          }
        }
#pragma unroll
        for (int e = 0; e < kN; ++e) sum[e] = 0.f;
        entered = false;
      }
    }
  }
}

// The run that leaves a piece having begun in it: its share there, the whole
// pieces it fills and its share of the piece where it ends.
template <int GT, int VEC>
__global__ void __launch_bounds__(kSegThreads) ns_embed_joins_kernel(const __grid_constant__ GradParams p) {
  const int b = blockIdx.x / p.chunks;
  const int last = (b + 1) * p.seg - 1;
  if (last + 1 >= p.n) return;
  const int id = p.keys[last];
  if (id >= p.vocab || p.keys[last + 1] != id) return;              // nothing leaves
  if (b > 0 && p.keys[b * p.seg] == id && p.keys[b * p.seg - 1] == id) return;  // began earlier
  // pieces b + 1 .. q begin with it: the CTA looks at kSegThreads of them at a time
  int q = b;
  for (int more = kSegThreads; more == kSegThreads;) {
    const int64_t i = static_cast<int64_t>(q + 1 + static_cast<int>(threadIdx.x)) * p.seg;
    more = __syncthreads_count(i < p.n && p.keys[i] == id);
    q += more;
  }
  const int c = ((blockIdx.x - b * p.chunks) * kSegThreads + threadIdx.x) * VEC;
  if (c >= p.dim) return;
  const float *parts = p.parts + static_cast<int64_t>(b) * 2 * p.dim_pad + c;
  float sum[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) sum[e] = parts[p.dim_pad + e];
  for (int k0 = b + 1; k0 <= q; k0 += kJoinAhead) {
    float v[kJoinAhead][VEC];
#pragma unroll
    for (int k = 0; k < kJoinAhead; ++k) {
      const float *at = parts + static_cast<int64_t>(min(k0 + k, q) - b) * 2 * p.dim_pad;
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[k][e] = at[e];  // parts are 16-byte aligned: one access
    }
#pragma unroll
    for (int k = 0; k < kJoinAhead; ++k)
      if (k0 + k <= q) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) sum[e] += v[k][e];
      }
  }
  write_row<GT, (VEC > 1)>(p, id, c, sum);
}

// ------------------------------------------------------------------ few positions
constexpr int kDirect = 1024;  // positions at most (the words of a list of matches are one per lane)

// CTAs [0, n * chunks): position t and a column range. The first position of
// an id adds the rows of all its positions; the list of them is a bitmap, so
// they come in order. The CTAs behind clear the absent rows.
template <int DT, int GT, bool WIDE>
__global__ void __launch_bounds__(kSegThreads)
    ns_embed_direct_kernel(const __grid_constant__ GradParams p, const __grid_constant__ ZeroParams zero) {
  using R = RowPart<DT, WIDE>;
  using E = typename R::E;
  constexpr int kN = R::kN;
  const int work = p.n * p.chunks;
  if (blockIdx.x >= work) {
    __shared__ Bitmap seen;
    zero_absent(zero, seen, blockIdx.x - work, gridDim.x - work);
    return;
  }
  __shared__ uint32_t match[kDirect / 32];
  const int t = blockIdx.x / p.chunks, chunk = blockIdx.x - t * p.chunks;
  const int id = zero.ids.get(t);
  if (id < 0) return;
  bool earlier = false;
  for (int i = threadIdx.x; i < kDirect; i += kSegThreads) {  // whole warps, a word each
    const bool same = i < p.n && zero.ids.get(i) == id;
    const uint32_t word = __ballot_sync(0xffffffffu, same);
    if ((threadIdx.x & 31) == 0) match[i >> 5] = word;
    earlier |= same && i < t;
  }
  if (__syncthreads_or(earlier)) return;
  const int c = R::first(chunk * kSegThreads + threadIdx.x);
  if (c >= p.dim) return;
  float sum[kN];
#pragma unroll
  for (int e = 0; e < kN; ++e) sum[e] = 0.f;
  const E *src = static_cast<const E *>(p.dout);
  int word = t >> 5;
  uint32_t left = match[word];
  const int words = (p.n + 31) >> 5;
  auto next = [&] {  // the next position with this id, -1 behind the last
    while (left == 0) {
      if (++word >= words) return -1;
      left = match[word];
    }
    const int i = (word << 5) + __ffs(left) - 1;
    left &= left - 1;
    return i;
  };
  for (int i = next(); i >= 0;) {
    R v[kSegAhead];
    int count = 0;
#pragma unroll
    for (int k = 0; k < kSegAhead; ++k)
      if (i >= 0) {
        v[k].template load<true>(src + static_cast<int64_t>(i) * p.ld_dout, c, p.dim);
        ++count;
        i = next();
      }
#pragma unroll
    for (int k = 0; k < kSegAhead; ++k)
      if (k < count) {
#pragma unroll
        for (int e = 0; e < kN; ++e) sum[e] += v[k].get(e);
      }
  }
  write_row<GT, WIDE>(p, id, c, sum);
}

template <int DT, bool WIDE>
int run_lookup(const LookupParams &p, cudaStream_t s) {
  const int span = 32 * kLookupPacks * RowPart<DT, WIDE>::kN;
  const int64_t items = p.count * ((p.dim + span - 1) / span);
  // an item per warp: 62 us at 32768 rows of 8 KB, 69 with as many warps as are resident walking over them
  const int grid = static_cast<int>(std::min<int64_t>((items + 7) / 8, INT32_MAX));
  ns_embed_lookup_kernel<DT, WIDE><<<grid, 256, 0, s>>>(p);
  count_launch();
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

int run_sort(const SortParams &p, const ZeroParams &zero, bool clear, int dev, int sms, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kSortCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kSortThreads, 1, 1);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int clusters = 1;
  if (clear) {  // as many clusters as are resident at once: every one looks through the ids first
    static int resident[64] = {};
    int &n = resident[dev & 63];
    if (n == 0) {
      cfg.gridDim = dim3(sms / kSortCluster * kSortCluster, 1, 1);
      if (cudaOccupancyMaxActiveClusters(&n, ns_embed_sort_kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
      }
    }
    clusters = std::max(2, n);
  }
  cfg.gridDim = dim3(kSortCluster * clusters, 1, 1);
  if (cudaLaunchKernelEx(&cfg, ns_embed_sort_kernel, p, zero) != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  count_launch();
  return 0;
}

template <int DT, int GT, bool WIDE>
int run_direct(const GradParams &p, const ZeroParams &zero, int sms, cudaStream_t s) {
  // the rows to clear: a CTA for 16 KB, as many as are resident at most
  const int64_t clear = p.accumulate ? 0 : (static_cast<int64_t>(p.vocab) * zero.row_bytes + 16383) / 16384;
  const int64_t grid = static_cast<int64_t>(p.n) * p.chunks + std::min<int64_t>(clear, sms * 8);
  ns_embed_direct_kernel<DT, GT, WIDE><<<static_cast<int>(grid), kSegThreads, 0, s>>>(p, zero);
  count_launch();
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

template <int DT, int GT, bool WIDE>
int run_segments(const GradParams &p, cudaStream_t s) {
  ns_embed_segments_kernel<DT, GT, WIDE><<<p.pieces * p.chunks, kSegThreads, 0, s>>>(p);
  count_launch();
  constexpr int kJoin = WIDE ? 4 : 1;  // a 16-byte word of the fp32 parts
  GradParams j = p;
  j.chunks = (p.dim + kSegThreads * kJoin - 1) / (kSegThreads * kJoin);
  ns_embed_joins_kernel<GT, kJoin><<<p.pieces * j.chunks, kSegThreads, 0, s>>>(j);
  count_launch();
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

template <int DT, int GT>
int run_grad(GradParams p, const ZeroParams &zero, bool wide, int sms, cudaStream_t s) {
  p.chunks = chunks_of(p.dim, DT == kBF16 ? 8 : 4);
  if (p.n <= kDirect) return wide ? run_direct<DT, GT, true>(p, zero, sms, s) : run_direct<DT, GT, false>(p, zero, sms, s);
  return wide ? run_segments<DT, GT, true>(p, s) : run_segments<DT, GT, false>(p, s);
}

}  // namespace
}  // namespace ns

using namespace ns;

extern "C" int ns_embed_lookup(const void *table, int64_t ld_table, int64_t vocab, int64_t dim, const void *ids,
                               int id_type, int64_t count, float scale, void *out, int64_t ld_out, int dtype,
                               void *stream) {
  if ((dtype != NS_F32 && dtype != NS_BF16) || (id_type != NS_I32 && id_type != NS_I64)) return NS_EINVAL;
  if (bad_shape(vocab, dim, ld_table) || bad_shape(count, dim, ld_out) || dim > kMaxRowCols) return NS_EINVAL;
  if (count == 0 || dim == 0) return NS_OK;
  if (!ids || !out || (!table && vocab > 0)) return NS_EINVAL;
  const int elt = dtype == NS_BF16 ? 2 : 4;
  if (misaligned(table, elt) || misaligned(out, elt) || misaligned(ids, id_type == NS_I64 ? 8 : 4)) return NS_EALIGN;
  const Range ro(out, count, dim, ld_out, elt);
  if (ro.overlaps(Range(table, vocab, dim, ld_table, elt)) ||
      ro.overlaps(Range(ids, 1, count, count, id_type == NS_I64 ? 8 : 4)))
    return NS_EINVAL;
  OpCall call(stream);
  if (call.rc) return call.rc;
  LookupParams p{table, out, {ids, id_type == NS_I64, static_cast<int>(vocab)}, count, ld_table, ld_out,
                 static_cast<int>(dim), scale, call.status};
  // 16-byte packs when every row allows them; else single elements
  const int vec = 16 / elt;
  const bool wide = dim % vec == 0 && rows_aligned(table, ld_table, elt, vec) && rows_aligned(out, ld_out, elt, vec);
  return call.launch(kOpLookup, [&] {
    if (dtype == NS_BF16) return wide ? run_lookup<kBF16, true>(p, call.s) : run_lookup<kBF16, false>(p, call.s);
    return wide ? run_lookup<kF32, true>(p, call.s) : run_lookup<kF32, false>(p, call.s);
  });
}

extern "C" int ns_embed_grad(const void *dout, int64_t ld_dout, const void *ids, int id_type, int64_t count,
                             float scale, void *grad, int64_t ld_grad, int64_t vocab, int64_t dim, int dtype,
                             int grad_dtype, int accumulate, void *stream) {
  if ((dtype != NS_F32 && dtype != NS_BF16) || (grad_dtype != NS_F32 && grad_dtype != NS_BF16) ||
      (id_type != NS_I32 && id_type != NS_I64) || (accumulate != 0 && accumulate != 1))
    return NS_EINVAL;
  if (bad_shape(vocab, dim, ld_grad) || bad_shape(count, dim, ld_dout) || vocab >= INT32_MAX) return NS_EINVAL;
  if (count > (1 << 30) || dim > (1 << 24) || (count / kSegLeast + 1) * (dim / kSegThreads + 1) > INT32_MAX) return NS_EINVAL;
  if (vocab == 0 || dim == 0 || (count == 0 && accumulate)) return NS_OK;
  if (!grad || (count > 0 && (!ids || !dout))) return NS_EINVAL;
  const int elt = dtype == NS_BF16 ? 2 : 4, gelt = grad_dtype == NS_BF16 ? 2 : 4;
  if (misaligned(dout, elt) || misaligned(grad, gelt) || misaligned(ids, id_type == NS_I64 ? 8 : 4)) return NS_EALIGN;
  const Range rg(grad, vocab, dim, ld_grad, gelt);
  if (rg.overlaps(Range(dout, count, dim, ld_dout, elt)) ||
      rg.overlaps(Range(ids, 1, count, count, id_type == NS_I64 ? 8 : 4)))
    return NS_EINVAL;
  OpCall call(stream);
  if (call.rc) return call.rc;
  const int n = static_cast<int>(count);
  GradParams p{};
  p.dout = dout;
  p.grad = grad;
  p.ld_dout = ld_dout;
  p.ld_grad = ld_grad;
  p.n = n;
  p.vocab = static_cast<int>(vocab);
  p.dim = static_cast<int>(dim);
  p.dim_pad = static_cast<int>((dim + 7) / 8 * 8);
  p.scale = scale;
  p.accumulate = accumulate;
  p.status = call.status;
  const Ids list_ids{ids, id_type == NS_I64, p.vocab};
  const ZeroParams zero{list_ids, n, static_cast<uint8_t *>(grad), ld_grad * gelt, static_cast<int>(dim * gelt),
                        static_cast<size_t>((vocab - 1) * ld_grad + dim) * gelt, call.status};
  const int vec = 16 / elt;
  const bool wide = dim % vec == 0 && rows_aligned(dout, ld_dout, elt, vec) && rows_aligned(grad, ld_grad, gelt, vec);
  if (n > kDirect) {
    // long pieces leave fewer parts to join (32768 ids of 8 KB rows: 6 us less with 64 than with 32), short ones give
    // few positions more CTAs: the longest that give an SM 12 CTAs
    p.seg = kSegMost;
    while (p.seg > kSegLeast && static_cast<int64_t>(n / p.seg) * chunks_of(p.dim, vec) < 12ll * call.sms) p.seg /= 2;
    p.pieces = (n + p.seg - 1) / p.seg;
    const size_t list = (static_cast<size_t>(n) * 4 + 255) / 256 * 256;
    uint8_t *ws = nullptr;
    int rc = call.workspace(kSlotEmbed, 4 * list + static_cast<size_t>(p.pieces) * 2 * p.dim_pad * 4, &ws);
    if (rc) return rc;
    SortParams sp{};
    sp.ids = list_ids;
    sp.n = n;
    for (int k = 0; k < 2; ++k) {
      sp.keys[k] = reinterpret_cast<int *>(ws + 2 * k * list);
      sp.pos[k] = reinterpret_cast<int *>(ws + (2 * k + 1) * list);
    }
    int bits = 1;
    while (bits < 31 && (vocab >> bits)) ++bits;  // keys are 0 .. vocab
    sp.passes = (bits + 8) / 9;
    sp.bits = (bits + sp.passes - 1) / sp.passes;
    sp.status = call.status;
    p.keys = sp.keys[0];
    p.pos = sp.pos[0];
    p.parts = reinterpret_cast<float *>(ws + 4 * list);
    if ((rc = call.launch(kOpSort, [&] { return run_sort(sp, zero, !accumulate, call.dev, call.sms, call.s); }))) return rc;
  }
  return call.launch(kOpEmbedGrad, [&] {
    if (dtype == NS_BF16)
      return grad_dtype == NS_BF16 ? run_grad<kBF16, kBF16>(p, zero, wide, call.sms, call.s)
                                   : run_grad<kBF16, kF32>(p, zero, wide, call.sms, call.s);
    return grad_dtype == NS_BF16 ? run_grad<kF32, kBF16>(p, zero, wide, call.sms, call.s)
                                 : run_grad<kF32, kF32>(p, zero, wide, call.sms, call.s);
  });
}
