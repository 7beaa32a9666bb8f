// ns_route.cu -- the router of a layer of experts (include/ns.h): top-k
// experts of every row with their weights, counts and the slots in the
// experts' order, a balance loss; and the gradient of the logits.
//
// Small data (rows x experts) read once: what counts is latency. Two launches
// forward. The first takes a warp per row, the row in registers and the next one
// under way: the k largest by repeated warp maxima of order-preserving keys, the
// softmax in the same pass. (Several rows a warp, their maxima by shuffles: 71 us
// against 39 for 32768 x 256, top 8.) A CTA walks over a stretch of rows and leaves its counts and its sum of
// probabilities per expert. In the second every CTA adds up the counts of the
// stretches before its own and ranks its slots from there, so the order is
// stable and no atomic decides anything; the first one also writes the totals
// and the loss, whose sums run in a fixed order. 32768 x 256 bf16, top 8: 44 us
// forward, 13 backward; 1021 x 76 fp32, top 3: 11 and 3.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "../../include/ns.h"
#include "ns_rows.cuh"

namespace ns {

namespace {

constexpr int kMaxExperts = 1024, kMaxTopK = 32;
// CTAs of a call: what the scratch holds. Every CTA of the second launch reads the parts of all, so no more than fill the SMs.
constexpr int kMaxStretches = 152;

struct RouteParams {
  const void *logits;
  int64_t ld;
  const uint8_t *live;
  int rows, experts, top_k, renormalise;
  int stretch;              // rows of a CTA
  int32_t *ids;
  float *weights;
  float *logz;
  int32_t *counts, *offsets, *order, *live_rows;
  float *loss;
  float balance, z;
  int32_t *part_count;      // stretches x experts
  float *part_prob;         // stretches x experts
  float *part_z;            // stretches
  int32_t *part_live;       // stretches
  size_t work_size;         // bytes of the scratch, which starts at part_count
  int *status;
};

// Order-preserving key of a float, NaN above everything; 0 stands for "not to be chosen" (-infinity).
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v);
  if (isnan(v)) return 0xffffffffu;
  if (b == 0xff800000u) return 0u;
  const uint32_t k = b & 0x80000000u ? ~b : b | 0x80000000u;
  return v == 0.f ? 0x80000000u : k;  // both zeros are equal
}

// A lane's logits still to be chosen from: expert e of the row is value e / 32 of lane e % 32. take() gives the warp's
// largest, lowest index first among equals, and takes it out; -1 when nothing is left.
template <int DT, int V>
struct Choice;
// fp32: the largest key, then the lowest index that has it.
template <int V>
struct Choice<kF32, V> {
  uint32_t left[V], best = 0;
  __device__ __forceinline__ void set(int i, int, float v) {
    left[i] = key_of(v);
    best = max(best, left[i]);
  }
  __device__ __forceinline__ int take() {
    const int lane = threadIdx.x & 31;
    const uint32_t m = __reduce_max_sync(0xffffffffu, best);
    if (m == 0) return -1;
    int at = INT32_MAX;
    if (best == m) {
#pragma unroll
      for (int i = V - 1; i >= 0; --i) at = left[i] == m ? i * 32 + lane : at;
    }
    const int e = __reduce_min_sync(0xffffffffu, at);
    if (at == e) {
      best = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        left[i] = e == i * 32 + lane ? 0u : left[i];
        best = max(best, left[i]);
      }
    }
    return e;
  }
};
// bf16: key and index fit one word, so all are different: one maximum gives both, and what is left is what is smaller.
template <int V>
struct Choice<kBF16, V> {
  uint32_t left[V], best = 0;
  __device__ __forceinline__ void set(int i, int e, float v) {
    const uint32_t k = key_of(v) & 0xffff0000u;  // the low half of a positive number's is 0, of a negative one's ones
    left[i] = k ? k | (0xffffu - static_cast<uint32_t>(e)) : 0u;
    best = max(best, left[i]);
  }
  __device__ __forceinline__ int take() {
    const uint32_t m = __reduce_max_sync(0xffffffffu, best);
    if (m == 0) return -1;
    if (best == m) {
      best = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) best = max(best, left[i] < m ? left[i] : 0u);
    }
    return static_cast<int>(0xffffu - (m & 0xffffu));
  }
};

// Rows by warps, V logits a lane.
template <int V> constexpr int kRowWarps = V <= 8 ? 32 : 256 / V;  // their sums fill up to 32 KB
template <int DT, int V>
__global__ void __launch_bounds__(32 * kRowWarps<V>) ns_route_rows_kernel(const __grid_constant__ RouteParams p) {
  using E = typename Elem<DT>::T;
  constexpr int kW = kRowWarps<V>;
  __shared__ int32_t hist[V * 32];
  __shared__ float sums[kW][V * 32];
  __shared__ float zs[kW];
  __shared__ int lives[kW];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.launch_dependents;");  // the slots' launch may set itself up
  for (int e = threadIdx.x; e < V * 32; e += kW * 32) hist[e] = 0;
  __syncthreads();
  const int first = min(p.rows, static_cast<int>(blockIdx.x) * p.stretch), end = min(p.rows, first + p.stretch);
  float prob[V];
#pragma unroll
  for (int i = 0; i < V; ++i) prob[i] = 0.f;
  float zsum = 0.f;
  int nlive = 0;
  const size_t slots = static_cast<size_t>(p.rows) * p.top_k;
  // the next row's logits are read while this one's are chosen from
  E next[V];
  bool next_live = false;
  auto read = [&](int t) {
    next_live = t < end && (!p.live || p.live[t] != 0);
    const E *x = static_cast<const E *>(p.logits) + static_cast<int64_t>(t) * p.ld + lane;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (next_live && i * 32 + lane < p.experts) next[i] = x[i * 32];
  };
  read(first + warp);
  for (int t = first + warp; t < end; t += kW) {
    float v[V];
    Choice<DT, V> choice;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[i] = next_live && i * 32 + lane < p.experts ? Elem<DT>::to_f(next[i]) : -INFINITY;
      choice.set(i, i * 32 + lane, v[i]);
    }
    read(t + kW);
    int mine = -1;  // lane j: the j-th choice
    for (int j = 0; j < p.top_k; ++j) {
      const int e = choice.take();
      if (e < 0) break;
      if (lane == j) mine = e;
    }
    const int e0 = __shfl_sync(0xffffffffu, mine, 0);
    const bool live = e0 >= 0;
    // a chosen one's logit, from where the lane that has it keeps the row
    auto logit_of = [&](int e) {
      float r = 0.f;
      const int from = e >= 0 ? e & 31 : 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float f = __shfl_sync(0xffffffffu, v[i], from);
        r = e / 32 == i ? f : r;
      }
      return r;
    };
    const float chosen = logit_of(mine), top = __shfl_sync(0xffffffffu, chosen, 0);
    float total = 0.f, q[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      q[i] = live ? expf(v[i] - top) : 0.f;
      total += q[i];
    }
    total = warp_sum(total);
    const float inv = live ? 1.f / total : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) prob[i] += q[i] * inv;
    const float lz = live ? top + logf(total) : 0.f;
    zsum += lz * lz;
    nlive += live ? 1 : 0;
    float w = mine >= 0 ? expf(chosen - top) : 0.f;
    const float sum = p.renormalise ? warp_sum(w) : total;
    w = live ? w / sum : 0.f;
    if (lane < p.top_k) {
      const int64_t at = static_cast<int64_t>(t) * p.top_k + lane;
      if (in_bounds(p.ids + at, 4, p.ids, slots * 4, p.status)) p.ids[at] = mine;
      if (in_bounds(p.weights + at, 4, p.weights, slots * 4, p.status)) p.weights[at] = w;
      if (mine >= 0) atomicAdd(&hist[mine], 1);
    }
    if (lane == 0 && in_bounds(p.logz + t, 4, p.logz, static_cast<size_t>(p.rows) * 4, p.status)) p.logz[t] = lz;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) sums[warp][i * 32 + lane] = prob[i];
  if (lane == 0) {
    zs[warp] = zsum;
    lives[warp] = nlive;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.experts; e += kW * 32) {
    float s = sums[0][e];
#pragma unroll
    for (int k = 1; k < kW; ++k) s += sums[k][e];
    const int64_t at = static_cast<int64_t>(blockIdx.x) * p.experts + e;
    put(p.part_prob + at, s, p.part_count, p.work_size, p.status);
    put(p.part_count + at, hist[e], p.part_count, p.work_size, p.status);
  }
  if (threadIdx.x == 0) {
    float z = 0.f;
    int n = 0;
    for (int k = 0; k < kW; ++k) {
      z += zs[k];
      n += lives[k];
    }
    put(p.part_z + blockIdx.x, z, p.part_count, p.work_size, p.status);
    put(p.part_live + blockIdx.x, n, p.part_count, p.work_size, p.status);
  }
}

template <int W>
__device__ __forceinline__ float block_sum(float v, float *red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  float s = 0.f;
  for (int k = 0; k < W; ++k) s += red[k];
  return s;
}

// Slots of the CTA's stretch in the experts' order, and the totals, by W warps.
template <int W>
__global__ void __launch_bounds__(W * 32) ns_route_order_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ int32_t nexts[];  // per warp and expert: place of its next slot
  __shared__ int32_t scan[W];
  __shared__ float red[W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int stretches = gridDim.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int first = min(p.rows, static_cast<int>(blockIdx.x) * p.stretch), end = min(p.rows, first + p.stretch);
  const int slot0 = first * p.top_k, nslots = (end - first) * p.top_k;
  const int share = ((nslots + W - 1) / W + 31) / 32 * 32;  // of a warp
  const int a = min(nslots, warp * share), b = min(nslots, a + share);
  for (int e = threadIdx.x; e < W * p.experts; e += W * 32) nexts[e] = 0;
  int32_t *mine = nexts + warp * p.experts;
  __syncthreads();
  // this stretch's slots per warp and expert
  constexpr int kAhead = 4;  // reads in flight
  for (int i0 = a; i0 < b; i0 += 32 * kAhead) {
    int e[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) e[k] = i0 + 32 * k + lane < b ? p.ids[slot0 + i0 + 32 * k + lane] : -1;
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (e[k] >= 0) atomicAdd(mine + e[k], 1);
  }
  __syncthreads();
  // Counts of all stretches and of those before this one: warps take 32 experts and a share of the stretches, many reads
  // in flight (one thread for an expert's stretches was 40 us).
  __shared__ int32_t part_all[kMaxExperts], part_before[kMaxExperts];
  __shared__ float part_prob[kMaxExperts];
  const int groups = (p.experts + 31) / 32, shares = max(1, W / groups);
  for (int item = warp; item < groups * shares; item += W) {
    const int e = item % groups * 32 + lane, part = item / groups;
    const int c0 = stretches * part / shares, c1 = stretches * (part + 1) / shares;
    int all = 0, before = 0;
    float prob = 0.f;
    if (e < p.experts) {
      constexpr int kDeep = 16;
      for (int c = c0; c < c1; c += kDeep) {
        int n[kDeep];
        float f[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
          const int64_t at = static_cast<int64_t>(c + k) * p.experts + e;
          n[k] = c + k < c1 ? p.part_count[at] : 0;
          f[k] = blockIdx.x == 0 && c + k < c1 ? p.part_prob[at] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
          all += n[k];
          before += c + k < static_cast<int>(blockIdx.x) ? n[k] : 0;
          prob += f[k];
        }
      }
      part_all[part * p.experts + e] = all;
      part_before[part * p.experts + e] = before;
      part_prob[part * p.experts + e] = prob;
    }
  }
  __syncthreads();
  // experts in turn by threads, W * 32 at a time: the slots of all experts before, of the stretches before, of the warps before
  int run = 0;
  float loss = 0.f;
  for (int e0 = 0; e0 < p.experts; e0 += W * 32) {
    const int e = e0 + threadIdx.x;
    int before = 0, all = 0;
    float prob = 0.f;
    if (e < p.experts)
      for (int k = 0; k < shares; ++k) {
        all += part_all[k * p.experts + e];
        before += part_before[k * p.experts + e];
        prob += part_prob[k * p.experts + e];
      }
    // exclusive prefix over the threads
    int incl = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int base = run;
    for (int k = 0; k < W; ++k) {
      if (k < warp) base += scan[k];
      run += scan[k];
    }
    const int offset = base + incl - all;
    if (e < p.experts) {
      int at = offset + before;
      for (int k = 0; k < W; ++k) {
        const int n = nexts[k * p.experts + e];
        nexts[k * p.experts + e] = at;
        at += n;
      }
      if (blockIdx.x == 0) {
        if (in_bounds(p.counts + e, 4, p.counts, static_cast<size_t>(p.experts) * 4, p.status)) p.counts[e] = all;
        if (in_bounds(p.offsets + e, 4, p.offsets, (static_cast<size_t>(p.experts) + 1) * 4, p.status)) p.offsets[e] = offset;
        loss += static_cast<float>(all) * prob;
      }
    }
  }
  __syncthreads();
  const size_t size = static_cast<size_t>(p.rows) * p.top_k * 4;
  for (int i0 = a; i0 < b; i0 += 32 * kAhead) {
    int ids[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) ids[k] = i0 + 32 * k + lane < b ? p.ids[slot0 + i0 + 32 * k + lane] : -1;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int e = ids[k];
      const uint32_t same = __match_any_sync(0xffffffffu, e);
      const uint32_t before = same & ((1u << lane) - 1u);
      int at = 0;
      if (e >= 0) at = mine[e] + __popc(before);
      __syncwarp();
      if (e >= 0 && before == 0) mine[e] += __popc(same);
      __syncwarp();
      if (e >= 0 && in_bounds(p.order + at, 4, p.order, size, p.status)) p.order[at] = slot0 + i0 + 32 * k + lane;
    }
  }
  // places that no slot has
  const int64_t slots = static_cast<int64_t>(p.rows) * p.top_k;
  for (int64_t i = run + static_cast<int64_t>(blockIdx.x) * W * 32 + threadIdx.x; i < slots; i += static_cast<int64_t>(stretches) * W * 32)
    if (in_bounds(p.order + i, 4, p.order, size, p.status)) p.order[i] = -1;
  if (blockIdx.x == 0) {
    float z = 0.f;
    int live = 0;
    for (int c = threadIdx.x; c < stretches; c += W * 32) {
      z += p.part_z[c];
      live += p.part_live[c];
    }
    loss = block_sum<W>(loss, red);
    z = block_sum<W>(z, red);
    live = __reduce_add_sync(0xffffffffu, live);
    __syncthreads();
    if (lane == 0) scan[warp] = live;
    __syncthreads();
    if (threadIdx.x == 0) {
      live = 0;
      for (int k = 0; k < W; ++k) live += scan[k];
      const double t = live;
      if (in_bounds(p.offsets + p.experts, 4, p.offsets, (static_cast<size_t>(p.experts) + 1) * 4, p.status)) p.offsets[p.experts] = run;
      put(p.live_rows, live, p.live_rows, 4, p.status);
      // logz^2 may be beyond fp32: with a coefficient of 0 its mean stays out (a NaN of a row is in the balance as well)
      const double squares = p.z != 0.f ? p.z * (z / t) : 0.;
      const double mean = p.balance * (p.experts * static_cast<double>(loss) / (p.top_k * t * t)) + squares;
      put(p.loss, live == 0 ? 0.f : static_cast<float>(mean), p.loss, 4, p.status);
    }
  }
}

struct RouteBackParams {
  const void *logits;
  int64_t ld;
  int rows, experts, top_k, renormalise;
  const int32_t *ids;
  const float *weights, *dweights, *logz;
  const int32_t *counts, *live_rows;
  float balance, z;
  void *dlogits;
  int64_t ld_d;
  int *status;
};

constexpr int kBackWarps = 8;
// dL = P (s - sum of P s + 2 z logz / T) with s = balance E counts / (k T^2), and the weights' own part. P is exp(l - logz)
// over the sum of these: logz is rounded to fp32 (at logits around 1e5 by up to 2^-8), so alone it gives no probabilities.
// As the offset of its row any number of that size will do, which spares the row's maximum; sum and division are 1 us of
// 13 at 32768 x 256. CTAs an SM: what 32, 40, 64 and 128 registers a thread allow (128 experts, 35 registers: 13.2 us
// against 11.0).
template <int V> constexpr int kBackCtas = V <= 4 ? 8 : V == 8 ? 6 : V == 16 ? 4 : 2;
template <int DT, int V>
__global__ void __launch_bounds__(kBackWarps * 32, kBackCtas<V>) ns_route_backward_kernel(const __grid_constant__ RouteBackParams p) {
  using E = typename Elem<DT>::T;
  __shared__ float slope[V * 32];
  __shared__ float part[kBackWarps][V * 32];  // a row's weights' part by expert; zero between rows
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float t = static_cast<float>(max(__ldg(p.live_rows), 1));
  const float factor = p.balance * static_cast<float>(p.experts) / static_cast<float>(p.top_k) / t / t;
  for (int e = threadIdx.x; e < V * 32; e += kBackWarps * 32) {
    slope[e] = e < p.experts ? factor * static_cast<float>(p.counts[e]) : 0.f;
#pragma unroll
    for (int k = 0; k < kBackWarps; ++k) part[k][e] = 0.f;
  }
  __syncthreads();
  const size_t size = static_cast<size_t>((p.rows - 1) * p.ld_d + p.experts) * sizeof(E);
  for (int r = blockIdx.x * kBackWarps + warp; r < p.rows; r += gridDim.x * kBackWarps) {
    const E *x = static_cast<const E *>(p.logits) + static_cast<int64_t>(r) * p.ld;
    E *out = static_cast<E *>(p.dlogits) + static_cast<int64_t>(r) * p.ld_d;
    int e = -1;
    float w = 0.f, dw = 0.f;
    if (lane < p.top_k) {
      const int64_t at = static_cast<int64_t>(r) * p.top_k + lane;
      e = p.ids[at];
      if (e >= p.experts) e = -1;
      if (e >= 0) {
        w = p.weights[at];
        dw = p.dweights ? p.dweights[at] : 0.f;
      }
    }
    const bool live = __shfl_sync(0xffffffffu, e, 0) >= 0;
    if (!live) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = i * 32 + lane;
        if (c < p.experts && in_bounds(out + c, sizeof(E), p.dlogits, size, p.status)) out[c] = Elem<DT>::from_f(0.f);
      }
      continue;
    }
    if (p.renormalise) dw = w * (dw - warp_sum(w * dw));
    if (e >= 0) part[warp][e] = dw;
    __syncwarp();
    const float lz = p.logz[r];
    float q[V], s[V], total = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * 32 + lane;
      q[i] = c < p.experts ? expf(Elem<DT>::to_f(x[c]) - lz) : 0.f;
      s[i] = slope[c] + (p.renormalise ? 0.f : part[warp][c]);
      total += q[i];
      dot += q[i] * s[i];
    }
    const float inv = 1.f / warp_sum(total);
    dot = warp_sum(dot) * inv - 2.f * p.z / t * lz;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * 32 + lane;
      float d = q[i] * inv * (s[i] - dot);
      if (p.renormalise) d += part[warp][c];
      if (c < p.experts && in_bounds(out + c, sizeof(E), p.dlogits, size, p.status)) out[c] = Elem<DT>::from_f(d);
    }
    __syncwarp();
    if (e >= 0) part[warp][e] = 0.f;
    __syncwarp();
  }
}

// The same for bf16 rows of more than 128 experts that allow packs: 8 consecutive experts a lane, N times, the next row read
// while this one is worked on (its slots, weights and logits are a chain of loads that a row otherwise waits for), and the
// fast exponential, which is off by less than (2 + 1.2 |l - logz|) 2^-23 (its documented bound), far below bf16's rounding.
template <int N>
__global__ void __launch_bounds__(kBackWarps * 32) ns_route_backward_packs_kernel(const __grid_constant__ RouteBackParams p) {
  using E = typename Elem<kBF16>::T;
  __shared__ float4 slope4[N * 64];
  __shared__ float4 part4[kBackWarps][N * 64];  // a row's weights' part by expert; zero between rows
  float *slope = reinterpret_cast<float *>(slope4);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float *part = reinterpret_cast<float *>(part4[warp]);
  const float t = static_cast<float>(max(__ldg(p.live_rows), 1));
  const float factor = p.balance * static_cast<float>(p.experts) / static_cast<float>(p.top_k) / t / t;
  for (int e = threadIdx.x; e < N * 256; e += kBackWarps * 32) slope[e] = e < p.experts ? factor * static_cast<float>(p.counts[e]) : 0.f;
  for (int e = lane; e < N * 256; e += 32) part[e] = 0.f;
  __syncthreads();
  const size_t size = static_cast<size_t>((p.rows - 1) * p.ld_d + p.experts) * sizeof(E);
  Pack<kBF16, 8> v[N], nv[N];
  int ne = -1;
  float nw = 0.f, ndw = 0.f, nlz = 0.f;
  const int step = gridDim.x * kBackWarps;
  auto fetch = [&](int r) {
    if (r >= p.rows) return;
    const E *x = static_cast<const E *>(p.logits) + static_cast<int64_t>(r) * p.ld;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * 32 + lane) * 8;
      if (c < p.experts) nv[i].load(x + c);
    }
    nlz = p.logz[r];
    ne = -1;
    nw = ndw = 0.f;
    if (lane < p.top_k) {
      const int64_t at = static_cast<int64_t>(r) * p.top_k + lane;
      ne = p.ids[at];
      nw = p.weights[at];
      if (p.dweights) ndw = p.dweights[at];
    }
  };
  int r = blockIdx.x * kBackWarps + warp;
  fetch(r);
  for (; r < p.rows; r += step) {
    E *out = static_cast<E *>(p.dlogits) + static_cast<int64_t>(r) * p.ld_d;
    const int e = ne >= p.experts ? -1 : ne;
    const float w = e >= 0 ? nw : 0.f, lz = nlz;
    float dw = e >= 0 ? ndw : 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = nv[i];
    fetch(r + step);
    const bool live = __shfl_sync(0xffffffffu, e, 0) >= 0;
    if (live) {
      if (p.renormalise) dw = w * (dw - warp_sum(w * dw));
      if (e >= 0) part[e] = dw;
      __syncwarp();
      float q[N][8], s[N][8], own[N][8], total = 0.f, dot = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (i * 32 + lane) * 8;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float4 a = slope4[c / 4 + h], b = part4[warp][c / 4 + h];
          const float sa[4] = {a.x, a.y, a.z, a.w}, sb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int j = 4 * h + k;
            const float z = c < p.experts ? v[i].get(j) - lz : -INFINITY;
            q[i][j] = __expf(z);
            own[i][j] = p.renormalise ? sb[k] : 0.f;
            s[i][j] = sa[k] + (p.renormalise ? 0.f : sb[k]);
            total += q[i][j];
            dot = fmaf(q[i][j], s[i][j], dot);
          }
        }
      }
      const float inv = 1.f / warp_sum(total);
      dot = warp_sum(dot) * inv - 2.f * p.z / t * lz;
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i].set(j, fmaf(q[i][j] * inv, s[i][j] - dot, own[i][j]));
      __syncwarp();
      if (e >= 0) part[e] = 0.f;
      __syncwarp();
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i].set(j, 0.f);
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * 32 + lane) * 8;
      if (c < p.experts) v[i].store_stream(out + c, p.dlogits, size, p.status);
    }
  }
}

template <typename F>
int by_width(int experts, F &&f) {
  return experts <= 32 ? f(std::integral_constant<int, 1>{}) : experts <= 64 ? f(std::integral_constant<int, 2>{})
         : experts <= 128 ? f(std::integral_constant<int, 4>{}) : experts <= 256 ? f(std::integral_constant<int, 8>{})
         : experts <= 512 ? f(std::integral_constant<int, 16>{}) : f(std::integral_constant<int, 32>{});
}

template <typename F>
int by_packs(int experts, F &&f) {
  return experts <= 256 ? f(std::integral_constant<int, 1>{}) : experts <= 512 ? f(std::integral_constant<int, 2>{})
                                                              : f(std::integral_constant<int, 4>{});
}

bool bad_dtype(int dtype) { return dtype != NS_F32 && dtype != NS_BF16; }
bool bad_sizes(int64_t rows, int experts, int top_k, int64_t ld, float balance, float z) {
  return bad_shape(rows, experts, ld) || experts < 1 || experts > kMaxExperts || top_k < 1 || top_k > kMaxTopK ||
         top_k > experts || rows > (1 << 30) / top_k || !std::isfinite(balance) || !std::isfinite(z);
}
size_t scratch_of(int64_t rows, int experts) {
  const int64_t n = std::min<int64_t>((rows + 15) / 16, kMaxStretches);
  return static_cast<size_t>(std::max<int64_t>(n, 1)) * (8 * static_cast<size_t>(experts) + 8);
}

}  // namespace
}  // namespace ns

using namespace ns;

extern "C" int64_t ns_route_workspace(int64_t rows, int experts) {
  return rows < 0 || experts < 1 || experts > kMaxExperts ? -1 : static_cast<int64_t>(scratch_of(rows, experts));
}

extern "C" int ns_route(const void *logits, int64_t ld_logits, int64_t rows, int experts, int top_k,
                        const uint8_t *live, int renormalise, float balance_coef, float z_coef, int32_t *ids,
                        float *weights, float *logz, int32_t *counts, int32_t *offsets, int32_t *order,
                        int32_t *live_rows, float *loss, void *workspace, size_t workspace_bytes, int dtype,
                        void *stream) {
  if (bad_dtype(dtype) || bad_sizes(rows, experts, top_k, ld_logits, balance_coef, z_coef) ||
      (renormalise != 0 && renormalise != 1))
    return NS_EINVAL;
  if (!counts || !offsets || !live_rows || !loss || !workspace) return NS_EINVAL;
  if (rows > 0 && (!logits || !ids || !weights || !logz || !order)) return NS_EINVAL;
  if (workspace_bytes < scratch_of(rows, experts)) return NS_ENOMEM;
  const int elt = dtype == NS_BF16 ? 2 : 4;
  if (misaligned(logits, elt) || misaligned(workspace, 4)) return NS_EALIGN;
  const void *words[] = {ids, weights, logz, counts, offsets, order, live_rows, loss};
  const int64_t slots = rows * top_k, lengths[] = {slots, slots, rows, experts, experts + 1, slots, 1, 1};
  const Range rx(logits, rows, experts, ld_logits, elt), rl(live, 1, rows, rows, 1);
  const Range rw(workspace, 1, static_cast<int64_t>(workspace_bytes), static_cast<int64_t>(workspace_bytes), 1);
  if (rw.overlaps(rx) || rw.overlaps(rl)) return NS_EINVAL;
  for (int i = 0; i < 8; ++i) {
    if (misaligned(words[i], 4)) return NS_EALIGN;
    const Range r(words[i], 1, lengths[i], lengths[i], 4);
    if (r.overlaps(rx) || r.overlaps(rl) || r.overlaps(rw)) return NS_EINVAL;
    for (int k = 0; k < i; ++k)
      if (r.overlaps(Range(words[k], 1, lengths[k], lengths[k], 4))) return NS_EINVAL;
  }
  OpCall call(stream);
  if (call.rc) return call.rc;
  RouteParams p{};
  p.logits = logits;
  p.ld = ld_logits;
  p.live = live;
  p.rows = static_cast<int>(rows);
  p.experts = experts;
  p.top_k = top_k;
  p.renormalise = renormalise;
  p.ids = ids;
  p.weights = weights;
  p.logz = logz;
  p.counts = counts;
  p.offsets = offsets;
  p.order = order;
  p.live_rows = live_rows;
  p.loss = loss;
  p.balance = balance_coef;
  p.z = z_coef;
  p.status = call.status;
  const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({(rows + 15) / 16, call.sms, kMaxStretches})));
  p.stretch = static_cast<int>((rows + grid - 1) / grid);
  p.part_count = static_cast<int32_t *>(workspace);
  p.work_size = workspace_bytes;
  p.part_prob = reinterpret_cast<float *>(p.part_count + static_cast<int64_t>(grid) * experts);
  p.part_z = p.part_prob + static_cast<int64_t>(grid) * experts;
  p.part_live = reinterpret_cast<int32_t *>(p.part_z + grid);
  return call.launch(kOpRoute, [&] {
    by_width(experts, [&](auto v) {
      constexpr int V = decltype(v)::value;
      if (dtype == NS_BF16)
        ns_route_rows_kernel<kBF16, V><<<grid, 32 * kRowWarps<V>, 0, call.s>>>(p);
      else
        ns_route_rows_kernel<kF32, V><<<grid, 32 * kRowWarps<V>, 0, call.s>>>(p);
      return 0;
    });
    count_launch();
    const auto order = [&](auto w) {
      constexpr int W = decltype(w)::value;
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[0].val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      cfg.stream = call.s;
      cfg.gridDim = dim3(grid, 1, 1);
      cfg.blockDim = dim3(W * 32, 1, 1);
      cfg.dynamicSmemBytes = static_cast<size_t>(W) * experts * 4;
      static SmemOptIn opt_in;
      if (opt_in.ensure(reinterpret_cast<const void *>(ns_route_order_kernel<W>), static_cast<int>(cfg.dynamicSmemBytes))) return -1;
      if (cudaLaunchKernelEx(&cfg, ns_route_order_kernel<W>, p) == cudaSuccess) return 0;
      cudaGetLastError();
      return -1;
    };
    // Every CTA reads the counts of all stretches: 32 warps where these are many (both launches, 16 warps / 32, us: 32768 x
    // 256 52 / 44, 8192 x 1024 94 / 70, 32768 x 64 29 / 26), 16 where barriers of few reads count more (32768 x 8 19.3 /
    // 19.7, 1021 x 76 11.4 / 12.2, one row of 256 9.7 / 11.4).
    const int rc = static_cast<int64_t>(grid) * experts > 8192 ? order(std::integral_constant<int, 32>{}) : order(std::integral_constant<int, 16>{});
    if (rc) return rc;
    count_launch();
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
  });
}

extern "C" int ns_route_backward(const void *logits, int64_t ld_logits, int64_t rows, int experts, int top_k,
                                 const int32_t *ids, const float *weights, const float *dweights, const float *logz,
                                 const int32_t *counts, const int32_t *live_rows, int renormalise, float balance_coef,
                                 float z_coef, void *dlogits, int64_t ld_dlogits, int dtype, void *stream) {
  if (bad_dtype(dtype) || bad_sizes(rows, experts, top_k, ld_logits, balance_coef, z_coef) ||
      bad_shape(rows, experts, ld_dlogits) || (renormalise != 0 && renormalise != 1))
    return NS_EINVAL;
  if (rows == 0) return NS_OK;
  if (!logits || !ids || !weights || !logz || !counts || !live_rows || !dlogits) return NS_EINVAL;
  const int elt = dtype == NS_BF16 ? 2 : 4;
  if (misaligned(logits, elt) || misaligned(dlogits, elt)) return NS_EALIGN;
  const Range rd(dlogits, rows, experts, ld_dlogits, elt);
  if (!(dlogits == logits && ld_dlogits == ld_logits) && rd.overlaps(Range(logits, rows, experts, ld_logits, elt))) return NS_EINVAL;
  const void *words[] = {ids, weights, dweights, logz, counts, live_rows};
  const int64_t slots = rows * top_k, lengths[] = {slots, slots, slots, rows, experts, 1};
  for (int i = 0; i < 6; ++i) {
    if (misaligned(words[i], 4)) return NS_EALIGN;
    if (rd.overlaps(Range(words[i], 1, lengths[i], lengths[i], 4))) return NS_EINVAL;
  }
  OpCall call(stream);
  if (call.rc) return call.rc;
  RouteBackParams p{logits, ld_logits, static_cast<int>(rows), experts, top_k, renormalise, ids, weights, dweights, logz,
                    counts, live_rows, balance_coef, z_coef, dlogits, ld_dlogits, call.status};
  // 32768 rows, us, packs against elements: 64 experts 11.3 / 9.0, 128 11.8 / 11.0, 192 12.1 / 17.7, 256 12.8 / 21.1;
  // 8192 rows of 512 7.6 / 9.3, of 1024 14.0 / 26.8. fp32 gains nothing by them (4096 x 256 4.6 / 4.5).
  const bool packs = dtype == NS_BF16 && experts > 128 && experts % 8 == 0 && rows_aligned(logits, ld_logits, elt, 8) &&
                     rows_aligned(dlogits, ld_dlogits, elt, 8);
  const auto grid = [&](int per_sm) {
    return static_cast<int>(std::min<int64_t>((rows + kBackWarps - 1) / kBackWarps, static_cast<int64_t>(call.sms) * per_sm));
  };
  return call.launch(kOpRoute, [&] {
    if (packs)
      by_packs(experts, [&](auto n) {
        // as many CTAs as their registers let stay
        ns_route_backward_packs_kernel<decltype(n)::value><<<grid(4 / decltype(n)::value), 32 * kBackWarps, 0, call.s>>>(p);
        return 0;
      });
    else
      by_width(experts, [&](auto v) {
        if (dtype == NS_BF16)
          ns_route_backward_kernel<kBF16, decltype(v)::value><<<grid(8), 32 * kBackWarps, 0, call.s>>>(p);
        else
          ns_route_backward_kernel<kF32, decltype(v)::value><<<grid(8), 32 * kBackWarps, 0, call.s>>>(p);
        return 0;
      });
    count_launch();
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
  });
}
