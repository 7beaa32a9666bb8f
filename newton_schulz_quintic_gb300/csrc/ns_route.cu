// ns_route.cu -- the router of a layer of experts (include/ns.h): top-k
// experts of every row with their weights, counts and the slots in the
// experts' order, a balance loss; and the gradient of the logits.
//
// Small data (rows x experts) read once: what counts is latency. Two launches
// forward. The first takes a warp per row, the row in registers: the k largest
// by repeated warp maxima of order-preserving keys, the softmax in the same
// pass. A CTA walks over a stretch of rows and leaves its counts and its sum of
// probabilities per expert. In the second every CTA adds up the counts of the
// stretches before its own and ranks its slots from there, so the order is
// stable and no atomic decides anything; the first one also writes the totals
// and the loss, whose sums run in a fixed order.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "../../include/ns.h"
#include "ns_rows.cuh"

namespace ns {

namespace {

constexpr int kWarps = 16, kThreads = kWarps * 32;
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

// L lanes a row, V logits a lane: expert e of the row is value e / L of lane e % L; 32 / L rows a warp. A group's largest
// key is found by shuffles among its lanes.
template <int L>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  if constexpr (L == 32) {
    return __reduce_max_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}
template <int L>
__device__ __forceinline__ int group_min(int v) {
  if constexpr (L == 32) {
    return __reduce_min_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// The float of a key (zero for either zero).
__device__ __forceinline__ float value_of(uint32_t key) {
  return key == 0xffffffffu ? __int_as_float(0x7fc00000) : __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

template <int L, int V> constexpr int kRowWarps = L * V <= 512 ? kWarps : kWarps / 2;  // their sums fill 32 KB
template <int DT, int L, int V>
__global__ void __launch_bounds__(32 * kRowWarps<L, V>) ns_route_rows_kernel(const __grid_constant__ RouteParams p) {
  using E = typename Elem<DT>::T;
  constexpr int kRows = 32 / L, kW = kRowWarps<L, V>;  // rows of a warp at a time, warps
  __shared__ int32_t hist[V * L];
  __shared__ float sums[kW][V * L];
  __shared__ float zs[kW];
  __shared__ int lives[kW];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % L, sub = lane / L;
  asm volatile("griddepcontrol.launch_dependents;");  // the slots' launch may set itself up
  for (int e = threadIdx.x; e < V * L; e += kW * 32) hist[e] = 0;
  __syncthreads();
  const int first = min(p.rows, static_cast<int>(blockIdx.x) * p.stretch), end = min(p.rows, first + p.stretch);
  float prob[V];
#pragma unroll
  for (int i = 0; i < V; ++i) prob[i] = 0.f;
  float zsum = 0.f;
  int nlive = 0;
  const size_t slots = static_cast<size_t>(p.rows) * p.top_k;
  for (int t0 = first + warp * kRows; t0 < end; t0 += kW * kRows) {
    const int t = t0 + sub;
    const E *x = static_cast<const E *>(p.logits) + static_cast<int64_t>(t) * p.ld;
    bool live = t < end && (!p.live || p.live[t] != 0);
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = i * L + l;
      key[i] = live && e < p.experts ? key_of(Elem<DT>::to_f(x[e])) : 0u;
    }
    // the k largest, one after the other: the lane that holds it takes it out of its own
    uint32_t left[V];
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      left[i] = key[i];
      best = max(best, key[i]);
    }
    uint32_t chosen[kMaxTopK / L > 0 ? kMaxTopK / L : 1];  // lane j % L: the j-th choice
    int mine[kMaxTopK / L > 0 ? kMaxTopK / L : 1];
    constexpr int kHeld = kMaxTopK / L > 0 ? kMaxTopK / L : 1;
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
      chosen[h] = 0;
      mine[h] = -1;
    }
    uint32_t top = 0;
    for (int j = 0; j < p.top_k; ++j) {
      const uint32_t m = group_max<L>(best);
      if (j == 0) top = m;
      if (!__any_sync(0xffffffffu, m != 0)) break;  // nothing left that may be chosen
      int at = INT32_MAX;
#pragma unroll
      for (int i = V - 1; i >= 0; --i) at = left[i] == m ? i * L + l : at;
      const int e = group_min<L>(m != 0 ? at : INT32_MAX);
      if (m != 0 && at == e) {
        best = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          left[i] = i * L + l == e ? 0u : left[i];
          best = max(best, left[i]);
        }
      }
#pragma unroll
      for (int h = 0; h < kHeld; ++h)
        if (m != 0 && l == j - h * L) {
          mine[h] = e;
          chosen[h] = m;
        }
    }
    live = top != 0;
    const float most = live ? value_of(top) : 0.f;
    float total = 0.f, q[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      q[i] = key[i] != 0 ? expf(value_of(key[i]) - most) : 0.f;
      total += q[i];
    }
    total = group_sum<L>(total);
    const float inv = live ? 1.f / total : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) prob[i] += q[i] * inv;
    const float lz = live ? most + logf(total) : 0.f;
    zsum += lz * lz;
    nlive += live ? 1 : 0;
    float w[kHeld], sum = 0.f;
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
      w[h] = mine[h] >= 0 ? expf(value_of(chosen[h]) - most) : 0.f;
      sum += w[h];
    }
    sum = group_sum<L>(sum);
    if (!p.renormalise) sum = total;
    if (t < end) {
#pragma unroll
      for (int h = 0; h < kHeld; ++h)
        if (h * L + l < p.top_k) {
          const int64_t at = static_cast<int64_t>(t) * p.top_k + h * L + l;
          if (in_bounds(p.ids + at, 4, p.ids, slots * 4, p.status)) p.ids[at] = mine[h];
          if (in_bounds(p.weights + at, 4, p.weights, slots * 4, p.status)) p.weights[at] = live ? w[h] / sum : 0.f;
          if (mine[h] >= 0) atomicAdd(&hist[mine[h]], 1);
        }
      if (l == 0 && in_bounds(p.logz + t, 4, p.logz, static_cast<size_t>(p.rows) * 4, p.status)) p.logz[t] = lz;
    }
  }
  // the warp's groups of lanes are added in order
#pragma unroll
  for (int o = L; o < 32; o <<= 1) {
    zsum += __shfl_down_sync(0xffffffffu, zsum, o);
    nlive += __shfl_down_sync(0xffffffffu, nlive, o);
#pragma unroll
    for (int i = 0; i < V; ++i) prob[i] += __shfl_down_sync(0xffffffffu, prob[i], o);
  }
  if (lane < L)
#pragma unroll
    for (int i = 0; i < V; ++i) sums[warp][i * L + l] = prob[i];
  if (lane == 0) {
    zs[warp] = zsum;
    lives[warp] = nlive;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.experts; e += kW * 32) {
    float s = sums[0][e];
#pragma unroll
    for (int k = 1; k < kW; ++k) s += sums[k][e];
    p.part_prob[static_cast<int64_t>(blockIdx.x) * p.experts + e] = s;
    p.part_count[static_cast<int64_t>(blockIdx.x) * p.experts + e] = hist[e];
  }
  if (threadIdx.x == 0) {
    float z = 0.f;
    int n = 0;
    for (int k = 0; k < kW; ++k) {
      z += zs[k];
      n += lives[k];
    }
    p.part_z[blockIdx.x] = z;
    p.part_live[blockIdx.x] = n;
  }
}

__device__ __forceinline__ float block_sum(float v, float *red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  float s = 0.f;
  for (int k = 0; k < kWarps; ++k) s += red[k];
  return s;
}

// Slots of the CTA's stretch in the experts' order, and the totals.
__global__ void __launch_bounds__(kThreads) ns_route_order_kernel(const __grid_constant__ RouteParams p) {
  extern __shared__ int32_t nexts[];  // per warp and expert: place of its next slot
  __shared__ int32_t scan[kWarps];
  __shared__ float red[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int stretches = gridDim.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int first = min(p.rows, static_cast<int>(blockIdx.x) * p.stretch), end = min(p.rows, first + p.stretch);
  const int slot0 = first * p.top_k, nslots = (end - first) * p.top_k;
  const int share = ((nslots + kWarps - 1) / kWarps + 31) / 32 * 32;  // of a warp
  const int a = min(nslots, warp * share), b = min(nslots, a + share);
  for (int e = threadIdx.x; e < kWarps * p.experts; e += kThreads) nexts[e] = 0;
  int32_t *mine = nexts + warp * p.experts;
  __syncthreads();
  // this stretch's slots per warp and expert
  for (int i = a + lane; i < b; i += 32) {
    const int e = p.ids[slot0 + i];
    if (e >= 0) atomicAdd(mine + e, 1);
  }
  __syncthreads();
  // Experts in turn by threads, kThreads at a time: all slots of the experts before, of the stretches before, of the warps before.
  int run = 0;
  float loss = 0.f;
  for (int e0 = 0; e0 < p.experts; e0 += kThreads) {
    const int e = e0 + threadIdx.x;
    int before = 0, all = 0;
    float prob = 0.f;
    if (e < p.experts) {
#pragma unroll 32
      for (int c = 0; c < stretches; ++c) {
        const int n = __ldg(p.part_count + static_cast<int64_t>(c) * p.experts + e);
        all += n;
        before += c < static_cast<int>(blockIdx.x) ? n : 0;
      }
      if (blockIdx.x == 0) {
#pragma unroll 32
        for (int c = 0; c < stretches; ++c) prob += p.part_prob[static_cast<int64_t>(c) * p.experts + e];
      }
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
    for (int k = 0; k < kWarps; ++k) {
      if (k < warp) base += scan[k];
      run += scan[k];
    }
    const int offset = base + incl - all;
    if (e < p.experts) {
      int at = offset + before;
      for (int k = 0; k < kWarps; ++k) {
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
  for (int i0 = a; i0 < b; i0 += 32) {
    const int i = i0 + lane;
    const int e = i < b ? p.ids[slot0 + i] : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    const uint32_t before = same & ((1u << lane) - 1u);
    int at = 0;
    if (e >= 0) at = mine[e] + __popc(before);
    __syncwarp();
    if (e >= 0 && before == 0) mine[e] += __popc(same);
    __syncwarp();
    if (e >= 0 && in_bounds(p.order + at, 4, p.order, size, p.status)) p.order[at] = slot0 + i;
  }
  // places that no slot has
  const int64_t slots = static_cast<int64_t>(p.rows) * p.top_k;
  for (int64_t i = run + static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < slots; i += static_cast<int64_t>(stretches) * kThreads)
    if (in_bounds(p.order + i, 4, p.order, size, p.status)) p.order[i] = -1;
  if (blockIdx.x == 0) {
    float z = 0.f;
    int live = 0;
    for (int c = threadIdx.x; c < stretches; c += kThreads) {
      z += p.part_z[c];
      live += p.part_live[c];
    }
    loss = block_sum(loss, red);
    z = block_sum(z, red);
    live = __reduce_add_sync(0xffffffffu, live);
    __syncthreads();
    if (lane == 0) scan[warp] = live;
    __syncthreads();
    if (threadIdx.x == 0) {
      live = 0;
      for (int k = 0; k < kWarps; ++k) live += scan[k];
      const double t = live;
      if (in_bounds(p.offsets + p.experts, 4, p.offsets, (static_cast<size_t>(p.experts) + 1) * 4, p.status)) p.offsets[p.experts] = run;
      *p.live_rows = live;
      *p.loss = live == 0 ? 0.f : static_cast<float>(p.balance * (p.experts * static_cast<double>(loss) / (p.top_k * t * t)) + p.z * (z / t));
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
// dL = P (s - sum of P s + 2 z logz / T) with s = balance E counts / (k T^2), and the weights' own part.
template <int DT, int V>
__global__ void __launch_bounds__(kBackWarps * 32) ns_route_backward_kernel(const __grid_constant__ RouteBackParams p) {
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
    float q[V], s[V], dot = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * 32 + lane;
      q[i] = c < p.experts ? expf(Elem<DT>::to_f(x[c]) - lz) : 0.f;
      s[i] = slope[c] + (p.renormalise ? 0.f : part[warp][c]);
      dot += q[i] * s[i];
    }
    dot = warp_sum(dot) - 2.f * p.z / t * lz;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = i * 32 + lane;
      float d = q[i] * (s[i] - dot);
      if (p.renormalise) d += part[warp][c];
      if (c < p.experts && in_bounds(out + c, sizeof(E), p.dlogits, size, p.status)) out[c] = Elem<DT>::from_f(d);
    }
    __syncwarp();
    if (e >= 0) part[warp][e] = 0.f;
    __syncwarp();
  }
}

// Lanes of a row and logits a lane of the first launch: rows of up to 256 experts share a warp, 16 logits a lane, so that a
// step of the choice serves several rows.
template <typename F>
int by_lanes(int experts, F &&f) {
  using std::integral_constant;
  return experts <= 16    ? f(integral_constant<int, 4>{}, integral_constant<int, 4>{})
         : experts <= 32  ? f(integral_constant<int, 4>{}, integral_constant<int, 8>{})
         : experts <= 64  ? f(integral_constant<int, 8>{}, integral_constant<int, 8>{})
         : experts <= 128 ? f(integral_constant<int, 8>{}, integral_constant<int, 16>{})
         : experts <= 256 ? f(integral_constant<int, 16>{}, integral_constant<int, 16>{})
         : experts <= 512 ? f(integral_constant<int, 32>{}, integral_constant<int, 16>{})
                          : f(integral_constant<int, 32>{}, integral_constant<int, 32>{});
}

template <typename F>
int by_width(int experts, F &&f) {
  return experts <= 32 ? f(std::integral_constant<int, 1>{}) : experts <= 64 ? f(std::integral_constant<int, 2>{})
         : experts <= 128 ? f(std::integral_constant<int, 4>{}) : experts <= 256 ? f(std::integral_constant<int, 8>{})
         : experts <= 512 ? f(std::integral_constant<int, 16>{}) : f(std::integral_constant<int, 32>{});
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
  p.part_prob = reinterpret_cast<float *>(p.part_count + static_cast<int64_t>(grid) * experts);
  p.part_z = p.part_prob + static_cast<int64_t>(grid) * experts;
  p.part_live = reinterpret_cast<int32_t *>(p.part_z + grid);
  return call.launch(kOpRoute, [&] {
    by_lanes(experts, [&](auto l, auto v) {
      if (dtype == NS_BF16)
        ns_route_rows_kernel<kBF16, decltype(l)::value, decltype(v)::value><<<grid, 32 * kRowWarps<decltype(l)::value, decltype(v)::value>, 0, call.s>>>(p);
      else
        ns_route_rows_kernel<kF32, decltype(l)::value, decltype(v)::value><<<grid, 32 * kRowWarps<decltype(l)::value, decltype(v)::value>, 0, call.s>>>(p);
      return 0;
    });
    count_launch();
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = call.s;
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(kWarps) * experts * 4;
    static SmemOptIn opt_in;
    if (opt_in.ensure(reinterpret_cast<const void *>(ns_route_order_kernel), static_cast<int>(cfg.dynamicSmemBytes))) return -1;
    if (cudaLaunchKernelEx(&cfg, ns_route_order_kernel, p) != cudaSuccess) {
      cudaGetLastError();
      return -1;
    }
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
  const int grid = static_cast<int>(std::min<int64_t>((rows + kBackWarps - 1) / kBackWarps, static_cast<int64_t>(call.sms) * 8));
  return call.launch(kOpRoute, [&] {
    by_width(experts, [&](auto v) {
      if (dtype == NS_BF16)
        ns_route_backward_kernel<kBF16, decltype(v)::value><<<grid, 32 * kBackWarps, 0, call.s>>>(p);
      else
        ns_route_backward_kernel<kF32, decltype(v)::value><<<grid, 32 * kBackWarps, 0, call.s>>>(p);
      return 0;
    });
    count_launch();
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
  });
}
