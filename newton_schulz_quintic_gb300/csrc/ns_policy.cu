// ns_policy.cu -- log probabilities of target tokens and the clipped policy
// loss with a KL term, with the gradient of the logits (include/ns.h).
//
// Per row, with m the largest logit, k = inv_temperature * log2(e) and s = sum
// of 2^((v - m) k) over the row's logits v: logp = ((v[y] - m) k - log2 s) /
// log2(e). The difference comes before the factor, so logits up to the type's
// largest and lowest values do not overflow. Each thread keeps a running
// maximum and sum; they are merged over the CTA (or over the cluster, where
// few rows leave SMs idle) in a fixed order.
//
// A row's gradient depends on nothing but the row, so the second pass
// (softmax times the row's coefficient) follows at once. It is the memory
// that bounds this: one read and one write of the logits. The second read
// comes from L2 as long as the rows in flight fit there.
// The loss is summed over the rows by one CTA in a fixed order.
#include <algorithm>
#include <cmath>

#include "../../include/ns.h"
#include "ns_rows.cuh"

namespace ns {

namespace {

struct PolicyParams {
  const void *logits;
  void *dlogits;  // nullptr: no gradient
  Ids targets;
  const float *old_logp, *ref_logp, *advantage, *weight;  // weight nullptr: log probabilities only
  float *logp, *kl, *loss, *row_loss;
  int64_t rows, ld, ld_d;
  int vocab;
  float inv_temp, clip_low, clip_high, kl_coef;
  int cluster;  // CTAs per row
  int *status;
};

constexpr int kMaxThreads = 1024;
constexpr int kMaxCluster = 8;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The largest logit m so far and s = sum of 2^((v - m) k); m = -inf, s = 0 is nothing.
struct MaxSum {
  float m, s;
};
__device__ __forceinline__ MaxSum merge(MaxSum a, MaxSum b, float k) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return MaxSum{m, a.s + b.s};  // nothing yet (or NaN sums, kept)
  return MaxSum{m, a.s * exp2_fast((a.m - m) * k) + b.s * exp2_fast((b.m - m) * k)};
}

struct RowResult {
  float logp, kl, loss, slope;
};

// The row's outputs from its target's log probability.
__device__ __forceinline__ RowResult policy_row(const PolicyParams &p, int64_t t, float logp) {
  RowResult r{logp, 0.f, 0.f, 0.f};
  if (!p.weight) return r;
  const float adv = p.advantage[t], w = p.weight[t];
  const float ratio = p.old_logp ? expf(logp - p.old_logp[t]) : 1.f;
  const float a = ratio * adv, b = fminf(fmaxf(ratio, 1.f - p.clip_low), 1.f + p.clip_high) * adv;
  float slope = a <= b ? -a : 0.f;
  if (p.ref_logp) {
    const float d = p.ref_logp[t] - logp, e = expm1f(d);
    r.kl = e - d;
    slope -= p.kl_coef * e;
  }
  r.loss = w * (p.kl_coef * r.kl - fminf(a, b));
  r.slope = w * slope * p.inv_temp;
  return r;
}

// Largest of a pack's values.
template <int DT, int VEC>
__device__ __forceinline__ float pack_max(const Pack<DT, VEC> &v) {
  if constexpr (DT == kBF16 && VEC == 8) {  // two at a time; NaN is passed over here and reaches the sum
    const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(v.w);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
  } else {
    float m = v.get(0);
#pragma unroll
    for (int e = 1; e < VEC; ++e) m = fmaxf(m, v.get(e));
    return m;
  }
}

// One row per cluster of p.cluster CTAs (1: no cluster); CTA rank r takes
// every p.cluster-th stretch of the row.
template <int DT, int VEC, bool GRAD>
__global__ void __launch_bounds__(kMaxThreads) ns_policy_kernel(const __grid_constant__ PolicyParams p) {
  using P = Pack<DT, VEC>;
  using E = typename P::E;
  __shared__ MaxSum part[kMaxThreads / 32];
  __shared__ MaxSum mine;  // this CTA's share of the row, read by the cluster
  __shared__ MaxSum all;
  __shared__ RowResult res;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int rank = p.cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int first = (rank * blockDim.x + threadIdx.x) * VEC, stride = p.cluster * blockDim.x * VEC;
  const float k = p.inv_temp * kLog2e;
  const size_t dsize = static_cast<size_t>((p.rows - 1) * p.ld_d + p.vocab) * sizeof(E);
  for (int64_t t = blockIdx.x / p.cluster; t < p.rows; t += gridDim.x / p.cluster) {
    const E *x = static_cast<const E *>(p.logits) + t * p.ld;
    E *g = GRAD ? static_cast<E *>(p.dlogits) + t * p.ld_d : nullptr;
    const int y = p.targets.get(t);
    bool live = y >= 0 && (!p.weight || p.weight[t] != 0.f);  // the same in every thread of the cluster
    MaxSum a{-INFINITY, 0.f};
    if (live) {
#pragma unroll 4
      for (int c = first; c < p.vocab; c += stride) {
        P v;
        v.load(x + c);
        const float top = pack_max<DT, VEC>(v);
        if (top > a.m) {
          a.s *= exp2_fast((a.m - top) * k);
          a.m = top;
        }
        // a pack of -inf alone adds 2^(-inf - 0) = 0; NaN reaches the sum either way
        const float m = a.m == -INFINITY ? 0.f : a.m;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) s += exp2_fast((v.get(e) - m) * k);
        a.s += s;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        a = merge(a, MaxSum{__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o)}, k);
      if (lane == 0) part[warp] = a;
      __syncthreads();
      if (warp == 0) {
        a = lane < warps ? part[lane] : MaxSum{-INFINITY, 0.f};
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          a = merge(a, MaxSum{__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o)}, k);
        if (lane == 0) mine = a;
      }
      if (p.cluster > 1) {
        cluster_sync();
        if (warp == 0) {
          MaxSum b{-INFINITY, 0.f};
          if (lane < p.cluster) {
            const uint32_t at = mapa_shared(smem_u32(&mine), lane);
            b.m = __uint_as_float(ld_shared_cluster_u32(at));
            b.s = __uint_as_float(ld_shared_cluster_u32(at + 4));
          }
          a = b;
#pragma unroll
          for (int o = kMaxCluster / 2; o > 0; o >>= 1)
            a = merge(a, MaxSum{__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o)}, k);
        }
      }
      if (threadIdx.x == 0) {
        all = a;
        RowResult r{0.f, 0.f, 0.f, 0.f};
        if (a.s != 0.f)  // else every logit is -inf: no distribution
          r = policy_row(p, t, ((Elem<DT>::to_f(x[y]) - a.m) * k - log2f(a.s)) * kLn2);
        res = r;
      }
      __syncthreads();
      a = all;
      if (a.s == 0.f) live = false;
    }
    if (threadIdx.x == 0 && rank == 0) {
      const RowResult r = live ? res : RowResult{0.f, 0.f, 0.f, 0.f};
      if (in_bounds(p.logp + t, 4, p.logp, p.rows * 4, p.status)) p.logp[t] = r.logp;
      if (p.weight) {
        if (in_bounds(p.kl + t, 4, p.kl, p.rows * 4, p.status)) p.kl[t] = r.kl;
        p.row_loss[t] = r.loss;
      }
    }
    if constexpr (GRAD) {
      if (live) {
        const float slope = res.slope, scale = -slope / a.s;
        const bool in_place = p.dlogits == p.logits;
        // in place, the target's logit is read by every CTA before any overwrites it
        if (p.cluster > 1 && in_place) cluster_sync();
#pragma unroll 4
        for (int c = first; c < p.vocab; c += stride) {
          P v;
          v.load_stream(x + c);
#pragma unroll
          for (int e = 0; e < VEC; ++e) v.set(e, scale * exp2_fast((v.get(e) - a.m) * k));
          if (static_cast<unsigned>(y - c) < VEC) {  // the target's pack, again with its 1
#pragma unroll
            for (int e = 0; e < VEC; ++e)
              if (c + e == y) v.set(e, fmaf(scale, exp2_fast((Elem<DT>::to_f(x[y]) - a.m) * k), slope));
          }
          v.store_stream(g + c, p.dlogits, dsize, p.status);
        }
      } else {
        P v;
#pragma unroll
        for (int e = 0; e < VEC; ++e) v.set(e, 0.f);
        for (int c = first; c < p.vocab; c += stride) v.store_stream(g + c, p.dlogits, dsize, p.status);
      }
    }
    // shared values are free for the next row (in a cluster: once all have read `mine`)
    if (p.cluster > 1)
      cluster_sync();
    else
      __syncthreads();
  }
}

// loss = sum of the rows' losses: one CTA, each thread a fixed stride, then a
// fixed tree.
__global__ void __launch_bounds__(1024) ns_policy_sum_kernel(const __grid_constant__ PolicyParams p) {
  __shared__ float part[32];
  float s = 0.f;
  for (int64_t t = threadIdx.x; t < p.rows; t += 1024) s += p.row_loss[t];
  s = warp_sum(s);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x < 32) {
    s = warp_sum(part[threadIdx.x]);
    if (threadIdx.x == 0 && in_bounds(p.loss, 4, p.loss, 4, p.status)) *p.loss = s;
  }
}

template <int DT, int VEC, bool GRAD>
int run_policy(PolicyParams p, int sms, cudaStream_t s) {
  if (p.rows > 0) {
    constexpr int elt = DT == kBF16 ? 2 : 4;
    // threads: two packs or more each, down to a warp
    int threads = kMaxThreads;
    while (threads > 32 && static_cast<int64_t>(threads) * 2 * VEC > p.vocab) threads /= 2;
    // few rows: a cluster of CTAs per row while SMs are idle and every thread keeps two packs
    p.cluster = 1;
    while (p.cluster < kMaxCluster && p.rows * p.cluster * 2 <= sms &&
           static_cast<int64_t>(threads) * p.cluster * 4 * VEC <= p.vocab)
      p.cluster *= 2;
    // as many CTAs as are resident, but no more rows in flight than L2 keeps
    // for the second read (kL2Rows bytes) unless that leaves SMs idle
    constexpr int64_t kL2Rows = int64_t(80) << 20;
    int64_t grid = static_cast<int64_t>(sms) * (2048 / threads);
    if (GRAD) grid = std::min(grid, std::max<int64_t>(sms, kL2Rows / std::max<int64_t>(1, static_cast<int64_t>(p.vocab) * elt)));
    grid = std::min(grid, p.rows * p.cluster) / p.cluster * p.cluster;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&cfg, ns_policy_kernel<DT, VEC, GRAD>, p) != cudaSuccess) {
      cudaGetLastError();
      return -1;
    }
    count_launch();
  }
  if (p.weight) {
    ns_policy_sum_kernel<<<1, 1024, 0, s>>>(p);
    count_launch();
  }
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

template <int DT, int VEC>
int run_policy(const PolicyParams &p, int sms, cudaStream_t s) {
  return p.dlogits ? run_policy<DT, VEC, true>(p, sms, s) : run_policy<DT, VEC, false>(p, sms, s);
}

int policy_call(PolicyParams &p, int dtype, void *stream) {
  OpCall call(stream);
  if (call.rc) return call.rc;
  p.status = call.status;
  const int elt = dtype == NS_BF16 ? 2 : 4;
  if (p.weight) {
    uint8_t *ws = nullptr;
    if (const int rc = call.workspace(kSlotPolicy, static_cast<size_t>(p.rows) * 4, &ws)) return rc;
    p.row_loss = reinterpret_cast<float *>(ws);
  }
  const int vec = 16 / elt;
  const bool wide = p.vocab % vec == 0 && rows_aligned(p.logits, p.ld, elt, vec) &&
                    (!p.dlogits || rows_aligned(p.dlogits, p.ld_d, elt, vec));
  return call.launch(kOpPolicy, [&] {
    if (dtype == NS_BF16) return wide ? run_policy<kBF16, 8>(p, call.sms, call.s) : run_policy<kBF16, 1>(p, call.sms, call.s);
    return wide ? run_policy<kF32, 4>(p, call.sms, call.s) : run_policy<kF32, 1>(p, call.sms, call.s);
  });
}

}  // namespace
}  // namespace ns

using namespace ns;

extern "C" int ns_token_logprobs(const void *logits, int64_t ld_logits, int64_t rows, int64_t vocab,
                                 const void *targets, int id_type, float inv_temperature, float *logp, int dtype,
                                 void *stream) {
  if ((dtype != NS_F32 && dtype != NS_BF16) || (id_type != NS_I32 && id_type != NS_I64)) return NS_EINVAL;
  if (bad_shape(rows, vocab, ld_logits) || !std::isfinite(inv_temperature) || inv_temperature <= 0) return NS_EINVAL;
  if (rows == 0) return NS_OK;
  if (!targets || !logp || (vocab > 0 && !logits)) return NS_EINVAL;
  const int elt = dtype == NS_BF16 ? 2 : 4, ielt = id_type == NS_I64 ? 8 : 4;
  if (misaligned(logits, elt) || misaligned(logp, 4) || misaligned(targets, ielt)) return NS_EALIGN;
  const Range out(logp, 1, rows, rows, 4);
  if (out.overlaps(Range(logits, rows, vocab, ld_logits, elt)) || out.overlaps(Range(targets, 1, rows, rows, ielt)))
    return NS_EINVAL;
  PolicyParams p{};
  p.logits = logits;
  p.targets = Ids{targets, id_type == NS_I64, static_cast<int>(vocab)};
  p.logp = logp;
  p.rows = rows;
  p.ld = ld_logits;
  p.vocab = static_cast<int>(vocab);
  p.inv_temp = inv_temperature;
  return policy_call(p, dtype, stream);
}

extern "C" int ns_policy_loss(const void *logits, int64_t ld_logits, int64_t rows, int64_t vocab,
                              const void *targets, int id_type, const float *old_logp, const float *ref_logp,
                              const float *advantage, const float *weight, float inv_temperature, float clip_low,
                              float clip_high, float kl_coef, float *loss, float *logp, float *kl, void *dlogits,
                              int64_t ld_dlogits, int dtype, void *stream) {
  if ((dtype != NS_F32 && dtype != NS_BF16) || (id_type != NS_I32 && id_type != NS_I64)) return NS_EINVAL;
  if (bad_shape(rows, vocab, ld_logits) || (dlogits && bad_shape(rows, vocab, ld_dlogits))) return NS_EINVAL;
  if (!std::isfinite(inv_temperature) || inv_temperature <= 0 || !std::isfinite(clip_low) || !std::isfinite(clip_high) ||
      !std::isfinite(kl_coef) || clip_low < 0 || clip_high < 0 || kl_coef < 0)
    return NS_EINVAL;
  if (!loss) return NS_EINVAL;
  if (rows > 0 && (!targets || !advantage || !weight || !logp || !kl || (vocab > 0 && !logits))) return NS_EINVAL;
  const int elt = dtype == NS_BF16 ? 2 : 4, ielt = id_type == NS_I64 ? 8 : 4;
  if (misaligned(logits, elt) || misaligned(dlogits, elt) || misaligned(targets, ielt) || misaligned(loss, 4) ||
      misaligned(logp, 4) || misaligned(kl, 4) || misaligned(old_logp, 4) || misaligned(ref_logp, 4) ||
      misaligned(advantage, 4) || misaligned(weight, 4))
    return NS_EALIGN;
  const Range in[] = {Range(targets, 1, rows, rows, ielt), Range(old_logp, 1, rows, rows, 4),
                      Range(ref_logp, 1, rows, rows, 4),   Range(advantage, 1, rows, rows, 4),
                      Range(weight, 1, rows, rows, 4),     Range(logits, rows, vocab, ld_logits, elt)};
  const Range out[] = {Range(loss, 1, 1, 1, 4), Range(logp, 1, rows, rows, 4), Range(kl, 1, rows, rows, 4),
                       Range(dlogits, rows, vocab, ld_dlogits, elt)};
  for (int i = 0; i < 4; ++i) {
    for (int k = 0; k < 6; ++k)
      if (out[i].overlaps(in[k]) && !(i == 3 && k == 5 && dlogits == logits && ld_dlogits == ld_logits)) return NS_EINVAL;
    for (int k = 0; k < i; ++k)
      if (out[i].overlaps(out[k])) return NS_EINVAL;
  }
  static const float none = 0.f;  // rows == 0: nothing is read
  PolicyParams p{};
  p.logits = logits;
  p.dlogits = dlogits;
  p.targets = Ids{targets, id_type == NS_I64, static_cast<int>(vocab)};
  p.old_logp = old_logp;
  p.ref_logp = ref_logp;
  p.advantage = advantage;
  p.weight = rows > 0 ? weight : &none;
  p.logp = logp;
  p.kl = kl;
  p.loss = loss;
  p.rows = rows;
  p.ld = ld_logits;
  p.ld_d = ld_dlogits;
  p.vocab = static_cast<int>(vocab);
  p.inv_temp = inv_temperature;
  p.clip_low = clip_low;
  p.clip_high = clip_high;
  p.kl_coef = kl_coef;
  return policy_call(p, dtype, stream);
}
