// ns_policy.cu -- log probabilities of target tokens and the clipped policy
// loss with a KL term, with the gradient of the logits (include/ns.h).
//
// Per row: one pass over the logits keeps each thread's running maximum m and
// sum of exp(z - m); merged over the CTA they give logp = z[y] - m - log(sum).
// A row's gradient depends on nothing but the row, so the second pass
// (softmax times the row's coefficient) follows at once. The loss is summed
// over the rows by one CTA in a fixed order.
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
  int *status;
};

constexpr int kPolicyThreads = 512;

// (m, s) stands for s * exp(m); m = -inf, s = 0 is nothing.
struct MaxSum {
  float m, s;
};
__device__ __forceinline__ MaxSum merge(MaxSum a, MaxSum b) {
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return MaxSum{m, a.s + b.s};  // nothing yet (or NaN sums, kept)
  return MaxSum{m, a.s * __expf(a.m - m) + b.s * __expf(b.m - m)};
}

struct RowResult {
  float logp, kl, loss, slope;
};

// The row's outputs from its target's z - max and log(sum).
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

template <int DT, int VEC>
__global__ void __launch_bounds__(kPolicyThreads) ns_policy_kernel(const __grid_constant__ PolicyParams p) {
  using P = Pack<DT, VEC>;
  using E = typename P::E;
  __shared__ MaxSum part[kPolicyThreads / 32];
  __shared__ MaxSum all;
  __shared__ RowResult res;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t dsize = static_cast<size_t>((p.rows - 1) * p.ld_d + p.vocab) * sizeof(E);
  for (int64_t t = blockIdx.x; t < p.rows; t += gridDim.x) {
    const E *x = static_cast<const E *>(p.logits) + t * p.ld;
    E *g = p.dlogits ? static_cast<E *>(p.dlogits) + t * p.ld_d : nullptr;
    const int y = p.targets.get(t);
    bool live = y >= 0 && (!p.weight || p.weight[t] != 0.f);
    MaxSum a{-INFINITY, 0.f};
    if (live) {
      for (int c = threadIdx.x * VEC; c < p.vocab; c += kPolicyThreads * VEC) {
        P v;
        v.load(x + c);
        float top = -INFINITY;
#pragma unroll
        for (int e = 0; e < VEC; ++e) top = fmaxf(top, v.get(e) * p.inv_temp);
        if (top > a.m) {
          a.s *= __expf(a.m - top);
          a.m = top;
        }
        // a pack of -inf alone adds exp(-inf - 0) = 0; NaN reaches the sum either way
        const float m = a.m == -INFINITY ? 0.f : a.m;
#pragma unroll
        for (int e = 0; e < VEC; ++e) a.s += __expf(fmaf(v.get(e), p.inv_temp, -m));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        a = merge(a, MaxSum{__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o)});
      if (lane == 0) part[warp] = a;
      __syncthreads();
      if (threadIdx.x == 0) {
        for (int k = 1; k < kPolicyThreads / 32; ++k) a = merge(a, part[k]);
        all = a;
        RowResult r{0.f, 0.f, 0.f, 0.f};
        if (a.s != 0.f) {  // else every logit is -inf: no distribution
          const float z = Elem<DT>::to_f(x[y]) * p.inv_temp;
          r = policy_row(p, t, (z - a.m) - logf(a.s));
        }
        res = r;
      }
      __syncthreads();
      a = all;
      if (a.s == 0.f) live = false;
    } else if (threadIdx.x == 0) {
      res = RowResult{0.f, 0.f, 0.f, 0.f};
    }
    if (threadIdx.x == 0) {
      if (in_bounds(p.logp + t, 4, p.logp, p.rows * 4, p.status)) p.logp[t] = res.logp;
      if (p.weight) {
        if (in_bounds(p.kl + t, 4, p.kl, p.rows * 4, p.status)) p.kl[t] = res.kl;
        p.row_loss[t] = res.loss;
      }
    }
    if (g) {
      const float slope = live ? res.slope : 0.f, scale = live ? -slope / a.s : 0.f;
      for (int c = threadIdx.x * VEC; c < p.vocab; c += kPolicyThreads * VEC) {
        P v;
        if (live) {
          v.load(x + c);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            float d = scale * __expf(fmaf(v.get(e), p.inv_temp, -a.m));
            if (c + e == y) d += slope;
            v.set(e, d);
          }
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) v.set(e, 0.f);
        }
        v.store(g + c, p.dlogits, dsize, p.status);
      }
    }
    __syncthreads();  // `all`, `res` and `part` are free for the next row
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

template <int DT, int VEC>
int run_policy(const PolicyParams &p, int sms, cudaStream_t s) {
  if (p.rows > 0) {
    const int grid = static_cast<int>(p.rows < sms * 4 ? p.rows : sms * 4);
    ns_policy_kernel<DT, VEC><<<grid, kPolicyThreads, 0, s>>>(p);
    count_launch();
  }
  if (p.weight) {
    ns_policy_sum_kernel<<<1, 1024, 0, s>>>(p);
    count_launch();
  }
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
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
