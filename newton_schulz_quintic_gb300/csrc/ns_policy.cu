// ns_policy.cu -- log probabilities of target tokens and the clipped policy
// loss with a KL term, with the gradient of the logits (include/ns.h).
//
// Per row, with m the largest logit, k = inv_temperature * log2(e) and s = sum
// of 2^(v k - m k) over the row's logits v: logp = (v[y] - m) inv_temperature -
// log s, corrected by what rounding m k left out (the few operations of that
// line in fp64: its terms are about 10 where the KL term wants its differences
// from old and reference to 1e-7). A row's gradient depends on nothing but the row, so it follows at
// once: softmax times the row's coefficient.
//
// One CTA per row (a cluster of up to 8 where few rows leave SMs idle), in two
// passes. What bounds this is one read and one write of the logits: between
// the passes a row stays in shared memory as far as that goes (110 KB a CTA,
// two CTAs an SM) and in L2 beyond. That leaves the instructions per element:
// packed maxima and pairs of fp32 operations. Measured at 8192 x 131072 bf16
// with a quarter of the rows masked: 660 us, 85 % of the copy bandwidth (564
// us). On the way there: separate fp32 operations 800 us; CTAs that walk over
// the rows in a fixed stride 754 us, because masked rows are cheap and leave
// some CTAs with more work, where the block scheduler hands rows out as CTAs
// finish; and a row held in the registers of 8 CTAs, 1160 us, a cluster
// barrier a row.
//
// Packs of 16 bytes sit on 16-byte boundaries whatever a row's own alignment
// is; the ragged ends go element by element, and so does a gradient whose
// rows lie differently on those boundaries than the logits'. All sums run in
// a fixed order that depends on the logits' shape and alignment alone, so log
// probabilities are the same bits with and without a gradient. The loss is
// summed over the rows, in a fixed order, by the CTA that finishes last, or by
// a launch of its own where that CTA would be long at it.
#include <algorithm>
#include <cmath>
#include <type_traits>

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
  int kept;     // packs per thread that stay in shared memory between the passes
  int *done;    // rows finished, 0 between calls; nullptr: the loss is summed by ns_policy_sum_kernel
  int packed;   // the gradient's rows take the packs that the logits' rows are read in
  int *status;
};

constexpr int kMaxThreads = 512;
constexpr int kMaxCluster = 8;
constexpr int64_t kKeepBytes = 216 * 1024;  // shared memory of an SM for rows kept between the passes
constexpr float kLog2e = 1.44269504088896340736f;
constexpr double kLn2 = 0.69314718055994530942;
constexpr float kLargest = 3.402823466e38f;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// How a logit v becomes the power 2^((v - m) k). As long as |m k| is below
// kPlain, by one fused multiply-add: v k - mk, with mk = m k rounded, is off by
// that rounding (2^-5 at most), the same for every v. Logits beyond (the
// type's largest and lowest values, or tiny temperatures) take the difference
// first. m = -inf: nothing but -inf so far, whose powers are 0.
// (Here and below, products and sums that a compiler may contract one way in one
// instance of the kernel and another way in the next are written out, so that
// all of them round alike.)
constexpr float kPlain = 1048576.f;
struct Scale {
  float k, m, mk;
  bool plain;
  __device__ __forceinline__ Scale(float top, float factor) {
    k = factor;
    m = top == -INFINITY ? 0.f : top;
    mk = __fmul_rn(m, k);
    plain = fabsf(mk) <= kPlain;
  }
  // what the powers are relative to, over 2^(m k), as an exponent
  __device__ __forceinline__ float left_out() const { return plain ? fmaf(m, k, -mk) : 0.f; }
  __device__ __forceinline__ float power(float v) const {
    return exp2_fast(plain ? fmaf(v, k, -mk) : __fmul_rn(__fadd_rn(v, -m), k));
  }
};

// The largest logit m so far and s = sum of the powers relative to it; m = -inf, s = 0 is nothing.
struct MaxSum {
  float m, s;
};
// What a sum relative to `from` is multiplied by to be relative to m >= from.
__device__ __forceinline__ float rebase(float from, float m, float k) {
  if (from == m) return 1.f;
  if (from == -INFINITY) return 0.f;
  const Scale a(from, k), b(m, k);
  if (a.plain && b.plain) return exp2_fast(a.mk - b.mk);  // both as rounded
  return exp2_fast(fmaf(from - m, k, b.left_out() - a.left_out()));
}
__device__ __forceinline__ MaxSum merge(MaxSum a, MaxSum b, float k) {
  const float m = fmaxf(a.m, b.m);
  return MaxSum{m, fmaf(a.s, rebase(a.m, m, k), __fmul_rn(b.s, rebase(b.m, m, k)))};
}

// log s, with the exponent's part in fp64 (s is 1 or more as a rule; infinities and NaN pass through).
__device__ __forceinline__ double log_of(float s) {
  if (!(s >= 1.f && s <= kLargest)) return logf(s);
  const int e = (__float_as_int(s) >> 23) - 127;
  const float f = __int_as_float((__float_as_int(s) & 0x7fffff) | 0x3f800000);  // 1 .. 2
  return e * kLn2 + logf(f);
}

struct RowInputs {
  float old_logp, ref_logp, advantage, weight;
};
struct RowResult {
  float logp, kl, loss, slope;
};

__device__ __forceinline__ RowInputs row_inputs(const PolicyParams &p, int64_t t) {
  RowInputs r{0.f, 0.f, 0.f, 0.f};
  if (!p.weight) return r;
  r.weight = p.weight[t];
  r.advantage = p.advantage[t];
  if (p.old_logp) r.old_logp = p.old_logp[t];
  if (p.ref_logp) r.ref_logp = p.ref_logp[t];
  return r;
}

// The smaller and the larger of two, NaN where either is (fminf and fmaxf take the other).
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// The row's outputs from its target's log probability.
__device__ __forceinline__ RowResult policy_row(const PolicyParams &p, const RowInputs &in, double logp) {
  RowResult r{static_cast<float>(logp), 0.f, 0.f, 0.f};
  if (!p.weight) return r;
  const float apart = p.old_logp ? static_cast<float>(logp - in.old_logp) : 0.f;
  const float ratio = p.old_logp ? expf(apart) : 1.f;
  // a ratio beyond fp32's largest value is finite all the same, and 0 times no advantage
  const float a = in.advantage == 0.f && fabsf(apart) <= kLargest ? 0.f : ratio * in.advantage;
  const float b = min_nan(max_nan(ratio, 1.f - p.clip_low), 1.f + p.clip_high) * in.advantage;
  const float gain = min_nan(a, b);
  float slope = a <= b ? -a : a > b ? 0.f : gain;  // neither: NaN
  if (p.ref_logp) {
    const float d = static_cast<float>(in.ref_logp - logp), e = expm1f(d);
    r.kl = e - d;
    if (p.kl_coef != 0.f) slope -= p.kl_coef * e;  // 0 times a term beyond fp32's range is NaN
  }
  r.loss = in.weight * ((p.kl_coef != 0.f ? p.kl_coef * r.kl : 0.f) - gain);
  r.slope = in.weight * slope * p.inv_temp;
  return r;
}

// Writes a row's scalars.
__device__ __forceinline__ void write_result(const PolicyParams &p, int64_t t, const RowResult &r) {
  if (in_bounds(p.logp + t, 4, p.logp, p.rows * 4, p.status)) p.logp[t] = r.logp;
  if (p.weight) {
    if (in_bounds(p.kl + t, 4, p.kl, p.rows * 4, p.status)) p.kl[t] = r.kl;
    p.row_loss[t] = r.loss;
  }
}

// Sum of the rows' losses by the calling CTA, in thread 0: each thread a
// fixed stride, then a fixed tree. part: a float per warp.
__device__ __forceinline__ float sum_losses(const PolicyParams &p, float *part) {
  float s = 0.f;
#pragma unroll 8
  for (int64_t t = threadIdx.x; t < p.rows; t += blockDim.x) s += __ldcg(p.row_loss + t);
  s = warp_sum(s);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
  __syncthreads();
  s = threadIdx.x < blockDim.x >> 5 ? part[threadIdx.x] : 0.f;
  return threadIdx.x < 32 ? warp_sum(s) : 0.f;
}

// 16 bytes of a row.
template <int DT>
struct RowPack {
  static constexpr int VEC = DT == kBF16 ? 8 : 4;
  using E = typename Elem<DT>::T;
  Pack<DT, VEC> v;
  // its i-th pair of values
  __device__ __forceinline__ float2 pair(int i) const {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(v.w);
    if constexpr (DT == kBF16)
      return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    else
      return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  }
  __device__ __forceinline__ void set_pair(int i, float2 x) {
    uint32_t *w = reinterpret_cast<uint32_t *>(v.w);
    if constexpr (DT == kBF16) {
      const __nv_bfloat162 b = __float22bfloat162_rn(x);
      w[i] = *reinterpret_cast<const uint32_t *>(&b);
    } else {
      w[2 * i] = __float_as_uint(x.x);
      w[2 * i + 1] = __float_as_uint(x.y);
    }
  }
  // largest value; NaN is passed over here and reaches the sum
  __device__ __forceinline__ float top() const {
    if constexpr (DT == kBF16) {
      const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(v.w);
      const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
      return fmaxf(__low2float(m), __high2float(m));
    } else {
      return fmaxf(fmaxf(v.get(0), v.get(1)), fmaxf(v.get(2), v.get(3)));
    }
  }
  template <bool PLAIN>
  __device__ __forceinline__ float2 powers(int i, const Scale &f) const {
    const float2 v = pair(i), k = make_float2(f.k, f.k);
    const float2 x = PLAIN ? __ffma2_rn(v, k, make_float2(-f.mk, -f.mk))
                           : __fmul2_rn(__fadd2_rn(v, make_float2(-f.m, -f.m)), k);
    return make_float2(exp2_fast(x.x), exp2_fast(x.y));
  }
  template <bool PLAIN>
  __device__ __forceinline__ float sum(const Scale &f) const {
    float2 s = powers<PLAIN>(0, f);
#pragma unroll
    for (int i = 1; i < VEC / 2; ++i) s = __fadd2_rn(s, powers<PLAIN>(i, f));
    return __fadd_rn(s.x, s.y);
  }
  template <bool PLAIN>
  __device__ __forceinline__ void to_gradient(float scale, const Scale &f) {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) set_pair(i, __fmul2_rn(make_float2(scale, scale), powers<PLAIN>(i, f)));
  }
};

// A row as its packs: `count` of them, the first starting `phase` elements
// before the row. Packs [full0, full1) lie in it whole; the one before and
// the one after, if any, are its ragged ends.
struct RowPacks {
  int phase, full0, full1;
  template <int DT>
  static __device__ __forceinline__ RowPacks of(const void *row, int vocab) {
    constexpr int VEC = RowPack<DT>::VEC;
    RowPacks r;
    r.phase = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / (16 / VEC));
    r.full0 = r.phase ? 1 : 0;
    r.full1 = (vocab + r.phase) / VEC;  // may be below full0: a row inside one pack
    return r;
  }
};

constexpr int kAhead = 4;  // packs in flight per thread

template <int DT, bool GRAD>
__global__ void __launch_bounds__(kMaxThreads, 2) ns_policy_kernel(const __grid_constant__ PolicyParams p) {
  using RP = RowPack<DT>;
  using E = typename RP::E;
  constexpr int VEC = RP::VEC;
  extern __shared__ uint4 keep[];  // [pack][thread]
  __shared__ MaxSum part[kMaxThreads / 32];
  __shared__ MaxSum mine;  // this CTA's share of the row, read by the cluster
  __shared__ MaxSum all;
  __shared__ RowResult res;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int rank = p.cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int first = rank * blockDim.x + threadIdx.x, stride = p.cluster * blockDim.x;
  const float k = p.inv_temp * kLog2e;
  const size_t dsize = static_cast<size_t>((p.rows - 1) * p.ld_d + p.vocab) * sizeof(E);
  const int64_t t = blockIdx.x / p.cluster;
  const E *x = static_cast<const E *>(p.logits) + t * p.ld;
  const RowPacks packs = RowPacks::of<DT>(x, p.vocab);
  const E *base = x - packs.phase;  // pack j is base + j * VEC
  // the two ragged ends, at most VEC - 1 elements each: thread 0's and thread 1's
  int edge0 = 0, edge1 = 0;
  if (first == 0) {
    edge1 = min(p.vocab, packs.full0 * VEC - packs.phase);
  } else if (first == 1) {
    edge0 = max(packs.full1 * VEC - packs.phase, min(p.vocab, packs.full0 * VEC - packs.phase));
    edge1 = p.vocab;
  }
  const int y = p.targets.get(t);
  bool live = y >= 0 && (!p.weight || p.weight[t] != 0.f);  // the same in every thread of the cluster
  MaxSum a{-INFINITY, 0.f};
  if (live) {
    RowInputs in;
    float target = 0.f;
    if (threadIdx.x == 0) {  // asked for now, needed after the reduction
      in = row_inputs(p, t);
      target = Elem<DT>::to_f(x[y]);
    }
    Scale f(-INFINITY, k);
    auto raise = [&](float top) {  // a new largest logit
      a.s = __fmul_rn(a.s, rebase(a.m, top, k));
      a.m = top;
      f = Scale(top, k);
    };
    for (int n = 0, j0 = packs.full0 + first; j0 < packs.full1; j0 += kAhead * stride, n += kAhead) {
      RP v[kAhead];
      const int left = packs.full1 - j0;  // pack u of these is there if u * stride < left
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (u * stride < left) v[u].v.load(base + static_cast<int64_t>(j0 + u * stride) * VEC);
      float top = -INFINITY;
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (u * stride < left) {
          if (GRAD && n < p.kept) keep[(n + u) * blockDim.x + threadIdx.x] = v[u].v.w[0];
          top = fmaxf(top, v[u].top());
        }
      if (top > a.m) raise(top);
      auto add = [&](auto plain) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
          if (u * stride < left) a.s = __fadd_rn(a.s, v[u].template sum<decltype(plain)::value>(f));
      };
      if (f.plain)
        add(std::true_type());
      else
        add(std::false_type());
    }
    for (int c = edge0; c < edge1; ++c) {
      const float v = Elem<DT>::to_f(x[c]);
      if (v > a.m) raise(v);
      a.s = __fadd_rn(a.s, f.power(v));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      a = merge(a, MaxSum{__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o)}, k);
    if (lane == 0) part[warp] = a;
    __syncthreads();
    if (warp == 0) {
      a = lane < warps ? part[lane] : MaxSum{-INFINITY, 0.f};
#pragma unroll
      for (int o = kMaxThreads / 64; o > 0; o >>= 1)
        a = merge(a, MaxSum{__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o)}, k);
      if (lane == 0) mine = a;
    }
    if (p.cluster > 1) {
      cluster_sync();
      if (warp == 0) {
        a = MaxSum{-INFINITY, 0.f};
        if (lane < p.cluster) {
          const uint32_t at = mapa_shared(smem_u32(&mine), lane);
          a.m = __uint_as_float(ld_shared_cluster_u32(at));
          a.s = __uint_as_float(ld_shared_cluster_u32(at + 4));
        }
#pragma unroll
        for (int o = kMaxCluster / 2; o > 0; o >>= 1)
          a = merge(a, MaxSum{__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o)}, k);
      }
    }
    if (threadIdx.x == 0) {
      all = a;
      RowResult r{0.f, 0.f, 0.f, 0.f};
      if (a.s != 0.f) {  // else every logit is -inf: no distribution
        const Scale f(a.m, k);
        // the powers are relative to m k as rounded
        r = policy_row(p, in, (static_cast<double>(target) - a.m) * p.inv_temp + f.left_out() * kLn2 - log_of(a.s));
      }
      res = r;
      if (rank == 0) write_result(p, t, r);
    }
    __syncthreads();
    a = all;
    if (a.s == 0.f) live = false;
  } else if (threadIdx.x == 0 && rank == 0) {
    write_result(p, t, RowResult{0.f, 0.f, 0.f, 0.f});
  }
  if constexpr (GRAD) {
    E *g = static_cast<E *>(p.dlogits) + t * p.ld_d;
    E *gbase = g - packs.phase;
    // in place, every CTA has read the target's logit before any overwrites it
    if (live && p.cluster > 1 && p.dlogits == p.logits) cluster_sync();
    const float slope = live ? res.slope : 0.f, scale = live ? -slope / a.s : 0.f;
    const Scale f(a.m, k);
    auto put = [&](int j, const RP &v) {
      if (p.packed) {
        v.v.store_stream(gbase + static_cast<int64_t>(j) * VEC, p.dlogits, dsize, p.status);
      } else {
        E *to = gbase + static_cast<int64_t>(j) * VEC;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (in_bounds(to + e, sizeof(E), p.dlogits, dsize, p.status)) to[e] = reinterpret_cast<const E *>(v.v.w)[e];
      }
    };
    auto put_one = [&](int c, float v) {
      if (in_bounds(g + c, sizeof(E), p.dlogits, dsize, p.status)) g[c] = Elem<DT>::from_f(v);
    };
    if (live) {
      const int target_pack = (y + packs.phase) / VEC;
      auto second_pass = [&](auto plain) {
        for (int n = 0, j0 = packs.full0 + first; j0 < packs.full1; j0 += kAhead * stride, n += kAhead) {
          RP v[kAhead];
          const int left = packs.full1 - j0;  // pack u of these is there if u * stride < left
          if (n < p.kept) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
              if (u * stride < left) v[u].v.w[0] = keep[(n + u) * blockDim.x + threadIdx.x];
          } else {
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
              if (u * stride < left) v[u].v.load_stream(base + static_cast<int64_t>(j0 + u * stride) * VEC);
          }
#pragma unroll
          for (int u = 0; u < kAhead; ++u) {
            if (u * stride >= left) break;
            const int j = j0 + u * stride;
            if (j != target_pack) {
              v[u].template to_gradient<decltype(plain)::value>(scale, f);
            } else {
              const int at = y + packs.phase - j * VEC;
#pragma unroll
              for (int e = 0; e < VEC; ++e) {
                const float d = scale * f.power(v[u].v.get(e));
                v[u].v.set(e, e == at ? d + slope : d);
              }
            }
            put(j, v[u]);
          }
        }
      };
      if (f.plain)
        second_pass(std::true_type());
      else
        second_pass(std::false_type());
      for (int c = edge0; c < edge1; ++c) {
        const float d = scale * f.power(Elem<DT>::to_f(x[c]));
        put_one(c, c == y ? d + slope : d);
      }
    } else {
      RP v;
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) v.set_pair(i, make_float2(0.f, 0.f));
      for (int j = packs.full0 + first; j < packs.full1; j += stride) put(j, v);
      for (int c = edge0; c < edge1; ++c) put_one(c, 0.f);
    }
  }
  if (p.cluster > 1) cluster_sync();  // no CTA leaves while another may read its share
  if (p.weight && p.done && rank == 0) {
    __shared__ bool last;
    if (threadIdx.x == 0) {
      __threadfence();  // the row's loss before its count
      last = atomicAdd(p.done, 1) == static_cast<int>(p.rows) - 1;
      __threadfence();
    }
    __syncthreads();
    if (last) {
      const float s = sum_losses(p, reinterpret_cast<float *>(part));
      if (threadIdx.x == 0) {
        if (in_bounds(p.loss, 4, p.loss, 4, p.status)) *p.loss = s;
        *p.done = 0;
      }
    }
  }
}

__global__ void __launch_bounds__(1024) ns_policy_sum_kernel(const __grid_constant__ PolicyParams p) {
  __shared__ float part[32];
  const float s = sum_losses(p, part);
  if (threadIdx.x == 0 && in_bounds(p.loss, 4, p.loss, 4, p.status)) *p.loss = s;
}

template <int DT, bool GRAD>
int run_rows(PolicyParams p, int sms, cudaStream_t s, bool *summed) {
  constexpr int elt = DT == kBF16 ? 2 : 4, VEC = 16 / elt;
  p.packed = ((reinterpret_cast<uintptr_t>(p.logits) ^ reinterpret_cast<uintptr_t>(p.dlogits)) % 16 == 0) &&
             (p.ld_d - p.ld) * elt % 16 == 0;
  // Threads: 16 packs each where the row has them, down to a warp; fewer, and
  // so more rows at a time on an SM, beat more threads a row (8192 x 32000
  // bf16: 205 us, 225 with 8 packs each, 260 with 4).
  int threads = kMaxThreads;
  while (threads > 32 && static_cast<int64_t>(threads) * 4 * kAhead * VEC > p.vocab) threads /= 2;
  // the last CTA sums the loss if that is at most 32 rows a thread
  if (p.rows > static_cast<int64_t>(threads) * 32) p.done = nullptr;
  *summed = p.done != nullptr;
  // few rows: a cluster of CTAs per row while SMs are idle and threads keep kAhead packs
  p.cluster = 1;
  while (p.cluster < kMaxCluster && p.rows * p.cluster * 2 <= sms &&
         static_cast<int64_t>(threads) * p.cluster * 2 * kAhead * VEC <= p.vocab)
    p.cluster *= 2;
  // shared memory for what is read twice: the row's packs, or an equal share of the SM
  int smem = 0;
  if (GRAD) {
    const int64_t step = static_cast<int64_t>(threads) * 16 * kAhead;  // bytes of kAhead packs of every thread
    const int64_t row = (static_cast<int64_t>(p.vocab) * elt / p.cluster + step - 1) / step * step;
    const int64_t share = kKeepBytes * threads / (2 * kMaxThreads) / step * step;
    smem = static_cast<int>(std::min(row, share));
    p.kept = static_cast<int>(smem / step) * kAhead;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(p.rows * p.cluster), 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster > 1 ? 1 : 0;
  static SmemOptIn opt_in;
  if (smem > 0 && opt_in.ensure(reinterpret_cast<const void *>(ns_policy_kernel<DT, GRAD>), smem)) return -1;
  if (cudaLaunchKernelEx(&cfg, ns_policy_kernel<DT, GRAD>, p) != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  count_launch();
  return 0;
}

template <int DT>
int run_policy(const PolicyParams &p, int sms, cudaStream_t s) {
  int rc = 0;
  bool summed = false;
  if (p.rows > 0) rc = p.dlogits ? run_rows<DT, true>(p, sms, s, &summed) : run_rows<DT, false>(p, sms, s, &summed);
  if (rc == 0 && p.weight && !summed) {
    ns_policy_sum_kernel<<<1, 1024, 0, s>>>(p);
    count_launch();
    rc = cudaGetLastError() == cudaSuccess ? 0 : -1;
  }
  return rc;
}

int policy_call(PolicyParams &p, int dtype, void *stream) {
  OpCall call(stream);
  if (call.rc) return call.rc;
  p.status = call.status;
  if (p.weight) {
    uint8_t *ws = nullptr;
    // a counter that every call leaves at 0, then the rows' losses
    if (const int rc = call.workspace(kSlotPolicy, 256 + static_cast<size_t>(p.rows) * 4, &ws, 256)) return rc;
    p.done = reinterpret_cast<int *>(ws);
    p.row_loss = reinterpret_cast<float *>(ws + 256);
  }
  return call.launch(kOpPolicy, [&] {
    return dtype == NS_BF16 ? run_policy<kBF16>(p, call.sms, call.s) : run_policy<kF32>(p, call.sms, call.s);
  });
}

}  // namespace
}  // namespace ns

using namespace ns;

extern "C" int ns_token_logprobs(const void *logits, int64_t ld_logits, int64_t rows, int64_t vocab,
                                 const void *targets, int id_type, float inv_temperature, float *logp, int dtype,
                                 void *stream) {
  if ((dtype != NS_F32 && dtype != NS_BF16) || (id_type != NS_I32 && id_type != NS_I64)) return NS_EINVAL;
  if (bad_shape(rows, vocab, ld_logits) || vocab > kMaxRowCols || !std::isfinite(inv_temperature) || inv_temperature <= 0) return NS_EINVAL;
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
  if (bad_shape(rows, vocab, ld_logits) || (dlogits && bad_shape(rows, vocab, ld_dlogits)) || vocab > kMaxRowCols)
    return NS_EINVAL;
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
