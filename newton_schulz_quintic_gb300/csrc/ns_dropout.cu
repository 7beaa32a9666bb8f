// ns_dropout.cu -- dropout from a counter-based generator (include/ns.h).
//
// The mask is a function of (seed, counter), so nothing of it is stored: the
// backward pass is the same call on the gradient. A lane takes 8 consecutive
// columns, which share one counter, and draws 16 bits for each with one
// Philox4x32-10. The 16 bits are the upper half of a 32-bit number; its lower
// half, a second Philox, is drawn only when an upper half equals the limit's,
// once in 65536 elements, so p holds to 2^-32 at half of the arithmetic. That
// arithmetic is what bounds it (issue slots 70 % busy): 16384 x 8192 bf16 in 118 us
// (4.6 TB/s), added to a residual in 138 us (5.9 TB/s). Product and sum take one
// rounding: 0.08 % of the bf16 results at prob 0.1 are another neighbour than with the
// product rounded first, at the same distance from 64 bits (46.3559 against 46.3559 in
// the norm over 2^27 elements).
#include <cmath>

#include "../../include/ns.h"
#include "ns_rows.cuh"

namespace ns {

namespace {

constexpr int kThreads = 256;

struct DropoutParams {
  const void *x, *residual;
  void *out;
  int64_t ld_x, ld_r, ld_o, rows;
  int cols;
  uint32_t limit_high, limit_low;  // dropped: high * 65536 + low below this (limit_high 65536: all)
  float scale;
  uint64_t seed, offset;
  const uint64_t *state;           // nullptr, or {seed, offset} to add
  int lanes_log2;
  int *status;
};

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as easy as 1, 2, 3", 2011).
__device__ __forceinline__ uint4 philox(uint64_t n, uint32_t third, uint64_t key) {
  uint32_t a = static_cast<uint32_t>(n), b = static_cast<uint32_t>(n >> 32), c = third, d = 0;
  uint32_t k0 = static_cast<uint32_t>(key), k1 = static_cast<uint32_t>(key >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p = static_cast<uint64_t>(a) * 0xD2511F53u, q = static_cast<uint64_t>(c) * 0xCD9E8D57u;
    a = static_cast<uint32_t>(q >> 32) ^ b ^ k0;
    b = static_cast<uint32_t>(q);
    c = static_cast<uint32_t>(p >> 32) ^ d ^ k1;
    d = static_cast<uint32_t>(p);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(a, b, c, d);
}
__device__ __forceinline__ uint32_t half_of(const uint4 &w, int e) {
  const uint32_t v = e < 2 ? w.x : e < 4 ? w.y : e < 6 ? w.z : w.w;
  return e & 1 ? v >> 16 : v & 0xffffu;
}

template <int XT, int RT, bool ADD, bool WIDE>
__global__ void __launch_bounds__(kThreads) ns_dropout_kernel(const __grid_constant__ DropoutParams p) {
  using X = typename Elem<XT>::T;
  using R = typename Elem<RT>::T;
  __shared__ uint4 stages[WIDE ? 1 : kThreads / 32][WIDE ? 1 : Eight<RT, WIDE>::kStage];
  uint4 *stage = stages[WIDE ? 0 : threadIdx.x / 32];
  const int c = ((blockIdx.x << p.lanes_log2) + (threadIdx.x & ((1 << p.lanes_log2) - 1))) * 8;
  const int height = kThreads >> p.lanes_log2;
  const int64_t step = static_cast<int64_t>(gridDim.y) * height;
  const uint64_t seed = p.seed + (p.state ? __ldg(p.state) : 0), offset = p.offset + (p.state ? __ldg(p.state + 1) : 0);
  const uint64_t packs = (static_cast<uint64_t>(p.cols) + 7) / 8;
  const size_t size = static_cast<size_t>((p.rows - 1) * p.ld_o + p.cols) * sizeof(R);
  for (int64_t t0 = static_cast<int64_t>(blockIdx.y) * height; t0 < p.rows; t0 += step) {
    const int64_t t = t0 + (threadIdx.x >> p.lanes_log2);
    const bool row = t < p.rows;
    Eight<XT, WIDE> x;
    Eight<RT, WIDE> r;
    x.load(static_cast<const X *>(p.x) + t * p.ld_x, c, p.cols, row);
    if constexpr (ADD) r.load(static_cast<const R *>(p.residual) + t * p.ld_r, c, p.cols, row);
    const uint64_t n = offset + static_cast<uint64_t>(t) * packs + static_cast<uint64_t>(c / 8);
    const uint4 high = philox(n, 0, seed);
    uint32_t keep = 0;
    bool close = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t h = half_of(high, e);
      keep |= (h >= p.limit_high ? 1u : 0u) << e;
      close = close || h == p.limit_high;
    }
    if (close && p.limit_low != 0) {
      const uint4 low = philox(n, 1, seed);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (half_of(high, e) == p.limit_high && half_of(low, e) < p.limit_low) keep &= ~(1u << e);
    }
    x.settle(stage);
    if constexpr (ADD) r.settle(stage);
    Eight<RT, WIDE> o;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool k = (keep >> e) & 1u;  // a dropped value has no part in the result, whatever it is
      if constexpr (ADD)
        o.set(e, k ? fmaf(x.get(e), p.scale, r.get(e)) : r.get(e));
      else
        o.set(e, k ? x.get(e) * p.scale : 0.f);
    }
    o.store(static_cast<R *>(p.out) + t * p.ld_o, c, p.cols, row, stage, p.out, size, p.status);
  }
}

template <int XT, int RT, bool ADD>
int run_dropout(DropoutParams &p, bool wide, int sms, cudaStream_t s) {
  const EightGrid g(p.rows, p.cols, kThreads, wide, 2, sms, wide ? 64 : 32);
  p.lanes_log2 = g.lanes_log2;
  if (wide)
    ns_dropout_kernel<XT, RT, ADD, true><<<g.grid, kThreads, 0, s>>>(p);
  else
    ns_dropout_kernel<XT, RT, ADD, false><<<g.grid, kThreads, 0, s>>>(p);
  count_launch();
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace
}  // namespace ns

using namespace ns;

extern "C" int ns_dropout(const void *x, int64_t ld_x, const void *residual, int64_t ld_residual, int64_t rows,
                          int64_t cols, double prob, uint64_t seed, uint64_t offset, const void *state, void *out,
                          int64_t ld_out, int dtype, int out_dtype, void *stream) {
  if ((dtype != NS_F32 && dtype != NS_BF16) || (out_dtype != NS_F32 && out_dtype != NS_BF16)) return NS_EINVAL;
  // a wider sum is for a residual stream in fp32; nothing narrows
  if (out_dtype != dtype && !(residual && out_dtype == NS_F32)) return NS_EINVAL;
  if (!(prob >= 0. && prob <= 1.)) return NS_EINVAL;
  if (bad_shape(rows, cols, ld_x) || bad_shape(rows, cols, ld_out) || (residual && bad_shape(rows, cols, ld_residual)) ||
      cols > kMaxRowCols)
    return NS_EINVAL;
  if (rows == 0 || cols == 0) return NS_OK;
  if (!x || !out) return NS_EINVAL;
  const int elt = dtype == NS_BF16 ? 2 : 4, oelt = out_dtype == NS_BF16 ? 2 : 4;
  if (misaligned(x, elt) || misaligned(out, oelt) || misaligned(residual, oelt) || misaligned(state, 8)) return NS_EALIGN;
  const Range ro(out, rows, cols, ld_out, oelt);
  if (!(out == x && ld_out == ld_x && oelt == elt) && ro.overlaps(Range(x, rows, cols, ld_x, elt))) return NS_EINVAL;
  if (residual && !(out == residual && ld_out == ld_residual) && ro.overlaps(Range(residual, rows, cols, ld_residual, oelt)))
    return NS_EINVAL;
  if (ro.overlaps(Range(state, 1, 2, 2, 8))) return NS_EINVAL;
  OpCall call(stream);
  if (call.rc) return call.rc;
  DropoutParams p{};
  p.x = x;
  p.residual = residual;
  p.out = out;
  p.ld_x = ld_x;
  p.ld_r = ld_residual;
  p.ld_o = ld_out;
  p.rows = rows;
  p.cols = static_cast<int>(cols);
  const uint64_t limit = static_cast<uint64_t>(std::nearbyint(prob * 4294967296.));
  p.limit_high = static_cast<uint32_t>(limit >> 16);
  p.limit_low = static_cast<uint32_t>(limit & 0xffffu);
  p.scale = limit == uint64_t(1) << 32 ? 0.f : static_cast<float>(4294967296. / static_cast<double>((uint64_t(1) << 32) - limit));
  p.seed = seed;
  p.offset = offset;
  p.state = static_cast<const uint64_t *>(state);
  p.status = call.status;
  const bool wide = cols % 8 == 0 && rows_aligned(x, ld_x, elt, 8) && rows_aligned(out, ld_out, oelt, 8) &&
                    (!residual || rows_aligned(residual, ld_residual, oelt, 8));
  return call.launch(kOpDropout, [&] {
    if (!residual)
      return dtype == NS_BF16 ? run_dropout<kBF16, kBF16, false>(p, wide, call.sms, call.s)
                              : run_dropout<kF32, kF32, false>(p, wide, call.sms, call.s);
    if (out_dtype == NS_BF16) return run_dropout<kBF16, kBF16, true>(p, wide, call.sms, call.s);
    return dtype == NS_BF16 ? run_dropout<kBF16, kF32, true>(p, wide, call.sms, call.s)
                            : run_dropout<kF32, kF32, true>(p, wide, call.sms, call.s);
  });
}
