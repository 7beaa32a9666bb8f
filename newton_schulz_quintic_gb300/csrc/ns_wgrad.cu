// ns_wgrad.cu -- weight gradients from an input held in 8 bits
// (include/ns.h): G[e] (+)= dY[e]^T X[e] over the rows of each group.
//
// CUDA-core form: a 64 x 64 tile of one group's G per CTA, 16 rows of both
// operands at a time in shared memory as fp32, 4 x 4 sums per thread.
#include <algorithm>

#include "../../include/ns.h"
#include "ns_rows.cuh"

namespace ns {

namespace {

struct WgradParams {
  const void *dy;
  const int8_t *q;
  const uint8_t *s;
  const int32_t *offsets;  // nullptr: one group of all rows
  void *grad;
  int64_t ld_dy;
  int rows, n_out, n_in, pitch, scale_pitch, groups;
  int accumulate;
  int *status;
};

constexpr int kTile = 64;
constexpr int kDepth = 16;

template <int DT, int GT>
__global__ void __launch_bounds__(256) ns_wgrad_simt_kernel(const __grid_constant__ WgradParams p) {
  using E = typename Elem<DT>::T;
  using G = typename Elem<GT>::T;
  __shared__ float sa[kDepth][kTile], sb[kDepth][kTile];
  const int tn = (p.n_out + kTile - 1) / kTile, tk = (p.n_in + kTile - 1) / kTile;
  const int per = tn * tk;
  const int e = blockIdx.x / per, tile = blockIdx.x - e * per;
  const int n0 = tile / tk * kTile, k0 = tile % tk * kTile;
  int lo = 0, hi = p.rows;
  if (p.offsets) {
    lo = min(max(p.offsets[e], 0), p.rows);
    hi = min(max(p.offsets[e + 1], lo), p.rows);
  }
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int t0 = lo; t0 < hi; t0 += kDepth) {
    __syncthreads();
    for (int i = threadIdx.x; i < kDepth * kTile; i += 256) {
      const int r = i / kTile, c = i % kTile, t = t0 + r;
      float a = 0.f, b = 0.f;
      if (t < hi && n0 + c < p.n_out) a = Elem<DT>::to_f(static_cast<const E *>(p.dy)[t * p.ld_dy + n0 + c]);
      if (t < hi && k0 + c < p.n_in) {
        const int ex = p.s[static_cast<int64_t>(t) * p.scale_pitch + (k0 + c) / 32];
        const float unit = ex == 255 ? __int_as_float(0x7fc00000) : __int_as_float((max(ex, 7) - 6) << 23);
        b = static_cast<float>(p.q[static_cast<int64_t>(t) * p.pitch + k0 + c]) * unit;
      }
      sa[r][c] = a;
      sb[r][c] = b;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kDepth; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[r][ty * 4 + i], sb[r][tx * 4 + j], acc[i][j]);
  }
  const size_t size = static_cast<size_t>(p.groups) * p.n_out * p.n_in * sizeof(G);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + ty * 4 + i, k = k0 + tx * 4 + j;
      if (n >= p.n_out || k >= p.n_in) continue;
      G *g = static_cast<G *>(p.grad) + (static_cast<int64_t>(e) * p.n_out + n) * p.n_in + k;
      if (in_bounds(g, sizeof(G), p.grad, size, p.status))
        *g = Elem<GT>::from_f(p.accumulate ? Elem<GT>::to_f(*g) + acc[i][j] : acc[i][j]);
    }
}

template <int DT, int GT>
int run_simt(const WgradParams &p, cudaStream_t s) {
  const int64_t tiles = static_cast<int64_t>((p.n_out + kTile - 1) / kTile) * ((p.n_in + kTile - 1) / kTile) * p.groups;
  if (tiles > INT32_MAX) return -1;
  ns_wgrad_simt_kernel<DT, GT><<<static_cast<int>(tiles), 256, 0, s>>>(p);
  count_launch();
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

}  // namespace
}  // namespace ns

using namespace ns;

extern "C" int ns_ckpt_wgrad(const void *dy, int64_t ld_dy, int64_t rows, int64_t n_out, const void *q,
                             const void *scales, int64_t n_in, const int32_t *offsets, int groups, void *grad,
                             int dtype, int grad_dtype, int accumulate, void *stream) {
  if ((dtype != NS_F32 && dtype != NS_BF16) || (grad_dtype != NS_F32 && grad_dtype != NS_BF16) ||
      (accumulate != 0 && accumulate != 1) || groups < 0)
    return NS_EINVAL;
  if (bad_shape(rows, n_out, ld_dy) || bad_shape(n_out, n_in, n_in) || n_out > (1 << 30) || n_in > (1 << 30) ||
      rows > (1 << 30))
    return NS_EINVAL;
  if (!offsets && groups != 1) return NS_EINVAL;
  if (groups > 0 && n_out * n_in > (int64_t(1) << 42) / groups) return NS_EINVAL;
  if (groups == 0 || n_out == 0 || n_in == 0 || (rows == 0 && accumulate)) return NS_OK;
  if (!grad || (rows > 0 && (!dy || !q || !scales))) return NS_EINVAL;
  const int elt = dtype == NS_BF16 ? 2 : 4, gelt = grad_dtype == NS_BF16 ? 2 : 4;
  if (misaligned(dy, elt) || misaligned(grad, gelt) || misaligned(q, 16) || misaligned(scales, 16) ||
      misaligned(offsets, 4))
    return NS_EALIGN;
  WgradParams p{};
  p.pitch = static_cast<int>(ns_ckpt_pitch(n_in));
  p.scale_pitch = static_cast<int>(ns_ckpt_scale_pitch(n_in));
  const Range rg(grad, static_cast<int64_t>(groups) * n_out, n_in, n_in, gelt);
  if (rg.overlaps(Range(dy, rows, n_out, ld_dy, elt)) || rg.overlaps(Range(q, rows, p.pitch, p.pitch, 1)) ||
      rg.overlaps(Range(scales, rows, p.scale_pitch, p.scale_pitch, 1)) ||
      rg.overlaps(Range(offsets, 1, groups + 1, groups + 1, 4)))
    return NS_EINVAL;
  OpCall call(stream);
  if (call.rc) return call.rc;
  p.dy = dy;
  p.q = static_cast<const int8_t *>(q);
  p.s = static_cast<const uint8_t *>(scales);
  p.offsets = offsets;
  p.grad = grad;
  p.ld_dy = ld_dy;
  p.rows = static_cast<int>(rows);
  p.n_out = static_cast<int>(n_out);
  p.n_in = static_cast<int>(n_in);
  p.groups = groups;
  p.accumulate = accumulate;
  p.status = call.status;
  return call.launch(kOpWgrad, [&] {
    if (dtype == NS_BF16) return grad_dtype == NS_BF16 ? run_simt<kBF16, kBF16>(p, call.s) : run_simt<kBF16, kF32>(p, call.s);
    return grad_dtype == NS_BF16 ? run_simt<kF32, kBF16>(p, call.s) : run_simt<kF32, kF32>(p, call.s);
  });
}
