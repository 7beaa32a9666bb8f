// ns_block_norm.cu -- the norms after and before a block, fused with the
// block's gate and the residual scale (include/ns.h), and their backward pass.
//
//     u = y * rsqrt(mean y^2 + eps) * post,  r = a x + b g u,  z = r * rsqrt(mean r^2 + eps) * pre
//
// Bound by HBM: forward reads x and y and writes r and z, backward reads the
// two gradients, x and y and writes two gradients (r is formed again, in fp32,
// from the kept 1 / rms of y). A row is held in the registers of its threads
// between the sums over it. So that memory stays busy while threads wait for
// one another at those sums, rows come through a ring in shared memory that a
// warp keeps full by bulk copies (the ends of rows that are not 16-byte aligned
// element by element). With reads straight into registers, 16384 rows of 8192 bf16
// took 268 us forward and 603 back; now 172, 92 % of the copy rate, and 393 to 404 (232
// without pre, where X is not read). Forward has two rows of 256 threads in hand: one of
// 512 took 221.
// The weights' gradients are sums over rows: a CTA walks over rows and adds in
// fp32, each thread its own columns, and a second launch adds the CTAs' parts in
// order.
#include "ns_block_norm.cuh"

namespace ns {

namespace {
using namespace block_norm;

template <int XT, int YT, bool WIDE, int NP>
__global__ void __launch_bounds__(kMostThreads<WIDE, NP>) ns_block_norm_kernel(const __grid_constant__ NormParams p,
                                                            const __grid_constant__ RingShape ring) {
  using X = typename Elem<XT>::T;
  using Y = typename Elem<YT>::T;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ RowSums reds;
  reds.clear();
  RingBarriers *bar = start_ring(ring, smem);
  uint8_t *slots = smem + kRingHead;
  const Waiter w{&bar->abort, p.status, p.wait_limit_ns};
  const int consumers = ring.threads * ring.height;
  Filler<WIDE> filler;
  if (!WIDE && static_cast<int>(threadIdx.x) >= consumers) {
    filler.all(ring, bar, slots, p.rows, w);
    return;
  }
  const bool fills = WIDE && threadIdx.x < 32;
  if (fills) filler.first(ring, bar, slots, p.rows, w);
  const int group = threadIdx.x / ring.threads, thread = threadIdx.x - group * ring.threads;
  RowSum sum{reds.red[group], ring.threads, 1 + group, 0, thread};
  const size_t rsize = static_cast<size_t>((p.rows - 1) * p.ld_r + p.cols) * sizeof(X);
  const size_t zsize = static_cast<size_t>((p.rows - 1) * p.ld_z + p.cols) * sizeof(Y);
  const float inv_n = 1.f / static_cast<float>(p.cols);
  int c[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i)
    c[i] = WIDE ? (i * ring.threads + thread) * 8 : (i * ring.threads + (thread & ~31)) * 8 + (thread & 31);
  const ColumnWeights<WIDE, NP> held{reinterpret_cast<float4 *>(slots + ring.slots * ring.slot_bytes) + thread, ring.threads};
  if (p.hold && group == 0) held.keep(p, c);
  asm volatile("bar.sync 15, %0;" ::"r"(consumers) : "memory");
  RowReader reader;
  bool ok = true;
  const uint32_t rows = static_cast<uint32_t>(p.rows), step = gridDim.x * ring.height;
  uint32_t t = blockIdx.x * ring.height + group;
  const StreamRow<XT, WIDE, 0> xs(ring, group);
  const StreamRow<YT, WIDE, 1> ys(ring, group);
  X *to = static_cast<X *>(p.r) + t * p.ld_r;
  Y *zt = static_cast<Y *>(p.z) + t * p.ld_z;
  int64_t ahead = blockIdx.x + static_cast<int64_t>(ring.slots) * gridDim.x;
  for (uint32_t t0 = blockIdx.x * ring.height; t0 < rows; t0 += step, t += step, to += step * p.ld_r, zt += step * p.ld_z,
                ahead += gridDim.x) {
    const uint8_t *at = reader.wait(ring, bar, slots, w, ok);
    if (t >= rows) {  // (never the first group)
      reader.release(ring, bar);
      continue;
    }
    Eight2 r[NP], y[NP];
    float2 s2 = both(0.f);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      xs.load(ring, at, t, c[i], p.cols, r[i]);
      if (p.y) {
        ys.load(ring, at, t, c[i], p.cols, y[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) s2 = __ffma2_rn(y[i].v[j], y[i].v[j], s2);
      }
    }
    reader.release(ring, bar);
    if (p.y) {
      float k = p.b * (p.gate_form == kGateRows ? one_of(p.gate, t * p.ld_gate, p.gate_type) : 1.f);
      if (p.post) {
        const float ry = rsqrtf(sum(s2.x + s2.y) * inv_n + p.eps);
        if (thread == 0 && ok) put(p.post_rstd + t, ry, p.post_rstd, static_cast<size_t>(p.rows) * 4, p.status);
        k *= ry;
      }
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        Eight2 f;
        weights_of<WIDE, NP>(p, held, 0, i, c[i], f);
        if (p.gate_form == kGateFull) {
          Eight2 g;
          load_any<WIDE>(at_row(p.gate, t, p.ld_gate, p.gate_type), p.gate_type, c[i], p.cols, g);
#pragma unroll
          for (int j = 0; j < 4; ++j) f.v[j] = __fmul2_rn(f.v[j], g.v[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          r[i].v[j] = __ffma2_rn(__fmul2_rn(y[i].v[j], both(k)), f.v[j], __fmul2_rn(r[i].v[j], both(p.a)));
      }
    } else {
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) r[i].v[j] = __fmul2_rn(r[i].v[j], both(p.a));
    }
    if (fills) filler.fill(ring, bar, slots, p.rows, ahead, w);
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (ok) store8<XT, WIDE>(to, c[i], p.cols, r[i], p.r, rsize, p.status);
    if (p.pre) {
      s2 = both(0.f);
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s2 = __ffma2_rn(r[i].v[j], r[i].v[j], s2);
      const float rr = rsqrtf(sum(s2.x + s2.y) * inv_n + p.eps);
      if (thread == 0 && ok) put(p.pre_rstd + t, rr, p.pre_rstd, static_cast<size_t>(p.rows) * 4, p.status);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        Eight2 f;
        weights_of<WIDE, NP>(p, held, 1, i, c[i], f);
#pragma unroll
        for (int j = 0; j < 4; ++j) f.v[j] = __fmul2_rn(f.v[j], __fmul2_rn(r[i].v[j], both(rr)));
        if (ok) store8<YT, WIDE>(zt, c[i], p.cols, f, p.z, zsize, p.status);
      }
    }
  }
  if (fills) filler.end(ring, bar, w);
}

}  // namespace
}  // namespace ns

using namespace ns;
using namespace ns::block_norm;

extern "C" int64_t ns_block_norm_workspace(int64_t rows, int64_t cols) {
  if (rows < 0 || cols < 0 || cols > kMaxCols) return -1;
  return std::max<int64_t>(1, std::min<int64_t>(rows, kMaxParts)) * 2 * cols * 4;
}

extern "C" int ns_block_norm(const void *x, int64_t ld_x, const void *y, int64_t ld_y, const void *gate, int gate_form,
                             int64_t ld_gate, const void *post, const void *pre, int64_t rows, int64_t cols, float a,
                             float b, float eps, void *residual, int64_t ld_r, void *normed, int64_t ld_z,
                             float *post_rstd, float *pre_rstd, int dtype, int block_dtype, int weight_dtype,
                             int gate_dtype, void *stream) {
  NormParams p{};
  if (int rc = check(p, x, ld_x, y, ld_y, gate, gate_form, ld_gate, post, pre, rows, cols, a, b, dtype, block_dtype,
                     weight_dtype, gate_dtype))
    return rc;
  if (!(eps >= 0.f) || !std::isfinite(eps) || bad_shape(rows, cols, ld_r) || (pre && bad_shape(rows, cols, ld_z))) return NS_EINVAL;
  if (rows == 0 || cols == 0) return NS_OK;
  if (!x || !residual || (pre && (!normed || !pre_rstd)) || (post && !post_rstd)) return NS_EINVAL;
  const int xe = size_of(dtype), ye = size_of(block_dtype), we = size_of(weight_dtype);
  if (misaligned(residual, xe) || misaligned(normed, ye) || misaligned(post_rstd, 4) || misaligned(pre_rstd, 4)) return NS_EALIGN;
  const Range in[] = {Range(x, rows, cols, ld_x, xe), Range(y, rows, cols, ld_y, ye),
                      gate_range(gate, gate_form, rows, cols, ld_gate, gate_dtype), Range(post, 1, cols, cols, we),
                      Range(pre, 1, cols, cols, we)};
  const Range out[] = {Range(residual, rows, cols, ld_r, xe), Range(pre ? normed : nullptr, rows, cols, ld_z, ye),
                       Range(post ? post_rstd : nullptr, 1, rows, rows, 4), Range(pre ? pre_rstd : nullptr, 1, rows, rows, 4)};
  // a thread reads its part of a row before it writes there: residual may be x, normed may be y
  const bool over_x = residual == x && ld_r == ld_x, over_y = normed == y && ld_z == ld_y;
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 5; ++i)
      if (!(o == 0 && i == 0 && over_x) && !(o == 1 && i == 1 && over_y) && out[o].overlaps(in[i])) return NS_EINVAL;
    for (int k = 0; k < o; ++k)
      if (out[o].overlaps(out[k])) return NS_EINVAL;
  }
  OpCall call(stream);
  if (call.rc) return call.rc;
  p.r = residual;
  p.z = normed;
  p.ld_r = ld_r;
  p.ld_z = ld_z;
  p.post_rstd = post_rstd;
  p.pre_rstd = pre_rstd;
  p.eps = eps;
  p.status = call.status;
  p.wait_limit_ns = kWaitLimitNs;
  const bool wide = packs_fit(p, dtype, block_dtype) && rows_aligned(residual, ld_r, xe, 8) && (!pre || rows_aligned(normed, ld_z, ye, 8));
  const Shape sh(p, false, wide, dtype, block_dtype, call.sms);
  p.hold = sh.hold;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(sh.batches(rows), static_cast<int64_t>(call.sms) * sh.per_sm));
  return call.launch(kOpBlockNorm, [&] {
    const int rc = by_types(dtype, block_dtype, wide, [&](auto xt, auto yt, auto w) {
      return by_packs(sh.packs, [&](auto np) {
        auto *kernel = ns_block_norm_kernel<decltype(xt)::value, decltype(yt)::value, decltype(w)::value, decltype(np)::value>;
        static SmemOptIn opt_in;
        if (opt_in.ensure(reinterpret_cast<const void *>(kernel), sh.smem)) return -1;
        kernel<<<grid, sh.block(wide), sh.smem, call.s>>>(p, sh.ring);
        return 0;
      });
    });
    if (rc) return rc;
    count_launch();
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
  });
}
