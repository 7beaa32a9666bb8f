// ns_block_norm_back.cu -- backward pass of the block norms (include/ns.h; the forward pass and the layout of the work
// are described in ns_block_norm.cu).
#include "ns_block_norm.cuh"

namespace ns {

namespace {
using namespace block_norm;

// The columns' sums are in registers, or for rows of more than 2 packs a thread in shared memory behind the ring and the
// weights ([2][NP][8][threads of a row] floats for each row of the CTA, every thread its own).
template <int NP> constexpr bool kInRegs = NP <= 2;
template <int XT, int YT, bool WIDE, int NP>
__global__ void __launch_bounds__(kMostThreads<WIDE, NP>) ns_block_norm_backward_kernel(const __grid_constant__ NormParams p,
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
  const int step = ring.threads;
  uint8_t *behind = slots + ring.slots * ring.slot_bytes;  // the weights, then the sums
  const ColumnWeights<WIDE, NP> held{reinterpret_cast<float4 *>(behind) + thread, ring.threads};
  float *acc = reinterpret_cast<float *>(kInRegs<NP> ? slots : behind + (p.hold ? 2 * NP * 8 * 4 * step : 0)) +
               group * (2 * NP * 8 * step) + thread;
  int c[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i)
    c[i] = WIDE ? (i * ring.threads + thread) * 8 : (i * ring.threads + (thread & ~31)) * 8 + (thread & 31);
  RowSum sum{reds.red[group], ring.threads, 1 + group, 0, thread};
  const size_t xsize = static_cast<size_t>((p.rows - 1) * p.ld_dx + p.cols) * sizeof(X);
  const size_t ysize = static_cast<size_t>((p.rows - 1) * p.ld_dy + p.cols) * sizeof(Y);
  const float inv_n = 1.f / static_cast<float>(p.cols);
  float2 sums[2][kInRegs<NP> ? NP : 1][4];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (kInRegs<NP>)
          sums[k][i][j] = both(0.f);
        else
          acc[((k * NP + i) * 8 + 2 * j) * step] = acc[((k * NP + i) * 8 + 2 * j + 1) * step] = 0.f;
      }
  auto add = [&](int k, int i, int j, float2 a, float2 b) {  // a * b
    if constexpr (kInRegs<NP>) {
      sums[k][i][j] = __ffma2_rn(a, b, sums[k][i][j]);
    } else {
      float *own = acc + ((k * NP + i) * 8 + 2 * j) * step;
      own[0] = fmaf(a.x, b.x, own[0]);
      own[step] = fmaf(a.y, b.y, own[step]);
    }
  };
  if (p.hold && group == 0) held.keep(p, c);
  asm volatile("bar.sync 15, %0;" ::"r"(consumers) : "memory");
  RowReader reader;
  bool ok = true;
  const uint32_t rows = static_cast<uint32_t>(p.rows), stride = gridDim.x * ring.height;
  uint32_t t = blockIdx.x * ring.height + group;
  const StreamRow<XT, WIDE, 0> xs(ring, group);
  const StreamRow<YT, WIDE, 1> ys(ring, group);
  const StreamRow<YT, WIDE, 2> zs(ring, group);
  const StreamRow<XT, WIDE, 3> drs(ring, group);
  X *to = static_cast<X *>(p.dx) + t * p.ld_dx;
  Y *yt = static_cast<Y *>(p.dy) + t * p.ld_dy;
  int64_t ahead = blockIdx.x + static_cast<int64_t>(ring.slots) * gridDim.x;
  const bool post = p.y && p.post;
  float ry_next = t < rows && post ? p.post_rstd[t] : 1.f, rr_next = t < rows && p.pre ? p.pre_rstd[t] : 0.f;
  for (uint32_t t0 = blockIdx.x * ring.height; t0 < rows; t0 += stride, t += stride, to += stride * p.ld_dx, yt += stride * p.ld_dy,
                ahead += gridDim.x) {
    const bool here = t < rows;
    const float ry = ry_next, rr = rr_next;
    {  // the next row's, and this row's dR where it is read past the ring
      const uint32_t next = t + stride;
      ry_next = next < rows && post ? p.post_rstd[next] : 1.f;
      rr_next = next < rows && p.pre ? p.pre_rstd[next] : 0.f;
      if (p.dr && here && !ring.row_bytes[3])
#pragma unroll
        for (int i = 0; i < NP; ++i)
          if (c[i] < p.cols) asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<uint64_t>(ring.src[3] + t * ring.ld_bytes[3] + c[i] * sizeof(X))));
    }
    const float grow = here && p.gate_form == kGateRows ? one_of(p.gate, t * p.ld_gate, p.gate_type) : 1.f;
    const uint8_t *at = reader.wait(ring, bar, slots, w, ok);
    if (!here) {  // (never the first group)
      reader.release(ring, bar);
      continue;
    }
    Eight2 y[NP], d[NP];  // Y / rms; R / rms, then the gradient of r
    if (p.pre) {
      float2 s2 = both(0.f);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        xs.load(ring, at, t, c[i], p.cols, d[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) d[i].v[j] = __fmul2_rn(d[i].v[j], both(p.a));
        Eight2 f;
        if (p.y) {
          ys.load(ring, at, t, c[i], p.cols, y[i]);
          weights_of<WIDE, NP>(p, held, 0, i, c[i], f);
          if (p.gate_form == kGateFull) {
            Eight2 full;
            load_any<WIDE>(at_row(p.gate, t, p.ld_gate, p.gate_type), p.gate_type, c[i], p.cols, full);
#pragma unroll
            for (int j = 0; j < 4; ++j) f.v[j] = __fmul2_rn(f.v[j], full.v[j]);
          }
          const float k = p.b * grow;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            y[i].v[j] = __fmul2_rn(y[i].v[j], both(ry));
            d[i].v[j] = __ffma2_rn(__fmul2_rn(y[i].v[j], both(k)), f.v[j], d[i].v[j]);
          }
        }
        Eight2 z;
        zs.load(ring, at, t, c[i], p.cols, z);
        weights_of<WIDE, NP>(p, held, 1, i, c[i], f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          d[i].v[j] = __fmul2_rn(d[i].v[j], both(rr));
          add(0, i, j, z.v[j], d[i].v[j]);
          s2 = __ffma2_rn(__fmul2_rn(z.v[j], f.v[j]), d[i].v[j], s2);
        }
      }
      const float m = -sum(s2.x + s2.y) * inv_n;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        // dZ again from the ring: registers for it would be spilled
        Eight2 z, f, o;
        zs.load(ring, at, t, c[i], p.cols, z);
        weights_of<WIDE, NP>(p, held, 1, i, c[i], f);
        if (p.dr)
          drs.load(ring, at, t, c[i], p.cols, o);
        else
          o.fill(0.f);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          d[i].v[j] = __ffma2_rn(both(rr), __ffma2_rn(d[i].v[j], both(m), __fmul2_rn(z.v[j], f.v[j])), o.v[j]);
      }
      reader.release(ring, bar);
    } else {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        drs.load(ring, at, t, c[i], p.cols, d[i]);
        if (p.y) {
          ys.load(ring, at, t, c[i], p.cols, y[i]);
#pragma unroll
          for (int j = 0; j < 4; ++j) y[i].v[j] = __fmul2_rn(y[i].v[j], both(ry));
        }
      }
      reader.release(ring, bar);
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      Eight2 o;
#pragma unroll
      for (int j = 0; j < 4; ++j) o.v[j] = __fmul2_rn(d[i].v[j], both(p.a));
      if (ok) store8<XT, WIDE>(to, c[i], p.cols, o, p.dx, xsize, p.status);
    }
    if (!p.y) {
      if (fills) filler.fill(ring, bar, slots, p.rows, ahead, w);
      continue;
    }
    // through the gate: d * yh enters the sums (with a row's or a full gate's factor; the columns' comes at their end);
    // the gradient of y's norm is b gate post d
    float2 s2 = both(0.f);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      Eight2 f;
      weights_of<WIDE, NP>(p, held, 0, i, c[i], f);
#pragma unroll
      for (int j = 0; j < 4; ++j) f.v[j] = __fmul2_rn(f.v[j], both(p.b));
      if (p.gate_form == kGateFull) {
        Eight2 g, og;
        load_any<WIDE>(at_row(p.gate, t, p.ld_gate, p.gate_type), p.gate_type, c[i], p.cols, g);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          og.v[j] = __fmul2_rn(__fmul2_rn(f.v[j], d[i].v[j]), y[i].v[j]);
          d[i].v[j] = __fmul2_rn(d[i].v[j], g.v[j]);
        }
        const size_t gsize = static_cast<size_t>((p.rows - 1) * p.ld_dgate + p.cols) * (p.gate_type == kBF16 ? 2 : 4);
        void *gt = const_cast<void *>(at_row(p.dgate, t, p.ld_dgate, p.gate_type));
        if (ok && p.gate_type == kBF16)
          store8<kBF16, WIDE>(gt, c[i], p.cols, og, p.dgate, gsize, p.status);
        else if (ok)
          store8<kF32, WIDE>(gt, c[i], p.cols, og, p.dgate, gsize, p.status);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 dyh = __fmul2_rn(d[i].v[j], y[i].v[j]);
        add(1, i, j, both(grow), dyh);
        s2 = __ffma2_rn(f.v[j], dyh, s2);
        d[i].v[j] = __fmul2_rn(d[i].v[j], __fmul2_rn(f.v[j], both(grow)));
      }
    }
    if (fills) filler.fill(ring, bar, slots, p.rows, ahead, w);
    const float s = p.post || p.gate_form == kGateRows ? sum(s2.x + s2.y) : 0.f;
    if (p.gate_form == kGateRows && thread == 0 && ok) {
      const size_t places = static_cast<size_t>((p.rows - 1) * p.ld_dgate + 1);
      if (p.gate_type == kBF16)
        put(static_cast<__nv_bfloat16 *>(p.dgate) + t * p.ld_dgate, __float2bfloat16_rn(s), p.dgate, places * 2, p.status);
      else
        put(static_cast<float *>(p.dgate) + t * p.ld_dgate, s, p.dgate, places * 4, p.status);
    }
    const float m = p.post ? -s * grow * inv_n : 0.f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      Eight2 o;
#pragma unroll
      for (int j = 0; j < 4; ++j) o.v[j] = __fmul2_rn(__ffma2_rn(y[i].v[j], both(m), d[i].v[j]), both(ry));
      if (ok) store8<YT, WIDE>(yt, c[i], p.cols, o, p.dy, ysize, p.status);
    }
  }
  if (fills) filler.end(ring, bar, w);
  if constexpr (kInRegs<NP>) {
    // the ring is done with once every thread is here: it takes the sums
    asm volatile("bar.sync 15, %0;" ::"r"(consumers) : "memory");
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[((k * NP + i) * 8 + 2 * j) * step] = sums[k][i][j].x;
          acc[((k * NP + i) * 8 + 2 * j + 1) * step] = sums[k][i][j].y;
        }
  }
  asm volatile("bar.sync 15, %0;" ::"r"(consumers) : "memory");
  // the CTA's rows added in order, to its part
  if (group == 0) {
    float *part = p.parts + static_cast<int64_t>(blockIdx.x) * 2 * p.cols;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int at = (k * NP + i) * 8 + e, col = col_of<WIDE>(c[i], e);
          float v = acc[at * step];
          for (int j = 1; j < ring.height; ++j) v += acc[at * step + j * (2 * NP * 8 * step)];
          if (col < p.cols) put(part + k * p.cols + col, v, p.parts, p.parts_size, p.status);
        }
  }
}

struct JoinParams {
  const float *parts;
  int count, cols, gate_form, gate_type, weight_type;
  const void *gate, *post;
  void *dgate, *dpost, *dpre;
  float b;
  int *status;
};

// Weights' gradients from the CTAs' parts: 32 columns a CTA, its warps take parts in turn.
__global__ void __launch_bounds__(512) ns_block_norm_join_kernel(const __grid_constant__ JoinParams p) {
  __shared__ float red[2][16][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float s0 = 0.f, s1 = 0.f;
  if (col < p.cols)
#pragma unroll 4
    for (int k = warp; k < p.count; k += 16) {
      s0 += p.parts[(static_cast<int64_t>(k) * 2) * p.cols + col];
      s1 += p.parts[(static_cast<int64_t>(k) * 2 + 1) * p.cols + col];
    }
  red[0][warp][lane] = s0;
  red[1][warp][lane] = s1;
  __syncthreads();
  if (warp != 0 || col >= p.cols) return;
  for (int k = 1; k < 16; ++k) {
    s0 += red[0][k][lane];
    s1 += red[1][k][lane];
  }
  auto write = [&](void *out, int type, float v) {
    const size_t size = static_cast<size_t>(p.cols) * (type == kBF16 ? 2 : 4);
    if (type == kBF16) {
      __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(out) + col;
      if (in_bounds(to, 2, out, size, p.status)) *to = __float2bfloat16_rn(v);
    } else {
      float *to = static_cast<float *>(out) + col;
      if (in_bounds(to, 4, out, size, p.status)) *to = v;
    }
  };
  if (p.dpre) write(p.dpre, p.weight_type, s0);
  const float post = p.post ? one_of(p.post, col, p.weight_type) : 1.f;
  if (p.dpost) write(p.dpost, p.weight_type, p.b * s1 * (p.gate_form == kGateCols ? one_of(p.gate, col, p.gate_type) : 1.f));
  if (p.gate_form == kGateCols) write(p.dgate, p.gate_type, p.b * s1 * post);
}

}  // namespace
}  // namespace ns

using namespace ns;
using namespace ns::block_norm;

extern "C" int ns_block_norm_backward(const void *dresidual, int64_t ld_dr, const void *dnormed, int64_t ld_dz,
                                      const void *x, int64_t ld_x, const void *y, int64_t ld_y, const void *gate,
                                      int gate_form, int64_t ld_gate, const void *post, const void *pre,
                                      const float *post_rstd, const float *pre_rstd, int64_t rows, int64_t cols, float a,
                                      float b, void *dx, int64_t ld_dx, void *dy, int64_t ld_dy, void *dgate,
                                      int64_t ld_dgate, void *dpost, void *dpre, void *workspace,
                                      size_t workspace_bytes, int dtype, int block_dtype, int weight_dtype,
                                      int gate_dtype, void *stream) {
  NormParams p{};
  if (int rc = check(p, x, ld_x, y, ld_y, gate, gate_form, ld_gate, post, pre, rows, cols, a, b, dtype, block_dtype,
                     weight_dtype, gate_dtype))
    return rc;
  if ((dresidual && bad_shape(rows, cols, ld_dr)) || (pre && bad_shape(rows, cols, ld_dz)) || bad_shape(rows, cols, ld_dx) ||
      (y && bad_shape(rows, cols, ld_dy)) || (gate_form == kGateFull && bad_shape(rows, cols, ld_dgate)) ||
      (gate_form == kGateRows && bad_shape(rows, 1, ld_dgate)))
    return NS_EINVAL;
  if (cols == 0 && (rows == 0 || gate_form != kGateRows)) return NS_OK;
  if (cols == 0) {  // a row's gate has a gradient all the same: a sum over no columns
    const int ge = size_of(gate_dtype);
    if (!dgate) return NS_EINVAL;
    if (misaligned(dgate, ge)) return NS_EALIGN;
    if (Range(dgate, rows, 1, ld_dgate, ge).overlaps(Range(gate, rows, 1, ld_gate, ge))) return NS_EINVAL;
    OpCall call(stream);
    if (call.rc) return call.rc;
    return call.launch(kOpBlockNorm, [&] {
      if (cudaMemset2DAsync(dgate, static_cast<size_t>(ld_dgate) * ge, 0, ge, rows, call.s) == cudaSuccess) return 0;
      cudaGetLastError();
      return -1;
    });
  }
  if ((post && !dpost) || (pre && !dpre) || (gate_form == kGateCols && !dgate) || !workspace) return NS_EINVAL;
  if (rows > 0 && (!x || !dx || (y && !dy) || (pre && (!dnormed || !pre_rstd)) || (post && !post_rstd) ||
                   (gate_form != kGateNone && !dgate) || (!dresidual && !pre)))
    return NS_EINVAL;
  if (workspace_bytes < static_cast<size_t>(ns_block_norm_workspace(rows, cols))) return NS_ENOMEM;
  const int xe = size_of(dtype), ye = size_of(block_dtype), we = size_of(weight_dtype), ge = size_of(gate_dtype);
  if (misaligned(dresidual, xe) || misaligned(dnormed, ye) || misaligned(dx, xe) || misaligned(dy, ye) || misaligned(dgate, ge) ||
      misaligned(dpost, we) || misaligned(dpre, we) || misaligned(post_rstd, 4) || misaligned(pre_rstd, 4) || misaligned(workspace, 4))
    return NS_EALIGN;
  const Range in[] = {Range(dresidual, rows, cols, ld_dr, xe), Range(pre ? dnormed : nullptr, rows, cols, ld_dz, ye),
                      Range(x, rows, cols, ld_x, xe), Range(y, rows, cols, ld_y, ye),
                      gate_range(gate, gate_form, rows, cols, ld_gate, gate_dtype), Range(post, 1, cols, cols, we),
                      Range(pre, 1, cols, cols, we), Range(post ? post_rstd : nullptr, 1, rows, rows, 4),
                      Range(pre ? pre_rstd : nullptr, 1, rows, rows, 4)};
  const Range out[] = {Range(dx, rows, cols, ld_dx, xe), Range(y ? dy : nullptr, rows, cols, ld_dy, ye),
                       gate_range(dgate, gate_form, rows, cols, ld_dgate, gate_dtype),
                       Range(post ? dpost : nullptr, 1, cols, cols, we), Range(pre ? dpre : nullptr, 1, cols, cols, we),
                       Range(workspace, 1, static_cast<int64_t>(workspace_bytes), static_cast<int64_t>(workspace_bytes), 1)};
  const bool over_r = dx == dresidual && ld_dx == ld_dr, over_z = dy == dnormed && ld_dy == ld_dz;
  for (int o = 0; o < 6; ++o) {
    for (int i = 0; i < 9; ++i)
      if (!(o == 0 && i == 0 && over_r) && !(o == 1 && i == 1 && over_z) && out[o].overlaps(in[i])) return NS_EINVAL;
    for (int k = 0; k < o; ++k)
      if (out[o].overlaps(out[k])) return NS_EINVAL;
  }
  OpCall call(stream);
  if (call.rc) return call.rc;
  p.dr = dresidual;
  p.dz = dnormed;
  p.dx = dx;
  p.dy = dy;
  p.dgate = dgate;
  p.ld_dr = ld_dr;
  p.ld_dz = ld_dz;
  p.ld_dx = ld_dx;
  p.ld_dy = ld_dy;
  p.ld_dgate = ld_dgate;
  p.post_rstd = const_cast<float *>(post_rstd);
  p.pre_rstd = const_cast<float *>(pre_rstd);
  p.parts = static_cast<float *>(workspace);
  p.parts_size = workspace_bytes;
  p.status = call.status;
  p.wait_limit_ns = kWaitLimitNs;
  const bool wide = packs_fit(p, dtype, block_dtype) && rows_aligned(dresidual, ld_dr, xe, 8) && rows_aligned(dnormed, ld_dz, ye, 8) &&
                    rows_aligned(dx, ld_dx, xe, 8) && rows_aligned(dy, ld_dy, ye, 8) &&
                    (gate_form != kGateFull || rows_aligned(dgate, ld_dgate, ge, 8));
  const Shape sh(p, true, wide, dtype, block_dtype, call.sms);
  p.hold = sh.hold;
  const int grid = static_cast<int>(std::min<int64_t>({sh.batches(rows), static_cast<int64_t>(call.sms) * sh.per_sm, kMaxParts}));
  const JoinParams j{p.parts, grid, p.cols, gate_form, gate_dtype, weight_dtype, gate, post, dgate, post ? dpost : nullptr,
                     pre ? dpre : nullptr, b, call.status};
  return call.launch(kOpBlockNorm, [&] {
    int rc = 0;
    if (grid > 0) {
      rc = by_types(dtype, block_dtype, wide, [&](auto xt, auto yt, auto w) {
        return by_packs(sh.packs, [&](auto np) {
          auto *kernel = ns_block_norm_backward_kernel<decltype(xt)::value, decltype(yt)::value, decltype(w)::value, decltype(np)::value>;
          static SmemOptIn opt_in;
          if (opt_in.ensure(reinterpret_cast<const void *>(kernel), sh.smem)) return -1;
          kernel<<<grid, sh.block(wide), sh.smem, call.s>>>(p, sh.ring);
          return 0;
        });
      });
      if (rc) return rc;
      count_launch();
    }
    if (j.dpre || j.dpost || gate_form == kGateCols) {
      ns_block_norm_join_kernel<<<(p.cols + 31) / 32, 512, 0, call.s>>>(j);
      count_launch();
    }
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
  });
}
