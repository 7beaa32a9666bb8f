// ns_block_norm.cu -- the norms after and before a block, fused with the
// block's gate and the residual scale (include/ns.h), and their backward pass.
//
//     u = y * rsqrt(mean y^2 + eps) * post,  r = a x + b g u,  z = r * rsqrt(mean r^2 + eps) * pre
//
// Bound by HBM: forward reads x and y and writes r and z, backward reads the
// two gradients, x and y and writes two gradients (r is formed again, in fp32,
// from the kept 1 / rms of y). A row is held in the registers of its threads
// between the sums over it. The weights' gradients are sums over rows: a CTA
// walks over rows and adds in fp32, each thread its own columns, and a second
// launch adds the CTAs' parts in order.
#include <algorithm>
#include <cmath>

#include "../../include/ns.h"
#include "ns_rows.cuh"

namespace ns {

namespace {

enum Gate : int { kGateNone, kGateCols, kGateRows, kGateFull };
constexpr int kMaxCols = 16384;
constexpr int kMaxParts = 304;  // CTAs of a backward call: what the scratch holds

struct NormParams {
  const void *x, *y, *gate, *post, *pre;
  void *r, *z;              // forward
  float *post_rstd, *pre_rstd;
  const void *dr, *dz;      // backward
  void *dx, *dy, *dgate;
  float *parts;             // CTAs x 2 x cols: sums of dz * rh, and of the gate's (none, cols: drt * yh; else: g * drt * yh)
  int64_t ld_x, ld_y, ld_gate, ld_r, ld_z, ld_dr, ld_dz, ld_dx, ld_dy, ld_dgate;
  int64_t rows;
  int cols, gate_form, gate_type, weight_type;
  float a, b, eps;
  int *status;
};

// Value e of 8 that a thread holds from column c on: consecutive where rows allow packs (WIDE), else every 32nd.
template <bool WIDE>
__device__ __forceinline__ int col_of(int c, int e) { return WIDE ? c + e : c + 32 * e; }

template <int DT, bool WIDE>
__device__ __forceinline__ void load8(const void *row, int c, int cols, Pack<DT, 8> &v) {
  using E = typename Elem<DT>::T;
  const E *p = static_cast<const E *>(row);
  if constexpr (WIDE) {
    if (c < cols) {
      v.load(p + c);
      return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v.set(e, 0.f);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) reinterpret_cast<E *>(v.w)[e] = c + 32 * e < cols ? p[c + 32 * e] : Elem<DT>::from_f(0.f);
  }
}
template <int DT, bool WIDE>
__device__ __forceinline__ void store8(void *row, int c, int cols, const float (&f)[8], const void *base, size_t size, int *status) {
  using E = typename Elem<DT>::T;
  E *p = static_cast<E *>(row);
  Pack<DT, 8> v;
#pragma unroll
  for (int e = 0; e < 8; ++e) v.set(e, f[e]);
  if constexpr (WIDE) {
    if (c < cols) v.store_stream(p + c, base, size, status);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + 32 * e < cols && in_bounds(p + c + 32 * e, sizeof(E), base, size, status)) __stcs(p + c + 32 * e, reinterpret_cast<const E *>(v.w)[e]);
  }
}
// 8 values of either type as floats; 1 where there are none
template <bool WIDE>
__device__ __forceinline__ void load_any(const void *row, int type, int c, int cols, float (&f)[8]) {
  if (!row) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 1.f;
  } else if (type == kBF16) {
    Pack<kBF16, 8> v;
    load8<kBF16, WIDE>(row, c, cols, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = v.get(e);
  } else {
    Pack<kF32, 8> v;
    load8<kF32, WIDE>(row, c, cols, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = v.get(e);
  }
}
__device__ __forceinline__ const void *at_row(const void *p, int64_t row, int64_t ld, int type) {
  return static_cast<const uint8_t *>(p) + row * ld * (type == kBF16 ? 2 : 4);
}
__device__ __forceinline__ float one_of(const void *p, int64_t i, int type) {
  return type == kBF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]) : static_cast<const float *>(p)[i];
}

// Sum over the TPR threads of a row, the same on all, in a fixed order. red: 2 x TPR / 32 floats of the row's
// threads, used in turn, so one barrier a sum is enough.
struct RowSum {
  float *red;
  int threads, id, turn;
  __device__ __forceinline__ float operator()(float v) {
    v = warp_sum(v);
    if (threads == 32) return v;
    float *at = red + turn * (threads / 32);
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) at[(threadIdx.x % threads) / 32] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
    float s = 0.f;
    for (int k = 0; k < threads / 32; ++k) s += at[k];
    return s;
  }
};

// blockDim: (threads of a row, rows of a CTA)
template <int XT, int YT, bool WIDE, int NP>
__global__ void __launch_bounds__(512) ns_block_norm_kernel(const __grid_constant__ NormParams p) {
  using X = typename Elem<XT>::T;
  using Y = typename Elem<YT>::T;
  __shared__ float reds[8][32];
  RowSum sum{reds[threadIdx.y], static_cast<int>(blockDim.x), 1 + static_cast<int>(threadIdx.y), 0};
  const size_t rsize = static_cast<size_t>((p.rows - 1) * p.ld_r + p.cols) * sizeof(X);
  const size_t zsize = static_cast<size_t>((p.rows - 1) * p.ld_z + p.cols) * sizeof(Y);
  const float n = static_cast<float>(p.cols);
  int c[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i)
    c[i] = WIDE ? (i * blockDim.x + threadIdx.x) * 8 : (i * blockDim.x + (threadIdx.x & ~31u)) * 8 + (threadIdx.x & 31);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y; t < p.rows; t += static_cast<int64_t>(gridDim.x) * blockDim.y) {
    Pack<XT, 8> x[NP];
    Pack<YT, 8> y[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      load8<XT, WIDE>(at_row(p.x, t, p.ld_x, XT), c[i], p.cols, x[i]);
      if (p.y) load8<YT, WIDE>(at_row(p.y, t, p.ld_y, YT), c[i], p.cols, y[i]);
    }
    float r[NP][8];
    if (p.y) {
      float ry = 1.f;
      if (p.post) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NP; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) s = fmaf(y[i].get(e), y[i].get(e), s);
        ry = rsqrtf(sum(s) / n + p.eps);
        if (threadIdx.x == 0) p.post_rstd[t] = ry;
      }
      const float k = p.b * ry * (p.gate_form == kGateRows ? one_of(p.gate, t * p.ld_gate, p.gate_type) : 1.f);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        float w[8], g[8];
        load_any<WIDE>(p.post, p.weight_type, c[i], p.cols, w);
        const void *gate = p.gate_form == kGateCols ? p.gate : p.gate_form == kGateFull ? at_row(p.gate, t, p.ld_gate, p.gate_type) : nullptr;
        load_any<WIDE>(gate, p.gate_type, c[i], p.cols, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[i][e] = fmaf(y[i].get(e) * k, w[e] * g[e], p.a * x[i].get(e));
      }
    } else {
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) r[i][e] = p.a * x[i].get(e);
    }
    X *to = static_cast<X *>(p.r) + t * p.ld_r;
#pragma unroll
    for (int i = 0; i < NP; ++i) store8<XT, WIDE>(to, c[i], p.cols, r[i], p.r, rsize, p.status);
    if (p.pre) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(r[i][e], r[i][e], s);
      const float rr = rsqrtf(sum(s) / n + p.eps);
      if (threadIdx.x == 0) p.pre_rstd[t] = rr;
      Y *zt = static_cast<Y *>(p.z) + t * p.ld_z;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        float w[8];
        load_any<WIDE>(p.pre, p.weight_type, c[i], p.cols, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] *= r[i][e] * rr;
        store8<YT, WIDE>(zt, c[i], p.cols, w, p.z, zsize, p.status);
      }
    }
  }
}

// Backward. Shared memory: the columns' sums, [2][NP][8][threads of a row] floats for each row of the CTA, every
// thread its own.
template <int XT, int YT, bool WIDE, int NP>
__global__ void __launch_bounds__(512) ns_block_norm_backward_kernel(const __grid_constant__ NormParams p) {
  using X = typename Elem<XT>::T;
  using Y = typename Elem<YT>::T;
  extern __shared__ float sums[];
  __shared__ float reds[8][32];
  RowSum sum{reds[threadIdx.y], static_cast<int>(blockDim.x), 1 + static_cast<int>(threadIdx.y), 0};
  float *acc = sums + threadIdx.y * (2 * NP * 8 * blockDim.x) + threadIdx.x;
  const int step = blockDim.x;
#pragma unroll
  for (int i = 0; i < 2 * NP * 8; ++i) acc[i * step] = 0.f;
  const size_t xsize = static_cast<size_t>((p.rows - 1) * p.ld_dx + p.cols) * sizeof(X);
  const size_t ysize = static_cast<size_t>((p.rows - 1) * p.ld_dy + p.cols) * sizeof(Y);
  const float n = static_cast<float>(p.cols);
  int c[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i)
    c[i] = WIDE ? (i * blockDim.x + threadIdx.x) * 8 : (i * blockDim.x + (threadIdx.x & ~31u)) * 8 + (threadIdx.x & 31);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y; t < p.rows; t += static_cast<int64_t>(gridDim.x) * blockDim.y) {
    Pack<XT, 8> x[NP], dr[NP];
    Pack<YT, 8> y[NP], dz[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      load8<XT, WIDE>(at_row(p.x, t, p.ld_x, XT), c[i], p.cols, x[i]);
      if (p.y) load8<YT, WIDE>(at_row(p.y, t, p.ld_y, YT), c[i], p.cols, y[i]);
      if (p.pre) load8<YT, WIDE>(at_row(p.dz, t, p.ld_dz, YT), c[i], p.cols, dz[i]);
      if (p.dr) load8<XT, WIDE>(at_row(p.dr, t, p.ld_dr, XT), c[i], p.cols, dr[i]);
    }
    const float ry = p.y && p.post ? p.post_rstd[t] : 1.f, rr = p.pre ? p.pre_rstd[t] : 0.f;
    const float grow = p.gate_form == kGateRows ? one_of(p.gate, t * p.ld_gate, p.gate_type) : 1.f;
    float d[NP][8];  // the gradient of r
    if (p.pre) {
      float rh[NP][8], s = 0.f;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        float w[8], g[8];
        load_any<WIDE>(p.y ? p.post : nullptr, p.weight_type, c[i], p.cols, w);
        const void *gate = p.gate_form == kGateCols ? p.gate : p.gate_form == kGateFull ? at_row(p.gate, t, p.ld_gate, p.gate_type) : nullptr;
        load_any<WIDE>(gate, p.gate_type, c[i], p.cols, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float r = p.y ? fmaf(y[i].get(e) * (p.b * ry * grow), w[e] * g[e], p.a * x[i].get(e)) : p.a * x[i].get(e);
          rh[i][e] = r * rr;
        }
        load_any<WIDE>(p.pre, p.weight_type, c[i], p.cols, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float z = dz[i].get(e);
          acc[(i * 8 + e) * step] += z * rh[i][e];
          d[i][e] = z * w[e];
          s = fmaf(d[i][e], rh[i][e], s);
        }
      }
      s = sum(s) / n;
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) d[i][e] = fmaf(rr, d[i][e] - rh[i][e] * s, p.dr ? dr[i].get(e) : 0.f);
    } else {
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) d[i][e] = p.dr ? dr[i].get(e) : 0.f;
    }
    X *to = static_cast<X *>(p.dx) + t * p.ld_dx;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = p.a * d[i][e];
      store8<XT, WIDE>(to, c[i], p.cols, o, p.dx, xsize, p.status);
    }
    if (!p.y) continue;
    // through the gate: d * yh enters the sums; the gradient of y's norm is k = b g post d
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      float w[8], g[8];
      load_any<WIDE>(p.post, p.weight_type, c[i], p.cols, w);
      const void *gate = p.gate_form == kGateCols ? p.gate : p.gate_form == kGateFull ? at_row(p.gate, t, p.ld_gate, p.gate_type) : nullptr;
      load_any<WIDE>(gate, p.gate_type, c[i], p.cols, g);
      float og[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float yh = y[i].get(e) * ry, dyh = d[i][e] * yh;
        og[e] = p.b * w[e] * dyh;  // the gate's gradient
        acc[(NP * 8 + i * 8 + e) * step] += p.gate_form == kGateFull ? g[e] * dyh : grow * dyh;
        s = fmaf(og[e], g[e], s);
        d[i][e] *= p.b * grow * g[e] * w[e];
      }
      if (p.gate_form == kGateFull) {
        const size_t gsize = static_cast<size_t>((p.rows - 1) * p.ld_dgate + p.cols) * (p.gate_type == kBF16 ? 2 : 4);
        void *gt = const_cast<void *>(at_row(p.dgate, t, p.ld_dgate, p.gate_type));
        if (p.gate_type == kBF16)
          store8<kBF16, WIDE>(gt, c[i], p.cols, og, p.dgate, gsize, p.status);
        else
          store8<kF32, WIDE>(gt, c[i], p.cols, og, p.dgate, gsize, p.status);
      }
    }
    s = p.post || p.gate_form == kGateRows ? sum(s) : 0.f;
    if (p.gate_form == kGateRows && threadIdx.x == 0) {
      if (p.gate_type == kBF16)
        static_cast<__nv_bfloat16 *>(p.dgate)[t * p.ld_dgate] = __float2bfloat16_rn(s);
      else
        static_cast<float *>(p.dgate)[t * p.ld_dgate] = s;
    }
    const float k = p.post ? s * grow / n : 0.f;
    Y *yt = static_cast<Y *>(p.dy) + t * p.ld_dy;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      float o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = ry * (d[i][e] - y[i].get(e) * ry * k);
      store8<YT, WIDE>(yt, c[i], p.cols, o, p.dy, ysize, p.status);
    }
  }
  __syncthreads();
  // the CTA's rows added in order, to its part
  if (threadIdx.y == 0) {
    float *part = p.parts + static_cast<int64_t>(blockIdx.x) * 2 * p.cols;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int at = (k * NP + i) * 8 + e, col = col_of<WIDE>(c[i], e);
          float s = acc[at * step];
          for (int j = 1; j < static_cast<int>(blockDim.y); ++j) s += acc[at * step + j * (2 * NP * 8 * step)];
          if (col < p.cols) part[k * p.cols + col] = s;
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

// Threads of a row and packs a thread for `cols` columns, and rows of a CTA of about 256 threads.
struct Shape {
  int threads, packs, rows;
  Shape(int cols) {
    const int lanes = (cols + 7) / 8;
    packs = lanes <= 256 ? 1 : lanes <= 512 ? 2 : 4;
    threads = ((lanes + packs - 1) / packs + 31) / 32 * 32;
    rows = threads >= 256 ? 1 : std::min(8, 256 / threads);
  }
};

template <typename F>
int by_packs(int packs, F &&f) {
  return packs == 1 ? f(std::integral_constant<int, 1>{}) : packs == 2 ? f(std::integral_constant<int, 2>{}) : f(std::integral_constant<int, 4>{});
}
template <typename F>
int by_types(int xt, int yt, bool wide, F &&f) {
  using B = std::integral_constant<int, kBF16>;
  using S = std::integral_constant<int, kF32>;
  if (xt == kBF16) return wide ? f(B{}, B{}, std::true_type{}) : f(B{}, B{}, std::false_type{});
  if (yt == kBF16) return wide ? f(S{}, B{}, std::true_type{}) : f(S{}, B{}, std::false_type{});
  return wide ? f(S{}, S{}, std::true_type{}) : f(S{}, S{}, std::false_type{});
}

bool bad_type(int t) { return t != NS_F32 && t != NS_BF16; }
int size_of(int t) { return t == NS_BF16 ? 2 : 4; }
int backward_parts(int64_t rows, int sms, const Shape &sh) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({(rows + sh.rows - 1) / sh.rows, 2 * sms, kMaxParts})));
}

// The checks that both directions share; fills p. `written`: ranges of the outputs to come are checked by the caller.
int check(NormParams &p, const void *x, int64_t ld_x, const void *y, int64_t ld_y, const void *gate, int gate_form,
          int64_t ld_gate, const void *post, const void *pre, int64_t rows, int64_t cols, float a, float b, int dtype,
          int block_dtype, int weight_dtype, int gate_dtype) {
  if (bad_type(dtype) || bad_type(block_dtype) || bad_type(weight_dtype) || bad_type(gate_dtype)) return NS_EINVAL;
  if (dtype == NS_BF16 && block_dtype == NS_F32) return NS_EINVAL;  // a residual narrower than the block's output
  if (bad_shape(rows, cols, ld_x) || cols > kMaxCols || gate_form < kGateNone || gate_form > kGateFull) return NS_EINVAL;
  if (!std::isfinite(a) || !std::isfinite(b)) return NS_EINVAL;
  if (y && bad_shape(rows, cols, ld_y)) return NS_EINVAL;
  if (!y && (gate_form != kGateNone || post)) return NS_EINVAL;
  if (!y && !pre && rows > 0) return NS_EINVAL;  // nothing to do
  if ((gate_form != kGateNone) != (gate != nullptr) && rows > 0) return NS_EINVAL;
  if (gate_form == kGateFull && bad_shape(rows, cols, ld_gate)) return NS_EINVAL;
  if (gate_form == kGateRows && bad_shape(rows, 1, ld_gate)) return NS_EINVAL;
  if (misaligned(x, size_of(dtype)) || misaligned(y, size_of(block_dtype)) || misaligned(gate, size_of(gate_dtype)) ||
      misaligned(post, size_of(weight_dtype)) || misaligned(pre, size_of(weight_dtype)))
    return NS_EALIGN;
  p.x = x;
  p.y = y;
  p.gate = gate;
  p.post = post;
  p.pre = pre;
  p.ld_x = ld_x;
  p.ld_y = ld_y;
  p.ld_gate = ld_gate;
  p.rows = rows;
  p.cols = static_cast<int>(cols);
  p.gate_form = gate_form;
  p.gate_type = gate_dtype;
  p.weight_type = weight_dtype;
  p.a = a;
  p.b = b;
  return NS_OK;
}
// Whether every operand that is read in packs allows it.
bool packs_fit(const NormParams &p, int dtype, int block_dtype) {
  return p.cols % 8 == 0 && rows_aligned(p.x, p.ld_x, size_of(dtype), 8) && rows_aligned(p.y, p.ld_y, size_of(block_dtype), 8) &&
         !misaligned(p.post, 16) && !misaligned(p.pre, 16) &&
         (p.gate_form == kGateCols ? !misaligned(p.gate, 16)
                                   : p.gate_form != kGateFull || rows_aligned(p.gate, p.ld_gate, size_of(p.gate_type), 8));
}
Range gate_range(const void *gate, int form, int64_t rows, int64_t cols, int64_t ld, int type) {
  return form == kGateCols   ? Range(gate, 1, cols, cols, size_of(type))
         : form == kGateRows ? Range(gate, rows, 1, ld, size_of(type))
         : form == kGateFull ? Range(gate, rows, cols, ld, size_of(type))
                             : Range(nullptr, 0, 0, 0, 1);
}

}  // namespace
}  // namespace ns

using namespace ns;

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
  const Shape sh(p.cols);
  const bool wide = packs_fit(p, dtype, block_dtype) && rows_aligned(residual, ld_r, xe, 8) && (!pre || rows_aligned(normed, ld_z, ye, 8));
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>((rows + sh.rows - 1) / sh.rows, static_cast<int64_t>(call.sms) * 32));
  return call.launch(kOpBlockNorm, [&] {
    by_types(dtype, block_dtype, wide, [&](auto xt, auto yt, auto w) {
      return by_packs(sh.packs, [&](auto np) {
        ns_block_norm_kernel<decltype(xt)::value, decltype(yt)::value, decltype(w)::value, decltype(np)::value>
            <<<grid, dim3(sh.threads, sh.rows), 0, call.s>>>(p);
        return 0;
      });
    });
    count_launch();
    return cudaGetLastError() == cudaSuccess ? 0 : -1;
  });
}

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
  if (cols == 0) return NS_OK;
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
  p.status = call.status;
  const Shape sh(p.cols);
  const bool wide = packs_fit(p, dtype, block_dtype) && rows_aligned(dresidual, ld_dr, xe, 8) && rows_aligned(dnormed, ld_dz, ye, 8) &&
                    rows_aligned(dx, ld_dx, xe, 8) && rows_aligned(dy, ld_dy, ye, 8) &&
                    (gate_form != kGateFull || rows_aligned(dgate, ld_dgate, ge, 8));
  const int grid = rows == 0 ? 0 : backward_parts(rows, call.sms, sh);
  const int smem = 2 * sh.packs * 8 * sh.threads * sh.rows * 4;
  const JoinParams j{p.parts, grid, p.cols, gate_form, gate_dtype, weight_dtype, gate, post, dgate, post ? dpost : nullptr,
                     pre ? dpre : nullptr, b, call.status};
  return call.launch(kOpBlockNorm, [&] {
    int rc = 0;
    if (grid > 0) {
      rc = by_types(dtype, block_dtype, wide, [&](auto xt, auto yt, auto w) {
        return by_packs(sh.packs, [&](auto np) {
          auto *kernel = ns_block_norm_backward_kernel<decltype(xt)::value, decltype(yt)::value, decltype(w)::value, decltype(np)::value>;
          static SmemOptIn opt_in;
          if (opt_in.ensure(reinterpret_cast<const void *>(kernel), smem)) return -1;
          kernel<<<grid, dim3(sh.threads, sh.rows), smem, call.s>>>(p);
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
