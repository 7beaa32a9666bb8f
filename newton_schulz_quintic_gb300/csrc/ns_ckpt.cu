// ns_ckpt.cu -- activations held for the backward pass in 8 bits, and the
// gated activation around them (include/ns.h).
//
// Element-wise work bound by HBM, so each operator is one pass that reads its
// inputs and writes its outputs once. A lane holds kLane consecutive values
// of a row and the lanes of a 32-value block find its largest magnitude by
// shuffles; the scale is a power of two, so quantising multiplies by an exact
// factor and rounds once. Two lane widths: 16 values (16-byte accesses of q)
// when every row allows it, else one value per lane, a block per warp access,
// which stays coalesced for any pitch and alignment.
#include <algorithm>

#include "../../include/ns.h"
#include "ns_rows.cuh"

namespace ns {

namespace {

constexpr int kBlock = 32;  // values per scale

struct Held {  // a checkpoint
  int8_t *q;
  uint8_t *s;
};

struct CkptParams {
  const void *in[2];   // store: x; gated forward: gate, up; gated backward: dh
  void *out[3];        // load: values; forward: h; backward: dgate, dup, h (or nullptr)
  Held held[2];
  int64_t rows;
  int64_t ld_in, ld_out[3];
  int cols, pitch, scale_pitch;
  int *status;
};

// Exponent byte of a block whose largest magnitude has the float bits `top`.
__device__ __forceinline__ int block_exponent(uint32_t top) { return max(static_cast<int>(top >> 23), 7); }
__device__ __forceinline__ float up_factor(int e) { return __int_as_float((260 - min(e, 254)) << 23); }  // 2^(133-e)
// 2^(e-133); a padding or corrupt byte below 7 reads as 7, 255 as NaN
__device__ __forceinline__ float unit_of(int e) {
  return e == 255 ? __int_as_float(0x7fc00000) : __int_as_float((max(e, 7) - 6) << 23);
}
__device__ __forceinline__ int quantise(float x, float up) {
  return max(-127, min(127, __float2int_rn(x * up)));
}

// Largest magnitude (as float bits; NaN is the largest of all) over the lanes
// of a block: LANE values per lane, so 32 / LANE neighbouring lanes.
template <int LANE>
__device__ __forceinline__ uint32_t block_top(uint32_t top) {
  if constexpr (LANE == 1) {
    return __reduce_max_sync(0xffffffffu, top);
  } else {
#pragma unroll
    for (int o = 1; o < kBlock / LANE; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    return top;
  }
}

// The values of one lane quantised and written: x[0..LANE) at row t, columns
// c.. (values beyond the row are 0 and become the padding bytes).
template <int LANE>
__device__ __forceinline__ void hold(const CkptParams &p, const Held &h, int64_t t, int c, float (&x)[LANE]) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < LANE; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
  top = block_top<LANE>(top);
  const int ex = block_exponent(top);
  const float up = up_factor(ex);
  Pack<kF32, LANE / 4 + (LANE < 4)> bytes;  // LANE bytes as words
  int8_t *q8 = reinterpret_cast<int8_t *>(bytes.w);
#pragma unroll
  for (int e = 0; e < LANE; ++e) {
    const int q = ex == 255 ? 0 : quantise(x[e], up);
    q8[e] = static_cast<int8_t>(q);
    x[e] = static_cast<float>(q) * unit_of(ex);  // what is held
  }
  const size_t qsize = static_cast<size_t>(p.rows) * p.pitch, ssize = static_cast<size_t>(p.rows) * p.scale_pitch;
  if (c < p.pitch) {
    int8_t *q = h.q + t * p.pitch + c;
    if (LANE == 1) {
      if (in_bounds(q, 1, h.q, qsize, p.status)) *q = q8[0];
    } else {
      bytes.store(reinterpret_cast<float *>(q), h.q, qsize, p.status);
    }
  }
  const int b = c / kBlock;
  if (c % kBlock == 0 && b < p.scale_pitch) {
    uint8_t *s = h.s + t * p.scale_pitch + b;
    if (in_bounds(s, 1, h.s, ssize, p.status)) *s = c < p.cols ? static_cast<uint8_t>(ex) : 0;
  }
}

// The values a checkpoint holds at row t, columns c.. (0 beyond the row).
template <int LANE>
__device__ __forceinline__ void recall(const CkptParams &p, const Held &h, int64_t t, int c, float (&x)[LANE]) {
  if (c >= p.cols) {
#pragma unroll
    for (int e = 0; e < LANE; ++e) x[e] = 0.f;
    return;
  }
  const float unit = unit_of(h.s[t * p.scale_pitch + c / kBlock]);
  const int8_t *q = h.q + t * p.pitch + c;
  if (LANE == 1) {
    x[0] = static_cast<float>(*q) * unit;
  } else {
    Pack<kF32, LANE / 4 + (LANE < 4)> bytes;
    bytes.load(reinterpret_cast<const float *>(q));
    const int8_t *q8 = reinterpret_cast<const int8_t *>(bytes.w);
#pragma unroll
    for (int e = 0; e < LANE; ++e) x[e] = static_cast<float>(q8[e]) * unit;
  }
}

template <int DT, int LANE>
__device__ __forceinline__ void read_row(const void *base, int64_t off, int c, int cols, float (&x)[LANE]) {
  using P = Pack<DT, LANE>;
  P v;
  if (c < cols) v.load_stream(static_cast<const typename P::E *>(base) + off + c);
#pragma unroll
  for (int e = 0; e < LANE; ++e) x[e] = c < cols ? v.get(e) : 0.f;
}
template <int DT, int LANE>
__device__ __forceinline__ void write_row(const CkptParams &p, int which, int64_t t, int c, const float (&x)[LANE]) {
  using P = Pack<DT, LANE>;
  if (c >= p.cols) return;
  P v;
#pragma unroll
  for (int e = 0; e < LANE; ++e) v.set(e, x[e]);
  typename P::E *base = static_cast<typename P::E *>(p.out[which]);
  v.store(base + t * p.ld_out[which] + c, base,
          static_cast<size_t>((p.rows - 1) * p.ld_out[which] + p.cols) * sizeof(typename P::E), p.status);
}

template <int DT>
__device__ __forceinline__ float sigmoid(float x) {
  return 1.f / (1.f + (DT == kF32 ? expf(-x) : __expf(-x)));
}

enum Op : int { kStore, kLoad, kForward, kBackward };

// One warp per (row, 32 * LANE columns).
template <int OP, int DT, int LANE>
__global__ void __launch_bounds__(256) ns_ckpt_kernel(const __grid_constant__ CkptParams p) {
  const int lane = threadIdx.x & 31;
  const int span = 32 * LANE;
  // store and forward also write the padding bytes behind the last column
  const int extent = OP == kStore || OP == kForward ? max(p.pitch, p.scale_pitch * kBlock) : p.cols;
  const int per_row = (extent + span - 1) / span;
  const int64_t items = p.rows * per_row;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); it < items;
       it += static_cast<int64_t>(gridDim.x) * 8) {
    const int64_t t = it / per_row;
    const int c = static_cast<int>(it - t * per_row) * span + lane * LANE;
    if (OP == kStore) {
      float x[LANE];
      read_row<DT, LANE>(p.in[0], t * p.ld_in, c, p.cols, x);
      hold<LANE>(p, p.held[0], t, c, x);
    } else if (OP == kLoad) {
      float x[LANE];
      recall<LANE>(p, p.held[0], t, c, x);
      write_row<DT, LANE>(p, 0, t, c, x);
    } else if (OP == kForward) {
      float g[LANE], u[LANE], h[LANE];
      read_row<DT, LANE>(p.in[0], t * p.ld_in, c, p.cols, g);
      read_row<DT, LANE>(p.in[1], t * p.ld_in, c, p.cols, u);
#pragma unroll
      for (int e = 0; e < LANE; ++e) h[e] = g[e] * sigmoid<DT>(g[e]) * u[e];
      write_row<DT, LANE>(p, 0, t, c, h);
      hold<LANE>(p, p.held[0], t, c, g);
      hold<LANE>(p, p.held[1], t, c, u);
    } else {
      float d[LANE], g[LANE], u[LANE], h[LANE];
      read_row<DT, LANE>(p.in[0], t * p.ld_in, c, p.cols, d);
      recall<LANE>(p, p.held[0], t, c, g);
      recall<LANE>(p, p.held[1], t, c, u);
#pragma unroll
      for (int e = 0; e < LANE; ++e) {
        const float s = sigmoid<DT>(g[e]), act = g[e] * s;
        h[e] = act * u[e];
        g[e] = d[e] * u[e] * (s * fmaf(g[e], 1.f - s, 1.f));
        u[e] = d[e] * act;
      }
      write_row<DT, LANE>(p, 0, t, c, g);
      write_row<DT, LANE>(p, 1, t, c, u);
      if (p.out[2]) write_row<DT, LANE>(p, 2, t, c, h);
    }
  }
}

template <int OP, int DT, int LANE>
int run_one(const CkptParams &p, int sms, cudaStream_t s) {
  const int span = 32 * LANE;
  const int64_t extent = std::max<int64_t>(p.pitch, static_cast<int64_t>(p.scale_pitch) * kBlock);
  const int64_t items = p.rows * ((extent + span - 1) / span);
  const int grid = static_cast<int>(std::min<int64_t>((items + 7) / 8, static_cast<int64_t>(sms) * 16));
  ns_ckpt_kernel<OP, DT, LANE><<<grid, 256, 0, s>>>(p);
  count_launch();
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

template <int OP>
int ckpt_call(CkptParams &p, int dtype, bool wide, void *stream) {
  OpCall call(stream);
  if (call.rc) return call.rc;
  p.status = call.status;
  return call.launch(kOpCkpt, [&] {
    if (dtype == NS_BF16)
      return wide ? run_one<OP, kBF16, 16>(p, call.sms, call.s) : run_one<OP, kBF16, 1>(p, call.sms, call.s);
    return wide ? run_one<OP, kF32, 16>(p, call.sms, call.s) : run_one<OP, kF32, 1>(p, call.sms, call.s);
  });
}

bool bad_dtype(int dtype) { return dtype != NS_F32 && dtype != NS_BF16; }
constexpr int64_t kMaxCols = int64_t(1) << 30;

// Two rows x cols matrices with one pitch: disjoint, or the interleaved halves of wider rows.
bool halves_overlap(const void *a, const void *b, int64_t rows, int64_t cols, int64_t ld, int elt) {
  if (!Range(a, rows, cols, ld, elt).overlaps(Range(b, rows, cols, ld, elt))) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  const uintptr_t d = x < y ? y - x : x - y;
  const uintptr_t in_row = d % (static_cast<uintptr_t>(ld) * elt);  // d is less than a matrix: some row lies beside another
  return in_row < static_cast<uintptr_t>(cols) * elt || in_row > static_cast<uintptr_t>(ld - cols) * elt;
}

}  // namespace
}  // namespace ns

using namespace ns;

extern "C" int64_t ns_ckpt_pitch(int64_t cols) { return cols < 0 ? -1 : (cols + 15) / 16 * 16; }
extern "C" int64_t ns_ckpt_scale_pitch(int64_t cols) { return cols < 0 ? -1 : ((cols + 31) / 32 + 3) / 4 * 4; }

extern "C" int ns_ckpt_store(const void *x, int64_t ld_x, int64_t rows, int64_t cols, void *q, void *scales,
                             int dtype, void *stream) {
  if (bad_dtype(dtype) || bad_shape(rows, cols, ld_x) || cols > kMaxCols) return NS_EINVAL;
  if (rows == 0 || cols == 0) return NS_OK;
  if (!x || !q || !scales) return NS_EINVAL;
  const int elt = dtype == NS_BF16 ? 2 : 4;
  if (misaligned(x, elt) || misaligned(q, 16) || misaligned(scales, 16)) return NS_EALIGN;
  CkptParams p{};
  p.pitch = static_cast<int>(ns_ckpt_pitch(cols));
  p.scale_pitch = static_cast<int>(ns_ckpt_scale_pitch(cols));
  const Range rx(x, rows, cols, ld_x, elt), rq(q, rows, p.pitch, p.pitch, 1), rs(scales, rows, p.scale_pitch, p.scale_pitch, 1);
  if (rq.overlaps(rx) || rs.overlaps(rx) || rq.overlaps(rs)) return NS_EINVAL;
  p.in[0] = x;
  p.ld_in = ld_x;
  p.rows = rows;
  p.cols = static_cast<int>(cols);
  p.held[0] = Held{static_cast<int8_t *>(q), static_cast<uint8_t *>(scales)};
  return ckpt_call<kStore>(p, dtype, cols % 16 == 0 && rows_aligned(x, ld_x, elt, 16), stream);
}

extern "C" int ns_ckpt_load(const void *q, const void *scales, int64_t rows, int64_t cols, void *out, int64_t ld_out,
                            int dtype, void *stream) {
  if (bad_dtype(dtype) || bad_shape(rows, cols, ld_out) || cols > kMaxCols) return NS_EINVAL;
  if (rows == 0 || cols == 0) return NS_OK;
  if (!out || !q || !scales) return NS_EINVAL;
  const int elt = dtype == NS_BF16 ? 2 : 4;
  if (misaligned(out, elt) || misaligned(q, 16) || misaligned(scales, 16)) return NS_EALIGN;
  CkptParams p{};
  p.pitch = static_cast<int>(ns_ckpt_pitch(cols));
  p.scale_pitch = static_cast<int>(ns_ckpt_scale_pitch(cols));
  const Range ro(out, rows, cols, ld_out, elt);
  if (ro.overlaps(Range(q, rows, p.pitch, p.pitch, 1)) || ro.overlaps(Range(scales, rows, p.scale_pitch, p.scale_pitch, 1)))
    return NS_EINVAL;
  p.out[0] = out;
  p.ld_out[0] = ld_out;
  p.rows = rows;
  p.cols = static_cast<int>(cols);
  p.held[0] = Held{static_cast<int8_t *>(const_cast<void *>(q)), static_cast<uint8_t *>(const_cast<void *>(scales))};
  return ckpt_call<kLoad>(p, dtype, cols % 16 == 0 && rows_aligned(out, ld_out, elt, 16), stream);
}

extern "C" int ns_gated_forward(const void *gate, const void *up, int64_t ld_in, int64_t rows, int64_t cols, void *h,
                                int64_t ld_h, void *q_gate, void *s_gate, void *q_up, void *s_up, int dtype,
                                void *stream) {
  if (bad_dtype(dtype) || bad_shape(rows, cols, ld_in) || bad_shape(rows, cols, ld_h) || cols > kMaxCols) return NS_EINVAL;
  if (rows == 0 || cols == 0) return NS_OK;
  if (!gate || !up || !h || !q_gate || !s_gate || !q_up || !s_up) return NS_EINVAL;
  const int elt = dtype == NS_BF16 ? 2 : 4;
  if (misaligned(gate, elt) || misaligned(up, elt) || misaligned(h, elt) || misaligned(q_gate, 16) ||
      misaligned(s_gate, 16) || misaligned(q_up, 16) || misaligned(s_up, 16))
    return NS_EALIGN;
  CkptParams p{};
  p.pitch = static_cast<int>(ns_ckpt_pitch(cols));
  p.scale_pitch = static_cast<int>(ns_ckpt_scale_pitch(cols));
  const Range in[] = {Range(gate, rows, cols, ld_in, elt), Range(up, rows, cols, ld_in, elt)};
  const Range out[] = {Range(h, rows, cols, ld_h, elt), Range(q_gate, rows, p.pitch, p.pitch, 1),
                       Range(s_gate, rows, p.scale_pitch, p.scale_pitch, 1), Range(q_up, rows, p.pitch, p.pitch, 1),
                       Range(s_up, rows, p.scale_pitch, p.scale_pitch, 1)};
  for (int i = 0; i < 5; ++i) {
    if (out[i].overlaps(in[0]) || out[i].overlaps(in[1])) return NS_EINVAL;
    for (int k = 0; k < i; ++k)
      if (out[i].overlaps(out[k])) return NS_EINVAL;
  }
  p.in[0] = gate;
  p.in[1] = up;
  p.ld_in = ld_in;
  p.out[0] = h;
  p.ld_out[0] = ld_h;
  p.rows = rows;
  p.cols = static_cast<int>(cols);
  p.held[0] = Held{static_cast<int8_t *>(q_gate), static_cast<uint8_t *>(s_gate)};
  p.held[1] = Held{static_cast<int8_t *>(q_up), static_cast<uint8_t *>(s_up)};
  const bool wide = cols % 16 == 0 && rows_aligned(gate, ld_in, elt, 16) && rows_aligned(up, ld_in, elt, 16) &&
                    rows_aligned(h, ld_h, elt, 16);
  return ckpt_call<kForward>(p, dtype, wide, stream);
}

extern "C" int ns_gated_backward(const void *dh, int64_t ld_dh, const void *q_gate, const void *s_gate,
                                 const void *q_up, const void *s_up, int64_t rows, int64_t cols, void *dgate,
                                 void *dup, int64_t ld_d, void *h, int64_t ld_h, int dtype, void *stream) {
  if (bad_dtype(dtype) || bad_shape(rows, cols, ld_dh) || bad_shape(rows, cols, ld_d) ||
      (h && bad_shape(rows, cols, ld_h)) || cols > kMaxCols)
    return NS_EINVAL;
  if (rows == 0 || cols == 0) return NS_OK;
  if (!dh || !dgate || !dup || !q_gate || !s_gate || !q_up || !s_up) return NS_EINVAL;
  const int elt = dtype == NS_BF16 ? 2 : 4;
  if (misaligned(dh, elt) || misaligned(dgate, elt) || misaligned(dup, elt) || misaligned(h, elt) ||
      misaligned(q_gate, 16) || misaligned(s_gate, 16) || misaligned(q_up, 16) || misaligned(s_up, 16))
    return NS_EALIGN;
  CkptParams p{};
  p.pitch = static_cast<int>(ns_ckpt_pitch(cols));
  p.scale_pitch = static_cast<int>(ns_ckpt_scale_pitch(cols));
  const Range in[] = {Range(dh, rows, cols, ld_dh, elt), Range(q_gate, rows, p.pitch, p.pitch, 1),
                      Range(s_gate, rows, p.scale_pitch, p.scale_pitch, 1), Range(q_up, rows, p.pitch, p.pitch, 1),
                      Range(s_up, rows, p.scale_pitch, p.scale_pitch, 1)};
  const Range out[] = {Range(dgate, rows, cols, ld_d, elt), Range(dup, rows, cols, ld_d, elt), Range(h, rows, cols, ld_h, elt)};
  for (const Range &o : out)
    for (const Range &i : in)
      if (o.overlaps(i)) return NS_EINVAL;
  if (out[2].overlaps(out[0]) || out[2].overlaps(out[1]) || halves_overlap(dgate, dup, rows, cols, ld_d, elt)) return NS_EINVAL;
  p.in[0] = dh;
  p.ld_in = ld_dh;
  p.out[0] = dgate;
  p.out[1] = dup;
  p.out[2] = h;
  p.ld_out[0] = p.ld_out[1] = ld_d;
  p.ld_out[2] = ld_h;
  p.rows = rows;
  p.cols = static_cast<int>(cols);
  p.held[0] = Held{static_cast<int8_t *>(const_cast<void *>(q_gate)), static_cast<uint8_t *>(const_cast<void *>(s_gate))};
  p.held[1] = Held{static_cast<int8_t *>(const_cast<void *>(q_up)), static_cast<uint8_t *>(const_cast<void *>(s_up))};
  const bool wide = cols % 16 == 0 && rows_aligned(dh, ld_dh, elt, 16) && rows_aligned(dgate, ld_d, elt, 16) &&
                    rows_aligned(dup, ld_d, elt, 16) && (!h || rows_aligned(h, ld_h, elt, 16));
  return ckpt_call<kBackward>(p, dtype, wide, stream);
}
