// ns_ckpt.cu -- activations held for the backward pass in 8 bits, and the
// gated activation around them (include/ns.h).
//
// Element-wise work bound by HBM, so each operator is one pass that reads its
// inputs and writes its outputs once, and what is left is to keep the
// instructions per element well below what the copies take. A lane holds 8
// consecutive values of a row and the four lanes of a 32-value block find its
// largest magnitude by shuffles. The scale is a power of two, so quantising
// is one fused multiply-add: x * 2^k + 1.5 * 2^23 rounds the exact product
// half to even and leaves q in the sum's low byte. Rows whose pitch or base
// does not allow 16-byte accesses go through a warp's piece of shared memory:
// element by element and coalesced on the memory's side, 8 values a lane on
// the other (a block per warp access and a value per lane instead costs 33
// instructions per 32 values: 57 against 45 us for fp32 4093 x 6143 stored and
// loaded).
//
// 16384 x 14336 bf16: gated forward 298 us, 6.4 TB/s; backward 357 us, 6.6 TB/s
// (95 and 99 % of the copy rate). fp32 4093 x 6143, unaligned, stored and loaded:
// 45 us, 5.6 TB/s.
#include <algorithm>

#include "../../include/ns.h"
#include "ns_rows.cuh"

namespace ns {

namespace {

constexpr int kBlock = 32;  // values per scale
constexpr int kN = 8;       // consecutive values per lane
constexpr int kThreads = 256;

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
  int lanes_log2;      // lanes per row in a block: kThreads >> lanes_log2 rows at a time
  int *status;
};

// Exponent byte of a block whose largest magnitude has the float bits `top`.
__device__ __forceinline__ int block_exponent(uint32_t top) { return max(static_cast<int>(top >> 23), 7); }
__device__ __forceinline__ float up_factor(int e) { return __int_as_float((260 - min(e, 254)) << 23); }  // 2^(133-e)
// 2^(e-133); a padding or corrupt byte below 7 reads as 7, 255 as NaN
__device__ __forceinline__ float unit_of(int e) {
  return e == 255 ? __int_as_float(0x7fc00000) : __int_as_float((max(e, 7) - 6) << 23);
}
constexpr float kRound = 12582912.f;  // 1.5 * 2^23: a float this size has whole units

template <typename T>
__device__ __forceinline__ void put(T *at, T v, const void *base, size_t size, int *status) {
  if (in_bounds(at, sizeof(T), base, size, status)) *at = v;
}

// A lane's kN values of a row, columns c..., as they were read; zeros beyond the row.
template <int DT>
struct Values {
  using E = typename Elem<DT>::T;
  Pack<DT, kN> v;
  // rows that allow 16-byte accesses
  __device__ __forceinline__ void load(const E *row, int c, bool here) {
    if (here) {
      v.load_stream(row + c);
    } else {
#pragma unroll
      for (int e = 0; e < kN; ++e) v.set(e, 0.f);
    }
  }
  // other rows: the warp's 32 * kN columns from c0 on, lane by lane, to be exchanged afterwards
  __device__ __forceinline__ void load_spread(const E *row, int c0, int cols, bool row_here) {
    const int left = row_here ? cols - c0 - static_cast<int>(threadIdx.x & 31) : 0;
    const E *at = row + c0 + (threadIdx.x & 31);
#pragma unroll
    for (int e = 0; e < kN; ++e)
      reinterpret_cast<E *>(v.w)[e] = e * 32 < left ? __ldcs(at + e * 32) : Elem<DT>::from_f(0.f);
  }
  __device__ __forceinline__ void exchange(uint4 *stage) {
    const int lane = threadIdx.x & 31;
    E *s = reinterpret_cast<E *>(stage);
    __syncwarp();
#pragma unroll
    for (int e = 0; e < kN; ++e) s[e * 32 + lane] = reinterpret_cast<const E *>(v.w)[e];
    __syncwarp();
    constexpr int kW = sizeof(v.w) / 16;
#pragma unroll
    for (int i = 0; i < kW; ++i) reinterpret_cast<uint4 *>(v.w)[i] = stage[lane * kW + i];
  }
  // largest magnitude as float bits; NaN is the largest of all
  __device__ __forceinline__ uint32_t top() const {
    uint32_t m = 0;
    if constexpr (DT == kBF16) {
#pragma unroll
      for (int i = 0; i < kN / 2; ++i) m = __vmaxu2(m, reinterpret_cast<const uint32_t *>(v.w)[i] & 0x7fff7fffu);  // two at a time
      return max(m & 0xffff0000u, m << 16);
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i) m = max(m, __float_as_uint(v.get(i)) & 0x7fffffffu);
      return m;
    }
  }
};

// The bits whose low byte is q: x in a block whose largest magnitude has the
// bits `top`. 127.5 units and above would round to 128, and blocks with
// infinities or NaN hold zeros: both rare, both told by `top`.
__device__ __forceinline__ bool plain_block(uint32_t top) { return (top & 0x7fffffu) < 0x7f0000u && top < 0x7f800000u; }
__device__ __forceinline__ uint32_t quantise(float x, float up) { return __float_as_uint(fmaf(x, up, kRound)); }
__device__ __forceinline__ uint32_t quantise_rare(float x, float up, int ex) {
  return ex == 255 ? 0u : __float_as_uint(fminf(fmaxf(x * up, -127.f), 127.f) + kRound);
}

// Quantises a lane's values and writes them (with the padding behind the row)
// where `row`. All lanes of the warp call it.
template <int DT>
__device__ __forceinline__ void hold(const CkptParams &p, const Held &h, int64_t t, int c, bool row, const Values<DT> &x) {
  const size_t qsize = static_cast<size_t>(p.rows) * p.pitch, ssize = static_cast<size_t>(p.rows) * p.scale_pitch;
  uint32_t top = x.top();
#pragma unroll
  for (int o = 1; o < kBlock / kN; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const int ex = block_exponent(top);
  const float up = up_factor(ex);
  uint32_t b[kN];
  if (plain_block(top)) {
#pragma unroll
    for (int e = 0; e < kN; ++e) b[e] = quantise(x.v.get(e), up);
  } else {
#pragma unroll
    for (int e = 0; e < kN; ++e) b[e] = quantise_rare(x.v.get(e), up, ex);
  }
  if (!row) return;
  if (c < p.pitch) {
    auto four = [&](int i) {
      return __byte_perm(__byte_perm(b[i], b[i + 1], 0x0040), __byte_perm(b[i + 2], b[i + 3], 0x0040), 0x5410);
    };
    put(reinterpret_cast<uint2 *>(h.q + t * p.pitch + c), make_uint2(four(0), four(4)), h.q, qsize, p.status);
  }
  if (c % kBlock == 0 && c / kBlock < p.scale_pitch)
    put(h.s + t * p.scale_pitch + c / kBlock, static_cast<uint8_t>(c < p.cols ? ex : 0), h.s, ssize, p.status);
}

// What a checkpoint holds in a lane's columns of row t: the bytes and the scale.
struct HeldValues {
  uint2 w;
  int e;
  __device__ __forceinline__ void load(const CkptParams &p, const Held &h, int64_t t, int c) {
    e = __ldcs(h.s + t * p.scale_pitch + c / kBlock);
    w = __ldcs(reinterpret_cast<const uint2 *>(h.q + t * p.pitch + c));
  }
  // the i-th value: (byte + 128) + 2^23 as a float, minus both, in units; exact
  __device__ __forceinline__ float get(int i) const {
    const uint32_t u = __byte_perm((i < 4 ? w.x : w.y) ^ 0x80808080u, 0x4B000000u, 0x7540 + i % 4);
    return (__uint_as_float(u) - 8388736.f) * unit_of(e);
  }
};

// Writes a lane's values at row t, columns c..., where `here`; through `stage`
// by the whole warp (c0: its first column) for rows without 16-byte accesses.
template <int DT, bool WIDE>
__device__ __forceinline__ void write_row(const CkptParams &p, int which, int64_t t, int c, int c0, bool row, bool here,
                                          const float (&x)[kN], uint4 *stage) {
  using E = typename Elem<DT>::T;
  E *base = static_cast<E *>(p.out[which]);
  E *to = base + t * p.ld_out[which];
  const size_t size = static_cast<size_t>((p.rows - 1) * p.ld_out[which] + p.cols) * sizeof(E);
  Pack<DT, kN> v;
#pragma unroll
  for (int e = 0; e < kN; ++e) v.set(e, x[e]);
  if constexpr (WIDE) {
    if (here) v.store(to + c, base, size, p.status);
  } else {
    const int lane = threadIdx.x & 31;
    constexpr int kW = sizeof(v.w) / 16;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kW; ++i) stage[lane * kW + i] = reinterpret_cast<const uint4 *>(v.w)[i];
    __syncwarp();
    const E *s = reinterpret_cast<const E *>(stage) + lane;
    const int left = row ? p.cols - c0 - lane : 0;
    E *at = to + c0 + lane;
#pragma unroll
    for (int e = 0; e < kN; ++e)
      if (e * 32 < left) put(at + e * 32, s[e * 32], base, size, p.status);
  }
}

// 1 / (1 + exp(-x)). The fast division holds for divisors up to 2^126 and gives
// 0 beyond, where x is below -87.3 and the value 2^-126; so neither form divides
// by 1 + exp(-x) itself. fp32 data: below zero t / (1 + t) with t = exp(x), to a
// few units in the last place (of the smallest subnormal, where that is more).
// bf16 data: both sides of the fraction times 2^-24, which the exponential's
// argument takes in, to within 24 + |x| units of fp32, far below bf16's rounding.
// 16384 x 14336 bf16 both ways: 654 us (681 in the form for fp32); 8192 x 14336 fp32: 244
// us forward, 332 backward.
template <int DT>
__device__ __forceinline__ float sigmoid(float x) {
  if constexpr (DT == kF32) {
    const float t = expf(-fabsf(x));
    return __fdividef(x >= 0.f ? 1.f : t, 1.f + t);
  } else {
    constexpr float kLog2e = 1.44269504088896340736f, kDown = 1.f / 16777216.f;
    float t;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(x, -kLog2e, -24.f)));
    return __fdividef(kDown, kDown + t);
  }
}

enum Op : int { kStore, kLoad, kForward, kBackward };

// A block of threads covers kThreads >> lanes_log2 rows of 1 << lanes_log2
// lanes, further columns by blockIdx.x, and walks down the rows.
template <int OP, int DT, bool WIDE>
__global__ void __launch_bounds__(kThreads) ns_ckpt_kernel(const __grid_constant__ CkptParams p) {
  using E = typename Elem<DT>::T;
  __shared__ uint4 stages[WIDE ? 1 : kThreads / 32][WIDE ? 1 : 32 * kN * sizeof(E) / 16];
  uint4 *stage = stages[WIDE ? 0 : threadIdx.x / 32];
  const int c = ((blockIdx.x << p.lanes_log2) + (threadIdx.x & ((1 << p.lanes_log2) - 1))) * kN;
  const int c0 = c - (threadIdx.x & 31) * kN;  // the warp's first column (one row per warp where that is used)
  const int height = kThreads >> p.lanes_log2;
  const int64_t step = static_cast<int64_t>(gridDim.y) * height;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.y) * height; t0 < p.rows; t0 += step) {
    const int64_t t = t0 + (threadIdx.x >> p.lanes_log2);
    const bool row = t < p.rows, here = row && c < p.cols;
    auto read = [&](int which, Values<DT> &v) {
      const E *x = static_cast<const E *>(p.in[which]) + t * p.ld_in;
      if constexpr (WIDE)
        v.load(x, c, here);
      else
        v.load_spread(x, c0, p.cols, row);
    };
    auto write = [&](int which, const float (&x)[kN]) { write_row<DT, WIDE>(p, which, t, c, c0, row, here, x, stage); };
    Values<DT> a, b;
    HeldValues ga, ub;
    if constexpr (OP != kLoad) read(0, a);
    if constexpr (OP == kForward) read(1, b);
    if constexpr (OP == kLoad || OP == kBackward)
      if (here) ga.load(p, p.held[0], t, c);
    if constexpr (OP == kBackward)
      if (here) ub.load(p, p.held[1], t, c);
    if constexpr (!WIDE && OP != kLoad) a.exchange(stage);
    if constexpr (!WIDE && OP == kForward) b.exchange(stage);

    if constexpr (OP == kStore) hold<DT>(p, p.held[0], t, c, row, a);
    const bool compute = WIDE ? here : true;  // where lanes exchange values, all of them
    if (OP == kLoad && compute) {
      float v[kN];
#pragma unroll
      for (int e = 0; e < kN; ++e) v[e] = ga.get(e);
      write(0, v);
    }
    if constexpr (OP == kForward) {
      if (compute) {
        float h[kN];
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          const float g = a.v.get(e);
          h[e] = g * sigmoid<DT>(g) * b.v.get(e);
        }
        write(0, h);
      }
      hold<DT>(p, p.held[0], t, c, row, a);
      hold<DT>(p, p.held[1], t, c, row, b);
    }
    if (OP == kBackward && compute) {
      float dg[kN], du[kN], h[kN];
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        const float g = ga.get(e), u = ub.get(e), d = a.v.get(e);
        const float s = sigmoid<DT>(g), act = g * s;
        h[e] = act * u;
        du[e] = d * act;
        dg[e] = d * u * (s * fmaf(g, 1.f - s, 1.f));
      }
      write(0, dg);
      write(1, du);
      if (p.out[2]) write(2, h);
    }
  }
}

template <int OP, int DT, bool WIDE>
int run_one(CkptParams p, int sms, cudaStream_t s) {
  // store and forward also write the padding behind the last column
  const int64_t extent =
      OP == kStore || OP == kForward ? std::max<int64_t>(p.pitch, static_cast<int64_t>(p.scale_pitch) * kBlock) : p.cols;
  // lanes that cover a row: whole blocks of 32 values (4 lanes), whole warps where they exchange values
  const int64_t lanes = (extent + kN - 1) / kN;
  p.lanes_log2 = WIDE ? 2 : 5;
  while (p.lanes_log2 < 8 && (1 << p.lanes_log2) < lanes) ++p.lanes_log2;
  const int64_t gx = (lanes + (1 << p.lanes_log2) - 1) >> p.lanes_log2;
  const int height = kThreads >> p.lanes_log2;
  // Blocks beyond the resident ones even out the end; too many repeat the setup: 16384 x 14336 gated, both ways, with
  // a sigmoid that has since made 660 us 654: 675 us at 32 a SM, 660 at 128, 722 without a limit. (Two row steps in
  // flight per thread cost registers: 10 % slower.)
  const int64_t want = (p.rows + height - 1) / height;
  const int64_t most = std::max<int64_t>(1, static_cast<int64_t>(sms) * (WIDE ? 128 : 32) / gx);
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(std::min<int64_t>({want, most, 65535})), 1);
  ns_ckpt_kernel<OP, DT, WIDE><<<grid, kThreads, 0, s>>>(p);
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
      return wide ? run_one<OP, kBF16, true>(p, call.sms, call.s) : run_one<OP, kBF16, false>(p, call.sms, call.s);
    return wide ? run_one<OP, kF32, true>(p, call.sms, call.s) : run_one<OP, kF32, false>(p, call.sms, call.s);
  });
}

bool bad_dtype(int dtype) { return dtype != NS_F32 && dtype != NS_BF16; }
constexpr int64_t kMaxCols = int64_t(1) << 30;

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
  return ckpt_call<kStore>(p, dtype, cols % kN == 0 && rows_aligned(x, ld_x, elt, kN), stream);
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
  return ckpt_call<kLoad>(p, dtype, cols % kN == 0 && rows_aligned(out, ld_out, elt, kN), stream);
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
  const bool wide = cols % kN == 0 && rows_aligned(gate, ld_in, elt, kN) && rows_aligned(up, ld_in, elt, kN) &&
                    rows_aligned(h, ld_h, elt, kN);
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
  if (out[2].overlaps(out[0]) || out[2].overlaps(out[1]) || out[0].overlaps(out[1])) return NS_EINVAL;
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
  const bool wide = cols % kN == 0 && rows_aligned(dh, ld_dh, elt, kN) && rows_aligned(dgate, ld_d, elt, kN) &&
                    rows_aligned(dup, ld_d, elt, kN) && (!h || rows_aligned(h, ld_h, elt, kN));
  return ckpt_call<kBackward>(p, dtype, wide, stream);
}
