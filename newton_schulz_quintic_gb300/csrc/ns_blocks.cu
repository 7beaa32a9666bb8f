// ns_blocks.cu -- matrices held in e4m3 with a power-of-two scale for each
// block of 128 (include/ns.h): rows with 1 x 128 blocks, rows gathered on the
// way, and weights with 128 x 128 blocks; and the values read back. Their
// product is in ns_blocks_mm.cu.
//
// The scale is the smallest power of two that brings a block's largest
// magnitude to 448 or less, found in the bits of that magnitude, so x * 2^-e is
// exact and the conversion to e4m3 rounds once, half to even.
//
// Element-wise work bound by HBM: one read, one write. Rows: a lane holds 16
// consecutive values (8 where rows allow no packs) and the lanes of a block find
// its largest magnitude by shuffles. Weights: a CTA holds one 128 x 128 block in
// registers between the two steps. Stored: 16384 x 8192 bf16 rows in 60 us, 6.7
// TB/s, 8 x 8192 x 6144 weights in 181 us, 6.7 TB/s; read back 68 and 206 us, 5.9 TB/s;
// 38912 rows gathered from 9728 of 6144: 94 us (rows that left L2 are read again).
#include <algorithm>

#include "../../include/ns.h"
#include "ns_rows.cuh"

namespace ns {

namespace {

constexpr int kThreads = 256;
constexpr int kBlock = 128;

struct BlocksParams {
  const void *x;          // store: values; load: nothing
  void *out;              // load: values
  int64_t ld;             // pitch of the values
  int64_t rows;           // rows of q (of one matrix of a stack)
  int64_t src_rows;       // rows form: rows of x
  const int32_t *index;   // rows form: row r holds x[index[r] / per]; nullptr: x[r]
  uint32_t per, per_mul;  // a division by per of numbers below 2^31: (mulhi(n, per_mul) + n) >> per_shift
  int per_shift;
  uint8_t *q, *s;
  int cols, pitch, scale_pitch;
  int groups;             // matrices of a stack (tiles)
  int tiles;              // load: 128 x 128 blocks
  int lanes_log2;
  int *status;
};

// The scale byte of a block whose largest magnitude has the float bits `top`, and 2^(127 - byte).
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  return top >= 0x7f800000u ? 255u : static_cast<uint32_t>(max(static_cast<int>((top + 0x1fffffu) >> 23) - 8, 1));
}
__device__ __forceinline__ float up_of(uint32_t s) {  // NaN for a block with infinities or NaN: every value of it
  return __uint_as_float(s == 255 ? 0x7fc00000u : (254u - s) << 23);
}
__device__ __forceinline__ float unit_of(uint32_t s) {  // a padding byte 0 reads as 1
  return __uint_as_float(s == 255 ? 0x7fc00000u : max(s, 1u) << 23);
}
__device__ __forceinline__ uint32_t to_e4m3x2(float low, float high) {
  uint16_t v;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(high), "f"(low));
  return v;
}
// Two e4m3 values as floats, exactly (every e4m3 value is an fp16 value).
__device__ __forceinline__ void from_e4m3x2(uint32_t v, float &low, float &high) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
  asm("{.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;}" : "=f"(low), "=f"(high) : "r"(h));
}

// Largest magnitude of a lane's 8 values as float bits; NaN is the largest of all.
template <int DT, typename V>
__device__ __forceinline__ uint32_t top_of(const V &v) {
  uint32_t m = 0;
  if constexpr (DT == kBF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, reinterpret_cast<const uint32_t *>(v.w)[i] & 0x7fff7fffu);
    return max(m & 0xffff0000u, m << 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v.get(i)) & 0x7fffffffu);
    return m;
  }
}
template <typename V>
__device__ __forceinline__ uint2 eight_e4m3(const V &v, float up) {
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __fmul2_rn(make_float2(v.get(2 * i), v.get(2 * i + 1)), make_float2(up, up));
    b[i] = to_e4m3x2(f.x, f.y);
  }
  return make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
}

// Rows that allow packs: 16 columns a lane, 8 lanes a block, so that what a lane does for its row and block (addresses,
// the scale, shuffles) is spread over 16 values. What bounds it is instructions: 8 columns a lane took 162 a warp for 256
// values of bf16, 102 us at 16384 x 8192.
template <int DT, bool GATHER>
__global__ void __launch_bounds__(kThreads) ns_blocks_store_rows_kernel(const __grid_constant__ BlocksParams p) {
  using E = typename Elem<DT>::T;
  const int lanes = 1 << p.lanes_log2;
  const int c = ((blockIdx.x << p.lanes_log2) + (threadIdx.x & (lanes - 1))) * 16;
  const int height = kThreads >> p.lanes_log2, step = gridDim.y * height;
  const size_t qsize = static_cast<size_t>(p.rows) * p.pitch, ssize = static_cast<size_t>(p.rows) * p.scale_pitch;
  const E *x = static_cast<const E *>(p.x) + c;
  const int rows = static_cast<int>(p.rows), src_rows = static_cast<int>(p.src_rows);
  const bool in0 = c < p.cols, in1 = c + 8 < p.cols;
  asm volatile("griddepcontrol.launch_dependents;");  // a product may set itself up meanwhile
  int t = blockIdx.y * height + (threadIdx.x >> p.lanes_log2);
  auto index_at = [&](int r) { return GATHER && r < rows ? __ldg(p.index + r) : -1; };
  int32_t index = index_at(t);
  for (int t0 = blockIdx.y * height; t0 < rows; t0 += step, t += step) {
    int from = t;
    bool here = t < rows;
    if (GATHER) {
      // index / per: the product with the rounded-up reciprocal, for dividends below 2^31
      from = static_cast<int>((__umulhi(static_cast<uint32_t>(index), p.per_mul) + static_cast<uint32_t>(index)) >> p.per_shift);
      here = index >= 0 && from < src_rows;
      index = index_at(t + step);
    }
    const E *at = x + static_cast<int64_t>(from) * p.ld;
    Pack<DT, 8> v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (here && (h == 0 ? in0 : in1)) {
        if (GATHER)
          v[h].load(at + 8 * h);  // rows that are read again stay in the caches
        else
          v[h].load_stream(at + 8 * h);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[h].set(e, 0.f);
      }
    }
    uint32_t top = max(top_of<DT>(v[0]), top_of<DT>(v[1]));
#pragma unroll
    for (int o = 1; o < kBlock / 16; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t sb = scale_byte(top);
    const float up = up_of(sb);
    const uint2 lo = eight_e4m3(v[0], up), hi = eight_e4m3(v[1], up);
    if (t < rows) {
      if (in0) {  // the padding behind the row is part of its last 16
        const uint2 high = in1 ? hi : make_uint2(0, 0);  // zeros behind a NaN block too
        uint4 *to = reinterpret_cast<uint4 *>(p.q + static_cast<int64_t>(t) * p.pitch + c);
        if (in_bounds(to, 16, p.q, qsize, p.status)) {
          if (GATHER)
            __stcs(to, make_uint4(lo.x, lo.y, high.x, high.y));
          else
            *to = make_uint4(lo.x, lo.y, high.x, high.y);
        }
      }
      if (c % kBlock == 0 && c / kBlock < p.scale_pitch)
        put(p.s + static_cast<int64_t>(t) * p.scale_pitch + c / kBlock, static_cast<uint8_t>(in0 ? sb : 0), p.s, ssize, p.status);
    }
  }
}

// Any rows: 8 columns a lane, through shared memory.
template <int DT>
__global__ void __launch_bounds__(kThreads) ns_blocks_store_any_kernel(const __grid_constant__ BlocksParams p) {
  using E = typename Elem<DT>::T;
  using V = Eight<DT, false>;
  __shared__ uint4 stages[kThreads / 32][V::kStage];
  uint4 *stage = stages[threadIdx.x / 32];
  const int c = ((blockIdx.x << p.lanes_log2) + (threadIdx.x & ((1 << p.lanes_log2) - 1))) * 8;
  const int height = kThreads >> p.lanes_log2;
  const int64_t step = static_cast<int64_t>(gridDim.y) * height;
  const size_t qsize = static_cast<size_t>(p.rows) * p.pitch, ssize = static_cast<size_t>(p.rows) * p.scale_pitch;
  asm volatile("griddepcontrol.launch_dependents;");
  for (int64_t t0 = static_cast<int64_t>(blockIdx.y) * height; t0 < p.rows; t0 += step) {
    const int64_t t = t0 + (threadIdx.x >> p.lanes_log2);
    int64_t from = t < p.rows ? t : -1;
    if (p.index && t < p.rows) {
      const int32_t i = __ldg(p.index + t);
      from = i < 0 ? -1 : static_cast<int64_t>(static_cast<uint32_t>(i) / p.per);
      if (from >= p.src_rows) from = -1;
    }
    V x;
    x.load(static_cast<const E *>(p.x) + (from >= 0 ? from : 0) * p.ld, c, p.cols, from >= 0);
    x.settle(stage);
    uint32_t top = top_of<DT>(x.v);
#pragma unroll
    for (int o = 1; o < kBlock / 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t sb = scale_byte(top);
    uint2 v = eight_e4m3(x, up_of(sb));
    if (sb == 255 && c + 8 > p.cols) {  // behind the row lie zeros, in a NaN block too
      uint8_t *b = reinterpret_cast<uint8_t *>(&v);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e >= p.cols) b[e] = 0;
    }
    if (t < p.rows && c < p.pitch) put(p.q + t * p.pitch + c, v, p.q, qsize, p.status);
    if (t < p.rows && c % kBlock == 0 && c / kBlock < p.scale_pitch)
      put(p.s + t * p.scale_pitch + c / kBlock, static_cast<uint8_t>(c < p.cols ? sb : 0), p.s, ssize, p.status);
  }
}

// One CTA per 128 x 128 block: thread i holds columns (i % 16) * 8.. of rows i / 16 + 16 k.
template <int DT, bool WIDE>
__global__ void __launch_bounds__(kThreads) ns_blocks_store_tiles_kernel(const __grid_constant__ BlocksParams p) {
  using E = typename Elem<DT>::T;
  __shared__ uint32_t tops[kThreads / 32];
  const int tiles_x = (p.cols + kBlock - 1) / kBlock;
  const int64_t tiles_y = (p.rows + kBlock - 1) / kBlock;
  const int64_t per = tiles_x * tiles_y, total = per * p.groups;
  const size_t qsize = static_cast<size_t>(p.groups) * p.rows * p.pitch;
  const size_t ssize = static_cast<size_t>(p.groups) * tiles_y * p.scale_pitch;
  for (int64_t i = blockIdx.x; i < total; i += gridDim.x) {
    const int64_t g = i / per, in = i - g * per, ty = in / tiles_x;
    const int tx = static_cast<int>(in - ty * tiles_x);
    const int c = tx * kBlock + static_cast<int>(threadIdx.x % 16) * 8;
    const int64_t r0 = ty * kBlock + threadIdx.x / 16;
    const E *x = static_cast<const E *>(p.x) + (g * p.rows) * p.ld;
    Pack<DT, 8> v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t r = r0 + 16 * k;
      if (WIDE && r < p.rows && c < p.cols) {
        v[k].load_stream(x + r * p.ld + c);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          reinterpret_cast<E *>(v[k].w)[e] = !WIDE && r < p.rows && c + e < p.cols ? __ldcs(x + r * p.ld + c + e) : Elem<DT>::from_f(0.f);
      }
    }
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, top_of<DT>(v[k]));
    top = __reduce_max_sync(0xffffffffu, top);
    __syncthreads();  // the last block's have been read
    if (threadIdx.x % 32 == 0) tops[threadIdx.x / 32] = top;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) top = max(top, tops[k]);
    const uint32_t sb = scale_byte(top);
    const float up = up_of(sb);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int64_t r = r0 + 16 * k;
      if (r >= p.rows || c >= p.pitch) continue;
      uint2 w = eight_e4m3(v[k], up);
      if (sb == 255 && c + 8 > p.cols) {
        uint8_t *b = reinterpret_cast<uint8_t *>(&w);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e >= p.cols) b[e] = 0;
      }
      put(p.q + (g * p.rows + r) * p.pitch + c, w, p.q, qsize, p.status);
    }
    // the row of scales up to its pitch: the last block of a row also writes the zeros behind it
    const int last = tx + 1 == tiles_x ? p.scale_pitch : tx + 1;
    if (tx + static_cast<int>(threadIdx.x) < last)
      put(p.s + (g * tiles_y + ty) * p.scale_pitch + tx + threadIdx.x, static_cast<uint8_t>(threadIdx.x == 0 ? sb : 0), p.s,
          ssize, p.status);
  }
}

// Row of scales that belongs to row t of all.
__device__ __forceinline__ int64_t scale_row(const BlocksParams &p, int64_t t, int64_t bands) {
  if (!p.tiles) return t;
  if (p.groups == 1) return t / kBlock;
  const int64_t g = t / p.rows;
  return g * bands + (t - g * p.rows) / kBlock;
}
template <int DT>
__device__ __forceinline__ void eight_values(uint2 w, float unit, Pack<DT, 8> &v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    from_e4m3x2((i < 2 ? w.x : w.y) >> (16 * (i % 2)), a, b);
    const float2 f = __fmul2_rn(make_float2(a, b), make_float2(unit, unit));
    v.set(2 * i, f.x);
    v.set(2 * i + 1, f.y);
  }
}

// Rows that allow packs: 16 columns a lane.
template <int DT>
__global__ void __launch_bounds__(kThreads) ns_blocks_load_kernel(const __grid_constant__ BlocksParams p) {
  using E = typename Elem<DT>::T;
  const int c = ((blockIdx.x << p.lanes_log2) + (threadIdx.x & ((1 << p.lanes_log2) - 1))) * 16;
  const int height = kThreads >> p.lanes_log2;
  const int64_t step = static_cast<int64_t>(gridDim.y) * height, all = p.rows * p.groups;
  const int64_t bands = (p.rows + kBlock - 1) / kBlock;
  const size_t size = static_cast<size_t>((all - 1) * p.ld + p.cols) * sizeof(E);
  if (c >= p.cols) return;
  for (int64_t t = static_cast<int64_t>(blockIdx.y) * height + (threadIdx.x >> p.lanes_log2); t < all; t += step) {
    const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(p.q + t * p.pitch + c));
    const float unit = unit_of(p.s[scale_row(p, t, bands) * p.scale_pitch + c / kBlock]);
    E *to = static_cast<E *>(p.out) + t * p.ld + c;
    Pack<DT, 8> v;
    eight_values<DT>(make_uint2(w.x, w.y), unit, v);
    v.store_stream(to, p.out, size, p.status);
    if (c + 8 < p.cols) {
      eight_values<DT>(make_uint2(w.z, w.w), unit, v);
      v.store_stream(to + 8, p.out, size, p.status);
    }
  }
}

template <int DT>
__global__ void __launch_bounds__(kThreads) ns_blocks_load_any_kernel(const __grid_constant__ BlocksParams p) {
  using E = typename Elem<DT>::T;
  using V = Eight<DT, false>;
  __shared__ uint4 stages[kThreads / 32][V::kStage];
  uint4 *stage = stages[threadIdx.x / 32];
  const int c = ((blockIdx.x << p.lanes_log2) + (threadIdx.x & ((1 << p.lanes_log2) - 1))) * 8;
  const int height = kThreads >> p.lanes_log2;
  const int64_t step = static_cast<int64_t>(gridDim.y) * height, all = p.rows * p.groups;
  const int64_t bands = (p.rows + kBlock - 1) / kBlock;
  const size_t size = static_cast<size_t>((all - 1) * p.ld + p.cols) * sizeof(E);
  for (int64_t t0 = static_cast<int64_t>(blockIdx.y) * height; t0 < all; t0 += step) {
    const int64_t t = t0 + (threadIdx.x >> p.lanes_log2);
    V o;
    if (t < all && c < p.cols)
      eight_values<DT>(__ldcs(reinterpret_cast<const uint2 *>(p.q + t * p.pitch + c)),
                       unit_of(p.s[scale_row(p, t, bands) * p.scale_pitch + c / kBlock]), o.v);
    o.store(static_cast<E *>(p.out) + t * p.ld, c, p.cols, t < all, stage, p.out, size, p.status);
  }
}

template <int DT>
int run_store(BlocksParams &p, bool tiles, bool wide, int sms, cudaStream_t s) {
  if (tiles) {
    const int64_t total = (p.rows + kBlock - 1) / kBlock * ((p.cols + kBlock - 1) / kBlock) * p.groups;
    const unsigned grid = static_cast<unsigned>(std::min<int64_t>(total, static_cast<int64_t>(sms) * 64));
    if (wide)
      ns_blocks_store_tiles_kernel<DT, true><<<grid, kThreads, 0, s>>>(p);
    else
      ns_blocks_store_tiles_kernel<DT, false><<<grid, kThreads, 0, s>>>(p);
  } else {
    const int64_t extent = std::max<int64_t>(p.pitch, static_cast<int64_t>(p.scale_pitch) * kBlock);
    if (wide) {
      const EightGrid g(p.rows, (extent + 1) / 2, kThreads, true, 3, sms, 128);  // 16 columns a lane
      p.lanes_log2 = g.lanes_log2;
      if (p.index)
        ns_blocks_store_rows_kernel<DT, true><<<g.grid, kThreads, 0, s>>>(p);
      else
        ns_blocks_store_rows_kernel<DT, false><<<g.grid, kThreads, 0, s>>>(p);
    } else {
      const EightGrid g(p.rows, extent, kThreads, false, 4, sms, 32);
      p.lanes_log2 = g.lanes_log2;
      ns_blocks_store_any_kernel<DT><<<g.grid, kThreads, 0, s>>>(p);
    }
  }
  count_launch();
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

template <int DT>
int run_load(BlocksParams &p, bool wide, int sms, cudaStream_t s) {
  if (wide) {
    const EightGrid g(p.rows * p.groups, (p.cols + 1) / 2, kThreads, true, 2, sms, 128);
    p.lanes_log2 = g.lanes_log2;
    ns_blocks_load_kernel<DT><<<g.grid, kThreads, 0, s>>>(p);
  } else {
    const EightGrid g(p.rows * p.groups, p.cols, kThreads, false, 5, sms, 32);
    p.lanes_log2 = g.lanes_log2;
    ns_blocks_load_any_kernel<DT><<<g.grid, kThreads, 0, s>>>(p);
  }
  count_launch();
  return cudaGetLastError() == cudaSuccess ? 0 : -1;
}

bool bad_dtype(int dtype) { return dtype != NS_F32 && dtype != NS_BF16; }

}  // namespace
}  // namespace ns

using namespace ns;

extern "C" int64_t ns_blocks_pitch(int64_t cols) { return cols < 0 ? -1 : (cols + 15) / 16 * 16; }
extern "C" int64_t ns_blocks_scale_pitch(int64_t cols) { return cols < 0 ? -1 : ((cols + 127) / 128 + 3) / 4 * 4; }

extern "C" int ns_blocks_store_rows(const void *x, int64_t ld_x, int64_t x_rows, const int32_t *index, int per,
                                    int64_t rows, int64_t cols, void *q, void *scales, int dtype, void *stream) {
  if (bad_dtype(dtype) || bad_shape(x_rows, cols, ld_x) || bad_shape(rows, cols, cols) || cols > kMaxRowCols || rows > (1 << 30) ||
      x_rows > (1 << 30) || per < 1)
    return NS_EINVAL;
  if (rows == 0 || cols == 0) return NS_OK;
  if (!index && (rows != x_rows || per != 1)) return NS_EINVAL;
  if ((!x && x_rows > 0) || !q || !scales) return NS_EINVAL;
  const int elt = dtype == NS_BF16 ? 2 : 4;
  if (misaligned(x, elt) || misaligned(index, 4) || misaligned(q, 16) || misaligned(scales, 16)) return NS_EALIGN;
  BlocksParams p{};
  p.pitch = static_cast<int>(ns_blocks_pitch(cols));
  p.scale_pitch = static_cast<int>(ns_blocks_scale_pitch(cols));
  const Range rx(x, x_rows, cols, ld_x, elt), ri(index, 1, rows, rows, 4);
  const Range rq(q, rows, p.pitch, p.pitch, 1), rs(scales, rows, p.scale_pitch, p.scale_pitch, 1);
  if (rq.overlaps(rx) || rs.overlaps(rx) || rq.overlaps(rs) || rq.overlaps(ri) || rs.overlaps(ri)) return NS_EINVAL;
  OpCall call(stream);
  if (call.rc) return call.rc;
  p.x = x;
  p.ld = ld_x;
  p.rows = rows;
  p.src_rows = x_rows;
  p.index = index;
  p.per = static_cast<uint32_t>(per);
  while ((uint64_t(1) << p.per_shift) < p.per) ++p.per_shift;
  p.per_mul = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << p.per_shift) - p.per)) / p.per + 1);
  p.q = static_cast<uint8_t *>(q);
  p.s = static_cast<uint8_t *>(scales);
  p.cols = static_cast<int>(cols);
  p.groups = 1;
  p.status = call.status;
  const bool wide = cols % 8 == 0 && rows_aligned(x, ld_x, elt, 8);
  return call.launch(kOpBlocks, [&] {
    return dtype == NS_BF16 ? run_store<kBF16>(p, false, wide, call.sms, call.s) : run_store<kF32>(p, false, wide, call.sms, call.s);
  });
}

extern "C" int ns_blocks_store_tiles(const void *x, int64_t ld_x, int groups, int64_t rows, int64_t cols, void *q,
                                     void *scales, int dtype, void *stream) {
  if (bad_dtype(dtype) || groups < 0 || bad_shape(rows, cols, ld_x) || cols > kMaxRowCols ||
      (groups > 0 && bad_shape(static_cast<int64_t>(groups) * rows, cols, ld_x)))
    return NS_EINVAL;
  if (groups == 0 || rows == 0 || cols == 0) return NS_OK;
  if (!x || !q || !scales) return NS_EINVAL;
  const int elt = dtype == NS_BF16 ? 2 : 4;
  if (misaligned(x, elt) || misaligned(q, 16) || misaligned(scales, 16)) return NS_EALIGN;
  BlocksParams p{};
  p.pitch = static_cast<int>(ns_blocks_pitch(cols));
  p.scale_pitch = static_cast<int>(ns_blocks_scale_pitch(cols));
  const int64_t all = static_cast<int64_t>(groups) * rows, bands = static_cast<int64_t>(groups) * ((rows + kBlock - 1) / kBlock);
  const Range rx(x, all, cols, ld_x, elt), rq(q, all, p.pitch, p.pitch, 1), rs(scales, bands, p.scale_pitch, p.scale_pitch, 1);
  if (rq.overlaps(rx) || rs.overlaps(rx) || rq.overlaps(rs)) return NS_EINVAL;
  OpCall call(stream);
  if (call.rc) return call.rc;
  p.x = x;
  p.ld = ld_x;
  p.rows = rows;
  p.q = static_cast<uint8_t *>(q);
  p.s = static_cast<uint8_t *>(scales);
  p.cols = static_cast<int>(cols);
  p.groups = groups;
  p.status = call.status;
  const bool wide = cols % 8 == 0 && rows_aligned(x, ld_x, elt, 8);
  return call.launch(kOpBlocks, [&] {
    return dtype == NS_BF16 ? run_store<kBF16>(p, true, wide, call.sms, call.s) : run_store<kF32>(p, true, wide, call.sms, call.s);
  });
}

extern "C" int ns_blocks_load(const void *q, const void *scales, int tiles, int groups, int64_t rows, int64_t cols,
                              void *out, int64_t ld_out, int dtype, void *stream) {
  if (bad_dtype(dtype) || groups < 0 || (tiles != 0 && tiles != 1) || (!tiles && groups != 1) ||
      bad_shape(rows, cols, ld_out) || cols > kMaxRowCols ||
      (groups > 0 && bad_shape(static_cast<int64_t>(groups) * rows, cols, ld_out)))
    return NS_EINVAL;
  if (groups == 0 || rows == 0 || cols == 0) return NS_OK;
  if (!out || !q || !scales) return NS_EINVAL;
  const int elt = dtype == NS_BF16 ? 2 : 4;
  if (misaligned(out, elt) || misaligned(q, 16) || misaligned(scales, 16)) return NS_EALIGN;
  BlocksParams p{};
  p.pitch = static_cast<int>(ns_blocks_pitch(cols));
  p.scale_pitch = static_cast<int>(ns_blocks_scale_pitch(cols));
  const int64_t all = static_cast<int64_t>(groups) * rows;
  const int64_t bands = tiles ? static_cast<int64_t>(groups) * ((rows + kBlock - 1) / kBlock) : all;
  const Range ro(out, all, cols, ld_out, elt);
  if (ro.overlaps(Range(q, all, p.pitch, p.pitch, 1)) || ro.overlaps(Range(scales, bands, p.scale_pitch, p.scale_pitch, 1)))
    return NS_EINVAL;
  OpCall call(stream);
  if (call.rc) return call.rc;
  p.out = out;
  p.ld = ld_out;
  p.rows = rows;
  p.q = static_cast<uint8_t *>(const_cast<void *>(q));
  p.s = static_cast<uint8_t *>(const_cast<void *>(scales));
  p.cols = static_cast<int>(cols);
  p.groups = groups;
  p.tiles = tiles;
  p.status = call.status;
  const bool wide = cols % 8 == 0 && rows_aligned(out, ld_out, elt, 8);
  return call.launch(kOpBlocks, [&] {
    return dtype == NS_BF16 ? run_load<kBF16>(p, wide, call.sms, call.s) : run_load<kF32>(p, wide, call.sms, call.s);
  });
}
