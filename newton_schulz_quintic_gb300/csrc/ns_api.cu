// ns_api.cu -- C ABI of libns (include/ns.h) and its host planner.
//
// The planner validates the batch, decides per matrix between the
// shared-memory resident kernel (small m) and the GEMM path, orders the
// GEMM-path matrices by Newton-Schulz cost max(M,N)*min(M,N)^2 (largest
// first, the ordering rule of the second page's "Changes" items 1-2), lays out
// one device workspace, builds the per-phase tile lists and TMA descriptors,
// uploads them, and launches:
//   resident kernel (all small matrices at once)
//   bf16: tile norms -> norm finish -> steps x { gram -> square -> apply }
//   fp32: norm -> prep -> steps x { gram -> square -> apply }  (all large matrices)
// The megabatch of the first page's "Concrete repro" is just `count`
// matrices of one shape; remainder batches (the xtuner PR's ragged
// all-to-all commit) are calls with a smaller `count`, so no zero matrix is
// ever orthogonalised.
#include <cuda.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <cstring>
#include <map>
#include <memory>
#include <mutex>
#include <vector>

#include "../../include/ns.h"
#include "ns_internal.h"

namespace ns {

static std::atomic<int64_t> g_launches{0};
void count_launch() { g_launches.fetch_add(1, std::memory_order_relaxed); }
static std::atomic<int64_t> g_allocations{0};
// Largest workspace the library's cache may hold per (device, stream, slot);
// 0 = no limit (ns_set_workspace_limit).
static std::atomic<size_t> g_ws_limit{0};

int SmemOptIn::ensure(const void *kernel, int bytes) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  int &have = allowed[dev & 63];
  if (bytes <= have) return 0;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  have = bytes;
  return 0;
}

// Device status word (one per device, file-scope; see ns_get_status) and the
// flag the wait self-test reports through.
__device__ int g_status_word;
__device__ int g_probe_word;

namespace {

constexpr float kDefaultCoeffs[3] = {3.4445f, -4.7750f, 2.0315f};
constexpr int kResidentMaxM = 64;
#ifndef NS_RASTER_GROUP
#define NS_RASTER_GROUP 8
#endif
constexpr int kRasterGroup = NS_RASTER_GROUP;  // tile rows per rasterisation group
constexpr int kResidentSmemMax = 200 * 1024;
constexpr size_t kAlign = 1024;

size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
int64_t round8(int64_t v) { return (v + 7) / 8 * 8; }

// ------------------------------------------------------------ device info
struct DevInfo {
  bool ok = false;
  int sms = 0;
  int *status = nullptr;
  int *probe = nullptr;
};
std::mutex g_mu;
std::map<int, DevInfo> g_dev;

// cudaGetDevice, with "no CUDA driver or device" reported as NS_ENODEV and
// any other failure as NS_ECUDA
int current_device(int *dev) {
  const cudaError_t e = cudaGetDevice(dev);
  if (e == cudaSuccess) return NS_OK;
  cudaGetLastError();
  return e == cudaErrorNoDevice || e == cudaErrorInsufficientDriver ? NS_ENODEV : NS_ECUDA;
}

int device_info(DevInfo **out) {
  int dev = 0;
  if (const int rc = current_device(&dev)) return rc;
  auto it = g_dev.find(dev);
  if (it == g_dev.end()) {
    DevInfo di;
    cudaDeviceProp prop;
    if (cudaGetDeviceProperties(&prop, dev) != cudaSuccess) return NS_ECUDA;
    di.ok = prop.major == 10;  // sm_100 family (sm_103a is what this library is built for)
    di.sms = prop.multiProcessorCount;
    void *sym = nullptr;
    if (cudaGetSymbolAddress(&sym, g_status_word) != cudaSuccess) return NS_ECUDA;
    di.status = static_cast<int *>(sym);
    if (cudaGetSymbolAddress(&sym, g_probe_word) != cudaSuccess) return NS_ECUDA;
    di.probe = static_cast<int *>(sym);
    it = g_dev.emplace(dev, di).first;
  }
  *out = &it->second;
  return it->second.ok ? NS_OK : NS_ENODEV;
}

// ------------------------------------------------------------ TMA encode
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn g_encode = nullptr;

int get_encode() {
  if (g_encode) return NS_OK;
  void *fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) !=
          cudaSuccess ||
      q != cudaDriverEntryPointSuccess || !fn)
    return NS_ECUDA;
  g_encode = reinterpret_cast<EncodeFn>(fn);
  return NS_OK;
}

// bf16 row-major rows x cols matrix with a pitch of `pitch` elements; box
// {64 columns, box_rows rows} with 128-byte swizzle; out-of-range reads give 0.
int encode_bf16(CUtensorMap *map, void *base, int64_t rows, int64_t cols, int64_t pitch, int box_rows) {
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(std::max<int64_t>(cols, 1)),
                        static_cast<cuuint64_t>(std::max<int64_t>(rows, 1))};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch * 2)};
  cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? NS_OK : NS_ECUDA;
}

// The three bf16 slices of a rows x cols tensor (fp32 path), `slice` elements
// apart, as one 3-D map whose third coordinate is the slice; boxes
// {64 columns, box_rows rows, 1 slice} with 128-byte swizzle.
int encode_bf16_sliced(CUtensorMap *map, void *base, int64_t rows, int64_t cols, int64_t pitch, int64_t slice,
                       int box_rows) {
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(std::max<int64_t>(cols, 1)),
                        static_cast<cuuint64_t>(std::max<int64_t>(rows, 1)), 3};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(pitch * 2), static_cast<cuuint64_t>(slice * 2)};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? NS_OK : NS_ECUDA;
}

int encode_iterate_sliced(CUtensorMap *kmajor, CUtensorMap *mnmajor, void *base, int64_t rows, int64_t cols,
                          int64_t pitch) {
  const int64_t slice = rows * pitch;
  int rc = encode_bf16_sliced(kmajor, base, rows, cols, pitch, slice, kTcBM);
  return rc ? rc : encode_bf16_sliced(mnmajor, base, rows, cols, pitch, slice, 64);
}

// The two maps of one tensor read both ways: K-major box {64, 128}, MN-major box {64, 64}.
int encode_iterate(CUtensorMap *kmajor, CUtensorMap *mnmajor, void *base, int64_t rows, int64_t cols,
                   int64_t pitch) {
  int rc = encode_bf16(kmajor, base, rows, cols, pitch, kTcBM);
  return rc ? rc : encode_bf16(mnmajor, base, rows, cols, pitch, 64);
}

// ------------------------------------------------------------ layout
struct BigMat {
  int index;  // caller index
  int64_t M, N, m, n, pm, pn;
  int transposed;
  int t01, t2;  // tiles of this matrix in the gram/square list and in the apply list
  int64_t ps;   // bf16 path: pitch of the iterate buffers (caller's orientation)
  size_t off_x, off_xt0, off_xt1, off_s0, off_s1, off_a, off_b;
};

// Resident matrices of one cluster size: entries [start, start + count) of
// the resident descriptor table, one launch.
struct ResGroup {
  int cluster, start, count, smem;
};

struct Layout {
  int dtype = 0;
  int elt = 2;
  bool split = false;        // fp32 on the tensor cores (three bf16 slices per tensor)
  bool tc() const { return dtype == NS_BF16 || split; }
  std::vector<BigMat> big;   // cost order
  std::vector<int> res;      // caller indices on the resident path, grouped by cluster size
  std::vector<int> res_ns;   // their slice widths
  std::vector<ResGroup> res_groups;
  std::vector<Tile> tiles01, tiles2;
  std::vector<int> prefix;   // prep tile prefix, big.size()+1
  size_t off_mats = 0, off_res = 0, off_t01 = 0, off_t2 = 0, off_prefix = 0, blob_end = 0;
  size_t off_partials = 0, off_tilepart = 0, off_tileext = 0, off_rscale = 0, off_ext = 0, off_done = 0,
         off_buffers = 0, total = 0;
};

int validate(void *const *X, const int64_t *shapes, int count, int steps, int dtype, bool check_ptrs) {
  if (count < 0 || steps < 0) return NS_EINVAL;
  if (dtype != NS_F32 && dtype != NS_BF16) return NS_EINVAL;
  if (count == 0) return NS_OK;
  if (!shapes || (check_ptrs && !X)) return NS_EINVAL;
  const size_t elt = dtype == NS_BF16 ? 2 : 4;
  for (int i = 0; i < count; ++i) {
    const int64_t M = shapes[2 * i], N = shapes[2 * i + 1];
    if (M < 0 || N < 0) return NS_EINVAL;
    if (M > INT32_MAX / 2 || N > INT32_MAX / 2) return NS_EINVAL;
    if (M * N > (int64_t(1) << 40)) return NS_EINVAL;
    if (check_ptrs && M * N > 0) {
      if (!X[i]) return NS_EINVAL;
      if (reinterpret_cast<uintptr_t>(X[i]) % elt) return NS_EALIGN;
    }
  }
  if (check_ptrs) {
    // matrices must not overlap: the last step of one writes its matrix in
    // place while another may still be reading its own
    std::vector<std::pair<uintptr_t, uintptr_t>> r;
    r.reserve(count);
    for (int i = 0; i < count; ++i) {
      const int64_t M = shapes[2 * i], N = shapes[2 * i + 1];
      if (M * N == 0) continue;
      const uintptr_t b = reinterpret_cast<uintptr_t>(X[i]);
      r.emplace_back(b, b + static_cast<uintptr_t>(M * N) * elt);
    }
    std::sort(r.begin(), r.end());
    for (size_t k = 1; k < r.size(); ++k)
      if (r[k].first < r[k - 1].second) return NS_EINVAL;
  }
  return NS_OK;
}

// Whether a small matrix takes the shared-memory resident path: m <= 64 and
// the whole matrix, with its m x m products, would fit one CTA's shared memory.
bool resident_fits(int64_t m, int64_t n, int dtype) {
  if (m > kResidentMaxM) return false;
  const int64_t elt = dtype == NS_BF16 ? 2 : 4;
  const int64_t mp = (m + 3) / 4 * 4, np = (n + 3) / 4 * 4;
  return mp * np * elt + 2 * mp * (mp + 1) * 4 + 16 * 1024 <= kResidentSmemMax;
}

// Large fp32 matrices: the tensor-core path (three bf16 slices per tensor,
// six slice products per GEMM) by default, or the CUDA-core GEMMs
// (ns_set_f32_gemm). The tensor cores' accumulation error grows with the
// contraction length (max(M, N) in gram); past kF32TensorMaxK a call runs on
// the CUDA cores, whose fp32 FMAs round to nearest.
std::atomic<int> g_f32_gemm{NS_F32_TENSOR};
constexpr int64_t kF32TensorMaxK = 16384;

void build_layout(const int64_t *shapes, int count, int dtype, Layout &L) {
  L = Layout();
  L.dtype = dtype;
  L.elt = dtype == NS_BF16 ? 2 : 4;
  L.split = dtype == NS_F32 && g_f32_gemm.load() == NS_F32_TENSOR;
  std::vector<int> order;
  std::vector<int> res_cluster;  // indexed by caller index
  for (int i = 0; i < count; ++i) {
    const int64_t M = shapes[2 * i], N = shapes[2 * i + 1];
    if (M == 0 || N == 0) continue;
    const int64_t m = std::min(M, N), n = std::max(M, N);
    bool res = resident_fits(m, n, dtype);
    if (res) {  // and one CTA's slice of it fits as laid out
      const int c = resident_cluster(static_cast<int>(m), static_cast<int>(n));
      res = resident_smem_bytes(static_cast<int>(m), resident_slice(static_cast<int>(n), c), dtype, c) <=
            kResidentSmemMax;
    }
    if (res)
      L.res.push_back(i);
    else
      order.push_back(i);
  }
  // resident matrices: one launch per cluster size (largest first), each
  // matrix's cluster size from its own shape
  auto cl = [&](int i) {
    const int64_t M = shapes[2 * i], N = shapes[2 * i + 1];
    return resident_cluster(static_cast<int>(std::min(M, N)), static_cast<int>(std::max(M, N)));
  };
  std::stable_sort(L.res.begin(), L.res.end(), [&](int a, int b) { return cl(a) > cl(b); });
  for (size_t k = 0; k < L.res.size(); ++k) {
    const int i = L.res[k];
    const int64_t M = shapes[2 * i], N = shapes[2 * i + 1];
    const int m = static_cast<int>(std::min(M, N)), n = static_cast<int>(std::max(M, N));
    const int c = cl(i), ns = resident_slice(n, c);
    L.res_ns.push_back(ns);
    if (L.res_groups.empty() || L.res_groups.back().cluster != c)
      L.res_groups.push_back(ResGroup{c, static_cast<int>(k), 0, 0});
    ResGroup &g = L.res_groups.back();
    ++g.count;
    g.smem = std::max(g.smem, resident_smem_bytes(m, ns, dtype, c));
  }
  if (L.split)
    for (int i : order)
      if (std::max(shapes[2 * i], shapes[2 * i + 1]) > kF32TensorMaxK) L.split = false;
  // largest Newton-Schulz cost first; ties keep the caller's order
  std::stable_sort(order.begin(), order.end(), [&](int a, int b) {
    return ns_cost(shapes[2 * a], shapes[2 * a + 1]) > ns_cost(shapes[2 * b], shapes[2 * b + 1]);
  });
  const int BM = L.tc() ? kTcPairM : kSimtBM;  // tensor cores: rows of one CTA pair
  const int BN = L.tc() ? kTcBN : kSimtBN;
  L.prefix.push_back(0);
  for (int idx : order) {
    BigMat b{};
    b.index = idx;
    b.M = shapes[2 * idx];
    b.N = shapes[2 * idx + 1];
    b.transposed = b.M > b.N;
    b.m = std::min(b.M, b.N);
    b.n = std::max(b.M, b.N);
    b.pm = round8(b.m);
    b.pn = round8(b.n);
    b.ps = round8(b.N);
    const int mi = static_cast<int>(L.big.size());
    // Tiles in groups of kRasterGroup tile rows: within a group, column by
    // column, so the tiles in flight at once share a few operand row blocks
    // of each side and the working set stays in L2.
    const size_t n01_before = L.tiles01.size(), n2_before = L.tiles2.size();
    const int64_t gstep = static_cast<int64_t>(kRasterGroup) * BM;
    // gram / square: tiles with some column index >= some row index
    for (int64_t g0 = 0; g0 < b.m; g0 += gstep)
      for (int64_t c0 = 0; c0 < b.m; c0 += BN)
        for (int64_t r0 = g0; r0 < std::min(b.m, g0 + gstep); r0 += BM)
          if (c0 + BN > r0) L.tiles01.push_back(Tile{mi, static_cast<int>(r0), static_cast<int>(c0), 0});
    // apply: tensor cores, tiles of the next iterate in the caller's
    // orientation (M x N); CUDA cores, tiles of W'^T (n x m)
    const int64_t arows = L.tc() ? b.M : b.n, acols = L.tc() ? b.N : b.m;
    for (int64_t g0 = 0; g0 < arows; g0 += gstep)
      for (int64_t c0 = 0; c0 < acols; c0 += BN)
        for (int64_t r0 = g0; r0 < std::min(arows, g0 + gstep); r0 += BM)
          L.tiles2.push_back(Tile{mi, static_cast<int>(r0), static_cast<int>(c0), 0});
    b.t01 = static_cast<int>(L.tiles01.size() - n01_before);
    b.t2 = static_cast<int>(L.tiles2.size() - n2_before);
    const int64_t pt = ((b.M + kPrepTile - 1) / kPrepTile) * ((b.N + kPrepTile - 1) / kPrepTile);
    L.prefix.push_back(L.prefix.back() + static_cast<int>(pt));
    L.big.push_back(b);
  }
  size_t off = 0;
  L.off_mats = off;
  off = align_up(off + L.big.size() * sizeof(MatDesc), kAlign);
  L.off_res = off;
  off = align_up(off + L.res.size() * sizeof(ResDesc), 256);
  L.off_t01 = off;
  off = align_up(off + L.tiles01.size() * sizeof(Tile), 256);
  L.off_t2 = off;
  off = align_up(off + L.tiles2.size() * sizeof(Tile), 256);
  L.off_prefix = off;
  off = align_up(off + L.prefix.size() * sizeof(int), 256);
  L.blob_end = off;
  L.off_partials = off;
  off = align_up(off + L.big.size() * kNormBlocks * sizeof(float), 256);
  L.off_tilepart = off;
  off = align_up(off + static_cast<size_t>(L.prefix.back()) * sizeof(float), 256);
  L.off_tileext = off;
  off = align_up(off + static_cast<size_t>(L.prefix.back()) * 2 * sizeof(int), 256);
  L.off_rscale = off;
  off = align_up(off + L.big.size() * sizeof(float), 256);
  L.off_ext = off;
  off = align_up(off + L.big.size() * 2 * sizeof(int), 256);
  L.off_done = off;  // per matrix completion counters, then the ticket counter
  off = align_up(off + (L.big.size() + 1) * sizeof(int), kAlign);
  L.off_buffers = off;
  for (BigMat &b : L.big) {
    if (L.split) {  // iterates, A and B as three bf16 slices each
      b.off_s0 = off;
      off = align_up(off + 3 * static_cast<size_t>(b.M * b.ps) * 2, kAlign);
      b.off_s1 = off;
      off = align_up(off + 3 * static_cast<size_t>(b.M * b.ps) * 2, kAlign);
      b.off_a = off;
      off = align_up(off + 3 * static_cast<size_t>(b.m * b.pm) * 2, kAlign);
      b.off_b = off;
      off = align_up(off + 3 * static_cast<size_t>(b.m * b.pm) * 2, kAlign);
      continue;
    }
    if (dtype == NS_BF16) {  // two iterate buffers in the caller's orientation
      b.off_s0 = off;
      off = align_up(off + static_cast<size_t>(b.M * b.ps) * L.elt, kAlign);
      b.off_s1 = off;
      off = align_up(off + static_cast<size_t>(b.M * b.ps) * L.elt, kAlign);
    } else {  // W and two W^T buffers
      b.off_x = off;
      off = align_up(off + static_cast<size_t>(b.m * b.pn) * L.elt, kAlign);
      b.off_xt0 = off;
      off = align_up(off + static_cast<size_t>(b.n * b.pm) * L.elt, kAlign);
      b.off_xt1 = off;
      off = align_up(off + static_cast<size_t>(b.n * b.pm) * L.elt, kAlign);
    }
    b.off_a = off;
    off = align_up(off + static_cast<size_t>(b.m * b.pm) * L.elt, kAlign);
    b.off_b = off;
    off = align_up(off + static_cast<size_t>(b.m * b.pm) * L.elt, kAlign);
  }
  L.total = std::max<size_t>(off, 256);
}

// Step 0 of the bf16 path reads the caller's Y through TMA when its base and
// row pitch are 16-byte aligned, and when a later step (not step 0 itself)
// is the one that overwrites it.
bool reads_y_directly(const void *y, int64_t N, int steps) {
  return steps >= 2 && (reinterpret_cast<uintptr_t>(y) & 15) == 0 && (N * 2) % 16 == 0;
}

int build_blob(const Layout &L, void *const *X, const int64_t *shapes, int steps, uint8_t *ws,
               std::vector<uint8_t> &blob) {
  blob.assign(L.blob_end, 0);
  if (L.tc() && !L.big.empty()) {
    int rc = get_encode();
    if (rc) return rc;
  }
  uint8_t *mats = blob.data() + L.off_mats;  // host bytes; copied, never dereferenced as MatDesc
  for (size_t k = 0; k < L.big.size(); ++k) {
    const BigMat &b = L.big[k];
    MatDesc d;
    std::memset(&d, 0, sizeof(d));
    if (L.tc()) {
      d.s[0] = ws + b.off_s0;
      d.s[1] = ws + b.off_s1;
    } else {
      d.x = ws + b.off_x;
      d.xt[0] = ws + b.off_xt0;
      d.xt[1] = ws + b.off_xt1;
    }
    d.a = ws + b.off_a;
    d.b = ws + b.off_b;
    d.user = X[b.index];
    d.M = static_cast<int>(b.M);
    d.N = static_cast<int>(b.N);
    d.m = static_cast<int>(b.m);
    d.n = static_cast<int>(b.n);
    d.pm = static_cast<int>(b.pm);
    d.pn = static_cast<int>(b.pn);
    d.ps = static_cast<int>(b.ps);
    d.transposed = b.transposed;
    d.index = b.index;
    d.t01 = b.t01;
    d.t2 = b.t2;
    if (L.split) {  // step 0 reads s[0], which the preparation fills
      int rc = encode_iterate_sliced(&d.tm_a, &d.tm_a_mn, d.a, b.m, b.m, b.pm);
      rc = rc ? rc : encode_iterate_sliced(&d.tm_b, &d.tm_b_mn, d.b, b.m, b.m, b.pm);
      rc = rc ? rc : encode_iterate_sliced(&d.tm_s[0], &d.tm_s_mn[0], d.s[0], b.M, b.N, b.ps);
      rc = rc ? rc : encode_iterate_sliced(&d.tm_s[1], &d.tm_s_mn[1], d.s[1], b.M, b.N, b.ps);
      if (rc) return rc;
    } else if (L.dtype == NS_BF16) {
      d.direct = reads_y_directly(d.user, b.N, steps);
      int rc = encode_iterate(&d.tm_a, &d.tm_a_mn, d.a, b.m, b.m, b.pm);
      rc = rc ? rc : encode_iterate(&d.tm_b, &d.tm_b_mn, d.b, b.m, b.m, b.pm);
      rc = rc ? rc : encode_iterate(&d.tm_s[0], &d.tm_s_mn[0], d.s[0], b.M, b.N, b.ps);
      rc = rc ? rc : encode_iterate(&d.tm_s[1], &d.tm_s_mn[1], d.s[1], b.M, b.N, b.ps);
      if (!rc && d.direct) rc = encode_iterate(&d.tm_y, &d.tm_y_mn, d.user, b.M, b.N, b.N);
      if (rc) return rc;
    }
    std::memcpy(mats + k * sizeof(MatDesc), &d, sizeof(d));
  }
  uint8_t *res = blob.data() + L.off_res;
  for (size_t k = 0; k < L.res.size(); ++k) {
    const int i = L.res[k];
    ResDesc r{};
    r.user = X[i];
    r.M = static_cast<int>(shapes[2 * i]);
    r.N = static_cast<int>(shapes[2 * i + 1]);
    r.transposed = r.M > r.N;
    r.m = std::min(r.M, r.N);
    r.n = std::max(r.M, r.N);
    r.ns = L.res_ns[k];
    std::memcpy(res + k * sizeof(ResDesc), &r, sizeof(r));
  }
  if (!L.tiles01.empty())
    std::memcpy(blob.data() + L.off_t01, L.tiles01.data(), L.tiles01.size() * sizeof(Tile));
  if (!L.tiles2.empty()) std::memcpy(blob.data() + L.off_t2, L.tiles2.data(), L.tiles2.size() * sizeof(Tile));
  std::memcpy(blob.data() + L.off_prefix, L.prefix.data(), L.prefix.size() * sizeof(int));
  return NS_OK;
}

// Everything a call's plan and descriptor table depend on besides the
// workspace: the matrices' pointers and shapes, the step count (step 0 may
// read Y itself), the data type and the fp32 GEMM mode.
std::vector<int64_t> call_key(void *const *X, const int64_t *shapes, int count, int steps, int dtype) {
  std::vector<int64_t> k;
  k.reserve(4 + 3 * static_cast<size_t>(count));
  k.push_back(count);
  k.push_back(steps);
  k.push_back(dtype);
  k.push_back(g_f32_gemm.load());
  for (int i = 0; i < count; ++i) {
    k.push_back(static_cast<int64_t>(reinterpret_cast<uintptr_t>(X[i])));
    k.push_back(shapes[2 * i]);
    k.push_back(shapes[2 * i + 1]);
  }
  return k;
}

// ------------------------------------------------------------ workspace cache
// A descriptor table (matrix descriptors with their TMA maps, tile lists)
// resident on the device, and the host bytes it was uploaded from.
struct DevBlob {
  uint8_t *ptr = nullptr;
  std::vector<uint8_t> bytes;
  uint64_t last_use = 0;
  // the call it was last planned for (call_key) and that plan: a repeat of
  // the call reuses both without planning or encoding anything
  std::vector<int64_t> key;
  std::shared_ptr<const Layout> layout;
};
// Tables kept per workspace: a caller that alternates between a few batches
// on one stream (remainder batches, several parameter groups) finds each
// table already on the device, so a call uploads nothing and never waits for
// a staging copy behind the stream's earlier work.
constexpr size_t kBlobsPerWs = 8;

struct CachedWs {
  uint8_t *ptr = nullptr;  // scratch of the largest batch seen (its descriptor-table area unused)
  size_t bytes = 0;
  std::vector<DevBlob> blobs;  // tables whose pointers refer to this scratch
  uint64_t uses = 0;
  // A captured call's graph keeps the addresses of the scratch and of the
  // tables. Once a capture has used this scratch, it and the tables are kept
  // when they are replaced, not freed, until ns_release_workspace.
  bool captured = false;
  std::vector<uint8_t *> kept;
};

bool capturing(cudaStream_t s) {
  cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &st) == cudaSuccess) return st != cudaStreamCaptureStatusNone;
  cudaGetLastError();
  return false;
}

// A block of the cache that no later call uses.
int drop_block(CachedWs &c, uint8_t *p, cudaStream_t s) {
  if (c.captured) {
    c.kept.push_back(p);
    return NS_OK;
  }
  return cudaFreeAsync(p, s) == cudaSuccess ? NS_OK : NS_ECUDA;
}

void drop_blobs(CachedWs &c, cudaStream_t s) {
  for (DevBlob &b : c.blobs) drop_block(c, b.ptr, s);
  c.blobs.clear();
}

// A device block for calls on stream s, its first `fill` bytes copied from
// `from`, or zero where that is nullptr; ordered on s. While s is being
// captured the block is made and filled outside the capture, at once: inside,
// it would be memory that exists only while the graph runs, filled only by it,
// and calls outside the graph use it too.
int new_block(uint8_t **out, size_t bytes, const void *from, size_t fill, cudaStream_t s) {
  g_allocations.fetch_add(1, std::memory_order_relaxed);
  void *p = nullptr;
  auto fill_on = [&](cudaStream_t on) {
    if (fill == 0) return cudaSuccess;
    return from ? cudaMemcpyAsync(p, from, fill, cudaMemcpyHostToDevice, on) : cudaMemsetAsync(p, 0, fill, on);
  };
  int rc = NS_OK;
  if (!capturing(s)) {
    if (cudaMallocAsync(&p, bytes, s) != cudaSuccess) {
      cudaGetLastError();
      return NS_ENOMEM;
    }
    if (fill_on(s) != cudaSuccess) {
      cudaFreeAsync(p, s);
      rc = NS_ECUDA;
    }
  } else {
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return NS_ECUDA;
    cudaStream_t own = nullptr;
    if (cudaMalloc(&p, bytes) != cudaSuccess) {
      cudaGetLastError();
      rc = NS_ENOMEM;
    } else if (fill > 0) {
      if (cudaStreamCreateWithFlags(&own, cudaStreamNonBlocking) != cudaSuccess || fill_on(own) != cudaSuccess ||
          cudaStreamSynchronize(own) != cudaSuccess) {
        cudaFree(p);
        rc = NS_ECUDA;
      }
      if (own) cudaStreamDestroy(own);
    }
    cudaThreadExchangeStreamCaptureMode(&mode);
  }
  if (rc == NS_OK) *out = static_cast<uint8_t *>(p);
  return rc;
}
// keyed by (device, stream, slot): slot 0 serves the device entry points,
// slot 1 holds the host entry point's device copies, slot 2 + g the workspace
// of its g-th pipeline group
struct WsKey {
  int dev;
  cudaStream_t stream;
  unsigned long long id;  // cudaStreamPerThread is one handle for a stream of every thread: which of them; else 0
  int slot;
  bool operator<(const WsKey &o) const {
    if (dev != o.dev) return dev < o.dev;
    if (stream != o.stream) return stream < o.stream;
    if (id != o.id) return id < o.id;
    return slot < o.slot;
  }
};
std::map<WsKey, CachedWs> g_ws;

CachedWs &cached_ws(int dev, cudaStream_t s, int slot) {
  WsKey key{dev, s, 0, slot};
  if (s == cudaStreamPerThread && cudaStreamGetId(s, &key.id) != cudaSuccess) cudaGetLastError();
  return g_ws[key];
}

// The cached scratch grown to `bytes`; its first `zero` bytes are zero when it
// is made.
int ensure_ws(CachedWs &c, size_t bytes, cudaStream_t s, size_t zero = 0) {
  const bool now = capturing(s);
  c.captured = c.captured || now;
  if (c.ptr && c.bytes >= bytes) return NS_OK;
  const size_t limit = g_ws_limit.load();
  if (limit && bytes > limit) return NS_ENOMEM;  // refused before any allocation
  drop_blobs(c, s);  // their descriptors point into the old scratch
  if (c.ptr) {
    if (const int rc = drop_block(c, c.ptr, s)) return rc;
    c.ptr = nullptr;
    c.bytes = 0;
  }
  c.captured = now;
  if (const int rc = new_block(&c.ptr, bytes, nullptr, zero, s)) return rc;
  c.bytes = bytes;
  return NS_OK;
}

// ------------------------------------------------------------ kernel timing
// kinds: 0 norm pass (the read of the caller's matrices), 1 norm finish (bf16:
// per-matrix scale), 2 gram, 3 square, 4 apply, 5 resident, 6 gemm (one
// launch running every step and phase), 7 prep (fp32: the normalising copy),
// 8 momentum (ns_muon_update_batched's element-wise step), 9.. the training
// operators (OpKind in ns_internal.h)
constexpr int kKinds = kOpKindEnd;

// How the tensor-core path is launched (ns_set_gemm_schedule): one launch per
// step and phase (default) or one launch per call with per-matrix counters.
std::atomic<int> g_gemm_schedule{NS_SCHED_PHASE};
bool phase_launches() { return g_gemm_schedule.load() != NS_SCHED_SINGLE; }
struct TimedLaunch {
  int kind;
  cudaEvent_t start, stop;
};
bool g_timing = false;
std::vector<TimedLaunch> g_timed;

// NVTX ranges around every launch and every call (for profilers' timelines),
// off unless ns_set_nvtx(1) or the environment variable NS_NVTX=1.
std::atomic<int> g_nvtx{-1};
bool nvtx_on() {
  int v = g_nvtx.load();
  if (v < 0) {
    const char *e = std::getenv("NS_NVTX");
    v = (e && e[0] == '1') ? 1 : 0;
    g_nvtx.store(v);
  }
  return v != 0;
}
const char *const kKindNames[] = {"ns norm pass", "ns norm finish", "ns gram", "ns square", "ns apply",
                                  "ns resident", "ns gemm (all phases)", "ns prep", "ns momentum",
                                  "ns embed lookup", "ns embed sort", "ns embed grad", "ns policy",
                                  "ns checkpoint", "ns wgrad"};
static_assert(sizeof(kKindNames) / sizeof(kKindNames[0]) == kKinds, "one name per kind");
struct NvtxRange {
  bool on;
  explicit NvtxRange(const char *name) : on(nvtx_on()) {
    if (on) nvtxRangePushA(name);
  }
  ~NvtxRange() {
    if (on) nvtxRangePop();
  }
};

// Launch `fn` bracketed by events when timing is on (and by an NVTX range
// when those are on).
template <typename F>
int timed(int kind, cudaStream_t s, F &&fn) {
  NvtxRange range(kKindNames[kind]);
  if (!g_timing) return fn();
  TimedLaunch t{kind, nullptr, nullptr};
  if (cudaEventCreate(&t.start) != cudaSuccess || cudaEventCreate(&t.stop) != cudaSuccess) return -1;
  cudaEventRecord(t.start, s);
  const int rc = fn();
  cudaEventRecord(t.stop, s);
  g_timed.push_back(t);
  return rc;
}

// ------------------------------------------------------------ execution
// Options of one call that tests use: the limit of the kernels' bounded waits,
// and the dependency-timeout self-test (the single-launch schedule with every
// completion signal held back).
struct RunOpts {
  uint64_t wait_limit_ns = kWaitLimitNs;
  bool hold_signals = false;
  float out_scale = 1.0f;  // the result is multiplied by it before it is written
};

// co: one (a, b, c) triple for every step (table == false) or a steps x 3 table
// ws: the scratch (offsets at and past L.blob_end); blob: the device copy of
// the descriptor table (offsets below L.blob_end), at the front of ws or apart.
int execute(const Layout &L, uint8_t *ws, const uint8_t *blob, int steps, const float *co, bool table, float eps,
            DevInfo *di, cudaStream_t s, const RunOpts &opt) {
  const MatDesc *mats = reinterpret_cast<const MatDesc *>(blob + L.off_mats);
  for (const ResGroup &g : L.res_groups) {
    ResParams rp{};
    rp.mats = reinterpret_cast<const ResDesc *>(blob + L.off_res) + g.start;
    rp.nmats = g.count;
    rp.cluster = g.cluster;
    rp.dtype = L.dtype;
    rp.steps = steps;
    rp.ncoef = table ? steps : 1;
    for (int k = 0; k < (table ? steps : 1); ++k)
      for (int u = 0; u < 3; ++u) rp.coef[k][u] = co[3 * k + u];
    rp.eps = eps;
    rp.out_scale = opt.out_scale;
    rp.status = di->status;
    if (timed(5, s, [&] { return launch_resident(rp, g.smem, s); })) return NS_ECUDA;
  }
  if (L.big.empty()) return NS_OK;
  const int nbig = static_cast<int>(L.big.size());
  int *ext = reinterpret_cast<int *>(ws + L.off_ext);
  int *done = reinterpret_cast<int *>(ws + L.off_done);
  // extents, completion counters and the ticket counter start at zero (they are adjacent)
  if (cudaMemsetAsync(ext, 0, L.off_done + (nbig + 1) * sizeof(int) - L.off_ext, s) != cudaSuccess) return NS_ECUDA;
  PrepParams pp{};
  pp.mats = mats;
  pp.nmats = nbig;
  pp.partials = reinterpret_cast<float *>(ws + L.off_partials);
  pp.ext = ext;
  pp.tile_prefix = reinterpret_cast<const int *>(blob + L.off_prefix);
  pp.eps = eps;
  pp.dtype = L.dtype;
  pp.to_user = steps == 0;
  pp.tile_partials = reinterpret_cast<float *>(ws + L.off_tilepart);
  pp.tile_ext = reinterpret_cast<int *>(ws + L.off_tileext);
  pp.rscale = reinterpret_cast<float *>(ws + L.off_rscale);
  pp.out_scale = opt.out_scale;
  pp.status = di->status;
  // bf16 with steps: one pass sums Y (and copies it unscaled into the first
  // iterate buffer where step 0 cannot read Y itself); the first step's
  // epilogues apply 1/(||Y|| + eps). Otherwise: norm, then a scaled copy.
  const bool fused = L.dtype == NS_BF16 && steps > 0;
  if (fused) {
    if (timed(0, s, [&] { return launch_norm_tiles(pp, L.prefix.back(), 2 * di->sms, s); })) return NS_ECUDA;
    if (timed(1, s, [&] { return launch_norm_finish(pp, s); })) return NS_ECUDA;
  } else if (L.split && steps > 0) {  // fp32 on the tensor cores: the slices of Y / (||Y|| + eps) into s[0]
    if (timed(0, s, [&] { return launch_norm(pp, s); })) return NS_ECUDA;
    if (timed(7, s, [&] { return launch_split_prep(pp, L.prefix.back(), s); })) return NS_ECUDA;
  } else {
    if (timed(0, s, [&] { return launch_norm(pp, s); })) return NS_ECUDA;
    if (timed(7, s, [&] { return launch_prep(pp, L.prefix.back(), s); })) return NS_ECUDA;
  }
  const Tile *t01 = reinterpret_cast<const Tile *>(blob + L.off_t01);
  const Tile *t2 = reinterpret_cast<const Tile *>(blob + L.off_t2);
  if (steps == 0) return NS_OK;
  if (L.tc()) {
    TcParams tp{};
    tp.tiles01 = t01;
    tp.tiles2 = t2;
    tp.n01 = static_cast<int>(L.tiles01.size());
    tp.n2 = static_cast<int>(L.tiles2.size());
    tp.steps = steps;
    tp.mats = mats;
    tp.ext = ext;
    tp.status = di->status;
    tp.done = done;
    tp.ticket = done + nbig;
    tp.rscale = L.split ? nullptr : pp.rscale;  // the fp32 slices are already normalised
    tp.split = L.split ? 1 : 0;
    tp.wait_limit_ns = opt.wait_limit_ns;
    tp.out_scale = opt.out_scale;
    tp.hold_signals = opt.hold_signals ? 1 : 0;
    tp.ncoef = table ? steps : 1;
    for (int k = 0; k < (table ? steps : 1); ++k)
      for (int u = 0; u < 3; ++u) tp.coef[k][u] = co[3 * k + u];
    const int per_step = 2 * tp.n01 + tp.n2;
    int rc = 1;
    if (!L.split && (opt.hold_signals || !phase_launches()) &&
        static_cast<int64_t>(steps) * per_step < (int64_t(1) << 30)) {
      // one launch: every step and phase, items ordered by per-matrix counters
      tp.g_begin = 0;
      tp.g_end = steps * per_step;
      tp.wait = 1;
      tp.tickets = 1;
      rc = timed(6, s, [&] { return launch_tc(tp, di->sms, s); });
      if (rc < 0) return NS_ECUDA;
    }
    if (rc == 1 && opt.hold_signals) return NS_ECUDA;  // the self-test needs the single launch
    if (rc == 1) {  // one launch per step and phase
      tp.wait = 0;
      tp.tickets = 0;
      const int begin[3] = {0, tp.n01, 2 * tp.n01}, count[3] = {tp.n01, tp.n01, tp.n2};
      for (int step = 0; step < steps; ++step)
        for (int phase = 0; phase < 3; ++phase) {
          tp.g_begin = step * per_step + begin[phase];
          tp.g_end = tp.g_begin + count[phase];
          if (timed(2 + phase, s, [&] { return launch_tc(tp, di->sms, s); })) return NS_ECUDA;
        }
    }
    return NS_OK;
  }
  PhaseParams ph{};
  ph.out_scale = opt.out_scale;
  ph.mats = mats;
  ph.ext = ext;
  ph.status = di->status;
  for (int step = 0; step < steps; ++step) {
    const float *cs = table ? co + 3 * step : co;
    ph.ca = cs[0];
    ph.cb = cs[1];
    ph.cc = cs[2];
    ph.step = step;
    ph.final_step = step == steps - 1;
    for (int phase = 0; phase < 3; ++phase) {
      ph.tiles = phase < 2 ? t01 : t2;
      ph.ntiles = static_cast<int>(phase < 2 ? L.tiles01.size() : L.tiles2.size());
      if (timed(2 + phase, s, [&] { return launch_simt_phase(phase, ph, s); })) return NS_ECUDA;
    }
  }
  return NS_OK;
}

int run(void *const *X, const int64_t *shapes, int count, int steps, const float *coeffs, float eps, int dtype,
        void *user_ws, size_t user_ws_bytes, cudaStream_t s, int slot = 0, bool table = false,
        const RunOpts &opt = RunOpts()) {
  NvtxRange range("ns call");
  int rc = validate(X, shapes, count, steps, dtype, true);
  if (rc) return rc;
  if (table && steps > 0 && (!coeffs || steps > kMaxTableSteps)) return NS_EINVAL;
  if (!(eps >= 0.f)) return NS_EINVAL;
  if (count == 0) return NS_OK;
  std::lock_guard<std::mutex> lock(g_mu);
  DevInfo *di = nullptr;
  rc = device_info(&di);
  if (rc) return rc;
  const float *co = coeffs ? coeffs : kDefaultCoeffs;
  std::vector<int64_t> key;
  if (!user_ws) {
    // a repeat of a call whose table is still on the device (same pointers,
    // shapes, steps and types; the same scratch, or the table would have been
    // dropped with it) runs from that plan: nothing is planned, encoded or uploaded
    int dev = 0;
    cudaGetDevice(&dev);
    CachedWs &c = cached_ws(dev, s, slot);
    key = call_key(X, shapes, count, steps, dtype);
    for (DevBlob &b : c.blobs)
      if (b.layout && b.key == key) {
        c.captured = c.captured || capturing(s);
        b.last_use = ++c.uses;
        return execute(*b.layout, c.ptr, b.ptr, steps, co, table, eps, di, s, opt);
      }
  }
  Layout L;
  build_layout(shapes, count, dtype, L);
  if (L.big.empty() && L.res.empty()) return NS_OK;

  uint8_t *ws = nullptr;
  std::vector<uint8_t> blob;
  CachedWs *cache = nullptr;
  if (user_ws) {
    if (user_ws_bytes < L.total) return NS_ENOMEM;
    if (reinterpret_cast<uintptr_t>(user_ws) % 256) return NS_EALIGN;
    ws = static_cast<uint8_t *>(user_ws);
  } else {
    int dev = 0;
    cudaGetDevice(&dev);
    cache = &cached_ws(dev, s, slot);
    rc = ensure_ws(*cache, L.total, s);
    if (rc) return rc;
    ws = cache->ptr;
  }
  rc = build_blob(L, X, shapes, steps, ws, blob);
  if (rc) return rc;
  const uint8_t *blob_dev = ws;
  if (!cache) {  // caller workspace: the table goes at its front, every call
    if (cudaMemcpyAsync(ws, blob.data(), blob.size(), cudaMemcpyHostToDevice, s) != cudaSuccess) return NS_ECUDA;
  } else {
    DevBlob *hit = nullptr;
    for (DevBlob &b : cache->blobs)
      if (b.bytes == blob) hit = &b;
    if (!hit) {
      if (cache->blobs.size() >= kBlobsPerWs) {  // evict the least recently used table (stream-ordered free)
        auto lru = std::min_element(cache->blobs.begin(), cache->blobs.end(),
                                    [](const DevBlob &a, const DevBlob &b) { return a.last_use < b.last_use; });
        drop_block(*cache, lru->ptr, s);
        cache->blobs.erase(lru);
      }
      DevBlob nb;
      if ((rc = new_block(&nb.ptr, std::max<size_t>(blob.size(), 256), blob.data(), blob.size(), s))) return rc;
      nb.bytes = std::move(blob);
      cache->blobs.push_back(std::move(nb));
      hit = &cache->blobs.back();
    }
    hit->last_use = ++cache->uses;
    hit->key = std::move(key);
    hit->layout = std::make_shared<const Layout>(L);
    blob_dev = hit->ptr;
  }
  return execute(L, ws, blob_dev, steps, co, table, eps, di, s, opt);
}

// ------------------------------------------------------------ host pipeline
// Streams and events of the host entry point, created once per device.
struct HostPipe {
  cudaStream_t h2d = nullptr, d2h = nullptr;
  cudaStream_t comp2 = nullptr;  // second compute stream: odd groups run there
  std::vector<cudaEvent_t> ev;
};
std::map<int, HostPipe> g_pipe;

int host_pipe(int dev, size_t nev, HostPipe **out) {
  HostPipe &hp = g_pipe[dev];
  if (!hp.h2d && cudaStreamCreateWithFlags(&hp.h2d, cudaStreamNonBlocking) != cudaSuccess) return NS_ECUDA;
  if (!hp.d2h && cudaStreamCreateWithFlags(&hp.d2h, cudaStreamNonBlocking) != cudaSuccess) return NS_ECUDA;
  if (!hp.comp2 && cudaStreamCreateWithFlags(&hp.comp2, cudaStreamNonBlocking) != cudaSuccess) return NS_ECUDA;
  while (hp.ev.size() < nev) {
    cudaEvent_t e;
    if (cudaEventCreateWithFlags(&e, cudaEventDisableTiming) != cudaSuccess) return NS_ECUDA;
    hp.ev.push_back(e);
  }
  *out = &hp;
  return NS_OK;
}

}  // namespace

// Every check a call makes before it touches the GPU: the arguments, then the
// current device (see ns_internal.h).
int check_call(void *const *X, const int64_t *shapes, int count, int steps, int dtype) {
  const int rc = validate(X, shapes, count, steps, dtype, true);
  if (rc || count == 0) return rc;
  std::lock_guard<std::mutex> lock(g_mu);
  DevInfo *di = nullptr;
  return device_info(&di);
}

// ------------------------------------------------------------ operator calls
OpCall::OpCall(void *stream) : s(static_cast<cudaStream_t>(stream)), lock(g_mu) {
  if (nvtx_on()) {
    nvtxRangePushA("ns call");
    ranged = true;
  }
  // the maps behind these allocate; an exception must not reach the C boundary
  try {
    DevInfo *di = nullptr;
    rc = device_info(&di);
    if (rc) return;
    sms = di->sms;
    status = di->status;
    cudaGetDevice(&dev);
  } catch (...) {
    rc = NS_ENOMEM;
  }
}

OpCall::~OpCall() {
  if (ranged) nvtxRangePop();
}

int OpCall::workspace(int slot, size_t bytes, uint8_t **ptr, size_t zero) {
  try {
    CachedWs &c = cached_ws(dev, s, slot);
    const int e = ensure_ws(c, std::max<size_t>(bytes, 256), s, zero);
    *ptr = c.ptr;
    return e;
  } catch (...) {
    return NS_ENOMEM;
  }
}

int OpCall::tensor_map(CUtensorMap *map, int elt, const void *base, int rank, const int64_t *dims,
                       const int64_t *pitch_bytes, const int *box) {
  if (const int e = get_encode()) return e;
  cuuint64_t d[3], st[2];
  cuuint32_t bx[3], one[3] = {1, 1, 1};
  for (int i = 0; i < rank; ++i) {
    d[i] = static_cast<cuuint64_t>(std::max<int64_t>(dims[i], 1));
    bx[i] = static_cast<cuuint32_t>(box[i]);
    if (i) st[i - 1] = static_cast<cuuint64_t>(pitch_bytes[i - 1]);
  }
  const CUresult r = g_encode(map, elt == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                              static_cast<cuuint32_t>(rank), const_cast<void *>(base), d, st, bx, one,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? NS_OK : NS_ECUDA;
}

int OpCall::timed_launch(int kind, int (*fn)(void *), void *arg) {
  try {
    return timed(kind, s, [&] { return fn(arg); }) ? NS_ECUDA : NS_OK;
  } catch (...) {
    return NS_ENOMEM;
  }
}

}  // namespace ns

using namespace ns;

extern "C" {

int64_t ns_cost(int64_t M, int64_t N) {
  if (M < 0 || N < 0) return -1;
  const int64_t hi = M > N ? M : N, lo = M > N ? N : M;
  return hi * lo * lo;
}

int ns_orthogonalize_batched(void *const *X, const int64_t *shapes, int count, int steps, const float *coeffs,
                             int dtype, void *stream) {
  return run(X, shapes, count, steps, coeffs, 1e-7f, dtype, nullptr, 0, static_cast<cudaStream_t>(stream));
}

int ns_orthogonalize_batched_ex(void *const *X, const int64_t *shapes, int count, int steps, const float *coeffs,
                                float eps, int dtype, void *workspace, size_t workspace_bytes, void *stream) {
  if (!workspace && count > 0) return NS_EINVAL;
  return run(X, shapes, count, steps, coeffs, eps, dtype, workspace, workspace_bytes,
             static_cast<cudaStream_t>(stream));
}

int ns_orthogonalize_batched_sched(void *const *X, const int64_t *shapes, int count, int steps,
                                   const float *coeff_table, int dtype, void *stream) {
  return run(X, shapes, count, steps, coeff_table, 1e-7f, dtype, nullptr, 0, static_cast<cudaStream_t>(stream), 0,
             true);
}

int ns_muon_update_batched(void *const *G, void *const *Mom, void *const *Out, const int64_t *shapes, int count,
                           int steps, const float *coeffs, float mu, int nesterov, float scale, int dtype,
                           void *stream) {
  int rc = validate(G, shapes, count, steps, dtype, true);
  if (!rc) rc = validate(Mom, shapes, count, steps, dtype, true);
  if (!rc) rc = validate(Out, shapes, count, steps, dtype, true);
  if (rc) return rc;
  if (!std::isfinite(mu) || !std::isfinite(scale) || (nesterov != 0 && nesterov != 1)) return NS_EINVAL;
  if (count == 0) return NS_OK;
  // the three buffers of every matrix, and of different matrices, must not
  // overlap; the one exception is an output buffer that is the matrix's own
  // gradient buffer (the update written over the gradient)
  {
    const size_t elt = dtype == NS_BF16 ? 2 : 4;
    std::vector<std::pair<uintptr_t, uintptr_t>> r;
    r.reserve(3 * static_cast<size_t>(count));
    for (int i = 0; i < count; ++i) {
      const int64_t n = shapes[2 * i] * shapes[2 * i + 1];
      if (n == 0) continue;
      const uintptr_t bytes = static_cast<uintptr_t>(n) * elt;
      for (void *const *arr : {G, Mom, Out}) {
        if (arr == Out && Out[i] == G[i]) continue;
        const uintptr_t b = reinterpret_cast<uintptr_t>(arr[i]);
        r.emplace_back(b, b + bytes);
      }
    }
    std::sort(r.begin(), r.end());
    for (size_t k = 1; k < r.size(); ++k)
      if (r[k].first < r[k - 1].second) return NS_EINVAL;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int sms = 0;
  int *status = nullptr;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    DevInfo *di = nullptr;
    rc = device_info(&di);
    if (rc) return rc;
    sms = di->sms;
    status = di->status;
  }
  for (int k0 = 0; k0 < count; k0 += kMomChunk) {
    MomentumParams mp{};
    mp.status = status;
    mp.mu = mu;
    mp.nesterov = nesterov;
    for (int i = k0; i < std::min(count, k0 + kMomChunk); ++i) {
      const int64_t n = shapes[2 * i] * shapes[2 * i + 1];
      if (n == 0) continue;
      mp.g[mp.count] = G[i];
      mp.mom[mp.count] = Mom[i];
      mp.out[mp.count] = Out[i];
      mp.numel[mp.count] = n;
      ++mp.count;
    }
    if (timed(8, s, [&] { return launch_momentum(mp, dtype, sms, s); })) return NS_ECUDA;
  }
  RunOpts opt;
  opt.out_scale = scale;
  return run(Out, shapes, count, steps, coeffs, 1e-7f, dtype, nullptr, 0, s, 0, false, opt);
}

size_t ns_workspace_bytes(const int64_t *shapes, int count, int dtype) {
  if (validate(nullptr, shapes, count, 0, dtype, false)) return 0;
  Layout L;
  build_layout(shapes, count, dtype, L);
  return L.total;
}

int ns_orthogonalize_batched_host(void *const *X_host, const int64_t *shapes, int count, int steps,
                                  const float *coeffs, int dtype, void *stream) {
  int rc = validate(X_host, shapes, count, steps, dtype, true);
  if (rc) return rc;
  if (count == 0) return NS_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t elt = dtype == NS_BF16 ? 2 : 4;
  std::vector<size_t> off(count), bytes(count);
  size_t total = 0;
  for (int i = 0; i < count; ++i) {
    bytes[i] = static_cast<size_t>(shapes[2 * i] * shapes[2 * i + 1]) * elt;
    off[i] = total;
    total = align_up(total + bytes[i], 256);
  }
  // contiguous groups of about total/G bytes: group g's copies in, its
  // Newton-Schulz and group g-1's copies out overlap. G is at most 8 and
  // groups hold at least 32 MiB: a group's kernels take about as long for one
  // small matrix as for many (one CTA per small matrix), so splitting a small
  // batch would only repeat that latency.
  constexpr int kMaxGroups = 8;
  constexpr size_t kMinGroupBytes = size_t(32) << 20;
  const int max_groups = static_cast<int>(std::min<size_t>(kMaxGroups, std::max<size_t>(1, total / kMinGroupBytes)));
  std::vector<int> gstart{0};
  size_t acc = 0;
  for (int i = 0; i < count; ++i) {
    acc += bytes[i];
    if (acc * max_groups >= total * gstart.size() && i + 1 < count &&
        static_cast<int>(gstart.size()) < max_groups)
      gstart.push_back(i + 1);
  }
  gstart.push_back(count);
  const int ngroups = static_cast<int>(gstart.size()) - 1;

  uint8_t *dbuf = nullptr;
  HostPipe *hp = nullptr;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    DevInfo *di = nullptr;
    rc = device_info(&di);
    if (rc) return rc;
    int dev = 0;
    cudaGetDevice(&dev);
    CachedWs &c = cached_ws(dev, s, 1);
    rc = ensure_ws(c, std::max<size_t>(total, 256), s);
    if (rc) return rc;
    dbuf = c.ptr;
    rc = host_pipe(dev, 2 * static_cast<size_t>(ngroups) + 2, &hp);
    if (rc) return rc;
  }
  std::vector<void *> dptr(count);
  for (int i = 0; i < count; ++i) dptr[i] = dbuf + off[i];
  cudaEvent_t ev_start = hp->ev[2 * ngroups], ev_comp2 = hp->ev[2 * ngroups + 1];
  // Odd groups compute on a second stream, so the partial last wave of one
  // group's launches shares the GPU with the start of the next group's (the
  // per-phase launches never wait on one another). The single-launch schedule
  // keeps every group on the caller's stream: its cooperative launch must
  // have the whole GPU.
  cudaStream_t comp[2] = {s, phase_launches() ? hp->comp2 : s};
  // the copies in and the second compute stream start after earlier work on the caller's stream
  if (cudaEventRecord(ev_start, s) != cudaSuccess || cudaStreamWaitEvent(hp->h2d, ev_start, 0) != cudaSuccess ||
      cudaStreamWaitEvent(hp->comp2, ev_start, 0) != cudaSuccess)
    return NS_ECUDA;
  for (int g = 0; g < ngroups; ++g) {
    const int i0 = gstart[g], i1 = gstart[g + 1];
    cudaStream_t cs = comp[g & 1];
    cudaEvent_t ev_in = hp->ev[2 * g], ev_out = hp->ev[2 * g + 1];
    for (int i = i0; i < i1; ++i)
      if (bytes[i] && cudaMemcpyAsync(dptr[i], X_host[i], bytes[i], cudaMemcpyHostToDevice, hp->h2d) != cudaSuccess)
        return NS_ECUDA;
    if (cudaEventRecord(ev_in, hp->h2d) != cudaSuccess || cudaStreamWaitEvent(cs, ev_in, 0) != cudaSuccess)
      return NS_ECUDA;
    rc = run(dptr.data() + i0, shapes + 2 * i0, i1 - i0, steps, coeffs, 1e-7f, dtype, nullptr, 0, cs, 2 + g);
    if (rc) return rc;
    if (cudaEventRecord(ev_out, cs) != cudaSuccess || cudaStreamWaitEvent(hp->d2h, ev_out, 0) != cudaSuccess)
      return NS_ECUDA;
    for (int i = i0; i < i1; ++i)
      if (bytes[i] && cudaMemcpyAsync(X_host[i], dptr[i], bytes[i], cudaMemcpyDeviceToHost, hp->d2h) != cudaSuccess)
        return NS_ECUDA;
  }
  // the caller's stream is ordered after the second compute stream's work
  if (cudaEventRecord(ev_comp2, hp->comp2) != cudaSuccess || cudaStreamWaitEvent(s, ev_comp2, 0) != cudaSuccess)
    return NS_ECUDA;
  if (cudaStreamSynchronize(hp->d2h) != cudaSuccess) return NS_ECUDA;
  return cudaStreamSynchronize(s) == cudaSuccess ? NS_OK : NS_ECUDA;
}

int ns_plan_shards(const int64_t *shapes, const int64_t *numels, int count, int nshards, double numel_eps,
                   int order, int64_t *loads, int *assign) {
  if (count < 0 || nshards <= 0 || (count > 0 && (!shapes || !assign))) return NS_EINVAL;
  if (order != NS_PLAN_COST && order != NS_PLAN_NUMEL) return NS_EINVAL;
  std::vector<int64_t> size(count), numel(count);
  int64_t total = 0;
  for (int i = 0; i < count; ++i) {
    const int64_t M = shapes[2 * i], N = shapes[2 * i + 1];
    if (M < 0 || N < 0 || (numels && numels[i] < 0)) return NS_EINVAL;
    numel[i] = numels ? numels[i] : M * N;
    size[i] = order == NS_PLAN_COST ? ns_cost(M, N) : numel[i];
    total += numel[i];
  }
  std::vector<int64_t> load(nshards, 0), placed(nshards, 0);
  if (loads)
    for (int s = 0; s < nshards; ++s) load[s] = loads[s];
  // largest first; ties keep the caller's order
  std::vector<int> idx(count);
  for (int i = 0; i < count; ++i) idx[i] = i;
  std::stable_sort(idx.begin(), idx.end(), [&](int a, int b) { return size[a] > size[b]; });
  const bool capped = numel_eps >= 0.0;
  const double cap = capped ? std::ceil((1.0 + numel_eps) * static_cast<double>(total) / nshards) : 0.0;
  for (int i : idx) {
    int best = -1;
    if (capped || order == NS_PLAN_COST) {
      for (int s = 0; s < nshards; ++s) {
        if (capped && static_cast<double>(placed[s] + numel[i]) > cap) continue;
        if (best < 0 || load[s] < load[best] || (load[s] == load[best] && placed[s] < placed[best])) best = s;
      }
    }
    if (best < 0) {  // least-numel fallback
      best = 0;
      for (int s = 1; s < nshards; ++s)
        if (placed[s] < placed[best]) best = s;
    }
    assign[i] = best;
    load[best] += size[i];
    placed[best] += numel[i];
  }
  if (loads)
    for (int s = 0; s < nshards; ++s) loads[s] = load[s];
  return NS_OK;
}

int ns_get_status(void *stream) {
  int dev = 0;
  if (const int rc = current_device(&dev)) return rc;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return NS_ECUDA;
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_status_word, sizeof(int)) != cudaSuccess) return NS_ECUDA;
  const int zero = 0;
  if (cudaMemcpyToSymbol(g_status_word, &zero, sizeof(int)) != cudaSuccess) return NS_ECUDA;
  // device status codes: 1 a bounded wait gave up, 2 a CTA pair's TMEM
  // allocations disagreed, 3 a debug build's bounds check caught a store
  return v == 0 ? NS_OK : v == 3 ? NS_EBOUNDS : v == 2 ? NS_ECUDA : NS_ETIMEOUT;
}

const char *ns_strerror(int code) {
  switch (code) {
    case NS_OK: return "success";
    case NS_EINVAL: return "invalid argument";
    case NS_EALIGN: return "matrix pointer not aligned to its element size";
    case NS_ENOMEM: return "workspace allocation failed or caller workspace too small";
    case NS_ECUDA: return "CUDA runtime or driver error";
    case NS_ETIMEOUT: return "a bounded device-side wait gave up";
    case NS_ENODEV: return "no CUDA device or driver, or the current device is not sm_100-family";
    case NS_ETOOBIG: return "batch needs more scratch than the no-allocation entry point's 256 MiB array";
    case NS_EBOUNDS: return "a debug build's bounds check caught a store outside its buffer (not made)";
    default: return "unknown status";
  }
}

int ns_release_workspace(void) {
  std::lock_guard<std::mutex> lock(g_mu);
  int dev = 0;
  if (const int rc = current_device(&dev)) return rc;
  if (cudaDeviceSynchronize() != cudaSuccess) return NS_ECUDA;
  for (auto it = g_ws.begin(); it != g_ws.end();) {
    if (it->first.dev == dev) {
      for (DevBlob &b : it->second.blobs) cudaFree(b.ptr);
      for (uint8_t *p : it->second.kept) cudaFree(p);
      if (it->second.ptr) cudaFree(it->second.ptr);
      it = g_ws.erase(it);
    } else {
      ++it;
    }
  }
  return NS_OK;
}

int64_t ns_num_kernel_launches(void) { return g_launches.load(); }

int64_t ns_num_workspace_allocations(void) { return g_allocations.load(); }

int ns_set_workspace_limit(size_t bytes) {
  g_ws_limit.store(bytes);
  return NS_OK;
}

int ns_set_nvtx(int enable) {
  g_nvtx.store(enable ? 1 : 0);
  return NS_OK;
}

int ns_set_f32_gemm(int mode) {
  if (mode != NS_F32_TENSOR && mode != NS_F32_SIMT) return NS_EINVAL;
  g_f32_gemm.store(mode);
  return NS_OK;
}

int ns_set_gemm_schedule(int mode) {
  if (mode != NS_SCHED_PHASE && mode != NS_SCHED_SINGLE) return NS_EINVAL;
  g_gemm_schedule.store(mode);
  return NS_OK;
}

int ns_selftest_wait_timeout(int limit_us, void *stream) {
  if (limit_us <= 0 || limit_us > 10000000) return NS_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  DevInfo *di = nullptr;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    const int rc = device_info(&di);
    if (rc) return rc;
  }
  int *gave_up = di->probe;
  if (cudaMemsetAsync(gave_up, 0, sizeof(int), s) != cudaSuccess) return NS_ECUDA;
  if (launch_wait_probe(di->status, static_cast<uint64_t>(limit_us) * 1000ull, gave_up, s)) return NS_ECUDA;
  int h = 0;
  if (cudaMemcpyAsync(&h, gave_up, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess) return NS_ECUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return NS_ECUDA;
  return h ? NS_OK : NS_ECUDA;
}

int ns_selftest_dependency_timeout(int limit_us, void *stream) {
  if (limit_us <= 0 || limit_us > 10000000) return NS_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  {
    std::lock_guard<std::mutex> lock(g_mu);
    DevInfo *di = nullptr;
    const int rc = device_info(&di);
    if (rc) return rc;
  }
  // two small non-zero bf16 matrices (every element 0x3C3C) and their own
  // workspace, allocated here and released before returning
  const int64_t shapes[4] = {512, 768, 512, 768};
  const size_t mat_bytes = 512 * 768 * 2;
  const size_t ws_bytes = ns_workspace_bytes(shapes, 2, NS_BF16);
  void *buf = nullptr;
  if (cudaMallocAsync(&buf, 2 * mat_bytes + ws_bytes, s) != cudaSuccess) {
    cudaGetLastError();
    return NS_ENOMEM;
  }
  uint8_t *base = static_cast<uint8_t *>(buf);
  void *X[2] = {base, base + mat_bytes};
  int rc = cudaMemsetAsync(base, 0x3C, 2 * mat_bytes, s) == cudaSuccess ? NS_OK : NS_ECUDA;
  RunOpts opt;
  opt.wait_limit_ns = static_cast<uint64_t>(limit_us) * 1000ull;
  opt.hold_signals = true;
  if (rc == NS_OK) rc = run(X, shapes, 2, 2, nullptr, 1e-7f, NS_BF16, base + 2 * mat_bytes, ws_bytes, s, 0, false, opt);
  const cudaError_t sync = cudaStreamSynchronize(s);
  cudaFreeAsync(buf, s);
  if (cudaStreamSynchronize(s) != cudaSuccess || sync != cudaSuccess) return NS_ECUDA;
  if (rc) return rc;
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_status_word, sizeof(int)) != cudaSuccess) return NS_ECUDA;
  return v != 0 ? NS_OK : NS_ECUDA;
}

int ns_selftest_bounds_check(void *stream) {
  DevInfo *di = nullptr;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    const int rc = device_info(&di);
    if (rc) return rc;
  }
#ifndef NS_DEBUG_BOUNDS
  (void)stream;
  return NS_EINVAL;  // a release build: no bounds checks to exercise
#else
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (launch_bounds_probe(di->status, di->probe, s)) return NS_ECUDA;
  return cudaStreamSynchronize(s) == cudaSuccess ? NS_OK : NS_ECUDA;
#endif
}

static void drop_timed() {
  for (auto &t : g_timed) {
    cudaEventDestroy(t.start);
    cudaEventDestroy(t.stop);
  }
  g_timed.clear();
}

int ns_set_kernel_timing(int enable) {
  std::lock_guard<std::mutex> lock(g_mu);
  drop_timed();
  g_timing = enable != 0;
  return NS_OK;
}

int ns_get_kernel_times(double *ms, int64_t *launches, int n) {
  std::lock_guard<std::mutex> lock(g_mu);
  if (n < 0 || n > kKinds || (n > 0 && (!ms || !launches))) return NS_EINVAL;
  double acc[kKinds] = {};
  int64_t cnt[kKinds] = {};
  for (auto &t : g_timed) {
    if (cudaEventSynchronize(t.stop) != cudaSuccess) return NS_ECUDA;
    float e = 0.f;
    if (cudaEventElapsedTime(&e, t.start, t.stop) != cudaSuccess) return NS_ECUDA;
    acc[t.kind] += e;
    cnt[t.kind] += 1;
  }
  for (int k = 0; k < n; ++k) {
    ms[k] = acc[k];
    launches[k] = cnt[k];
  }
  return NS_OK;
}

}  // extern "C"
