// uf_layers.cu -- the C ABI of the head's operators and the optimizer: argument checks, scratch
// layout, TMA tensor maps and the launches on the caller's stream.  No allocation, no
// synchronisation.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <initializer_list>
#include <memory>
#include <new>
#include <utility>

#include "../../include/uf_layers.h"
#include "layers.h"

using namespace ufc;

namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 512;  // row coordinates of the tensor maps are 32-bit
constexpr int kMaxWidth = 1 << 24;

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int elem_size(int type) { return type == UF_F32 ? 4 : type == UF_BF16 ? 2 : 1; }
bool float_type(int type) { return type == UF_BF16 || type == UF_F32; }
bool act_ok(int act) { return act >= UF_ACT_NONE && act <= UF_ACT_SILU; }

// A buffer of a call: [lo, hi), empty for NULL.
struct Range {
  uintptr_t lo, hi;
};
Range vec(const void* p, int64_t n, int elem) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Range{a, p && n > 0 ? a + static_cast<uintptr_t>(n) * elem : a};
}
// A matrix of rows x cols with row stride ld (elements).
Range mat(const void* p, int64_t rows, int64_t cols, int64_t ld, int elem) {
  return vec(p, rows > 0 ? (rows - 1) * ld + cols : 0, elem);
}
// No written range overlaps another one or a range that is read.
bool disjoint(std::initializer_list<Range> written, std::initializer_list<Range> read) {
  auto overlap = [](const Range& x, const Range& y) { return x.lo < x.hi && y.lo < y.hi && x.lo < y.hi && y.lo < x.hi; };
  for (auto i = written.begin(); i != written.end(); ++i) {
    for (auto j = i + 1; j != written.end(); ++j)
      if (overlap(*i, *j)) return false;
    for (const Range& r : read)
      if (overlap(*i, r)) return false;
  }
  return true;
}

// The ranges of a long list of buffers, sorted by their start.  Lists come as a few ascending runs (one
// of parameters, one of states, ...), so runs are merged as they are found: the 960 ranges of 160
// tensors take 6 us of a call, 17 in random order.
struct Ranges {
  std::unique_ptr<Range[]> own;
  Range* r = nullptr;
  int n = 0;
  explicit Ranges(int64_t most) : own(new (std::nothrow) Range[2 * static_cast<size_t>(most)]), r(own.get()), most_(most) {}
  void add(const Range& x) {
    if (x.lo < x.hi) r[n++] = x;
  }
  void sort() {
    const auto before = [](const Range& x, const Range& y) { return x.lo < y.lo; };
    Range* to = r == own.get() ? r + most_ : own.get();
    for (int runs = 2; runs > 1; std::swap(r, to)) {
      runs = 0;
      for (Range* i = r; i < r + n; ++runs) {
        Range* mid = std::is_sorted_until(i, r + n, before);
        Range* end = std::is_sorted_until(mid, r + n, before);
        std::merge(i, mid, mid, end, to + (i - r), before);
        i = end;
      }
    }
  }

 private:
  int64_t most_;
};
// disjoint() of long lists, which it sorts.
bool disjoint(Ranges& written, Ranges& read) {
  written.sort();
  read.sort();
  for (int i = 1; i < written.n; ++i)
    if (written.r[i].lo < written.r[i - 1].hi) return false;
  for (int i = 0, j = 0; i < written.n && j < read.n;) {
    const Range &w = written.r[i], &x = read.r[j];
    if (w.lo < x.hi && x.lo < w.hi) return false;
    if (x.hi <= w.lo)
      ++j;
    else
      ++i;
  }
  return true;
}

// A matrix operand or output of a product: rows on 16-byte boundaries.
bool rows16(const void* p, int64_t ld, int64_t cols, int elem) {
  return aligned(p, 16) && ld >= cols && (ld * elem) % 16 == 0;
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// [rows][cols] elements of elem bytes (1: e4m3, 2: bf16, 4: fp32), boxes of box_cols by box_rows
// with the swizzle of their width (128 or 64 bytes).
bool encode(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t ld, int elem, int box_cols, int box_rows) {
  const auto enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * elem};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t es[2] = {1, 1};
  const CUtensorMapDataType type = elem == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                   : elem == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                               : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  return enc(m, type, 2, const_cast<void*>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_cols * elem == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Every kernel of the library is loaded and sized once per device; later calls see it without
// taking the set-up's lock.
std::atomic<uint64_t> g_ready{0};
uf_status_t ready() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return UF_CUDA_ERROR;
  if (dev >= 0 && dev < 64 && (g_ready.load(std::memory_order_relaxed) >> dev & 1)) return UF_OK;
  const uf_status_t st = uf_contrastive_init(dev);
  if (st == UF_OK) g_ready.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  return st;
}

uf_status_t status_of(cudaError_t e) { return e == cudaSuccess ? UF_OK : UF_CUDA_ERROR; }

// A product's operands and result.  mn false: an operand is [rows][kdim] (K-major); true: [kdim][rows].
struct Operand {
  const void* p;
  int64_t ld;
  bool mn;
};
struct Product {
  Operand a, b;
  int64_t kdim;
  Epilogue e;
};

size_t part_bytes(const DensePlan& pl, int n) {
  size_t bytes = 0;
  for (int k = 0; k < n; ++k) bytes += align256(pl.p[k].part_bytes);
  return bytes;
}

// q[k].e.rows x q[k].e.cols = A B^T (gated: B holds the gate's rows, then as many of the up
// projection's); a product of no rows is left out.
cudaError_t products(const Product* q, int n, DenseKind kind, void* part, int* status, cudaStream_t stream) {
  const bool gated = kind == kDenseGated;
  const int elem = kind == kDenseLinear8 ? 1 : 2;
  DenseShape shapes[2];
  for (int k = 0; k < n; ++k) shapes[k] = DenseShape{q[k].e.rows, q[k].e.cols, q[k].kdim};
  const DensePlan pl = plan_dense(shapes, n, kind);
  const int wide = 128 / elem, out = dense_store_cols(pl.bn, gated);
  DenseMaps maps[2];
  DenseParams params[2] = {};
  uint8_t* scratch = static_cast<uint8_t*>(part);
  for (int k = 0; k < n; ++k) {
    const Epilogue& e = q[k].e;
    const Operand &a = q[k].a, &b = q[k].b;
    const DensePlan::Product& s = pl.p[k];
    params[k].e = e;
    params[k].up_row = e.cols;
    params[k].part = reinterpret_cast<float*>(scratch);
    scratch += align256(s.part_bytes);
    if (e.rows == 0) continue;
    const int64_t b_rows = gated ? 2 * e.cols : e.cols;
    DenseMaps& m = maps[k];
    bool ok = a.mn ? encode(&m.a, a.p, q[k].kdim, e.rows, a.ld, 2, 64, 64)
                   : encode(&m.a, a.p, e.rows, q[k].kdim, a.ld, elem, wide, 128);
    ok = ok && (b.mn ? encode(&m.b, b.p, q[k].kdim, b_rows, b.ld, 2, 64, 64)
                     : encode(&m.b, b.p, b_rows, q[k].kdim, b.ld, elem, wide, pl.bn / 2));
    if (s.rest > 0) ok = ok && encode(&m.part, params[k].part, static_cast<int64_t>(s.splits) * s.rest * 256, pl.bn, pl.bn, 4, 32, 32);
    if (s.full > 0) {
      ok = ok && encode(&m.y, e.y, e.rows, e.cols, e.ldy, 2, out, 32);
      if (e.pre) ok = ok && encode(&m.p0, e.pre, e.rows, e.cols, e.ldp, 2, out, 32);
      if (e.pre && gated) ok = ok && encode(&m.p1, e.pre + e.cols, e.rows, e.cols, e.ldp, 2, out, 32);
    }
    if (!ok) return cudaErrorInvalidValue;
  }
  return launch_dense(maps, params, pl, n, kind, status, stream);
}

size_t product_bytes(int64_t rows, int64_t cols, int64_t kdim, DenseKind kind) {
  const DenseShape s{rows, cols, kdim};
  return part_bytes(plan_dense(&s, 1, kind), 1);
}

// The gradients' products of a layer, of which dx (rows x inner) or dW (outer x inner) may not be
// asked for: scratch for each case (0 rows: left out).
size_t grads_bytes(int64_t rows, int64_t inner, int64_t outer) {
  size_t most = 0;
  for (const int asked : {1, 2, 3}) {
    const DenseShape s[2] = {{asked & 1 ? rows : 0, inner, outer}, {asked & 2 ? outer : 0, inner, rows}};
    const size_t b = part_bytes(plan_dense(s, 2, kDenseGrads), 2);
    most = b > most ? b : most;
  }
  return most;
}

bool sizes_ok(int64_t rows, int inner, int outer, int multiple) {
  return rows >= 0 && rows <= kMaxRows && inner >= multiple && outer >= multiple && inner <= kMaxWidth &&
         outer <= kMaxWidth && inner % multiple == 0 && outer % multiple == 0;
}

bool workspace_ok(const void* ws, size_t have, size_t need, uf_status_t* st) {
  if (need == 0) return true;
  if (!ws || !aligned(ws, 256)) {
    *st = UF_INVALID_ARGUMENT;
    return false;
  }
  if (have < need) {
    *st = UF_WORKSPACE_TOO_SMALL;
    return false;
  }
  return true;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------------------ RMS norm
uf_status_t uf_rmsnorm_fwd(const void* x, int64_t ldx, int x_type, const void* residual, int64_t ldr, int stream_type,
                           const void* weight, int weight_type, int64_t rows, int width, float eps, void* y, int64_t ldy,
                           int y_type, float* y_scale, void* stream_out, int64_t lds, float* rstd, void* stream) {
  if (rows < 0 || rows > kMaxRows || width < 1 || !float_type(x_type) || !float_type(weight_type)) return UF_INVALID_ARGUMENT;
  if (width > kNormMaxWidth) return UF_UNSUPPORTED;
  if (y_type != UF_BF16 && y_type != UF_E4M3) return UF_INVALID_ARGUMENT;
  if (residual && !float_type(stream_type)) return UF_INVALID_ARGUMENT;
  if (residual && x_type != UF_BF16) return UF_UNSUPPORTED;
  if ((residual == nullptr) != (stream_out == nullptr) || (y_type == UF_E4M3) != (y_scale != nullptr))
    return UF_INVALID_ARGUMENT;
  if (!(eps >= 0.f) || !std::isfinite(eps) || !weight) return UF_INVALID_ARGUMENT;
  if (rows > 0 && (!x || !y)) return UF_INVALID_ARGUMENT;
  if (ldx < width || ldy < width || (residual && (ldr < width || lds < width))) return UF_INVALID_ARGUMENT;
  const int xe = elem_size(x_type), se = elem_size(stream_type), we = elem_size(weight_type), ye = elem_size(y_type);
  if (!aligned(x, xe) || !aligned(weight, we) || !aligned(y, ye) || !aligned(rstd, 4) || !aligned(y_scale, 4) ||
      (residual && (!aligned(residual, se) || !aligned(stream_out, se))))
    return UF_INVALID_ARGUMENT;
  if (!disjoint({mat(y, rows, width, ldy, ye), vec(y_scale, rows, 4), mat(stream_out, rows, width, lds, se), vec(rstd, rows, 4)},
                {mat(x, rows, width, ldx, xe), mat(residual, rows, width, ldr, se), vec(weight, width, we)}))
    return UF_INVALID_ARGUMENT;
  if (rows == 0) return UF_OK;
  const uf_status_t st = ready();
  if (st != UF_OK) return st;
  NormFwdParams p{};
  p.x = x, p.ldx = ldx, p.x_type = x_type;
  p.res = residual, p.ldr = ldr, p.stream_type = stream_type;
  p.weight = weight, p.weight_type = weight_type;
  p.rows = rows, p.width = width, p.eps = eps;
  p.y = y, p.ldy = ldy, p.y_type = y_type, p.y_scale = y_scale;
  p.s = stream_out, p.lds = lds, p.rstd = rstd;
  return status_of(launch_norm_fwd(p, static_cast<cudaStream_t>(stream)));
}

size_t uf_rmsnorm_bwd_workspace(int64_t rows, int width) {
  if (rows < 0 || rows > kMaxRows || width < 1 || width > kNormMaxWidth) return 0;
  return align256(sizeof(float) * static_cast<size_t>(norm_bwd_blocks(rows, width)) * width);
}

uf_status_t uf_rmsnorm_bwd(const void* dy, int64_t lddy, int dy_type, const void* s, int64_t lds, int stream_type,
                           const void* weight, int weight_type, const float* rstd, const void* d_stream, int64_t ldds,
                           int64_t rows, int width, void* dx, int64_t lddx, float* dweight, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (rows < 0 || rows > kMaxRows || width < 1 || !float_type(dy_type) || !float_type(stream_type) || !float_type(weight_type))
    return UF_INVALID_ARGUMENT;
  if (width > kNormMaxWidth) return UF_UNSUPPORTED;
  if (!weight || (rows > 0 && (!dy || !s || !rstd || !dx))) return UF_INVALID_ARGUMENT;
  if (lddy < width || lds < width || lddx < width || (d_stream && ldds < width)) return UF_INVALID_ARGUMENT;
  const int ge = elem_size(dy_type), se = elem_size(stream_type), we = elem_size(weight_type);
  if (!aligned(dy, ge) || !aligned(s, se) || !aligned(dx, se) || !aligned(d_stream, se) || !aligned(weight, we) ||
      !aligned(rstd, 4) || !aligned(dweight, 4))
    return UF_INVALID_ARGUMENT;
  uf_status_t st = UF_OK;
  const size_t need = dweight ? uf_rmsnorm_bwd_workspace(rows, width) : 0;
  if (!workspace_ok(workspace, workspace_bytes, need, &st)) return st;
  if (!disjoint({mat(dx, rows, width, lddx, se), vec(dweight, width, 4), vec(workspace, need, 1)},
                {mat(dy, rows, width, lddy, ge), mat(s, rows, width, lds, se), vec(weight, width, we), vec(rstd, rows, 4),
                 mat(d_stream, rows, width, ldds, se)}))
    return UF_INVALID_ARGUMENT;
  if (rows == 0 && !dweight) return UF_OK;
  if ((st = ready()) != UF_OK) return st;
  NormRowsBwdParams p{};
  p.dy = dy, p.lddy = lddy, p.dy_type = dy_type;
  p.s = s, p.lds = lds, p.stream_type = stream_type;
  p.weight = weight, p.weight_type = weight_type;
  p.rstd = rstd;
  p.ds = d_stream, p.ldds = ldds;
  p.dx = dx, p.lddx = lddx;
  p.rows = rows, p.width = width;
  p.part = dweight ? static_cast<float*>(workspace) : nullptr;
  p.dweight = dweight;
  return status_of(launch_norm_rows_bwd(p, static_cast<cudaStream_t>(stream)));
}

// -------------------------------------------------------------------- linear projection
size_t uf_linear_fwd_workspace(int64_t rows, int inner, int outer, int type) {
  if ((type != UF_BF16 && type != UF_E4M3) || !sizes_ok(rows, inner, outer, type == UF_E4M3 ? 16 : 8)) return 0;
  return skinny_takes(rows, static_cast<int64_t>(inner) * (type == UF_E4M3 ? 1 : 2), outer)
             ? 0
             : product_bytes(rows, outer, inner, type == UF_E4M3 ? kDenseLinear8 : kDenseLinear);
}

uf_status_t uf_linear_fwd(const void* x, int64_t ldx, const void* W, int64_t ldw, int type, const float* x_scale,
                          const float* w_scale, const void* bias, int bias_type, const void* residual, int64_t ldr, int act,
                          int64_t rows, int inner, int outer, void* y, int64_t ldy, void* pre, int64_t ldp, void* workspace,
                          size_t workspace_bytes, int* device_status, void* stream) {
  if ((type != UF_BF16 && type != UF_E4M3) || !act_ok(act) || (bias && !float_type(bias_type))) return UF_INVALID_ARGUMENT;
  const bool e4m3 = type == UF_E4M3;
  if (!sizes_ok(rows, inner, outer, e4m3 ? 16 : 8)) return UF_INVALID_ARGUMENT;
  if (!W || (rows > 0 && (!x || !y)) || (rows > 0 && e4m3 && !x_scale) || e4m3 != (w_scale != nullptr) || (!e4m3 && x_scale))
    return UF_INVALID_ARGUMENT;
  const int e = elem_size(type), be = elem_size(bias_type);
  if (!rows16(x, ldx, inner, e) || !rows16(W, ldw, inner, e) || !rows16(y, ldy, outer, 2) ||
      (residual && !rows16(residual, ldr, outer, 2)) || (pre && !rows16(pre, ldp, outer, 2)) || !aligned(bias, 16) ||
      !aligned(x_scale, 4) || !aligned(w_scale, 16) || !aligned(device_status, 4))
    return UF_INVALID_ARGUMENT;
  uf_status_t st = UF_OK;
  const size_t need = uf_linear_fwd_workspace(rows, inner, outer, type);
  if (!workspace_ok(workspace, workspace_bytes, need, &st)) return st;
  if (!disjoint({mat(y, rows, outer, ldy, 2), mat(pre, rows, outer, ldp, 2), vec(workspace, need, 1), vec(device_status, 1, 4)},
                {mat(x, rows, inner, ldx, e), mat(W, outer, inner, ldw, e), vec(x_scale, rows, 4), vec(w_scale, outer, 4),
                 vec(bias, outer, be), mat(residual, rows, outer, ldr, 2)}))
    return UF_INVALID_ARGUMENT;
  if (rows == 0) return UF_OK;
  if ((st = ready()) != UF_OK) return st;
  Epilogue ep{};
  ep.act = act;
  ep.x_scale = x_scale, ep.w_scale = w_scale;
  ep.bias = bias, ep.bias_type = bias_type;
  ep.res = static_cast<const uint16_t*>(residual), ep.ldr = ldr;
  ep.y = static_cast<uint16_t*>(y), ep.ldy = ldy;
  ep.pre = static_cast<uint16_t*>(pre), ep.ldp = ldp;
  ep.rows = rows, ep.cols = outer;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (skinny_takes(rows, static_cast<int64_t>(inner) * e, outer)) {
    SkinnyParams p{};
    p.e = ep;
    p.x = static_cast<const uint8_t*>(x), p.ldx_bytes = ldx * e;
    p.w = static_cast<const uint8_t*>(W), p.ldw_bytes = ldw * e;
    p.k_bytes = static_cast<int64_t>(inner) * e;
    return status_of(launch_skinny(p, e, false, s));
  }
  const Product q{{x, ldx, false}, {W, ldw, false}, inner, ep};
  return status_of(products(&q, 1, e4m3 ? kDenseLinear8 : kDenseLinear, workspace, device_status, s));
}

}  // extern "C"

namespace {

// Scratch of a linear backward: dz, the bias gradient's parts, the products' splits.
struct LinearBwdScratch {
  size_t dz, db, part, total;
};
LinearBwdScratch linear_bwd_scratch(int64_t rows, int inner, int outer) {
  LinearBwdScratch s{};
  s.dz = 0;
  s.db = align256(2 * static_cast<size_t>(rows) * outer);
  s.part = s.db + align256(sizeof(float) * static_cast<size_t>(act_bwd_blocks(rows, outer)) * outer);
  s.total = s.part + (rows > 0 ? grads_bytes(rows, inner, outer) : 0);
  return s;
}

// dx = dz W (contracting dz's columns) and dW = dz^T x (contracting the rows).
uf_status_t grads(const void* dz, int64_t lddz, const void* x, int64_t ldx, const void* W, int64_t ldw, int64_t rows,
                  int64_t inner, int64_t outer, void* dx, int64_t lddx, void* dW, int64_t lddw, void* part, int* status,
                  cudaStream_t s) {
  Product q[2] = {{{dz, lddz, false}, {W, ldw, true}, outer, {}}, {{dz, lddz, true}, {x, ldx, true}, rows, {}}};
  q[0].e.cols = q[1].e.cols = inner;
  if (dx) q[0].e.y = static_cast<uint16_t*>(dx), q[0].e.ldy = lddx, q[0].e.rows = rows;
  if (dW) q[1].e.y = static_cast<uint16_t*>(dW), q[1].e.ldy = lddw, q[1].e.rows = outer;
  if (!dx && !dW) return UF_OK;
  return status_of(products(q, 2, kDenseGrads, part, status, s));
}

}  // namespace

extern "C" {

size_t uf_linear_bwd_workspace(int64_t rows, int inner, int outer) {
  return sizes_ok(rows, inner, outer, 8) ? linear_bwd_scratch(rows, inner, outer).total : 0;
}

uf_status_t uf_linear_bwd(const void* dy, int64_t lddy, int dy_type, const void* x, int64_t ldx, const void* W, int64_t ldw,
                          const void* pre, int64_t ldp, int act, int64_t rows, int inner, int outer, void* dx, int64_t lddx,
                          void* dW, int64_t lddw, float* dbias, void* workspace, size_t workspace_bytes, int* device_status,
                          void* stream) {
  if (!float_type(dy_type) || !act_ok(act) || !sizes_ok(rows, inner, outer, 8)) return UF_INVALID_ARGUMENT;
  const bool has_act = act != UF_ACT_NONE;
  if (rows > 0 && (!dy || (dW && !x) || (has_act && !pre))) return UF_INVALID_ARGUMENT;
  if (dx && !W) return UF_INVALID_ARGUMENT;
  if (!rows16(dy, lddy, outer, elem_size(dy_type)) || (dW && !rows16(x, ldx, inner, 2)) || (dx && !rows16(W, ldw, inner, 2)) ||
      (has_act && !rows16(pre, ldp, outer, 2)) || (dx && !rows16(dx, lddx, inner, 2)) || (dW && !rows16(dW, lddw, inner, 2)) ||
      !aligned(dbias, 4) || !aligned(device_status, 4))
    return UF_INVALID_ARGUMENT;
  uf_status_t st = UF_OK;
  const LinearBwdScratch sc = linear_bwd_scratch(rows, inner, outer);
  if (!workspace_ok(workspace, workspace_bytes, sc.total, &st)) return st;
  if (!disjoint({mat(dx, rows, inner, lddx, 2), mat(dW, outer, inner, lddw, 2), vec(dbias, outer, 4),
                 vec(workspace, sc.total, 1), vec(device_status, 1, 4)},
                {mat(dy, rows, outer, lddy, elem_size(dy_type)), mat(x, rows, inner, ldx, 2), mat(W, outer, inner, ldw, 2),
                 mat(has_act ? pre : nullptr, rows, outer, ldp, 2)}))
    return UF_INVALID_ARGUMENT;
  if (!dx && !dW && !dbias) return UF_OK;
  if ((st = ready()) != UF_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if (dW && cudaMemset2DAsync(dW, lddw * 2, 0, static_cast<size_t>(inner) * 2, outer, s) != cudaSuccess) return UF_CUDA_ERROR;
    if (dbias && cudaMemsetAsync(dbias, 0, sizeof(float) * outer, s) != cudaSuccess) return UF_CUDA_ERROR;
    return UF_OK;
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const bool as_is = !has_act && dy_type == UF_BF16;  // dz is dy
  const bool products = dx || dW;
  if (dbias || !as_is) {
    ActBwdParams p{};
    p.dy = dy, p.lddy = lddy, p.dy_type = dy_type;
    p.pre = has_act ? static_cast<const uint16_t*>(pre) : nullptr, p.ldp = ldp, p.act = act;
    p.dz = products && !as_is ? reinterpret_cast<uint16_t*>(ws + sc.dz) : nullptr, p.ldz = outer;
    p.part = dbias ? reinterpret_cast<float*>(ws + sc.db) : nullptr;
    p.rows = rows, p.n = outer;
    if (launch_act_bwd(p, s) != cudaSuccess) return UF_CUDA_ERROR;
    if (dbias && launch_col_sum(p.part, act_bwd_blocks(rows, outer), outer, dbias, s) != cudaSuccess) return UF_CUDA_ERROR;
  }
  return grads(as_is ? dy : ws + sc.dz, as_is ? lddy : outer, x, ldx, W, ldw, rows, inner, outer, dx, lddx, dW, lddw,
               ws + sc.part, device_status, s);
}

// -------------------------------------------------------------------- gated feed-forward
size_t uf_gated_fwd_workspace(int64_t rows, int inner, int outer) {
  if (!sizes_ok(rows, inner, outer, 8) || outer > kMaxWidth / 2) return 0;
  return skinny_takes(rows, 2 * static_cast<int64_t>(inner), outer) ? 0 : product_bytes(rows, outer, inner, kDenseGated);
}

uf_status_t uf_gated_fwd(const void* x, int64_t ldx, const void* W, int64_t ldw, int act, int64_t rows, int inner, int outer,
                         void* h, int64_t ldh, void* pre, int64_t ldp, void* workspace, size_t workspace_bytes,
                         int* device_status, void* stream) {
  if (!act_ok(act) || act == UF_ACT_NONE || !sizes_ok(rows, inner, outer, 8) || outer > kMaxWidth / 2) return UF_INVALID_ARGUMENT;
  if (!W || (rows > 0 && (!x || !h))) return UF_INVALID_ARGUMENT;
  if (!rows16(x, ldx, inner, 2) || !rows16(W, ldw, inner, 2) || !rows16(h, ldh, outer, 2) ||
      (pre && !rows16(pre, ldp, 2 * static_cast<int64_t>(outer), 2)) || !aligned(device_status, 4))
    return UF_INVALID_ARGUMENT;
  uf_status_t st = UF_OK;
  const size_t need = uf_gated_fwd_workspace(rows, inner, outer);
  if (!workspace_ok(workspace, workspace_bytes, need, &st)) return st;
  const int64_t two = 2 * static_cast<int64_t>(outer);
  if (!disjoint({mat(h, rows, outer, ldh, 2), mat(pre, rows, two, ldp, 2), vec(workspace, need, 1), vec(device_status, 1, 4)},
                {mat(x, rows, inner, ldx, 2), mat(W, two, inner, ldw, 2)}))
    return UF_INVALID_ARGUMENT;
  if (rows == 0) return UF_OK;
  if ((st = ready()) != UF_OK) return st;
  Epilogue ep{};
  ep.act = act;
  ep.y = static_cast<uint16_t*>(h), ep.ldy = ldh;
  ep.pre = static_cast<uint16_t*>(pre), ep.ldp = ldp;
  ep.rows = rows, ep.cols = outer;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (skinny_takes(rows, 2 * static_cast<int64_t>(inner), outer)) {
    SkinnyParams p{};
    p.e = ep;
    p.x = static_cast<const uint8_t*>(x), p.ldx_bytes = ldx * 2;
    p.w = static_cast<const uint8_t*>(W), p.ldw_bytes = ldw * 2;
    p.k_bytes = static_cast<int64_t>(inner) * 2;
    p.up_row = outer;
    return status_of(launch_skinny(p, 2, true, s));
  }
  const Product q{{x, ldx, false}, {W, ldw, false}, inner, ep};
  return status_of(products(&q, 1, kDenseGated, workspace, device_status, s));
}

size_t uf_gated_bwd_workspace(int64_t rows, int inner, int outer) {
  if (!sizes_ok(rows, inner, outer, 8) || outer > kMaxWidth / 2) return 0;
  const int two = 2 * outer;
  return align256(2 * static_cast<size_t>(rows) * two) + (rows > 0 ? grads_bytes(rows, inner, two) : 0);
}

uf_status_t uf_gated_bwd(const void* dh, int64_t lddh, const void* x, int64_t ldx, const void* W, int64_t ldw,
                         const void* pre, int64_t ldp, int act, int64_t rows, int inner, int outer, void* dx, int64_t lddx,
                         void* dW, int64_t lddw, void* workspace, size_t workspace_bytes, int* device_status, void* stream) {
  if (!act_ok(act) || act == UF_ACT_NONE || !sizes_ok(rows, inner, outer, 8) || outer > kMaxWidth / 2) return UF_INVALID_ARGUMENT;
  const int64_t two = 2 * static_cast<int64_t>(outer);
  if (rows > 0 && (!dh || !pre || (dW && !x))) return UF_INVALID_ARGUMENT;
  if (dx && !W) return UF_INVALID_ARGUMENT;
  if (!rows16(dh, lddh, outer, 2) || !rows16(pre, ldp, two, 2) || (dW && !rows16(x, ldx, inner, 2)) ||
      (dx && !rows16(W, ldw, inner, 2)) || (dx && !rows16(dx, lddx, inner, 2)) || (dW && !rows16(dW, lddw, inner, 2)) ||
      !aligned(device_status, 4))
    return UF_INVALID_ARGUMENT;
  uf_status_t st = UF_OK;
  const size_t need = uf_gated_bwd_workspace(rows, inner, outer);
  if (!workspace_ok(workspace, workspace_bytes, need, &st)) return st;
  if (!disjoint({mat(dx, rows, inner, lddx, 2), mat(dW, two, inner, lddw, 2), vec(workspace, need, 1), vec(device_status, 1, 4)},
                {mat(dh, rows, outer, lddh, 2), mat(x, rows, inner, ldx, 2), mat(W, two, inner, ldw, 2),
                 mat(pre, rows, two, ldp, 2)}))
    return UF_INVALID_ARGUMENT;
  if (!dx && !dW) return UF_OK;
  if ((st = ready()) != UF_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if (dW && cudaMemset2DAsync(dW, lddw * 2, 0, static_cast<size_t>(inner) * 2, two, s) != cudaSuccess) return UF_CUDA_ERROR;
    return UF_OK;
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  GatedActBwdParams p{};
  p.dh = static_cast<const uint16_t*>(dh), p.lddh = lddh;
  p.pre = static_cast<const uint16_t*>(pre), p.ldp = ldp;
  p.d = reinterpret_cast<uint16_t*>(ws);
  p.rows = rows, p.n = outer, p.act = act;
  if (launch_gated_act_bwd(p, s) != cudaSuccess) return UF_CUDA_ERROR;
  return grads(ws, two, x, ldx, W, ldw, rows, inner, two, dx, lddx, dW, lddw,
               ws + align256(2 * static_cast<size_t>(rows) * two), device_status, s);
}

// -------------------------------------------------------------------------------- AdamW
uf_status_t uf_adamw_step(int n, void* const* p, const void* const* g, void* const* m, void* const* v, float* const* m_scale,
                          float* const* v_scale, void* const* copy, const int64_t* sizes, int param_type, int grad_type,
                          int state_type, float lr, const float* lr_dev, double beta1, double beta2, float eps,
                          float weight_decay, int64_t step, const int64_t* step_dev, uint32_t seed,
                          const float* grad_scale_dev, void* stream) {
  if (n < 0 || (n > 0 && (!p || !g || !m || !v || !sizes))) return UF_INVALID_ARGUMENT;
  if (!float_type(param_type) || !float_type(grad_type) || (state_type != UF_F32 && state_type != UF_E4M3))
    return UF_INVALID_ARGUMENT;
  const bool e8 = state_type == UF_E4M3;
  if (n > 0 && e8 && (!m_scale || !v_scale)) return UF_INVALID_ARGUMENT;
  if (copy && param_type != UF_F32) return UF_INVALID_ARGUMENT;
  if (!(beta1 >= 0.f && beta1 < 1.f && beta2 >= 0.f && beta2 < 1.f && eps >= 0.f) || !std::isfinite(eps) ||
      !std::isfinite(weight_decay) || (!lr_dev && !std::isfinite(lr)) || (!step_dev && step < 1))
    return UF_INVALID_ARGUMENT;
  if (!aligned(lr_dev, 4) || !aligned(step_dev, 8) || !aligned(grad_scale_dev, 4)) return UF_INVALID_ARGUMENT;
  const int pe = elem_size(param_type), ge = elem_size(grad_type), se = elem_size(state_type);
  if (n == 0) return UF_OK;
  Ranges written(6 * static_cast<int64_t>(n)), read(static_cast<int64_t>(n) + 3);
  if (!written.r || !read.r) return UF_CUDA_ERROR;
  for (int i = 0; i < n; ++i) {
    if (sizes[i] < 0) return UF_INVALID_ARGUMENT;
    if (sizes[i] == 0) continue;
    if (!p[i] || !g[i] || !m[i] || !v[i] || (e8 && (!m_scale[i] || !v_scale[i]))) return UF_INVALID_ARGUMENT;
    if (!aligned(p[i], pe) || !aligned(g[i], ge) || !aligned(m[i], se) || !aligned(v[i], se)) return UF_INVALID_ARGUMENT;
    if (e8 && (!aligned(m_scale[i], 4) || !aligned(v_scale[i], 4))) return UF_INVALID_ARGUMENT;
    if (copy && !aligned(copy[i], 2)) return UF_INVALID_ARGUMENT;
    written.add(vec(p[i], sizes[i], pe));
    read.add(vec(g[i], sizes[i], ge));
  }
  // list by list: each is an ascending run of addresses as a rule
  for (int i = 0; i < n; ++i) written.add(vec(m[i], sizes[i], se));
  for (int i = 0; i < n; ++i) written.add(vec(v[i], sizes[i], se));
  for (int i = 0; copy && i < n; ++i) written.add(vec(copy[i], sizes[i], 2));
  for (auto* scale : {m_scale, v_scale})
    for (int i = 0; e8 && i < n; ++i) written.add(vec(scale[i], (sizes[i] + kAdamBlock - 1) / kAdamBlock, 4));
  read.add(vec(lr_dev, 1, 4));
  read.add(vec(step_dev, 1, 8));
  read.add(vec(grad_scale_dev, 1, 4));
  if (!disjoint(written, read)) return UF_INVALID_ARGUMENT;
  const uf_status_t st = ready();
  if (st != UF_OK) return st;
  AdamScalars sc{};
  sc.lr = lr, sc.eps = eps, sc.decay = weight_decay;
  sc.beta1 = static_cast<float>(beta1), sc.beta2 = static_cast<float>(beta2);
  sc.c1 = static_cast<float>(1.0 - beta1), sc.c2 = static_cast<float>(1.0 - beta2);
  sc.one = 1.f;
  sc.lr_dev = lr_dev, sc.step_dev = step_dev, sc.grad_scale = grad_scale_dev;
  sc.log_beta1 = static_cast<float>(std::log(beta1));
  sc.log_beta2 = static_cast<float>(std::log(beta2));
  if (!step_dev) {
    sc.bc1 = static_cast<float>(1.0 - std::pow(beta1, static_cast<double>(step)));
    sc.sqrt_bc2 = static_cast<float>(std::sqrt(1.0 - std::pow(beta2, static_cast<double>(step))));
  }
  sc.seed = seed;
  AdamTensor t[kAdamTensors];
  for (int first = 0; first < n; first += kAdamTensors) {
    sc.first = static_cast<uint32_t>(first);
    sc.n = n - first < kAdamTensors ? n - first : kAdamTensors;
    for (int i = 0; i < sc.n; ++i) {
      const int k = first + i;
      t[i] = AdamTensor{p[k], g[k], m[k], v[k], e8 ? m_scale[k] : nullptr, e8 ? v_scale[k] : nullptr,
                        copy ? static_cast<uint16_t*>(copy[k]) : nullptr, sizes[k], 0};
    }
    if (launch_adamw(t, sc, param_type, grad_type, state_type, static_cast<cudaStream_t>(stream)) != cudaSuccess)
      return UF_CUDA_ERROR;
  }
  return UF_OK;
}

}  // extern "C"
