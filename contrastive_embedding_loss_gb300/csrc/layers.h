// layers.h -- parameters and launchers of the head's operators and the optimizer (internal).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "launch.h"

namespace ufc {

enum Dtype : int { kBf16 = 0, kF32 = 1, kE4m3 = 2 };  // == uf_dtype_t
enum Act : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };  // == uf_activation_t

// ---------------------------------------------------------------- norm_kernels.cu
constexpr int kNormMaxWidth = 16384;

struct NormFwdParams {
  const void* x;
  const void* res;
  const void* weight;
  void* y;
  void* s;
  float* y_scale;
  float* rstd;
  int64_t ldx, ldr, ldy, lds, rows;
  int width, x_type, stream_type, weight_type, y_type;
  float eps;
};
cudaError_t norm_kernels_setup();
cudaError_t launch_norm_fwd(const NormFwdParams& p, cudaStream_t stream);

struct NormRowsBwdParams {
  const void* dy;
  const void* s;
  const void* weight;
  const float* rstd;
  const void* ds;
  void* dx;
  float* part;     // [blocks][width] partial weight gradients, or NULL
  float* dweight;  // with part
  int64_t lddy, lds, ldds, lddx, rows;
  int width, dy_type, stream_type, weight_type;
};
// The most blocks the backward's grid has: a function of the problem alone (it sizes the workspace).
int64_t norm_bwd_blocks(int64_t rows, int width);
cudaError_t launch_norm_rows_bwd(const NormRowsBwdParams& p, cudaStream_t stream);

// out[c] = sum_b part[b][c], in a fixed order.
cudaError_t launch_col_sum(const float* part, int64_t blocks, int64_t width, float* out, cudaStream_t stream);

// ---------------------------------------------------------------- act_kernels.cu
// dz = dy act'(z) in bf16, and its column sums (unrounded).
struct ActBwdParams {
  const void* dy;
  const uint16_t* pre;  // NULL: dz = dy
  uint16_t* dz;         // [rows][ldz], or NULL (only the column sums)
  float* part;          // [blocks][n] partial column sums, or NULL
  int64_t lddy, ldp, ldz, rows, n;
  int dy_type, act;
};
int64_t act_bwd_blocks(int64_t rows, int64_t n);  // row blocks: rows of part
cudaError_t launch_act_bwd(const ActBwdParams& p, cudaStream_t stream);

// [dg | du] of the gated block, in bf16.
struct GatedActBwdParams {
  const uint16_t* dh;
  const uint16_t* pre;  // [rows][2 n]: [g | u]
  uint16_t* d;          // [rows][2 n]
  int64_t lddh, ldp, rows, n;
  int act;
};
cudaError_t launch_gated_act_bwd(const GatedActBwdParams& p, cudaStream_t stream);

// ---------------------------------------------------------------- dense_kernel.cu
// What follows a matrix product's accumulator (linear: z = acc xs ws + bias, y = act(z) + res;
// gated: h = act(g) u).
struct Epilogue {
  int act;
  int bias_type;
  const float* x_scale;
  const float* w_scale;
  const void* bias;
  const uint16_t* res;
  uint16_t* y;
  uint16_t* pre;
  int64_t ldr, ldy, ldp;
  int64_t rows, cols;  // of y; gated: pre has 2 cols columns
};

// Products of a launch.  kDenseLinear(8): y from K-major bf16 (e4m3) operands.  kDenseGated: of 2
// cols columns, the gate's and the up projection's.  kDenseGrads: product 0 with a K-major A
// (dx = dz W), product 1 with an MN-major one (dW = dz^T x; the contraction index selects the
// row), both with an MN-major B; either may be empty.
enum DenseKind : int { kDenseLinear = 0, kDenseLinear8 = 1, kDenseGated = 2, kDenseGrads = 3 };
constexpr int kDensePairs = 76;    // CTA pairs of a GB300: a constant, so that the workspace's size is one too
constexpr int kDenseClasses = 4;   // whole tiles and split ones of two products

// D[rows][cols] = A B^T over kdim.
struct DenseShape {
  int64_t rows, cols, kdim;
};
struct DensePlan {
  int bn;               // tile columns: 256, 128 or 64 (rows: 256)
  struct Product {
    int tiles_m, tiles_n;
    int chunks;         // 128-byte chunks of the contraction
    int full;           // the first tiles, computed whole
    int rest, splits;   // the others' contraction is split: split s takes chunks s, s + splits, ...
    size_t part_bytes;  // scratch of the splits
  } p[2];
};
// A pure function of the problem.
DensePlan plan_dense(const DenseShape* shapes, int n, DenseKind kind);

struct DenseParams {
  Epilogue e;
  int64_t up_row;      // gated: first row of the up projection in B
  float* part;         // [split][rest tile][256][tile columns] fp32
  int tiles_m, tiles_n, chunks, full, rest, splits;  // from the plan (set by the launcher)
};
struct DenseArgs {
  DenseParams p[2];
  struct Class {
    int units, k, rest;  // of product k: its whole tiles, or its split ones
  } classes[kDenseClasses];
  int listed;            // the units are dealt by count, else in turn
  uint16_t count[kDenseClasses][kDensePairs];
  int* status;
};
cudaError_t dense_kernel_setup();
// Tensor maps, all with the swizzle of their box's width.
struct DenseMaps {
  CUtensorMap a;     // boxes of 128 rows x 128 bytes (K-major) or 64 x 64 elements (MN-major)
  CUtensorMap b;     // bn / 2 rows x 128 bytes (K-major) or 64 x 64 elements (MN-major)
  CUtensorMap y;     // stores: dense_store_cols columns x 32 rows
  CUtensorMap p0;    // pre, or the gate's half of it, as y
  CUtensorMap p1;    // the up projection's half
  CUtensorMap part;  // the scratch as rows of bn fp32 columns, 32 x 32
};
constexpr int dense_store_cols(int bn, bool gated) { return gated ? (bn == 256 ? 64 : 32) : (bn == 64 ? 32 : 64); }
// maps, products: n of each.
cudaError_t launch_dense(const DenseMaps* maps, const DenseParams* products, const DensePlan& plan, int n, DenseKind kind,
                         int* status, cudaStream_t stream);

// ---------------------------------------------------------------- skinny_kernel.cu
// Whether few rows go this way: up to 16 always, up to 32 where the kernel's blocks fit the GPU at
// once (17 to 32 rows of 4096 x 4096: 11.6 to 12.2 us against 14.0 by the tiles, of 1024 x 1024 4.3 to
// 4.8 against 7.8; two waves, as of gated 1024 x 8192, 13.7 to 14.8 against 12.1).
bool skinny_takes(int64_t rows, int64_t k_bytes, int64_t cols);
struct SkinnyParams {
  Epilogue e;
  const uint8_t* x;
  const uint8_t* w;
  int64_t ldx_bytes, ldw_bytes;
  int64_t k_bytes;
  int64_t up_row;
  int wk;              // warps of a block that share a contraction (a power of two)
  int cluster;         // CTAs that share a contraction
  int64_t span;        // bytes of the contraction per CTA of the cluster
};
cudaError_t launch_skinny(const SkinnyParams& p, int elem_bytes, bool gated, cudaStream_t stream);

// ---------------------------------------------------------------- adamw_kernel.cu
constexpr int kAdamBlock = 256;
constexpr int kAdamTensors = 256;  // tensors of one launch
struct AdamTensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  uint16_t* copy;
  int64_t size;
  int64_t wide;  // set by the launcher
};
struct AdamScalars {
  float lr, beta1, beta2, c1, c2, eps, decay;  // c1, c2: 1 - beta1, 1 - beta2
  float one;  // 1, as a value that the compiler does not know
  float log_beta1, log_beta2;
  float bc1, sqrt_bc2;  // 1 - beta1^t, sqrt(1 - beta2^t) (without step_dev)
  const float* lr_dev;
  const int64_t* step_dev;
  const float* grad_scale;
  uint32_t seed;
  uint32_t first;  // index of the launch's first tensor
  int n;
};
// tensors: host array of sc.n <= kAdamTensors entries.
cudaError_t launch_adamw(const AdamTensor* tensors, const AdamScalars& sc, int param_type, int grad_type, int state_type,
                         cudaStream_t stream);

}  // namespace ufc
