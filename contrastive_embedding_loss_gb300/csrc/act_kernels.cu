// act_kernels.cu -- the elementwise halves of the backward passes: dz = dy act'(z) with its
// column sums (the bias gradient), and the gated block's [dg | du].
//
// Bound by HBM, once the activations go two elements at a time: every array is read or written
// once, 16 bytes a thread and access.  A block of act_bwd owns up to 256 columns (8 a thread) and
// a range of rows (8 or more at a time); its column sums stay in registers, are joined across the
// row lanes in shared memory and written as one row of partial sums, which the column-sum kernel
// adds in a fixed order.  16384 x 4096 with gelu: 66 us (403 MB, 6.1 TB/s); the gated block's pass
// over 16384 x 2816: 64 us (461 MB).
//
// dz and [dg | du] are rounded to bf16, an fp32 dy's too, because the products that read them take
// bf16 operands: in fp32 they would go by tf32 at half the rate, or as two bf16 terms at a third of it.
// It puts the gradients 2.3e-3 of their norm from the exact ones, where the rounding of the outputs
// alone makes 1.7e-3.  The bias gradient sums the unrounded values.
#include <algorithm>
#include "layers.cuh"

namespace ufc {
namespace actk {

// Column groups (of 8) of a block, and its rows at a time.
__host__ __device__ constexpr int col_groups(int64_t n) { return n >= 256 ? 32 : static_cast<int>(n / 8); }
__host__ __device__ constexpr int row_lanes(int64_t n) { return 256 / col_groups(n); }

template <typename T>
struct alignas(16) Eight {
  T v[8];
};
constexpr int kBlocksPerSm = 4;  // resident: one wave
template <typename GT>
__global__ void __launch_bounds__(256, kBlocksPerSm) act_bwd_kernel(const ActBwdParams p, const int64_t rows_per_block) {
  griddep_enter();
  __shared__ float red[256 * 8];  // [row lane][column]
  const int groups = col_groups(p.n), lanes = row_lanes(p.n);
  const int g = threadIdx.x % groups, w = threadIdx.x / groups;
  const int64_t c = (static_cast<int64_t>(blockIdx.x) * groups + g) * 8;
  const int64_t r0 = blockIdx.y * rows_per_block;
  const int64_t r1 = r0 + rows_per_block < p.rows ? r0 + rows_per_block : p.rows;
  float2 sum[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) sum[j] = both(0.f);
  if (c < p.n && w < lanes) {
    for_act(p.pre ? p.act : kActNone, [&](auto act_c) {
      constexpr int ACT = decltype(act_c)::value;
      // two rows' loads ahead of the first store, which loads may not pass (three or four take
      // registers that resident threads need more)
      constexpr int kRows = 2;
      for (int64_t r = r0 + w; r < r1; r += kRows * lanes) {
        Eight<GT> dy[kRows];
        uint4 z[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i)
          if (r + i * lanes < r1) {
            dy[i] = *reinterpret_cast<const Eight<GT>*>(static_cast<const GT*>(p.dy) + (r + i * lanes) * p.lddy + c);
            if constexpr (ACT != kActNone) z[i] = *reinterpret_cast<const uint4*>(p.pre + (r + i * lanes) * p.ldp + c);
          }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          if (r + i * lanes >= r1) break;
          float d[8];
          load8(reinterpret_cast<const GT*>(&dy[i]), d);
          if constexpr (ACT != kActNone) {
            float v[8];
            unpack8(z[i], v);
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
              float2 a, da;
              act_grad2<ACT>(make_float2(v[j], v[j + 1]), a, da);
              // (the sum's own product: the same bits whether dz is asked for or not)
              sum[j / 2] = fma2(make_float2(d[j], d[j + 1]), da, sum[j / 2]);
              const float2 dz = mul2(make_float2(d[j], d[j + 1]), da);
              d[j] = dz.x, d[j + 1] = dz.y;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] = add2(sum[j], make_float2(d[2 * j], d[2 * j + 1]));
          }
          if (p.dz) store8(p.dz + (r + i * lanes) * p.ldz + c, d);
        }
      }
    });
  }
  if (!p.part) return;
  if (w < lanes) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      red[(w * groups + g) * 8 + 2 * j] = sum[j].x;
      red[(w * groups + g) * 8 + 2 * j + 1] = sum[j].y;
    }
  }
  __syncthreads();
  const int64_t col = static_cast<int64_t>(blockIdx.x) * groups * 8 + threadIdx.x;
  if (static_cast<int>(threadIdx.x) < groups * 8 && col < p.n) {
    float v = 0.f;
    for (int i = 0; i < lanes; ++i) v += red[i * groups * 8 + threadIdx.x];
    p.part[static_cast<int64_t>(blockIdx.y) * p.n + col] = v;
  }
}

__global__ void __launch_bounds__(256) gated_kernel(const GatedActBwdParams p) {
  griddep_enter();
  const int64_t per_row = p.n / 8;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t r = i / per_row, c = (i - r * per_row) * 8;
  if (r >= p.rows) return;
  float dh[8], g[8], u[8];
  load8(p.dh + r * p.lddh + c, dh);
  load8(p.pre + r * p.ldp + c, g);
  load8(p.pre + r * p.ldp + p.n + c, u);
  for_act(p.act, [&](auto act_c) {
    constexpr int ACT = decltype(act_c)::value;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      float2 a, da;
      act_grad2<ACT>(make_float2(g[j], g[j + 1]), a, da);
      const float2 d = make_float2(dh[j], dh[j + 1]);
      const float2 dg = mul2(mul2(d, make_float2(u[j], u[j + 1])), da), du = mul2(d, a);
      g[j] = dg.x, g[j + 1] = dg.y, u[j] = du.x, u[j + 1] = du.y;
    }
  });
  store8(p.d + r * 2 * p.n + c, g);
  store8(p.d + r * 2 * p.n + p.n + c, u);
}

}  // namespace actk

int64_t act_bwd_blocks(int64_t rows, int64_t n) {
  const int64_t cols = (n + 255) / 256;
  const int64_t want = std::max<int64_t>(152 * actk::kBlocksPerSm / cols, 1);
  const int64_t turn = 2 * actk::row_lanes(n);  // two rows a thread at least
  const int64_t most = (rows + turn - 1) / turn;
  const int64_t b = want < most ? want : most;
  return b < 1 ? 1 : b;
}

cudaError_t launch_act_bwd(const ActBwdParams& p, cudaStream_t stream) {
  const int64_t blocks = act_bwd_blocks(p.rows, p.n);
  const int64_t per = (p.rows + blocks - 1) / blocks;
  const int64_t width = 8 * actk::col_groups(p.n);
  const dim3 grid(static_cast<unsigned>((p.n + width - 1) / width), static_cast<unsigned>(blocks));
  if (p.dy_type == kF32) return launch_pdl(actk::act_bwd_kernel<float>, grid, dim3(256), 0, stream, 1, p, per);
  return launch_pdl(actk::act_bwd_kernel<uint16_t>, grid, dim3(256), 0, stream, 1, p, per);
}

cudaError_t launch_gated_act_bwd(const GatedActBwdParams& p, cudaStream_t stream) {
  const int64_t items = p.rows * (p.n / 8);
  return launch_pdl(actk::gated_kernel, dim3(static_cast<unsigned>((items + 255) / 256)), dim3(256), 0, stream, 1, p);
}

}  // namespace ufc
