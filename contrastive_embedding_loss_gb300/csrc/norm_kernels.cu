// norm_kernels.cu -- RMS norm with the residual's addition, forward and backward.
//
//   forward:   s = x + r,  rho = (mean s^2 + eps)^-1/2,  y = s rho w   (bf16, or e4m3 with a
//              scale a row)
//   backward:  g = dy w,  xh = s rho,  dx = rho (g - xh mean(g xh)) + d_stream,
//              dw = sum_rows dy xh
//
// Both are bound by HBM.  A row stays in registers between its reduction and its output, so
// every array crosses HBM once: TPR threads share a row, 16 or 32 values each at most (TPR = 32 to
// 1024 by the width).  The backward's blocks walk rows with a stride and keep their columns'
// part of dw in registers; the blocks' parts are summed by a second small kernel in a fixed order.
// 16384 x 4096 with a bf16 residual to e4m3: 68 us (470 MB, 6.9 TB/s); the backward of 65536 x 1024
// with an fp32 stream: 139 us (940 MB, 6.7 TB/s).
//
// Rows of any width and alignment: a row is cut into a head of up to 7 elements that ends at a
// 16-byte boundary, vectors of 8, and a tail of up to 7; head and tail take one scalar access of
// one thread each.  That needs every array of the call to have the same misalignment in elements
// (contiguous tensors have); else all accesses are scalar.  A head's length repeats every 8 rows,
// and the backward's stride is a multiple of 8 rows, so a thread keeps its columns.
#include "layers.cuh"

namespace ufc {
namespace norm {

constexpr int kPerThread = 32;  // values of a row per thread at most

template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  if constexpr (TPR > 32) {
    __syncthreads();  // the previous reduction's reads are done
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) v += red[i];
  }
  return v;
}
template <int TPR>
__device__ __forceinline__ float row_max(float v, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
  if constexpr (TPR > 32) {
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < TPR / 32; ++i) v = fmaxf(v, red[i]);
  }
  return v;
}

struct NoRes {};

// Where a thread's values lie in its row.  VEC = 8: vectors from the head's end on, and one
// element of the head or tail for some threads; VEC = 1: single elements, TPR apart.
template <int TPR, int VEC>
struct Cut {
  int head, width, extra;  // extra: this thread's element of the head or tail, or -1
  template <typename T>
  __device__ __forceinline__ Cut(const T* row, int width_, int lane) : head(0), width(width_), extra(-1) {
    if constexpr (VEC == 8) {
      head = static_cast<int>(0u - static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) / sizeof(T))) & 7;
      if (head > width) head = width;
      const int tail = head + ((width - head) & ~7);
      if (lane < head) extra = lane;
      if (lane >= 8 && lane - 8 < width - tail) extra = tail + lane - 8;
    }
  }
  __device__ __forceinline__ int at(int i, int lane) const { return head + (i * TPR + lane) * VEC; }
  __device__ __forceinline__ bool in(int c) const { return c + VEC <= width; }
};

// VEC consecutive values as floats.
template <int VEC, typename T>
__device__ __forceinline__ void load(const T* p, float* v) {
  if constexpr (VEC == 8) {
    load8(p, *reinterpret_cast<float(*)[8]>(v));
  } else {
    v[0] = load1(p);
  }
}
template <int VEC, typename T>
__device__ __forceinline__ void store(T* p, const float* v) {
  if constexpr (VEC == 8) {
    store8(p, *reinterpret_cast<const float(*)[8]>(v));
  } else {
    store1(p, v[0]);
  }
}
__device__ __forceinline__ float weight1(const void* w, int type, int c) {
  return type == kF32 ? load1(static_cast<const float*>(w) + c) : load1(static_cast<const uint16_t*>(w) + c);
}
// VEC weights from column c on (VEC = 8: c is the head's length plus a multiple of 8, the weight
// itself 16-byte aligned).
template <int VEC>
__device__ __forceinline__ void load_weight(const void* w, int type, int c, int head, int width, float* v) {
  if constexpr (VEC == 1) {
    v[0] = weight1(w, type, c);
  } else {
    if (head == 0) {
      if (type == kF32)
        load<8>(static_cast<const float*>(w) + c, v);
      else
        load<8>(static_cast<const uint16_t*>(w) + c, v);
    } else if (type == kF32 && c + 11 < width) {
      // three aligned float4 that cover the 8 floats, and the 8 out of them
      const int sh = head & 3;
      const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(w) + (c - sh));
      const float4 f0 = q[0], f1 = q[1], f2 = q[2];
      const float f[12] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w, f2.x, f2.y, f2.z, f2.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = sh == 0 ? f[j] : sh == 1 ? f[j + 1] : sh == 2 ? f[j + 2] : f[j + 3];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = weight1(w, type, c + j);
    }
  }
}

template <typename XT, typename RT, int TPR, int VEC>
__global__ void __launch_bounds__(TPR == 32 ? 128 : TPR) fwd_kernel(const NormFwdParams p) {
  griddep_enter();
  constexpr int kChunks = kPerThread / VEC;
  constexpr bool kRes = !std::is_same<RT, NoRes>::value;
  using ResT = typename std::conditional<kRes, RT, float>::type;
  __shared__ float red[TPR / 32];
  const int lane = threadIdx.x % TPR;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / TPR) + threadIdx.x / TPR;
  if (row >= p.rows) return;  // whole warps (TPR = 32) or blocks
  const XT* x = static_cast<const XT*>(p.x) + row * p.ldx;
  const ResT* r = kRes ? static_cast<const ResT*>(p.res) + row * p.ldr : nullptr;
  ResT* out = kRes ? static_cast<ResT*>(p.s) + row * p.lds : nullptr;
  const Cut<TPR, VEC> cut(x, p.width, lane);
  float s[kPerThread], e = 0.f;
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = cut.at(i, lane);
    if (cut.in(c)) {
      load<VEC>(x + c, s + i * VEC);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) s[i * VEC + j] = 0.f;
    }
  }
  if (cut.extra >= 0) e = load1(x + cut.extra);
  if constexpr (kRes) {
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = cut.at(i, lane);
      if (cut.in(c)) {
        float v[VEC];
        load<VEC>(r + c, v);
#pragma unroll
        for (int j = 0; j < VEC; ++j) s[i * VEC + j] += v[j];
      }
    }
    if (cut.extra >= 0) {
      e += load1(r + cut.extra);
      store1(out + cut.extra, e);
    }
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = cut.at(i, lane);
      if (cut.in(c)) store<VEC>(out + c, s + i * VEC);
    }
  }
  float q = e * e;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) q = fmaf(s[i], s[i], q);
  q = row_sum<TPR>(q, red);
  const float rho = rsqrtf(q / static_cast<float>(p.width) + p.eps);
  if (p.rstd && lane == 0) p.rstd[row] = rho;
  // bf16: y = s (rho w).  e4m3: the codes 448 y / max |y| do not depend on rho, of which only the power
  // of two goes into y, the rest into the row's scale: one rounding less before the code is chosen, at
  // y's own size.  (A rho of 0, infinity or NaN goes to the scale.)
  const bool e4m3 = p.y_type == kE4m3;
  const float two = rho > 0.f && rho < __int_as_float(0x7F800000) ? __uint_as_float(__float_as_uint(rho) & 0x7F800000u) : 1.f;
  const float by = e4m3 ? two : rho;
  if (cut.extra >= 0) e *= by * weight1(p.weight, p.weight_type, cut.extra);
  float top = fabsf(e);
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = cut.at(i, lane);
    if (cut.in(c)) {
      float w[VEC];
      load_weight<VEC>(p.weight, p.weight_type, c, cut.head, p.width, w);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        s[i * VEC + j] *= by * w[j];
        top = fmaxf(top, fabsf(s[i * VEC + j]));
      }
    }
  }
  if (!e4m3) {
    uint16_t* y = static_cast<uint16_t*>(p.y) + row * p.ldy;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = cut.at(i, lane);
      if (cut.in(c)) store<VEC>(y + c, s + i * VEC);
    }
    if (cut.extra >= 0) store1(y + cut.extra, e);
    return;
  }
  top = row_max<TPR>(top, red);
  // (of a row whose y are all below 2^-116 the quotient is infinite: they count as zeros)
  if (top < 0x1p-116f) top = 0.f;
  const float inv = top > 0.f ? 448.f / top : 0.f;
  if (lane == 0) p.y_scale[row] = rho / two * top / 448.f;
  uint8_t* y = static_cast<uint8_t*>(p.y) + row * p.ldy;
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = cut.at(i, lane);
    if (cut.in(c)) {
      const float* v = s + i * VEC;
      if constexpr (VEC == 8) {
        uint2 o;
        o.x = pack_e4m3(v[0] * inv, v[1] * inv) | pack_e4m3(v[2] * inv, v[3] * inv) << 16;
        o.y = pack_e4m3(v[4] * inv, v[5] * inv) | pack_e4m3(v[6] * inv, v[7] * inv) << 16;
        *reinterpret_cast<uint2*>(y + c) = o;
      } else {
        y[c] = static_cast<uint8_t>(pack_e4m3(v[0] * inv, 0.f));
      }
    }
  }
  if (cut.extra >= 0) y[cut.extra] = static_cast<uint8_t>(pack_e4m3(e * inv, 0.f));
}

// The backward's blocks: kBwdBlock threads, or one row's if it has more.  A thread's sums of
// dy xh over its rows stay in registers; at the end the block writes one row of parts.
constexpr int kBwdBlock = 128;
template <int TPR>
constexpr int bwd_block() {
  return TPR < kBwdBlock ? kBwdBlock : TPR;
}
template <int TPR, int VEC, int N>
__device__ __forceinline__ void write_part(float* part, const Cut<TPR, VEC>& cut, int lane, const float (&dw)[N], float dwe,
                                           float* dw_sum) {
  constexpr int kGroups = bwd_block<TPR>() / TPR;
  if constexpr (kGroups > 1) {
    // the block's row groups' sums, one after another (their heads may differ)
    for (int c = threadIdx.x; c < cut.width; c += kBwdBlock) dw_sum[c] = 0.f;
    for (int w = 0; w < kGroups; ++w) {
      __syncthreads();
      if (static_cast<int>(threadIdx.x / TPR) == w) {
#pragma unroll
        for (int i = 0; i < N / VEC; ++i) {
          const int c = cut.at(i, lane);
          if (cut.in(c))
#pragma unroll
            for (int j = 0; j < VEC; ++j) dw_sum[c + j] += dw[i * VEC + j];
        }
        if (cut.extra >= 0) dw_sum[cut.extra] += dwe;
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < cut.width; c += kBwdBlock) part[c] = dw_sum[c];
  } else {
#pragma unroll
    for (int i = 0; i < N / VEC; ++i) {
      const int c = cut.at(i, lane);
      if (cut.in(c))
#pragma unroll
        for (int j = 0; j < VEC; ++j) part[c + j] = dw[i * VEC + j];
    }
    if (cut.extra >= 0) part[cut.extra] = dwe;
  }
}

// Sum over the TPR threads of a row; red: one float per warp of the block, twice (alternating, so
// that one barrier a sum is enough).
template <int TPR>
__device__ __forceinline__ float group_sum(float v, float* red, uint32_t turn) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  if constexpr (TPR > 32) {
    constexpr int kWarps = bwd_block<TPR>() / 32;
    float* slot = red + (turn & 1) * kWarps;
    if ((threadIdx.x & 31) == 0) slot[threadIdx.x >> 5] = v;
    named_bar_sync(1 + threadIdx.x / TPR, TPR);
    const int first = threadIdx.x / TPR * (TPR / 32);
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) v += slot[first + i];
  }
  return v;
}

// 16 bytes asynchronously.  An fp32 array's 32 bytes a thread go as two of these, whose sectors
// the first leaves in L1 for the second; 16-bit arrays pass L1 by.
template <bool PAIR>
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  if constexpr (PAIR)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void ld_shared8(uint32_t at, uint32_t piece, const uint16_t*, float (&v)[8]) {
  uint4 q;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(at) : "memory");
  unpack8(q, v);
}
__device__ __forceinline__ void ld_shared8(uint32_t at, uint32_t piece, const float*, float (&v)[8]) {
  const float4 a = ld_shared_v4f(at), b = ld_shared_v4f(at + piece);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// Arrays in step (vector accesses).  What bounds the backward is how much is on its way: held in
// registers until the row's reduction, one row a warp leaves the memory idle through reductions
// and stores (bf16 rows ran at 3.7 TB/s so).  So every thread copies its own pieces of its next
// row into shared memory asynchronously while it works on this one, reads them back twice (for
// the reduction and for dx), and needs no barrier for it.  16 values a thread: with 32 the rings
// leave room for only 8 warps an SM, too few to cover their own latencies (250 us for 65536 fp32
// rows of 1024).
template <int TPR, int N>
constexpr int bwd_per_sm() {  // blocks whose registers fit
  const int threads = N == 16 && TPR > 128 ? 768 : 512;
  return threads < bwd_block<TPR>() ? 1 : threads / bwd_block<TPR>();
}
template <typename GT, typename ST, int TPR, int N>
__global__ void __launch_bounds__(bwd_block<TPR>(), (bwd_per_sm<TPR, N>()))
    bwd_kernel(const NormRowsBwdParams p, const int chunks, const int stages) {
  griddep_enter();
  constexpr int kBlock = bwd_block<TPR>();
  constexpr int kRows = kBlock / TPR;
  constexpr int kChunks = N / 8;
  constexpr uint32_t kPiece = kBlock * 16;  // piece q of thread t lies at q kPiece + 16 t
  constexpr uint32_t kS = sizeof(ST) / 2, kG = sizeof(GT) / 2;  // pieces per 8 values
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[2 * kBlock / 32];
  __shared__ float dw_sum[kRows > 1 ? N * TPR : 1];
  const int lane = threadIdx.x % TPR;
  const uint32_t per_chunk = (kS + kG + (p.ds ? kS : 0)) * kPiece;
  const uint32_t mine = smem_u32(ring) + threadIdx.x * 16;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / TPR;
  const Cut<TPR, 8> cut(static_cast<const ST*>(p.s) + row * p.lds, p.width, lane);
  const bool edge = cut.extra >= 0;
  // the thread's columns stay the same: its weights and its sums of dy xh
  float w[N], dw[N], dwe = 0.f;
  const float we = edge ? weight1(p.weight, p.weight_type, cut.extra) : 0.f;
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = cut.at(i, lane);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[i * 8 + j] = dw[i * 8 + j] = 0.f;
    if (cut.in(c)) load_weight<8>(p.weight, p.weight_type, c, cut.head, p.width, w + i * 8);
  }

  float rho_n = 0.f, xe_n = 0.f, ge_n = 0.f, de_n = 0.f;  // the next row's statistics and edge elements
  auto fetch = [&](int64_t r, uint32_t stage) {
    if (r < p.rows) {
      const ST* sp = static_cast<const ST*>(p.s) + r * p.lds;
      const GT* gp = static_cast<const GT*>(p.dy) + r * p.lddy;
      const ST* dp = p.ds ? static_cast<const ST*>(p.ds) + r * p.ldds : nullptr;
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        const int c = cut.at(i, lane);
        if (!cut.in(c)) continue;
        const uint32_t at = mine + (stage * chunks + i) * per_chunk;
#pragma unroll
        for (uint32_t k = 0; k < kS; ++k) cp_async16<kS == 2>(at + k * kPiece, reinterpret_cast<const uint8_t*>(sp + c) + 16 * k);
#pragma unroll
        for (uint32_t k = 0; k < kG; ++k)
          cp_async16<kG == 2>(at + (kS + k) * kPiece, reinterpret_cast<const uint8_t*>(gp + c) + 16 * k);
        if (dp)
#pragma unroll
          for (uint32_t k = 0; k < kS; ++k)
            cp_async16<kS == 2>(at + (kS + kG + k) * kPiece, reinterpret_cast<const uint8_t*>(dp + c) + 16 * k);
      }
      rho_n = p.rstd[r];
      if (edge) {
        xe_n = load1(sp + cut.extra);
        ge_n = load1(gp + cut.extra);
        if (dp) de_n = load1(dp + cut.extra);
      }
    }
    cp_async_commit();
  };

  fetch(row, 0);
  for (uint32_t it = 0; row < p.rows; row += stride, ++it) {
    const float rho = rho_n, se = xe_n, xe = xe_n * rho_n, de = de_n;
    float ge = ge_n;
    if (stages == 2) {
      fetch(row + stride, (it + 1) & 1);
      cp_async_wait<1>();  // this row's pieces have landed
    } else {
      cp_async_wait<0>();
    }
    const uint32_t base = mine + (stages == 2 ? it & 1 : 0) * chunks * per_chunk;
    dwe = fmaf(ge, xe, dwe);
    ge *= we;
    float dot = xe * ge;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      if (cut.in(cut.at(i, lane))) {
        float x[8], g[8];
        ld_shared8(base + i * per_chunk, kPiece, static_cast<const ST*>(nullptr), x);
        ld_shared8(base + i * per_chunk + kS * kPiece, kPiece, static_cast<const GT*>(nullptr), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float gx = g[j] * (x[j] * rho);
          dw[i * 8 + j] += gx;
          dot = fmaf(gx, w[i * 8 + j], dot);
        }
      }
    }
    // dx = rho g + d_stream - (rho^2 mean(g xh)) s
    const float along = -rho * rho * group_sum<TPR>(dot, red, it) / static_cast<float>(p.width);
    ST* dx = static_cast<ST*>(p.dx) + row * p.lddx;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = cut.at(i, lane);
      if (cut.in(c)) {
        float x[8], g[8], o[8];
        ld_shared8(base + i * per_chunk, kPiece, static_cast<const ST*>(nullptr), x);
        ld_shared8(base + i * per_chunk + kS * kPiece, kPiece, static_cast<const GT*>(nullptr), g);
        if (p.ds) {
          ld_shared8(base + i * per_chunk + (kS + kG) * kPiece, kPiece, static_cast<const ST*>(nullptr), o);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = fmaf(along, x[j], fmaf(rho * w[i * 8 + j], g[j], o[j]));
        store8(dx + c, o);
      }
    }
    if (edge) store1(dx + cut.extra, fmaf(along, se, fmaf(rho, ge, de)));
    if (stages == 1) fetch(row + stride, 0);
  }
  cp_async_wait<0>();
  if (p.part) write_part(p.part + static_cast<int64_t>(blockIdx.x) * p.width, cut, lane, dw, dwe, dw_sum);
}

// Arrays of different misalignments: element by element, through registers.
template <typename GT, typename ST, int TPR>
__global__ void __launch_bounds__(TPR == 32 ? 128 : TPR) bwd_scalar_kernel(const NormRowsBwdParams p) {
  griddep_enter();
  constexpr int kRows = TPR == 32 ? 4 : 1;
  constexpr int kGroup = 8;  // values of d_stream loaded at once
  __shared__ float red[TPR / 32];
  __shared__ float dw_sum[TPR == 32 ? kPerThread * 32 : 1];
  const int lane = threadIdx.x % TPR;
  float dw[kPerThread];
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) dw[i] = 0.f;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / TPR;
  const Cut<TPR, 1> cut(static_cast<const ST*>(p.s), p.width, lane);
  for (; row < p.rows; row += stride) {
    const GT* dy = static_cast<const GT*>(p.dy) + row * p.lddy;
    const ST* sp = static_cast<const ST*>(p.s) + row * p.lds;
    const ST* ds = p.ds ? static_cast<const ST*>(p.ds) + row * p.ldds : nullptr;
    const float rho = p.rstd[row];
    float xh[kPerThread], g[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int c = cut.at(i, lane);
      xh[i] = cut.in(c) ? load1(sp + c) : 0.f;
      g[i] = cut.in(c) ? load1(dy + c) : 0.f;
    }
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int c = cut.at(i, lane);
      if (cut.in(c)) {
        xh[i] *= rho;
        dw[i] = fmaf(g[i], xh[i], dw[i]);
        g[i] *= weight1(p.weight, p.weight_type, c);
        dot = fmaf(g[i], xh[i], dot);
      }
    }
    const float along = -row_sum<TPR>(dot, red) / static_cast<float>(p.width);
    ST* dx = static_cast<ST*>(p.dx) + row * p.lddx;
    // a load behind a store to memory it might share waits for a round trip: eight loads at a time
#pragma unroll
    for (int i0 = 0; i0 < kPerThread; i0 += kGroup) {
      float a[kGroup];
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        const int c = cut.at(i0 + i, lane);
        a[i] = ds && cut.in(c) ? load1(ds + c) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        const int c = cut.at(i0 + i, lane);
        if (cut.in(c)) store1(dx + c, fmaf(rho, fmaf(along, xh[i0 + i], g[i0 + i]), a[i]));
      }
    }
  }
  if (p.part) write_part(p.part + static_cast<int64_t>(blockIdx.x) * p.width, cut, lane, dw, 0.f, dw_sum);
}

// 32 columns a block, 32 rows of parts at a time, eight loads in flight a thread.
__global__ void __launch_bounds__(1024) col_sum_kernel(const float* part, int64_t blocks, int64_t width, float* out) {
  griddep_enter();
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float v = 0.f;
  if (c < width) {
#pragma unroll 8
    for (int64_t b = w; b < blocks; b += 32) v += part[b * width + c];
  }
  red[w][lane] = v;
  __syncthreads();
  v = red[lane][w];  // column w of the block, part lane
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + w;
  if (lane == 0 && col < width) out[col] = v;
}

int threads_per_row(int width) {
  return width <= 32 * kPerThread ? 32 : width <= 128 * kPerThread ? 128 : width <= 256 * kPerThread ? 256 : 512;
}

// Whether array p (element size elem, row stride ld) has 16-byte boundaries at the same elements
// of every row as q, with 8 elements to a vector.
bool in_step(const void* p, int64_t ld, int elem, const void* q, int64_t ldq, int elem_q) {
  const uint64_t m = elem == 4 ? 4 : 8;
  const uint64_t a = reinterpret_cast<uintptr_t>(p) / elem, b = reinterpret_cast<uintptr_t>(q) / elem_q;
  return (a - b) % m == 0 && static_cast<uint64_t>(ld - ldq) % m == 0;
}
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
int elem_of(int type) { return type == kF32 ? 4 : type == kBf16 ? 2 : 1; }

template <typename XT, typename RT, int VEC>
cudaError_t fwd(const NormFwdParams& p, cudaStream_t stream) {
  const int tpr = threads_per_row(p.width);
  if (tpr == 32)
    return launch_pdl(fwd_kernel<XT, RT, 32, VEC>, dim3(static_cast<unsigned>((p.rows + 3) / 4)), dim3(128), 0, stream, 1,
                      p);
  const dim3 grid(static_cast<unsigned>(p.rows));
  if (tpr == 128) return launch_pdl(fwd_kernel<XT, RT, 128, VEC>, grid, dim3(128), 0, stream, 1, p);
  if (tpr == 256) return launch_pdl(fwd_kernel<XT, RT, 256, VEC>, grid, dim3(256), 0, stream, 1, p);
  return launch_pdl(fwd_kernel<XT, RT, 512, VEC>, grid, dim3(512), 0, stream, 1, p);
}
template <int VEC>
cudaError_t fwd_types(const NormFwdParams& p, cudaStream_t stream) {
  if (!p.res) return p.x_type == kF32 ? fwd<float, NoRes, VEC>(p, stream) : fwd<uint16_t, NoRes, VEC>(p, stream);
  return p.stream_type == kF32 ? fwd<uint16_t, float, VEC>(p, stream) : fwd<uint16_t, uint16_t, VEC>(p, stream);
}

// Blocks of the backward: as many as can be resident with their rings of rows.  A multiple of 8
// where blocks take several turns, so that a thread's rows keep one misalignment.
constexpr int kMostBlocksPerSm = 12;
int64_t bwd_blocks(int64_t rows, int rows_per_block, int per_sm) {
  // with few rows, no more than two blocks an SM until each has four turns: every block writes a
  // row of parts
  const int64_t most = 152 * per_sm, some = 152 * 2;
  const int64_t turns = (rows + rows_per_block - 1) / rows_per_block;
  const int64_t n = turns <= some ? turns : turns / 4 < some ? some : turns / 4 / 8 * 8;
  return n < 1 ? 1 : n < most ? n : most;
}
constexpr int kMostRing = 220 * 1024;  // bytes, beside the static arrays
template <typename GT, typename ST, int TPR, int N>
cudaError_t bwd_async(const NormRowsBwdParams& p, int64_t* blocks, cudaStream_t stream) {
  constexpr int kBlock = bwd_block<TPR>();
  const int chunks = (p.width / 8 + TPR - 1) / TPR;
  const int stage = chunks * static_cast<int>(8 * (sizeof(GT) + sizeof(ST) * (p.ds ? 2 : 1))) * kBlock;
  const int stages = 2 * stage <= kMostRing ? 2 : 1;  // (one: the longest rows with fp32 dy or stream)
  const int smem = stages * stage;
  // fp32 arrays need room in L1 for the other half of their sectors
  int per_sm = (sizeof(GT) + sizeof(ST) > 4 ? 168 : 220) * 1024 / (smem + 2 * 1024);
  per_sm = per_sm < bwd_per_sm<TPR, N>() ? per_sm : bwd_per_sm<TPR, N>();
  per_sm = per_sm < 1 ? 1 : per_sm > kMostBlocksPerSm ? kMostBlocksPerSm : per_sm;
  *blocks = bwd_blocks(p.rows, kBlock / TPR, per_sm);
  return launch_pdl(bwd_kernel<GT, ST, TPR, N>, dim3(static_cast<unsigned>(*blocks)), dim3(kBlock), smem, stream, 1, p, chunks,
                    stages);
}
// Calls f with the variant for a width.
template <int TPR, int N>
struct Variant {
  static constexpr int kTpr = TPR, kValues = N;
};
template <typename ST, typename F>
cudaError_t for_width(int width, F&& f) {
  if constexpr (sizeof(ST) == 2) {
    if (width <= 1024) return f(Variant<32, 32>{});
    if (width <= 4096) return f(Variant<128, 32>{});
    if (width <= 8192) return f(Variant<256, 32>{});
    return f(Variant<512, 32>{});
  } else {
    if (width <= 512) return f(Variant<32, 16>{});
    if (width <= 1024) return f(Variant<64, 16>{});
    if (width <= 2048) return f(Variant<128, 16>{});
    if (width <= 4096) return f(Variant<256, 16>{});
    if (width <= 8192) return f(Variant<512, 16>{});
    return f(Variant<1024, 16>{});
  }
}
// Every variant may take the largest ring: the limit is the function's, not a call's, so a call that
// set its own would race with other threads'.
template <typename GT, typename ST>
cudaError_t bwd_setup() {
  for (int width = 512; width <= kNormMaxWidth; width *= 2) {
    const cudaError_t e = for_width<ST>(width, [](auto v) {
      return cudaFuncSetAttribute(bwd_kernel<GT, ST, decltype(v)::kTpr, decltype(v)::kValues>,
                                  cudaFuncAttributeMaxDynamicSharedMemorySize, kMostRing);
    });
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}
template <typename GT, typename ST>
cudaError_t bwd(const NormRowsBwdParams& p, bool vec, int64_t* blocks, cudaStream_t stream) {
  if (vec)
    return for_width<ST>(p.width, [&](auto v) {
      return bwd_async<GT, ST, decltype(v)::kTpr, decltype(v)::kValues>(p, blocks, stream);
    });
  const int tpr = threads_per_row(p.width);
  *blocks = bwd_blocks(p.rows, tpr == 32 ? 4 : 1, tpr == 512 ? 1 : tpr == 256 ? 2 : 4);
  const dim3 grid(static_cast<unsigned>(*blocks));
  if (tpr == 32) return launch_pdl(bwd_scalar_kernel<GT, ST, 32>, grid, dim3(128), 0, stream, 1, p);
  if (tpr == 128) return launch_pdl(bwd_scalar_kernel<GT, ST, 128>, grid, dim3(128), 0, stream, 1, p);
  if (tpr == 256) return launch_pdl(bwd_scalar_kernel<GT, ST, 256>, grid, dim3(256), 0, stream, 1, p);
  return launch_pdl(bwd_scalar_kernel<GT, ST, 512>, grid, dim3(512), 0, stream, 1, p);
}

}  // namespace norm

cudaError_t launch_norm_fwd(const NormFwdParams& p, cudaStream_t stream) {
  using namespace norm;
  const int xe = elem_of(p.x_type), se = elem_of(p.stream_type);
  const bool w = aligned16(p.weight) && in_step(p.y, p.ldy, elem_of(p.y_type), p.x, p.ldx, xe) &&
                 (!p.res || (in_step(p.res, p.ldr, se, p.x, p.ldx, xe) && in_step(p.s, p.lds, se, p.x, p.ldx, xe)));
  return w ? fwd_types<8>(p, stream) : fwd_types<1>(p, stream);
}

cudaError_t norm_kernels_setup() {
  cudaError_t e = norm::bwd_setup<float, float>();
  if (e == cudaSuccess) e = norm::bwd_setup<float, uint16_t>();
  if (e == cudaSuccess) e = norm::bwd_setup<uint16_t, float>();
  return e == cudaSuccess ? norm::bwd_setup<uint16_t, uint16_t>() : e;
}

int64_t norm_bwd_blocks(int64_t rows, int width) {
  // fewer rows a block and more blocks an SM than any variant has
  return norm::bwd_blocks(rows, 1, width <= 4096 ? norm::kMostBlocksPerSm : 4);
}

cudaError_t launch_norm_rows_bwd(const NormRowsBwdParams& p, cudaStream_t stream) {
  using namespace norm;
  const int st = elem_of(p.stream_type), ge = elem_of(p.dy_type);
  const bool w = aligned16(p.weight) && in_step(p.dy, p.lddy, ge, p.s, p.lds, st) &&
                 in_step(p.dx, p.lddx, st, p.s, p.lds, st) && (!p.ds || in_step(p.ds, p.ldds, st, p.s, p.lds, st));
  int64_t blocks = 0;
  const cudaError_t e =
      p.dy_type == kF32
          ? (p.stream_type == kF32 ? bwd<float, float>(p, w, &blocks, stream) : bwd<float, uint16_t>(p, w, &blocks, stream))
          : (p.stream_type == kF32 ? bwd<uint16_t, float>(p, w, &blocks, stream) : bwd<uint16_t, uint16_t>(p, w, &blocks, stream));
  if (e != cudaSuccess || !p.part) return e;
  return launch_col_sum(p.part, blocks, p.width, p.dweight, stream);
}

cudaError_t launch_col_sum(const float* part, int64_t blocks, int64_t width, float* out, cudaStream_t stream) {
  return launch_pdl(norm::col_sum_kernel, dim3(static_cast<unsigned>((width + 31) / 32)), dim3(1024), 0, stream, 1, part,
                    blocks, width, out);
}

}  // namespace ufc
