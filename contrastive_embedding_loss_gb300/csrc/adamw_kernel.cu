// adamw_kernel.cu -- one AdamW step over many tensors.
//
//   m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2;
//   p -= lr (m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps) + decay p)
//
// Bound by HBM: 30 bytes an element with fp32 states, gradients and parameters and a bf16 copy,
// 16 with 8-bit states and bf16 gradients.  The table of tensors is a kernel argument (no copy
// to the device, so a step can be captured); a warp takes blocks of 256 elements with a stride
// of the grid's warps, 8 elements a lane, and walks the table forward as it goes.  A block's loads
// are issued before the block before it is worked on.  389 M elements with 8-bit states: 1038 us
// (6.0 TB/s); 18 M with fp32 states 84 us (6.5 TB/s).
//
// 8-bit states: e4m3 codes of m and of r = sqrt(v) with an fp32 scale per block of 256 elements,
// the block's largest magnitude standing at code 448.  One step moves v by about 1 - b2 = 0.1 %
// while codes of r are 6 to 12 % apart, so rounding to nearest would freeze v: the codes are
// rounded at random, up with the probability that makes m and v (r squared, not r: E[r^2] exceeds
// E[r]^2, which would inflate v at every step) unbiased.  A nonzero v never rounds to code 0,
// which would make its next update m / eps.  A block in which v overflows keeps an infinite scale, and
// every code of it becomes 126: from then on its elements take no step, as sqrt(v) = inf has it.
#include "layers.cuh"

namespace ufc {
namespace adam {

constexpr int kThreads = 256;
constexpr float kMinNormal = 0.015625f;  // 2^-6: e4m3's smallest normal number
constexpr float kMinTop = 0x1p-116f;     // the least block maximum with codes: 448 / it is finite

// A mix of 32 bits by two multiplications, found by search: C. Wellons, Prospecting for Hash Functions
// (2018), shifts 16, 15, 16.
__device__ __forceinline__ uint32_t hash32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7FEB352Du;
  x ^= x >> 15;
  x *= 0x846CA68Bu;
  return x ^ (x >> 16);
}

template <int CAP>
struct Table {
  AdamTensor t[CAP];
  int64_t first_block[CAP + 1];
};

// The codes come in the low byte.  SUB: some value may lie below 2^-6, where the codes are 2^-9
// apart, as they are in [2^-6, 2^-5): adding 2^-6 there makes one rule of both.  Few blocks have
// such a value next to their largest (28672 times as large), and the rule for
// the others is much shorter: it took 389 M elements from 1133 us to 1020.  (Of a block with a NaN or
// an infinity the scale tells.)

// The e4m3 code of n, |n| <= 448, rounded away from 0 with the probability of |n|'s place between
// its neighbours (u: 16 random bits at bits 4 to 19, below the code's bits).
template <bool SUB>
__device__ __forceinline__ uint32_t code_linear(float n, uint32_t u) {
  const float x = fabsf(n);
  const bool sub = SUB && x < kMinNormal;
  // (448 itself has no bits below its code's, and n exceeds it by 3 units of the last place at most:
  // no carry)
  const uint32_t c = ((__float_as_uint(sub ? x + kMinNormal : x) + u) >> 20) - (sub ? 968u : 960u);
  return c | (__float_as_uint(n) >> 24 & 0x80u);
}
// The same for two values n >= 0, unbiased in n^2: up when u < (n^2 - lo^2) / (hi^2 - lo^2), u in
// [0, 1), lo and hi the neighbours; a nonzero n is at least code 1.  minus_u: -u.  May exceed 126.
template <bool SUB>
__device__ __forceinline__ void code_square2(float2 n, float2 minus_u, uint32_t& ca, uint32_t& cb) {
  const bool sa = SUB && n.x < kMinNormal, sb = SUB && n.y < kMinNormal;
  const float2 minus = make_float2(-1.f, -1.f);
  const float2 off = make_float2(sa ? kMinNormal : 0.f, sb ? kMinNormal : 0.f);
  const float2 x = SUB ? add2(n, off) : n;
  const uint32_t ba = __float_as_uint(x.x) & ~0xFFFFFu, bb = __float_as_uint(x.y) & ~0xFFFFFu;
  float2 lo = make_float2(__uint_as_float(ba), __uint_as_float(bb));
  float2 hi = make_float2(__uint_as_float(ba + 0x100000u), __uint_as_float(bb + 0x100000u));
  if constexpr (SUB) lo = fma2(off, minus, lo), hi = fma2(off, minus, hi);
  const float2 lo2 = mul2(lo, lo);
  const float2 over = fma2(lo2, minus, mul2(n, n)), span = fma2(lo2, minus, mul2(hi, hi));
  const float2 d = fma2(minus_u, span, over);  // over - u span, rounded once: its sign is exact
  ca = (__float_as_uint(x.x) >> 20) - (sa ? 968u : 960u) + (d.x > 0.f ? 1u : 0u);
  cb = (__float_as_uint(x.y) >> 20) - (sb ? 968u : 960u) + (d.y > 0.f ? 1u : 0u);
  if constexpr (SUB) {
    ca = max(ca, min(__float_as_uint(n.x), 1u));
    cb = max(cb, min(__float_as_uint(n.y), 1u));
  }
}
// Four e4m3 codes to floats.
__device__ __forceinline__ void from_e4m3(uint32_t q, float* v) {
  const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(q & 0xFFFFu), __NV_E4M3);
  const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(q >> 16), __NV_E4M3);
  const float2 x = __half22float2(__half2(a)), y = __half22float2(__half2(b));
  v[0] = x.x, v[1] = x.y, v[2] = y.x, v[3] = y.y;
}
// The step's constants, prepared once a thread:
//   m = beta1 m + c1 g,  v = beta2 v + c2 g g
//   p -= lr (m a / (sqrt(v) + e) + decay p),  a = sqrt(1 - b2^t) / (1 - b1^t),  e = eps sqrt(1 - b2^t)
// m and v are rounded after every operation, not fused: a code is chosen by where its value lies
// between two others, so a last bit more or less decides codes, and these are the roundings that
// the formula has in any other fp32 program.
struct Step {
  float lr, beta1, beta2, c1, c2, scale, one, a, e, decay;
};

// sqrt(v) to the nearest: an approximate reciprocal root y, r = v y, and one step of the coupled
// Newton iteration (Markstein), r + (v - r^2) y / 2.  A subnormal v's root comes out too small, by up to
// 2^-63: update() uses it only beside an e that hides that.  Of an infinite v the sum
// is NaN (inf 0); v 2^-70, which is below the root of every finite v, is infinite there, and a maximum
// takes the other operand of a NaN.  (A NaN v makes both NaN.)
__device__ __forceinline__ float2 sqrt2(float2 v) {
  float2 y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(fmaxf(v.x, 1.18e-38f)));
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(fmaxf(v.y, 1.18e-38f)));
  const float2 r = mul2(v, y);
  const float2 left = fma2(mul2(r, both(-1.f)), r, v);
  const float2 root = fma2(left, mul2(y, both(0.5f)), r), below = mul2(v, both(0x1p-70f));
  return make_float2(fmaxf(root.x, below.x), fmaxf(root.y, below.y));
}
// 1 / x to the nearest, by one Newton step.
__device__ __forceinline__ float reciprocal(float x) {
  const float y = rcp_approx(x);
  return fmaf(fmaf(-y, x, 1.f), y, y);
}

// Two elements: the new moments, sqrt(v), and the new parameters (whose fast reciprocal is good
// to about 2^-22 of the step).  EXACT: for an e below 2^-38; from there on an error of r of 2^-63 is within
// the rounding of r + e.
template <bool EXACT>
__device__ __forceinline__ float2 update(const Step& h, float2 p, float2 g, float2& m, float2& v, float2& r) {
  g = mul2(g, both(h.scale));
  // x 1 + y: a packed addition of two packed products would be contracted to a fused operation
  // (which skips a rounding), a fused one is left alone
  m = fma2(mul2(m, both(h.beta1)), both(h.one), mul2(g, both(h.c1)));
  v = fma2(mul2(v, both(h.beta2)), both(h.one), mul2(mul2(g, both(h.c2)), g));
  if constexpr (EXACT)
    r = make_float2(sqrtf(v.x), sqrtf(v.y));
  else
    r = sqrt2(v);
  const float2 den = add2(r, both(h.e));
  const float2 d = mul2(m, make_float2(rcp_approx(den.x), rcp_approx(den.y)));
  return fma2(both(-h.lr), fma2(d, both(h.a), mul2(p, both(h.decay))), p);
}

// Eight elements as they lie in memory; past `left` they are 0.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p, int64_t left, bool wide) {
    if (wide && left >= 8) {
      a = reinterpret_cast<const float4*>(p)[0];
      b = reinterpret_cast<const float4*>(p)[1];
    } else {
      a.x = left > 0 ? p[0] : 0.f, a.y = left > 1 ? p[1] : 0.f, a.z = left > 2 ? p[2] : 0.f, a.w = left > 3 ? p[3] : 0.f;
      b.x = left > 4 ? p[4] : 0.f, b.y = left > 5 ? p[5] : 0.f, b.z = left > 6 ? p[6] : 0.f, b.w = left > 7 ? p[7] : 0.f;
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};
template <>
struct Raw8<uint16_t> {
  uint4 q;
  __device__ __forceinline__ void load(const uint16_t* p, int64_t left, bool wide) {
    if (wide && left >= 8) {
      q = *reinterpret_cast<const uint4*>(p);
    } else {
      auto at = [&](int j) { return left > j ? static_cast<uint32_t>(p[j]) : 0u; };
      q = make_uint4(at(0) | at(1) << 16, at(2) | at(3) << 16, at(4) | at(5) << 16, at(6) | at(7) << 16);
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const { unpack8(q, v); }
};
template <>
struct Raw8<uint8_t> {  // e4m3 codes
  uint2 q;
  __device__ __forceinline__ void load(const uint8_t* p, int64_t left, bool wide) {
    if (wide && left >= 8) {
      q = *reinterpret_cast<const uint2*>(p);
    } else {
      auto at = [&](int j) { return left > j ? static_cast<uint32_t>(p[j]) << (8 * (j & 3)) : 0u; };
      q = make_uint2(at(0) | at(1) | at(2) | at(3), at(4) | at(5) | at(6) | at(7));
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const { from_e4m3(q.x, v), from_e4m3(q.y, v + 4); }
};

// CAP: entries of the table; a small one keeps the argument block of a short list small.  EXACT: a
// kernel of its own, as a branch on it (the same for the whole grid) kept the loads' unpacking and
// the update apart, 4 % of the time.
template <typename PT, typename GT, bool E8, int CAP, bool EXACT>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Table<CAP> tab, const AdamScalars sc) {
  griddep_enter();
  const int lane = threadIdx.x & 31;
  float scale = 1.f, bc1 = sc.bc1, sqrt_bc2 = sc.sqrt_bc2;
  uint32_t seed = sc.seed;
  if (sc.grad_scale) scale = *sc.grad_scale;
  if (sc.step_dev) {  // 1 - b^t = -expm1(t log b)
    const int64_t t = *sc.step_dev;
    seed += static_cast<uint32_t>(t);
    bc1 = -expm1f(static_cast<float>(t) * sc.log_beta1);
    sqrt_bc2 = sqrtf(-expm1f(static_cast<float>(t) * sc.log_beta2));
  }
  Step h;
  h.lr = sc.lr_dev ? *sc.lr_dev : sc.lr;
  h.beta1 = sc.beta1, h.beta2 = sc.beta2;
  h.c1 = sc.c1, h.c2 = sc.c2;
  h.scale = scale;
  h.one = sc.one;
  h.a = sqrt_bc2 / bc1;
  h.e = sc.eps * sqrt_bc2;
  h.decay = sc.decay;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  const int64_t total = tab.first_block[sc.n];
  using MT = typename std::conditional<E8, uint8_t, float>::type;
  // a lane's part of a block as it lies in memory
  struct Part {
    Raw8<PT> p;
    Raw8<GT> g;
    Raw8<MT> m, v;
    float ms, vs;
  };
  int64_t blk = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  int k = 0;
  auto fetch = [&](Part& q) {
    while (blk >= tab.first_block[k + 1]) ++k;
    const AdamTensor& t = tab.t[k];
    const int64_t b = blk - tab.first_block[k], i0 = b * kAdamBlock + lane * 8;
    const int64_t left = t.size - i0;
    q.p.load(static_cast<const PT*>(t.p) + i0, left, t.wide);
    q.g.load(static_cast<const GT*>(t.g) + i0, left, t.wide);
    q.m.load(static_cast<const MT*>(t.m) + i0, left, t.wide);
    q.v.load(static_cast<const MT*>(t.v) + i0, left, t.wide);
    if (E8) {
      q.ms = t.ms[b];
      q.vs = t.vs[b];
    }
  };
  Part next;
  if (blk < total) fetch(next);
  while (blk < total) {
    // the next block's loads are on their way while this one is worked on
    const Part part = next;
    const int kt = k;
    const AdamTensor& t = tab.t[kt];
    const int64_t b = blk - tab.first_block[kt];
    const int64_t i0 = b * kAdamBlock + lane * 8;
    blk += warps;
    if (blk < total) fetch(next);
    const int left = t.size - i0 >= 8 ? 8 : t.size > i0 ? static_cast<int>(t.size - i0) : 0;
    const bool wide = left == 8 && t.wide;
    PT* pp = static_cast<PT*>(t.p) + i0;
    uint16_t* cp = t.copy ? t.copy + i0 : nullptr;
    float p[8], g[8], m[8], v[8], r[8];
    part.p.get(p);
    part.g.get(g);
    part.m.get(m);
    part.v.get(v);
    if constexpr (E8) {
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float2 m2 = mul2(make_float2(m[j], m[j + 1]), both(part.ms));
        const float2 r2 = mul2(make_float2(v[j], v[j + 1]), both(part.vs));
        const float2 v2 = mul2(r2, r2);
        m[j] = m2.x, m[j + 1] = m2.y, v[j] = v2.x, v[j + 1] = v2.y;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      float2 m2 = make_float2(m[j], m[j + 1]), v2 = make_float2(v[j], v[j + 1]), r2;
      const float2 p2 =
          update<EXACT>(h, make_float2(p[j], p[j + 1]), make_float2(g[j], g[j + 1]), m2, v2, r2);
      p[j] = p2.x, p[j + 1] = p2.y;
      m[j] = m2.x, m[j + 1] = m2.y;
      v[j] = v2.x, v[j + 1] = v2.y;
      r[j] = r2.x, r[j + 1] = r2.y;
    }
    uint32_t rnd[8];
    if constexpr (E8 || sizeof(PT) == 2) {
      const uint32_t key = hash32(seed + 0x9E3779B9u * (sc.first + static_cast<uint32_t>(kt)));
#pragma unroll
      for (int j = 0; j < 8; ++j) rnd[j] = hash32(static_cast<uint32_t>(i0 + j) + key);
    }
    if constexpr (sizeof(PT) == 2) {
      // 16 random bits below the bf16's own, then cut (a NaN's would carry into its sign)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t up = __float_as_uint(p[j]) + (hash32(rnd[j] ^ 0x9E3779B9u) & 0xFFFFu);
        if (!isnan(p[j])) p[j] = __uint_as_float(up & 0xFFFF0000u);
      }
    }
    if (wide) {
      store8(pp, p);
      if (cp) store8(cp, p);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < left) {
          store1(pp + j, p[j]);
          if (cp) store1(cp + j, p[j]);
        }
    }
    if constexpr (E8) {
      if (left < 8) {  // 0 times an infinite scale is not 0
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j >= left) m[j] = r[j] = 0.f;
      }
      float mt = 0.f, ml = fabsf(m[0]), rl = r[0];
      uint32_t rt = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        mt = fmaxf(mt, fabsf(m[j]));
        ml = fminf(ml, fabsf(m[j]));
        rl = fminf(rl, r[j]);
        rt = max(rt, __float_as_uint(r[j]));  // as bits: a NaN is the largest
      }
      mt = __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(mt)));
      const float vt = __uint_as_float(__reduce_max_sync(~0u, rt));
      // Momentum that is not fed halves every 7 steps (beta1 = 0.9) and gets here in some 750.  (A nonzero sqrt(v)
      // is above 2^-75.)
      if (mt < kMinTop) mt = 0.f;
      if (isnan(vt)) mt = vt;  // a NaN gradient makes both scales NaN
      const float mi = mt > 0.f ? reciprocal(mt) * 448.f : 0.f, vi = vt > 0.f ? reciprocal(vt) * 448.f : 0.f;
      if (lane == 0) {
        t.ms[b] = mt * (1.f / 448.f);
        t.vs[b] = vt * (1.f / 448.f);
      }
      uint2 mq, vq;
      auto encode = [&](auto sub_c) {
        constexpr bool SUB = decltype(sub_c)::value;
        uint32_t cm[8], cv[8];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float2 n = mul2(make_float2(m[j], m[j + 1]), both(mi));
          cm[j] = code_linear<SUB>(n.x, rnd[j] << 4 & 0xFFFF0u);
          cm[j + 1] = code_linear<SUB>(n.y, rnd[j + 1] << 4 & 0xFFFF0u);
          const float2 minus_u = fma2(make_float2(__uint_as_float(rnd[j] >> 9 & 0x7FFF80u | 0x3F800000u),
                                                  __uint_as_float(rnd[j + 1] >> 9 & 0x7FFF80u | 0x3F800000u)),
                                      both(-1.f), both(1.f));
          code_square2<SUB>(mul2(make_float2(r[j], r[j + 1]), both(vi)), minus_u, cv[j], cv[j + 1]);
        }
        auto bytes = [](const uint32_t* c) {
          return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
        };
        // two 16-bit codes at a time, 126 at most
        auto bytes126 = [](const uint32_t* c) {
          return __byte_perm(__vminu2(__byte_perm(c[0], c[1], 0x5410), 0x7E007Eu),
                             __vminu2(__byte_perm(c[2], c[3], 0x5410), 0x7E007Eu), 0x6420);
        };
        mq = make_uint2(bytes(cm), bytes(cm + 4)), vq = make_uint2(bytes126(cv), bytes126(cv + 4));
      };
      if (__any_sync(~0u, fminf(ml * mi, rl * vi) < kMinNormal))
        encode(std::true_type{});
      else
        encode(std::false_type{});
      uint8_t* mp = static_cast<uint8_t*>(t.m) + i0;
      uint8_t* vp = static_cast<uint8_t*>(t.v) + i0;
      if (wide) {
        *reinterpret_cast<uint2*>(mp) = mq;
        *reinterpret_cast<uint2*>(vp) = vq;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < left) {
            mp[j] = static_cast<uint8_t>((j < 4 ? mq.x : mq.y) >> (8 * (j & 3)));
            vp[j] = static_cast<uint8_t>((j < 4 ? vq.x : vq.y) >> (8 * (j & 3)));
          }
      }
    } else {
      float* mp = static_cast<float*>(t.m) + i0;
      float* vp = static_cast<float*>(t.v) + i0;
      if (wide) {
        store8(mp, m);
        store8(vp, v);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < left) {
            mp[j] = m[j];
            vp[j] = v[j];
          }
      }
    }
  }
}

template <typename PT, typename GT, bool E8, int CAP, bool EXACT>
cudaError_t launch(const AdamTensor* t, const AdamScalars& sc, cudaStream_t stream) {
  Table<CAP> tab;
  tab.first_block[0] = 0;
  for (int i = 0; i < sc.n; ++i) {
    tab.t[i] = t[i];
    // wide accesses need every array's 16-byte alignment (8 for the codes)
    const uintptr_t any = reinterpret_cast<uintptr_t>(t[i].p) | reinterpret_cast<uintptr_t>(t[i].g) |
                          reinterpret_cast<uintptr_t>(t[i].copy);
    const uintptr_t states = reinterpret_cast<uintptr_t>(t[i].m) | reinterpret_cast<uintptr_t>(t[i].v);
    tab.t[i].wide = (any & 15) == 0 && (states & (E8 ? 7 : 15)) == 0;
    tab.first_block[i + 1] = tab.first_block[i] + (t[i].size + kAdamBlock - 1) / kAdamBlock;
  }
  const int64_t blocks = (tab.first_block[sc.n] + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks == 0) return cudaSuccess;
  const int64_t most = static_cast<int64_t>(current_sm_count()) * 8;
  return launch_pdl(adamw_kernel<PT, GT, E8, CAP, EXACT>, dim3(static_cast<unsigned>(blocks < most ? blocks : most)),
                    dim3(kThreads), 0, stream, 1, tab, sc);
}
template <typename PT, typename GT, bool E8>
cudaError_t launch_cap(const AdamTensor* t, const AdamScalars& sc, cudaStream_t stream) {
  // eps sqrt(1 - beta2^t), at its least at the first step
  if (sc.eps * sqrtf(sc.c2) < 0x1p-38f) return launch<PT, GT, E8, kAdamTensors, true>(t, sc, stream);
  return sc.n <= 32 ? launch<PT, GT, E8, 32, false>(t, sc, stream) : launch<PT, GT, E8, kAdamTensors, false>(t, sc, stream);
}
template <typename PT, typename GT>
cudaError_t launch_state(const AdamTensor* t, const AdamScalars& sc, int state_type, cudaStream_t stream) {
  return state_type == kE4m3 ? launch_cap<PT, GT, true>(t, sc, stream) : launch_cap<PT, GT, false>(t, sc, stream);
}

}  // namespace adam

cudaError_t launch_adamw(const AdamTensor* t, const AdamScalars& sc, int param_type, int grad_type, int state_type,
                         cudaStream_t stream) {
  if (param_type == kF32)
    return grad_type == kF32 ? adam::launch_state<float, float>(t, sc, state_type, stream)
                             : adam::launch_state<float, uint16_t>(t, sc, state_type, stream);
  return grad_type == kF32 ? adam::launch_state<uint16_t, float>(t, sc, state_type, stream)
                           : adam::launch_state<uint16_t, uint16_t>(t, sc, state_type, stream);
}

}  // namespace ufc
