// Products of 8-bit integers with a scale for each token and each output channel:
//   q[t, i] = rint(x[t, i] / sx[t]),   sx[t] = max_i |x[t, i]| / 127          (quantize_rows_i8)
//   Y[t, n] = sx[t] * sw[n] * sum_i q[t, i] * w[n, i]  (+ bias[n])            (qgemm_i8)
// The sums are exact int32 on every path, so the paths agree bit for bit and results are
// deterministic; what is rounded is float(sum) (one rounding above 2^24), the two scalings, the
// bias and the store, in this order.
//
// No page describes this step: the pages' CPU engines hold activations as int8 blocks for their
// integer dots (Camelid README, "Engine status"); this is the whole-row form that a batch of
// tokens needs, with weights that are int8 rows.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "host_common.h"
#include "i8_cut.h"
#include "tcgen05.cuh"

namespace bqg {

// ---------------------------------------------------------------- element types
template <typename T>
struct Elem;
// Raw: eight values as they are stored.  most(): a running max|x| (NaN if there is one), two at a time for
// the 16-bit types, which starts at 0 and as_float() ends.
template <>
struct Elem<float> {
  struct Raw {
    uint32_t w[8];
  };
  static __device__ __forceinline__ Raw load8(const float* p) {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
  }
  static __device__ __forceinline__ void set(Raw& r, int i, float v) { r.w[i] = __float_as_uint(v); }
  static __device__ __forceinline__ void values(const Raw& r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.w[i]);
  }
  static __device__ __forceinline__ void most(uint32_t& top, const Raw& r) {
    float t = __uint_as_float(top);
#pragma unroll
    for (int i = 0; i < 8; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(t) : "f"(fabsf(__uint_as_float(r.w[i]))));
    top = __float_as_uint(t);
  }
  static __device__ __forceinline__ float as_float(uint32_t top) { return __uint_as_float(top); }
};
struct Raw16 {
  uint32_t w[4];
};
template <typename T>
__device__ __forceinline__ Raw16 load8_16(const T* p) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  return {{a.x, a.y, a.z, a.w}};
}
__device__ __forceinline__ void set16(Raw16& r, int i, uint32_t bits) {
  r.w[i >> 1] = i & 1 ? (r.w[i >> 1] & 0xFFFFu) | bits << 16 : (r.w[i >> 1] & 0xFFFF0000u) | bits;
}
template <>
struct Elem<__half> {
  using Raw = Raw16;
  static __device__ __forceinline__ Raw load8(const __half* p) { return load8_16(p); }
  static __device__ __forceinline__ void set(Raw& r, int i, __half v) { set16(r, i, __half_as_ushort(v)); }
  static __device__ __forceinline__ void values(const Raw& r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ void most(uint32_t& top, const Raw& r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(top) : "r"(r.w[i] & 0x7FFF7FFFu));
  }
  static __device__ __forceinline__ float as_float(uint32_t top) {
    asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(top) : "r"(top >> 16 | top << 16));
    return __half2float(__ushort_as_half(static_cast<unsigned short>(top & 0xFFFFu)));
  }
  static __device__ __forceinline__ uint32_t bits(float f) { return __half_as_ushort(__float2half_rn(f)); }
};
template <>
struct Elem<__nv_bfloat16> {
  using Raw = Raw16;
  static __device__ __forceinline__ Raw load8(const __nv_bfloat16* p) { return load8_16(p); }
  static __device__ __forceinline__ void set(Raw& r, int i, __nv_bfloat16 v) { set16(r, i, __bfloat16_as_ushort(v)); }
  static __device__ __forceinline__ void values(const Raw& r, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(r.w[i] << 16);
      v[2 * i + 1] = __uint_as_float(r.w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void most(uint32_t& top, const Raw& r) {
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(r.w[i] & 0x7FFF7FFFu));
  }
  static __device__ __forceinline__ float as_float(uint32_t top) {
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(top >> 16 | top << 16));
    return __uint_as_float(top << 16);
  }
  static __device__ __forceinline__ uint32_t bits(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }
};

// ---------------------------------------------------------------- rows to int8
// TPR threads own a row (32: 8 rows per CTA, else one row per CTA of TPR threads).  A thread keeps up
// to kQrChunks chunks of 8 values in registers, so rows of up to TPR * 32 values are read once; longer
// rows read the rest a second time (from L2).  Bytes bound it: 1 read and 1 write of the row; of the
// TPR that hold a row, the smallest has the most bytes in flight (8192 x 4096 bf16: 128 threads a row
// 21.9 us, bound by instructions: 3.0 of 4 issue slots a clock; 256, and every rounding decided the long
// way, 40 us), the largest the shortest way for few rows.  fp32 rows of 4096: 27.3 us, 6.1 TB/s.  VEC false
// (rows off 16 bytes, read value by value): 30.4 and 38.6 us.
//
// The rounding is decided exactly.  t = x * (1 / s) + 1.5 * 2^23 is rounded once, to a whole number
// n (in t's low bits); x * (1 / s) is off from x / s by less than 127 * 2^-24 * 1.1, so wherever it
// lies within 0.4999 of n, so does x / s within 1/2.  Otherwise, next to a border: with f = floor(x *
// (1 / s)) (off by at most one), q is f or f + 1 by the sign of fma(-(f + 1/2), s, x), which is the
// sign of the exact difference (f + 1/2 has at most 9 bits; a fused result is 0 only for an exact tie,
// since s >= 2^-100 keeps it clear of underflow).  A tie goes to the even integer.  A plain rint(x *
// (1 / s)) would miss borders: bf16 rows meet exact ties often.
constexpr int kQrThreads = 256;
constexpr int kQrChunks = 4;
constexpr int kQrFewRows = 592;  // four rows an SM
constexpr float kQrTinyScale = 7.888609052210118e-31f;  // 2^-100: a row below it is held as zeros

__device__ __forceinline__ int round_quotient(float x, float s, float inv) {
  const float f = floorf(x * inv);
  const float d = fmaf(-(f + 0.5f), s, x);
  const int i = int(f);
  return i + ((d > 0.f || (d == 0.f && (i & 1))) ? 1 : 0);
}

template <typename T, int TPR, bool VEC>
__global__ void __launch_bounds__(TPR == 32 ? kQrThreads : TPR) k_quantize_rows(const T* __restrict__ X, long long ldx,
                                                              int8_t* __restrict__ Q, long long ldq,
                                                              float* __restrict__ scale, int rows, int k) {
  constexpr int kRows = TPR == 32 ? kQrThreads / 32 : 1;
  __shared__ uint32_t wmax[TPR / 32];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = TPR == 32 ? (threadIdx.x & 31) : threadIdx.x;
  const long long row = (long long)blockIdx.x * kRows + (TPR == 32 ? threadIdx.x >> 5 : 0);
  if (TPR == 32 && row >= rows) return;
  const T* x = X + row * ldx;
  int8_t* q = Q + row * ldq;
  const int kmain = min(k, TPR * 8 * kQrChunks);

  using Raw = typename Elem<T>::Raw;
  auto load = [&](int i0) -> Raw {  // values i0 .. i0 + 7 (0 past the row's end)
    if (VEC && i0 + 8 <= k) return Elem<T>::load8(x + i0);
    Raw r{};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i0 + j < k) Elem<T>::set(r, j, x[i0 + j]);
    return r;
  };
  uint32_t top = 0u;
  Raw keep[kQrChunks];
#pragma unroll
  for (int c = 0; c < kQrChunks; ++c) {
    const int i0 = (c * TPR + tid) * 8;
    keep[c] = Raw{};
    if (i0 < kmain) keep[c] = load(i0);
  }
#pragma unroll
  for (int c = 0; c < kQrChunks; ++c) Elem<T>::most(top, keep[c]);
  for (int i0 = (kQrChunks * TPR + tid) * 8; i0 < k; i0 += TPR * 8) Elem<T>::most(top, load(i0));
  // as an unsigned integer, which keeps the order and puts Inf and NaN above every finite value
  uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(Elem<T>::as_float(top)));
  if (TPR > 32) {
    if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < TPR / 32; ++w) most = max(most, wmax[w]);
  }
  float s = __fdiv_rn(__uint_as_float(most), 127.f);
  const bool finite = most < 0x7F800000u;
  if (!finite) s = __uint_as_float(0x7FC00000u);  // the whole row of the product becomes NaN
  else if (s < kQrTinyScale) s = 0.f;
  if (tid == 0) scale[row] = s;
  const bool zero = !(s > 0.f);
  const float inv = zero ? 0.f : __fdiv_rn(1.f, s);

  auto store = [&](int i0, const Raw& r) {
    float v[8];
    Elem<T>::values(r, v);
    uint32_t w[2] = {0u, 0u};
    if (!zero) {
      constexpr float kWhole = 12582912.f;  // 1.5 * 2^23
      uint32_t b[8];
      bool border = false;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = fmaf(v[j], inv, kWhole);
        border |= fabsf(fmaf(v[j], inv, -(t - kWhole))) > 0.4999f;
        b[j] = __float_as_uint(t);
      }
      if (border) {
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = uint32_t(round_quotient(v[j], s, inv));
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
        w[j] = __byte_perm(__byte_perm(b[4 * j], b[4 * j + 1], 0x0040), __byte_perm(b[4 * j + 2], b[4 * j + 3], 0x0040), 0x5410);
    }
    if (i0 + 8 <= k) {
      *reinterpret_cast<uint2*>(q + i0) = make_uint2(w[0], w[1]);
    } else {
      for (int j = 0; j < 8 && i0 + j < k; ++j) q[i0 + j] = int8_t(w[j >> 2] >> (8 * (j & 3)));
    }
  };
#pragma unroll
  for (int c = 0; c < kQrChunks; ++c) {
    const int i0 = (c * TPR + tid) * 8;
    if (i0 < kmain) store(i0, keep[c]);
  }
  for (int i0 = (kQrChunks * TPR + tid) * 8; i0 < k; i0 += TPR * 8) store(i0, load(i0));
}

// ---------------------------------------------------------------- the product: arguments
struct I8Params {
  const int8_t* X;
  const int8_t* W;
  const float* sx;
  const float* sw;
  const float* bias;  // or null
  void* Y;
  long long ldx, ldw, ldy;
  int tokens, n, k;
  int out;   // BQG_F32, BQG_F16 or BQG_BF16
  int pair;  // 16-bit outputs: rows of Y are 4-byte aligned, two values per store
  int split; // parts of k, CTAs of a cluster (k_i8_gemm<BN, true>)
};

__device__ __forceinline__ float i8_value(int sum, float sx, float sw, float bias, bool has_bias) {
  // spelled out, so that no copy of this fuses a product with the bias: all paths round alike
  const float v = __fmul_rn(__fmul_rn(__int2float_rn(sum), sx), sw);
  return has_bias ? __fadd_rn(v, bias) : v;
}

__device__ __forceinline__ void i8_store(const I8Params& P, long long t, int n, float v) {
  const long long at = t * P.ldy + n;
  if (P.out == BQG_F32) static_cast<float*>(P.Y)[at] = v;
  else if (P.out == BQG_F16) static_cast<__half*>(P.Y)[at] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(P.Y)[at] = __float2bfloat16_rn(v);
}

// ---------------------------------------------------------------- few tokens: a GEMV per token on dp4a
// A warp owns kIgRows rows of W and walks k in 512-byte steps: lane l reads 16 bytes of each row
// (coalesced) and of each token's x (from L1, shared by every warp of the SM); 4 dp4a per 16
// bytes, row and token.  Bound by the weight stream where the rows fill the SMs (1 x 4096 x 14336: 11.8 us,
// 5.0 TB/s), by a warp's steps one after another otherwise.  i8_few says which products come here.
constexpr int kIgThreads = 256;
constexpr int kIgRows = 4;

__device__ __forceinline__ uint4 load16_tail(const int8_t* p, int bytes) {  // 1..15 bytes, the rest 0
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  for (int i = 0; i < bytes; ++i) w[i >> 2] |= uint32_t(uint8_t(p[i])) << (8 * (i & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ int dp16(const uint4& a, const uint4& b, int c) {
  c = __dp4a(int(a.x), int(b.x), c);
  c = __dp4a(int(a.y), int(b.y), c);
  c = __dp4a(int(a.z), int(b.z), c);
  return __dp4a(int(a.w), int(b.w), c);
}

template <int NT>
__global__ void __launch_bounds__(kIgThreads) k_i8_gemv(const __grid_constant__ I8Params P) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const long long warps = (long long)gridDim.x * (kIgThreads / 32);
  const int full = P.k / 16, tail = P.k % 16;
  const int groups = (P.n + kIgRows - 1) / kIgRows;
  for (long long g = (long long)blockIdx.x * (kIgThreads / 32) + (threadIdx.x >> 5); g < groups; g += warps) {
    const int n0 = int(g) * kIgRows;
    const int8_t* wrow[kIgRows];
#pragma unroll
    for (int r = 0; r < kIgRows; ++r) wrow[r] = P.W + (long long)min(n0 + r, P.n - 1) * P.ldw;
    int acc[kIgRows][NT];
#pragma unroll
    for (int r = 0; r < kIgRows; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[r][t] = 0;
    auto step = [&](const uint4 (&w)[kIgRows], const uint4& xv, int t) {
#pragma unroll
      for (int r = 0; r < kIgRows; ++r) acc[r][t] = dp16(w[r], xv, acc[r][t]);
    };
#pragma unroll 2
    for (int c = lane; c < full; c += 32) {
      uint4 w[kIgRows];
#pragma unroll
      for (int r = 0; r < kIgRows; ++r) w[r] = __ldcs(reinterpret_cast<const uint4*>(wrow[r]) + c);
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (t < P.tokens) step(w, __ldg(reinterpret_cast<const uint4*>(P.X + t * P.ldx) + c), t);
    }
    if (tail > 0 && lane == (full & 31)) {  // the last 1..15 values of each row, byte by byte
      uint4 w[kIgRows];
#pragma unroll
      for (int r = 0; r < kIgRows; ++r) w[r] = load16_tail(wrow[r] + full * 16, tail);
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (t < P.tokens) step(w, load16_tail(P.X + t * P.ldx + full * 16, tail), t);
    }
    __syncwarp();
    int mine = 0;  // lane r * NT + t holds row r of token t
#pragma unroll
    for (int r = 0; r < kIgRows; ++r)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int v = __reduce_add_sync(0xffffffffu, acc[r][t]);
        if (lane == r * NT + t) mine = v;
      }
    const int r = lane / NT, t = lane % NT;
    if (r < kIgRows && t < P.tokens && n0 + r < P.n)
      i8_store(P, t, n0 + r,
               i8_value(mine, __ldg(P.sx + t), __ldg(P.sw + n0 + r), P.bias ? __ldg(P.bias + n0 + r) : 0.f,
                        P.bias != nullptr));
  }
}

// ---------------------------------------------------------------- many tokens: tcgen05 kind::i8
// One tile is 128 output channels (rows of W, the MMA's M side: tensor-memory lanes) x BN tokens
// (N side: columns).  Lane = channel makes the store of one token's column 32 consecutive values
// of Y per warp, at any pitch, and lets small token counts take a small N.
//   warp 0     TMA: per stage 128 k of W (128 rows) and of X (BN rows), 128-byte swizzle; rows and
//              columns past the tensors read as 0
//   warp 1     allocates tensor memory, issues 4 MMAs (M 128, N BN, K 32) per stage into one of two
//              int32 accumulators
//   warps 2-5  scale, convert and store the other accumulator (one warp per 32 lanes)
// Persistent: CTA b takes tiles b, b + grid, ...
constexpr int kItThreads = 192;
constexpr int kItRaster = 8;  // token tiles walked together (their X and the W tiles of a wave stay in L2)
__host__ __device__ constexpr int it_stage_bytes(int bn) { return (kItM + bn) * kItK; }
__host__ __device__ constexpr int it_stages(int bn) {
  return (216 * 1024) / it_stage_bytes(bn) < 10 ? (216 * 1024) / it_stage_bytes(bn) : 10;
}
__host__ __device__ constexpr size_t it_smem_bytes(int bn) {
  return 1024 + size_t(it_stages(bn)) * it_stage_bytes(bn) + 2 * 256 * sizeof(float) + 256;
}
static_assert(it_smem_bytes(256) <= 227 * 1024 && it_smem_bytes(128) <= 227 * 1024 && it_smem_bytes(16) <= 227 * 1024,
              "int8 product shared memory");

// kind::i8, A and B signed, int32 sums.
__host__ __device__ constexpr uint32_t umma_idesc_s8(int m, int n) {
  return (2u << 4) | (1u << 7) | (1u << 10) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}
__device__ __forceinline__ void umma_i8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}

// N accumulator columns (tokens t0 ..) of this lane's channel.
template <typename T, int N>
__device__ __forceinline__ void it_store_h(const I8Params& P, const uint32_t (&v)[N], const float* sx, int t0, int n,
                                           float sw, float bias, bool has_bias) {
  const int lane = threadIdx.x & 31;
  T* Y = static_cast<T*>(P.Y);
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    const uint32_t a = Elem<T>::bits(i8_value(int(v[c]), sx[c], sw, bias, has_bias));
    const uint32_t b = Elem<T>::bits(i8_value(int(v[c + 1]), sx[c + 1], sw, bias, has_bias));
    if (P.pair) {
      // lanes 2i and 2i + 1 swap a value each: the even lane then holds token c of channels n,
      // n + 1, the odd lane token c + 1 of channels n - 1, n
      const bool odd = lane & 1;
      const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
      const int t = t0 + c + (odd ? 1 : 0), m = n - (odd ? 1 : 0);
      const uint32_t two = odd ? (got | (b << 16)) : (a | (got << 16));
      if (t < P.tokens) {
        T* y = Y + (long long)t * P.ldy + m;
        if (m + 1 < P.n) *reinterpret_cast<uint32_t*>(y) = two;
        else if (m < P.n) *reinterpret_cast<uint16_t*>(y) = uint16_t(two);
      }
    } else if (n < P.n) {
      if (t0 + c < P.tokens) reinterpret_cast<uint16_t*>(Y)[(long long)(t0 + c) * P.ldy + n] = uint16_t(a);
      if (t0 + c + 1 < P.tokens) reinterpret_cast<uint16_t*>(Y)[(long long)(t0 + c + 1) * P.ldy + n] = uint16_t(b);
    }
  }
}

template <int N>
__device__ __forceinline__ void it_store(const I8Params& P, const uint32_t (&v)[N], const float* sx, int t0, int n, float sw,
                                         float bias, bool has_bias) {
  if (P.out == BQG_F32) {
    if (n < P.n) {
      float* y = static_cast<float*>(P.Y) + (long long)t0 * P.ldy + n;
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (t0 + j < P.tokens) y[j * P.ldy] = i8_value(int(v[j]), sx[j], sw, bias, has_bias);
    }
  } else if (P.out == BQG_F16) {
    it_store_h<__half, N>(P, v, sx, t0, n, sw, bias, has_bias);
  } else {
    it_store_h<__nv_bfloat16, N>(P, v, sx, t0, n, sw, bias, has_bias);
  }
}

// The tile's columns of one warp's 32 channels: scale, convert, store.
__device__ __forceinline__ void it_store_tile(const I8Params& P, uint32_t lane_base, int columns, const float* sx, int t0,
                                              int n, float sw, float bias, bool has_bias) {
  const int ncol = min(columns, P.tokens - t0);
#pragma unroll 1
  for (int c = 0; c < ncol; c += 16) {
    uint32_t v[16];
    tmem_ld16(lane_base + uint32_t(c), v);
    it_store<16>(P, v, sx + c, t0 + c, n, sw, bias, has_bias);
  }
}

// The storing warps' barrier (THREADS of them), which tells each whether all have what they waited for: a warp
// whose wait gave up comes here once more, and all of them leave together.
template <int THREADS>
__device__ __forceinline__ bool it_all_go_on(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(uint32_t(ok)), "n"(THREADS)
      : "memory");
  return all != 0;
}

// SPLIT: where the tiles would leave SMs idle, a cluster of CTAs takes one tile, each a part of k; they
// exchange their int32 sums through shared memory, each adding and storing its share of the tokens.
// 24 x 4096 x 4096: 11.0 us on 32 SMs, 7.4 us on 128; 30 x 8192 x 1000: 19.4 and 7.6 us.
template <int BN, bool SPLIT>
__global__ void __launch_bounds__(kItThreads, 1)
    k_i8_gemm(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
              const __grid_constant__ I8Params P) {
  constexpr int kStages = it_stages(BN);
  constexpr int kABytes = kItM * kItK, kBBytes = BN * kItK;
  constexpr int kCols = 2 * BN < 32 ? 32 : 2 * BN;  // tensor-memory columns: two accumulators
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* a_ring = smem;
  uint8_t* b_ring = a_ring + size_t(kStages) * kABytes;
  float* sx_s = reinterpret_cast<float*>(b_ring + size_t(kStages) * kBBytes);  // [2][256]
  uint64_t* full = reinterpret_cast<uint64_t*>(sx_s + 2 * 256);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;  // [2]
  uint64_t* acc_empty = acc_full + 2;    // [2]
  uint64_t* done = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  static_assert((2 * kStages + 5) * 8 + 4 <= 256, "barrier area");
  constexpr int kSumPitch = BN + 4;  // words of a channel's sums; 16-byte accesses of a warp in different banks
  static_assert(!SPLIT || 128 * kSumPitch * 4 <= kStages * (kABytes + kBBytes), "sums of a split tile");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 128);
    }
    mbar_init(done, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_launch_dependents();
  griddep_wait();

  const int ntn = (P.n + kItM - 1) / kItM, ntt = (P.tokens + BN - 1) / BN;
  const long long tiles = (long long)ntn * ntt;
  const int nk = (P.k + kItK - 1) / kItK;
  const int split = SPLIT ? P.split : 1, rank = SPLIT ? int(cluster_ctarank()) : 0;
  const int k0 = nk * rank / split, k1 = nk * (rank + 1) / split;
  const long long tile0 = SPLIT ? blockIdx.x / split : blockIdx.x, tile_step = SPLIT ? tiles : gridDim.x;
  // tile i: groups of kItRaster token tiles, token tile fastest inside a group
  auto place = [&](long long i, int& tn, int& tt) {
    const long long per = (long long)kItRaster * ntn;
    const int g = int(i / per);
    const int w = min(kItRaster, ntt - g * kItRaster);
    const int r = int(i - g * per);
    tn = r / w;
    tt = g * kItRaster + r - tn * w;
  };

  if (warp == 0) {
    if (lane == 0) {
      long long s = 0;  // stages issued
      bool ok = true;
      for (long long i = tile0; i < tiles && ok; i += tile_step) {
        int tn, tt;
        place(i, tn, tt);
        for (int kk = k0; kk < k1; ++kk, ++s) {
          const int st = int(s % kStages);
          if (s >= kStages && !mbar_wait(&empty[st], uint32_t(s / kStages - 1) & 1u)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[st], uint32_t(kABytes + kBBytes));
          tma_load_2d(a_ring + size_t(st) * kABytes, &tmap_w, kk * kItK, tn * kItM, &full[st]);
          tma_load_2d(b_ring + size_t(st) * kBBytes, &tmap_x, kk * kItK, tt * BN, &full[st]);
        }
      }
      // bounded wait for the last copies, so that none lands after the CTA has gone, whoever gave up
      for (long long q = (s > kStages ? s - kStages : 0); q < s; ++q)
        mbar_wait(&full[q % kStages], uint32_t(q / kStages) & 1u);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = umma_idesc_s8(kItM, BN);
      long long s = 0;
      int it = 0;
      bool ok = true;
      for (long long i = tile0; i < tiles && ok; i += tile_step, ++it) {
        const int buf = it & 1;
        if (it >= 2 && !mbar_wait(&acc_empty[buf], uint32_t(it / 2 - 1) & 1u)) break;
        tc_fence_after();
        const uint32_t acc = tmem + uint32_t(buf * BN);
        for (int kk = k0; kk < k1; ++kk, ++s) {
          const int st = int(s % kStages);
          if (!mbar_wait(&full[st], uint32_t(s / kStages) & 1u)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = smem_u32(a_ring + size_t(st) * kABytes), b = smem_u32(b_ring + size_t(st) * kBBytes);
#pragma unroll
          for (int j = 0; j < kItK / 32; ++j)
            umma_i8(acc, umma_desc_sw128(a + 32 * j), umma_desc_sw128(b + 32 * j), idesc, (kk > k0 || j > 0) ? 1u : 0u);
          umma_commit(&empty[st]);
        }
        if (ok) umma_commit(&acc_full[buf]);
      }
      umma_commit(done);  // every MMA issued here has completed before tensor memory is freed
      mbar_wait(done, 0);
    }
  } else {
    const int quarter = warp & 3;
    const int et = int(threadIdx.x) - 64;  // 0..127
    const bool has_bias = P.bias != nullptr;
    int it = 0;
    bool ok = true;
    for (long long i = tile0; i < tiles; i += tile_step, ++it) {
      const int buf = it & 1;
      int tn, tt;
      place(i, tn, tt);
      const int n = tn * kItM + quarter * 32 + lane, t0 = tt * BN;
      float* sx = sx_s + buf * 256;
      for (int c = et; c < BN; c += 128) sx[c] = t0 + c < P.tokens ? __ldg(P.sx + t0 + c) : 0.f;
      const float sw = n < P.n ? __ldg(P.sw + n) : 0.f;
      const float bias = has_bias && n < P.n ? __ldg(P.bias + n) : 0.f;
      if (!it_all_go_on<128>(ok)) break;
      ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[buf], uint32_t(it / 2) & 1u));
      if (!ok) continue;
      tc_fence_after();
      const uint32_t lane_base = tmem + uint32_t(buf * BN) + (uint32_t(quarter * 32) << 16);
      if constexpr (SPLIT) {  // every MMA has read its stages: their memory takes the sums
        const uint32_t at = smem_u32(a_ring) + 4 * (quarter * 32 + lane) * kSumPitch;
#pragma unroll 1
        for (int c = 0; c < BN; c += 16) {
          uint32_t v[16];
          tmem_ld16(lane_base + uint32_t(c), v);
#pragma unroll
          for (int j = 0; j < 16; j += 4) sts128(at + 4 * (c + j), v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
      } else {
        it_store_tile(P, lane_base, BN, sx, t0, n, sw, bias, has_bias);
      }
      tc_fence_before();
      mbar_arrive(&acc_empty[buf]);
    }
  }
  if constexpr (SPLIT) {
    __syncwarp();
    cluster_sync();
    if (warp >= 2) {
      int tn, tt;
      place(tile0, tn, tt);
      const int quarter = warp & 3, n = tn * kItM + quarter * 32 + lane, t0 = tt * BN;
      const bool has_bias = P.bias != nullptr;
      const float sw = n < P.n ? __ldg(P.sw + n) : 0.f, bias = has_bias && n < P.n ? __ldg(P.bias + n) : 0.f;
      const int share = BN / split;  // at least 4 columns
      const uint32_t at = smem_u32(a_ring) + 4 * (quarter * 32 + lane) * kSumPitch;
#pragma unroll 2
      for (int c = share * rank; c < share * (rank + 1); c += 4) {
        uint32_t v[4] = {0u, 0u, 0u, 0u};
#pragma unroll 4
        for (int r = 0; r < split; ++r) {
          const float4 p = ld_dsmem_f32x4(at + 4 * c, uint32_t(r));
          v[0] += __float_as_uint(p.x);
          v[1] += __float_as_uint(p.y);
          v[2] += __float_as_uint(p.z);
          v[3] += __float_as_uint(p.w);
        }
        it_store<4>(P, v, sx_s + c, t0 + c, n, sw, bias, has_bias);
      }
    }
    __syncwarp();
    cluster_sync();  // a CTA's sums stay until all have read them
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols));
  }
}

// ---------------------------------------------------------------- large products: tiles of a CTA pair
// One tile is 256 output channels x 256 tokens, computed by the two CTAs of a cluster (cta_group::2):
// each holds 128 channels of W and 128 tokens of X in its shared memory and the sums of its channels in
// its tensor memory; the first CTA issues M 256, N 256 MMAs that read both.  A CTA then loads 32 KB per
// 128 k for the same MMAs that take 48 KB as a 128 x 256 tile of its own, whose 94 bytes a clock are
// more than an SM gets from L2.  The warps' parts are k_i8_gemm's, but eight warps store.
// 8192 tokens, k 4096, n 14336, bf16 out: 457 us as 128 x 256 tiles (2.1 POP/s), 435 us with four storing
// warps (a tile's 256 columns took longer than its 32 stages), 322 us (3.0 POP/s; tensor pipe 87 % active).
constexpr int kI2Half = 128;
constexpr int kI2Threads = 320;  // 8 warps store: a quarter of the channels and half of the tokens each
constexpr int kI2StageBytes = 2 * kI2Half * kItK;
constexpr int kI2Stages = 6;
constexpr size_t kI2SmemBytes = 1024 + size_t(kI2Stages) * kI2StageBytes + 2 * 256 * sizeof(float) + 256;
static_assert(kI2SmemBytes <= 227 * 1024, "int8 pair product shared memory");

__device__ __forceinline__ void umma_i8_pair(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}
// Arrives on `bar` of both CTAs once the MMAs issued so far have completed.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_u32(bar)),
      "h"(uint16_t(3))
      : "memory");
}
// The first CTA's copy of a barrier.
__device__ __forceinline__ uint32_t first_cta(uint64_t* bar) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(bar)));
  return a;
}
// A load into this CTA's shared memory whose bytes count on a barrier of the pair.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kI2Threads, 1)
    k_i8_gemm_pair(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                   const __grid_constant__ I8Params P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* a_ring = smem;
  uint8_t* b_ring = a_ring + kI2Stages * kI2Half * kItK;
  float* sx_s = reinterpret_cast<float*>(b_ring + kI2Stages * kI2Half * kItK);  // [2][256]
  uint64_t* full = reinterpret_cast<uint64_t*>(sx_s + 2 * 256);  // the first CTA's counts both CTAs' bytes
  uint64_t* empty = full + kI2Stages;
  uint64_t* acc_full = empty + kI2Stages;  // [2]
  uint64_t* acc_empty = acc_full + 2;      // [2], the first CTA's: both CTAs' storing warps
  uint64_t* done = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  static_assert((2 * kI2Stages + 5) * 8 + 4 <= 256, "barrier area");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = int(cluster_ctarank());
  if (threadIdx.x == 0) {
    for (int i = 0; i < kI2Stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 16);
    }
    mbar_init(done, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_launch_dependents();
  griddep_wait();

  const int ntn = (P.n + kI2M - 1) / kI2M, ntt = (P.tokens + kI2N - 1) / kI2N;
  const long long tiles = (long long)ntn * ntt, pairs = gridDim.x / 2;
  const int nk = (P.k + kItK - 1) / kItK;
  auto place = [&](long long i, int& tn, int& tt) {  // as in k_i8_gemm
    const long long per = (long long)kItRaster * ntn;
    const int g = int(i / per);
    const int w = min(kItRaster, ntt - g * kItRaster);
    const int r = int(i - g * per);
    tn = r / w;
    tt = g * kItRaster + r - tn * w;
  };

  if (warp == 0) {
    if (lane == 0) {
      long long s = 0;  // stages issued
      bool ok = true;
      for (long long i = blockIdx.x / 2; i < tiles && ok; i += pairs) {
        int tn, tt;
        place(i, tn, tt);
        for (int kk = 0; kk < nk; ++kk, ++s) {
          const int st = int(s % kI2Stages);
          if (s >= kI2Stages && !mbar_wait(&empty[st], uint32_t(s / kI2Stages - 1) & 1u)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&full[st], uint32_t(2 * kI2StageBytes));
          const uint32_t bar = first_cta(&full[st]);
          tma_load_2d_pair(a_ring + st * kI2Half * kItK, &tmap_w, kk * kItK, tn * kI2M + rank * kI2Half, bar);
          tma_load_2d_pair(b_ring + st * kI2Half * kItK, &tmap_x, kk * kItK, tt * kI2N + rank * kI2Half, bar);
        }
      }
      if (rank == 0)  // bounded wait for the last copies, so that none lands after the pair has gone, whoever gave up
        for (long long q = (s > kI2Stages ? s - kI2Stages : 0); q < s; ++q)
          mbar_wait(&full[q % kI2Stages], uint32_t(q / kI2Stages) & 1u);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      if (rank == 0) {
        const uint32_t idesc = umma_idesc_s8(kI2M, kI2N);
        long long s = 0;
        int it = 0;
        bool ok = true;
        for (long long i = blockIdx.x / 2; i < tiles && ok; i += pairs, ++it) {
          const int buf = it & 1;
          if (it >= 2 && !mbar_wait(&acc_empty[buf], uint32_t(it / 2 - 1) & 1u)) break;
          tc_fence_after();
          const uint32_t acc = tmem + uint32_t(buf * kI2N);
          for (int kk = 0; kk < nk; ++kk, ++s) {
            const int st = int(s % kI2Stages);
            if (!mbar_wait(&full[st], uint32_t(s / kI2Stages) & 1u)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a = smem_u32(a_ring + st * kI2Half * kItK), b = smem_u32(b_ring + st * kI2Half * kItK);
#pragma unroll
            for (int j = 0; j < kItK / 32; ++j)
              umma_i8_pair(acc, umma_desc_sw128(a + 32 * j), umma_desc_sw128(b + 32 * j), idesc, (kk > 0 || j > 0) ? 1u : 0u);
            umma_commit_pair(&empty[st]);
          }
          if (ok) umma_commit_pair(&acc_full[buf]);
        }
        umma_commit_pair(done);
      }
    }
  } else {
    const int quarter = warp & 3, col = (warp - 2) / 4 * kI2Half;
    const int et = int(threadIdx.x) - 64;  // 0..255
    const bool has_bias = P.bias != nullptr;
    int it = 0;
    bool ok = true;
    for (long long i = blockIdx.x / 2; i < tiles; i += pairs, ++it) {
      const int buf = it & 1;
      int tn, tt;
      place(i, tn, tt);
      const int n = tn * kI2M + rank * kI2Half + quarter * 32 + lane, t0 = tt * kI2N;
      float* sx = sx_s + buf * 256;
      sx[et] = t0 + et < P.tokens ? __ldg(P.sx + t0 + et) : 0.f;
      const float sw = n < P.n ? __ldg(P.sw + n) : 0.f;
      const float bias = has_bias && n < P.n ? __ldg(P.bias + n) : 0.f;
      if (!it_all_go_on<256>(ok)) break;
      ok = __all_sync(0xffffffffu, mbar_wait(&acc_full[buf], uint32_t(it / 2) & 1u));
      if (!ok) continue;
      tc_fence_after();
      it_store_tile(P, tmem + uint32_t(buf * kI2N + col) + (uint32_t(quarter * 32) << 16), kI2Half, sx + col, t0 + col, n, sw,
                    bias, has_bias);
      tc_fence_before();
      __syncwarp();
      if (lane == 0)
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(first_cta(&acc_empty[buf])) : "memory");
    }
  }
  // Every MMA has completed before tensor memory is freed and the barriers that its commits arrive on go.
  // Waited for behind the storing warps, which the last tile's MMAs let go: the second CTA, which issues
  // none, would otherwise wait from the start on, and a product of more than two seconds would look stuck.
  __syncthreads();
  if (threadIdx.x == 32) mbar_wait(done, 0);
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // neither CTA's memory is freed while the other still uses it
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

// ---------------------------------------------------------------- host side
// The last tile's rows and columns, past the tensors' ends too, are 32-bit indexes.
static_assert(0x7FFFFFFF - BQG_MAX_I8_ROWS >= kI2M && 0x7FFFFFFF - BQG_MAX_I8_ROWS >= 256, "a tile past the last row");
inline size_t i8_type_bytes(int type) { return type == BQG_F32 ? 4 : (type == BQG_F16 || type == BQG_BF16) ? 2 : 0; }

template <typename T>
inline int launch_quantize_rows(const void* X, size_t ldx, int8_t* Q, size_t ldq, float* scale, int rows, int k,
                                cudaStream_t s) {
  // 8 values a thread by 16-byte loads where every row starts on 16 bytes; one by one otherwise
  const bool vec = aligned(X, 16) && ldx * sizeof(T) % 16 == 0;
  const T* x = static_cast<const T*>(X);
  const long long lx = (long long)ldx, lq = (long long)ldq;
  auto launch = [&](auto kernel, int tpr) {
    const unsigned grid = tpr == 32 ? unsigned((rows + 7) / 8) : unsigned(rows);
    return launch_pdl(kernel, dim3(grid), dim3(unsigned(tpr == 32 ? kQrThreads : tpr)), 0, s, x, lx, Q, lq, scale, rows, k);
  };
  // the smallest that keeps a row in registers; for one row and a few, as many threads as there are
  constexpr int kHeld = 8 * kQrChunks;
  if (k <= 32 * kHeld && rows > 1)
    return vec ? launch(k_quantize_rows<T, 32, true>, 32) : launch(k_quantize_rows<T, 32, false>, 32);
  if (k <= 64 * kHeld && rows > kQrFewRows)
    return vec ? launch(k_quantize_rows<T, 64, true>, 64) : launch(k_quantize_rows<T, 64, false>, 64);
  if (k <= 128 * kHeld && rows > kQrFewRows)
    return vec ? launch(k_quantize_rows<T, 128, true>, 128) : launch(k_quantize_rows<T, 128, false>, 128);
  return vec ? launch(k_quantize_rows<T, 256, true>, 256) : launch(k_quantize_rows<T, 256, false>, 256);
}

inline bool i8_encode(CUtensorMap* m, const int8_t* p, size_t pitch, int rows, int k, int box_rows) {
  EncodeTiledFn encode = encode_tiled_fn();
  if (encode == nullptr) return false;
  const cuuint64_t dims[2] = {cuuint64_t(k), cuuint64_t(rows)};
  const cuuint64_t strides[1] = {cuuint64_t(pitch)};
  const cuuint32_t box[2] = {cuuint32_t(kItK), cuuint32_t(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(p), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline SmemAttrOnce g_i8_attr[10];  // tiles of 16 to 256 tokens, of pairs, and of 16 to 128 in parts of k

template <int BN>
inline int launch_i8_gemm(const I8Params& P, int dev, const DeviceInfo* info, cudaStream_t s) {
  CUtensorMap tw, tx;
  if (!i8_encode(&tw, P.W, size_t(P.ldw), P.n, P.k, kItM) || !i8_encode(&tx, P.X, size_t(P.ldx), P.tokens, P.k, BN))
    return BQG_ERR_CUDA;
  constexpr int slot = BN == 16 ? 0 : BN == 32 ? 1 : BN == 64 ? 2 : BN == 128 ? 3 : 4;
  const long long tiles = (long long)((P.n + kItM - 1) / kItM) * ((P.tokens + BN - 1) / BN);
  if constexpr (BN <= 128) {
    if (P.split > 1) {
      const int st = g_i8_attr[6 + slot].ensure(dev, k_i8_gemm<BN, true>, it_smem_bytes(BN));
      if (st != BQG_OK) return st;
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3(unsigned(tiles * P.split));
      cfg.blockDim = dim3(kItThreads);
      cfg.dynamicSmemBytes = it_smem_bytes(BN);
      cfg.stream = s;
      cudaLaunchAttribute attr[2];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = unsigned(P.split);
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[1].val.programmaticStreamSerializationAllowed = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 2;
      if (cudaLaunchKernelEx(&cfg, k_i8_gemm<BN, true>, tw, tx, P) != cudaSuccess) {
        (void)cudaGetLastError();
        return BQG_ERR_CUDA;
      }
      return launch_status();
    }
  }
  const int st = g_i8_attr[slot].ensure(dev, k_i8_gemm<BN, false>, it_smem_bytes(BN));
  if (st != BQG_OK) return st;
  const int grid = int(tiles < info->sm_count ? tiles : info->sm_count);
  return launch_pdl(k_i8_gemm<BN, false>, dim3(unsigned(grid)), dim3(kItThreads), it_smem_bytes(BN), s, tw, tx, P);
}

inline int launch_i8_gemm_pair(const I8Params& P, int dev, const DeviceInfo* info, cudaStream_t s) {
  CUtensorMap tw, tx;
  if (!i8_encode(&tw, P.W, size_t(P.ldw), P.n, P.k, kI2Half) || !i8_encode(&tx, P.X, size_t(P.ldx), P.tokens, P.k, kI2Half))
    return BQG_ERR_CUDA;
  const int st = g_i8_attr[5].ensure(dev, k_i8_gemm_pair, kI2SmemBytes);
  if (st != BQG_OK) return st;
  const long long tiles = (long long)((P.n + kI2M - 1) / kI2M) * ((P.tokens + kI2N - 1) / kI2N);
  const int pairs = int(tiles < info->sm_count / 2 ? tiles : info->sm_count / 2);
  return launch_pdl(k_i8_gemm_pair, dim3(unsigned(2 * pairs)), dim3(kI2Threads), kI2SmemBytes, s, tw, tx, P);
}

// Clusters of 2 and of 4 CTAs that run at once on the device (a CTA of k_i8_gemm takes a whole SM, and a
// cluster's CTAs one cluster of SMs: 74 of 2, 33 of 4 on a B200).  Asked once per device.
inline I8Clusters i8_clusters(int dev) {
  static std::atomic<int> known[kMaxDevices][2] = {};  // count + 1
  int n[2] = {0, 0};
  for (int i = 0; i < 2; ++i) {
    n[i] = known[dev][i].load(std::memory_order_relaxed) - 1;
    if (n[i] >= 0) continue;
    n[i] = 0;
    if (g_i8_attr[6].ensure(dev, k_i8_gemm<16, true>, it_smem_bytes(16)) != BQG_OK) continue;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2u << i);
    cfg.blockDim = dim3(kItThreads);
    cfg.dynamicSmemBytes = it_smem_bytes(16);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2u << i;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int count = 0;
    if (cudaOccupancyMaxActiveClusters(&count, k_i8_gemm<16, true>, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();
      continue;  // no parts of k in this call; the next one asks again
    }
    n[i] = count;
    known[dev][i].store(count + 1, std::memory_order_relaxed);
  }
  return I8Clusters{n[0], n[1]};
}
static_assert(it_smem_bytes(16) > 114 * 1024 && it_smem_bytes(32) > 114 * 1024 && it_smem_bytes(64) > 114 * 1024 &&
                  it_smem_bytes(128) > 114 * 1024,
              "one CTA an SM, whatever the tile");

}  // namespace bqg

extern "C" int quantize_rows_i8(int type, const void* X, size_t ldx, int8_t* Xq, size_t ldq, float* scale, int rows,
                                int k, void* stream) {
  using namespace bqg;
  if (X == nullptr || Xq == nullptr || scale == nullptr || rows < 1 || k < 1) return BQG_ERR_ARG;
  const size_t size = i8_type_bytes(type);
  if (size == 0) return BQG_ERR_ARG;
  if (k > BQG_MAX_I8_COLS || rows > BQG_MAX_I8_ROWS) return BQG_ERR_LIMIT;
  if (ldx < size_t(k) || ldq < size_t(k) || ldq % 16 != 0) return BQG_ERR_SHAPE;
  if (!aligned(X, size) || !aligned(Xq, 16) || !aligned(scale, 4)) return BQG_ERR_ALIGN;
  int dev;
  DeviceInfo* info;
  const int st = current_device(&dev, &info);
  if (st != BQG_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (type == BQG_F32) return launch_quantize_rows<float>(X, ldx, Xq, ldq, scale, rows, k, s);
  if (type == BQG_F16) return launch_quantize_rows<__half>(X, ldx, Xq, ldq, scale, rows, k, s);
  return launch_quantize_rows<__nv_bfloat16>(X, ldx, Xq, ldq, scale, rows, k, s);
}

extern "C" int qgemm_i8(const int8_t* Xq, size_t ldx, const float* sx, const int8_t* Wq, size_t ldw, const float* sw,
                        const float* bias, int out_type, void* Y, size_t ldy, int tokens, int n, int k, void* stream) {
  using namespace bqg;
  if (Xq == nullptr || sx == nullptr || Wq == nullptr || sw == nullptr || Y == nullptr || tokens < 1 || n < 1 || k < 1)
    return BQG_ERR_ARG;
  const size_t size = i8_type_bytes(out_type);
  if (size == 0) return BQG_ERR_ARG;
  if (k > BQG_MAX_I8_COLS || tokens > BQG_MAX_I8_ROWS || n > BQG_MAX_I8_ROWS) return BQG_ERR_LIMIT;
  if (ldx < size_t(k) || ldw < size_t(k) || ldy < size_t(n) || ldx % 16 != 0 || ldw % 16 != 0) return BQG_ERR_SHAPE;
  if (!aligned(Xq, 16) || !aligned(Wq, 16) || !aligned(sx, 4) || !aligned(sw, 4) || !aligned(bias, 4) ||
      !aligned(Y, size))
    return BQG_ERR_ALIGN;
  int dev;
  DeviceInfo* info;
  const int st = current_device(&dev, &info);
  if (st != BQG_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  I8Params P{};
  P.X = Xq;
  P.W = Wq;
  P.sx = sx;
  P.sw = sw;
  P.bias = bias;
  P.Y = Y;
  P.ldx = (long long)ldx;
  P.ldw = (long long)ldw;
  P.ldy = (long long)ldy;
  P.tokens = tokens;
  P.n = n;
  P.k = k;
  P.out = out_type;
  P.pair = size == 2 && ldy % 2 == 0 && aligned(Y, 4);
  if (i8_few(tokens, n, k, info->sm_count)) {
    const int groups = (n + kIgRows - 1) / kIgRows;
    const int want = (groups + kIgThreads / 32 - 1) / (kIgThreads / 32);
    const int most = info->sm_count * 6;
    const dim3 grid(unsigned(want < most ? want : most));
    if (tokens == 1) return launch_pdl(k_i8_gemv<1>, grid, dim3(kIgThreads), 0, s, P);
    if (tokens == 2) return launch_pdl(k_i8_gemv<2>, grid, dim3(kIgThreads), 0, s, P);
    return launch_pdl(k_i8_gemv<4>, grid, dim3(kIgThreads), 0, s, P);
  }
  const I8Cut cut = i8_cut(tokens, n, k, info->sm_count, i8_clusters(dev));
  P.split = cut.split;
  switch (cut.tokens) {
    case 16: return launch_i8_gemm<16>(P, dev, info, s);
    case 32: return launch_i8_gemm<32>(P, dev, info, s);
    case 64: return launch_i8_gemm<64>(P, dev, info, s);
    case 128: return launch_i8_gemm<128>(P, dev, info, s);
    case 256: return launch_i8_gemm<256>(P, dev, info, s);
    default: return launch_i8_gemm_pair(P, dev, info, s);
  }
}
